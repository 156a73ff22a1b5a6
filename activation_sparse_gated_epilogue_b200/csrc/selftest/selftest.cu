// Self-test of the failure handling of the tcgen05 GEMM engines (a
// test-only library, libsge_selftest.so, not part of libsge.so).
//
// Every wait of the engines is bounded: a wait that runs out sets
// SGE_FLAG_TIMEOUT in the caller's diag word, raises the CTA's abort flag,
// and the CTA drains its in-flight loads and MMAs (again with bounded waits),
// frees its tensor memory and returns, leaving the context usable.  This
// library builds the engines with a 20 ms deadline and runs them on a tile
// pipeline whose stage barriers can never complete: the B operand's tensor
// map has a box half as tall as the stage the producer arms for, so every
// stage receives fewer bytes than it expects.  The copies themselves are in
// bounds; only the barriers' transaction counts stay above zero.  The MMA
// issuer's first wait then runs out, and the abort and drain paths run.
#define SGE_WAIT_NS 20000000ull

#include "../../../include/sge_selftest.h"
#include "../i8_gemm.cuh"
#include "../tc_launch.cuh"

namespace sge {

// Counts the output tiles whose accumulators reached the epilogue (none may).
struct EpiCountTiles {
  int* tiles_done;
  template <int BN>
  __device__ __forceinline__ void run(uint32_t, int64_t, int, int lane) const {
    if (lane == 0) atomicAdd(tiles_done, 1);
  }
};

// The same for the 8-bit engine's epilogue interfaces: whole sums, and block by
// block with a scale for each row and 128 of k.
struct EpiCountI8 {
  int* tiles_done;
  const float* scales;  // [k / 128][rows]
  int64_t rows;
  template <int COLS>
  __device__ __forceinline__ void run(const I8Out& o, int) const {
    if (o.lane == 0) atomicAdd(tiles_done, 1);
  }
  __device__ __forceinline__ const float* block_scales(const I8Out& o) const {
    return scales + (o.row < rows ? o.row : rows - 1);
  }
  __device__ __forceinline__ int64_t scale_pitch() const { return rows; }
  template <int COLS>
  __device__ __forceinline__ void store(const I8Out& o, const float (&sum)[COLS], int) const {
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < COLS; ++j) s += sum[j];
    if (o.lane == 0) atomicAdd(tiles_done, s == 0.0f ? 1 : 2);
  }
};

// `b` read through a map whose box has half the rows that a stage expects.
template <class Shape>
static int i8_wait_timeout(const void* a, const void* b, int64_t m, int64_t n, int64_t k, const EpiCountI8& epi,
                           int32_t* diag, cudaStream_t st) {
  const I8Problem p{static_cast<int>(m), static_cast<int>(n), static_cast<int>(k), 1, 1, nullptr};
  I8Maps maps;
  const int8_t* b0 = static_cast<const int8_t*>(b);
  int rc = make_i8_maps<Shape>(&maps, p, static_cast<const int8_t*>(a), k, b0, Shape::NB == 2 ? b0 : nullptr, k);
  if (!rc) rc = make_tmap_i8(&maps.b0, b, n, k, k, Shape::B_ROWS / 2);
  if (rc) return rc;
  return launch_i8_gemm<Shape>(maps, p, epi, diag, st, "selftest (8-bit engine)");
}

}  // namespace sge

using namespace sge;

extern "C" int sge_selftest_wait_timeout(int pair, const void* a, const void* b, int64_t m, int64_t n,
                                         int64_t k, int32_t* diag, int32_t* tiles_done, void* stream) {
  clear_error();
  if (!a || !b || !diag || !tiles_done || m < 1 || n < 1 || k < 64 || m > (1 << 20) || n > (1 << 20) ||
      k > (1 << 20) || !aligned16(a) || !aligned16(b))
    return fail(SGE_ERR_ARG, "sge_selftest_wait_timeout: bad arguments");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  EpiCountTiles epi{tiles_done};
  if (pair >= 2) {  // the 8-bit engine
    if (pair > 7 || k % 16) return fail(SGE_ERR_ARG, "sge_selftest_wait_timeout: bad arguments");
    // a's bytes as block scales (copied, not used): [k / 128][m] floats fit in its m x k
    const EpiCountI8 e8{tiles_done, static_cast<const float*>(a), m};
    switch (pair) {
      case 2: return i8_wait_timeout<I8Shape<128, 1, 2, 1, false, false, false, 0>>(a, b, m, n, k, e8, diag, st);
      case 3: return i8_wait_timeout<I8Shape<256, 1, 2, 2, true, false, false, 0>>(a, b, m, n, k, e8, diag, st);
      case 4: return i8_wait_timeout<GateUpOne>(a, b, m, n, k, e8, diag, st);
      case 5: return i8_wait_timeout<GateUpPair>(a, b, m, n, k, e8, diag, st);
      case 6: return i8_wait_timeout<DownOne>(a, b, m, n, k, e8, diag, st);
      default: return i8_wait_timeout<DownPair>(a, b, m, n, k, e8, diag, st);
    }
  }
  CUtensorMap ma, mb;
  if (pair) {
    using S = TcPairShape<256, 1>;
    int rc = make_tmap_bf16(&ma, a, m, k, k, kBM);
    // half the rows the stage expects: its barrier is never satisfied
    if (!rc) rc = make_tmap_bf16(&mb, b, n, k, k, S::BN / 4);
    if (rc) return rc;
    return launch_tc_gemm_pair<S>(ma, mb, mb, m, n, k, epi, diag, st, "selftest (pair engine)");
  }
  using S = TcShape<128, 1>;
  int rc = make_tmap_bf16(&ma, a, m, k, k, a_box_rows(m));
  if (!rc) rc = make_tmap_bf16(&mb, b, n, k, k, S::BN / 2);
  if (rc) return rc;
  return launch_tc_gemm<S>(ma, mb, mb, m, n, k, epi, diag, st, "selftest (single-CTA engine)");
}
