// Products of 8-bit integers with a scale for each token and channel.
//
//   int8_quant_rows        activation rows -> int8 rows and their scales
//   int8_linear            y[n][m] = (sum_k xq[n][k] wq[m][k]) * sx[n] * sw[m]
//   twell_gate_pack_int8   the same product as the gate projection, ReLU and
//                          the TwELL pack in its epilogue
//
// The sums are exact 32-bit integers (i8_gemm.cuh); y is their conversion to
// fp32 times the two scales, in this order, rounded once more to a bf16 y.
#include "i8_gemm.cuh"
#include "i8_quant.cuh"
#include "i8_small.cuh"

namespace sge {

// ------------------------------------------------------------ quantisation

// One warp per row: the row stays in registers between its maximum and its
// rounding, so it is read once.  Bound by HBM: 16384 x 2560 bf16 (84 MB in, 42 MB
// out) takes 25 us, 5.0 TB/s.
template <class T, bool VEC>
__global__ void __launch_bounds__(256) i8_quant_kernel(const T* __restrict__ x, int64_t ldx, int64_t rows,
                                                       int cols, int8_t* __restrict__ q, int64_t ldq,
                                                       float* __restrict__ scale) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  int8_t* dst = q + row * ldq;
  uint32_t amax;
  quant_row<T, VEC, 8>(x + row * ldx, cols, lane, amax,
                       [&](int c, const auto& f, float inv) { store_q(dst + c, f, inv); });
  // the bytes past the row: zeros, so that 16-byte reads of rows see nothing else
  for (int c = ((cols + 3) & ~3) + 4 * lane; c < ldq; c += 128) *reinterpret_cast<uint32_t*>(dst + c) = 0;
  if (lane == 0) scale[row] = quant_scale(amax).scale;
}

template <class T>
static int quant_rows(const void* x, int64_t ldx, int64_t rows, int64_t cols, int8_t* q, int64_t ldq,
                      float* scale, cudaStream_t st) {
  constexpr int V = Vec16<T>::N;
  const dim3 grid(static_cast<unsigned>((rows + 7) / 8));
  auto kern = cols % V == 0 && ldx % V == 0 ? i8_quant_kernel<T, true> : i8_quant_kernel<T, false>;
  return launch_pdl(kern, grid, dim3(256), 0, st, "int8_quant_rows", static_cast<const T*>(x), ldx, rows,
                    static_cast<int>(cols), q, ldq, scale);
}

// --------------------------------------------------------------- epilogues

// 32 accumulator columns as scaled floats: acc * sx * sw[col].
SGE_DEV void i8_scaled32(uint32_t taddr, float sx, const float* __restrict__ sw, int col0, int n,
                         float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  tmem_ld_wait();
  if (col0 + 32 <= n) {
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const float4 s = __ldg(reinterpret_cast<const float4*>(sw + col0 + j));
      v[j] = __int2float_rn(static_cast<int>(r[j])) * sx * s.x;
      v[j + 1] = __int2float_rn(static_cast<int>(r[j + 1])) * sx * s.y;
      v[j + 2] = __int2float_rn(static_cast<int>(r[j + 2])) * sx * s.z;
      v[j + 3] = __int2float_rn(static_cast<int>(r[j + 3])) * sx * s.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      v[j] = col0 + j < n ? __int2float_rn(static_cast<int>(r[j])) * sx * __ldg(sw + col0 + j) : 0.0f;
  }
}

// y's columns, 128 bytes of a row at a time through staging memory (16384 x 2560
// x 10240 bf16: 276 us at full clocks, 3.1 POPS, against 340 us with each thread
// storing its own row; the tensor pipe is busy 77% of the cycles, and in a
// sustained run the power cap sets the time).
template <class T>
struct EpiI8Linear {
  T* y;
  const float* sx;
  const float* sw;

  template <int COLS>
  __device__ __forceinline__ void run(const I8Out& o, int n) const {
    using Rows = StagedRows<T>;
    static_assert(COLS % Rows::COLS == 0, "whole rows of 128 bytes");
    const float s = o.row_ok ? __ldg(sx + o.row) : 0.0f;
#pragma unroll 1
    for (int c = 0; c < COLS; c += Rows::COLS) {
      if (o.col0 + c >= n) break;
#pragma unroll
      for (int part = 0; part < Rows::COLS; part += 32) {
        float v[32];
        i8_scaled32(o.taddr + c + part, s, sw, o.col0 + c + part, n, v);
        Rows::put(o.stage, o.lane, part, v);
      }
      Rows::flush(o.stage, o.lane, y, o.row - o.lane, o.row_end, o.col0 + c, n);
    }
  }
};

// ReLU and the TwELL pack; each thread owns a row, so a tile's entries come out
// in ascending order (8192 x 2048 x 8192 at 1% density: 87 us, 3.15 POPS, as fast
// as the main loop alone).
template <int T>
struct EpiI8Twell {
  uint8_t* count;
  uint8_t* idx;
  uint16_t* val;  // bf16 bits
  int cap;
  int32_t* diag;
  const float* sx;
  const float* sw;

  // Per 32 columns the bit mask of active ones (g > 0; NaN inactive), whose
  // set bits are visited in ascending order.
  template <int COLS>
  __device__ __forceinline__ void run(const I8Out& o, int n) const {
    static_assert(COLS % T == 0 && (T == 16 || T % 32 == 0), "whole tiles");
    const float s = o.row_ok ? __ldg(sx + o.row) : 0.0f;
    const int64_t nt = n / T;
    int overflow = 0, c = 0;
#pragma unroll 1
    for (int ch = 0; ch < COLS / 32; ++ch) {
      const int col0 = o.col0 + ch * 32;
      if (col0 >= n) break;
      float v[32];
      i8_scaled32(o.taddr + ch * 32, s, sw, col0, n, v);
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) m |= (v[j] > 0.0f ? 1u : 0u) << j;
      constexpr int PARTS = T == 16 ? 2 : 1;
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        const int col = col0 + part * T;
        const bool ok = o.row_ok && col < n;
        const int64_t seg = o.row * nt + col / T;
        const int in_tile = col % T;
        if (in_tile == 0) c = 0;
        uint32_t left = PARTS == 1 ? m : part ? m >> 16 : m & 0xffffu;
        while (left) {
          const int j = __ffs(left) - 1;
          left &= left - 1;
          if (ok && c < cap) {
            idx[seg * cap + c] = static_cast<uint8_t>(in_tile + j);
            val[seg * cap + c] = f32_to_bf16_bits(select32(v, part * 16 + j));
          }
          ++c;
        }
        if (in_tile + 32 >= T && ok) {
          count[seg] = static_cast<uint8_t>(c);
          overflow += c > cap;
        }
      }
    }
    if (overflow && diag) atomicAdd(reinterpret_cast<int*>(diag + SGE_DIAG_OVERFLOW_TILES), overflow);
  }
};

// --------------------------------------------------------------- dispatch

// Whether single-CTA tiles (128 rows, bn columns) leave every SM at most one: the
// product then takes the narrowest such tiles, else pairs of 256 x 256.  us of the
// product alone, weights from HBM, tokens x d -> columns:
//   int8_linear                    64 columns  128 columns  pairs
//   256 x 2560 -> 1024                    9.9         10.7   14.7
//   1024 x 2560 -> 1024                  10.0         10.8   14.4
//   2048 x 2560 -> 1024                  15.3         10.9   14.3
//   4096 x 2560 -> 1024                  26.0         16.9   15.1
//   257 / 512 / 1024 x 2560 -> 2560  10.1 / 15.2 / 20.7  10.9 / 11.3 / 16.6  14.8 / 15.0 / 15.5
//   128 / 256 / 257 x 2048 -> 8192   9.6 / 13.7 / 17.9  10.3 / 10.4 / 14.7  14.6 / 14.7 / 14.4
//   32 / 129 x 2560 -> 10240         15.4 / 20.8  11.4 / 17.0  17.3 / 15.7
//   4096 x 1024 -> 64                     5.7          6.0    7.4
// (at d = 1024 two rounds of 128 columns still beat pairs: 4096 -> 1024 10.2
// against 11.6; the rule does not look at d.)
//   gate, 1% open                             128 columns  pairs
//   2048 / 4096 x 2560 -> 1024                12.0 / 18.1  13.3 / 14.0
//   512 / 1024 x 2560 -> 2560                 12.6 / 17.6  14.1 / 14.6
//   256 / 257 x 2048 -> 8192                  12.1 / 15.9  14.0 / 13.5
//   128 / 129 x 2560 -> 10240                 15.2 / 21.0  17.7 / 17.0
static bool one_tile_each(int64_t n, int64_t m, int bn) {
  return ((n + kBM - 1) / kBM) * ((m + bn - 1) / bn) <= sm_count();
}

template <class Shape, class Epi>
static int i8_product(const int8_t* xq, int64_t ldx, const int8_t* wq, int64_t ldw, int64_t n, int64_t m,
                      int64_t k, const Epi& epi, int32_t* diag, cudaStream_t st, const char* what) {
  const I8Problem p{static_cast<int>(n), static_cast<int>(m), static_cast<int>(k), 1, 1, nullptr};
  I8Maps maps;
  const int rc = make_i8_maps<Shape>(&maps, p, xq, ldx, wq, nullptr, ldw);
  if (rc) return rc;
  return launch_i8_gemm<Shape>(maps, p, epi, diag, st, what);
}

template <class T>
static int linear(const int8_t* xq, int64_t ldx, const float* sx, const int8_t* wq, int64_t ldw,
                  const float* sw, void* y, int64_t n, int64_t m, int64_t k, int32_t* diag, cudaStream_t st) {
  if (n <= kSmallLinear) {
    auto kern = n == 1 ? i8_linear_small_kernel<T, 1> : i8_linear_small_kernel<T, 2>;
    return launch_pdl(kern, dim3(static_cast<unsigned>((m + 7) / 8)), dim3(256), 0, st, "int8_linear (few tokens)",
                      xq, ldx, sx, wq, ldw, sw, static_cast<T*>(y), static_cast<int>(n), static_cast<int>(m),
                      static_cast<int>(k));
  }
  const EpiI8Linear<T> epi{static_cast<T*>(y), sx, sw};
  if (one_tile_each(n, m, 64))
    return i8_product<I8Shape<64, 1, 2, 1, false, false, false, 4096>>(xq, ldx, wq, ldw, n, m, k, epi, diag, st,
                                                                       "int8_linear");
  if (one_tile_each(n, m, 128))
    return i8_product<I8Shape<128, 1, 2, 2, false, false, false, 4096>>(xq, ldx, wq, ldw, n, m, k, epi, diag, st,
                                                                        "int8_linear");
  return i8_product<I8Shape<256, 1, 2, 2, true, false, false, 4096>>(xq, ldx, wq, ldw, n, m, k, epi, diag, st,
                                                                     "int8_linear (CTA pairs)");
}

template <int T>
static int gate(const int8_t* xq, int64_t ldx, const float* sx, const int8_t* wq, int64_t ldw, const float* sw,
                int64_t n, int64_t f, int64_t k, int cap, uint8_t* count, uint8_t* idx, void* val,
                int32_t* diag, cudaStream_t st) {
  const EpiI8Twell<T> epi{count, idx, static_cast<uint16_t*>(val), cap, diag, sx, sw};
  if (one_tile_each(n, f, 128))
    return i8_product<I8Shape<128, 1, 2, 1, false, false, false, 0>>(xq, ldx, wq, ldw, n, f, k, epi, diag, st,
                                                    "twell_gate_pack_int8");
  return i8_product<I8Shape<256, 1, 2, 2, true, false, false, 0>>(xq, ldx, wq, ldw, n, f, k, epi, diag, st,
                                                 "twell_gate_pack_int8 (CTA pairs)");
}

// Checks that int8_linear and twell_gate_pack_int8 share.
static int check_product(const char* fn, const int8_t* xq, int64_t ldx, const float* sx, const int8_t* wq,
                         int64_t ldw, const float* sw, int64_t k, const int32_t* diag) {
  if (!xq || !sx || !wq || !sw) return fail(SGE_ERR_ARG, "%s: null pointer", fn);
  if (!aligned16(xq) || !aligned16(sx) || !aligned16(wq) || !aligned16(sw) || (diag && !aligned16(diag)))
    return fail(SGE_ERR_ARG, "%s: pointer not 16-byte aligned", fn);
  if (ldx < k || ldw < k || ldx % 16 || ldw % 16)
    return fail(SGE_ERR_ARG, "%s: row pitches ldx=%lld, ldw=%lld must be multiples of 16, at least k=%lld", fn,
                (long long)ldx, (long long)ldw, (long long)k);
  return SGE_OK;
}

}  // namespace sge

using namespace sge;

extern "C" int int8_quant_rows(const void* x, int64_t ldx, int64_t n_rows, int64_t n_cols, int dtype, int8_t* q,
                               int64_t ldq, float* scale, void* stream) {
  NvtxRange nvtx_range("int8_quant_rows");
  clear_error();
  if (n_rows < 0 || n_cols < 1)
    return fail(SGE_ERR_ARG, "int8_quant_rows: bad sizes rows=%lld cols=%lld", (long long)n_rows,
                (long long)n_cols);
  if (dtype != SGE_BF16 && dtype != SGE_F32) return fail(SGE_ERR_UNSUPPORTED, "int8_quant_rows: dtype %d", dtype);
  if (n_rows >= (1LL << 31) || n_cols >= (1LL << 30) || ldq >= (1LL << 30))
    return fail(SGE_ERR_UNSUPPORTED, "int8_quant_rows: rows beyond 2^31, or a row beyond 2^30");
  if (ldx < n_cols) return fail(SGE_ERR_ARG, "int8_quant_rows: ldx below the row length");
  if (ldq < n_cols || ldq % 16)
    return fail(SGE_ERR_ARG, "int8_quant_rows: ldq must be a multiple of 16, at least the row length");
  if (n_rows == 0) return SGE_OK;
  if (!x || !q || !scale) return fail(SGE_ERR_ARG, "int8_quant_rows: null pointer");
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale))
    return fail(SGE_ERR_ARG, "int8_quant_rows: pointer not 16-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SGE_BF16) return quant_rows<__nv_bfloat16>(x, ldx, n_rows, n_cols, q, ldq, scale, st);
  return quant_rows<float>(x, ldx, n_rows, n_cols, q, ldq, scale, st);
}

extern "C" int int8_linear(const int8_t* xq, int64_t ldx, const float* sx, const int8_t* wq, int64_t ldw,
                           const float* sw, void* y, int64_t n_tokens, int64_t n_out, int64_t n_in, int dtype,
                           int32_t* diag, void* stream) {
  NvtxRange nvtx_range("int8_linear");
  clear_error();
  if (n_tokens < 0 || n_out < 1 || n_in < 1)
    return fail(SGE_ERR_ARG, "int8_linear: bad sizes tokens=%lld out=%lld in=%lld", (long long)n_tokens,
                (long long)n_out, (long long)n_in);
  if (dtype != SGE_BF16 && dtype != SGE_F32) return fail(SGE_ERR_UNSUPPORTED, "int8_linear: dtype %d", dtype);
  if (n_in > kI8MaxK)
    return fail(SGE_ERR_UNSUPPORTED, "int8_linear: n_in %lld beyond %lld (the 32-bit sums' bound)",
                (long long)n_in, (long long)kI8MaxK);
  if (n_tokens >= kI8MaxRows || n_out >= kI8MaxRows)
    return fail(SGE_ERR_UNSUPPORTED, "int8_linear: size beyond 2^30");
  if (n_tokens == 0) return SGE_OK;
  if (!y) return fail(SGE_ERR_ARG, "int8_linear: null pointer");
  if (!aligned16(y)) return fail(SGE_ERR_ARG, "int8_linear: pointer not 16-byte aligned");
  const int rc = check_product("int8_linear", xq, ldx, sx, wq, ldw, sw, n_in, diag);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SGE_BF16)
    return linear<__nv_bfloat16>(xq, ldx, sx, wq, ldw, sw, y, n_tokens, n_out, n_in, diag, st);
  return linear<float>(xq, ldx, sx, wq, ldw, sw, y, n_tokens, n_out, n_in, diag, st);
}

extern "C" int twell_gate_pack_int8(const int8_t* xq, int64_t ldx, const float* sx, const int8_t* wg_q,
                                    int64_t ldw, const float* sw, int64_t n_tokens, int64_t d_model,
                                    int64_t d_ff, int tile, int cap, uint8_t* count, uint8_t* idx, void* val,
                                    int32_t* diag, void* stream) {
  NvtxRange nvtx_range("twell_gate_pack_int8");
  clear_error();
  const char* fn = "twell_gate_pack_int8";
  if (n_tokens < 0 || d_model < 1 || d_ff < 1)
    return fail(SGE_ERR_ARG, "%s: bad sizes N=%lld d=%lld F=%lld", fn, (long long)n_tokens, (long long)d_model,
                (long long)d_ff);
  if (tile != 16 && tile != 32 && tile != 64 && tile != 128)
    return fail(SGE_ERR_UNSUPPORTED, "%s: tile %d not in {16,32,64,128}", fn, tile);
  if (d_ff % tile) return fail(SGE_ERR_ARG, "%s: d_ff %% tile != 0", fn);
  if (cap < 1 || cap > tile) return fail(SGE_ERR_ARG, "%s: cap %d outside [1, tile]", fn, cap);
  if (d_model > kI8MaxK)
    return fail(SGE_ERR_UNSUPPORTED, "%s: d_model %lld beyond %lld (the 32-bit sums' bound)", fn,
                (long long)d_model, (long long)kI8MaxK);
  if (n_tokens >= kI8MaxRows || d_ff >= kI8MaxRows) return fail(SGE_ERR_UNSUPPORTED, "%s: size beyond 2^30", fn);
  if (n_tokens == 0) return SGE_OK;
  if (!count || !idx || !val) return fail(SGE_ERR_ARG, "%s: null pointer", fn);
  if (!aligned16(count) || !aligned16(idx) || !aligned16(val))
    return fail(SGE_ERR_ARG, "%s: pointer not 16-byte aligned", fn);
  const int rc = check_product(fn, xq, ldx, sx, wg_q, ldw, sw, d_model, diag);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (tile) {
    case 16: return gate<16>(xq, ldx, sx, wg_q, ldw, sw, n_tokens, d_ff, d_model, cap, count, idx, val, diag, st);
    case 32: return gate<32>(xq, ldx, sx, wg_q, ldw, sw, n_tokens, d_ff, d_model, cap, count, idx, val, diag, st);
    case 64: return gate<64>(xq, ldx, sx, wg_q, ldw, sw, n_tokens, d_ff, d_model, cap, count, idx, val, diag, st);
    default: return gate<128>(xq, ldx, sx, wg_q, ldw, sw, n_tokens, d_ff, d_model, cap, count, idx, val, diag, st);
  }
}
