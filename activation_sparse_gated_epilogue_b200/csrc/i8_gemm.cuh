// Persistent tcgen05 GEMM engine for 8-bit integers on sm_100a:
//   D[r][c] = sum_k A[r][k] * B[c][k]   (int8 operands, K-major; exact int32
//   accumulation in tensor memory, kind::i8)
// with a pluggable epilogue, over one matrix or over groups of rows: with
// `offsets` the rows [offsets[g], offsets[g+1]) of A multiply the g-th block
// of p.n rows of B (the experts of a routed feed-forward block).  The integer
// sums are exact, so results do not depend on the order of the k blocks.
//
// The roles, the stage ring, the bounded waits and the abort/drain protocol
// are those of the bf16 engine (tc_gemm.cuh): warp 0 loads tiles by TMA
// (128-byte swizzle rows = 128 int8), one thread of warp 1 issues the MMAs,
// the other warps drain the accumulators.  PAIR: two CTAs on 256-row tiles
// (cta_group::2), each loading its half of the operands; no multicast loads.
//
// PER_BLOCK: every 128-wide k block gets an accumulator of its own, which the
// epilogue scales (one factor per row and k block) and adds in 32-bit floats:
// the down projection of the feed-forward block, whose activations carry one
// scale per token and 128 hidden units.
#pragma once

#include "i8_host.h"
#include "i8_quant.cuh"
#include "sge_host.h"
#include "tc_gemm.cuh"

namespace sge {

constexpr int kI8BK = 128;  // k per stage: one 128-byte swizzle row
constexpr int kMaxGroups = 256;
constexpr int64_t kI8MaxK = 131071;        // k * 128 * 128 stays below 2^31
constexpr int64_t kI8MaxRows = 1LL << 30;  // row and column indices of a tile stay 32-bit

// GROUPED: the engine takes group bounds.  STAGING: bytes of shared memory per
// epilogue warp.
template <int BN_, int NB_, int NACC_, int HALVES_, bool PAIR_, bool GROUPED_, bool PER_BLOCK_, int STAGING_>
struct I8Shape {
  static constexpr bool GROUPED = GROUPED_;
  static constexpr int STAGING = STAGING_;
  static constexpr int BN = BN_, NB = NB_, NACC = NACC_, HALVES = HALVES_;
  static constexpr bool PAIR = PAIR_, PER_BLOCK = PER_BLOCK_;
  // warps before the epilogue's: 2, or a warpgroup of 4 where registers move
  // from it to the epilogue (setmaxnreg works on whole warpgroups)
  static constexpr bool MOVE_REGS = PER_BLOCK && HALVES == 2 && BN / HALVES > 64;
  static constexpr int FIRST_EPI = MOVE_REGS ? 4 : 2;
  // what the warpgroups ask for with setmaxnreg: it draws on the registers of
  // the launch, so their sum may not pass those (launch_i8_gemm checks it)
  static constexpr int FEW_REGS = 56, MANY_REGS = 224;
  static constexpr int THREADS = 32 * FIRST_EPI + 128 * HALVES;
  static constexpr int BM = PAIR ? 2 * kBM : kBM;
  // B rows of one load.  NB = 2: two matrices' tiles of BN rows side by side
  // are one operand of 2 BN rows (one MMA with N = 256 reads A once; two with
  // N = 128 took 1.3 times as long); of a pair each CTA loads one matrix's.
  static constexpr int B_ROWS = PAIR ? NB * BN / 2 : BN;
  static constexpr int B_LOADS = PAIR ? 1 : NB;
  static constexpr int MMA_N = NB * BN;
  static constexpr int A_BYTES = kBM * kI8BK;
  static constexpr int B_BYTES = B_ROWS * kI8BK;
  static constexpr int STAGE_BYTES = A_BYTES + B_LOADS * B_BYTES;
  static constexpr int SCALES_AHEAD = PER_BLOCK ? 8 : 0;  // slots of block scales per epilogue thread
  static constexpr int STAGING_BYTES = 4 * HALVES * STAGING + SCALES_AHEAD * 128 * HALVES * 4;
  // the stage ring takes what is left of 227 KB (2 KB of it: the tile list)
  static constexpr int RING = 227 * 1024 - (GROUPED ? 2304 : 256) - 1024 - 512 - STAGING_BYTES;
  static constexpr int STAGES = RING / STAGE_BYTES > 8 ? 8 : RING / STAGE_BYTES;
  static constexpr int ACC_COLS = BN * NB;
  static constexpr int USED_COLS = NACC * ACC_COLS;
  static constexpr int TMEM_COLS = USED_COLS <= 32 ? 32 : USED_COLS <= 64 ? 64 : USED_COLS <= 128 ? 128
                                   : USED_COLS <= 256 ? 256 : 512;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + STAGING_BYTES + 1024 /*align slack*/ + 512 /*barriers*/;
  static_assert(USED_COLS <= 512, "TMEM columns");
  static_assert(MMA_N % (PAIR ? 32 : 16) == 0 && MMA_N <= 256, "UMMA N");
  static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "1024-byte aligned sub-tiles");
  static_assert(HALVES == 1 || NB == 1, "column halves need one accumulator");
  static_assert(!PER_BLOCK || NB == 1, "per-block scales: one accumulator");
  // PER_BLOCK epilogues wait on the stages' barriers: at most NACC blocks behind
  // the MMAs, they must not miss a phase
  static_assert(!PER_BLOCK || STAGES >= NACC, "stages");
};

// The products of the gated feed-forward block.
using GateUpPair = I8Shape<128, 2, 2, 1, true, true, false, 0>;
using GateUpOne = I8Shape<128, 2, 2, 1, false, true, false, 0>;
using DownPair = I8Shape<256, 1, 2, 2, true, true, true, 4096>;
using DownOne = I8Shape<128, 1, 4, 2, false, true, true, 4096>;

struct I8Problem {
  int rows;    // rows of A
  int n;       // output columns of a group (rows of B per group)
  int k;       // bytes of a row
  int groups;  // 1..kMaxGroups
  int splits;  // K is cut into this many parts, none empty, each an output of its own
  const int32_t* offsets;  // [groups + 1] row bounds on the device, or null (one group)
};

// One output tile: rows [row0, row_end) (at most BM of them are computed),
// columns [col0, col0 + BN) of group `group`, k blocks [kb0, kb1).
struct I8Tile {
  int group, row0, row_end, col0, split, kb0, kb1;
};

// The tile list, built in shared memory from the group bounds.
template <class Shape>
struct I8Sched {
  static constexpr int GROUPS = Shape::GROUPED ? kMaxGroups : 1;
  int off[GROUPS + 1];    // clamped group bounds
  int first[GROUPS + 1];  // row blocks before group g

  // one whole warp
  __device__ __forceinline__ void build(const I8Problem& p, int lane) {
    int run = 0, floor = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
      const int g = g0 + lane;
      // group g ends at hi and begins where the one before ends; bounds that
      // are out of range or out of order give fewer rows, never an overlap or
      // an access out of range
      int hi = p.rows, begin = 0;
      if (p.offsets) {
        hi = g < p.groups ? checked_bound(p.offsets[g + 1], 0, p.rows) : 0;
        if (g == 0) begin = checked_bound(p.offsets[0], 0, p.rows);
        hi = max(hi, max(begin, floor));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, hi, o);
          if (lane >= o) hi = max(hi, u);
        }
      }
      int lo = __shfl_up_sync(0xffffffffu, hi, 1);
      if (lane == 0) lo = g == 0 ? begin : floor;
      floor = __shfl_sync(0xffffffffu, hi, 31);
      const int blocks = g < p.groups ? (hi - lo + Shape::BM - 1) / Shape::BM : 0;
      int incl = blocks;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      if (g < p.groups) {
        off[g] = lo;
        first[g] = run + incl - blocks;
        if (g == p.groups - 1) off[p.groups] = hi;
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) first[p.groups] = run;
  }

  __device__ __forceinline__ I8Tile tile(const I8Problem& p, int t, int k_blocks) const {
    I8Tile r;
    r.split = t % p.splits;
    t /= p.splits;
    const int m_blocks = first[p.groups];
    const int mb = t % m_blocks;
    r.col0 = t / m_blocks * Shape::BN;
    int lo = 0, hi = p.groups;  // the last group whose first block is <= mb
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= mb) lo = mid;
      else hi = mid;
    }
    r.group = lo;
    r.row0 = off[lo] + (mb - first[lo]) * Shape::BM;
    r.row_end = off[lo + 1];
    const int per = (k_blocks + p.splits - 1) / p.splits;
    r.kb0 = min(k_blocks, r.split * per);
    r.kb1 = min(k_blocks, r.kb0 + per);
    return r;
  }

  __device__ __forceinline__ int tiles(const I8Problem& p) const {
    return first[p.groups] * ((p.n + Shape::BN - 1) / Shape::BN) * p.splits;
  }
};

// Instruction descriptor: kind::i8, signed A and B, 32-bit integer
// accumulator, both operands K-major, tile M x N.
constexpr uint32_t umma_idesc_i8(int m, int n) {
  return (2u << 4)                                // D format: s32
         | (1u << 7)                              // A format: signed 8 bit
         | (1u << 10)                             // B format: signed 8 bit
         | (static_cast<uint32_t>(n >> 3) << 17)  // N / 8
         | (static_cast<uint32_t>(m >> 4) << 24); // M / 16
}

template <bool PAIR>
SGE_DEV void umma_i8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

template <bool PAIR>
SGE_DEV void i8_commit(uint64_t* bar) {
  if constexpr (PAIR) umma2_commit_mc(bar, 0x3);
  else umma_commit(bar);
}

// Rows of 128 bytes from one warp's staging memory to global memory.  A lane
// holds one row of a tile, but 32 rows' 16-byte stores are 32 lines each; via
// shared memory (16-byte pieces swizzled by row, so that neither side has bank
// conflicts) a store covers four whole rows, and where the matrix's pitch leaves
// rows unaligned, 32 neighbouring elements.
template <class T>
struct StagedRows {
  static constexpr int COLS = 128 / static_cast<int>(sizeof(T));  // columns at a time
  static constexpr int PER = 16 / static_cast<int>(sizeof(T));

  SGE_DEV static uint8_t* piece(uint8_t* stage, int row, int p) { return stage + row * 128 + ((p ^ (row & 7)) * 16); }

  // this lane's row: columns [c, c + W) of the 128 bytes
  template <int W>
  SGE_DEV static void put(uint8_t* stage, int lane, int c, const float (&v)[W]) {
#pragma unroll
    for (int j = 0; j < W; j += PER) {
      uint32_t w[4];
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = static_cast<uint32_t>(f32_to_bf16_bits(v[j + 2 * i])) |
                 (static_cast<uint32_t>(f32_to_bf16_bits(v[j + 2 * i + 1])) << 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[j + i]);
      }
      *reinterpret_cast<uint4*>(piece(stage, lane, (c + j) / PER)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }

  // all lanes: rows [row0, row0 + 32) (those below row_end) of a matrix of
  // `pitch` columns, its columns [col0, col0 + COLS) (those below pitch)
  SGE_DEV static void flush(uint8_t* stage, int lane, T* out, int64_t row0, int64_t row_end, int col0, int pitch) {
    __syncwarp();
    if (pitch % PER == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + lane / 8, p = lane % 8;
        const uint4 v = *reinterpret_cast<const uint4*>(piece(stage, r, p));
        const int col = col0 + p * PER;
        if (row0 + r < row_end && col < pitch) *reinterpret_cast<uint4*>(out + (row0 + r) * pitch + col) = v;
      }
    } else {
#pragma unroll 8
      for (int r = 0; r < 32; ++r) {
#pragma unroll
        for (int c = lane; c < COLS; c += 32) {
          const T v = reinterpret_cast<const T*>(piece(stage, r, c / PER))[c % PER];
          if (row0 + r < row_end && col0 + c < pitch) out[(row0 + r) * pitch + col0 + c] = v;
        }
      }
    }
    __syncwarp();
  }
};

// Arrive on a barrier of another CTA of the cluster.  CTA scope: what it
// orders is this warp's tensor-memory reads, done before the tcgen05 fence in
// front of it; cluster scope would also wait for the warp's global stores and
// loads in flight, once per accumulator.
SGE_DEV void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// What an epilogue call gets: the accumulator's TMEM address (this warp's
// lanes, its first column), this thread's row and its tile.
struct I8Out {
  uint32_t taddr;
  int64_t row;      // row of A of this thread
  int64_t row_end;  // end of the tile's group
  bool row_ok;      // row < row_end
  int lane;
  int col0;     // first column (within the group) of this warp's share
  int group, split;
  uint8_t* stage;  // this warp's staging memory
};

template <class Shape, class Epilogue>
__global__ void __launch_bounds__(Shape::THREADS, 1)
    i8_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b0,
                   const __grid_constant__ CUtensorMap map_b1, const I8Problem p, const Epilogue epi,
                   int32_t* diag) {
  constexpr int BN = Shape::BN, NB = Shape::NB, NACC = Shape::NACC, STAGES = Shape::STAGES;
  constexpr bool PAIR = Shape::PAIR, PER_BLOCK = Shape::PER_BLOCK;
  extern __shared__ uint8_t smem_raw[];
  __shared__ I8Sched<Shape> sched;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* staging = smem + STAGES * Shape::STAGE_BYTES;
  float* scales = reinterpret_cast<float*>(staging + 4 * Shape::HALVES * Shape::STAGING);
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + Shape::STAGING_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tmem_full = empty + STAGES;
  uint64_t* tmem_empty = tmem_full + NACC;
  uint64_t* drain = tmem_empty + NACC;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0;
  const bool leader = rank == 0;
  const int worker = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int n_workers = PAIR ? static_cast<int>(cluster_count_x()) : static_cast<int>(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < NACC; ++a) {
      mbar_init(&tmem_full[a], 1);
      mbar_init(&tmem_empty[a], (PAIR ? 8 : 4) * Shape::HALVES);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_b0);
    if (NB == 2) tma_prefetch_desc(&map_b1);
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc_pair(tmem_holder, Shape::TMEM_COLS);
    else tmem_alloc(tmem_holder, Shape::TMEM_COLS);
  }
  // the set-up above overlaps the previous kernel; what it wrote (the group
  // bounds among it) is read only below
  grid_dep_wait();
  grid_dep_launch();
  if (warp == 0) sched.build(p, lane);
  tc_fence_before();
  if constexpr (PAIR) cluster_sync();  // both CTAs' barriers exist before any remote arrive / TMA
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int k_blocks = (p.k + kI8BK - 1) / kI8BK;
  const int num_tiles = sched.tiles(p);

  // MOVE_REGS: 384 threads start with 168 registers each (64,512 in all); 56 for
  // the first warpgroup and 224 for the two epilogue warpgroups are as many
  if (warp < Shape::FIRST_EPI) {
    if constexpr (Shape::MOVE_REGS) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Shape::FEW_REGS));
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- TMA producer
      int s = 0;
      uint32_t ph = 0, armed = 0, armed_par = 0;
      const uint32_t bytes =
          PAIR ? 2 * Shape::STAGE_BYTES : a_box_rows(p.rows) * kI8BK + Shape::B_LOADS * Shape::B_BYTES;
      for (int t = worker; t < num_tiles && !*abort_flag; t += n_workers) {
        const I8Tile tc = sched.tile(p, t, k_blocks);
        const int a_row = tc.row0 + static_cast<int>(rank) * kBM;
        const int b_row = tc.group * p.n + tc.col0 + (NB == 1 ? static_cast<int>(rank) * Shape::B_ROWS : 0);
        for (int kb = tc.kb0; kb < tc.kb1; ++kb) {
          if (!wait_or_abort(&empty[s], ph ^ 1, abort_flag, diag)) break;
          uint8_t* sa = smem + s * Shape::STAGE_BYTES;
          if (leader) mbar_arrive_expect_tx(&full[s], bytes);
          if constexpr (PAIR) {
            tma_load_2d_pair(sa, &map_a, &full[s], kb * kI8BK, a_row);
            tma_load_2d_pair(sa + Shape::A_BYTES, NB == 1 || leader ? &map_b0 : &map_b1, &full[s], kb * kI8BK,
                             b_row);
          } else {
            tma_load_2d(sa, &map_a, &full[s], kb * kI8BK, a_row);
            tma_load_2d(sa + Shape::A_BYTES, &map_b0, &full[s], kb * kI8BK, b_row);
            if (NB == 2)
              tma_load_2d(sa + Shape::A_BYTES + Shape::B_BYTES, &map_b1, &full[s], kb * kI8BK, b_row);
          }
          armed |= 1u << s;
          armed_par = (armed_par & ~(1u << s)) | (ph << s);
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // Drain: no load of this CTA (PAIR: of either CTA) is in flight after this.
      if (leader)
        for (int t = 0; t < STAGES; ++t)
          if (armed & (1u << t)) mbar_wait(&full[t], (armed_par >> t) & 1, diag);
    } else if (warp == 1 && leader) {
      // ------------------------------------------------------ MMA issuer
      // The whole warp walks the loop and one elected thread issues: with
      // uniform control flow around them the instructions go out several
      // times faster than from a single diverged lane (one lane took about
      // 700 cycles for the four MMAs of a stage, whatever their N).
      constexpr uint32_t idesc = umma_idesc_i8(Shape::BM, Shape::MMA_N);
      const uint64_t adesc0 = umma_desc_sw128(smem_u32(smem));
      const uint64_t bdesc0 = umma_desc_sw128(smem_u32(smem) + Shape::A_BYTES);
      const bool elected = elect_one_sync();
      int s = 0, acc = 0;
      uint32_t ph = 0, acc_ph = 0;
      bool ok = true;
      for (int t = worker; ok && t < num_tiles && !*abort_flag; t += n_workers) {
        const I8Tile tc = sched.tile(p, t, k_blocks);
        for (int kb = tc.kb0; kb < tc.kb1; ++kb) {
          const bool fresh = PER_BLOCK || kb == tc.kb0;
          if (fresh) {
            ok = __all_sync(0xffffffffu, wait_or_abort(&tmem_empty[acc], acc_ph ^ 1, abort_flag, diag));
            if (!ok) break;
          }
          ok = __all_sync(0xffffffffu, wait_or_abort(&full[s], ph, abort_flag, diag));
          if (!ok) break;
          tc_fence_after();
          if (elected) {
            const uint32_t d_tmem = tmem_base + acc * Shape::ACC_COLS;
            const uint64_t at = static_cast<uint64_t>(s * (Shape::STAGE_BYTES >> 4));
#pragma unroll
            for (int k = 0; k < kI8BK / 32; ++k)
              umma_i8<PAIR>(d_tmem, adesc0 + at + 2 * k, bdesc0 + at + 2 * k, idesc, (!fresh || k != 0) ? 1u : 0u);
            // frees the stage; PER_BLOCK it also says that the block's sums are there
            i8_commit<PAIR>(&empty[s]);
            if (!PER_BLOCK && kb == tc.kb1 - 1) i8_commit<PAIR>(&tmem_full[acc]);
          }
          __syncwarp();
          if (++s == STAGES) {
            s = 0;
            ph ^= 1;
          }
          if ((PER_BLOCK || kb == tc.kb1 - 1) && ++acc == NACC) {
            acc = 0;
            acc_ph ^= 1;
          }
        }
      }
      if (elected) i8_commit<PAIR>(drain);  // completes once every MMA issued above has
      __syncwarp();
    }
    if (warp == 1 && lane == 0) mbar_wait(drain, 0, diag);
    __syncwarp();
  } else {
    // --------------------------------------------------------- epilogue
    if constexpr (Shape::MOVE_REGS) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Shape::MANY_REGS));
    const int quarter = warp & 3;      // TMEM lanes this warp may access
    const int half = (warp - Shape::FIRST_EPI) >> 2;  // column half (HALVES = 2)
    constexpr int COLS = BN / Shape::HALVES;
    const uint32_t lane_base = tmem_base + half * COLS + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t release0 = PAIR ? mapa_shared(smem_u32(&tmem_empty[0]), 0) : 0;
    int acc = 0, s_done = 0;  // s_done: the stage of the block at hand (PER_BLOCK)
    uint32_t acc_ph = 0, s_ph = 0;
    const auto release = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_remote(release0 + acc * 8);
        else mbar_arrive(&tmem_empty[acc]);
      }
      if (++acc == NACC) {
        acc = 0;
        acc_ph ^= 1;
      }
    };
    // this thread's place in a tile
    const auto place = [&](const I8Tile& tc) {
      I8Out o;
      o.row = static_cast<int64_t>(tc.row0) + rank * kBM + quarter * 32 + lane;
      o.row_end = tc.row_end;
      o.row_ok = o.row < tc.row_end;
      o.lane = lane;
      o.stage = staging + (warp - Shape::FIRST_EPI) * Shape::STAGING;
      o.col0 = tc.col0 + half * COLS;
      o.group = tc.group;
      o.split = tc.split;
      return o;
    };
    // PER_BLOCK: the blocks' scales come by asynchronous copies to this thread's
    // own slots, SCALES_AHEAD blocks early: a load from L2 takes longer than a
    // block, and there are no registers left to hold values in flight.
    constexpr int AHEAD = Shape::SCALES_AHEAD;
    const uint32_t slots = smem_u32(scales + threadIdx.x - 32 * Shape::FIRST_EPI);
    const auto fetch_scale = [&](const float* src, int kb, int kb1, int slot) {
      if constexpr (PER_BLOCK) {
        if (kb < kb1)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(slots + slot * (128 * Shape::HALVES * 4)),
                       "l"(src + static_cast<int64_t>(kb) * epi.scale_pitch())
                       : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
      }
    };
    // the first scales of tile t (the tile before's are all used by then)
    const auto fetch_first = [&](int t) {
      if constexpr (PER_BLOCK) {
        if (t >= num_tiles) return;
        const I8Tile tc = sched.tile(p, t, k_blocks);
        const float* src = epi.block_scales(place(tc));
#pragma unroll 1
        for (int i = 0; i < AHEAD; ++i) fetch_scale(src, tc.kb0 + i, tc.kb1, i);
      }
    };
    bool ok = true;
    // A single CTA fetches a tile's first scales before it stores the tile
    // before (5-10% of the block where experts leave it short tiles); a pair as
    // the tile begins: there the other order costs registers (171 -> 179 us for
    // the down product at the 1B shape).
    if (!PAIR) fetch_first(worker);
    for (int t = worker; ok && t < num_tiles; t += n_workers) {
      const I8Tile tc = sched.tile(p, t, k_blocks);  // no split is empty: the host sees to it
      const I8Out o = place(tc);
      // a warp whose rows all lie past the group's end only keeps the pace
      const bool any = (PAIR && PER_BLOCK) || __any_sync(0xffffffffu, o.row_ok);
      if (PAIR) fetch_first(t);
      if constexpr (PER_BLOCK) {
        float sum[COLS];
#pragma unroll
        for (int j = 0; j < COLS; ++j) sum[j] = 0.0f;
        const float* src_scale = epi.block_scales(o);
        int slot = 0;
#pragma unroll 1
        for (int kb = tc.kb0; kb < tc.kb1; ++kb) {
          asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
          float scale;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(scale) : "r"(slots + slot * (128 * Shape::HALVES * 4)) : "memory");
          fetch_scale(src_scale, kb + AHEAD, tc.kb1, slot);
          slot = slot + 1 == AHEAD ? 0 : slot + 1;
          // the commit that frees the block's stage also says that its sums are there
          ok = __all_sync(0xffffffffu, wait_or_abort(&empty[s_done], s_ph, abort_flag, diag));
          if (!ok) break;
          if (++s_done == STAGES) {
            s_done = 0;
            s_ph ^= 1;
          }
          tc_fence_after();
          if (!any) {
            release();
            continue;
          }
          const uint32_t src = lane_base + acc * Shape::ACC_COLS;
          uint32_t r[2][32];
          tmem_ld32(src, r[0]);
#pragma unroll
          for (int ch = 0; ch < COLS / 32; ++ch) {
            tmem_ld_wait();
            if (ch + 1 < COLS / 32) tmem_ld32(src + (ch + 1) * 32, r[(ch + 1) & 1]);
            else release();  // the block's last sums are in registers: the MMA may write over them
#pragma unroll
            for (int j = 0; j < 32; ++j)
              sum[ch * 32 + j] = fmaf(__int2float_rn(static_cast<int>(r[ch & 1][j])), scale, sum[ch * 32 + j]);
          }
        }
        if (!ok) break;
        if (!PAIR) fetch_first(t + n_workers);
        if (any) epi.template store<COLS>(o, sum, p.n);
      } else {
        ok = __all_sync(0xffffffffu, wait_or_abort(&tmem_full[acc], acc_ph, abort_flag, diag));
        if (!ok) break;
        tc_fence_after();
        if (any) {
          I8Out at = o;
          at.taddr = lane_base + acc * Shape::ACC_COLS;
          epi.template run<COLS>(at, p.n);
        }
        release();
      }
    }
    // every scale that is used has been waited for; a warp that gives up leaves
    // copies to its slots in flight
    if constexpr (PER_BLOCK) asm volatile("cp.async.wait_all;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // no CTA leaves while its pair may still touch its barriers or TMEM
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, Shape::TMEM_COLS);
    else tmem_dealloc(tmem_base, Shape::TMEM_COLS);
  }
}

// ------------------------------------------------------------- launchers

// Tensor maps of an engine call.  B: `b_rows` rows of k bytes, pitch ldb.
struct I8Maps {
  CUtensorMap a, b0, b1;
};

template <class Shape>
int make_i8_maps(I8Maps* m, const I8Problem& p, const int8_t* a, int64_t lda, const int8_t* b0,
                 const int8_t* b1, int64_t ldb) {
  const uint32_t a_box = Shape::PAIR ? kBM : a_box_rows(p.rows);
  const uint64_t b_rows = static_cast<uint64_t>(p.n) * p.groups;
  int rc = make_tmap_i8(&m->a, a, p.rows, p.k, lda, a_box);
  if (!rc) rc = make_tmap_i8(&m->b0, b0, b_rows, p.k, ldb, Shape::B_ROWS);
  if (!rc && b1) rc = make_tmap_i8(&m->b1, b1, b_rows, p.k, ldb, Shape::B_ROWS);
  if (!b1) m->b1 = m->b0;  // not used
  return rc;
}

// CTAs (PAIR: CTA pairs) of a kernel that can be resident at once, per device.
template <class Shape, class Epi>
int i8_workers() {
  if constexpr (!Shape::PAIR) return sm_count();
  static PerDevice cached;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return sm_count() / 2;
  return cached.get(dev, [] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (sm_count() / 2));
    cfg.blockDim = dim3(Shape::THREADS);
    cfg.dynamicSmemBytes = Shape::SMEM_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const void* kern = reinterpret_cast<const void*>(i8_gemm_kernel<Shape, Epi>);
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = sm_count() / 2;
    }
    return n;
  });
}

template <class Shape, class Epi>
int launch_i8_gemm(const I8Maps& m, const I8Problem& p, const Epi& epi, int32_t* diag, cudaStream_t st,
                   const char* what) {
  auto kern = i8_gemm_kernel<Shape, Epi>;
  int rc = set_smem_limit(reinterpret_cast<const void*>(kern), Shape::SMEM_BYTES);
  if (rc) return rc;
  // the most row blocks there can be: with groups, one partial block more for each
  if constexpr (Shape::MOVE_REGS) {
    static const int launch_regs = [&] {
      cudaFuncAttributes attr = {};
      return cudaFuncGetAttributes(&attr, reinterpret_cast<const void*>(kern)) == cudaSuccess ? attr.numRegs : 0;
    }();
    if (launch_regs * Shape::THREADS < 128 * Shape::FEW_REGS + 256 * Shape::MANY_REGS)
      return fail(SGE_ERR_CUDA, "%s: built with %d registers a thread, too few for its warpgroups' shares", what,
                  launch_regs);
  }
  int64_t m_blocks = (p.rows + Shape::BM - 1) / Shape::BM;
  if (p.offsets) m_blocks += p.groups - 1 < p.rows ? p.groups - 1 : p.rows;
  const int64_t tiles = m_blocks * ((p.n + Shape::BN - 1) / Shape::BN) * p.splits;
  const int64_t slots = i8_workers<Shape, Epi>();
  const int workers = static_cast<int>(tiles < slots ? tiles : slots);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(Shape::PAIR ? 2 * workers : workers);
  cfg.blockDim = dim3(Shape::THREADS);
  cfg.dynamicSmemBytes = Shape::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = Shape::PAIR ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, m.a, m.b0, m.b1, p, epi, diag);
  if (e != cudaSuccess) return fail(SGE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

}  // namespace sge
