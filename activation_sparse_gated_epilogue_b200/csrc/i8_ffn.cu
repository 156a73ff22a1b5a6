// The gated feed-forward block on 8-bit weights, of one expert or of the
// experts that a route chose:
//
//   xq, sx    the tokens' rows, quantised (int8_quant_rows), in expert order
//   g, u      (sum xq wg) * sx * sg  and  (sum xq wu) * sx * su, fp32
//   h         ReLU(g) * u, quantised per token and group of 128 hidden units
//   z         sum over groups of (sum hq wd) * sh, times sd
//   y         z, or the sum of a token's experts' z with its weights
//
// The hidden activation's scale is per token and 128 hidden units, not per
// token, because a whole row's largest value is known only when every column
// tile of the first product is done: that would take a wider copy of h to
// HBM and back.  128 units are one tile of the first product's epilogue and
// one k block of the second product, whose integer sums over a block are
// exact; the blocks are scaled and added in fp32.
#include "i8_gemm.cuh"
#include "i8_quant.cuh"
#include "i8_small.cuh"

namespace sge {

// ------------------------------------------- quantise and order the tokens

// One warp per token; its row goes to every place of the token (pos null: to
// its own row).  8192 x 2048 bf16, one place: 14 us (33.5 MB in, 16.8 MB out).
template <class T>
__global__ void __launch_bounds__(256) i8_dispatch_kernel(const T* __restrict__ x, int64_t n, int d, int k,
                                                          const int32_t* __restrict__ pos, int rows,
                                                          int8_t* __restrict__ q, int64_t ldq,
                                                          float* __restrict__ scale) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= n) return;
  // the token's places; a number outside [0, rows): none
  __shared__ uint32_t s_place[8][16];
  uint32_t* place = s_place[threadIdx.x >> 5];
  if (lane < k) place[lane] = pos ? checked_place(pos[row * k + lane], rows) : static_cast<uint32_t>(row);
  __syncwarp();
  uint32_t amax;
  quant_row<T, true, 8>(x + row * d, d, lane, amax, [&](int c, const auto& f, float inv) {
    for (int j = 0; j < k; ++j) {
      const uint32_t p = place[j];
      if (p < static_cast<uint32_t>(rows)) store_q(q + p * ldq + c, f, inv);
    }
  });
  const float s = quant_scale(amax).scale;
  for (int j = 0; j < k; ++j) {
    const uint32_t p = place[j];
    if (p >= static_cast<uint32_t>(rows)) continue;
    if (lane == 0) scale[p] = s;
    // a row ends with at most 8 bytes of padding (d % 8 == 0)
    if (lane == 1 && d % 16) *reinterpret_cast<uint2*>(q + p * ldq + d) = make_uint2(0, 0);
  }
}

// --------------------------------------------------------------- epilogues

// h = ReLU(g) * u of one row and 128 hidden units, quantised.  A thread holds
// its row's 128 values in registers between their maximum and their rounding.
// 8192 x 2048 x 8192: 168 us for both projections, 3.27 POPS, tensor pipe 87%.
struct EpiI8Gated {
  int8_t* hq;
  int64_t ldh;
  float* hs;  // [groups of 128][rows]
  int64_t rows;
  const float* sx;
  const float* sg;
  const float* su;

  template <int COLS>
  __device__ __forceinline__ void run(const I8Out& o, int n) const {
    static_assert(COLS == kHGroup, "a tile's columns are one group");
    const float s = o.row_ok ? __ldg(sx + o.row) : 0.0f;
    const float* cg = sg + static_cast<int64_t>(o.group) * n + o.col0;
    const float* cu = su + static_cast<int64_t>(o.group) * n + o.col0;
    float h[COLS];
    uint32_t amax = 0;
#pragma unroll
    for (int ch = 0; ch < COLS / 32; ++ch) {
      uint32_t g[32], u[32];
      tmem_ld32(o.taddr + ch * 32, g);
      tmem_ld32(o.taddr + COLS + ch * 32, u);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; j += 4) {
        // n % 8 == 0: four columns are inside the group's weights or all outside
        const bool in = o.col0 + ch * 32 + j < n;
        const float4 a = in ? __ldg(reinterpret_cast<const float4*>(cg + ch * 32 + j)) : make_float4(0, 0, 0, 0);
        const float4 b = in ? __ldg(reinterpret_cast<const float4*>(cu + ch * 32 + j)) : make_float4(0, 0, 0, 0);
        const float sa[4] = {a.x, a.y, a.z, a.w}, sb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float gv = __int2float_rn(static_cast<int>(g[j + i])) * s * sa[i];
          const float uv = __int2float_rn(static_cast<int>(u[j + i])) * s * sb[i];
          // a NaN (from a token that is not finite) stays one
          const float v = in ? (gv < 0.0f ? 0.0f : gv) * uv : 0.0f;
          h[ch * 32 + j + i] = v;
          amax = max(amax, abs_bits(v));
        }
      }
    }
    if (!o.row_ok) return;
    const QuantScale qs = quant_scale(amax);
    int8_t* dst = hq + o.row * ldh + o.col0;
#pragma unroll
    for (int j = 0; j < COLS; j += 16)
      if (o.col0 + j < ldh)
        *reinterpret_cast<uint4*>(dst + j) = make_uint4(
            quant_pack4(h[j], h[j + 1], h[j + 2], h[j + 3], qs.inv),
            quant_pack4(h[j + 4], h[j + 5], h[j + 6], h[j + 7], qs.inv),
            quant_pack4(h[j + 8], h[j + 9], h[j + 10], h[j + 11], qs.inv),
            quant_pack4(h[j + 12], h[j + 13], h[j + 14], h[j + 15], qs.inv));
    hs[static_cast<int64_t>(o.col0 / kHGroup) * rows + o.row] = qs.scale;
  }
};

// Block sums scaled and added (in the engine), then the channel's scale.  8192 x
// 8192 x 2048: 173 us, 1.6 POPS: two instructions for each of the 1.07 x 10^9 block
// sums (conversion, multiply-add) keep the epilogue busier than the tensor pipe
// (46%), and 256 tiles are 3.5 waves of 74 pairs.
template <class T>
struct EpiI8Down {
  T* z;  // [splits][rows][n]
  int64_t rows;
  const float* hs;
  const float* sd;

  // this thread's row's scales, one every scale_pitch() floats (rows past the
  // group's: some row's, their sums are not stored)
  __device__ __forceinline__ const float* block_scales(const I8Out& o) const {
    return hs + (o.row < rows ? o.row : rows - 1);
  }
  __device__ __forceinline__ int64_t scale_pitch() const { return rows; }

  template <int COLS>
  __device__ __forceinline__ void store(const I8Out& o, const float (&sum)[COLS], int n) const {
    const float* cd = sd + static_cast<int64_t>(o.group) * n;
    using Rows = StagedRows<T>;
    T* out = z + o.split * rows * n;
    // all scales of 32 columns at once, those of the next 32 in flight while
    // these are stored (n % 8 == 0: four columns are inside or outside together)
    float4 next[8];
    const auto fetch = [&](int c) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        next[j] = __ldg(reinterpret_cast<const float4*>(cd + min(o.col0 + c + 4 * j, n - 4)));
    };
    fetch(0);
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
      float4 sc[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) sc[j] = next[j];
      if (c + 32 < COLS) fetch(c + 32);
      float v[32];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[4 * j] = sum[c + 4 * j] * sc[j].x;
        v[4 * j + 1] = sum[c + 4 * j + 1] * sc[j].y;
        v[4 * j + 2] = sum[c + 4 * j + 2] * sc[j].z;
        v[4 * j + 3] = sum[c + 4 * j + 3] * sc[j].w;
      }
      Rows::put(o.stage, o.lane, c % Rows::COLS, v);
      if ((c + 32) % Rows::COLS == 0)
        Rows::flush(o.stage, o.lane, out, o.row - o.lane, o.row_end, o.col0 + c + 32 - Rows::COLS, n);
    }
  }
};

// y[t] = sum over the token's places of w * (sum over splits of z), in the
// order of the token's experts and of the splits.  z is kept in fp32 whatever
// the activations' type, so that y is rounded once, in the end, on every path:
// with z in bf16 a token's result was less exact (0.0023 against 0.0017 of its
// norm) in the batches whose down product is not split than in the others.
// One warp per token and 256 columns, eight a lane; columns are clamped, not
// branched around, so that the loads of several splits and places are in flight
// together (with a branch before each it took 1.6 times as long).  8000 tokens
// over 16 experts of 2048 x 2048, two a token: the block took 238 us with z in
// bf16 and takes 253 us (131 MB more through HBM; this kernel alone 34 us, 131 MB
// read).  Sixteen columns a lane spill
// at four blocks per SM (64 registers): 1-3% more of the block at 2048 to 12000
// tokens over 8 to 32 experts.
template <class T>
__global__ void __launch_bounds__(256, 6)
    i8_combine_kernel(const float* __restrict__ z, int rows, int splits, int64_t n, int d, int k,
                      const float* __restrict__ w, const int32_t* __restrict__ pos,
                      const int32_t* __restrict__ offsets, int experts, T* __restrict__ y) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int W = 8, N = Vec16<float>::N;
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (t >= n) return;
  // the experts' rows, all together: only there has z been written
  int begin = 0, end = rows;
  if (offsets) {
    begin = checked_bound(offsets[0], 0, rows);
    end = 0;
    for (int i = lane; i <= experts; i += 32) end = max(end, checked_bound(offsets[i], 0, rows));
    end = __reduce_max_sync(0xffffffffu, end);
  }
  uint32_t my_place = 0xffffffffu;
  float my_w = 1.0f;
  if (lane < k) {
    my_place = pos ? checked_place(pos[t * k + lane], rows) : static_cast<uint32_t>(t);
    if (w) my_w = w[t * k + lane];
  }
  const int col = (blockIdx.y * 32 + lane) * W, from = min(col, d - W);  // d % 8 == 0
  float sum[W];
#pragma unroll
  for (int j = 0; j < W; ++j) sum[j] = 0.0f;
  const int64_t split_step = static_cast<int64_t>(rows) * d;
#pragma unroll 2
  for (int a = 0; a < k; ++a) {
    const uint32_t p = __shfl_sync(0xffffffffu, my_place, a);
    const float wt = __shfl_sync(0xffffffffu, my_w, a);
    if (p < static_cast<uint32_t>(begin) || p >= static_cast<uint32_t>(end)) continue;
    const float* src = z + static_cast<int64_t>(p) * d + from;
    float part[W];
#pragma unroll
    for (int j = 0; j < W; ++j) part[j] = 0.0f;
#pragma unroll 2
    for (int s = 0; s < splits; ++s) {
      uint4 raw[W / N];
#pragma unroll
      for (int j = 0; j < W / N; ++j) raw[j] = *reinterpret_cast<const uint4*>(src + s * split_step + j * N);
#pragma unroll
      for (int j = 0; j < W / N; ++j) {
        float f[N];
        Vec16<float>::unpack(raw[j], f);
#pragma unroll
        for (int m = 0; m < N; ++m) part[j * N + m] += f[m];
      }
    }
#pragma unroll
    for (int j = 0; j < W; ++j) sum[j] = fmaf(wt, part[j], sum[j]);
  }
  if (col < d) store8(y + t * d + col, sum);
}

// ------------------------------------------------------------------- host

static int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

struct FfnPlan {
  int64_t rows;     // assignments: n, or n * k
  bool small;       // the kernels for a few tokens
  bool pairs;       // CTA-pair tiles
  int splits;       // parts of the down projection's K
  bool combine;     // y is summed from z (fp32) by the combine kernel
  int64_t ldx, ldh;
  size_t xq, sx, hq, hs, z, total;  // workspace offsets
};

// Of a split down product.  This and the plan's other bounds are numbers of this
// GPU's 148 SMs, not of the current device: the size query for the workspace may
// be made without one, and the call must come to the same plan.
constexpr int64_t kSplitTiles = 148, kMaxSplits = 16;

static FfnPlan ffn_plan(int64_t n, int64_t d, int64_t f, int e, int k, bool routed) {
  FfnPlan p = {};
  p.rows = routed ? n * k : n;
  // A few tokens whose quantised rows fit a block's shared memory, at most two
  // for each expert that can have any: 2048 x 8192 without experts took 18 / 21
  // / 31 us for 1 / 2 / 4 tokens there and 28 to 31 us on tiles, weights in L2 (20 /
  // 23 us for 1 / 2, 34 on tiles, from HBM); 32 experts of 1024 x 1024, 4 of them a
  // token, 28 us for 8 tokens and 39 us for 9 on tiles (30 and 45 from HBM).
  p.small = n <= kSmallTokens && p.rows <= 2 * (e < p.rows ? e : p.rows) && kSmallTokens * round16(d) <= 128 * 1024;
  // CTA pairs (256-row, 256-column tiles) when an expert has rows for more than
  // two of them on average and the down product's tiles fill most of the 74
  // pairs: 2048 x 8192 without experts took 70 / 111 us for 1024 / 1536 tokens
  // on single CTAs and 80 / 93 us on pairs; 32 experts of 1024 x 1024 with 512
  // rows each 125 and 135 us.
  p.pairs = p.rows / e > 512 && (p.rows / 256) * ((d + 255) / 256) >= 40;
  p.splits = 1;
  const int64_t kb = (f + kI8BK - 1) / kI8BK;
  if (!p.pairs && !p.small) {
    // few output tiles: cut K so that about every SM (of 148) has one, at
    // least 4 blocks (512 hidden units) each, no part empty
    const int64_t groups = e < p.rows ? e : p.rows;  // experts that can have rows
    const int64_t tiles = (p.rows / kBM + groups) * ((d + DownOne::BN - 1) / DownOne::BN);
    int64_t s = tiles ? kSplitTiles / tiles : 1;
    if (s > kb / 4) s = kb / 4;
    if (s > kMaxSplits) s = kMaxSplits;
    if (s < 1) s = 1;
    const int64_t per = (kb + s - 1) / s;
    p.splits = static_cast<int>((kb + per - 1) / per);
  }
  p.combine = !p.small && (routed || p.splits > 1);
  p.ldx = round16(d);
  p.ldh = round16(f);
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  p.xq = take(static_cast<size_t>(p.rows) * p.ldx);
  p.sx = take(static_cast<size_t>(p.rows) * 4);
  p.hq = take(static_cast<size_t>(p.rows) * p.ldh);
  p.hs = take(static_cast<size_t>(p.rows) * kb * 4);
  p.z = p.combine ? take(static_cast<size_t>(p.rows) * p.splits * d * 4) : 0;
  p.total = at;
  return p;
}

// Bytes that a batch of n tokens or fewer needs, so that a program's workspace
// for its largest batch serves all: a smaller batch whose down product is split
// may keep more partial results than n tokens do.  Its tiles (128 x 128, at least
// the rows and columns of z) times its splits are at most kSplitTiles.
static size_t ffn_workspace(int64_t n, int64_t d, int64_t f, int e, int k, bool routed) {
  const FfnPlan p = ffn_plan(n, d, f, e, k, routed);
  const size_t z = p.combine ? align256(static_cast<size_t>(p.rows) * p.splits * d * 4) : 0;
  const size_t most = static_cast<size_t>(kSplitTiles) * kBM * DownOne::BN * 4;
  const size_t all = align256(static_cast<size_t>(p.rows) * kMaxSplits * d * 4);
  const size_t split = all < most ? all : most;
  return p.total - z + (z > split ? z : split);
}

struct FfnArgs {
  const void* x;
  const int8_t *wg, *wu, *wd;
  const float *sg, *su, *sd;
  const float* w;
  const int32_t *offsets, *pos;
  void* y;
  int64_t n, d, f;
  int e, k;
  uint8_t* ws;
  int32_t* diag;
  cudaStream_t st;
};

template <class Shape, class Z>
static int ffn_down(const FfnArgs& a, const FfnPlan& p, const I8Problem& pr, Z* z) {
  I8Maps m;
  const int rc = make_i8_maps<Shape>(&m, pr, reinterpret_cast<int8_t*>(a.ws + p.hq), p.ldh, a.wd, nullptr, p.ldh);
  if (rc) return rc;
  const EpiI8Down<Z> epi{z, p.rows, reinterpret_cast<float*>(a.ws + p.hs), a.sd};
  return launch_i8_gemm<Shape>(m, pr, epi, a.diag, a.st, "int8 ffn (down)");
}

template <class Shape>
static int ffn_gate_up(const FfnArgs& a, const FfnPlan& p, const I8Problem& pr) {
  I8Maps m;
  const int rc = make_i8_maps<Shape>(&m, pr, reinterpret_cast<int8_t*>(a.ws + p.xq), p.ldx, a.wg, a.wu, p.ldx);
  if (rc) return rc;
  const EpiI8Gated epi{reinterpret_cast<int8_t*>(a.ws + p.hq), p.ldh, reinterpret_cast<float*>(a.ws + p.hs), p.rows,
                       reinterpret_cast<float*>(a.ws + p.sx), a.sg, a.su};
  return launch_i8_gemm<Shape>(m, pr, epi, a.diag, a.st, "int8 ffn (gate, up)");
}

template <class T>
static int ffn_combine(const FfnArgs& a, const FfnPlan& p) {
  const dim3 grid(static_cast<unsigned>((a.n + 7) / 8), static_cast<unsigned>((a.d + 255) / 256));
  return launch_pdl(i8_combine_kernel<T>, grid, dim3(256), 0, a.st, "int8 ffn (combine)",
                    reinterpret_cast<const float*>(a.ws + p.z), static_cast<int>(p.rows), p.splits, a.n,
                    static_cast<int>(a.d), a.k, a.w, a.pos, a.offsets, a.e, static_cast<T*>(a.y));
}

template <class T>
static int ffn_small(const FfnArgs& a, const FfnPlan& p) {
  const SmallFfn s = {a.n,  static_cast<int>(a.d), static_cast<int>(a.f), a.e, a.k, p.ldx, p.ldh, a.wg, a.wu, a.wd,
                      a.sg, a.su, a.sd, a.w, a.offsets, a.pos, reinterpret_cast<int8_t*>(a.ws + p.hq),
                      reinterpret_cast<float*>(a.ws + p.hs)};
  const int nt = a.n == 1 ? 1 : a.n <= 4 ? 4 : 8;
  auto kern = nt == 1 ? i8_small_up_kernel<T, 1> : nt == 4 ? i8_small_up_kernel<T, 4> : i8_small_up_kernel<T, 8>;
  const int smem = static_cast<int>(nt * p.ldx);
  int rc = set_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (rc) return rc;
  const int64_t used = a.e < p.rows ? a.e : p.rows;  // experts that can have rows
  rc = launch_pdl(kern, dim3(static_cast<unsigned>((a.f + kHGroup - 1) / kHGroup), static_cast<unsigned>(used)),
                  dim3(512), smem, a.st, "int8 ffn (gate, up; few tokens)", static_cast<const T*>(a.x), s);
  if (rc) return rc;
  return launch_pdl(i8_small_down_kernel<T>, dim3(static_cast<unsigned>((a.d + kDownChannels - 1) / kDownChannels)),
                    dim3(512), 0, a.st, "int8 ffn (down; few tokens)", s, static_cast<T*>(a.y));
}

template <class T>
static int ffn(const FfnArgs& a, const FfnPlan& p) {
  if (p.small) return ffn_small<T>(a, p);
  int rc = launch_pdl(i8_dispatch_kernel<T>, dim3(static_cast<unsigned>((a.n + 7) / 8)), dim3(256), 0, a.st,
                      "int8 ffn (quantise)", static_cast<const T*>(a.x), a.n, static_cast<int>(a.d), a.k, a.pos,
                      static_cast<int>(p.rows), reinterpret_cast<int8_t*>(a.ws + p.xq), p.ldx,
                      reinterpret_cast<float*>(a.ws + p.sx));
  if (rc) return rc;
  const I8Problem up{static_cast<int>(p.rows), static_cast<int>(a.f), static_cast<int>(a.d), a.e, 1, a.offsets};
  const I8Problem down{static_cast<int>(p.rows), static_cast<int>(a.d), static_cast<int>(a.f), a.e, p.splits, a.offsets};
  rc = p.pairs ? ffn_gate_up<GateUpPair>(a, p, up) : ffn_gate_up<GateUpOne>(a, p, up);
  if (rc) return rc;
  if (!p.combine) {
    T* y = static_cast<T*>(a.y);
    return p.pairs ? ffn_down<DownPair>(a, p, down, y) : ffn_down<DownOne>(a, p, down, y);
  }
  float* z = reinterpret_cast<float*>(a.ws + p.z);
  rc = p.pairs ? ffn_down<DownPair>(a, p, down, z) : ffn_down<DownOne>(a, p, down, z);
  return rc ? rc : ffn_combine<T>(a, p);
}

static int check_ffn_sizes(const char* fn, int64_t n, int64_t d, int64_t f, int e, int k, int dtype) {
  if (n < 0 || d < 1 || f < 1 || e < 1 || k < 1 || k > e)
    return fail(SGE_ERR_ARG, "%s: bad sizes N=%lld d=%lld F=%lld E=%d k=%d", fn, (long long)n, (long long)d,
                (long long)f, e, k);
  if (d % 8 || f % 8) return fail(SGE_ERR_ARG, "%s: d_model and d_ff must be multiples of 8", fn);
  if (dtype != SGE_BF16 && dtype != SGE_F32) return fail(SGE_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  if (e > kMaxGroups || k > 16) return fail(SGE_ERR_UNSUPPORTED, "%s: more than %d experts, or top_k above 16", fn, kMaxGroups);
  if (d > kI8MaxK) return fail(SGE_ERR_UNSUPPORTED, "%s: d_model beyond %lld (the 32-bit sums' bound)", fn, (long long)kI8MaxK);
  if (n >= kI8MaxRows / k || f >= kI8MaxRows / e || d >= kI8MaxRows / e)
    return fail(SGE_ERR_UNSUPPORTED, "%s: size beyond 2^30", fn);
  return SGE_OK;
}

static int run_ffn(const char* fn, FfnArgs a, int dtype, bool routed, void* workspace, size_t workspace_bytes) {
  const int rc = check_ffn_sizes(fn, a.n, a.d, a.f, a.e, a.k, dtype);
  if (rc) return rc;
  if (a.n == 0) return SGE_OK;
  if (!a.x || !a.wg || !a.sg || !a.wu || !a.su || !a.wd || !a.sd || !a.y || !workspace ||
      (routed && (!a.w || !a.offsets || !a.pos)))
    return fail(SGE_ERR_ARG, "%s: null pointer", fn);
  if (!aligned16(a.x) || !aligned16(a.wg) || !aligned16(a.sg) || !aligned16(a.wu) || !aligned16(a.su) ||
      !aligned16(a.wd) || !aligned16(a.sd) || !aligned16(a.y) || !aligned16(a.w) || !aligned16(a.offsets) ||
      !aligned16(a.pos) || !aligned16(a.diag) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(SGE_ERR_ARG, "%s: pointer not 16-byte aligned (workspace: 256)", fn);
  const FfnPlan p = ffn_plan(a.n, a.d, a.f, a.e, a.k, routed);
  if (workspace_bytes < p.total)
    return fail(SGE_ERR_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, p.total);
  a.ws = static_cast<uint8_t*>(workspace);
  return dtype == SGE_BF16 ? ffn<__nv_bfloat16>(a, p) : ffn<float>(a, p);
}

}  // namespace sge

using namespace sge;

extern "C" size_t int8_ffn_workspace_bytes(int64_t n_tokens, int64_t d_model, int64_t d_ff, int n_experts, int top_k,
                                           int dtype) {
  if (check_ffn_sizes("int8_ffn_workspace_bytes", n_tokens, d_model, d_ff, n_experts, top_k, dtype)) return 0;
  // int8_ffn_fwd and moe_int8_ffn_fwd both take it
  const size_t routed = ffn_workspace(n_tokens, d_model, d_ff, n_experts, top_k, true);
  const size_t dense = ffn_workspace(n_tokens, d_model, d_ff, n_experts, top_k, false);
  return n_experts > 1 || routed > dense ? routed : dense;
}

extern "C" int int8_ffn_fwd(const void* x, const int8_t* wg_q, const float* sg, const int8_t* wu_q, const float* su,
                            const int8_t* wd_q, const float* sd, void* y, int64_t n_tokens, int64_t d_model,
                            int64_t d_ff, int dtype, void* workspace, size_t workspace_bytes, int32_t* diag,
                            void* stream) {
  NvtxRange nvtx_range("int8_ffn_fwd");
  clear_error();
  const FfnArgs a = {x, wg_q, wu_q, wd_q, sg, su, sd, nullptr, nullptr, nullptr, y, n_tokens, d_model, d_ff, 1, 1,
                     nullptr, diag, static_cast<cudaStream_t>(stream)};
  return run_ffn("int8_ffn_fwd", a, dtype, false, workspace, workspace_bytes);
}

extern "C" int moe_int8_ffn_fwd(const void* x, const int8_t* wg_q, const float* sg, const int8_t* wu_q,
                                const float* su, const int8_t* wd_q, const float* sd, const float* w,
                                const int32_t* offsets, const int32_t* pos, void* y, int64_t n_tokens,
                                int64_t d_model, int64_t d_ff, int n_experts, int top_k, int dtype, void* workspace,
                                size_t workspace_bytes, int32_t* diag, void* stream) {
  NvtxRange nvtx_range("moe_int8_ffn_fwd");
  clear_error();
  const FfnArgs a = {x, wg_q, wu_q, wd_q, sg, su, sd, w, offsets, pos, y, n_tokens, d_model, d_ff, n_experts, top_k,
                     nullptr, diag, static_cast<cudaStream_t>(stream)};
  return run_ffn("moe_int8_ffn_fwd", a, dtype, true, workspace, workspace_bytes);
}
