// Router of a mixture of feed-forward experts: top-k experts and weights of
// each token, tokens per expert, the expert-ordered list of the assignments,
// the balance loss, and the gradient.
//
//   p = softmax(logits),  ids = the k largest logits (ties: lower index)
//   w_j = p[ids_j], or renormalised over the k chosen
//   counts_e = assignments of expert e,  f_e = counts_e / sum(counts)
//   loss = E * sum_e f_e * mean over live tokens of p_e
//
// One warp per row: lane l holds the logits of experts l, l + 32, ...  The
// k largest are found by k rounds of a warp-wide maximum over order-keeping
// 32-bit keys, then the lowest index that has it, so ties are exact.  Each
// block takes a contiguous range of rows, split into contiguous ranges of its
// warps, and leaves its count and probability sum of every expert; a second
// kernel adds these over the blocks (every block for itself: at most
// kRouteBlocks values per expert from L2) and walks its rows in order,
// so an assignment's place follows from sums of integers in a fixed order
// and equals a stable sort's.  Probability sums are added in a fixed order
// too (32 bits within a block, 64 across blocks): the same bits every run.
#include "block_scan.cuh"
#include "i8_quant.cuh"
#include "sge_host.h"

namespace sge {

constexpr int kRouteThreads = 1024, kRouteWarps = 32;
constexpr int kRouteBlocks = 148;  // most blocks of a call: one per SM
constexpr int kMaxExperts = 256, kMaxTopK = 16;

struct RouteArgs {
  const uint8_t* mask;  // [n] or null
  int64_t n;
  int experts, top_k, renorm;
  int64_t rows_per_warp;
  int blocks;
  int32_t* ids;
  float* w;
  int32_t* counts;
  int32_t* offsets;
  int32_t* pos;
  int32_t* order;
  float* loss;
  int32_t* n_live;
  int32_t* part_count;  // [blocks][experts + 1]: assignments of each expert, live rows
  float* part_p;        // [blocks][experts]
};

// Keys in the order of the floats (-0 as +0).
SGE_DEV uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
SGE_DEV float key_value(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu)); }
constexpr uint32_t kKeyMinusInf = 0x007fffffu;  // order_key(-inf); smaller: taken, or no expert

SGE_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A row's logits as floats; experts past the last: -inf.
template <class T, int V>
SGE_DEV void load_logits(const T* row, int experts, int lane, float (&l)[V]) {
#pragma unroll
  for (int v = 0; v < V; ++v)
    l[v] = lane + 32 * v < experts ? to_f32(row[lane + 32 * v]) : -INFINITY;
}

// Rows of block b, warp by warp: choose, weigh, count.
template <class T, int V>
SGE_DEV void route_choose(const T* __restrict__ logits, const RouteArgs& a, int b, int* hist, float* psum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.experts, K = a.top_k;
  for (int i = threadIdx.x; i <= E; i += kRouteThreads) hist[i] = 0;
  __syncthreads();
  const int64_t first = (static_cast<int64_t>(b) * kRouteWarps + warp) * a.rows_per_warp;
  const int64_t last = first + a.rows_per_warp < a.n ? first + a.rows_per_warp : a.n;
  float p[V];
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] = 0.0f;
  int live = 0;
  for (int64_t row = first; row < last; ++row) {
    int my_id = -1;
    float my_w = 0.0f;
    if (!a.mask || a.mask[row]) {
      float l[V];
      load_logits<T, V>(logits + row * E, E, lane, l);
      uint32_t key[V];
      bool bad = false;  // a NaN or +inf among the logits
#pragma unroll
      for (int v = 0; v < V; ++v) {
        bad |= !(l[v] < INFINITY);
        key[v] = order_key(l[v]);
      }
      if (__any_sync(0xffffffffu, bad)) {
        // routed nowhere; its probabilities, and with them the loss, are NaN
        ++live;
#pragma unroll
        for (int v = 0; v < V; ++v) p[v] = __uint_as_float(0x7fffffffu);
      } else {
        uint32_t top = 0, my_key = kKeyMinusInf;
        for (int j = 0; j < K; ++j) {
          uint32_t best = 0;
          int at = 0;
#pragma unroll
          for (int v = V - 1; v >= 0; --v)
            if (key[v] >= best) {
              best = key[v];
              at = v;
            }
          const uint32_t m = __reduce_max_sync(0xffffffffu, best);
          if (j == 0) top = m;
          if (m <= kKeyMinusInf) break;  // no expert left
          const int id = __reduce_min_sync(0xffffffffu, best == m ? lane + 32 * at : 0x7fffffff);
          if (lane == j) {
            my_id = id;
            my_key = m;
          }
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (id == lane + 32 * v) key[v] = 0;
        }
        if (top > kKeyMinusInf) {
          ++live;
          const float high = key_value(top);
          float e[V], sum = 0.0f;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            e[v] = expf(l[v] - high);
            sum += e[v];
          }
          const float inv = 1.0f / warp_sum(sum);
#pragma unroll
          for (int v = 0; v < V; ++v) p[v] += e[v] * inv;
          const float mine = my_id >= 0 ? expf(key_value(my_key) - high) : 0.0f;
          my_w = a.renorm ? mine / warp_sum(mine) : mine * inv;
          if (my_id >= 0) atomicAdd(&hist[my_id], 1);
        }
      }
    }
    if (lane < K) {
      a.ids[row * K + lane] = my_id;
      a.w[row * K + lane] = my_w;
    }
  }
  if (lane == 0) atomicAdd(&hist[E], live);
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane + 32 * v < E) psum[warp * E + lane + 32 * v] = p[v];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kRouteThreads) {
    float s = 0.0f;
    for (int w = 0; w < kRouteWarps; ++w) s += psum[w * E + e];
    a.part_p[static_cast<int64_t>(b) * E + e] = s;
  }
  for (int e = threadIdx.x; e <= E; e += kRouteThreads)
    a.part_count[static_cast<int64_t>(b) * (E + 1) + e] = hist[e];
}

// Places of block b's assignments; block 0 also writes counts, offsets and
// the loss.  smem: hist [kRouteWarps][E].
SGE_DEV void route_place(const RouteArgs& a, int b, int* hist) {
  __shared__ int s_total[4][kMaxExperts + 1], s_before[4][kMaxExperts];
  __shared__ int wsum[33];
  __shared__ double s_loss[kRouteWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.experts, K = a.top_k;
  // counts of every expert over all blocks, and over the blocks before this one
  const int part = threadIdx.x >> 8, e = threadIdx.x & 255;
  for (int c = e; c <= E; c += 256) {
    int total = 0, before = 0;
#pragma unroll 8
    for (int i = part; i < a.blocks; i += 4) {
      const int v = a.part_count[static_cast<int64_t>(i) * (E + 1) + c];
      total += v;
      before += i < b ? v : 0;
    }
    s_total[part][c] = total;
    if (c < E) s_before[part][c] = before;
  }
  for (int i = threadIdx.x; i < kRouteWarps * E; i += kRouteThreads) hist[i] = 0;
  __syncthreads();
  const bool mine = threadIdx.x < E;
  int count = 0;
  if (mine)
    count = s_total[0][threadIdx.x] + s_total[1][threadIdx.x] + s_total[2][threadIdx.x] + s_total[3][threadIdx.x];
  int all;
  const int begin = block_scan_exclusive(count, wsum, &all);
  // this block's assignments, by warp and expert
  const int64_t first = (static_cast<int64_t>(b) * kRouteWarps + warp) * a.rows_per_warp;
  const int64_t last = first + a.rows_per_warp < a.n ? first + a.rows_per_warp : a.n;
  for (int64_t i = first * K + lane; i < last * K; i += 32) {
    const int id = a.ids[i];
    if (id >= 0) atomicAdd(&hist[warp * E + id], 1);
  }
  __syncthreads();
  if (mine) {
    int at = begin + s_before[0][threadIdx.x] + s_before[1][threadIdx.x] + s_before[2][threadIdx.x] +
             s_before[3][threadIdx.x];
    for (int w = 0; w < kRouteWarps; ++w) {
      const int c = hist[w * E + threadIdx.x];
      hist[w * E + threadIdx.x] = at;
      at += c;
    }
  }
  __syncthreads();
  // row by row: a row's experts are distinct, so its lanes touch distinct cells
  for (int64_t row = first; row < last; ++row) {
    if (lane < K) {
      const int64_t i = row * K + lane;
      const int id = a.ids[i];
      int at = -1;
      if (id >= 0) {
        at = hist[warp * E + id]++;
        a.order[at] = static_cast<int32_t>(i);
      }
      a.pos[i] = at;
    }
    __syncwarp();
  }
  // no assignment behind the last one
  for (int64_t i = all + static_cast<int64_t>(b) * kRouteThreads + threadIdx.x; i < a.n * K;
       i += static_cast<int64_t>(a.blocks) * kRouteThreads)
    a.order[i] = -1;
  if (b) return;
  const int live = s_total[0][E] + s_total[1][E] + s_total[2][E] + s_total[3][E];
  double term = 0.0;
  if (mine) {
    a.counts[threadIdx.x] = count;
    a.offsets[threadIdx.x] = begin;
    double p = 0.0;
    for (int i = 0; i < a.blocks; ++i) p += a.part_p[static_cast<int64_t>(i) * E + threadIdx.x];
    term = p * count;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
  if (lane == 0) s_loss[warp] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < kRouteWarps; ++w) s += s_loss[w];
    a.offsets[E] = all;
    *a.n_live = live;
    // without an assignment the sum is 0, or NaN from a row that is not finite
    *a.loss = static_cast<float>(E * s / (static_cast<double>(max(all, 1)) * max(live, 1)));
  }
}

template <class T, int V>
__global__ void __launch_bounds__(kRouteThreads, 1) route_choose_kernel(const T* logits, const RouteArgs a) {
  extern __shared__ int smem[];
  grid_dep_wait();
  grid_dep_launch();
  route_choose<T, V>(logits, a, blockIdx.x, smem, reinterpret_cast<float*>(smem + a.experts + 1));
}

__global__ void __launch_bounds__(kRouteThreads, 1) route_place_kernel(const RouteArgs a) {
  extern __shared__ int smem[];
  grid_dep_wait();
  grid_dep_launch();
  route_place(a, blockIdx.x, smem);
}

// Few rows: one block does both.
template <class T, int V>
__global__ void __launch_bounds__(kRouteThreads, 1) route_one_kernel(const T* logits, const RouteArgs a) {
  extern __shared__ int smem[];
  grid_dep_wait();
  grid_dep_launch();
  route_choose<T, V>(logits, a, 0, smem, reinterpret_cast<float*>(smem + a.experts + 1));
  __syncthreads();
  route_place(a, 0, smem);
}

// ---------------------------------------------------------------- backward

struct RouteGradArgs {
  const uint8_t* mask;
  int64_t n;
  int experts, top_k, renorm;
  const int32_t* ids;
  const float* w;
  const int32_t* counts;
  const int32_t* offsets;
  const int32_t* n_live;
  const float* dloss;
  const float* dw;
};

// dloss reaches p_e through the mean (counts are constants): dp_e = dloss * E
// * f_e / live.  Raw weights add dw_j at ids_j; then dl = p (dp - <p, dp>).
// Renormalised weights are a softmax over the chosen logits: they add
// w_j (dw_j - <w, dw>) to dl at ids_j.
template <class T, int V>
__global__ void __launch_bounds__(256) route_bwd_kernel(const T* __restrict__ logits, const RouteGradArgs a,
                                                        T* __restrict__ dlogits) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const int E = a.experts, K = a.top_k;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  float share[V];
  {
    const double live = max(*a.n_live, 1), all = max(a.offsets[E], 1);
    const double d = a.dloss ? static_cast<double>(*a.dloss) * E / (live * all) : 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v)
      share[v] = lane + 32 * v < E ? static_cast<float>(d * a.counts[lane + 32 * v]) : 0.0f;
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < a.n; row += warps) {
    float dl[V];
#pragma unroll
    for (int v = 0; v < V; ++v) dl[v] = 0.0f;
    if (!a.mask || a.mask[row]) {
      float l[V], high = -INFINITY;
      load_logits<T, V>(logits + row * E, E, lane, l);
      bool bad = false;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        bad |= !(l[v] < INFINITY);
        high = fmaxf(high, l[v]);
      }
      high = key_value(__reduce_max_sync(0xffffffffu, order_key(high)));
      if (__any_sync(0xffffffffu, bad)) {
#pragma unroll
        for (int v = 0; v < V; ++v) dl[v] = __uint_as_float(0x7fffffffu);
      } else if (high > -INFINITY) {
        float p[V], sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          p[v] = expf(l[v] - high);
          sum += p[v];
        }
        const float inv = 1.0f / warp_sum(sum);
        int id = -1;
        float g = 0.0f, w = 0.0f;
        if (lane < K && a.dw) {
          id = a.ids[row * K + lane];
          if (id >= 0) {
            g = a.dw[row * K + lane];
            w = a.w[row * K + lane];
          }
        }
        if (a.renorm) g = w * (g - warp_sum(w * g));
        float dp[V], at[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          p[v] *= inv;
          dp[v] = share[v];
          at[v] = 0.0f;
        }
        if (a.dw)
          for (int j = 0; j < K; ++j) {
            const int idj = __shfl_sync(0xffffffffu, id, j);
            const float gj = __shfl_sync(0xffffffffu, g, j);
#pragma unroll
            for (int v = 0; v < V; ++v)
              if (idj == lane + 32 * v) at[v] += gj;
          }
        float dot = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (!a.renorm) dp[v] += at[v];
          dot += p[v] * dp[v];
        }
        dot = warp_sum(dot);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          dl[v] = p[v] * (dp[v] - dot);
          if (a.renorm) dl[v] += at[v];
        }
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane + 32 * v < E) from_f32(dl[v], dlogits + row * E + lane + 32 * v);
  }
}

// ------------------------------------------------------------------- host

static int route_blocks(int64_t n) {
  const int64_t b = (n + kRouteWarps - 1) / kRouteWarps;
  return static_cast<int>(b < 1 ? 1 : b < kRouteBlocks ? b : kRouteBlocks);
}

template <class T, int V>
static int route_fwd(const void* logits, RouteArgs& a, cudaStream_t st) {
  const T* l = static_cast<const T*>(logits);
  const size_t smem = (static_cast<size_t>(kRouteWarps + 1) * a.experts + 1) * 4;
  if (a.blocks == 1) {
    const int rc = set_smem_limit(reinterpret_cast<const void*>(route_one_kernel<T, V>), static_cast<int>(smem));
    if (rc) return rc;
    return launch_pdl(route_one_kernel<T, V>, dim3(1), dim3(kRouteThreads), smem, st, "moe_route_fwd", l, a);
  }
  const int rc = launch_pdl(route_choose_kernel<T, V>, dim3(a.blocks), dim3(kRouteThreads), smem, st,
                            "moe_route_fwd (choose)", l, a);
  if (rc) return rc;
  return launch_pdl(route_place_kernel, dim3(a.blocks), dim3(kRouteThreads), smem, st, "moe_route_fwd (place)", a);
}

template <class T, int V>
static int route_bwd(const void* logits, const RouteGradArgs& a, void* dlogits, cudaStream_t st) {
  const int64_t want = (a.n + 7) / 8, most = 8 * static_cast<int64_t>(sm_count());
  return launch_pdl(route_bwd_kernel<T, V>, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(256), 0,
                    st, "moe_route_bwd", static_cast<const T*>(logits), a, static_cast<T*>(dlogits));
}

static int check_route(const char* fn, int64_t n, int experts, int top_k, int dtype) {
  if (n < 0 || experts < 1 || top_k < 1 || top_k > experts)
    return fail(SGE_ERR_ARG, "%s: bad sizes N=%lld E=%d k=%d", fn, (long long)n, experts, top_k);
  if (dtype != SGE_BF16 && dtype != SGE_F32) return fail(SGE_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
  if (experts > kMaxExperts || top_k > kMaxTopK)
    return fail(SGE_ERR_UNSUPPORTED, "%s: more than %d experts, or top_k above %d", fn, kMaxExperts, kMaxTopK);
  if (n >= (1LL << 30) / top_k) return fail(SGE_ERR_UNSUPPORTED, "%s: 2^30 assignments or more", fn);
  return SGE_OK;
}

}  // namespace sge

using namespace sge;

extern "C" size_t moe_route_workspace_bytes(int64_t n_tokens, int n_experts) {
  if (n_tokens < 0 || n_experts < 1 || n_experts > kMaxExperts) return 0;
  return align256(static_cast<size_t>(route_blocks(n_tokens)) * (2 * n_experts + 1) * 4);
}

#define SGE_ROUTE_DISPATCH(FN, T, ...)           \
  (n_experts <= 32 ? FN<T, 1>(__VA_ARGS__)       \
   : n_experts <= 64 ? FN<T, 2>(__VA_ARGS__)     \
   : n_experts <= 128 ? FN<T, 4>(__VA_ARGS__)    \
                      : FN<T, 8>(__VA_ARGS__))

extern "C" int moe_route_fwd(const void* logits, const uint8_t* mask, int64_t n_tokens, int n_experts, int top_k,
                             int renorm, int dtype, int32_t* ids, float* w, int32_t* counts, int32_t* offsets,
                             int32_t* pos, int32_t* order, float* loss, int32_t* n_live, void* workspace,
                             size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("moe_route_fwd");
  clear_error();
  const char* fn = "moe_route_fwd";
  const int rc = check_route(fn, n_tokens, n_experts, top_k, dtype);
  if (rc) return rc;
  if (!counts || !offsets || !loss || !n_live || !workspace || (n_tokens && (!logits || !ids || !w || !pos || !order)))
    return fail(SGE_ERR_ARG, "%s: null pointer", fn);
  if (!aligned16(logits) || !aligned16(mask) || !aligned16(ids) || !aligned16(w) || !aligned16(counts) ||
      !aligned16(offsets) || !aligned16(pos) || !aligned16(order) || !aligned16(loss) || !aligned16(n_live) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(SGE_ERR_ARG, "%s: pointer not 16-byte aligned (workspace: 256)", fn);
  const size_t need = moe_route_workspace_bytes(n_tokens, n_experts);
  if (workspace_bytes < need)
    return fail(SGE_ERR_ARG, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, need);
  RouteArgs a = {};
  a.mask = mask;
  a.n = n_tokens;
  a.experts = n_experts;
  a.top_k = top_k;
  a.renorm = renorm != 0;
  a.blocks = route_blocks(n_tokens);
  a.rows_per_warp = (n_tokens + a.blocks * kRouteWarps - 1) / (a.blocks * kRouteWarps);
  a.ids = ids;
  a.w = w;
  a.counts = counts;
  a.offsets = offsets;
  a.pos = pos;
  a.order = order;
  a.loss = loss;
  a.n_live = n_live;
  a.part_count = static_cast<int32_t*>(workspace);
  a.part_p = reinterpret_cast<float*>(a.part_count + static_cast<int64_t>(a.blocks) * (n_experts + 1));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SGE_BF16) return SGE_ROUTE_DISPATCH(route_fwd, __nv_bfloat16, logits, a, st);
  return SGE_ROUTE_DISPATCH(route_fwd, float, logits, a, st);
}

extern "C" int moe_route_bwd(const void* logits, const uint8_t* mask, int64_t n_tokens, int n_experts, int top_k,
                             int renorm, int dtype, const int32_t* ids, const float* w, const int32_t* counts,
                             const int32_t* offsets, const int32_t* n_live, const float* dloss, const float* dw,
                             void* dlogits, void* stream) {
  NvtxRange nvtx_range("moe_route_bwd");
  clear_error();
  const char* fn = "moe_route_bwd";
  const int rc = check_route(fn, n_tokens, n_experts, top_k, dtype);
  if (rc) return rc;
  if (n_tokens == 0) return SGE_OK;
  if (!logits || !ids || !w || !counts || !offsets || !n_live || !dlogits)
    return fail(SGE_ERR_ARG, "%s: null pointer", fn);
  if (!aligned16(logits) || !aligned16(mask) || !aligned16(ids) || !aligned16(w) || !aligned16(counts) ||
      !aligned16(offsets) || !aligned16(n_live) || !aligned16(dloss) || !aligned16(dw) || !aligned16(dlogits))
    return fail(SGE_ERR_ARG, "%s: pointer not 16-byte aligned", fn);
  const RouteGradArgs a = {mask, n_tokens, n_experts, top_k, renorm != 0, ids, w, counts, offsets, n_live, dloss, dw};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SGE_BF16) return SGE_ROUTE_DISPATCH(route_bwd, __nv_bfloat16, logits, a, dlogits, st);
  return SGE_ROUTE_DISPATCH(route_bwd, float, logits, a, dlogits, st);
}
