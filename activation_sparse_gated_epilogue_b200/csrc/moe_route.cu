// Router of a mixture of feed-forward experts: top-k experts and weights of
// each token, tokens per expert, the expert-ordered list of the assignments,
// the balance loss, and the gradient.
//
//   p = softmax(logits),  ids = the k largest logits (ties: lower index)
//   w_j = p[ids_j], or renormalised over the k chosen
//   counts_e = assignments of expert e,  f_e = counts_e / sum(counts)
//   loss = E * sum_e f_e * mean over live tokens of p_e
//
// One warp per row: lane l holds the logits of experts l * V .. l * V + V - 1.
// The k largest are found by k rounds of a warp-wide maximum over order-keeping
// 32-bit keys, of which the lowest lane (the lowest index) gives its first, so
// ties are exact.  Each
// block takes a contiguous range of rows, split into contiguous ranges of its
// warps, and leaves its count and probability sum of every expert; a second
// kernel adds these over the blocks (every block for itself: at most
// kRouteBlocks values per expert from L2) and walks its rows in order,
// so an assignment's place follows from sums of integers in a fixed order
// and equals a stable sort's.  Probability sums are added in a fixed order
// too (32 bits over at most kFoldRows rows and within a block, 64 beyond): the
// same bits every run.
// Latency bounds small batches (one token of 64 experts: 6.0 us, ten block
// barriers), instructions large ones (16384 x 256 bf16, k = 8, call after call: 24.4
// us, about 560 instructions a row to choose; the gradient 9.2 us).
#include "block_scan.cuh"
#include "i8_quant.cuh"
#include "sge_host.h"

namespace sge {

constexpr int kRouteThreads = 1024, kRouteWarps = 32;
constexpr int kRouteBlocks = 148;  // most blocks of a call: one per SM
constexpr int kMaxExperts = 256, kMaxTopK = 16;
// Rows whose probabilities a warp adds in 32 bits: longer runs (more than 64 *
// 32 * 148 tokens) go to 64-bit sums in shared memory every so many rows.  A
// warp's 3543 rows of 16777216 tokens alone were off by 588 roundings.
constexpr int kFoldRows = 64;

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

// V consecutive values of a row from expert lane * V on, as floats; experts past
// the last: -inf.  VEC: E is a multiple of V, so that a lane's values are all
// there or all past the end, and aligned.
template <class T, int V, bool VEC>
SGE_DEV void load_logits(const T* row, int experts, int lane, float (&l)[V]) {
  const int e = lane * V;
  if constexpr (VEC) {
    constexpr int BYTES = V * static_cast<int>(sizeof(T));
    constexpr int UNIT = BYTES >= 16 ? 16 : BYTES;  // bytes of one load
    constexpr int PER = UNIT / static_cast<int>(sizeof(T));
    struct alignas(UNIT) Pack {
      T v[PER];
    };
#pragma unroll
    for (int u = 0; u < V / PER; ++u) {
      Pack p;
      if (e < experts) p = reinterpret_cast<const Pack*>(row + e)[u];
#pragma unroll
      for (int i = 0; i < PER; ++i) l[u * PER + i] = e < experts ? to_f32(p.v[i]) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = e + v < experts ? to_f32(row[e + v]) : -INFINITY;
  }
}
template <class T, int V, bool VEC>
SGE_DEV void store_logits(T* row, int experts, int lane, const float (&l)[V]) {
  const int e = lane * V;
  if constexpr (VEC) {
    constexpr int BYTES = V * static_cast<int>(sizeof(T));
    constexpr int UNIT = BYTES >= 16 ? 16 : BYTES;
    constexpr int PER = UNIT / static_cast<int>(sizeof(T));
    struct alignas(UNIT) Pack {
      T v[PER];
    };
    if (e >= experts) return;
#pragma unroll
    for (int u = 0; u < V / PER; ++u) {
      Pack p;
#pragma unroll
      for (int i = 0; i < PER; ++i) from_f32(l[u * PER + i], &p.v[i]);
      reinterpret_cast<Pack*>(row + e)[u] = p;
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e + v < experts) from_f32(l[v], row + e + v);
  }
}

// Sorts a lane's V keys, largest first (V = 1, 2, 4, 8: Batcher's networks).
SGE_DEV void sort2(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
template <int V>
SGE_DEV void sort_keys(uint32_t (&k)[V]) {
  if constexpr (V == 2) sort2(k[0], k[1]);
  if constexpr (V >= 4) {
#pragma unroll
    for (int h = 0; h < V; h += 4) {
      sort2(k[h], k[h + 1]);
      sort2(k[h + 2], k[h + 3]);
      sort2(k[h], k[h + 2]);
      sort2(k[h + 1], k[h + 3]);
      sort2(k[h + 1], k[h + 2]);
    }
  }
  if constexpr (V == 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sort2(k[i], k[i + 4]);
    sort2(k[2], k[4]);
    sort2(k[3], k[5]);
    sort2(k[1], k[2]);
    sort2(k[3], k[4]);
    sort2(k[5], k[6]);
  }
}

// The K largest of a row's values l: lane j < K gets the j-th one's expert and
// value (-1 where no expert is left); returns the largest value's key.
template <class T, int V>
SGE_DEV uint32_t top_k(const float (&l)[V], int K, int lane, int& my_id, float& my_value) {
  uint32_t key[V], top = 0;
  if constexpr (sizeof(T) == 2) {
    // A bf16 leaves the low half of its key free for the expert, so one
    // maximum finds value and index (complemented: ties go to the lower one),
    // and with a lane's keys sorted taking one is a shift: E = 256, k = 8 took
    // 1.6 times as long as with the general form below.
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = (order_key(l[v]) & 0xffff0000u) | (0xffffu - (lane * V + v));
    sort_keys<V>(key);
    uint32_t mine = 0;
    for (int j = 0; j < K; ++j) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, key[0]);
      if (j == 0) top = m;
      if ((m | 0xffffu) <= kKeyMinusInf) break;  // no expert left
      if (lane == j) mine = m;
      if (key[0] == m) {
#pragma unroll
        for (int v = 0; v + 1 < V; ++v) key[v] = key[v + 1];
        key[V - 1] = 0;
      }
    }
    if (mine) {
      my_id = static_cast<int>(0xffffu - (mine & 0xffffu));
      // the value's own bits: the low half of a bf16's pattern is zero (ones
      // in the key of a negative number)
      my_value = key_value((mine & 0x80000000u) ? (mine & 0xffff0000u) : (mine | 0xffffu));
    }
    return (top & 0x80000000u) ? (top & 0xffff0000u) : (top | 0xffffu);
  } else {
    uint32_t best = 0, my_key = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      key[v] = order_key(l[v]);
      best = max(best, key[v]);
    }
    for (int j = 0; j < K; ++j) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, best);
      if (j == 0) top = m;
      if (m <= kKeyMinusInf) break;  // no expert left
      const int owner = __ffs(__ballot_sync(0xffffffffu, best == m)) - 1;
      // the owner's first value equal to m is taken; its best is then the
      // largest that is left
      int at = 0;
      if (lane == owner) {
        best = 0;
        bool taken = false;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const bool here = key[v] == m && !taken;
          if (here) at = v;
          taken |= here;
          key[v] = here ? 0 : key[v];
          best = max(best, key[v]);
        }
      }
      const int id = owner * V + __shfl_sync(0xffffffffu, at, owner);
      if (lane == j) {
        my_id = id;
        my_key = m;
      }
    }
    if (my_key) my_value = key_value(my_key);
    return top;
  }
}

// Rows of block b, warp by warp: choose, weigh, count.  psum: [kRouteWarps][E];
// wide: the same in 64 bits, or null where no warp has more than kFoldRows rows.
template <class T, int V, bool VEC>
SGE_DEV void route_choose(const T* __restrict__ logits, const RouteArgs& a, int b, int* hist, float* psum,
                          double* wide) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.experts, K = a.top_k;
  const int64_t first = (static_cast<int64_t>(b) * kRouteWarps + warp) * a.rows_per_warp;
  const int64_t last = first + a.rows_per_warp < a.n ? first + a.rows_per_warp : a.n;
  float next[V];
  int next_live = 0;
  const auto fetch = [&](int64_t row) {
    if (row >= last) return;
    next_live = a.mask ? a.mask[row] : 1;
    load_logits<T, V, VEC>(logits + row * E, E, lane, next);
  };
  fetch(first);
  for (int i = threadIdx.x; i <= E; i += kRouteThreads) hist[i] = 0;
  __syncthreads();
  float p[V];
#pragma unroll
  for (int v = 0; v < V; ++v) p[v] = 0.0f;
  const auto fold = [&](bool start) {  // a lane's cells are its own
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (lane * V + v >= E) continue;
      double* cell = wide + warp * E + lane * V + v;
      *cell = start ? 0.0 : *cell + p[v];
      p[v] = 0.0f;
    }
  };
  if (wide) fold(true);
  int live = 0, run = 0;
  for (int64_t row = first; row < last; ++row) {
    if (wide && run++ == kFoldRows) {
      fold(false);
      run = 1;
    }
    float l[V];
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = next[v];
    const bool is_live = next_live != 0;
    fetch(row + 1);  // in flight while this row is worked on
    int my_id = -1;
    float my_w = 0.0f;
    if (is_live) {
      bool bad = false;  // a NaN or +inf among the logits
#pragma unroll
      for (int v = 0; v < V; ++v) bad |= !(l[v] < INFINITY);
      if (__any_sync(0xffffffffu, bad)) {
        // routed nowhere; its probabilities, and with them the loss, are NaN
        ++live;
#pragma unroll
        for (int v = 0; v < V; ++v) p[v] = __uint_as_float(0x7fffffffu);
      } else {
        float my_value = 0.0f;
        const uint32_t top = top_k<T, V>(l, K, lane, my_id, my_value);
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
          const float mine = my_id >= 0 ? expf(my_value - high) : 0.0f;
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
  if (wide) fold(false);
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane * V + v < E) psum[warp * E + lane * V + v] = p[v];
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kRouteThreads) {
    float s = 0.0f;
    if (wide) {
      double d = 0.0;
      for (int w = 0; w < kRouteWarps; ++w) d += wide[w * E + e];
      s = static_cast<float>(d);
    } else {
      for (int w = 0; w < kRouteWarps; ++w) s += psum[w * E + e];
    }
    a.part_p[static_cast<int64_t>(b) * E + e] = s;
  }
  for (int e = threadIdx.x; e <= E; e += kRouteThreads)
    a.part_count[static_cast<int64_t>(b) * (E + 1) + e] = hist[e];
}

// Places of block b's assignments; block 0 also writes counts, offsets and
// the loss.  smem: hist [kRouteWarps][E + 1] (the odd pitch keeps a column's
// cells in different banks).
SGE_DEV void route_place(const RouteArgs& a, int b, int* hist) {
  __shared__ int s_total[4][kMaxExperts], s_before[4][kMaxExperts], s_live;
  __shared__ double s_p[4][kMaxExperts];
  __shared__ int s_at[kMaxExperts];
  __shared__ int wsum[33];
  __shared__ double s_loss[kRouteWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.experts, K = a.top_k, pitch = E + 1;
  // this block's ids: a lane's of its warp's first rows stay in registers
  const int64_t first = (static_cast<int64_t>(b) * kRouteWarps + warp) * a.rows_per_warp;
  const int64_t last = first + a.rows_per_warp < a.n ? first + a.rows_per_warp : a.n;
  constexpr int KEEP = 4;
  int kept[KEEP];
#pragma unroll
  for (int r = 0; r < KEEP; ++r) kept[r] = lane < K && first + r < last ? a.ids[(first + r) * K + lane] : -1;
  // counts of every expert over all blocks, and over the blocks before this
  // one, in four parts (every fourth block), loads in batches
  const int part = threadIdx.x >> 8, e = threadIdx.x & 255;
  constexpr int BATCH = 19;  // half of a part of kRouteBlocks
  if (e < E) {
    int total = 0, before = 0;
    for (int i0 = part; i0 < a.blocks; i0 += 4 * BATCH) {
      const int32_t* src = a.part_count + i0 * (E + 1) + e;  // at most kRouteBlocks * 257: 32 bits do
      int v[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) v[i] = i0 + 4 * i < a.blocks ? src[i * 4 * (E + 1)] : 0;
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        total += v[i];
        before += i0 + 4 * i < b ? v[i] : 0;
      }
    }
    s_total[part][e] = total;
    s_before[part][e] = before;
  }
  if (b == 0 && e < E) {
    double p = 0.0;
    for (int i0 = part; i0 < a.blocks; i0 += 4 * BATCH) {
      const float* src = a.part_p + i0 * E + e;
      float v[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) v[i] = i0 + 4 * i < a.blocks ? src[i * 4 * E] : 0.0f;
#pragma unroll
      for (int i = 0; i < BATCH; ++i) p += v[i];
    }
    s_p[part][e] = p;
  }
  const int block_live =
      b == 0 && threadIdx.x < a.blocks ? a.part_count[static_cast<int64_t>(threadIdx.x) * (E + 1) + E] : 0;
  if (threadIdx.x == 0) s_live = 0;
  for (int i = threadIdx.x; i < kRouteWarps * pitch; i += kRouteThreads) hist[i] = 0;
  __syncthreads();
  if (block_live) atomicAdd(&s_live, block_live);
  const bool mine = threadIdx.x < E;
  int count = 0;
  if (mine)
    count = s_total[0][threadIdx.x] + s_total[1][threadIdx.x] + s_total[2][threadIdx.x] + s_total[3][threadIdx.x];
#pragma unroll
  for (int r = 0; r < KEEP; ++r)
    if (kept[r] >= 0) atomicAdd(&hist[warp * pitch + kept[r]], 1);
  for (int64_t i = (first + KEEP) * K + lane; i < last * K; i += 32) {
    const int id = a.ids[i];
    if (id >= 0) atomicAdd(&hist[warp * pitch + id], 1);
  }
  int all;
  const int begin = block_scan_exclusive(count, wsum, &all);
  if (mine)
    s_at[threadIdx.x] = begin + s_before[0][threadIdx.x] + s_before[1][threadIdx.x] + s_before[2][threadIdx.x] +
                        s_before[3][threadIdx.x];
  __syncthreads();
  // where each warp's assignments of an expert begin: one warp per expert, a
  // lane per warp, a prefix sum over the lanes
  for (int c = warp; c < E; c += kRouteWarps) {
    const int n = hist[lane * pitch + c];
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    hist[lane * pitch + c] = s_at[c] + incl - n;
  }
  __syncthreads();
  // row by row: a row's experts are distinct, so its lanes touch distinct cells
  const auto place = [&](int64_t row, int id) {
    if (lane < K) {
      const int64_t i = row * K + lane;
      int at = -1;
      if (id >= 0) {
        at = hist[warp * pitch + id]++;
        a.order[at] = static_cast<int32_t>(i);
      }
      a.pos[i] = at;
    }
    __syncwarp();
  };
#pragma unroll
  for (int r = 0; r < KEEP; ++r)
    if (first + r < last) place(first + r, kept[r]);
  for (int64_t row = first + KEEP; row < last; ++row) place(row, lane < K ? a.ids[row * K + lane] : -1);
  // no assignment behind the last one
  for (int64_t i = all + static_cast<int64_t>(b) * kRouteThreads + threadIdx.x; i < a.n * K;
       i += static_cast<int64_t>(a.blocks) * kRouteThreads)
    a.order[i] = -1;
  if (b) return;
  const int live = s_live;
  double term = 0.0;
  if (mine) {
    a.counts[threadIdx.x] = count;
    a.offsets[threadIdx.x] = begin;
    term = ((s_p[0][threadIdx.x] + s_p[1][threadIdx.x]) + (s_p[2][threadIdx.x] + s_p[3][threadIdx.x])) * count;
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

// Shared words of a block: counts and sums, or the places' [kRouteWarps][E + 1];
// even, so that 64-bit sums may follow.
__host__ __device__ constexpr int route_words(int experts) { return ((kRouteWarps + 1) * (experts + 1) + 1) & ~1; }

template <class T, int V, bool VEC>
__global__ void __launch_bounds__(kRouteThreads, 1) route_choose_kernel(const T* logits, const RouteArgs a) {
  extern __shared__ __align__(16) int smem[];
  grid_dep_wait();
  grid_dep_launch();
  float* psum = reinterpret_cast<float*>(smem + a.experts + 1);
  double* wide = reinterpret_cast<double*>(smem + route_words(a.experts));
  route_choose<T, V, VEC>(logits, a, blockIdx.x, smem, psum, a.rows_per_warp > kFoldRows ? wide : nullptr);
}

__global__ void __launch_bounds__(kRouteThreads, 1) route_place_kernel(const RouteArgs a) {
  extern __shared__ __align__(16) int smem[];
  grid_dep_wait();
  grid_dep_launch();
  route_place(a, blockIdx.x, smem);
}

// Few rows: one block does both, its counts and sums stay in shared memory.
template <class T, int V, bool VEC>
__global__ void __launch_bounds__(kRouteThreads, 1) route_one_kernel(const T* logits, const RouteArgs args) {
  extern __shared__ __align__(16) int smem[];
  __shared__ int s_count[kMaxExperts + 1];
  __shared__ float s_sum[kMaxExperts];
  RouteArgs a = args;
  a.part_count = s_count;
  a.part_p = s_sum;
  grid_dep_wait();
  grid_dep_launch();
  route_choose<T, V, VEC>(logits, a, 0, smem, reinterpret_cast<float*>(smem + a.experts + 1), nullptr);
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
template <class T, int V, bool VEC>
__global__ void __launch_bounds__(256) route_bwd_kernel(const T* __restrict__ logits, const RouteGradArgs a,
                                                        T* __restrict__ dlogits) {
  // per warp: what the weights' gradient adds at each of a row's experts
  __shared__ __align__(16) float s_at[8][32 * V];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  float* row_at = s_at[threadIdx.x >> 5];
  const int E = a.experts, K = a.top_k;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  float share[V];
  {
    const float live = __int2float_rn(max(*a.n_live, 1)), all = __int2float_rn(max(a.offsets[E], 1));
    const float d = a.dloss ? *a.dloss * E / live / all : 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
      share[v] = lane * V + v < E ? d * __int2float_rn(a.counts[lane * V + v]) : 0.0f;
  }
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < a.n; row += warps) {
    float dl[V], l[V];
    load_logits<T, V, VEC>(logits + row * E, E, lane, l);
    int id = -1;
    float g = 0.0f, w = 0.0f;
    if (lane < K && a.dw) {
      id = a.ids[row * K + lane];
      g = a.dw[row * K + lane];
      w = a.w[row * K + lane];
    }
    if (id < 0) g = w = 0.0f;  // whatever dw holds there
#pragma unroll
    for (int v = 0; v < V; ++v) dl[v] = 0.0f;
    if (!a.mask || a.mask[row]) {
      float high = -INFINITY;
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
        if (a.renorm) g = w * (g - warp_sum(w * g));
        float dp[V], at[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          p[v] *= inv;
          dp[v] = share[v];
          at[v] = 0.0f;
        }
        if (a.dw) {
          // a row's experts are distinct: its lanes write distinct cells
#pragma unroll
          for (int v = 0; v < V; ++v) row_at[lane * V + v] = 0.0f;
          __syncwarp();
          if (checked_place(id, E) < static_cast<uint32_t>(E)) row_at[id] = g;
          __syncwarp();
#pragma unroll
          for (int v = 0; v < V; ++v) at[v] = row_at[lane * V + v];
          __syncwarp();
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
    store_logits<T, V, VEC>(dlogits + row * E, E, lane, dl);
  }
}

// ------------------------------------------------------------------- host

static int route_blocks(int64_t n) {
  const int64_t b = (n + kRouteWarps - 1) / kRouteWarps;
  return static_cast<int>(b < 1 ? 1 : b < kRouteBlocks ? b : kRouteBlocks);
}

template <class T, int V, bool VEC>
static int route_fwd_as(const void* logits, RouteArgs& a, cudaStream_t st) {
  const T* l = static_cast<const T*>(logits);
  const size_t smem = static_cast<size_t>(route_words(a.experts)) * 4;
  const void* last = a.blocks == 1 ? reinterpret_cast<const void*>(route_one_kernel<T, V, VEC>)
                                   : reinterpret_cast<const void*>(route_place_kernel);
  int rc = set_smem_limit(last, static_cast<int>(smem));  // with its static share it may pass 48 KB
  if (rc) return rc;
  if (a.blocks == 1)
    return launch_pdl(route_one_kernel<T, V, VEC>, dim3(1), dim3(kRouteThreads), smem, st, "moe_route_fwd", l, a);
  size_t choose_smem = smem;
  if (a.rows_per_warp > kFoldRows) {
    choose_smem += static_cast<size_t>(kRouteWarps) * a.experts * 8;
    rc = set_smem_limit(reinterpret_cast<const void*>(route_choose_kernel<T, V, VEC>), static_cast<int>(choose_smem));
    if (rc) return rc;
  }
  rc = launch_pdl(route_choose_kernel<T, V, VEC>, dim3(a.blocks), dim3(kRouteThreads), choose_smem, st,
                  "moe_route_fwd (choose)", l, a);
  if (rc) return rc;
  return launch_pdl(route_place_kernel, dim3(a.blocks), dim3(kRouteThreads), smem, st, "moe_route_fwd (place)", a);
}

template <class T, int V>
static int route_fwd(const void* logits, RouteArgs& a, cudaStream_t st) {
  return a.experts % V == 0 ? route_fwd_as<T, V, true>(logits, a, st) : route_fwd_as<T, V, false>(logits, a, st);
}

template <class T, int V>
static int route_bwd(const void* logits, const RouteGradArgs& a, void* dlogits, cudaStream_t st) {
  const int64_t want = (a.n + 7) / 8, most = 8 * static_cast<int64_t>(sm_count());
  auto kern = a.experts % V == 0 ? route_bwd_kernel<T, V, true> : route_bwd_kernel<T, V, false>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(256), 0, st, "moe_route_bwd",
                    static_cast<const T*>(logits), a, static_cast<T*>(dlogits));
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
