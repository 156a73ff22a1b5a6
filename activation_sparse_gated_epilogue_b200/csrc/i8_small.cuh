// The 8-bit operators for a few tokens: products of weight rows with a few
// vectors, bound by the bytes of the weights.  CUDA cores (four products per
// __dp4a) instead of tensor-core tiles, whose 128 rows would be mostly empty
// and whose column tiles leave SMs idle.  Integer sums, so any split of a row
// gives the same result.
#pragma once

#include "i8_gemm.cuh"
#include "i8_quant.cuh"

namespace sge {

constexpr int kSmallTokens = 8;  // of the feed-forward block, where experts leave each weight few of them
// int8_linear, weights from HBM, us for 1 / 2 / 3 / 4 tokens here and for any of
// them on the tiles: 2048 -> 64 2.6 / 3.4 / 4.2 / 4.9 and 7.5, 2048 -> 1024 3.1 /
// 3.7 / 4.5 / 5.3 and 8.6, 2560 -> 2560 4.6 / 5.1 / 6.1 / 7.1 and 9.8, 2048 -> 8192
// 4.2 / 4.9 / 9.2 / 10.9 and 9.3 (from L2 3.3 / 4.4 / 8.8 / 10.4 and 7.8).  Three
// and four tokens lose at the widest: the limit is the number that wins at all of these.
constexpr int kSmallLinear = 2;
constexpr int kHGroup = 128;  // hidden units of the feed-forward block that share a scale

SGE_DEV int dot16(const uint4& a, const uint4& b, int acc) {
  acc = __dp4a(static_cast<int>(a.x), static_cast<int>(b.x), acc);
  acc = __dp4a(static_cast<int>(a.y), static_cast<int>(b.y), acc);
  acc = __dp4a(static_cast<int>(a.z), static_cast<int>(b.z), acc);
  return __dp4a(static_cast<int>(a.w), static_cast<int>(b.w), acc);
}

// Bytes [left, 16) of v cleared (left >= 16: none).
SGE_DEV uint4 keep_bytes(uint4 v, int left) {
  const auto keep = [&](uint32_t w, int at) {
    const int n = left - at;
    return n >= 4 ? w : n <= 0 ? 0u : w & ((1u << (8 * n)) - 1u);
  };
  return make_uint4(keep(v.x, 0), keep(v.y, 4), keep(v.z, 8), keep(v.w, 12));
}

SGE_DEV uint4 load_weights(const int8_t* p) {
  uint4 v;  // read once: not worth a place in L1
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// ------------------------------------------------------------- int8_linear

// One warp per output channel, 16 bytes of its row a lane, four loads in
// flight; NT tokens' rows come from L1.  1 x 2048 -> 8192, one call after another:
// 4.2 us with the weights from HBM (4.0 TB/s), 3.3 us from L2.
template <class T, int NT>
__global__ void __launch_bounds__(256) i8_linear_small_kernel(const int8_t* __restrict__ xq, int64_t ldx,
                                                              const float* __restrict__ sx,
                                                              const int8_t* __restrict__ wq, int64_t ldw,
                                                              const float* __restrict__ sw, T* __restrict__ y,
                                                              int n, int m, int k) {
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int8_t* row = wq + static_cast<int64_t>(min(c, m - 1)) * ldw;
  // towards L2 while the kernel before (the quantiser) still runs; what is
  // read is read after the wait
  for (int b = 128 * lane; b < k; b += 128 * 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + b));
  grid_dep_wait();
  grid_dep_launch();
  if (c >= m) return;
  int acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = 0;
  constexpr int U = 4;
  for (int b0 = 16 * lane; b0 < k; b0 += 512 * U) {
    uint4 w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + 512 * u;
      w[u] = b < k ? load_weights(row + b) : make_uint4(0, 0, 0, 0);
      w[u] = keep_bytes(w[u], k - b);  // bytes past the row are no part of it
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + 512 * u;
      if (b < k)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          if (t < n) acc[t] = dot16(w[u], __ldg(reinterpret_cast<const uint4*>(xq + t * ldx + b)), acc[t]);
    }
  }
  const float s = __ldg(sw + c);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int sum = __reduce_add_sync(0xffffffffu, acc[t]);
    if (t < n && lane == t) from_f32(__int2float_rn(sum) * __ldg(sx + t) * s, y + static_cast<int64_t>(t) * m + c);
  }
}

// ------------------------------------------------------ feed-forward block

struct SmallFfn {
  int64_t n;
  int d, f, experts, k;
  int64_t ldx, ldh;
  const int8_t *wg, *wu, *wd;
  const float *sg, *su, *sd;
  const float* w;            // [n][k], or null (one block for all)
  const int32_t* offsets;    // [experts + 1], or null
  const int32_t* pos;        // [n][k], or null
  int8_t* hq;                // [n * k][ldh]
  float* hs;                 // [groups of 128][n * k]
};

constexpr int kSmallRows = kSmallTokens * 16;  // places of at most kSmallTokens tokens

// The experts' row bounds, as the tile engine makes them (out of range or out of
// order they give fewer rows, never an overlap), and the experts that have rows,
// in order (any block size; experts <= 256, rows <= 128): expert e has the rows
// [bounds[e], bounds[e + 1]), so at most min(experts, rows) have any.  Returns
// their number.  list: experts bytes; bounds: experts + 1 bytes; scratch: 8 ints.
SGE_DEV int used_experts(const SmallFfn& a, int rows, uint8_t* list, uint8_t* bounds, int* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = threadIdx.x;
  int lo = 0, hi = 0;
  if (e < a.experts) {
    lo = a.offsets ? checked_bound(a.offsets[e], 0, rows) : 0;
    hi = a.offsets ? checked_bound(a.offsets[e + 1], 0, rows) : rows;
    bounds[e] = static_cast<uint8_t>(lo);
    if (e == a.experts - 1) bounds[a.experts] = static_cast<uint8_t>(hi);
  }
  // scratch[w]: warp w's used experts, and a high bit if its bounds descend
  // somewhere (a route's do not: a scan for everyone took 0.5 us of each kernel's 10)
  constexpr int DESCENDS = 1 << 16;
  uint32_t mask = __ballot_sync(0xffffffffu, hi > lo);
  const uint32_t down = __ballot_sync(0xffffffffu, hi < lo);
  if (lane == 0 && warp < 8) scratch[warp] = __popc(mask) | (down ? DESCENDS : 0);
  __syncthreads();
  const auto count = [&](int& before) {
    int all = 0;
    before = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += scratch[w];
      all += scratch[w];
    }
    return all;
  };
  int before, all = count(before);
  if (all >= DESCENDS) {
    __syncthreads();
    if (warp == 0) {  // each bound becomes the largest up to it
      int top = 0;
      for (int i0 = 0; i0 <= a.experts; i0 += 32) {
        int v = i0 + lane <= a.experts ? max(static_cast<int>(bounds[i0 + lane]), top) : top;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v = max(v, u);
        }
        if (i0 + lane <= a.experts) bounds[i0 + lane] = static_cast<uint8_t>(v);
        top = __shfl_sync(0xffffffffu, v, 31);
      }
    }
    __syncthreads();
    if (e < a.experts) {
      lo = bounds[e];
      hi = bounds[e + 1];
    }
    mask = __ballot_sync(0xffffffffu, hi > lo);
    if (lane == 0 && warp < 8) scratch[warp] = __popc(mask);
    __syncthreads();
    all = count(before);
  }
  if (hi > lo) list[before + __popc(mask & ((1u << lane) - 1u))] = static_cast<uint8_t>(e);
  __syncthreads();
  return all;
}

// Gate and up projections, h and its quantisation: one block per used expert
// and group of 128 hidden units, 16 warps of 8 units.  The block quantises its
// tokens' rows itself (a launch less).  NT: rows of an expert at a time.  With
// the kernel below 19.8 us for one token of 2048 x 8192 (50 MB of weights) with the
// weights from HBM, 18.1 from L2; 11.4 and 10.6 us for one over four of 32 experts
// of 1024 x 1024.
template <class T, int NT>
__global__ void __launch_bounds__(512, 1) i8_small_up_kernel(const T* __restrict__ x, const SmallFfn a) {
  extern __shared__ __align__(16) int8_t s_x[];  // [NT][ldx]
  __shared__ __align__(16) float s_h[NT][kHGroup];  // read in 16-byte pieces
  __shared__ float s_scale[NT];
  __shared__ int s_scratch[8], s_token[kSmallRows];
  __shared__ uint8_t s_list[kMaxGroups], s_bounds[kMaxGroups + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = static_cast<int>(a.n) * a.k;
  const int group = blockIdx.x, u0 = group * kHGroup;
  grid_dep_wait();
  grid_dep_launch();
  for (int i = threadIdx.x; i < rows; i += 512) s_token[i] = a.pos ? -1 : i;
  const int used = used_experts(a, rows, s_list, s_bounds, s_scratch);
  if (blockIdx.y >= used) return;
  const int e = s_list[blockIdx.y];
  const int lo = s_bounds[e], hi = s_bounds[e + 1];
  if (a.pos) {
    for (int i = threadIdx.x; i < rows; i += 512) {
      const uint32_t p = checked_place(a.pos[i], rows);
      if (p < static_cast<uint32_t>(rows)) s_token[p] = i / a.k;
    }
    __syncthreads();
  }
  const int8_t* wg = a.wg + (static_cast<int64_t>(e) * a.f + u0) * a.ldx;
  const int8_t* wu = a.wu + (static_cast<int64_t>(e) * a.f + u0) * a.ldx;
  const int units = min(kHGroup, a.f - u0);
  if (threadIdx.x < 2)  // the block's weights on their way to L2 while its tokens are quantised
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(threadIdx.x ? wu : wg),
                 "r"(static_cast<uint32_t>(units * a.ldx))
                 : "memory");
  for (int r0 = lo; r0 < hi; r0 += NT) {
    const int nr = min(NT, hi - r0);
    if (warp < nr) {
      // a place that no token names holds nothing
      const int token = s_token[r0 + warp];
      uint32_t amax = 0;
      int8_t* dst = s_x + warp * a.ldx;
      if (token >= 0)
        quant_row<T, true, 4>(x + static_cast<int64_t>(token) * a.d, a.d, lane, amax,
                              [&](int c, const auto& v, float inv) { store_q(dst + c, v, inv); });
      else
        for (int c = 16 * lane; c < a.ldx; c += 512) *reinterpret_cast<uint4*>(dst + c) = make_uint4(0, 0, 0, 0);
      if (lane == 0) s_scale[warp] = quant_scale(amax).scale;
      if (lane == 1 && a.d % 16) *reinterpret_cast<uint2*>(dst + a.d) = make_uint2(0, 0);
    }
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      const int j0 = warp * 8 + pass * 4;  // four units: eight weight rows
      int g[4][NT], u[4][NT];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) g[i][t] = u[i][t] = 0;
#pragma unroll 1
      for (int b = 16 * lane; b < a.ldx; b += 512) {
        uint4 vg[4], vu[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t at = static_cast<int64_t>(min(j0 + i, units - 1)) * a.ldx + b;
          vg[i] = load_weights(wg + at);
          vu[i] = load_weights(wu + at);
        }
        // bytes of a weight row past d meet zeros
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if (t >= nr) break;
          const uint4 xv = *reinterpret_cast<const uint4*>(s_x + t * a.ldx + b);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            g[i][t] = dot16(vg[i], xv, g[i][t]);
            u[i][t] = dot16(vu[i], xv, u[i][t]);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t >= nr) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int sum_g = __reduce_add_sync(0xffffffffu, g[i][t]);
          const int sum_u = __reduce_add_sync(0xffffffffu, u[i][t]);
          if (lane == i) {
            const int j = j0 + i;
            float h = 0.0f;
            if (j < units) {
              const int64_t c = static_cast<int64_t>(e) * a.f + u0 + j;
              const float gv = __int2float_rn(sum_g) * s_scale[t] * __ldg(a.sg + c);
              const float uv = __int2float_rn(sum_u) * s_scale[t] * __ldg(a.su + c);
              h = (gv < 0.0f ? 0.0f : gv) * uv;
            }
            s_h[t][j] = h;
          }
        }
      }
    }
    __syncthreads();
    if (warp < nr) {
      const float4 h = *reinterpret_cast<const float4*>(&s_h[warp][4 * lane]);
      const uint32_t amax = __reduce_max_sync(
          0xffffffffu, max(max(abs_bits(h.x), abs_bits(h.y)), max(abs_bits(h.z), abs_bits(h.w))));
      const QuantScale qs = quant_scale(amax);
      if (u0 + 4 * lane < a.ldh)
        *reinterpret_cast<uint32_t*>(a.hq + static_cast<int64_t>(r0 + warp) * a.ldh + u0 + 4 * lane) =
            quant_pack4(h.x, h.y, h.z, h.w, qs.inv);
      if (lane == 0) a.hs[static_cast<int64_t>(group) * rows + r0 + warp] = qs.scale;
    }
    __syncthreads();
  }
}

// Down projection and the weighted sum over a token's experts: one block per
// four output channels; a channel's weights (its row of every used expert, in
// pieces of 2 KB) are dealt to four warps.  Every warp adds its pieces' sums
// for each token in order, the four warps' sums are added in order.
constexpr int kDownChannels = 4, kDownSlices = 4, kDownPiece = 2048;

template <class T>
__global__ void __launch_bounds__(512) i8_small_down_kernel(const SmallFfn a, T* __restrict__ y) {
  __shared__ float s_sum[kDownSlices][kDownChannels][kSmallTokens];
  __shared__ int s_scratch[8], s_token[kSmallRows];
  __shared__ uint8_t s_list[kMaxGroups], s_bounds[kMaxGroups + 1];
  __shared__ float s_w[kSmallRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = warp % kDownChannels, slice = warp / kDownChannels;
  const int rows = static_cast<int>(a.n) * a.k;
  const int c = blockIdx.x * kDownChannels + ch;
  grid_dep_wait();
  grid_dep_launch();
  if (threadIdx.x < kDownSlices * kDownChannels * kSmallTokens) (&s_sum[0][0][0])[threadIdx.x] = 0.0f;
  for (int i = threadIdx.x; i < rows; i += 512) {
    s_token[i] = a.pos ? -1 : i;
    s_w[i] = a.pos ? 0.0f : 1.0f;
  }
  const int used = used_experts(a, rows, s_list, s_bounds, s_scratch);
  if (a.pos) {
    for (int i = threadIdx.x; i < rows; i += 512) {
      const uint32_t p = checked_place(a.pos[i], rows);
      if (p < static_cast<uint32_t>(rows)) {
        s_token[p] = i / a.k;
        s_w[p] = a.w[i];
      }
    }
    __syncthreads();
  }
  const int pieces = (a.f + kDownPiece - 1) / kDownPiece;
  if (c < a.d)
    for (int item = slice; item < used * pieces; item += kDownSlices) {
      const int e = s_list[item / pieces], b0 = item % pieces * kDownPiece + 16 * lane;
      const int8_t* row = a.wd + (static_cast<int64_t>(e) * a.d + c) * a.ldh;
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = b0 + 512 * i < a.f ? load_weights(row + b0 + 512 * i) : make_uint4(0, 0, 0, 0);
      const float sd = __ldg(a.sd + static_cast<int64_t>(e) * a.d + c);
      const int lo = s_bounds[e], hi = s_bounds[e + 1];
      for (int r = lo; r < hi; ++r) {
        const int token = s_token[r];
        float part = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int b = b0 + 512 * i;
          if (b < a.f) {
            // bytes of a weight row past f meet zeros of hq
            const uint4 h = __ldg(reinterpret_cast<const uint4*>(a.hq + static_cast<int64_t>(r) * a.ldh + b));
            const float hs = __ldg(a.hs + static_cast<int64_t>(b / kHGroup) * rows + r);
            part = fmaf(__int2float_rn(dot16(v[i], h, 0)), hs, part);
          }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        if (lane == 0 && token >= 0) s_sum[slice][ch][token] = fmaf(s_w[r], part * sd, s_sum[slice][ch][token]);
      }
    }
  __syncthreads();
  if (threadIdx.x < kDownChannels * kSmallTokens) {
    const int t = threadIdx.x / kDownChannels, j = threadIdx.x % kDownChannels;
    const int col = blockIdx.x * kDownChannels + j;
    if (t < a.n && col < a.d) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kDownSlices; ++i) s += s_sum[i][j][t];
      from_f32(s, y + static_cast<int64_t>(t) * a.d + col);
    }
  }
}

}  // namespace sge
