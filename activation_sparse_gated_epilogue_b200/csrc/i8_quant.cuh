// Symmetric 8-bit quantisation with one scale per row (or group):
//   amax = max |x|,  scale = amax / 127,  q = rint(x * (127 / amax))
// each operation in 32-bit floats, rounded to nearest even, so that every
// kernel that quantises (and any restatement of it) gives the same integers.
#pragma once

#include "debug_checks.cuh"
#include "sge_common.cuh"

namespace sge {

// Rows whose largest magnitude is below this are taken as zeros (scale 0):
// 127 / amax stays finite, and the scale a normal number.
constexpr float kQuantTiny = 7.8886090522101181e-31f;  // 2^-100

struct QuantScale {
  float scale;  // stored with the row
  float inv;    // what values are multiplied by; 0 when the row is all zeros or not finite
};

// `amax_bits`: the largest bit pattern of |x| of the row (as integers, so that
// a NaN, whose pattern is above infinity's, is not lost).  A row that holds
// an infinity or a NaN gets the scale NaN: its products come out NaN, not
// as wrong finite numbers.
SGE_DEV QuantScale quant_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return QuantScale{__uint_as_float(0x7fffffffu), 0.0f};
  const float amax = __uint_as_float(amax_bits);
  if (amax < kQuantTiny) return QuantScale{0.0f, 0.0f};
  return QuantScale{__fdiv_rn(amax, 127.0f), __fdiv_rn(127.0f, amax)};
}

SGE_DEV int quant_value(float x, float inv) {
  // |x * inv| <= 127 * (1 + 2^-23): rounds to at most 127.  A row that is not
  // finite has inv = 0 and stores zeros (0 * inf is a NaN, which converts to 0).
  return __float2int_rn(x * inv);
}

SGE_DEV uint32_t quant_pack4(float a, float b, float c, float d, float inv) {
  return (static_cast<uint32_t>(quant_value(a, inv)) & 0xffu) |
         ((static_cast<uint32_t>(quant_value(b, inv)) & 0xffu) << 8) |
         ((static_cast<uint32_t>(quant_value(c, inv)) & 0xffu) << 16) |
         (static_cast<uint32_t>(quant_value(d, inv)) << 24);
}

SGE_DEV uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// A place of a token's assignment: itself if it is one of `rows` places, else
// a number that is not.  -1 means no place; others out of range are left out
// too, and flagged by the debug build.
SGE_DEV uint32_t checked_place(int32_t p, uint32_t rows) {
#ifdef SGE_DEBUG
  if (p != -1 && static_cast<uint32_t>(p) >= rows) debug_flag();
#endif
  return static_cast<uint32_t>(p) < rows ? static_cast<uint32_t>(p) : 0xffffffffu;
}

// A group bound, moved into [lo, rows].
SGE_DEV int checked_bound(int b, int lo, int rows) {
#ifdef SGE_DEBUG
  if (b < lo || b > rows) debug_flag();
#endif
  return min(max(b, lo), rows);
}

// 16 bytes of an activation row as floats: 8 bf16 or 4 fp32.
template <class T>
struct Vec16;
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  SGE_DEV static void unpack(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  SGE_DEV static void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
};

// Eight values to a 16-byte aligned row.
SGE_DEV void store8(__nv_bfloat16* out, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i])) |
           (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i + 1])) << 16);
  *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
}
SGE_DEV void store8(float* out, const float (&v)[8]) {
  *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(out + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

SGE_DEV float to_f32(float v) { return v; }
SGE_DEV float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
SGE_DEV void from_f32(float v, float* o) { *o = v; }
SGE_DEV void from_f32(float v, __nv_bfloat16* o) { *o = __float2bfloat16_rn(v); }

// Four bytes of q at `dst` (4-byte aligned).
SGE_DEV void store_q(int8_t* dst, const float (&f)[4], float inv) {
  *reinterpret_cast<uint32_t*>(dst) = quant_pack4(f[0], f[1], f[2], f[3], inv);
}
SGE_DEV void store_q(int8_t* dst, const float (&f)[8], float inv) {
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(quant_pack4(f[0], f[1], f[2], f[3], inv), quant_pack4(f[4], f[5], f[6], f[7], inv));
}

// One warp quantises one row of `cols` values: emit(c, f, inv) gets the values
// f of columns c, c + 1, ... (zeros past the row) to be multiplied by inv and
// rounded.  VEC: the row is 16-byte aligned and cols a multiple of a 16-byte
// vector; otherwise it is read element by element.  Up to KEEP vectors a lane
// stay in registers between the two passes; longer rows are read again (from
// L1 / L2).
template <class T, bool VEC, int KEEP, class Emit>
SGE_DEV void quant_row(const T* x, int cols, int lane, uint32_t& amax_out, Emit&& emit) {
  using V = Vec16<T>;
  uint32_t amax = 0;
  if constexpr (VEC) {
    const uint4* xv = reinterpret_cast<const uint4*>(x);
    const int nv = cols / V::N;
    uint4 keep[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      keep[i] = lane + 32 * i < nv ? __ldg(xv + lane + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      float f[V::N];
      V::unpack(keep[i], f);
#pragma unroll
      for (int j = 0; j < V::N; ++j) amax = max(amax, abs_bits(f[j]));
    }
    for (int v = lane + 32 * KEEP; v < nv; v += 32) {
      float f[V::N];
      V::unpack(__ldg(xv + v), f);
#pragma unroll
      for (int j = 0; j < V::N; ++j) amax = max(amax, abs_bits(f[j]));
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    const float inv = quant_scale(amax).inv;
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (lane + 32 * i < nv) {
        float f[V::N];
        V::unpack(keep[i], f);
        emit((lane + 32 * i) * V::N, f, inv);
      }
    for (int v = lane + 32 * KEEP; v < nv; v += 32) {
      float f[V::N];
      V::unpack(__ldg(xv + v), f);
      emit(v * V::N, f, inv);
    }
  } else {
    // four consecutive elements a lane, kept like the vectors above
    const auto four = [&](int i, float (&f)[4]) {
      const int c = 4 * (lane + 32 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = c + j < cols ? to_f32(x[c + j]) : 0.0f;
    };
    const int n4 = (cols + 3) / 4;
    float keep[KEEP][4];
#pragma unroll
    for (int i = 0; i < KEEP; ++i) four(i, keep[i]);
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) amax = max(amax, abs_bits(keep[i][j]));
    for (int i = KEEP; 32 * i < n4; ++i) {
      float f[4];
      four(i, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) amax = max(amax, abs_bits(f[j]));
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    const float inv = quant_scale(amax).inv;
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
      if (lane + 32 * i < n4) emit(4 * (lane + 32 * i), keep[i], inv);
    for (int v = lane + 32 * KEEP; v < n4; v += 32) {
      float f[4];
      four((v - lane) / 32, f);
      emit(4 * v, f, inv);
    }
  }
  amax_out = amax;
}

}  // namespace sge
