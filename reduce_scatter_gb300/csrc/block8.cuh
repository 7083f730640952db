// block8.cuh -- 8-bit values (e4m3 / e5m2) with one fp32 scale for each block of
// 128 columns (of one row, or of 128): how a block's values are found from its
// largest magnitude.
//
//   c = amax / top  (top: the largest finite value; 1 for a block of zeros, at least 2^-126)
//   q = the nearest 8-bit value of x top / amax   (ties to even)
//   powers of two: c = 2^ceil(log2(amax / top)), q = the nearest value of x / c
//
// x top is exact for 16-bit x and the division is correctly rounded, so what lies
// halfway between two 8-bit values stays there: the rounding is that of the
// definition, not of an approximate multiplier (with x * (top / amax) 0.3 % of
// bf16 values, those near a tie, went to the other neighbour).  amax is over the
// block's finite values; a NaN or an infinity becomes NaN and stays alone.
#pragma once

#include "pairs.cuh"
#include "rows.cuh"

namespace dgl {

struct Quantizer {
  float c;            // the scale
  float num, den, rcp;  // q = x num / den; rcp: 1 / den, correctly rounded

  __device__ __forceinline__ Quantizer() {}
  // amax: finite, not negative
  __device__ __forceinline__ Quantizer(float amax, bool e5m2, bool pow2) {
    const int top_exp = e5m2 ? 15 : 8;  // top = 1.75 * 2^top_exp
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23);  // biased
    den = rcp = 1.f;
    bool least;
    if (pow2) {
      const int f = e - top_exp + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // the scale's biased exponent
      least = f <= 1;
      c = __uint_as_float((uint32_t)f << 23);
      num = __uint_as_float((uint32_t)(254 - f) << 23);
    } else {
      c = __fdiv_rn(amax, e5m2 ? kE5M2Max : kE4M3Max);
      least = !(c > kMinScale);
      // both sides times 2^-exponent of amax, so that no product leaves fp32's range
      num = __uint_as_float((uint32_t)(254 + top_exp - e) << 23 | 0x600000u);
      if (!least) {
        den = __uint_as_float((b & 0x7fffffu) | 0x3f800000u);
        rcp = __frcp_rn(den);
      }
    }
    if (least) c = kMinScale, num = 0x1p126f;
    if (amax == 0.f) c = num = 1.f;
  }
  // The correctly rounded quotients from the correctly rounded reciprocal: one
  // product and one residual (Markstein's theorem).  (POW2: den is 1.)
  template <bool POW2>
  __device__ __forceinline__ void all(Eight& v) const {
    const uint64_t n = pair_of(num, num), r = pair_of(rcp, rcp), d = pair_of(-den, -den);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t t = mul2(v.p[k], n);
      if constexpr (POW2) {
        v.p[k] = t;
      } else {
        const uint64_t q = mul2(t, r);
        v.p[k] = fma2(fma2(d, q, t), r, q);
      }
    }
  }
};

// x as it enters a block: an infinity as NaN.
__device__ __forceinline__ float block_value(float x) { return isinf(x) ? __uint_as_float(0x7fc00000u) : x; }

// Eight values of 128: over the 16 threads (half a warp) that hold the block.
__device__ __forceinline__ float block_max16(float m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// The same scale and one multiplier, for values that are themselves the result of
// fp32 arithmetic (or for powers of two, where the product is exact): two
// roundings from x to the 8 bits' own, so what lies within 3 2^-24 of itself from
// halfway between two 8-bit values may go to either.  Values of few bits do lie
// there (the norm of rows of one value, or with weights of zero, is the bias): the
// Quantizer takes the even neighbour of those, this one of the two.
struct Multiplier {
  float c, mul;
  __device__ __forceinline__ Multiplier(float amax, bool e5m2, bool pow2) {
    const int top_exp = e5m2 ? 15 : 8;  // top = 1.75 * 2^top_exp
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23);  // biased
    bool least;
    if (pow2) {
      const int f = e - top_exp + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);  // the scale's biased exponent
      least = f <= 1;
      c = __uint_as_float((uint32_t)f << 23);
      mul = __uint_as_float((uint32_t)(254 - f) << 23);
    } else {
      // quotients from reciprocals and their residuals, Newton's step and Markstein's (of a power of two less where a
      // reciprocal would be subnormal)
      const float top = e5m2 ? kE5M2Max : kE4M3Max, inv = e5m2 ? 1.f / kE5M2Max : 1.f / kE4M3Max, c0 = amax * inv;
      c = fmaf(fmaf(-top, c0, amax), inv, c0);
      least = !(c > kMinScale);
      const float a = __uint_as_float((b & 0x7fffffu) | 0x3f800000u), n = __uint_as_float((uint32_t)(254 + top_exp - e) << 23 | 0x600000u);
      float r;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
      r = fmaf(fmaf(-a, r, 1.f), r, r);
      const float q = n * r;
      mul = fmaf(fmaf(-a, q, n), r, q);
    }
    if (least) c = kMinScale, mul = 0x1p126f;
    if (amax == 0.f) c = mul = 1.f;
  }
};

__device__ __forceinline__ uint2 pack_fp8(const float (&v)[8], __nv_fp8_interpretation_t fmt) {
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k], v[4 * k + 1]), __NV_SATFINITE, fmt);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k + 2], v[4 * k + 3]), __NV_SATFINITE, fmt);
    w[k] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}
// Two 8-bit values (the low 16 bits) as floats.
__device__ __forceinline__ float2 unpack_fp8x2(uint32_t two, __nv_fp8_interpretation_t fmt) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, fmt);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ void unpack_fp8(uint2 u, __nv_fp8_interpretation_t fmt, float (&v)[8]) {
  const uint32_t w[4] = {u.x & 0xffffu, u.x >> 16, u.y & 0xffffu, u.y >> 16};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpack_fp8x2(w[k], fmt);
    v[2 * k] = f.x, v[2 * k + 1] = f.y;
  }
}

// 8-bit blocks of 1 x 128 as they are written.
struct Blocks {
  uint8_t* values;
  float* scales;
  int64_t s_row, s_block;
  int e5m2;
};

// Vector i (of `hidden`) of a row into its block, by all threads of a warp; `in`:
// it is in the row.
__device__ __forceinline__ void store_blocks(const Blocks& o, bool pow2, int64_t row, int hidden, int i, bool in, Eight v) {
  float f[8], m = 0.f;
  v.to_floats(f);
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));  // (passes over NaN)
  if (!in) m = 0.f;
  m = block_max16(m);
  if (__any_sync(0xffffffffu, isinf(m))) {  // an infinity does not enter the scale
    m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] = block_value(f[j]);
      m = fmaxf(m, fabsf(f[j]));
    }
    if (!in) m = 0.f;
    m = block_max16(m);
    v.from_floats(f);
  }
  const Multiplier by(m, o.e5m2 != 0, pow2);
  if (!in) return;
  const uint64_t mul = pair_of(by.mul, by.mul);
#pragma unroll
  for (int j = 0; j < 4; ++j) v.p[j] = mul2(v.p[j], mul);
  v.to_floats(f);
  *reinterpret_cast<uint2*>(o.values + row * hidden + i) = o.e5m2 ? pack_fp8(f, __NV_E5M2) : pack_fp8(f, __NV_E4M3);
  if ((threadIdx.x & 15) == 0) o.scales[row * o.s_row + (int64_t)(i >> 7) * o.s_block] = by.c;
}

// The same of four vectors of each thread, `step` values apart.  The sixteen threads
// of a half warp hold four blocks: they share out the largest magnitudes as they
// reduce them (5 exchanges instead of 16), so that each finds one block's scale
// and passes its multiplier on.
__device__ __forceinline__ void store_blocks4(const Blocks& o, bool pow2, int64_t row, int hidden, int i0, int step, Eight (&v)[4]) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1, second = lane & 2;
  const int block = (odd ? 2 : 0) + (second ? 1 : 0);  // this lane's
  auto top = [&]() {
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f[8];
      v[k].to_floats(f);
      m[k] = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m[k] = fmaxf(m[k], fabsf(f[j]));  // (passes over NaN)
      if (i0 + k * step >= hidden) m[k] = 0.f;
    }
    const float a = fmaxf(odd ? m[2] : m[0], __shfl_xor_sync(0xffffffffu, odd ? m[0] : m[2], 1));
    const float b = fmaxf(odd ? m[3] : m[1], __shfl_xor_sync(0xffffffffu, odd ? m[1] : m[3], 1));
    float c = fmaxf(second ? b : a, __shfl_xor_sync(0xffffffffu, second ? a : b, 2));
    c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, 4));
    return fmaxf(c, __shfl_xor_sync(0xffffffffu, c, 8));
  };
  float m = top();
  if (__any_sync(0xffffffffu, isinf(m))) {  // an infinity does not enter the scale
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f[8];
      v[k].to_floats(f);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = block_value(f[j]);
      v[k].from_floats(f);
    }
    m = top();
  }
  const Multiplier by(m, o.e5m2 != 0, pow2);
  const int first = i0 - (lane & 15) * 8;  // of this half warp's first block
  if ((lane & 15) < 4 && first + block * step < hidden)
    o.scales[row * o.s_row + (int64_t)((first + block * step) >> 7) * o.s_block] = by.c;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float f = __shfl_sync(0xffffffffu, by.mul, (lane & 16) + ((k >> 1) | (k & 1) << 1));
    const uint64_t mul = pair_of(f, f);
    if (i0 + k * step >= hidden) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[k].p[j] = mul2(v[k].p[j], mul);
    float g[8];
    v[k].to_floats(g);
    *reinterpret_cast<uint2*>(o.values + row * hidden + i0 + k * step) = o.e5m2 ? pack_fp8(g, __NV_E5M2) : pack_fp8(g, __NV_E4M3);
  }
}

}  // namespace dgl
