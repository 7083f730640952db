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
  // The correctly rounded quotient from the correctly rounded reciprocal: one
  // product and one residual (Markstein's theorem).
  __device__ __forceinline__ float operator()(float x) const {
    const float t = x * num, q = t * rcp;
    return fmaf(fmaf(-den, q, t), rcp, q);
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
// fp32 arithmetic, where nothing lies exactly halfway (or for powers of two,
// where the product is exact): four roundings from x to the 8 bits' own, and a
// handful of instructions a block instead of two divisions.
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
      c = amax * (e5m2 ? 1.f / kE5M2Max : 1.f / kE4M3Max);
      least = !(c > kMinScale);
      float r;  // of amax without its exponent, so that neither it nor its reciprocal is subnormal
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__uint_as_float((b & 0x7fffffu) | 0x3f800000u)));
      mul = __uint_as_float((uint32_t)(254 + top_exp - e) << 23 | 0x600000u) * r;
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

__device__ __forceinline__ void unpack_fp8(uint2 u, bool e5m2, Eight& v) {
  float f[8];
  if (e5m2)
    unpack_fp8(u, __NV_E5M2, f);
  else
    unpack_fp8(u, __NV_E4M3, f);
  v.from_floats(f);
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

inline bool is_fp8(int t) { return t == DG_TYPE_E4M3 || t == DG_TYPE_E5M2; }

}  // namespace dgl
