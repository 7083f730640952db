// pairs.cuh -- two fp32 values in one 64-bit register pair: the packed
// arithmetic takes half the instructions of the separate one.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace dgl {

__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// a b + c
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum_of(uint64_t p) {
  const float2 f = unpair(p);
  return f.x + f.y;
}

// Eight values: one 16-byte vector of bf16, or two of fp32.
struct Eight {
  uint64_t p[4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = 0;
  }
  __device__ __forceinline__ void from_bf16(uint4 u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = pair_of(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
  }
  __device__ __forceinline__ void from_f32(uint4 a, uint4 b) {
    p[0] = pair_of(__uint_as_float(a.x), __uint_as_float(a.y)), p[1] = pair_of(__uint_as_float(a.z), __uint_as_float(a.w));
    p[2] = pair_of(__uint_as_float(b.x), __uint_as_float(b.y)), p[3] = pair_of(__uint_as_float(b.z), __uint_as_float(b.w));
  }
  __device__ __forceinline__ uint4 to_bf16() const {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpair(p[k]);
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 to_f32(int half) const {
    const float2 a = unpair(p[2 * half]), b = unpair(p[2 * half + 1]);
    return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
  }
  __device__ __forceinline__ void to_floats(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpair(p[k]);
      v[2 * k] = f.x, v[2 * k + 1] = f.y;
    }
  }
  __device__ __forceinline__ void from_floats(const float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = pair_of(v[2 * k], v[2 * k + 1]);
  }
};
// Vector i of a matrix in memory.
__device__ __forceinline__ void load8(bool f32, const void* base, int64_t i, Eight& v) {
  if (f32) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i);
    v.from_f32(p[0], p[1]);
  } else {
    v.from_bf16(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i));
  }
}
__device__ __forceinline__ void store8(bool f32, void* base, int64_t i, const Eight& v) {
  if (f32) {
    uint4* p = reinterpret_cast<uint4*>(static_cast<float*>(base) + i);
    p[0] = v.to_f32(0), p[1] = v.to_f32(1);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) = v.to_bf16();
  }
}

}  // namespace dgl
