// rows.cuh -- what the kernels that go over rows of a matrix share: vectors of
// bf16, fp32 and 8-bit values, reductions over the threads of a row, per-thread
// asynchronous copies into shared memory.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "launch.cuh"

namespace dgl {

constexpr float kE4M3Max = 448.f, kE5M2Max = 57344.f;
constexpr float kMinScale = 0x1p-126f;  // the least row scale: the smallest normal number

// ---------------------------------------------------------------- vectors

// VW consecutive bf16 or fp32 values as floats: VW = 8 by 16-byte accesses
// (the caller has checked alignment), VW = 1 by one element.
template <int VW>
__device__ __forceinline__ void load_bf16(const void* base, int64_t i, float (&v)[VW]) {
  if constexpr (VW == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  } else {
    v[0] = __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
  }
}

template <int VW>
__device__ __forceinline__ void load_f32(const void* base, int64_t i, float (&v)[VW]) {
  if constexpr (VW == 8) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = static_cast<const float*>(base)[i];
  }
}

template <int VW>
__device__ __forceinline__ void load_any(bool f32, const void* base, int64_t i, float (&v)[VW]) {
  if (f32)
    load_f32<VW>(base, i, v);
  else
    load_bf16<VW>(base, i, v);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int VW>
__device__ __forceinline__ void store_bf16(void* base, int64_t i, const float (&v)[VW]) {
  if constexpr (VW == 8)
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) =
        make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  else
    static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v[0]);
}

template <int VW>
__device__ __forceinline__ void store_f32(void* base, int64_t i, const float (&v)[VW]) {
  if constexpr (VW == 8) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    static_cast<float*>(base)[i] = v[0];
  }
}

template <int VW>
__device__ __forceinline__ void store_fp8(void* base, int64_t i, const float (&v)[VW], __nv_fp8_interpretation_t fmt) {
  if constexpr (VW == 8) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k], v[4 * k + 1]), __NV_SATFINITE, fmt);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k + 2], v[4 * k + 3]), __NV_SATFINITE, fmt);
      w[k] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(base) + i) = make_uint2(w[0], w[1]);
  } else {
    static_cast<uint8_t*>(base)[i] = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, fmt);
  }
}

// --------------------------------------------------------------- reductions

struct Add {
  __device__ static float of(float a, float b) { return a + b; }
};
struct Max {
  __device__ static float of(float a, float b) { return fmaxf(a, b); }  // ignores NaN
};

// Over the blockDim.x threads of one row (threadIdx.y: the block's rows, one
// warp each when there are several); every thread gets the result, always
// added in the same order.  `part`: 33 floats of shared memory per use.
template <class Op>
__device__ __forceinline__ float row_reduce(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = Op::of(v, __shfl_xor_sync(0xffffffffu, v, o));
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  // the neutral value of both uses (sums of squares, maxima of magnitudes) is 0,
  // and every partial result of a plain sum meets lanes of zeros
  v = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = Op::of(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The sums of two values at once; `part`: 66 floats.
__device__ __forceinline__ float2 row_sum2(float a, float b, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o), b += __shfl_xor_sync(0xffffffffu, b, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return make_float2(a, b);
  const int lane = threadIdx.x & 31;
  float2* p2 = reinterpret_cast<float2*>(part);
  if (lane == 0) p2[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < warps ? p2[lane] : make_float2(0.f, 0.f);
  a = v.x, b = v.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o), b += __shfl_xor_sync(0xffffffffu, b, o);
  return make_float2(a, b);
}

// ------------------------------------------------------------------ spread

// Rows without 16-byte alignment, element by element: thread i holds the values
// i, i + blockDim.x, ...  All loads of a row are issued before the first is used
// (indices past the row read its last value, which is then dropped): with a
// branch around each load they went out one at a time, at 1.7 TB/s.
template <int N, class T>
__device__ __forceinline__ void load_spread(const T* p, int hidden, T (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = p[min((int)(threadIdx.x + k * blockDim.x), hidden - 1)];
}
__device__ __forceinline__ float as_float(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float as_float(float f) { return f; }

// N values per thread of a bf16 or fp32 row, 0 past its end.
template <bool F32, int N>
struct Spread {
  using T = std::conditional_t<F32, float, uint16_t>;
  T v[N];
  __device__ __forceinline__ void load(const void* base, int64_t at, int hidden) {
    load_spread<N, T>(static_cast<const T*>(base) + at, hidden, v);
  }
  __device__ __forceinline__ float at(int k, int hidden) const {
    return (int)(threadIdx.x + k * blockDim.x) < hidden ? as_float(v[k]) : 0.f;
  }
};

// Rows longer than the other kernels hold: each thread goes over its values, 8
// at a time, again for the maximum and for the output (its own stores of the
// sum, still in cache).  VEC: 8 consecutive values, else 8 spread over the block.
template <bool F32, bool VEC>
__device__ __forceinline__ void load_chunk(const void* base, int64_t at, int64_t from, int64_t hidden, float (&v)[8]) {
  if constexpr (VEC) {
    load_any<8>(F32, base, at + from + threadIdx.x * 8, v);  // (the caller has checked that the vector is in the row)
  } else {
    using T = std::conditional_t<F32, float, uint16_t>;
    T t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t i = from + threadIdx.x + k * blockDim.x;
      t[k] = static_cast<const T*>(base)[at + (i < hidden ? i : hidden - 1)];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = from + threadIdx.x + k * blockDim.x < hidden ? as_float(t[k]) : 0.f;
  }
}
template <bool VEC, class Store1, class Store8>
__device__ __forceinline__ void store_chunk(int64_t from, int64_t hidden, const float (&v)[8], Store1 store1, Store8 store8) {
  if constexpr (VEC) {
    store8(from + threadIdx.x * 8, v);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t i = from + threadIdx.x + k * blockDim.x;
      const float one[1] = {v[k]};
      if (i < hidden) store1(i, one);
    }
  }
}

// ----------------------------------------------------- asynchronous copies

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// By way of L1, for the halves of 32 bytes that two copies share: past it each would fetch the whole from L2.
__device__ __forceinline__ void copy_half(uint32_t dst, const void* src, int bytes = 16) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// The first `bytes` of 16 (zeros for the rest).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void unpack8(const uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}

// A thread's 16-byte slots in the dynamic shared memory: `stage`, then vector
// and part of it, then the thread (neighbours are 16 bytes apart).
template <int PARTS>
struct Slots {
  uint8_t* base;
  __device__ __forceinline__ uint4* at(int stage, int part) const {
    return reinterpret_cast<uint4*>(base) + ((int64_t)stage * PARTS + part) * blockDim.x + threadIdx.x;
  }
  __device__ __forceinline__ void fetch(int stage, int part, const void* src) const {
    copy16((uint32_t)__cvta_generic_to_shared(at(stage, part)), src);
  }
  __device__ __forceinline__ void fetch(int stage, int part, const void* src, int bytes) const {
    copy16((uint32_t)__cvta_generic_to_shared(at(stage, part)), src, bytes);
  }
  __device__ __forceinline__ void fetch_half(int stage, int part, const void* src, int bytes = 16) const {
    copy_half((uint32_t)__cvta_generic_to_shared(at(stage, part)), src, bytes);
  }
  // eight values: one slot of bf16 or two of fp32
  template <bool F32>
  __device__ __forceinline__ void read(int stage, int part, float (&v)[8]) const {
    const uint4 a = *at(stage, part);
    if constexpr (F32) {
      const uint4 b = *at(stage, part + 1);
      v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
      v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
    } else {
      unpack8(a, v);
    }
  }
};

// -------------------------------------------------------------------- host

inline int round32(int v) { return (v + 31) / 32 * 32; }

inline bool rows16(const void* p, int64_t ld, int64_t esz) {
  return !p || (dgl::aligned16(p) && (ld * esz) % 16 == 0);
}

inline bool bf16_or_f32(int t) { return t == DG_TYPE_BF16 || t == DG_TYPE_F32; }

}  // namespace dgl
