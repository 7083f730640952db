// block8.cu -- 8-bit values with an fp32 scale for each block of 128 columns:
// quantisation and its inverse (dg_layer_block8_quantize, _dequantize).
//
// Bound by memory traffic: each value is read once and stays in its thread's
// registers until its block's largest magnitude is known.  8192 x 8192 in 16 bits:
// 32 us (6.3 TB/s) in either form of blocks, and 32 us back; with the magnitudes
// and quotients one at a time 38.

#include "block8.cuh"

namespace {

using namespace dgl;

struct QuantArgs {
  const void* x;
  uint8_t* values;
  float* scales;
  int64_t ld_x, rows, cols, s_row, s_block;  // scales' strides: from row (or row block) to row, from column block to column block
  int e5m2;
};

// 16 values of a thread.
template <bool F32>
struct Raw16 {
  uint4 u[F32 ? 4 : 2];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + i * (F32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (F32 ? 4 : 2); ++k) u[k] = __ldg(p + k);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < (F32 ? 4 : 2); ++k) u[k] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(int half, Eight& v) const {
    if constexpr (F32)
      v.from_f32(u[2 * half], u[2 * half + 1]);
    else
      v.from_bf16(u[half]);
  }
  // The largest magnitude, past NaN (an infinity is seen).
  __device__ __forceinline__ float top() const {
    if constexpr (F32) {
      float m = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Eight e;
        float v[8];
        get(h, e);
        e.to_floats(v);
#pragma unroll
        for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(v[k]));
      }
      return m;
    } else {  // (two values at a time)
      const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[k] & 0x7fff7fffu));
      return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
  }
  // Infinities as NaN, so that they do not enter the block's scale.
  __device__ __forceinline__ void drop_infinities() {
    auto word = [](uint32_t& w) {
      if constexpr (F32) {
        if ((w & 0x7fffffffu) == 0x7f800000u) w |= 0x400000u;
      } else {
        if ((w & 0x7fffu) == 0x7f80u) w |= 0x40u;
        if ((w & 0x7fff0000u) == 0x7f800000u) w |= 0x400000u;
      }
    };
#pragma unroll
    for (int k = 0; k < (F32 ? 4 : 2); ++k) word(u[k].x), word(u[k].y), word(u[k].z), word(u[k].w);
  }
  template <bool POW2>
  __device__ __forceinline__ uint4 quantize(const Quantizer& q, bool e5m2) const {
    uint2 w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Eight e;
      float v[8];
      get(h, e);
      q.template all<POW2>(e);
      e.to_floats(v);
      w[h] = e5m2 ? pack_fp8(v, __NV_E5M2) : pack_fp8(v, __NV_E4M3);
    }
    return make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
  }
};

// Blocks of 1 x 128: eight threads to a block, a warp to 512 columns of a row;
// each warp takes kRowsEach rows, whose loads are in flight together.
constexpr int kQuantWarps = 8, kRowsEach = 4;
template <bool F32, bool POW2>
__global__ void __launch_bounds__(32 * kQuantWarps) block8_rows_kernel(const __grid_constant__ QuantArgs p) {
  begin_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)blockIdx.x * (kQuantWarps * kRowsEach) + warp;
  for (int64_t seg = blockIdx.y; seg * 512 < p.cols; seg += gridDim.y) {
    const int64_t col = seg * 512 + lane * 16;
    Raw16<F32> x[kRowsEach];
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k) {
      const int64_t row = row0 + k * kQuantWarps;
      if (row < p.rows && col < p.cols)
        x[k].load(p.x, row * p.ld_x + col);
      else
        x[k].zero();
    }
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k) {
      const int64_t row = row0 + k * kQuantWarps;
      auto block_top = [&]() {
        float m = x[k].top();
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
      };
      float m = block_top();
      if (__any_sync(0xffffffffu, isinf(m))) {
        x[k].drop_infinities();
        m = block_top();
      }
      const Quantizer q(m, p.e5m2 != 0, POW2);
      if (row < p.rows && col < p.cols) {
        *reinterpret_cast<uint4*>(p.values + row * p.cols + col) = x[k].template quantize<POW2>(q, p.e5m2 != 0);
        if ((lane & 7) == 0) p.scales[row * p.s_row + (col / 128) * p.s_block] = q.c;
      }
    }
  }
}

// Blocks of 128 x 128: a thread block each.
template <bool F32, bool POW2>
__global__ void __launch_bounds__(256) block8_tiles_kernel(const __grid_constant__ QuantArgs p) {
  __shared__ float part[8];
  begin_kernel();
  const int64_t row0 = (int64_t)blockIdx.x * 128 + (threadIdx.x >> 3);
  for (int64_t blk = blockIdx.y; blk * 128 < p.cols; blk += gridDim.y) {
    const int64_t col = blk * 128 + (threadIdx.x & 7) * 16;
    Raw16<F32> x[4];
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (row0 + 32 * k < p.rows && col < p.cols)
        x[k].load(p.x, (row0 + 32 * k) * p.ld_x + col);
      else
        x[k].zero();
    }
    auto block_top = [&]() {  // (the barrier before it: the last one's partials have been read)
      m = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) m = fmaxf(m, x[k].top());
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      __syncthreads();
      if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 8; ++k) m = fmaxf(m, part[k]);
    };
    block_top();
    if (isinf(m)) {  // (all threads have the same)
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k].drop_infinities();
      block_top();
    }
    const Quantizer q(m, p.e5m2 != 0, POW2);
    if (threadIdx.x == 0) p.scales[blockIdx.x * p.s_row + blk * p.s_block] = q.c;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (row0 + 32 * k < p.rows && col < p.cols)
        *reinterpret_cast<uint4*>(p.values + (row0 + 32 * k) * p.cols + col) = x[k].template quantize<POW2>(q, p.e5m2 != 0);
  }
}

struct DequantArgs {
  const uint8_t* values;
  const float* scales;
  void* y;
  int64_t rows, cols, s_row, s_block;
  int e5m2, row_shift;  // rows of a block: 2^row_shift
};

// Sixteen bytes of y to a thread and row, so that a warp's stores fill whole lines
// (sixteen values, in two stores 32 bytes apart: 8192 x 8192 37 us), and eight rows in flight.
constexpr int kValueRows = 8;
template <bool F32>
__global__ void __launch_bounds__(32 * kQuantWarps) block8_values_kernel(const __grid_constant__ DequantArgs p) {
  constexpr int N = F32 ? 4 : 8;  // values
  begin_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = (int64_t)blockIdx.x * (kQuantWarps * kValueRows) + warp;
  const __nv_fp8_interpretation_t fmt = p.e5m2 ? __NV_E5M2 : __NV_E4M3;
  for (int64_t seg = blockIdx.y; seg * (32 * N) < p.cols; seg += gridDim.y) {
    const int64_t col = seg * (32 * N) + lane * N;
    if (col >= p.cols) continue;
    uint2 u[kValueRows];
    float s[kValueRows];
#pragma unroll
    for (int k = 0; k < kValueRows; ++k) {
      const int64_t row = min(row0 + k * kQuantWarps, p.rows - 1);
      const uint8_t* from = p.values + row * p.cols + col;
      if constexpr (F32)
        u[k] = make_uint2(__ldg(reinterpret_cast<const uint32_t*>(from)), 0);
      else
        u[k] = __ldg(reinterpret_cast<const uint2*>(from));
      s[k] = __ldg(p.scales + (row >> p.row_shift) * p.s_row + (col / 128) * p.s_block);
    }
#pragma unroll
    for (int k = 0; k < kValueRows; ++k) {
      const int64_t row = row0 + k * kQuantWarps;
      if (row >= p.rows) break;
      float v[8];
      unpack_fp8(u[k], fmt, v);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] *= s[k];
      if constexpr (F32)
        *reinterpret_cast<float4*>(static_cast<float*>(p.y) + row * p.cols + col) = make_float4(v[0], v[1], v[2], v[3]);
      else
        store_bf16<8>(p.y, row * p.cols + col, v);
    }
  }
}

// A thread block's rows and columns, as a grid (its second dimension loops).
dim3 grid_of(int64_t rows, int rows_each, int64_t cols, int cols_each) {
  const int64_t y = (cols + cols_each - 1) / cols_each;
  return dim3((unsigned)((rows + rows_each - 1) / rows_each), (unsigned)(y < 65535 ? y : 65535));
}

int check_shape(int type, int64_t rows, int64_t cols, int block_rows) {
  if (!is_fp8(type)) return fail(DG_ERR_ARG, "8-bit blocks hold e4m3 or e5m2 (got type %d)", type);
  if (rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX)
    return fail(DG_ERR_ARG, "rows %lld, cols %lld out of range", (long long)rows, (long long)cols);
  if (block_rows != 1 && block_rows != 128) return fail(DG_ERR_ARG, "a block has 1 or 128 rows (got %d)", block_rows);
  if (cols % 16) return fail(DG_ERR_SHAPE, "cols %% 16 must be 0 (got %lld)", (long long)cols);
  return DG_OK;
}

}  // namespace

extern "C" int dg_layer_block8_quantize(const void* x, int64_t ld_x, int x_type, void* values, int type, float* scales,
                                        int64_t s_row, int64_t s_block, int block_rows, int pow2, int64_t rows,
                                        int64_t cols, void* stream) {
  if (int rc = check_shape(type, rows, cols, block_rows)) return rc;
  if (!bf16_or_f32(x_type)) return fail(DG_ERR_ARG, "x is bf16 or fp32 (got type %d)", x_type);
  if (rows == 0 || cols == 0) return DG_OK;
  if (!x || !values || !scales) return fail(DG_ERR_ARG, "x, values and scales must not be null");
  const bool f32 = x_type == DG_TYPE_F32;
  if (!aligned16(values) || !rows16(x, ld_x, f32 ? 4 : 2)) return fail(DG_ERR_ARG, "x, its pitch and values must be multiples of 16 bytes");
  const QuantArgs p{x, static_cast<uint8_t*>(values), scales, ld_x, rows, cols, s_row, s_block, type == DG_TYPE_E5M2};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (block_rows == 1)
    return dgl::launch(f32 ? (pow2 ? block8_rows_kernel<true, true> : block8_rows_kernel<true, false>)
                           : (pow2 ? block8_rows_kernel<false, true> : block8_rows_kernel<false, false>), grid_of(rows, kQuantWarps * kRowsEach, cols, 512),
                       dim3(32 * kQuantWarps), 0, s, p);
  return dgl::launch(f32 ? (pow2 ? block8_tiles_kernel<true, true> : block8_tiles_kernel<true, false>)
                         : (pow2 ? block8_tiles_kernel<false, true> : block8_tiles_kernel<false, false>), grid_of(rows, 128, cols, 128), dim3(256), 0, s, p);
}

extern "C" int dg_layer_block8_dequantize(const void* values, int type, const float* scales, int64_t s_row, int64_t s_block,
                                          int block_rows, void* y, int y_type, int64_t rows, int64_t cols, void* stream) {
  if (int rc = check_shape(type, rows, cols, block_rows)) return rc;
  if (!bf16_or_f32(y_type)) return fail(DG_ERR_ARG, "y is bf16 or fp32 (got type %d)", y_type);
  if (rows == 0 || cols == 0) return DG_OK;
  if (!values || !scales || !y) return fail(DG_ERR_ARG, "values, scales and y must not be null");
  if (!aligned16(values) || !aligned16(y)) return fail(DG_ERR_ARG, "values and y must be 16-byte aligned");
  const DequantArgs p{static_cast<const uint8_t*>(values), scales, y, rows, cols, s_row, s_block, type == DG_TYPE_E5M2,
                      block_rows == 128 ? 7 : 0};
  const bool f32 = y_type == DG_TYPE_F32;
  return dgl::launch(f32 ? block8_values_kernel<true> : block8_values_kernel<false>,
                     grid_of(rows, kQuantWarps * kValueRows, cols, f32 ? 128 : 256), dim3(32 * kQuantWarps), 0,
                     static_cast<cudaStream_t>(stream), p);
}
