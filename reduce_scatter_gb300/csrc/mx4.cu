// mx4.cu -- microscaled 4-bit quantisation and its inverse
// (dg_layer_mx4_quantize, dg_layer_mx4_dequantize).
//
//   a = max|x| over 32 columns;  E = max(floor(log2 a) - 2, -127);  code = e2m1(x / 2^E)
//
// The exponent is read from the maximum's bits, 2^-E is exact in fp32 and so is
// the scaled value, so the one rounding is the conversion to e2m1 (nearest,
// ties to even, saturating at 6).  Bound by memory: 2 bytes read and 17/32
// written per bf16 value.

#include <cuda_bf16.h>

#include "layer_common.h"

namespace {

__device__ __forceinline__ float pow2(int e) {  // 2^e, -127 <= e <= 127 (2^-127 is subnormal)
  return e > -127 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(1u << 22);
}

// Scale byte of a block whose largest magnitude has the fp32 bits `top`.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return 255u;  // an infinity or a NaN in the block
  // biased exponent of the maximum (0 for zeros and fp32 subnormals, whose
  // scale is the smallest one)
  const uint32_t e = top >> 23;
  return e > 2u ? e - 2u : 0u;
}

// Two fp32 values as e2m1 codes: lo in the low half of the byte.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint16_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "cvt.u16.u8 %0, b;\n\t}"
      : "=h"(r)
      : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ int64_t scale_offset(int64_t row, int64_t block, int64_t col_tiles) {
  return ((row >> 7) * col_tiles + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (block & 3);
}

// One warp per 256 columns (8 blocks): a lane holds 8 consecutive values, four
// lanes a block, so reads are 16 (or 32) bytes and writes 4 bytes a lane, and
// the warp's 8 scale bytes are two 4-byte words of the row's place in two
// tiles.  ROWS rows per warp keep that many loads in flight per lane.  The grid
// covers the scale layout's padding, which is written as 0.
template <bool F32, int ROWS>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const void* x, int64_t ld, uint8_t* codes, uint8_t* scales,
                                                           int64_t rows, int64_t cols, int chunks) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int chunk = (int)(w % chunks);
  const int64_t row0 = w / chunks * ROWS;
  if (row0 >= (rows + 127) / 128 * 128) return;
  const int64_t col = (int64_t)chunk * 256 + lane * 8;
  float v[ROWS][8];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (row0 + r < rows && col < cols) {
      const int64_t i = (row0 + r) * ld + col;
      if constexpr (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
        const float4 a = __ldcs(p), b = __ldcs(p + 1);
        v[r][0] = a.x, v[r][1] = a.y, v[r][2] = a.z, v[r][3] = a.w;
        v[r][4] = b.x, v[r][5] = b.y, v[r][6] = b.z, v[r][7] = b.w;
      } else {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + i));
        const uint32_t b[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[r][2 * k] = __uint_as_float(b[k] << 16);
          v[r][2 * k + 1] = __uint_as_float(b[k] & 0xffff0000u);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[r][k] = 0.f;
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t row = row0 + r;
    // magnitudes compare as integers; a NaN is above every other value
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(v[r][k]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t byte = scale_byte(top);
    const float inv = byte == 255u ? 0.f : pow2(127 - (int)byte);
    uint32_t c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) c |= e2m1x2(v[r][2 * k] * inv, v[r][2 * k + 1] * inv) << (8 * k);
    if (byte == 255u) c = 0;
    if (row < rows && col < cols) *reinterpret_cast<uint32_t*>(codes + row * (cols / 2) + col / 2) = c;
    // lanes 0 and 16 gather the four bytes of blocks 0-3 and 4-7
    uint32_t word = byte;
    word |= __shfl_down_sync(0xffffffffu, word, 4) << 8;
    word |= __shfl_down_sync(0xffffffffu, word, 8) << 16;
    if ((lane & 15) == 0)
      *reinterpret_cast<uint32_t*>(scales + scale_offset(row, (int64_t)chunk * 8 + lane / 4, (int64_t)chunks * 2)) = word;
  }
}

// Eight values per thread: 4 bytes of codes in, 16 (or 32) bytes out.
template <bool F32>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, void* y,
                                                             int64_t rows, int64_t cols, int64_t col_tiles) {
  const int64_t per_row = cols / 8, n = rows * per_row, stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
    const int64_t row = i / per_row, col = (i - row * per_row) * 8;
    const uint32_t c = __ldcs(reinterpret_cast<const uint32_t*>(codes) + i);
    const uint32_t byte = __ldg(scales + scale_offset(row, col / 32, col_tiles));
    const float s = byte == 255u ? __uint_as_float(0x7fc00000u) : pow2((int)byte - 127);
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t q = (c >> (4 * k)) & 15u, e = (q >> 1) & 3u, m = q & 1u;
      // e2m1: (1 + m / 2) 2^(e - 1), or m / 2 for e = 0
      const float mag = e ? __uint_as_float(((e + 126u) << 23) | (m << 22)) : 0.5f * (float)m;
      v[k] = (q & 8u ? -mag : mag) * s;
    }
    if constexpr (F32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(y) + i * 8);
      __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
      __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
    } else {
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        o[k] = *reinterpret_cast<const uint32_t*>(&b);
      }
      __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(y) + i * 8), make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

int check_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX)
    return dgl::fail(DG_ERR_ARG, "%lld x %lld out of range", (long long)rows, (long long)cols);
  if (cols % 32 != 0) return dgl::fail(DG_ERR_SHAPE, "the columns (%lld) must be a multiple of 32", (long long)cols);
  return DG_OK;
}

template <bool F32, int ROWS>
int launch_quantize(const void* x, int64_t ld, void* codes, void* scales, int64_t rows, int64_t cols, cudaStream_t s) {
  const int64_t chunks = (cols + 255) / 256, warps = chunks * ((rows + 127) / 128 * 128 / ROWS);
  mx4_quantize_kernel<F32, ROWS><<<(unsigned)((warps + 7) / 8), 256, 0, s>>>(
      x, ld, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), rows, cols, (int)chunks);
  DGL_LAUNCHED();
  return DG_OK;
}

}  // namespace

extern "C" size_t dg_layer_mx4_scale_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return (size_t)((rows + 127) / 128) * (size_t)((cols + 255) / 256) * 1024;
}

extern "C" int dg_layer_mx4_quantize(const void* x, int64_t ld_x, int x_type, void* codes, void* scales, int64_t rows,
                                     int64_t cols, void* stream) {
  if (int rc = check_shape(rows, cols)) return rc;
  if (x_type != DG_TYPE_BF16 && x_type != DG_TYPE_F32) return dgl::fail(DG_ERR_ARG, "x is bf16 or fp32 (got type %d)", x_type);
  if (rows == 0 || cols == 0) return DG_OK;
  if (!x || !codes || !scales) return dgl::fail(DG_ERR_ARG, "x, codes and scales must not be null");
  const bool f32 = x_type == DG_TYPE_F32;
  if (!dgl::aligned16(x) || ld_x * (f32 ? 4 : 2) % 16 != 0 || !dgl::aligned16(codes) || !dgl::aligned16(scales))
    return dgl::fail(DG_ERR_ARG, "x (and its rows), codes and scales must be 16-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // small inputs: one row per warp, so that more SMs take part
  const bool small = (rows + 127) / 128 * 128 * ((cols + 255) / 256) < 65536;
  if (f32) return small ? launch_quantize<true, 1>(x, ld_x, codes, scales, rows, cols, s)
                        : launch_quantize<true, 4>(x, ld_x, codes, scales, rows, cols, s);
  return small ? launch_quantize<false, 1>(x, ld_x, codes, scales, rows, cols, s)
               : launch_quantize<false, 4>(x, ld_x, codes, scales, rows, cols, s);
}

extern "C" int dg_layer_mx4_dequantize(const void* codes, const void* scales, void* y, int y_type, int64_t rows,
                                       int64_t cols, void* stream) {
  if (int rc = check_shape(rows, cols)) return rc;
  if (y_type != DG_TYPE_BF16 && y_type != DG_TYPE_F32) return dgl::fail(DG_ERR_ARG, "y is bf16 or fp32 (got type %d)", y_type);
  if (rows == 0 || cols == 0) return DG_OK;
  if (!codes || !scales || !y) return dgl::fail(DG_ERR_ARG, "codes, scales and y must not be null");
  if (!dgl::aligned16(y) || !dgl::aligned16(codes) || !dgl::aligned16(scales))
    return dgl::fail(DG_ERR_ARG, "codes, scales and y must be 16-byte aligned");
  int sms = 0;
  if (int rc = dgl::sm_count(&sms)) return rc;
  const int64_t n = rows * (cols / 8), want = (n + 255) / 256, most = (int64_t)sms * 32;
  const unsigned grid = (unsigned)(want < most ? want : most);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t col_tiles = (cols + 255) / 256 * 2;
  if (y_type == DG_TYPE_F32)
    mx4_dequantize_kernel<true><<<grid, 256, 0, s>>>(static_cast<const uint8_t*>(codes),
                                                     static_cast<const uint8_t*>(scales), y, rows, cols, col_tiles);
  else
    mx4_dequantize_kernel<false><<<grid, 256, 0, s>>>(static_cast<const uint8_t*>(codes),
                                                      static_cast<const uint8_t*>(scales), y, rows, cols, col_tiles);
  DGL_LAUNCHED();
  return DG_OK;
}
