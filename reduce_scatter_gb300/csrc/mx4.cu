// mx4.cu -- microscaled 4-bit quantisation and its inverse
// (dg_layer_mx4_quantize, dg_layer_mx4_dequantize).
//
//   a = max|x| over 32 columns;  E = max(floor(log2 a) - 2, -127);  code = e2m1(x / 2^E)
//
// The exponent is read from the maximum's bits, 2^-E is exact in fp32 and so is
// the scaled value, so the one rounding is the conversion to e2m1 (nearest,
// ties to even, saturating at 6).  Bound by memory: 2 bytes read and 17/32
// written per bf16 value.  8192 x 16384 back to back on a GB300: 53 us (6.4 TB/s),
// the way back 54 us (6.2 TB/s); two rows per warp 64 us, eight 59 and 55.

#include <cuda_bf16.h>

#include "launch.cuh"

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

// Eight fp32 values as e2m1 codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Larger of two pairs of 15-bit magnitudes (bf16 without signs; a NaN is above
// every other value).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.s16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Eight values of a row as fp32, and the fp32 bits of their largest magnitude.
template <bool F32>
struct Eight;
template <>
struct Eight<false> {
  uint4 u;
  __device__ __forceinline__ void load(const void* x, int64_t i) {
    u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + i));
  }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t t = max2(max2(u.x & m, u.y & m), max2(u.z & m, u.w & m));
    return max(t << 16, t & 0xffff0000u);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t b[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(b[k] << 16);
      v[2 * k + 1] = __uint_as_float(b[k] & 0xffff0000u);
    }
  }
};
template <>
struct Eight<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* x, int64_t i) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
    a = __ldcs(p), b = __ldcs(p + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ uint32_t top() const {
    float v[8];
    values(v);
    uint32_t t = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) t = max(t, __float_as_uint(v[k]) & 0x7fffffffu);
    return t;
  }
};

// Where a warp works: 256 columns (8 blocks) from `col`, ROWS rows from `row0`
// (ROWS divides 32, so that they lie in one run of the scale layout: 16 bytes
// from row to row).
template <int ROWS>
struct Place {
  int64_t row0, scale;  // scale: offset of (row0, first block) in the scale layout
  int64_t col;          // this lane's first column, -1: none
  __device__ __forceinline__ Place(int chunks) {
    const int lane = threadIdx.x & 31;
    const int chunk = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    row0 = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * ROWS;
    col = chunk < chunks ? (int64_t)chunk * 256 + lane * 8 : -1;
    scale = ((row0 >> 7) * (2 * (int64_t)chunks) + 2 * chunk) * 512 + (row0 & 31) * 16 + ((row0 >> 5) & 3) * 4;
  }
};

// One warp per 256 columns: a lane holds 8 consecutive values, four lanes a
// block, so reads are 16 (or 32) bytes and writes 4 bytes a lane, and the
// warp's 8 scale bytes of a row are two 4-byte words in two tiles.  ROWS rows
// per warp keep that many loads in flight per lane.  The grid covers the scale
// layout's padding, which is written as 0.  Index arithmetic is shared by the
// rows and magnitudes are compared two at a time: with 137 instructions per
// eight values, as a first form had, the kernel was bound by issue at 60 % of
// the bandwidth.
template <bool F32, int ROWS>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const void* x, int64_t ld, uint8_t* codes, uint8_t* scales,
                                                           int64_t rows, int64_t cols, int chunks) {
  dgl::begin_kernel();
  const Place<ROWS> at(chunks);
  if (at.col < 0 || at.row0 >= (rows + 127) / 128 * 128) return;
  const int lane = threadIdx.x & 31;
  // this lane's rows with data (none, or fewer than none, in the padding)
  const int ok = at.col < cols ? (int)min((int64_t)ROWS, rows - at.row0) : 0;
  Eight<F32> v[ROWS];
  const int64_t from = at.row0 * ld + at.col;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (r < ok)
      v[r].load(x, from + r * ld);
    else
      v[r].zero();
  }
  uint8_t* to = codes + (at.row0 * cols + at.col) / 2;
  uint8_t* sc = scales + at.scale + (lane >> 4) * 512;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    uint32_t top = v[r].top();
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t byte = scale_byte(top);
    // 2^(127 - byte), exact
    const float inv = __uint_as_float(byte == 255u ? 0u : (254u - byte) << 23);
    float f[8];
    v[r].values(f);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] *= inv;
    uint32_t c = e2m1x8(f);
    if (byte == 255u) c = 0;
    if (r < ok) *reinterpret_cast<uint32_t*>(to + r * (cols / 2)) = c;
    // lanes 0 and 16 gather the four bytes of blocks 0-3 and 4-7
    uint32_t word = byte | (__shfl_down_sync(0xffffffffu, byte, 4) << 8);
    word |= __shfl_down_sync(0xffffffffu, word, 8) << 16;
    if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(sc + r * 16) = word;
  }
}

// The values of four codes (16 bits) as two pairs of bf16: the magnitudes'
// bytes are picked from two eight-byte tables (0, 0.5, 1, 1.5, 2, 3, 4, 6 are
// 0x0000, 0x3f00, 0x3f80, 0x3fc0, 0x4000, 0x4040, 0x4080, 0x40c0), the signs
// moved to bits 15 and 31.
__device__ __forceinline__ void e2m1x4_bf16(uint32_t c, uint32_t& lo, uint32_t& hi) {
  const uint32_t sel = c & 0x7777u;
  const uint32_t high = __byte_perm(0x3f3f3f00u, 0x40404040u, sel), low = __byte_perm(0xc0800000u, 0xc0804000u, sel);
  lo = __byte_perm(low, high, 0x5140) | ((c & 0x8u) << 12) | ((c & 0x80u) << 24);
  hi = __byte_perm(low, high, 0x7362) | ((c & 0x800u) << 4) | ((c & 0x8000u) << 16);
}

// Eight values per lane and row: 4 bytes of codes in, 16 (or 32) bytes out.
// The product with the scale (a power of two) is exact in fp32 and in bf16.
template <bool F32, int ROWS>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, void* y,
                                                             int64_t rows, int64_t cols, int chunks) {
  dgl::begin_kernel();
  const Place<ROWS> at(chunks);
  if (at.col < 0 || at.col >= cols || at.row0 >= rows) return;
  const int lane = threadIdx.x & 31;
  const int ok = (int)min((int64_t)ROWS, rows - at.row0);
  const uint8_t* from = codes + (at.row0 * cols + at.col) / 2;
  const uint8_t* sc = scales + at.scale + (lane >> 4) * 512 + ((lane >> 2) & 3);
  uint32_t c[ROWS], byte[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    c[r] = byte[r] = 0;
    if (r < ok) c[r] = __ldcs(reinterpret_cast<const uint32_t*>(from + r * (cols / 2))), byte[r] = __ldg(sc + r * 16);
  }
  const int64_t to = at.row0 * cols + at.col;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const float s = byte[r] == 255u ? __uint_as_float(0x7fc00000u) : pow2((int)byte[r] - 127);
    uint32_t w[4];
    e2m1x4_bf16(c[r], w[0], w[1]);
    e2m1x4_bf16(c[r] >> 16, w[2], w[3]);
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16) * s;
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u) * s;
    }
    if (r < ok) {
      if constexpr (F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(y) + to + r * cols);
        __stcs(p, make_float4(v[0], v[1], v[2], v[3]));
        __stcs(p + 1, make_float4(v[4], v[5], v[6], v[7]));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
          w[k] = *reinterpret_cast<const uint32_t*>(&b);
        }
        __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(y) + to + r * cols),
               make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
  }
}

// Blocks of up to 8 warps, 2048 columns; the runs of `per` rows over y and z.
int warps_of(int chunks) { return chunks < 8 ? chunks : 8; }
dim3 grid_of(int64_t rows, int chunks, int per) {
  const int64_t runs = (rows + per - 1) / per, z = (runs + 32767) / 32768;
  return dim3((unsigned)((chunks + warps_of(chunks) - 1) / warps_of(chunks)), (unsigned)((runs + z - 1) / z), (unsigned)z);
}

int check_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX)
    return dgl::fail(DG_ERR_ARG, "%lld x %lld out of range", (long long)rows, (long long)cols);
  if (cols % 32 != 0) return dgl::fail(DG_ERR_SHAPE, "the columns (%lld) must be a multiple of 32", (long long)cols);
  return DG_OK;
}

template <bool F32, int ROWS>
int launch_quantize(const void* x, int64_t ld, void* codes, void* scales, int64_t rows, int64_t cols, cudaStream_t s) {
  const int chunks = (int)((cols + 255) / 256);
  return dgl::launch(mx4_quantize_kernel<F32, ROWS>, grid_of((rows + 127) / 128 * 128, chunks, ROWS),
                     dim3(32 * warps_of(chunks)), 0, s, x, ld, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales),
                     rows, cols, chunks);
}
template <bool F32, int ROWS>
int launch_dequantize(const void* codes, const void* scales, void* y, int64_t rows, int64_t cols, cudaStream_t s) {
  const int chunks = (int)((cols + 255) / 256);
  return dgl::launch(mx4_dequantize_kernel<F32, ROWS>, grid_of(rows, chunks, ROWS), dim3(32 * warps_of(chunks)), 0, s,
                     static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), y, rows, cols, chunks);
}

// Small inputs take one row per warp, so that more SMs take part.
bool is_small(int64_t rows, int64_t cols) { return (rows + 127) / 128 * 128 * ((cols + 255) / 256) < 65536; }

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
  const bool small = is_small(rows, cols);
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool small = is_small(rows, cols);
  if (y_type == DG_TYPE_F32) return small ? launch_dequantize<true, 1>(codes, scales, y, rows, cols, s)
                                          : launch_dequantize<true, 4>(codes, scales, y, rows, cols, s);
  return small ? launch_dequantize<false, 1>(codes, scales, y, rows, cols, s)
               : launch_dequantize<false, 4>(codes, scales, y, rows, cols, s);
}
