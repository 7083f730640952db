// norm.cu -- residual add + RMS norm with 16- or 8-bit output, and its
// gradient (dg_layer_add_rms_norm, dg_layer_add_rms_norm_backward).
//
//   h = x + r,  y = h s w,  s = rsqrt(mean h^2 + eps);   8 bits: q = y / c, c = max|y| / max finite
//   dx = s (g - xh mean(g xh)) + dh,  g = dy w,  xh = h s;   dw = sum over rows of dy xh
//
// Both are bound by memory traffic (a handful of operations per value), so a
// row is read once: its threads hold the row's sum in registers through the
// reductions (sum of squares, then the maximum for an 8-bit output) and write
// everything from there.  Many rows are streamed: a block walks rows, and each
// thread keeps its own vectors of the next rows in flight into its own slots of
// shared memory (asynchronous copies; no thread reads another's slots, so the
// hand-off needs no barrier), because a block that loads, reduces and stores by
// turns leaves the memory idle in between.
//
// Back to back on a GB300: 8192 x 16384, bf16 residual, to e4m3 141 us (6.7 TB/s;
// 186 us before streaming), 8192 x 8192 80 us, 16384 x 2048 45 us; 4 rows of 8192
// 2.8 us; fp32 residual, 8192 x 16384 316 us (4.7 TB/s, two stages), 8192 x 8192 144
// us; the gradient of 4099 x 8192 54 us with the weight's (4.9 TB/s), in fp32 114 us
// (4.1).  Without vectors 8192 x 3001 65 us (2.7 TB/s; bf16 output 56, gradient 94),
// 6437 x 10945 254 us (1.9; 222).  The gradients that loop (fp32 of 4099 x 16384 494
// us, 6437 x 10945 538) stay at 1.1 to 1.9 TB/s: partial sums in global memory, values
// loaded twice and one by one.  One vector per thread, or four, instead of two: 97
// and 121 us for 8192 x 8192.

#include "rows.cuh"

namespace {

using namespace dgl;

// ------------------------------------------------------------------ forward

struct NormArgs {
  const void *x, *residual, *weight;
  void *y, *sum;
  float *scale, *rstd;
  const float* scale_in;
  int64_t ld_x, ld_residual, ld_sum, rows;
  int hidden;
  float eps;
  int weight_f32, fp8;  // fp8: 0 bf16 output, else the dg_type
};

// The 8-bit value of y = h rstd w is y / c.  With rstd = f r, f a power of two and
// 1 <= r < 2, a thread forms t = (h f) w, where the product with f is exact, and
// rounds t mul to 8 bits.  |y| / 2 < |t| <= |y|: t leaves fp32's range only where y
// does, and mul stays below 2^128 (h w alone may be far below 1 or overflow while
// y is an ordinary number).  With the row's own scale c = top r / max, `top` the
// largest finite |t|, r cancels: mul = max / top, so q carries two roundings for
// bf16 h and w and hardly ever crosses a rounding boundary of the 8 bits that the
// exact value does not.
struct RowFactor {
  float f, r;
};
__device__ __forceinline__ RowFactor row_factor(float rstd, const float* given) {
  if (!(rstd > 0.f)) return RowFactor{0.f, rstd};  // a sum of squares beyond fp32 (finite values become 0), or a NaN
  const uint32_t b = __float_as_uint(rstd);        // normal (rsqrt of an fp32 value), or infinite: t and r are then too
  float f = __uint_as_float(b & 0x7f800000u), r = __uint_as_float((b & 0x007fffffu) | 0x3f800000u);
  // r / c stays finite for a subnormal c as well
  if (given && fabsf(__ldg(given)) < kMinScale) f *= 0x1p24f, r *= 0x1p-24f;
  return RowFactor{f, r};
}
struct RowScale {
  float c, mul;
};
// ORDINARY: `top` and r are within the bounds below, so that y and c are normal numbers.
template <bool ORDINARY = false>
__device__ __forceinline__ RowScale row_scale(float top, float r, const float* given, bool e5m2) {
  if (given) {
    const float c = __ldg(given);
    return RowScale{c, r / c};
  }
  const float most = e5m2 ? kE5M2Max : kE4M3Max, y = top * r;
  if (ORDINARY) return RowScale{y / most, most / top};
  if (!(y > 0.f)) return RowScale{1.f, r};  // a row of zeros (or one that is not finite, whose values stay so)
  const float c = isinf(y) ? top / most * r : y / most;
  return c > kMinScale ? RowScale{c, most / top} : RowScale{kMinScale, r / kMinScale};
}
// Where t = h w without the factor f serves as well, in the streamed kernel: rstd
// from 2^-40 to 2^60; a top product from 2^-64 (its row's 8-bit steps are then far
// above the subnormal one) to 2^60; with a given scale instead no infinite product
// and no multiplier above 2^100.
constexpr float kOrdinaryDev = 0x1p-40f, kOrdinaryMin = 0x1p-64f, kOrdinaryMax = 0x1p60f, kOrdinaryMul = 0x1p100f;
__device__ __forceinline__ float scaled_by(float h, float keep, float w) { return h * keep * w; }
__device__ __forceinline__ float finite_mag(float t) { return isinf(t) ? 0.f : fabsf(t); }

// RT: the residual's type (0 none, 1 bf16, 2 fp32).  The row stays in
// registers: NV vectors of 8 values per thread.
template <int RT, int NV, bool OUT8>
__global__ void __launch_bounds__(NV > 2 ? 512 : 1024) add_rms_norm_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float part[66];
  begin_kernel();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;  // several rows per block only with one warp each: no barrier below
  const int step = blockDim.x * 8;
  float h[NV][8];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = threadIdx.x * 8 + k * step;
    if (i < p.hidden) {
      load_bf16<8>(p.x, row * p.ld_x + i, h[k]);
      if constexpr (RT != 0) {
        float r[8];
        load_any<8>(RT == 2, p.residual, row * p.ld_residual + i, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[k][j] += r[j];
          // the norm is of the sum as it is stored, so that the gradient sees the same values
          if constexpr (RT == 1) h[k][j] = __bfloat162float(__float2bfloat16_rn(h[k][j]));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[k][j] = 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = threadIdx.x * 8 + k * step;
    if constexpr (RT != 0) {
      if (i < p.hidden) {
        if constexpr (RT == 2)
          store_f32<8>(p.sum, row * p.ld_sum + i, h[k]);
        else
          store_bf16<8>(p.sum, row * p.ld_sum + i, h[k]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(h[k][j], h[k][j], ss);
  }
  ss = row_reduce<Add>(ss, part);
  const float rstd = rsqrtf(ss / (float)p.hidden + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  float top = 0.f;
  const RowFactor by = OUT8 ? row_factor(rstd, p.scale_in) : RowFactor{rstd, 1.f};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = threadIdx.x * 8 + k * step;
    if (i < p.hidden) {
      float w[8];
      load_any<8>(p.weight_f32 != 0, p.weight, i, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[k][j] = scaled_by(h[k][j], by.f, w[j]);
        if constexpr (OUT8) top = fmaxf(top, finite_mag(h[k][j]));
      }
      if constexpr (!OUT8) store_bf16<8>(p.y, row * p.hidden + i, h[k]);
    }
  }
  if constexpr (OUT8) {
    const bool e5m2 = p.fp8 == DG_TYPE_E5M2;
    if (!p.scale_in) top = row_reduce<Max>(top, part + 33);
    const RowScale sc = row_scale(top, by.r, p.scale_in, e5m2);
    if (p.scale && threadIdx.x == 0) p.scale[row] = sc.c;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x * 8 + k * step;
      if (i < p.hidden) {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[k][j] *= sc.mul;
        store_fp8<8>(p.y, row * p.hidden + i, h[k], e5m2 ? __NV_E5M2 : __NV_E4M3);
      }
    }
  }
}

template <int RT, bool W32, int N, bool OUT8>
__global__ void __launch_bounds__(1024) add_rms_norm_spread_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float part[66];
  begin_kernel();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;  // several rows per block only with one warp each: no barrier below
  Spread<false, N> x;
  Spread<RT == 2, N> r;
  Spread<W32, N> w;
  x.load(p.x, row * p.ld_x, p.hidden);
  if constexpr (RT != 0) r.load(p.residual, row * p.ld_residual, p.hidden);
  float h[N], ss = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    h[k] = x.at(k, p.hidden);
    if constexpr (RT != 0) h[k] += r.at(k, p.hidden);
    if constexpr (RT == 1) h[k] = __bfloat162float(__float2bfloat16_rn(h[k]));
    ss = fmaf(h[k], h[k], ss);
  }
  if constexpr (RT != 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      const float v[1] = {h[k]};
      if (i < p.hidden) {
        if constexpr (RT == 2)
          store_f32<1>(p.sum, row * p.ld_sum + i, v);
        else
          store_bf16<1>(p.sum, row * p.ld_sum + i, v);
      }
    }
  }
  w.load(p.weight, 0, p.hidden);  // (in flight during the reduction, in the registers of x and r)
  ss = row_reduce<Add>(ss, part);
  const float rstd = rsqrtf(ss / (float)p.hidden + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  float top = 0.f;
  const RowFactor by = OUT8 ? row_factor(rstd, p.scale_in) : RowFactor{rstd, 1.f};
#pragma unroll
  for (int k = 0; k < N; ++k) {
    h[k] = scaled_by(h[k], by.f, w.at(k, p.hidden));
    if constexpr (OUT8) top = fmaxf(top, finite_mag(h[k]));
  }
  const bool e5m2 = p.fp8 == DG_TYPE_E5M2;
  float mul = 1.f;
  if constexpr (OUT8) {
    if (!p.scale_in) top = row_reduce<Max>(top, part + 33);
    const RowScale sc = row_scale(top, by.r, p.scale_in, e5m2);
    if (p.scale && threadIdx.x == 0) p.scale[row] = sc.c;
    mul = sc.mul;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    const float v[1] = {h[k] * mul};
    if (i < p.hidden) {
      if constexpr (OUT8)
        store_fp8<1>(p.y, row * p.hidden + i, v, e5m2 ? __NV_E5M2 : __NV_E4M3);
      else
        store_bf16<1>(p.y, row * p.hidden + i, v);
    }
  }
}

template <int RT, bool VEC, bool OUT8>
__global__ void __launch_bounds__(1024) add_rms_norm_long_kernel(const __grid_constant__ NormArgs p) {
  __shared__ float part[66];
  begin_kernel();
  const int64_t row = blockIdx.x, hidden = p.hidden, step = blockDim.x * 8;
  const void* hp = RT == 0 ? p.x : p.sum;
  const int64_t h0 = row * (RT == 0 ? p.ld_x : p.ld_sum), y0 = row * hidden;
  // (whole vectors: those past the row are skipped)
  auto chunks = [&](auto body) {
    for (int64_t from = 0; from < hidden; from += step)
      if (!VEC || from + threadIdx.x * 8 < hidden) body(from);
  };
  float ss = 0.f;
  chunks([&](int64_t from) {
    float h[8];
    load_chunk<false, VEC>(p.x, row * p.ld_x, from, hidden, h);
    if constexpr (RT != 0) {
      float r[8];
      load_chunk<RT == 2, VEC>(p.residual, row * p.ld_residual, from, hidden, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[j] += r[j];
        if constexpr (RT == 1) h[j] = __bfloat162float(__float2bfloat16_rn(h[j]));
      }
      if constexpr (RT == 2)
        store_chunk<VEC>(from, hidden, h, [&](int64_t i, const float(&v)[1]) { store_f32<1>(p.sum, h0 + i, v); },
                         [&](int64_t i, const float(&v)[8]) { store_f32<8>(p.sum, h0 + i, v); });
      else
        store_chunk<VEC>(from, hidden, h, [&](int64_t i, const float(&v)[1]) { store_bf16<1>(p.sum, h0 + i, v); },
                         [&](int64_t i, const float(&v)[8]) { store_bf16<8>(p.sum, h0 + i, v); });
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(h[j], h[j], ss);
  });
  ss = row_reduce<Add>(ss, part);
  const float rstd = rsqrtf(ss / (float)p.hidden + p.eps);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  const RowFactor by = OUT8 ? row_factor(rstd, p.scale_in) : RowFactor{rstd, 1.f};
  auto value = [&](int64_t from, float(&h)[8]) {
    float w[8];
    load_chunk<RT == 2, VEC>(hp, h0, from, hidden, h);
    if (p.weight_f32)
      load_chunk<true, VEC>(p.weight, 0, from, hidden, w);
    else
      load_chunk<false, VEC>(p.weight, 0, from, hidden, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = scaled_by(h[j], by.f, w[j]);
  };
  const bool e5m2 = p.fp8 == DG_TYPE_E5M2;
  float mul = 1.f;
  if constexpr (OUT8) {
    float top = 0.f;
    if (!p.scale_in) {
      chunks([&](int64_t from) {
        float h[8];
        value(from, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_mag(h[j]));
      });
      top = row_reduce<Max>(top, part + 33);
    }
    const RowScale sc = row_scale(top, by.r, p.scale_in, e5m2);
    if (p.scale && threadIdx.x == 0) p.scale[row] = sc.c;
    mul = sc.mul;
  }
  chunks([&](int64_t from) {
    float h[8];
    value(from, h);
    if constexpr (OUT8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] *= mul;
      const __nv_fp8_interpretation_t fmt = e5m2 ? __NV_E5M2 : __NV_E4M3;
      store_chunk<VEC>(from, hidden, h, [&](int64_t i, const float(&v)[1]) { store_fp8<1>(p.y, y0 + i, v, fmt); },
                       [&](int64_t i, const float(&v)[8]) { store_fp8<8>(p.y, y0 + i, v, fmt); });
    } else {
      store_chunk<VEC>(from, hidden, h, [&](int64_t i, const float(&v)[1]) { store_bf16<1>(p.y, y0 + i, v); },
                       [&](int64_t i, const float(&v)[8]) { store_bf16<8>(p.y, y0 + i, v); });
    }
  });
}

// ---------------------------------------------------------- streamed forward

constexpr int kStreamVecs = 2;        // vectors of 8 values per thread
constexpr int kStreamThreads = 1024;  // per SM (64 registers each)

template <int RT>
__host__ __device__ constexpr int norm_parts() {
  return kStreamVecs * (1 + RT);  // x, and the residual in 0, 1 or 2 slots
}

template <int RT, bool OUT8, int STAGES>
__global__ void __launch_bounds__(kStreamThreads) add_rms_norm_stream_kernel(const __grid_constant__ NormArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float part[2][99];
  constexpr int NV = kStreamVecs, PER = 1 + RT;
  const Slots<norm_parts<RT>()> slots{smem};
  begin_kernel();
  const int step = blockDim.x * 8, i0 = threadIdx.x * 8;
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.rows) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = i0 + k * step;
        if (i < p.hidden) {
          slots.fetch(stage, k * PER, static_cast<const __nv_bfloat16*>(p.x) + row * p.ld_x + i);
          if constexpr (RT == 1)
            slots.fetch(stage, k * PER + 1, static_cast<const __nv_bfloat16*>(p.residual) + row * p.ld_residual + i);
          if constexpr (RT == 2) {
            const float* r = static_cast<const float*>(p.residual) + row * p.ld_residual + i;
            slots.fetch(stage, k * PER + 1, r);
            slots.fetch(stage, k * PER + 2, r + 4);
          }
        }
      }
    }
    copies_commit();
  };
  float w[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[k][j] = 0.f;
    if (i0 + k * step < p.hidden) load_any<8>(p.weight_f32 != 0, p.weight, i0 + k * step, w[k]);
  }
#pragma unroll
  for (int s = 0; s < STAGES; ++s) fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
  int stage = 0, flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
    copies_wait<STAGES - 1>();
    float h[NV][8], ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = i0 + k * step;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[k][j] = 0.f;
      if (i < p.hidden) {
        slots.template read<false>(stage, k * PER, h[k]);
        if constexpr (RT != 0) {
          float r[8];
          slots.template read<RT == 2>(stage, k * PER + 1, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) h[k][j] += r[j];
          if constexpr (RT == 2) {
            store_f32<8>(p.sum, row * p.ld_sum + i, h[k]);
          } else {
            // the norm is of the sum as it is stored, so that the gradient sees the same values
            const uint4 u = make_uint4(pack2(h[k][0], h[k][1]), pack2(h[k][2], h[k][3]), pack2(h[k][4], h[k][5]),
                                       pack2(h[k][6], h[k][7]));
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.sum) + row * p.ld_sum + i) = u;
            unpack8(u, h[k]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(h[k][j], h[k][j], ss);
    }
    // this stage's values are in registers
    fetch(row + (int64_t)STAGES * gridDim.x, stage);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    ss = row_reduce<Add>(ss, part[flip]);
    const float rstd = rsqrtf(ss / (float)p.hidden + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
    if constexpr (OUT8) {
      float top = 0.f;
      // Ordinary rows do without the factor f, which costs a product per value (8192 x
      // 16384: 141 us, 162 with f in every row).
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[k][j] *= w[k][j];
          top = fmaxf(top, fabsf(h[k][j]));
        }
      const bool e5m2 = p.fp8 == DG_TYPE_E5M2;
      bool ordinary = rstd > kOrdinaryDev && rstd < kOrdinaryMax;
      if (p.scale_in) {  // (each thread for itself)
        ordinary = ordinary && !isinf(top) && fabsf(rstd / __ldg(p.scale_in)) < kOrdinaryMul;
      } else {  // the same for the whole row
        top = row_reduce<Max>(top, part[flip] + 33);
        ordinary = ordinary && top > kOrdinaryMin && top < kOrdinaryMax;
      }
      if (!ordinary) {  // products that left the range, or lost bits at its lower end: again from the stored sum, with f
        const RowFactor by = row_factor(rstd, p.scale_in);
        auto value = [&](int i, float(&t)[8]) {
          float v[8];
          load_any<8>(RT == 2, RT == 0 ? p.x : p.sum, row * (RT == 0 ? p.ld_x : p.ld_sum) + i, t);
          load_any<8>(p.weight_f32 != 0, p.weight, i, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) t[j] = scaled_by(t[j], by.f, v[j]);
        };
        top = 0.f;
        if (!p.scale_in) {
#pragma unroll 1
          for (int i = i0; i < p.hidden; i += step) {
            float t[8];
            value(i, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_mag(t[j]));
          }
          top = row_reduce<Max>(top, part[flip] + 66);
        }
        const RowScale sc = row_scale(top, by.r, p.scale_in, e5m2);
        if (p.scale && threadIdx.x == 0) p.scale[row] = sc.c;
#pragma unroll 1
        for (int i = i0; i < p.hidden; i += step) {
          float t[8];
          value(i, t);
#pragma unroll
          for (int j = 0; j < 8; ++j) t[j] *= sc.mul;
          store_fp8<8>(p.y, row * p.hidden + i, t, e5m2 ? __NV_E5M2 : __NV_E4M3);
        }
        continue;
      }
      const RowScale sc = row_scale<true>(top, rstd, p.scale_in, e5m2);
      if (p.scale && threadIdx.x == 0) p.scale[row] = sc.c;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = i0 + k * step;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[k][j] *= sc.mul;
        if (i < p.hidden) store_fp8<8>(p.y, row * p.hidden + i, h[k], e5m2 ? __NV_E5M2 : __NV_E4M3);
      }
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = i0 + k * step;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[k][j] = h[k][j] * rstd * w[k][j];
        if (i < p.hidden) store_bf16<8>(p.y, row * p.hidden + i, h[k]);
      }
    }
  }
  copies_wait<0>();
}

// The streamed kernels' dynamic shared memory: at most 1024 threads' slots in the
// forward (hidden <= 16384), and what run_grad admits in the gradient.  The limit
// is set to that whatever the call needs: it belongs to the process, and another
// thread's call must not find it lowered between this one's setting and launch.
constexpr int kStreamBytes = 220000;

// Blocks that fill the SMs, and the dynamic shared memory of one.
template <class Kernel>
int stream_shape(Kernel kernel, int hidden, int parts, int stages, int sms, int64_t rows, int* threads, int* blocks,
                 int* bytes) {
  *threads = (hidden / 8 + kStreamVecs - 1) / kStreamVecs;
  *threads = (*threads + 31) / 32 * 32;
  *bytes = stages * parts * 16 * *threads;
  const int64_t most = (int64_t)sms * (kStreamThreads / *threads);
  *blocks = (int)(rows < most ? rows : most);
  DGL_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamBytes));
  return DG_OK;
}

template <int RT, bool OUT8, int STAGES>
int stream_norm(const NormArgs& p, int sms, cudaStream_t s) {
  int threads, blocks, bytes;
  auto* kernel = add_rms_norm_stream_kernel<RT, OUT8, STAGES>;
  if (int rc = stream_shape(kernel, p.hidden, norm_parts<RT>(), STAGES, sms, p.rows, &threads, &blocks, &bytes)) return rc;
  return dgl::launch(kernel, dim3(blocks), dim3(threads), bytes, s, p);
}

template <int RT, int NV, bool OUT8>
int launch_norm(const NormArgs& p, int threads, cudaStream_t s) {
  const int per = threads == 32 ? 4 : 1;  // one warp per row: four rows to a block
  return dgl::launch(add_rms_norm_kernel<RT, NV, OUT8>, dim3((unsigned)((p.rows + per - 1) / per)),
                     dim3(threads, per), 0, s, p);
}

template <int RT, bool W32, bool OUT8>
int spread_norm(const NormArgs& p, cudaStream_t s) {
  const int n = p.hidden <= 1024 ? 4 : 16, threads = round32((p.hidden + n - 1) / n), per = threads == 32 ? 4 : 1;
  return dgl::launch(n == 4 ? add_rms_norm_spread_kernel<RT, W32, 4, OUT8> : add_rms_norm_spread_kernel<RT, W32, 16, OUT8>,
                     dim3((unsigned)((p.rows + per - 1) / per)), dim3(threads, per), 0, s, p);
}

template <int RT, bool OUT8>
int run_norm(const NormArgs& p, bool vec, int sms, cudaStream_t s) {
  if (vec) {
    const int n = p.hidden / 8;
    // Many long rows are streamed, in three stages (two of fp32 residuals: 96 KB
    // each at 16384).  Few rows: as many threads as the row has vectors, for the
    // shortest chain of loads; short rows are light enough for that too.
    if (p.rows > 2 * sms && n >= 256 && n <= 2048) return stream_norm<RT, OUT8, RT == 2 ? 2 : 3>(p, sms, s);
    if (n <= 1024) return launch_norm<RT, 1, OUT8>(p, round32(n), s);
    if (n <= 2048) return launch_norm<RT, 2, OUT8>(p, round32((n + 1) / 2), s);
    if (n <= 4096) return launch_norm<RT, 8, OUT8>(p, round32((n + 7) / 8), s);
    return dgl::launch(add_rms_norm_long_kernel<RT, true, OUT8>, dim3((unsigned)p.rows), dim3(1024), 0, s, p);
  } else {
    if (p.hidden <= 16384) return p.weight_f32 ? spread_norm<RT, true, OUT8>(p, s) : spread_norm<RT, false, OUT8>(p, s);
    return dgl::launch(add_rms_norm_long_kernel<RT, false, OUT8>, dim3((unsigned)p.rows), dim3(1024), 0, s, p);
  }
}

// ----------------------------------------------------------------- gradient

struct GradArgs {
  const void *dy, *h, *weight, *dh;
  const float* rstd;
  void *dx, *dweight;
  float* partial;  // blocks x hidden
  int64_t ld_dy, ld_h, ld_dh, rows;
  int hidden, weight_f32;
};

// Element by element, for rows without 16-byte alignment: N values per thread.
// A block walks the rows blockIdx.x, + gridDim.x, ...; the weight's gradient is
// summed in registers over its rows and written once as a row of `partial`.
template <bool F32, bool W32, int N, bool HAS_DH>
__global__ void __launch_bounds__(512) add_rms_norm_grad_kernel(const __grid_constant__ GradArgs p) {
  __shared__ float part[2][33];
  begin_kernel();
  Spread<W32, N> w;
  w.load(p.weight, 0, p.hidden);
  float dw[N];
#pragma unroll
  for (int k = 0; k < N; ++k) dw[k] = 0.f;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
    const float rstd = __ldg(p.rstd + row);
    Spread<false, N> dy;
    Spread<F32, N> h, dh;
    dy.load(p.dy, row * p.ld_dy, p.hidden);
    h.load(p.h, row * p.ld_h, p.hidden);
    if constexpr (HAS_DH) dh.load(p.dh, row * p.ld_dh, p.hidden);
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float t = dy.at(k, p.hidden) * (h.at(k, p.hidden) * rstd);
      dw[k] += t;
      dot = fmaf(t, w.at(k, p.hidden), dot);
    }
    // two sets of partials: a block's next row may start while a slow warp reads these
    dot = row_reduce<Add>(dot, part[flip]) / (float)p.hidden;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      float d[1] = {0.f};
      if constexpr (HAS_DH) d[0] = dh.at(k, p.hidden);
      d[0] = fmaf(rstd, dy.at(k, p.hidden) * w.at(k, p.hidden) - h.at(k, p.hidden) * rstd * dot, d[0]);
      if (i < p.hidden) {
        if constexpr (F32)
          store_f32<1>(p.dx, row * p.hidden + i, d);
        else
          store_bf16<1>(p.dx, row * p.hidden + i, d);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i < p.hidden) p.partial[(int64_t)blockIdx.x * p.hidden + i] = dw[k];
  }
}

// The gradient's rows streamed like the forward's: dy, h and dh of the next row
// are in flight while this one is reduced and written.  A row is read from its
// slots twice (for the dot product, and again for dx), which leaves registers
// to the weight and its gradient.
template <bool F32, bool HAS_DH>
__host__ __device__ constexpr int grad_parts() {
  return kStreamVecs * (1 + (F32 ? 2 : 1) * (HAS_DH ? 2 : 1));
}
constexpr int kGradStages = 2;

template <bool F32, bool HAS_DH>
__global__ void __launch_bounds__(kStreamThreads) add_rms_norm_grad_stream_kernel(const __grid_constant__ GradArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float part[2][33];
  constexpr int NV = kStreamVecs, HP = F32 ? 2 : 1, PER = 1 + HP * (HAS_DH ? 2 : 1);
  const Slots<grad_parts<F32, HAS_DH>()> slots{smem};
  begin_kernel();
  const int step = blockDim.x * 8, i0 = threadIdx.x * 8;
  const int hsz = F32 ? 4 : 2;
  auto fetch = [&](int64_t row, int stage) {
    if (row < p.rows) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int i = i0 + k * step;
        if (i < p.hidden) {
          slots.fetch(stage, k * PER, static_cast<const __nv_bfloat16*>(p.dy) + row * p.ld_dy + i);
          const uint8_t* h = static_cast<const uint8_t*>(p.h) + (row * p.ld_h + i) * hsz;
#pragma unroll
          for (int q = 0; q < HP; ++q) slots.fetch(stage, k * PER + 1 + q, h + 16 * q);
          if constexpr (HAS_DH) {
            const uint8_t* d = static_cast<const uint8_t*>(p.dh) + (row * p.ld_dh + i) * hsz;
#pragma unroll
            for (int q = 0; q < HP; ++q) slots.fetch(stage, k * PER + 1 + HP + q, d + 16 * q);
          }
        }
      }
    }
    copies_commit();
  };
  float dw[NV][8], w[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[k][j] = w[k][j] = 0.f;
    if (i0 + k * step < p.hidden) load_any<8>(p.weight_f32 != 0, p.weight, i0 + k * step, w[k]);
  }
#pragma unroll
  for (int s = 0; s < kGradStages; ++s) fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
  int stage = 0, flip = 0;
  float rstd_next = blockIdx.x < p.rows ? __ldg(p.rstd + blockIdx.x) : 0.f;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
    const float rstd = rstd_next;
    if (row + gridDim.x < p.rows) rstd_next = __ldg(p.rstd + row + gridDim.x);
    copies_wait<kGradStages - 1>();
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (i0 + k * step < p.hidden) {
        float dy[8], h[8];
        slots.template read<false>(stage, k * PER, dy);
        slots.template read<F32>(stage, k * PER + 1, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float t = dy[j] * (h[j] * rstd);
          dw[k][j] += t;
          dot = fmaf(t, w[k][j], dot);
        }
      }
    }
    // two sets of partials: a block's next row may start while a slow warp reads these
    dot = row_reduce<Add>(dot, part[flip]) / (float)p.hidden;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = i0 + k * step;
      if (i < p.hidden) {
        float dy[8], h[8], d[8];
        slots.template read<false>(stage, k * PER, dy);
        slots.template read<F32>(stage, k * PER + 1, h);
        if constexpr (HAS_DH)
          slots.template read<F32>(stage, k * PER + 1 + HP, d);
        else
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = fmaf(rstd, dy[j] * w[k][j] - h[j] * rstd * dot, d[j]);
        if constexpr (F32)
          store_f32<8>(p.dx, row * p.hidden + i, d);
        else
          store_bf16<8>(p.dx, row * p.hidden + i, d);
      }
    }
    fetch(row + (int64_t)kGradStages * gridDim.x, stage);
    stage ^= 1;
  }
  copies_wait<0>();
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (i0 + k * step < p.hidden) store_f32<8>(p.partial, (int64_t)blockIdx.x * p.hidden + i0 + k * step, dw[k]);
}

// Rows longer than the other kernels hold: two passes over each row; the
// weight's gradient accumulates in the block's row of `partial`.
template <bool F32, bool HAS_DH>
__global__ void __launch_bounds__(1024) add_rms_norm_grad_long_kernel(const __grid_constant__ GradArgs p) {
  __shared__ float part[2][33];
  begin_kernel();
  float* mine = p.partial + (int64_t)blockIdx.x * p.hidden;
  for (int64_t i = threadIdx.x; i < p.hidden; i += blockDim.x) mine[i] = 0.f;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
    const float rstd = __ldg(p.rstd + row);
    float dot = 0.f;
    for (int64_t i = threadIdx.x; i < p.hidden; i += blockDim.x) {
      float dy[1], h[1], w[1];
      load_bf16<1>(p.dy, row * p.ld_dy + i, dy);
      load_any<1>(F32, p.h, row * p.ld_h + i, h);
      load_any<1>(p.weight_f32 != 0, p.weight, i, w);
      mine[i] = fmaf(dy[0], h[0] * rstd, mine[i]);
      dot = fmaf(dy[0] * w[0], h[0] * rstd, dot);
    }
    dot = row_reduce<Add>(dot, part[flip]) / (float)p.hidden;
    for (int64_t i = threadIdx.x; i < p.hidden; i += blockDim.x) {
      float dy[1], h[1], w[1], d[1] = {0.f}, o[1];
      load_bf16<1>(p.dy, row * p.ld_dy + i, dy);
      load_any<1>(F32, p.h, row * p.ld_h + i, h);
      load_any<1>(p.weight_f32 != 0, p.weight, i, w);
      if constexpr (HAS_DH) load_any<1>(F32, p.dh, row * p.ld_dh + i, d);
      o[0] = fmaf(rstd, dy[0] * w[0] - h[0] * rstd * dot, d[0]);
      if constexpr (F32)
        store_f32<1>(p.dx, row * p.hidden + i, o);
      else
        store_bf16<1>(p.dx, row * p.hidden + i, o);
    }
  }
}

// dweight[i] = sum over the blocks' partial rows, in a fixed order: 32 columns
// x 32 threads, each thread a strided share of the rows, then a tree.
__global__ void __launch_bounds__(1024) norm_weight_grad_kernel(const float* partial, int blocks, int hidden,
                                                                void* dweight, int f32) {
  __shared__ float s[32][33];
  begin_kernel();
  const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (col < hidden)
#pragma unroll 8
    for (int b = threadIdx.y; b < blocks; b += 32) v += partial[(int64_t)b * hidden + col];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = s[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int64_t out = (int64_t)blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < hidden) {
    if (f32)
      static_cast<float*>(dweight)[out] = v;
    else
      static_cast<__nv_bfloat16*>(dweight)[out] = __float2bfloat16_rn(v);
  }
}

// Blocks of the gradient kernels: a fixed bound that the workspace is sized by.
constexpr int kGradBlocks = 1216;

// `most` blocks fill the SMs; a block takes four rows at least where there are
// enough of them, so that the partial sums stay small beside the rows.
int grad_blocks(int64_t rows, int sms, int64_t most) {
  if (most > kGradBlocks) most = kGradBlocks;
  const int64_t want = rows / 4 > sms ? rows / 4 : sms;
  const int64_t n = want < most ? want : most;
  return (int)(rows < n ? rows : n);
}

template <bool F32, bool HAS_DH>
int run_grad(GradArgs p, bool vec, int sms, cudaStream_t s) {
  const int n = p.hidden / 8;
  int blocks, rc;
  // 1024 threads hold 16384 values; fp32 rows of that length do not fit twice
  if (vec && n <= 2048 && grad_parts<F32, HAS_DH>() * 16 * kGradStages * (n / kStreamVecs + 31) <= kStreamBytes) {
    int threads, bytes;
    auto* kernel = add_rms_norm_grad_stream_kernel<F32, HAS_DH>;
    rc = stream_shape(kernel, p.hidden, grad_parts<F32, HAS_DH>(), kGradStages, sms, p.rows, &threads, &blocks, &bytes);
    if (rc != DG_OK) return rc;
    blocks = grad_blocks(p.rows, sms, (int64_t)sms * (kStreamThreads / threads));
    rc = dgl::launch(kernel, dim3(blocks), dim3(threads), bytes, s, p);
  } else {
    const bool small = !vec && p.hidden <= 1024, regs = !vec && p.hidden <= 8192;
    const int threads = small ? round32((p.hidden + 3) / 4) : regs ? round32((p.hidden + 15) / 16) : 1024;
    blocks = grad_blocks(p.rows, sms, (int64_t)sms * (threads < 512 ? 512 / threads : 1));
    auto* kernel = add_rms_norm_grad_long_kernel<F32, HAS_DH>;
    if (small)
      kernel = p.weight_f32 ? add_rms_norm_grad_kernel<F32, true, 4, HAS_DH> : add_rms_norm_grad_kernel<F32, false, 4, HAS_DH>;
    else if (regs)
      kernel = p.weight_f32 ? add_rms_norm_grad_kernel<F32, true, 16, HAS_DH> : add_rms_norm_grad_kernel<F32, false, 16, HAS_DH>;
    rc = dgl::launch(kernel, dim3(blocks), dim3(threads), 0, s, p);
  }
  if (rc != DG_OK) return rc;
  return dgl::launch(norm_weight_grad_kernel, dim3((unsigned)((p.hidden + 31) / 32)), dim3(32, 32), 0, s, p.partial, blocks,
                     p.hidden, p.dweight, p.weight_f32);
}

// Rows of no values: the scale of a row of zeros, and the reciprocal deviation of
// the mean of nothing, a NaN.
__global__ void __launch_bounds__(256) norm_of_nothing_kernel(float* scale, float* rstd, int64_t rows) {
  begin_kernel();
  const int64_t row = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (row >= rows) return;
  if (scale) scale[row] = 1.f;
  if (rstd) rstd[row] = __uint_as_float(0x7fc00000u);
}

}  // namespace

extern "C" int dg_layer_add_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                                     int residual_type, const void* weight, int weight_type, void* y, int y_type,
                                     void* sum_out, int64_t ld_sum, float* scale_out, const float* scale_in,
                                     float* rstd_out, int64_t rows, int64_t hidden, float eps, void* stream) {
  if (rows < 0 || hidden < 0 || rows > INT32_MAX || hidden > INT32_MAX)
    return dgl::fail(DG_ERR_ARG, "rows %lld, hidden %lld out of range", (long long)rows, (long long)hidden);
  if (!bf16_or_f32(weight_type) || (residual && !bf16_or_f32(residual_type)))
    return dgl::fail(DG_ERR_ARG, "the weight and the residual are bf16 or fp32");
  const bool out8 = y_type == DG_TYPE_E4M3 || y_type == DG_TYPE_E5M2;
  if (!out8 && y_type != DG_TYPE_BF16) return dgl::fail(DG_ERR_ARG, "y is bf16, e4m3 or e5m2 (got type %d)", y_type);
  if (!(eps >= 0.f)) return dgl::fail(DG_ERR_ARG, "eps must not be negative");
  if (rows == 0) return DG_OK;
  if (hidden == 0) {
    if (!scale_out && !rstd_out) return DG_OK;
    return dgl::launch(norm_of_nothing_kernel, dim3((unsigned)((rows + 255) / 256)), dim3(256), 0,
                       static_cast<cudaStream_t>(stream), scale_out, rstd_out, rows);
  }
  if (!x || !weight || !y) return dgl::fail(DG_ERR_ARG, "x, weight and y must not be null");
  if ((residual != nullptr) != (sum_out != nullptr))
    return dgl::fail(DG_ERR_ARG, "a residual and its sum come together");
  if (out8 && !scale_in && !scale_out) return dgl::fail(DG_ERR_ARG, "an 8-bit output needs scale_out or scale_in");
  int sms = 0;
  if (int rc = dgl::sm_count(&sms)) return rc;
  const int64_t rsz = residual_type == DG_TYPE_F32 ? 4 : 2;
  const bool vec = hidden % 8 == 0 && rows16(x, ld_x, 2) && rows16(residual, ld_residual, rsz) &&
                   rows16(sum_out, ld_sum, rsz) && dgl::aligned16(weight) && dgl::aligned16(y);
  NormArgs p{x, residual, weight, y, sum_out, scale_out, rstd_out, scale_in, ld_x, ld_residual, ld_sum, rows,
             (int)hidden, eps, weight_type == DG_TYPE_F32, out8 ? y_type : 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!residual) return out8 ? run_norm<0, true>(p, vec, sms, s) : run_norm<0, false>(p, vec, sms, s);
  if (residual_type == DG_TYPE_F32) return out8 ? run_norm<2, true>(p, vec, sms, s) : run_norm<2, false>(p, vec, sms, s);
  return out8 ? run_norm<1, true>(p, vec, sms, s) : run_norm<1, false>(p, vec, sms, s);
}

extern "C" size_t dg_layer_add_rms_norm_backward_workspace(int64_t rows, int64_t hidden) {
  if (rows <= 0 || hidden <= 0) return 0;
  return (size_t)(rows < kGradBlocks ? rows : kGradBlocks) * (size_t)hidden * sizeof(float);
}

extern "C" int dg_layer_add_rms_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, int h_type,
                                              const void* weight, int weight_type, const float* rstd, const void* dh,
                                              int64_t ld_dh, void* dx, void* dweight, void* workspace, int64_t rows,
                                              int64_t hidden, void* stream) {
  if (rows < 0 || hidden < 0 || rows > INT32_MAX || hidden > INT32_MAX)
    return dgl::fail(DG_ERR_ARG, "rows %lld, hidden %lld out of range", (long long)rows, (long long)hidden);
  if (!bf16_or_f32(weight_type) || !bf16_or_f32(h_type)) return dgl::fail(DG_ERR_ARG, "h and the weight are bf16 or fp32");
  if (hidden == 0) return DG_OK;
  if (!dweight) return dgl::fail(DG_ERR_ARG, "dweight must not be null");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    DGL_CUDA(cudaMemsetAsync(dweight, 0, (size_t)hidden * (weight_type == DG_TYPE_F32 ? 4 : 2), s));
    return DG_OK;
  }
  if (!dy || !h || !weight || !rstd || !dx || !workspace) return dgl::fail(DG_ERR_ARG, "a required pointer is null");
  if (!dgl::aligned16(workspace)) return dgl::fail(DG_ERR_ARG, "the workspace must be 16-byte aligned");
  int sms = 0;
  if (int rc = dgl::sm_count(&sms)) return rc;
  const int64_t hsz = h_type == DG_TYPE_F32 ? 4 : 2;
  const bool vec = hidden % 8 == 0 && rows16(dy, ld_dy, 2) && rows16(h, ld_h, hsz) && rows16(dh, ld_dh, hsz) &&
                   dgl::aligned16(weight) && dgl::aligned16(dx);
  GradArgs p{dy, h, weight, dh, rstd, dx, dweight, static_cast<float*>(workspace), ld_dy, ld_h, ld_dh, rows,
             (int)hidden, weight_type == DG_TYPE_F32};
  if (h_type == DG_TYPE_F32) return dh ? run_grad<true, true>(p, vec, sms, s) : run_grad<true, false>(p, vec, sms, s);
  return dh ? run_grad<false, true>(p, vec, sms, s) : run_grad<false, false>(p, vec, sms, s);
}
