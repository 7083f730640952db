// layer_norm.cu -- residual add + layer norm with 16-bit output or 8-bit blocks
// of 128, its input kept in 8 bits on request, and the gradient
// (dg_layer_layer_norm, dg_layer_layer_norm_backward).
//
//   h = x + r,  y = (h - mu) s w + b,  mu = mean h,  s = rsqrt(mean (h - mu)^2 + eps)
//   dx = s (g - mean g - xh mean(g xh)) + dh,  g = dy w,  xh = (h - mu) s
//   dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Bound by memory traffic.  A row is read once and stays in its threads'
// registers: first its sum, then, around the mean that it gives, the sums of the
// differences and of their squares (the first corrects the mean by what its
// rounding left, which matters where it is large beside the deviation), then the
// output.  A block of 128 columns lies with the 16 neighbouring threads of half
// a warp, so that its largest magnitude is four shuffles away.  Many rows are
// streamed as in norm.cu: a block walks rows, each thread with its vectors of the
// next rows in flight into its own slots of shared memory.
//
// 8192 x 16384 in 16 bits: 101 us (5.3 TB/s), with a residual 185 (5.8), with a
// residual to e4m3 166 (5.7), kept too 133; its gradient 138 (5.8), from kept rows 158.
// What is left of the way to a copy's rate is instructions: two steps of 512 threads
// over a row, with a barrier in between.

#include "block8.cuh"

namespace {

using namespace dgl;

struct Affine {
  const void *w, *b;  // null: 1 and 0
  int w_f32, b_f32;
};

struct Args {
  const void *x, *residual;
  void *sum, *y;
  Blocks y8, kept;  // y8: the output (y null); kept: h, with power-of-two scales (values null: not kept)
  float *mean, *rstd;
  Affine affine;
  int64_t ld_x, ld_residual, ld_sum, rows;
  int hidden, x_f32, r_f32;
  float eps;
};

// Vector i of w (or 1) and b (or 0).
__device__ __forceinline__ void affine8(const Affine& a, int i, Eight& w, Eight& b) {
#pragma unroll
  for (int j = 0; j < 4; ++j) w.p[j] = pair_of(1.f, 1.f), b.p[j] = 0;
  if (a.w) load8(a.w_f32 != 0, a.w, i, w);
  if (a.b) load8(a.b_f32 != 0, a.b, i, b);
}

// ------------------------------------------------------------- the moments
//
// Each warp finds the mean of its own values and the sum of the squared
// differences from it; the warps' are then put together around the first one's
// mean (a sum of squares grows by n (its mean - the row's)^2).  One barrier, and
// no difference of large numbers.

struct Moments {
  float mean, rstd;
};
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// How many values each warp holds, and their reciprocals.  (Products with these in
// place of divisions: what they leave in a mean the differences show.)
struct Share {
  float n, inv;
  __device__ __forceinline__ Share(int count) : n((float)count), inv(count > 0 ? 1.f / (float)count : 0.f) {}
};
// The second step of a warp's: from its mean as rounded, the sums of the
// differences from it and of their squares.  The first corrects the mean (below 2^-21 of
// the deviation the differences' own rounding is what their sum shows).
__device__ __forceinline__ float2 warp_moments(float mean, float d1, float d2, const Share& own) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d1 += __shfl_xor_sync(0xffffffffu, d1, o), d2 += __shfl_xor_sync(0xffffffffu, d2, o);
  const float off = d1 * own.inv, gone = off * d1;
  const bool far = gone > 0x1p-42f * d2;
  const float s = d2 - gone;
  return make_float2(far ? mean + off : mean, !far ? d2 : s < 0.f ? 0.f : s);
}
// The row's from lane l's warp l (none: a share of 0) of `hidden` values.
__device__ __forceinline__ Moments join_moments(float2 m, const Share& of, float inv_hidden, float eps) {
  const float first = __shfl_sync(0xffffffffu, m.x, 0);
  const float d = of.n == 0.f ? 0.f : m.x - first;
  const float off = warp_sum(of.n * d) * inv_hidden;
  const float s = warp_sum(of.n == 0.f ? 0.f : fmaf(of.n * (d - off), d - off, m.y));
  return Moments{first + off, rsqrtf(fmaf(s, inv_hidden, eps))};
}
__device__ __forceinline__ void keep_moments(const Args& p, int64_t row, const Moments& m) {
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = m.mean;
    if (p.rstd) p.rstd[row] = m.rstd;
  }
}
// Values of warp w whose threads hold NV vectors of 8, blockDim.x threads apart;
// the row starts `shift` values into the first vector.
template <int NV>
__device__ __forceinline__ int warp_count(int w, int hidden, int shift = 0) {
  int n = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int from = w * 256 + k * (int)blockDim.x * 8 - shift;
    n += max(min(from + 256, hidden) - max(from, 0), 0);
  }
  return n;
}
// Values of vector i that are not in the row become 0.
__device__ __forceinline__ void clip(Eight& v, int i, int hidden) {
  float f[8];
  v.to_floats(f);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = i + j < 0 || i + j >= hidden ? 0.f : f[j];
  v.from_floats(f);
}

// How the vectors of a row lie: every thread has its NV (kFull); whole vectors,
// not in every thread (kVectors); or the row starts and ends inside vectors
// (kEdges: rows without 16-byte alignment, of which each block takes those that
// start at the same place in a vector).
enum { kFull = 0, kVectors = 1, kEdges = 2 };

// A warp's moments from its vectors (those past the row: zeros).
template <int NV, int MODE = kVectors>
__device__ __forceinline__ float2 moments_of(const Eight (&h)[NV], int hidden, int i0, int step, const Share& own) {
  uint64_t sum = add2(h[0].p[0], h[0].p[1]);
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int j = k == 0 ? 2 : 0; j < 4; ++j) sum = add2(sum, h[k].p[j]);
  const float mean = warp_sum(sum_of(sum)) * own.inv;
  const uint64_t minus = pair_of(-mean, -mean);
  uint64_t d1 = 0, d2 = 0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = i0 + k * step;
    const uint64_t from = MODE == kFull || i < hidden ? minus : 0;  // (zeros stay zeros, without a branch)
    Eight d;
#pragma unroll
    for (int j = 0; j < 4; ++j) d.p[j] = add2(h[k].p[j], from);
    if (MODE == kEdges && (i < 0 || i + 8 > hidden)) clip(d, i, hidden);
#pragma unroll
    for (int j = 0; j < 4; ++j) d1 = add2(d1, d.p[j]), d2 = fma2(d.p[j], d.p[j], d2);
  }
  return warp_moments(mean, sum_of(d1), sum_of(d2), own);
}
// Vector i into a row at `at`; of one that is not whole, what is in the row.
template <int MODE>
__device__ __forceinline__ void store_row8(bool f32, void* base, int64_t at, int i, int hidden, const Eight& v) {
  if (MODE == kEdges && (i < 0 || i + 8 > hidden)) {
    float f[8];
    v.to_floats(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float one[1] = {f[j]};
      if (i + j < 0 || i + j >= hidden) continue;
      if (f32)
        store_f32<1>(base, at + i + j, one);
      else
        store_bf16<1>(base, at + i + j, one);
    }
  } else {
    store8(f32, base, at + i, v);
  }
}
// Vector i of a vector of `hidden` values (its nearest ones, where it is not whole).
template <int MODE>
__device__ __forceinline__ void load_row8(bool f32, const void* base, int i, int hidden, Eight& v) {
  if (MODE == kEdges) {  // (no alignment)
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float one[1];
      load_any<1>(f32, base, min(max(i + j, 0), hidden - 1), one);
      f[j] = one[0];
    }
    v.from_floats(f);
  } else {
    load8(f32, base, i, v);
  }
}

// Vector i of a row's output, from h.
template <bool OUT8>
__device__ __forceinline__ void finish(const Args& p, int64_t row, int i, bool in, const Moments& m, const Eight& h, const Eight& w,
                                       const Eight& b) {
  if (p.kept.values) store_blocks(p.kept, true, row, p.hidden, i, in, h);
  const uint64_t minus = pair_of(-m.mean, -m.mean), rstd = pair_of(m.rstd, m.rstd);
  Eight y;
#pragma unroll
  for (int j = 0; j < 4; ++j) y.p[j] = fma2(mul2(add2(h.p[j], minus), rstd), w.p[j], b.p[j]);
  if constexpr (OUT8)
    store_blocks(p.y8, false, row, p.hidden, i, in, y);
  else if (in)
    store8(false, p.y, row * p.hidden + i, y);
}

// ------------------------------------------------------ a row in registers

// NV vectors of 8 values per thread.
template <int NV, bool OUT8>
__global__ void __launch_bounds__(NV > 2 ? 512 : 1024) layer_norm_kernel(const __grid_constant__ Args p) {
  __shared__ float2 part[32];
  begin_kernel();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;  // several rows per block only with one warp each: no barrier below
  const int step = blockDim.x * 8, i0 = threadIdx.x * 8, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  Eight h[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = i0 + k * step;
    h[k].zero();
    if (i < p.hidden) {
      load8(p.x_f32 != 0, p.x, row * p.ld_x + i, h[k]);
      if (p.residual) {
        Eight r;
        load8(p.r_f32 != 0, p.residual, row * p.ld_residual + i, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[k].p[j] = add2(h[k].p[j], r.p[j]);
        store8(p.r_f32 != 0, p.sum, row * p.ld_sum + i, h[k]);
        // the norm is of the sum as it is stored, so that the gradient sees the same values
        if (!p.r_f32) h[k].from_bf16(h[k].to_bf16());
      }
    }
  }
  float2 mine = moments_of(h, p.hidden, i0, step, Share(warp_count<NV>(threadIdx.x >> 5, p.hidden)));
  if (warps > 1) {
    if (lane == 0) part[threadIdx.x >> 5] = mine;
    __syncthreads();
    mine = part[lane < warps ? lane : 0];
  }
  const Moments m = join_moments(mine, Share(lane < warps ? warp_count<NV>(lane, p.hidden) : 0), 1.f / (float)p.hidden, p.eps);
  keep_moments(p, row, m);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = i0 + k * step;
    const bool in = i < p.hidden;
    Eight w, b;
    affine8(p.affine, in ? i : 0, w, b);
    finish<OUT8>(p, row, i, in, m, h[k], w, b);
  }
}

// ------------------------------------------------------------ streamed rows

constexpr int kStages = 2;           // (three, or the next row's sums ahead of this one's output: 178 us instead of 167 for 8192 x 16384 to e4m3)
constexpr int kStreamVecs = 4;       // vectors of 8 values per thread
constexpr int kStreamThreads = 512;  // per SM (128 registers each)
constexpr int kSmBytes = 233472, kBlockBytes = 1024 + 1024;  // shared memory of an SM, and what a block takes besides
constexpr int kStreamBytes = 231936;  // dynamic shared memory that the streamed kernels may take, whatever the call needs

// XP, RP: 16-byte slots of eight values of x (1 bf16, 2 fp32) and of the
// residual (0 none).  A row goes through two steps, with a barrier in between: its
// warps' moments, and the output, for which h is read from the slots again
// (nothing is held in registers over the barrier).
template <int XP, int RP, bool OUT8, int MODE>
__global__ void __launch_bounds__(kStreamThreads) layer_norm_stream_kernel(const __grid_constant__ Args p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 part[2][32];  // (of two rows by turns: a warp's next sums may come before a slow one has read these)
  constexpr int NV = kStreamVecs, PER = XP + RP;
  constexpr bool H32 = RP == 2 || (RP == 0 && XP == 2);
  constexpr int HS = RP == 2 ? XP : 0;  // h's slot of a vector's
  const Slots<NV * PER> slots{smem};
  begin_kernel();
  const int shift = MODE == kEdges ? (int)((blockIdx.x & 7u) * (p.hidden & 7u) & 7u) : 0;
  const int step = blockDim.x * 8, i0 = threadIdx.x * 8 - shift, warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto in = [&](int k) { return MODE == kFull || i0 + k * step < p.hidden; };
  // a slot of up to 16 bytes of values from i on (the start of a row that begins inside it holds the end of the row before)
  auto copy = [&](int stage, int part, const uint8_t* src, int i, int size) {  // (8192 x 8192 in fp32 past L1: 102 us, now 72)
    // (zeros past the row, so that only stores ask where it ends: with a branch for each vector 4099 x 8208 52 us, now 47)
    const int bytes = MODE == kFull ? 16 : MODE == kEdges ? min(max((p.hidden - i) * size, 0), 16) : i < p.hidden ? 16 : 0;
    if (MODE != kFull && bytes == 0) src = static_cast<const uint8_t*>(p.x);
    if (size == 4)
      slots.fetch_half(stage, part, src, bytes);
    else if (MODE == kFull)
      slots.fetch(stage, part, src);
    else
      slots.fetch(stage, part, src, bytes);
  };
  // this thread's place in the next row to fetch
  int64_t next = blockIdx.x;
  const uint8_t* x_next = static_cast<const uint8_t*>(p.x) + (next * p.ld_x + i0) * (2 * XP);
  const uint8_t* r_next = RP ? static_cast<const uint8_t*>(p.residual) + (next * p.ld_residual + i0) * (2 * RP) : nullptr;
  const int64_t x_rows = gridDim.x * p.ld_x * (2 * XP), r_rows = gridDim.x * p.ld_residual * (2 * RP);
  auto fetch = [&](int stage) {
    if (next < p.rows) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int q = 0; q < XP; ++q) copy(stage, k * PER + q, x_next + k * step * (2 * XP) + 16 * q, i0 + k * step + 4 * q, 2 * XP);
        if constexpr (RP != 0)
#pragma unroll
          for (int q = 0; q < RP; ++q)
            copy(stage, k * PER + XP + q, r_next + k * step * (2 * RP) + 16 * q, i0 + k * step + 4 * q, 2 * RP);
      }
    }
    next += gridDim.x;
    x_next += x_rows;
    if (RP) r_next += r_rows;
    copies_commit();
  };
  auto read = [&](bool f32, int stage, int slot, Eight& v) {
    if (f32)
      v.from_f32(*slots.at(stage, slot), *slots.at(stage, slot + 1));
    else
      v.from_bf16(*slots.at(stage, slot));
  };
  // w in 16 bits stays in registers, b behind the stages (both in registers left too few for a row's output)
  auto bias_slot = [&](int k) { return slots.at(0, kStages * NV * PER + k); };
  uint4 w16[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = i0 + k * step;
    w16[k] = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    uint4 b16 = make_uint4(0, 0, 0, 0);
    if (in(k)) {
      Eight v;
      if (p.affine.w && !p.affine.w_f32) load_row8<MODE>(false, p.affine.w, i, p.hidden, v), w16[k] = v.to_bf16();
      if (p.affine.b && !p.affine.b_f32) load_row8<MODE>(false, p.affine.b, i, p.hidden, v), b16 = v.to_bf16();
    }
    *bias_slot(k) = b16;
  }
  const Share own(MODE == kFull ? NV * 256 : warp_count<NV>(warp, p.hidden, shift));
  const Share of(lane >= warps ? 0 : MODE == kFull ? NV * 256 : warp_count<NV>(lane, p.hidden, shift));
  const float inv_hidden = 1.f / (float)p.hidden;
  auto sums = [&](int64_t row, int stage) {
    Eight h[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = i0 + k * step;
      read(XP == 2, stage, k * PER, h[k]);
      if constexpr (RP != 0) {
        Eight r;
        read(RP == 2, stage, k * PER + XP, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[k].p[j] = add2(h[k].p[j], r.p[j]);
        if constexpr (RP == 2) {
          *slots.at(stage, k * PER + HS) = h[k].to_f32(0);
          *slots.at(stage, k * PER + HS + 1) = h[k].to_f32(1);
        } else {
          // the norm is of the sum as it is stored, so that the gradient sees the same values
          const uint4 u = h[k].to_bf16();
          *slots.at(stage, k * PER) = u;
          h[k].from_bf16(u);
        }
        if (in(k)) store_row8<MODE>(RP == 2, p.sum, row * p.ld_sum, i, p.hidden, h[k]);
      }
      if (MODE == kEdges && (i < 0 || i + 8 > p.hidden)) clip(h[k], i, p.hidden);
    }
    const float2 m = moments_of<NV, MODE>(h, p.hidden, i0, step, own);
    if (lane == 0) part[stage][warp] = m;
  };
  auto output = [&](int64_t row, int stage) {
    const Moments m = join_moments(part[stage][lane < warps ? lane : 0], of, inv_hidden, p.eps);
    keep_moments(p, row, m);
    const uint64_t minus = pair_of(-m.mean, -m.mean), rstd = pair_of(m.rstd, m.rstd);
    auto stored = [&](int k) {
      Eight h;
      read(H32, stage, k * PER + HS, h);
      return h;
    };
    if (MODE != kEdges && p.kept.values) {
      static_assert(NV == 4, "store_blocks4 takes four vectors");
      Eight h[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) h[k] = stored(k);
      store_blocks4(p.kept, true, row, p.hidden, i0, step, h);
    }
    Eight y[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = i0 + k * step;
      const Eight h = stored(k);
      Eight w, b;
      w.from_bf16(w16[k]), b.from_bf16(*bias_slot(k));
      if (in(k)) {
        if (p.affine.w_f32) load_row8<MODE>(true, p.affine.w, i, p.hidden, w);
        if (p.affine.b_f32) load_row8<MODE>(true, p.affine.b, i, p.hidden, b);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) y[k].p[j] = fma2(mul2(add2(h.p[j], minus), rstd), w.p[j], b.p[j]);
      if (!OUT8 && in(k)) store_row8<MODE>(false, p.y, row * p.hidden, i, p.hidden, y[k]);
    }
    if constexpr (OUT8) store_blocks4(p.y8, false, row, p.hidden, i0, step, y);
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) fetch(s);
  int stage = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, stage ^= 1) {
    copies_wait<kStages - 1>();
    sums(row, stage);
    __syncthreads();
    output(row, stage);
    fetch(stage);
  }
  copies_wait<0>();
}

// ------------------------------------------------ rows without alignment

// (16-bit output: rows of 8-bit blocks are multiples of 16 values, and come aligned)
template <bool X32, int RT, int N>
__global__ void __launch_bounds__(1024) layer_norm_spread_kernel(const __grid_constant__ Args p) {
  __shared__ float2 part[32];
  begin_kernel();
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  auto count = [&](int w) {
    int n = 0;
    for (int k = 0; k < N; ++k) n += min(max(p.hidden - (w * 32 + k * (int)blockDim.x), 0), 32);
    return n;
  };
  Spread<X32, N> x;
  Spread<RT == 2, N> r;
  x.load(p.x, row * p.ld_x, p.hidden);
  if constexpr (RT != 0) r.load(p.residual, row * p.ld_residual, p.hidden);
  float h[N], sum = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    h[k] = x.at(k, p.hidden);
    if constexpr (RT != 0) h[k] += r.at(k, p.hidden);
    if constexpr (RT == 1) h[k] = __bfloat162float(__float2bfloat16_rn(h[k]));
    if (RT != 0 && i < p.hidden) {
      const float v[1] = {h[k]};
      if constexpr (RT == 2)
        store_f32<1>(p.sum, row * p.ld_sum + i, v);
      else
        store_bf16<1>(p.sum, row * p.ld_sum + i, v);
    }
    sum += h[k];
  }
  const Share own(count(threadIdx.x >> 5));
  const float mean = warp_sum(sum) * own.inv;
  float d1 = 0.f, d2 = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k)
    if ((int)(threadIdx.x + k * blockDim.x) < p.hidden) {
      const float d = h[k] - mean;
      d1 += d, d2 = fmaf(d, d, d2);
    }
  float2 mine = warp_moments(mean, d1, d2, own);
  if (warps > 1) {
    if (lane == 0) part[threadIdx.x >> 5] = mine;
    __syncthreads();
    mine = part[lane < warps ? lane : 0];
  }
  const Moments m = join_moments(mine, Share(lane < warps ? count(lane) : 0), 1.f / (float)p.hidden, p.eps);
  keep_moments(p, row, m);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i < p.hidden) {
      float w[1] = {1.f}, b[1] = {0.f};
      if (p.affine.w) load_any<1>(p.affine.w_f32 != 0, p.affine.w, i, w);
      if (p.affine.b) load_any<1>(p.affine.b_f32 != 0, p.affine.b, i, b);
      const float v[1] = {fmaf((h[k] - m.mean) * m.rstd, w[0], b[0])};
      store_bf16<1>(p.y, row * p.hidden + i, v);
    }
  }
}

// ------------------------------------------------------------- longer rows

// Rows longer than the other kernels hold: each thread goes over its values, 8
// at a time, again for the differences and for the output.
template <bool VEC, bool OUT8>
__global__ void __launch_bounds__(1024) layer_norm_long_kernel(const __grid_constant__ Args p) {
  static_assert(VEC || !OUT8, "8-bit blocks come in vectors");
  __shared__ float part[100];
  begin_kernel();
  const int64_t row = blockIdx.x, hidden = p.hidden, step = blockDim.x * 8;
  const bool h_f32 = p.residual ? p.r_f32 != 0 : p.x_f32 != 0;
  const void* hp = p.residual ? p.sum : p.x;
  const int64_t h0 = row * (p.residual ? p.ld_sum : p.ld_x);
  auto load = [&](bool f32, const void* base, int64_t at, int64_t from, float (&v)[8]) {
    if (VEC && from + threadIdx.x * 8 >= hidden) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    } else if (f32) {
      load_chunk<true, VEC>(base, at, from, hidden, v);
    } else {
      load_chunk<false, VEC>(base, at, from, hidden, v);
    }
  };
  auto in_row = [&](int64_t from, int k) {
    return VEC ? from + threadIdx.x * 8 < hidden : from + threadIdx.x + (int64_t)k * blockDim.x < hidden;
  };
  float sum = 0.f;
  for (int64_t from = 0; from < hidden; from += step) {
    float h[8];
    load(p.x_f32 != 0, p.x, row * p.ld_x, from, h);
    if (p.residual) {
      float r[8];
      load(p.r_f32 != 0, p.residual, row * p.ld_residual, from, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] += r[j];
      if (!p.r_f32)
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = __bfloat162float(__float2bfloat16_rn(h[j]));
      if (!VEC || in_row(from, 0)) {
        if (p.r_f32)
          store_chunk<VEC>(from, hidden, h, [&](int64_t i, const float(&v)[1]) { store_f32<1>(p.sum, h0 + i, v); },
                           [&](int64_t i, const float(&v)[8]) { store_f32<8>(p.sum, h0 + i, v); });
        else
          store_chunk<VEC>(from, hidden, h, [&](int64_t i, const float(&v)[1]) { store_bf16<1>(p.sum, h0 + i, v); },
                           [&](int64_t i, const float(&v)[8]) { store_bf16<8>(p.sum, h0 + i, v); });
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += h[j];
  }
  const float mean = row_reduce<Add>(sum, part) / (float)p.hidden;
  float d1 = 0.f, d2 = 0.f;
  for (int64_t from = 0; from < hidden; from += step) {  // (a thread's own stores of the sum)
    float h[8];
    load(h_f32, hp, h0, from, h);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = in_row(from, j) ? h[j] - mean : 0.f;
      d1 += d, d2 = fmaf(d, d, d2);
    }
  }
  // (the whole row as one warp's: lane 0 holds it)
  const float2 all = row_sum2(d1, d2, part + 34);
  const float2 one = warp_moments(mean, (threadIdx.x & 31) == 0 ? all.x : 0.f, (threadIdx.x & 31) == 0 ? all.y : 0.f, Share((int)hidden));
  const Moments m{one.x, rsqrtf(one.y / (float)hidden + p.eps)};
  keep_moments(p, row, m);
  for (int64_t from = 0; from < hidden; from += step) {
    float h[8], w[8], b[8];
    load(h_f32, hp, h0, from, h);
    if constexpr (VEC) {
      const int i = (int)from + threadIdx.x * 8;  // (beyond the row by less than a step)
      const bool in = in_row(from, 0);
      Eight h8, w8, b8;
      h8.from_floats(h);
      affine8(p.affine, in ? i : 0, w8, b8);
      finish<OUT8>(p, row, i, in, m, h8, w8, b8);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = 1.f, b[j] = 0.f;
      if (p.affine.w) load(p.affine.w_f32 != 0, p.affine.w, 0, from, w);
      if (p.affine.b) load(p.affine.b_f32 != 0, p.affine.b, 0, from, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = fmaf((h[j] - m.mean) * m.rstd, w[j], b[j]);
      store_chunk<false>(from, hidden, h, [&](int64_t i, const float(&v)[1]) { store_bf16<1>(p.y, row * hidden + i, v); },
                         [&](int64_t, const float(&)[8]) {});
    }
  }
}

// ------------------------------------------------------------ forward launch

// Threads of a streamed row of n vectors.
constexpr int stream_threads(int n) { return ((n + kStreamVecs - 1) / kStreamVecs + 31) / 32 * 32; }

// Vectors of a row; one that starts inside a vector takes another.
constexpr int row_vectors(int hidden, bool vec) { return vec ? hidden / 8 : (hidden + 14) / 8; }

// Shared memory of a block: its stages of `slots` 16-byte slots a vector, and the bias.
constexpr int stream_bytes(int slots, int threads) { return (kStages * slots + 1) * kStreamVecs * 16 * threads; }

template <class Kernel>
int stream_shape(Kernel kernel, int vectors, int slots, int sms, int64_t rows, int* threads, int* blocks, int* bytes) {
  *threads = stream_threads(vectors);
  *bytes = stream_bytes(slots, *threads);
  const int by_threads = kStreamThreads / *threads, by_bytes = kSmBytes / (*bytes + kBlockBytes);
  const int64_t most = (int64_t)sms * (by_threads < by_bytes ? by_threads : by_bytes);
  *blocks = (int)(rows < most ? rows : most);
  DGL_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamBytes));
  return DG_OK;
}

template <int XP, int RP, bool OUT8>
int stream_norm(const Args& p, bool vec, int sms, cudaStream_t s) {
  int threads, blocks, bytes;
  auto* kernel = layer_norm_stream_kernel<XP, RP, OUT8, kVectors>;
  if constexpr (XP == 1 && RP < 2)
    if (p.hidden % (32 * 8 * kStreamVecs) == 0) kernel = layer_norm_stream_kernel<XP, RP, OUT8, kFull>;
  if constexpr (!OUT8)
    if (!vec) kernel = layer_norm_stream_kernel<XP, RP, false, kEdges>;
  if (int rc = stream_shape(kernel, row_vectors(p.hidden, vec), XP + RP, sms, p.rows, &threads, &blocks, &bytes))
    return rc;
  if (!vec) blocks = blocks / 8 * 8;  // (each block's rows start at the same place in a vector)
  return dgl::launch(kernel, dim3(blocks), dim3(threads), bytes, s, p);
}

template <int XP, int RP>
int run_spread(const Args& p, cudaStream_t s) {
  const int n = p.hidden <= 1024 ? 4 : 16, threads = round32((p.hidden + n - 1) / n), per = threads == 32 ? 4 : 1;
  return dgl::launch(n == 4 ? layer_norm_spread_kernel<XP == 2, RP, 4> : layer_norm_spread_kernel<XP == 2, RP, 16>,
                     dim3((unsigned)((p.rows + per - 1) / per)), dim3(threads, per), 0, s, p);
}

// vec: whole vectors; dense: else, rows that follow one another by their length from aligned bases.
template <int XP, int RP, bool OUT8>
int run_norm(const Args& p, bool vec, bool dense, int sms, cudaStream_t s) {
  // Many long rows are streamed; few rows take as many threads as they have vectors,
  // for the shortest chain of loads.
  const int vectors = row_vectors(p.hidden, vec);
  const bool fits = vectors <= 2048 && stream_bytes(XP + RP, stream_threads(vectors)) <= kStreamBytes;
  if (!vec) {
    if constexpr (!OUT8) {
      // 2047 x 5003: 20.8 us element by element
      if (dense && fits && p.rows > 2 * sms && vectors >= 64) return stream_norm<XP, RP, false>(p, false, sms, s);
      if (p.hidden <= 16384) return run_spread<XP, RP>(p, s);
      return dgl::launch(layer_norm_long_kernel<false, false>, dim3((unsigned)p.rows), dim3(1024), 0, s, p);
    }
    return fail(DG_ERR_ARG, "8-bit blocks need rows of whole 16-byte vectors");
  }
  const int n = vectors;
  if (fits && p.rows > 2 * sms && n >= 256) return stream_norm<XP, RP, OUT8>(p, true, sms, s);
  auto launch_rows = [&](auto* kernel, int threads) {
    const int per = threads == 32 ? 4 : 1;  // one warp per row: four rows to a block
    return dgl::launch(kernel, dim3((unsigned)((p.rows + per - 1) / per)), dim3(threads, per), 0, s, p);
  };
  if (n <= 1024) return launch_rows(layer_norm_kernel<1, OUT8>, round32(n));
  if (n <= 2048) return launch_rows(layer_norm_kernel<2, OUT8>, round32((n + 1) / 2));
  if (n <= 4096) return launch_rows(layer_norm_kernel<8, OUT8>, round32((n + 7) / 8));
  return dgl::launch(layer_norm_long_kernel<true, OUT8>, dim3((unsigned)p.rows), dim3(1024), 0, s, p);
}

template <int XP, int RP>
int run_out(const Args& p, bool vec, bool dense, int sms, cudaStream_t s) {
  return p.y ? run_norm<XP, RP, false>(p, vec, dense, sms, s) : run_norm<XP, RP, true>(p, vec, dense, sms, s);
}

// A matrix whose rows start at the same place in a vector as those of a densely packed one (or none).
bool like_dense(const void* p, int64_t ld, int64_t hidden) { return !p || (aligned16(p) && (ld - hidden) % 8 == 0); }

// ----------------------------------------------------------------- gradient

struct GradArgs {
  const void *dy, *h, *dh;
  const float *scales;  // of an 8-bit h
  int64_t s_row, s_block;
  Affine affine;
  const float *mean, *rstd;
  void *dx, *dweight, *dbias;
  float* partial;  // weight, then bias: blocks x hidden each; null without them
  int64_t ld_dy, ld_h, ld_dh, rows;
  int hidden, w_f32, b_f32;
};

// The type of h: bf16, fp32, or 8-bit blocks of 1 x 128 (of e4m3 and of e5m2 values).
enum { kH16 = 0, kH32 = 1, kH8 = 2, kH8wide = 3 };
__host__ __device__ constexpr bool in_blocks(int ht) { return ht >= kH8; }

// 16-byte slots of a vector: dy, h, and the gradient that reaches h on its other way.
template <int HT, bool HAS_DH>
__host__ __device__ constexpr int grad_parts() {
  return kStreamVecs * (1 + (HT == kH32 ? 2 : 1) * (HAS_DH ? 2 : 1));
}
// Two stages; three, with the next row's sums ahead of this one's output, for rows in
// blocks (8192 x 16384 159 us instead of 185; of 16 bits 164 instead of 146).
template <int HT, bool HAS_DH>
__host__ __device__ constexpr int grad_stages() {
  return in_blocks(HT) && !HAS_DH ? 3 : 2;
}
// Shared memory of a group of threads: their stages and their weights, and the scales of an 8-bit h's rows.
template <int HT, bool HAS_DH>
__host__ __device__ constexpr int grad_bytes(int threads) {
  return (grad_stages<HT, HAS_DH>() * grad_parts<HT, HAS_DH>() + kStreamVecs) * 16 * threads +
         (in_blocks(HT) ? (grad_stages<HT, HAS_DH>() + 1) * threads : 0);  // (a float for 128 values, of which a thread has 32)
}

template <int BYTES>
__device__ __forceinline__ void copy_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// Rows streamed like the forward's, in the same two steps: the sums, and dx, for
// which the row is read from its slots again, which leaves registers to the weight
// and the two gradients that are summed over the block's rows.  With
// e = h - mean: mean(g xh) = rstd mean(g e), dx = rstd (dy w - mean(g) - e (rstd mean(g xh))).
template <int HT, bool HAS_DH, int MODE>
__global__ void __launch_bounds__(kStreamThreads, 1) layer_norm_grad_stream_kernel(const __grid_constant__ GradArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 parts[2][16];  // (a group's warps)
  constexpr int NV = kStreamVecs, HP = HT == kH32 ? 2 : 1, PER = 1 + HP * (HAS_DH ? 2 : 1), hsz = HT == kH32 ? 4 : 2;
  constexpr int STAGES = grad_stages<HT, HAS_DH>();
  constexpr bool PIPE = STAGES > 2;
  constexpr int PARTS = grad_parts<HT, HAS_DH>();
  // every thread takes all of its vectors, zeros past the row, and only stores ask (4099 x 8208 71 us, now 55); not where a
  // row's scales end with it, nor where the vectors at its ends are clipped (2047 x 5003 with d_residual 34 us, 31 as it is)
  constexpr bool ALL = MODE == kVectors && !in_blocks(HT);
  const Slots<PARTS> slots{smem + threadIdx.y * grad_bytes<HT, HAS_DH>(blockDim.x)};
  float* const row_scales = reinterpret_cast<float*>(slots.base + (STAGES * PARTS + NV) * 16 * blockDim.x);
  // behind the stages: the weight's vectors of this thread, in bf16 (in registers they crowded out the row's)
  auto weight_slot = [&](int k) { return slots.at(0, STAGES * PARTS + k); };
  begin_kernel();
  // this group of threads takes the rows unit, unit + units, ...
  const uint32_t unit = blockIdx.x * blockDim.y + threadIdx.y, units = gridDim.x * blockDim.y, rows = (uint32_t)p.rows;
  const int shift = MODE == kEdges ? (int)((unit & 7u) * (p.hidden & 7u) & 7u) : 0;
  const int step = blockDim.x * 8, i0 = threadIdx.x * 8 - shift, warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto in = [&](int k) { return MODE == kFull || i0 + k * step < p.hidden; };
  auto copy = [&](int stage, int part, const uint8_t* src, int i, int size) {  // (as in the forward)
    const int bytes = MODE == kFull ? 16 : MODE == kEdges ? min(max((p.hidden - i) * size, 0), 16) : i < p.hidden ? 16 : 0;
    if (MODE != kFull && bytes == 0) src = static_cast<const uint8_t*>(p.dy);
    if (size == 4)
      slots.fetch_half(stage, part, src, bytes);
    else if (MODE == kFull)
      slots.fetch(stage, part, src);
    else
      slots.fetch(stage, part, src, bytes);
  };
  // this thread's place in the next row to fetch
  constexpr int HB = in_blocks(HT) ? 1 : hsz;  // bytes of a value of h
  uint32_t next = unit;
  int scale_next = 0;
  const uint8_t* dy_next = static_cast<const uint8_t*>(p.dy) + ((int64_t)next * p.ld_dy + i0) * 2;
  const uint8_t* h_next = static_cast<const uint8_t*>(p.h) + ((int64_t)next * p.ld_h + i0) * HB;
  const uint8_t* dh_next = HAS_DH ? static_cast<const uint8_t*>(p.dh) + ((int64_t)next * p.ld_dh + i0) * hsz : nullptr;
  auto fetch = [&](int stage) {
    if (next < rows) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (ALL || in(k)) {
          const int i = i0 + k * step;
          copy(stage, k * PER, dy_next + k * step * 2, i, 2);
          if constexpr (in_blocks(HT)) {
            copy_small<8>((uint32_t)__cvta_generic_to_shared(slots.at(stage, k * PER + 1)), h_next + k * step);
          } else {
#pragma unroll
            for (int q = 0; q < HP; ++q) copy(stage, k * PER + 1 + q, h_next + k * step * HB + 16 * q, i + 4 * q, hsz);
          }
          if constexpr (HAS_DH)
#pragma unroll
            for (int q = 0; q < HP; ++q) copy(stage, k * PER + 1 + HP + q, dh_next + k * step * hsz + 16 * q, i + 4 * q, hsz);
        }
      }
    }
    // a row's scales: one each for its first threads, which all read (so there is a place more than there are stages: the
    // one written here was last read before a barrier)
    if (in_blocks(HT)) {
      if (next < rows && (int)threadIdx.x * 128 < p.hidden)
        copy_small<4>((uint32_t)__cvta_generic_to_shared(row_scales + scale_next * (blockDim.x / 4) + threadIdx.x),
                      p.scales + (int64_t)next * p.s_row + threadIdx.x * p.s_block);
      scale_next = scale_next == STAGES ? 0 : scale_next + 1;
    }
    next += units;
    dy_next += units * p.ld_dy * 2, h_next += units * p.ld_h * HB;
    if (HAS_DH) dh_next += units * p.ld_dh * hsz;
    copies_commit();
  };
  // a row's mean (negated) and deviation, fetched ahead of their use, and the place of its scales
  struct Known {
    float m, r;
    int at;
  };
  int scale_known = 0;
  auto known = [&](uint32_t row, Known& n) {
    if (row < rows) n.m = -__ldg(p.mean + row), n.r = __ldg(p.rstd + row);
    if (in_blocks(HT)) {
      n.at = scale_known * (blockDim.x / 4);
      scale_known = scale_known == STAGES ? 0 : scale_known + 1;
    }
  };
  Eight dw[NV], db[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = i0 + k * step;
    uint4 w16 = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    if (in(k) && p.affine.w && !p.affine.w_f32) {
      Eight v;
      load_row8<MODE>(false, p.affine.w, i, p.hidden, v);
      w16 = v.to_bf16();
    }
    *weight_slot(k) = w16;
    dw[k].zero(), db[k].zero();
  }
  auto wide = [&](bool f32, int stage, int slot, Eight& v) {
    if (f32)
      v.from_f32(*slots.at(stage, slot), *slots.at(stage, slot + 1));
    else
      v.from_bf16(*slots.at(stage, slot));
  };
  // dy, h - mean and the weight of vector k
  auto read = [&](const Known& n, int stage, int k, uint64_t minus, Eight& dy, Eight& e, Eight& w) {
    wide(false, stage, k * PER, dy);
    if constexpr (in_blocks(HT)) {
      const float s = row_scales[n.at + ((i0 + k * step) >> 7)];
      const uint64_t scale = pair_of(s, s);
      float f[8];
      unpack_fp8(*reinterpret_cast<const uint2*>(slots.at(stage, k * PER + 1)), HT == kH8 ? __NV_E4M3 : __NV_E5M2, f);
      e.from_floats(f);
#pragma unroll
      for (int j = 0; j < 4; ++j) e.p[j] = fma2(e.p[j], scale, minus);
    } else {
      wide(HT == kH32, stage, k * PER + 1, e);
#pragma unroll
      for (int j = 0; j < 4; ++j) e.p[j] = add2(e.p[j], minus);
    }
    const int i = i0 + k * step;
    if (MODE == kEdges && (i < 0 || i + 8 > p.hidden)) clip(dy, i, p.hidden), clip(e, i, p.hidden);
    w.from_bf16(*weight_slot(k));
    if (p.affine.w_f32 && in(k)) load_row8<MODE>(true, p.affine.w, i, p.hidden, w);
  };
  const float inv_hidden = 1.f / (float)p.hidden;
  const int first_warp = threadIdx.y * warps;
  auto group_sync = [&]() {
    if (blockDim.y == 1)
      __syncthreads();
    else if (warps == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.y), "r"((int)blockDim.x) : "memory");
  };
  auto sums = [&](const Known& n, int stage, int flip) {
    const uint64_t minus = pair_of(n.m, n.m), rstd = pair_of(n.r, n.r);
    uint64_t s1 = 0, s2 = 0;
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (ALL || in(k)) {
        Eight dy, e, w;
        read(n, stage, k, minus, dy, e, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          db[k].p[j] = add2(db[k].p[j], dy.p[j]);
          dw[k].p[j] = fma2(mul2(dy.p[j], rstd), e.p[j], dw[k].p[j]);
          const uint64_t g = mul2(dy.p[j], w.p[j]);
          s1 = add2(s1, g);
          s2 = fma2(g, e.p[j], s2);
        }
      }
    float a = sum_of(s1), b = sum_of(s2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o), b += __shfl_xor_sync(0xffffffffu, b, o);
    if (lane == 0) parts[flip][first_warp + warp] = make_float2(a, b * n.r);
  };
  auto output = [&](const Known& n, uint32_t row, int stage, int flip) {
    const uint64_t minus = pair_of(n.m, n.m), rstd = pair_of(n.r, n.r);
    float2 s = parts[flip][first_warp + (lane < warps ? lane : 0)];
    if (lane >= warps) s = make_float2(0.f, 0.f);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s.x += __shfl_xor_sync(0xffffffffu, s.x, o), s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    const float c1 = -s.x * inv_hidden, c2 = -n.r * (s.y * inv_hidden);
    const uint64_t m1 = pair_of(c1, c1), m2 = pair_of(c2, c2);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (ALL || in(k)) {
        Eight dy, e, w, d;
        read(n, stage, k, minus, dy, e, w);
        if constexpr (HAS_DH) wide(HT == kH32, stage, k * PER + 1 + HP, d);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t t = fma2(e.p[j], m2, fma2(dy.p[j], w.p[j], m1));
          if constexpr (HAS_DH)
            d.p[j] = fma2(t, rstd, d.p[j]);
          else
            d.p[j] = mul2(t, rstd);
        }
        if (in(k)) store_row8<MODE>(HT == kH32, p.dx, (int64_t)row * p.hidden, i0 + k * step, p.hidden, d);
      }
    }
  };
  Known now, then;
  known(unit, now);
#pragma unroll
  for (int s = 0; s < STAGES; ++s) fetch(s);
  int stage = 0, flip = 0;
  auto after = [](int s) { return s + 1 == STAGES ? 0 : s + 1; };
  // (an 8-bit h's scales come through other threads' copies: a barrier after every wait)
  if (PIPE) {
    known(unit + units, then);
    copies_wait<STAGES - 2>();
    if (in_blocks(HT)) group_sync();
    if (unit < rows) sums(now, 0, 0);
    group_sync();
  }
  for (uint32_t row = unit; row < rows; row += units, flip ^= 1) {
    if constexpr (PIPE) {
      if (row + units < rows) sums(then, after(stage), flip ^ 1);
      output(now, row, stage, flip);
      now = then;
      known(row + 2 * units, then);
      fetch(stage);
      copies_wait<STAGES - 2>();
      group_sync();
    } else {
      known(row + units, then);
      copies_wait<STAGES - 1>();
      if (in_blocks(HT)) group_sync();
      sums(now, stage, flip);
      group_sync();
      output(now, row, stage, flip);
      now = then;
      fetch(stage);
    }
    stage = after(stage);
  }
  copies_wait<0>();
  if (!p.partial) return;
  // the groups' gradients side by side in shared memory, added up in their order to one row of `partial` for the block
  // (weight rows first, then the bias's).  A place is left out after every eight values: threads that are eight apart
  // write to different banks (without: 3 to 6 us a call).
  auto place = [](int c) { return c + (c >> 3); };
  __syncthreads();
  static_assert(grad_bytes<HT, HAS_DH>(32) >= 2 * 4 * (32 * NV * 8 * 9 / 8), "a group's gradients fit into its stages");
  float* const hand = reinterpret_cast<float*>(smem);
  const int each = place(p.hidden), all = blockDim.x * blockDim.y;
#pragma unroll
  for (int k = 0; k < NV; ++k)
    if (in(k)) {
      const int i = i0 + k * step;
      float* to = hand + threadIdx.y * 2 * each;
      float a[8], b[8];
      dw[k].to_floats(a), db[k].to_floats(b);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (MODE != kEdges || (i + j >= 0 && i + j < p.hidden)) to[place(i + j)] = a[j], to[each + place(i + j)] = b[j];
    }
  __syncthreads();
#pragma unroll 1
  for (int bias = 0; bias < 2; ++bias) {
    float* to = p.partial + (int64_t)(bias * gridDim.x + blockIdx.x) * p.hidden;
    const float* from = hand + bias * each;
#pragma unroll 4
    for (int c = threadIdx.y * blockDim.x + threadIdx.x; c < p.hidden; c += all) {
      float v = from[place(c)];
#pragma unroll 4
      for (int g = 1; g < blockDim.y; ++g) v += from[g * 2 * each + place(c)];
      to[c] = v;
    }
  }
}

// Rows of any alignment, element by element: N values per thread.
template <bool F32, int N, bool HAS_DH>
__global__ void __launch_bounds__(512) layer_norm_grad_kernel(const __grid_constant__ GradArgs p) {
  __shared__ float part[2][66];
  begin_kernel();
  float dw[N], db[N], w[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    dw[k] = db[k] = 0.f;
    float v[1] = {1.f};
    const int i = threadIdx.x + k * blockDim.x;
    if (p.affine.w && i < p.hidden) load_any<1>(p.affine.w_f32 != 0, p.affine.w, i, v);
    w[k] = v[0];
  }
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
    const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
    Spread<false, N> dy;
    Spread<F32, N> h, dh;
    dy.load(p.dy, row * p.ld_dy, p.hidden);
    h.load(p.h, row * p.ld_h, p.hidden);
    if constexpr (HAS_DH) dh.load(p.dh, row * p.ld_dh, p.hidden);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {  // (dy is 0 past the row)
      const float d = dy.at(k, p.hidden), xh = (h.at(k, p.hidden) - mean) * rstd;
      if ((int)(threadIdx.x + k * blockDim.x) < p.hidden) {
        db[k] += d;
        dw[k] = fmaf(d, xh, dw[k]);
        s1 += d * w[k];
        s2 = fmaf(d * w[k], xh, s2);
      }
    }
    const float2 s = row_sum2(s1, s2, part[flip]);
    const float m1 = s.x / (float)p.hidden, m2 = s.y / (float)p.hidden;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      float d[1] = {0.f};
      if constexpr (HAS_DH) d[0] = dh.at(k, p.hidden);
      d[0] = fmaf(rstd, fmaf(dy.at(k, p.hidden), w[k], -m1) - (h.at(k, p.hidden) - mean) * rstd * m2, d[0]);
      if (i < p.hidden) {
        if constexpr (F32)
          store_f32<1>(p.dx, row * p.hidden + i, d);
        else
          store_bf16<1>(p.dx, row * p.hidden + i, d);
      }
    }
  }
  if (p.partial)
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = threadIdx.x + k * blockDim.x;
      if (i < p.hidden) {
        p.partial[(int64_t)blockIdx.x * p.hidden + i] = dw[k];
        p.partial[(int64_t)(gridDim.x + blockIdx.x) * p.hidden + i] = db[k];
      }
    }
}

// Rows longer than the other kernels hold (above 16384 values; of fp32 rows with the
// gradient that reaches h, whose stages are the largest, above 10240): two passes over
// each row, a value at a time; the weight's and the bias's gradients accumulate in the
// block's rows of `partial`.  Such fp32 rows: 8192 x 10248 786 us (10240 streamed: 296),
// 8192 x 16384 1165.
template <int HT, bool HAS_DH>
__global__ void __launch_bounds__(1024) layer_norm_grad_long_kernel(const __grid_constant__ GradArgs p) {
  __shared__ float part[2][66];
  begin_kernel();
  float* mw = p.partial ? p.partial + (int64_t)blockIdx.x * p.hidden : nullptr;
  float* mb = p.partial ? p.partial + (int64_t)(gridDim.x + blockIdx.x) * p.hidden : nullptr;
  if (p.partial)
    for (int64_t i = threadIdx.x; i < p.hidden; i += blockDim.x) mw[i] = mb[i] = 0.f;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, flip ^= 1) {
    const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
    auto value = [&](int64_t i, float& dy, float& xh, float& w) {
      float d[1], h[1], v[1] = {1.f};
      load_bf16<1>(p.dy, row * p.ld_dy + i, d);
      if constexpr (in_blocks(HT))
        h[0] = unpack_fp8x2(static_cast<const uint8_t*>(p.h)[row * p.ld_h + i], HT == kH8 ? __NV_E4M3 : __NV_E5M2).x *
               __ldg(p.scales + row * p.s_row + (i >> 7) * p.s_block);
      else
        load_any<1>(HT == kH32, p.h, row * p.ld_h + i, h);
      if (p.affine.w) load_any<1>(p.affine.w_f32 != 0, p.affine.w, i, v);
      dy = d[0], xh = (h[0] - mean) * rstd, w = v[0];
    };
    float s1 = 0.f, s2 = 0.f;
    for (int64_t i = threadIdx.x; i < p.hidden; i += blockDim.x) {
      float dy, xh, w;
      value(i, dy, xh, w);
      if (p.partial) mw[i] = fmaf(dy, xh, mw[i]), mb[i] += dy;
      s1 += dy * w;
      s2 = fmaf(dy * w, xh, s2);
    }
    const float2 s = row_sum2(s1, s2, part[flip]);
    const float m1 = s.x / (float)p.hidden, m2 = s.y / (float)p.hidden;
    for (int64_t i = threadIdx.x; i < p.hidden; i += blockDim.x) {
      float dy, xh, w, d[1] = {0.f};
      value(i, dy, xh, w);
      if constexpr (HAS_DH) load_any<1>(HT == kH32, p.dh, row * p.ld_dh + i, d);
      d[0] = fmaf(rstd, fmaf(dy, w, -m1) - xh * m2, d[0]);
      if constexpr (HT == kH32)
        store_f32<1>(p.dx, row * p.hidden + i, d);
      else
        store_bf16<1>(p.dx, row * p.hidden + i, d);
    }
  }
}

// The weight's and the bias's gradient (blockIdx.y): sums over the blocks' partial
// rows, in a fixed order: 32 columns x kSumRows threads, each thread a strided share of
// the rows, then one after the other.  (32 threads a column: two rounds of blocks
// for rows of 5003 values.)
constexpr int kSumRows = 16;
__global__ void __launch_bounds__(32 * kSumRows) layer_norm_weight_grad_kernel(const __grid_constant__ GradArgs p, int blocks) {
  __shared__ float s[kSumRows][32];
  begin_kernel();
  const float* partial = p.partial + (blockIdx.y ? (int64_t)blocks * p.hidden : 0);
  const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
  float v = 0.f;
  if (col < p.hidden)
#pragma unroll 8
    for (int b = threadIdx.y; b < blocks; b += kSumRows) v += __ldcg(partial + (int64_t)b * p.hidden + col);
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  void* to = blockIdx.y ? p.dbias : p.dweight;
  if (threadIdx.y != 0 || col >= p.hidden || !to) return;
#pragma unroll
  for (int k = 1; k < kSumRows; ++k) v += s[k][threadIdx.x];
  if (blockIdx.y ? p.b_f32 : p.w_f32)
    static_cast<float*>(to)[col] = v;
  else
    static_cast<__nv_bfloat16*>(to)[col] = __float2bfloat16_rn(v);
}

// Blocks of the gradient kernels: a fixed bound that the workspace is sized by.
// (Rows of more than 4096 values take the threads of a whole SM, or of half of one.)
int64_t most_blocks(int64_t rows, int64_t hidden) {
  const int64_t most = hidden <= 4096 ? 1216 : 304;
  return rows < most ? rows : most;
}

// `fill` blocks fill the SMs; a block takes four rows at least where there are
// enough of them, so that the partial sums stay small beside the rows.
int grad_blocks(int64_t rows, int64_t hidden, int sms, int64_t fill) {
  const int64_t want = rows / 4 > sms ? rows / 4 : sms, most = most_blocks(rows, hidden);
  const int64_t n = want < fill ? want : fill;
  return (int)(n < most ? n : most);
}

// vec, dense: as in the forward.
template <int HT, bool HAS_DH>
int run_grad(const GradArgs& p, bool vec, bool dense, int sms, cudaStream_t s) {
  const int n = row_vectors(p.hidden, vec);
  int blocks, rc;
  // (2047 x 5003 element by element: 45 us)
  const bool edges = !in_blocks(HT) && !vec && dense && p.rows >= 8 && n >= 64;
  if ((vec || edges) && n <= 2048 && grad_bytes<HT, HAS_DH>(stream_threads(n)) <= kStreamBytes) {
    auto* kernel = layer_norm_grad_stream_kernel<HT, HAS_DH, kVectors>;
    if constexpr (HT != kH32)
      if (p.hidden % (32 * 8 * kStreamVecs) == 0) kernel = layer_norm_grad_stream_kernel<HT, HAS_DH, kFull>;
    if constexpr (!in_blocks(HT))
      if (!vec) kernel = layer_norm_grad_stream_kernel<HT, HAS_DH, kEdges>;
    DGL_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamBytes));
    const int threads = stream_threads(n), bytes = grad_bytes<HT, HAS_DH>(threads);
    // groups of threads, each with rows of its own, that fill an SM, and one block to an SM: its groups add their
    // weight gradients up, so that fewer partial rows go through memory (4096 x 1024: 1024 blocks of one warp
    // took 17.6 us, most of it there)
    const int most = kStreamThreads / threads < kStreamBytes / bytes ? kStreamThreads / threads : kStreamBytes / bytes;
    const int64_t want = (p.rows + sms - 1) / sms;
    const int groups = (int)(want < most ? want : most);
    const int64_t n_blocks = (p.rows + groups - 1) / groups;
    const int64_t fill = sms < most_blocks(p.rows, p.hidden) ? sms : most_blocks(p.rows, p.hidden);
    blocks = (int)(n_blocks < fill ? n_blocks : fill);
    if (!vec) blocks = blocks / 8 * 8;  // (eight rows at least: a group's rows start at the same place in a vector)
    rc = dgl::launch(kernel, dim3(blocks), dim3(threads, groups), bytes * groups, s, p);
  } else {
    const bool small = !in_blocks(HT) && p.hidden <= 1024, regs = !in_blocks(HT) && p.hidden <= 8192;
    const int threads = small ? round32((p.hidden + 3) / 4) : regs ? round32((p.hidden + 15) / 16) : 1024;
    blocks = grad_blocks(p.rows, p.hidden, sms, (int64_t)sms * (threads < 512 ? 512 / threads : 1));
    auto* kernel = layer_norm_grad_long_kernel<HT, HAS_DH>;
    if constexpr (!in_blocks(HT)) {
      if (small)
        kernel = layer_norm_grad_kernel<HT == kH32, 4, HAS_DH>;
      else if (regs)
        kernel = layer_norm_grad_kernel<HT == kH32, 16, HAS_DH>;
    }
    rc = dgl::launch(kernel, dim3(blocks), dim3(threads), 0, s, p);
  }
  if (rc != DG_OK || !p.partial) return rc;
  return dgl::launch(layer_norm_weight_grad_kernel, dim3((unsigned)((p.hidden + 31) / 32), 2), dim3(32, kSumRows), 0, s, p, blocks);
}

// Rows of no values: the deviation's reciprocal and the mean of nothing, a NaN.
__global__ void __launch_bounds__(256) layer_norm_of_nothing_kernel(float* mean, float* rstd, int64_t rows) {
  begin_kernel();
  const int64_t row = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (row >= rows) return;
  if (mean) mean[row] = __uint_as_float(0x7fc00000u);
  if (rstd) rstd[row] = __uint_as_float(0x7fc00000u);
}

int check_affine(const void* weight, int weight_type, const void* bias, int bias_type) {
  if ((weight && !bf16_or_f32(weight_type)) || (bias && !bf16_or_f32(bias_type)))
    return fail(DG_ERR_ARG, "the weight and the bias are bf16 or fp32");
  return DG_OK;
}

}  // namespace

extern "C" int dg_layer_layer_norm(const void* x, int64_t ld_x, int x_type, const void* residual, int64_t ld_residual,
                                   int residual_type, const void* weight, int weight_type, const void* bias, int bias_type,
                                   void* y, int y_type, float* y_scales, int64_t ys_row, int64_t ys_block, void* sum_out,
                                   int64_t ld_sum, void* kept, int kept_type, float* kept_scales, int64_t ks_row, int64_t ks_block,
                                   float* mean_out, float* rstd_out, int64_t rows, int64_t hidden, float eps, void* stream) {
  if (rows < 0 || hidden < 0 || rows > INT32_MAX || hidden > INT32_MAX - 8192)
    return fail(DG_ERR_ARG, "rows %lld, hidden %lld out of range", (long long)rows, (long long)hidden);
  if (!bf16_or_f32(x_type) || (residual && !bf16_or_f32(residual_type))) return fail(DG_ERR_ARG, "x and the residual are bf16 or fp32");
  if (int rc = check_affine(weight, weight_type, bias, bias_type)) return rc;
  const bool out8 = is_fp8(y_type);
  if (!out8 && y_type != DG_TYPE_BF16) return fail(DG_ERR_ARG, "y is bf16, e4m3 or e5m2 (got type %d)", y_type);
  if (kept && !is_fp8(kept_type)) return fail(DG_ERR_ARG, "kept rows are e4m3 or e5m2 (got type %d)", kept_type);
  if (!(eps >= 0.f)) return fail(DG_ERR_ARG, "eps must not be negative");
  if ((out8 || kept) && hidden % 16) return fail(DG_ERR_SHAPE, "8-bit blocks need hidden %% 16 == 0 (got %lld)", (long long)hidden);
  if (rows == 0) return DG_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (hidden == 0) {
    if (!mean_out && !rstd_out) return DG_OK;
    return dgl::launch(layer_norm_of_nothing_kernel, dim3((unsigned)((rows + 255) / 256)), dim3(256), 0, s, mean_out, rstd_out, rows);
  }
  if (!x || !y) return fail(DG_ERR_ARG, "x and y must not be null");
  if ((residual != nullptr) != (sum_out != nullptr)) return fail(DG_ERR_ARG, "a residual and its sum come together");
  if ((out8 && !y_scales) || (kept && !kept_scales)) return fail(DG_ERR_ARG, "8-bit blocks need their scales");
  int sms = 0;
  if (int rc = sm_count(&sms)) return rc;
  const int64_t xsz = x_type == DG_TYPE_F32 ? 4 : 2, rsz = residual_type == DG_TYPE_F32 ? 4 : 2;
  const bool vec = hidden % 8 == 0 && rows16(x, ld_x, xsz) && rows16(residual, ld_residual, rsz) && rows16(sum_out, ld_sum, rsz) &&
                   (!weight || aligned16(weight)) && (!bias || aligned16(bias)) && aligned16(y);
  if ((out8 || kept) && (!vec || (kept && !aligned16(kept))))
    return fail(DG_ERR_ARG, "8-bit blocks need 16-byte aligned pointers and pitches");
  Args p{};
  p.x = x, p.residual = residual, p.sum = sum_out, p.y = out8 ? nullptr : y;
  p.y8 = Blocks{out8 ? static_cast<uint8_t*>(y) : nullptr, y_scales, ys_row, ys_block, y_type == DG_TYPE_E5M2};
  p.kept = Blocks{static_cast<uint8_t*>(kept), kept_scales, ks_row, ks_block, kept_type == DG_TYPE_E5M2};
  p.mean = mean_out, p.rstd = rstd_out;
  p.affine = Affine{weight, bias, weight && weight_type == DG_TYPE_F32, bias && bias_type == DG_TYPE_F32};
  p.ld_x = ld_x, p.ld_residual = ld_residual, p.ld_sum = ld_sum, p.rows = rows;
  p.hidden = (int)hidden, p.x_f32 = x_type == DG_TYPE_F32, p.r_f32 = residual_type == DG_TYPE_F32, p.eps = eps;
  const bool dense = like_dense(x, ld_x, hidden) && like_dense(residual, ld_residual, hidden) && like_dense(sum_out, ld_sum, hidden) &&
                     aligned16(y);
  const int rp = !residual ? 0 : residual_type == DG_TYPE_F32 ? 2 : 1;
  if (x_type == DG_TYPE_F32)
    return rp == 0 ? run_out<2, 0>(p, vec, dense, sms, s) : rp == 1 ? run_out<2, 1>(p, vec, dense, sms, s) : run_out<2, 2>(p, vec, dense, sms, s);
  return rp == 0 ? run_out<1, 0>(p, vec, dense, sms, s) : rp == 1 ? run_out<1, 1>(p, vec, dense, sms, s) : run_out<1, 2>(p, vec, dense, sms, s);
}

extern "C" size_t dg_layer_layer_norm_backward_workspace(int64_t rows, int64_t hidden) {
  if (rows <= 0 || hidden <= 0) return 0;
  return 2 * (size_t)most_blocks(rows, hidden) * (size_t)hidden * sizeof(float);
}

extern "C" int dg_layer_layer_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, int h_type,
                                            const float* h_scales, int64_t hs_row, int64_t hs_block, const void* weight,
                                            int weight_type, const float* mean, const float* rstd, const void* dh, int64_t ld_dh,
                                            void* dx, void* dweight, void* dbias, int dbias_type, void* workspace, int64_t rows,
                                            int64_t hidden, void* stream) {
  if (rows < 0 || hidden < 0 || rows > INT32_MAX || hidden > INT32_MAX - 8192)
    return fail(DG_ERR_ARG, "rows %lld, hidden %lld out of range", (long long)rows, (long long)hidden);
  const bool h8 = is_fp8(h_type);
  if (!h8 && !bf16_or_f32(h_type)) return fail(DG_ERR_ARG, "h is bf16, fp32, e4m3 or e5m2 (got type %d)", h_type);
  if (int rc = check_affine(weight, weight_type, dbias, dbias_type)) return rc;
  if (dweight && !bf16_or_f32(weight_type)) return fail(DG_ERR_ARG, "the weight's gradient is bf16 or fp32");
  if (h8 && hidden % 16) return fail(DG_ERR_SHAPE, "8-bit blocks need hidden %% 16 == 0 (got %lld)", (long long)hidden);
  if (hidden == 0) return DG_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dweight) DGL_CUDA(cudaMemsetAsync(dweight, 0, (size_t)hidden * (weight_type == DG_TYPE_F32 ? 4 : 2), s));
    if (dbias) DGL_CUDA(cudaMemsetAsync(dbias, 0, (size_t)hidden * (dbias_type == DG_TYPE_F32 ? 4 : 2), s));
    return DG_OK;
  }
  if (!dy || !h || !mean || !rstd || !dx || (h8 && !h_scales)) return fail(DG_ERR_ARG, "a required pointer is null");
  const bool sums = dweight || dbias;
  if (sums && (!workspace || !aligned16(workspace))) return fail(DG_ERR_ARG, "the workspace must be there and 16-byte aligned");
  int sms = 0;
  if (int rc = sm_count(&sms)) return rc;
  const int64_t hsz = h_type == DG_TYPE_F32 ? 4 : h8 ? 1 : 2, dsz = h_type == DG_TYPE_F32 ? 4 : 2;
  const bool vec = hidden % 8 == 0 && rows16(dy, ld_dy, 2) && rows16(h, ld_h, hsz) && rows16(dh, ld_dh, dsz) &&
                   (!weight || aligned16(weight)) && aligned16(dx);
  GradArgs p{};
  p.dy = dy, p.h = h, p.dh = dh, p.scales = h_scales, p.s_row = hs_row, p.s_block = hs_block;
  p.affine = Affine{weight, nullptr, weight && weight_type == DG_TYPE_F32, 0};
  p.mean = mean, p.rstd = rstd, p.dx = dx, p.dweight = dweight, p.dbias = dbias;
  p.partial = sums ? static_cast<float*>(workspace) : nullptr;
  p.ld_dy = ld_dy, p.ld_h = ld_h, p.ld_dh = ld_dh, p.rows = rows, p.hidden = (int)hidden;
  p.w_f32 = weight_type == DG_TYPE_F32, p.b_f32 = dbias_type == DG_TYPE_F32;
  const bool dense = like_dense(dy, ld_dy, hidden) && like_dense(h, ld_h, hidden) && like_dense(dh, ld_dh, hidden) && aligned16(dx);
  if (h_type == DG_TYPE_E4M3) return dh ? run_grad<kH8, true>(p, vec, false, sms, s) : run_grad<kH8, false>(p, vec, false, sms, s);
  if (h8) return dh ? run_grad<kH8wide, true>(p, vec, false, sms, s) : run_grad<kH8wide, false>(p, vec, false, sms, s);
  if (h_type == DG_TYPE_F32) return dh ? run_grad<kH32, true>(p, vec, dense, sms, s) : run_grad<kH32, false>(p, vec, dense, sms, s);
  return dh ? run_grad<kH16, true>(p, vec, dense, sms, s) : run_grad<kH16, false>(p, vec, dense, sms, s);
}
