// mx4_gemm.cu -- product of two microscaled 4-bit tensors (dg_layer_mx4_matmul).
//
//   D[m, n] = sum over 32-blocks j of 2^(ea[m, j] + eb[n, j]) sum_{k in j} a[m, k] b[n, k]
//
// The block-scaled tensor core instruction (tcgen05.mma kind::mxf4, K = 64, two
// scales per row) applies the scales itself: codes stay packed in shared
// memory, the scales go to tensor memory.  CTA pairs, D^T orientation
// (ptx.cuh): P = b (features), Q = a (rows); a tile is 256 features x up to 192
// rows, so that two fp32 accumulators (384 columns) leave tensor memory for the
// scales of four K blocks.
//
// Scales of 128 rows x 128 columns are one 512-byte tile of the scale layout
// and four columns of tensor memory (tcgen05.cp 32x128b, copied to all four
// lane quarters).  A row tile of 192 starts at an even or odd multiple of 64:
// the odd ones start two columns into their scales.
//
// Bound by the tensor cores, and by the scales' copies between the MMAs: per K
// block four MMAs of 83 cycles and six copies of about 40 take about 500.
// 16384 x 13312 x 16384 back to back on a GB300: 1010 us (7070 TFLOP/s, under the
// power cap; alone 930); 8 x 8192 x 28672: 28 us (4.5 TB/s of weights).  At six
// times the measured bf16 rate, the chip's nominal ratio, the operations of the
// first take 630 us.

#include <cuda_bf16.h>

#include "launch.cuh"
#include "ptx.cuh"

namespace {

using namespace dgl;

constexpr int kTileRows = 192;
constexpr int kStages = 6;
constexpr int kBlockK = 256;                     // columns per K block: 128 bytes of codes
constexpr uint32_t kStageQ = (kTileRows / 2) * kRowBytes;
constexpr uint32_t kScaleP = 1024, kScaleQ = 2048;  // scales of 128 and of 256 rows x 256 columns
constexpr uint32_t kStage = kStageP + kStageQ + kScaleP + kScaleQ;
constexpr uint32_t kSmem = kStages * kStage + kEpiWarps * kStoreBuf + 256 + 1024;
constexpr uint32_t kTmemCols = 512, kScaleCol = 2 * kTileRows;
constexpr int kScaleBufs = 4;                    // 24 columns each: 2 x 4 for P, 2 x 8 for Q
constexpr int kBand = 16;  // row tiles of a band (8: 3 % slower on 16384 x 13312 x 16384)
constexpr int64_t kSlot = (int64_t)cut_slot_floats(kTileRows);

struct Args {
  CUtensorMap p, q[4];     // codes as bytes: boxes of 128 rows; of 96, 64, 32 and 16 rows
  CUtensorMap sp, sq;      // scales: (256 words, K block, row tile), boxes of one and two row tiles
  int rows, feats, kblocks, row_tiles;
  int high;                // rows of a tile: 192, or 64
  Raster raster;
  Divider per_unit;        // by the pairs of the launch
  void* out;
  uint32_t* counters;      // cut tiles
  float* partial;
  Watch watch;
};

__device__ __forceinline__ void scale_copy(uint32_t taddr, uint32_t saddr) {
  // 32 rows of 16 bytes without swizzle: groups of 8 rows 128 bytes apart
  const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t pdesc, uint64_t qdesc, uint32_t idesc, uint32_t psf,
                                        uint32_t qsf, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d),
      "l"(pdesc), "l"(qdesc), "r"(idesc), "r"(psf), "r"(qsf), "r"(acc)
      : "memory");
}

// Instruction descriptor of the block-scaled kinds: scale ids at bits 4 (Q) and
// 29 (P), e2m1 formats (1) at bits 7 and 10, columns / 8 at bit 17, e8m0 scales
// (bit 23), lanes / 16 at bit 24.
__device__ __forceinline__ uint32_t idesc_mx4(uint32_t n, uint32_t sf) {
  return (sf << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) | ((uint32_t)(kPairFeats >> 4) << 24) |
         (sf << 29);
}

struct Tile {
  int row0, rows, f0;
};
__device__ __forceinline__ Tile tile_at(const Args& p, int t) {
  int r, f;
  raster_at(p.raster, t, p.row_tiles, r, f);
  return Tile{r * p.high, min(p.high, p.rows - r * p.high), f * kPairFeats};
}

template <bool OUT32>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1) mx4_kernel(const __grid_constant__ Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* store_buf = smem + kStages * kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(store_buf + kEpiWarps * kStoreBuf);
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages, tempty = tfull + 16;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 4);
  volatile uint32_t* s_last = s_tmem + 1;
  volatile uint32_t* s_go = s_tmem + 2;  // [2]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t half = cluster_ctarank();
  const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;
  let_next_start();
  if (threadIdx.x < 4) prefetch_map(&p.q[threadIdx.x]);
  if (threadIdx.x >= 4 && threadIdx.x < 7) prefetch_map(threadIdx.x == 4 ? &p.p : threadIdx.x == 5 ? &p.sp : &p.sq);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(tfull + 8 * i, 1), mbar_init(tempty + 8 * i, 2 * kEpiWarps);
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(smem_u32(s_tmem), kTmemCols);
  wait_for_previous();
  fence_before();
  __syncwarp();
  cluster_sync();
  fence_after();
  const uint32_t tmem = *s_tmem, base = smem_u32(smem);
  const int total = p.row_tiles * p.raster.nf;
  const Cut cut = cut_of(total, units, p.per_unit, p.kblocks, (float)p.rows * (float)p.raster.nf);

  if (warp == 0) {
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    Item w;
    for (Walk walk(cut, unit, units, total); ok && walk.get(w);) {
      const Tile tl = tile_at(p, w.tile);
      const int n = (tl.rows + 31) / 32 * 32, mine = n / 2;
      const int f = tl.f0 + (int)half * kLanes, q0 = tl.row0 + (int)half * mine;
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        if (!(ok = mbar_wait_warp(p.watch, empty + 8 * stage, phase ^ 1, 0x100u | stage))) break;
        const uint32_t fb = mapa(full + 8 * stage, 0);
        const uint32_t sp = base + stage * kStage, sq = sp + kStageP, ss = sq + kStageQ;
        if (elect_one()) {
          if (half == 0) mbar_expect(full + 8 * stage, 2 * (kStageP + (uint32_t)mine * kRowBytes + kScaleP + kScaleQ));
          tma_2d(sp, &p.p, fb, kb * 128, f);
          if (mine == kTileRows / 2) {
            tma_2d(sq, &p.q[0], fb, kb * 128, q0);
          } else {
            int i = 0;
#pragma unroll
            for (int b = 1, r = 64; b < 4; ++b, r /= 2)
              if (mine & r) tma_2d(sq + i * kRowBytes, &p.q[b], fb, kb * 128, q0 + i), i += r;
          }
          tma_3d(ss, &p.sp, fb, 0, kb, f / 128);
          tma_3d(ss + kScaleP, &p.sq, fb, 0, kb, tl.row0 / 128);  // every row's: each CTA needs them all
        }
        __syncwarp();
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
    }
  } else if (warp == 1) {
    if (half == 0) {
      uint32_t stage = 0, phase = 0, it = 0, sbuf = 0;
      bool ok = true;
      Item w;
      for (Walk walk(cut, unit, units, total); ok && walk.get(w); ++it) {
        const Tile tl = tile_at(p, w.tile);
        const uint32_t n = (uint32_t)(tl.rows + 31) / 32 * 32, buf = it & 1;
        const uint32_t odd = (tl.row0 & 64) ? 2u : 0u;  // columns into the first scale tile
        if (!(ok = mbar_wait_warp(p.watch, tempty + 8 * buf, ((it >> 1) & 1) ^ 1, 0x200u | buf))) break;
        fence_after();
        const uint32_t d = tmem + buf * kTileRows;
        const uint32_t idesc0 = idesc_mx4(n, 0), idesc2 = idesc_mx4(n, 2);
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!(ok = mbar_wait_warp(p.watch, full + 8 * stage, phase, 0x300u | stage))) break;
          fence_after();
          const uint32_t sp = base + stage * kStage, sq = sp + kStageP, ss = sq + kStageQ;
          const uint32_t tp = tmem + kScaleCol + sbuf * 24, tq = tp + 8;
          const uint64_t pd = desc_k_major(sp), qd = desc_k_major(sq);
          if (elect_one()) {
            // copies and MMAs of one thread run in order
#pragma unroll
            for (uint32_t k = 0; k < 2; ++k) {
              scale_copy(tp + 4 * k, ss + 512 * k);
              scale_copy(tq + 8 * k, ss + kScaleP + 512 * k);
              scale_copy(tq + 8 * k + 4, ss + kScaleP + 1024 + 512 * k);
            }
#pragma unroll
            for (uint32_t s = 0; s < 4; ++s)
              mma_mx4(d, pd + 2 * s, qd + 2 * s, s & 1 ? idesc2 : idesc0, tp + 4 * (s >> 1), tq + 8 * (s >> 1) + odd,
                      kb != w.kb0 || s != 0);
            commit_pair(empty + 8 * stage);
          }
          __syncwarp();
          sbuf = (sbuf + 1) % kScaleBufs;
          if (++stage == kStages) stage = 0, phase ^= 1;
        }
        if (ok && elect_one()) commit_pair(tfull + 8 * buf);
        __syncwarp();
      }
    }
  } else {
    const int q = warp & 3;
    const int odd_steps = (warp - 2) >> 2;
    uint8_t* box = store_buf + (warp - 2) * kStoreBuf;
    uint32_t it = 0;
    Item w;
    for (Walk walk(cut, unit, units, total); walk.get(w); ++it) {
      const Tile tl = tile_at(p, w.tile);
      const uint32_t buf = it & 1;
      if (!epilogue_wait(p.watch, tfull, it, s_go)) break;
      const int f0 = tl.f0 + (int)half * kLanes + q * 32, feats_ok = min(32, p.feats - f0);
      const int nch = (tl.rows + kChunk - 1) / kChunk;
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * kTileRows;
      auto read = [&](int c, float(&v)[32]) {
        uint32_t u[32];
        tmem_ld32(acc + c * kChunk, u);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
      };
      auto release = [&]() {  // the accumulator has been read
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa(tempty + 8 * buf, 0));
      };
      int ways = 1, head = 0;
      if (w.tile < cut.tiles && (ways = cut_ways(cut, w.tile)) > 1) {
        head = cut_first(cut, w.tile);
        float* mine = p.partial + cut_slot(cut, w.tile, unit) * kSlot + half * (kSlot / 2);
#pragma unroll 1
        for (int c = odd_steps; c < nch; c += 2) {
          float v[32];
          read(c, v);
          store_partial(mine, c * kChunk, q * 32 + lane, v);
        }
        release();
        if (!cut_last(p.counters + 2 * w.tile + half, ways, s_last)) continue;
      } else if (odd_steps >= nch) {
        release();
      }
#pragma unroll 1
      for (int c = odd_steps; c < nch; c += 2) {
        float v[32];
        if (ways > 1) {
          join_partials(
              ways, [&](int j) { return p.partial + cut_slot(cut, w.tile, head + j) * kSlot + half * (kSlot / 2); },
              c * kChunk, q * 32 + lane, v);
        } else {
          read(c, v);
        }
        if (ways == 1 && c + 2 >= nch) release();
        const int64_t at = (int64_t)(tl.row0 + c * kChunk) * p.feats + f0;
        const int rows_ok = min(kChunk, tl.rows - c * kChunk);
        if constexpr (OUT32)
          store_box_f32(static_cast<float*>(p.out) + at, p.feats, rows_ok, feats_ok, lane, v);
        else
          store_box_bf16(static_cast<__nv_bfloat16*>(p.out) + at, p.feats, rows_ok, feats_ok, lane, v, box);
      }
    }
  }
  fence_before();
  __syncwarp();
  cluster_sync();
  fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_free(tmem, kTmemCols);
  }
}

template <bool OUT32>
int run(Args& p, cudaStream_t s) {
  int sms = 0;
  if (int rc = sm_count(&sms)) return rc;
  DGL_CUDA(cudaFuncSetAttribute(mx4_kernel<OUT32>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem));
  p.per_unit = divider_of((uint64_t)(sms / 2));
  return dgl::launch(mx4_kernel<OUT32>, dim3((unsigned)(sms / 2 * 2)), dim3(kThreads), kSmem, s, p);
}

}  // namespace

extern "C" int dg_layer_mx4_matmul(const void* a_codes, const void* a_scales, const void* b_codes,
                                   const void* b_scales, void* D, int d_type, int64_t M, int64_t N, int64_t K,
                                   void* workspace, void* status, void* stream) {
  if (M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX)
    return fail(DG_ERR_ARG, "M %lld, N %lld, K %lld out of range", (long long)M, (long long)N, (long long)K);
  if (d_type != DG_TYPE_BF16 && d_type != DG_TYPE_F32) return fail(DG_ERR_ARG, "D is bf16 or fp32 (got type %d)", d_type);
  if (N % 8 || K % 32) return fail(DG_ERR_SHAPE, "N %% 8 and K %% 32 must be 0 (N %lld, K %lld)", (long long)N, (long long)K);
  if (M == 0 || N == 0) return DG_OK;
  if (!D || !status) return fail(DG_ERR_ARG, "D and status must not be null");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) {
    DGL_CUDA(cudaMemsetAsync(D, 0, (size_t)M * N * (d_type == DG_TYPE_F32 ? 4 : 2), s));
    return DG_OK;
  }
  if (!a_codes || !a_scales || !b_codes || !b_scales || !workspace)
    return fail(DG_ERR_ARG, "codes, scales and the workspace must not be null");
  if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(b_codes) || !aligned16(b_scales) || !aligned16(D) || !aligned16(workspace))
    return fail(DG_ERR_ARG, "codes, scales, D and the workspace must be 16-byte aligned");
  const int64_t tiles = ((M + kTileRows - 1) / kTileRows) * ((N + kPairFeats - 1) / kPairFeats);
  if (tiles > INT32_MAX) return fail(DG_ERR_ARG, "M x N is too large (%lld tiles)", (long long)tiles);
  Args p{};
  const int64_t pitch[1] = {K / 2}, pd[2] = {K / 2, N}, qd[2] = {K / 2, M};
  if (int rc = encode_map(&p.p, b_codes, 1, 2, pd, pitch, kLanes)) return rc;
  for (int b = 0; b < 4; ++b)
    if (int rc = encode_map(&p.q[b], a_codes, 1, 2, qd, pitch, b == 0 ? kTileRows / 2 : 128 >> b)) return rc;
  p.kblocks = (int)((K + kBlockK - 1) / kBlockK);
  if (int rc = encode_scale_map(&p.sp, b_scales, p.kblocks, (N + 127) / 128, 1)) return rc;
  if (int rc = encode_scale_map(&p.sq, a_scales, p.kblocks, (M + 127) / 128, 2)) return rc;
  p.rows = (int)M, p.feats = (int)N, p.out = D;
  // more and shorter tiles end sooner where each still has a pair of its own (64
  // rows: a multiple of that, for the scales' columns); 2048 x 28672 with 200 rows
  // 29 -> 20 us
  int sms = 0;
  if (int rc = sm_count(&sms)) return rc;
  p.high = (M + 63) / 64 * ((N + kPairFeats - 1) / kPairFeats) > sms / 2 || N * K / 2 > kSharedBytes ? kTileRows : 64;
  p.row_tiles = (int)((M + p.high - 1) / p.high);
  p.raster = raster_of(N, kBand);
  p.counters = static_cast<uint32_t*>(workspace);
  p.partial = reinterpret_cast<float*>(p.counters + kCutCounters);
  p.watch = Watch{static_cast<unsigned long long*>(status), next_tag(), 4000000000ull};
  return d_type == DG_TYPE_F32 ? run<true>(p, s) : run<false>(p, s);
}
