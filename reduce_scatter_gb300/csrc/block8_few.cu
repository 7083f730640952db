// block8_few.cu -- product of up to 128 rows in 8-bit blocks of 128 (behind
// dg_layer_block8_matmul).
//
// Bound by the weights' way from memory.  As in the other products of few rows
// the features (b's) lie on the accumulator's 256 lanes of a CTA pair and the rows
// on its columns (D^T), so that a K block costs the rows' columns and not a whole
// tile's.  Each K block of 128 gets an accumulator of its own (4 to 16 of them in
// tensor memory), which eight warps multiply by its scales and add to the sums in
// their registers.  The tiles are cut along K (ptx.cuh); of a cut tile's sums the
// last pair adds the others' up in the order of K, and the accumulators in
// between go on filling while a pair leaves its own.  The loads of four K blocks go out
// together, rows before K blocks, so that neighbouring addresses follow each other.
// 8 x 8192 x 28672: 47 us (5.0 TB/s; as whole tiles of 256 rows 62), 64 x 8192 x
// 8192 24 (31), 128 rows 30.

#include "block8_few.h"

#include "launch.cuh"
#include "ptx.cuh"

namespace {

using namespace dgl;

constexpr int kStages = 8;
constexpr int kMostBufs = 16;                     // accumulators: as many as 512 columns hold, up to this
constexpr int kGroup = 4, kPart = 32;             // K blocks whose loads go out together, and rows of one load
constexpr int kJoins = 4;                         // partial sums whose loads are in flight at once
constexpr int kAhead = 4;                         // K blocks by which the scales' loads are ahead
constexpr int kStep = 16;                         // columns per load from tensor memory
constexpr int kSteps = kFewRows / kStep / 2;      // of one warp at most
constexpr uint32_t kStageQ = kFewRows / 2 * kRowBytes;
constexpr uint32_t kStage = kStageP + kStageQ;
constexpr uint32_t kTable = 2 * kFewRows / 2 * 4;  // a warp's: the scales of its rows, of two K blocks by turns
constexpr uint32_t kBarriers = 2 * kStages + 2 * kMostBufs;
constexpr uint32_t kSmem = kStages * kStage + kEpiWarps * kTable + 8 * kBarriers + 64 + 1024;
constexpr int64_t kSlot = (int64_t)cut_slot_floats(256);

struct Args {
  CUtensorMap p, q;        // b: boxes of 128 bytes x 128 rows; a: of 128 bytes x half the columns
  int rows, feats, kblocks, columns, bufs;
  int b_mn, out_f32;
  const float *sa, *sb;
  int64_t sa_m, sa_k, sb_n, sb_k;
  int a_shift, b_shift;
  uint32_t idesc;
  Divider per_unit;
  void* out;
  uint32_t* counters;
  float* partial;
  Watch watch;
};

// COLS: b has a scale for each of its rows (1 x 128).
template <bool COLS>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1) block8_few_kernel(const __grid_constant__ Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStage + kEpiWarps * kTable);
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages, tempty = tfull + 8 * kMostBufs;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + kBarriers);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t half = cluster_ctarank();
  const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;
  let_next_start();
  if (threadIdx.x < 2) prefetch_map(threadIdx.x == 0 ? &p.p : &p.q);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
    for (int i = 0; i < kMostBufs; ++i) mbar_init(tfull + 8 * i, 1), mbar_init(tempty + 8 * i, 2 * kEpiWarps);
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(smem_u32(s_tmem), 512);
  wait_for_previous();
  fence_before();
  __syncwarp();
  cluster_sync();
  fence_after();
  const uint32_t tmem = *s_tmem, base = smem_u32(smem);
  const int total = (p.feats + kPairFeats - 1) / kPairFeats;
  // (leaving and joining sums costs about 20 K blocks, as for a step of rows elsewhere: 96x2048x8192 31.6 us uncut)
  const Cut cut = cut_of(total, units, p.per_unit, p.kblocks, (float)kChunk * (float)total);

  if (warp == 0) {
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    Item w;
    const int mine = p.columns / 2, q0 = (int)half * mine;  // this CTA's share of the rows
    for (Walk walk(cut, unit, units, total); ok && walk.get(w);) {
      const int f = w.tile * kPairFeats + (int)half * kLanes;
      for (int kb = w.kb0; ok && kb < w.kb1; kb += kGroup) {
        const int many = min(kGroup, w.kb1 - kb);
        uint32_t st = stage, ph = phase;
        for (int j = 0; ok && j < many; ++j) {
          if (!(ok = mbar_wait_warp(p.watch, empty + 8 * st, ph ^ 1, 0x100u | st))) break;
          if (half == 0 && elect_one()) mbar_expect(full + 8 * st, 2 * (kStageP + (uint32_t)mine * kRowBytes));
          __syncwarp();
          if (++st == kStages) st = 0, ph ^= 1;
        }
        if (!ok) break;
        if (elect_one()) {
          for (int r = 0; r < kLanes / kPart; ++r) {
            st = stage;
            for (int j = 0; j < many; ++j) {
              const int k = (kb + j) * 128;
              const uint32_t fb = mapa(full + 8 * st, 0), sp = base + st * kStage;
              if (p.b_mn)
                tma_2d(sp + r * kPart * kRowBytes, &p.p, fb, f, k + r * kPart);
              else
                tma_2d(sp + r * kPart * kRowBytes, &p.p, fb, k, f + r * kPart);
              if (r == 0) tma_2d(sp + kStageP, &p.q, fb, k, q0);
              if (++st == kStages) st = 0;
            }
          }
        }
        __syncwarp();
        for (int j = 0; j < many; ++j)
          if (++stage == kStages) stage = 0, phase ^= 1;
      }
    }
  } else if (warp == 1) {
    if (half == 0) {
      uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 1;
      bool ok = true;
      Item w;
      const uint64_t p_step = p.b_mn ? 32 * kRowBytes / 16 : 2;  // 32 rows, or 32 bytes of a row
      for (Walk walk(cut, unit, units, total); ok && walk.get(w);) {
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!(ok = mbar_wait_warp(p.watch, tempty + 8 * buf, buf_phase, 0x200u | buf))) break;
          if (!(ok = mbar_wait_warp(p.watch, full + 8 * stage, phase, 0x300u | stage))) break;
          fence_after();
          const uint32_t sp = base + stage * kStage;
          const uint64_t pd = desc_k_major(sp), qd = desc_k_major(sp + kStageP);  // (MN-major: one swizzle span wide, the same fields)
          if (elect_one()) {
#pragma unroll
            for (uint32_t s = 0; s < 4; ++s) mma_pair<true>(tmem + buf * p.columns, pd + s * p_step, qd + 2 * s, p.idesc, s != 0);
            commit_pair(empty + 8 * stage);
            commit_pair(tfull + 8 * buf);
          }
          __syncwarp();
          if (++stage == kStages) stage = 0, phase ^= 1;
          if (++buf == (uint32_t)p.bufs) buf = 0, buf_phase ^= 1;
        }
      }
    }
  } else {
    const int q = warp & 3;            // the lanes that this warp may read
    const int side = (warp - 2) >> 2;  // it takes every other step of the columns
    const int steps = p.columns / kStep;
    const uint32_t table = smem_u32(smem + kStages * kStage) + (uint32_t)(warp - 2) * kTable;
    uint32_t buf = 0, buf_phase = 0;
    bool ok = true;
    Item w;
    for (Walk walk(cut, unit, units, total); ok && walk.get(w);) {
      const int f0 = w.tile * kPairFeats + (int)half * kLanes + q * 32;  // this warp's first feature
      const bool mine = f0 < p.feats && side < steps;
      // the scale of this lane's feature, and of two rows: lanes 0 to 15 have the first and third step's rows, the others
      // the second and fourth one's
      const float* sb = p.sb + (int64_t)(min(f0 + lane, p.feats - 1) >> p.b_shift) * p.sb_n + (int64_t)w.kb0 * p.sb_k;
      const float* sa[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = ((2 * i + (lane >> 4)) * 2 + side) * kStep + (lane & 15);
        sa[i] = p.sa + (int64_t)(min(row, p.rows - 1) >> p.a_shift) * p.sa_m + (int64_t)w.kb0 * p.sa_k;
      }
      const bool upper = steps > 4;  // (rows of a third and fourth step)
      // a ring of the scales of the next K blocks
      float b_ring[kAhead], a_ring[kAhead][2];
      int fetched = w.kb0;
      auto fetch = [&]() {
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) b_ring[k] = b_ring[k + 1], a_ring[k][0] = a_ring[k + 1][0], a_ring[k][1] = a_ring[k + 1][1];
        if (fetched++ < w.kb1) {
          b_ring[kAhead - 1] = __ldg(sb), a_ring[kAhead - 1][0] = __ldg(sa[0]);
          if (upper) a_ring[kAhead - 1][1] = __ldg(sa[1]);
          sb += p.sb_k, sa[0] += p.sa_k, sa[1] += p.sa_k;
        }
      };
#pragma unroll
      for (int k = 0; k < kAhead; ++k) b_ring[k] = a_ring[k][0] = a_ring[k][1] = 0.f;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) fetch();
      float acc[kSteps][kStep];
#pragma unroll
      for (int c = 0; c < kSteps; ++c)
#pragma unroll
        for (int i = 0; i < kStep; ++i) acc[c][i] = 0.f;
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        const float b = b_ring[0];
        const uint32_t at_table = table + (uint32_t)(kb & 1) * (kTable / 2);
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(at_table + lane * 4), "f"(COLS ? a_ring[0][0] : a_ring[0][0] * b) : "memory");
        if (upper) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at_table + 128 + lane * 4), "f"(COLS ? a_ring[0][1] : a_ring[0][1] * b) : "memory");
        __syncwarp();
        fetch();
        if (!(ok = mbar_wait_warp(p.watch, tfull + 8 * buf, buf_phase, 0x400u | buf))) break;
        fence_after();
        if (mine) {
          const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + buf * p.columns + side * kStep;
#pragma unroll
          for (int c = 0; c < kSteps; ++c) {
            if (2 * c + side < steps) {
              uint32_t u[16];
              tmem_ld16(at + 2 * c * kStep, u);
              tmem_ld_wait(u);
#pragma unroll
              for (int i = 0; i < kStep; i += 4) {
                float f[4];
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
                             : "r"(at_table + (c * kStep + i) * 4)
                             : "memory");
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float t = __uint_as_float(u[i + k]);
                  acc[c][i + k] = fmaf(t, COLS ? f[k] * b : f[k], acc[c][i + k]);
                }
              }
            }
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa(tempty + 8 * buf, 0));
        if (++buf == (uint32_t)p.bufs) buf = 0, buf_phase ^= 1;
      }
      if (!ok) break;
      if (!mine) continue;
      int ways = 1;
      if (w.tile < cut.tiles && (ways = cut_ways(cut, w.tile)) > 1) {
        const int head = cut_first(cut, w.tile);
        auto place = [&](int pair, int c) {
          return p.partial + cut_slot(cut, w.tile, pair) * kSlot + half * (kSlot / 2) + (int64_t)((2 * c + side) * kStep) * kLanes + q * 32 + lane;
        };
#pragma unroll
        for (int c = 0; c < kSteps; ++c)
          if (2 * c + side < steps)
#pragma unroll
            for (int i = 0; i < kStep; ++i) __stcg(place(unit, c) + i * kLanes, acc[c][i]);
        if (!warp_last(p.counters + 4 * w.tile + 2 * half + side, q, ways, lane)) continue;
        // the partial sums are added to each other in the order of K
#pragma unroll
        for (int c = 0; c < kSteps; ++c)
          if (2 * c + side < steps) {
#pragma unroll
            for (int i = 0; i < kStep; ++i) acc[c][i] = 0.f;
#pragma unroll 1
            for (int j = 0; j < ways; j += kJoins) {
              // (loads without a condition: behind one each waited for the one before, 31 000 cycles for 8 partials)
              float u[kJoins][kStep];
#pragma unroll
              for (int k = 0; k < kJoins; ++k) {
                const float* from = place(head + min(j + k, ways - 1), c);
#pragma unroll
                for (int i = 0; i < kStep; ++i) u[k][i] = __ldcg(from + i * kLanes);
              }
#pragma unroll
              for (int k = 0; k < kJoins; ++k)
#pragma unroll
                for (int i = 0; i < kStep; ++i) acc[c][i] += j + k < ways ? u[k][i] : 0.f;
            }
          }
      }
      if (f0 + lane < p.feats) {
#pragma unroll
        for (int c = 0; c < kSteps; ++c)
#pragma unroll
          for (int i = 0; i < kStep; ++i) {
            const int row = (2 * c + side) * kStep + i;
            if (row >= p.rows) break;
            const int64_t at = (int64_t)row * p.feats + f0 + lane;
            if (p.out_f32)
              static_cast<float*>(p.out)[at] = acc[c][i];
            else
              static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(acc[c][i]);
          }
      }
    }
    if (!ok) settle();
  }
  fence_before();
  __syncwarp();
  cluster_sync();  // both CTAs are done with each other's barriers and shared memory
  fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_free(tmem, 512);
  }
}

}  // namespace

namespace dgl {

int block8_few(const FewRows& f, void* stream) {
  int sms = 0;
  if (int rc = sm_count(&sms)) return rc;
  auto* kernel = f.b_shift == 0 ? block8_few_kernel<true> : block8_few_kernel<false>;
  DGL_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem));
  Args p{};
  p.columns = (int)((f.M + kStep - 1) / kStep * kStep);
  const int64_t pd[2] = {f.b_mn ? f.N : f.K, f.b_mn ? f.K : f.N}, pp[1] = {pd[0]}, qd[2] = {f.K, f.M}, qp[1] = {f.K};
  if (int rc = encode_map(&p.p, f.b, 1, 2, pd, pp, kPart)) return rc;
  if (int rc = encode_map(&p.q, f.a, 1, 2, qd, qp, p.columns / 2)) return rc;
  p.bufs = 512 / p.columns < kMostBufs ? 512 / p.columns : kMostBufs;
  p.rows = (int)f.M, p.feats = (int)f.N, p.kblocks = (int)((f.K + 127) / 128);
  p.b_mn = f.b_mn, p.out_f32 = f.d_f32, p.out = f.D;
  p.sa = f.sa, p.sb = f.sb, p.sa_m = f.sa_m, p.sa_k = f.sa_k, p.sb_n = f.sb_n, p.sb_k = f.sb_k;
  p.a_shift = f.a_shift, p.b_shift = f.b_shift;
  p.idesc = idesc_of(f.b_type == DG_TYPE_E5M2, f.a_type == DG_TYPE_E5M2, f.b_mn != 0, false) | idesc_columns((uint32_t)p.columns);
  p.per_unit = divider_of((uint64_t)(sms / 2));
  p.counters = static_cast<uint32_t*>(f.workspace);
  p.partial = reinterpret_cast<float*>(p.counters + kCutCounters);
  p.watch = Watch{static_cast<unsigned long long*>(f.status), next_tag(), 4000000000ull};
  return launch(kernel, dim3((unsigned)(sms / 2 * 2)), dim3(kThreads), kSmem, static_cast<cudaStream_t>(stream), p);
}

}  // namespace dgl
