// grouped.cu -- products grouped by expert (dg_layer_grouped_matmul,
// dg_layer_grouped_weight_grad).
//
//   D[t, n]     = sa[t] sb[e, n] sum_k A[t, k] B[e, n, k]      for the rows t of group e
//   dB[e, n, k] = sum over the rows t of group e of dD[t, n] A[t, k]
//
// One persistent kernel over CTA pairs, D^T orientation (ptx.cuh): P is the
// operand of the output's contiguous dimension (B's features; A's columns for
// the gradient), Q that of the output's rows (tokens; dD's columns).  A tile is
// 256 features x up to 256 rows.  The groups' ends live on the device, so every
// CTA scans them once into shared memory and walks the same list of tiles.
//
// Warp 0 loads (TMA, 128-byte swizzle, kStages stages), warp 1 issues the MMAs
// (even CTA of the pair), warps 2-9 empty the two accumulators.
//
// A tile of 256 rows moves 128 bytes a cycle through its SM's shared memory (what
// the loads write and the MMAs read), which is all it has: the tensor pipe is
// busy for 95 % of the cycles.  A shorter tile of n rows needs about 256 + n
// cycles a K block against 2 n of the MMAs, so few tall tiles are best where
// there are enough of them.  (That model gives 130 to 155 us of the 197 below; the
// rest is not accounted for.)  Back to back on a GB300: 16384 rows of 8 experts of
// 8192 x 8192 in bf16 1253 us even, 1317 uneven (1755, 1670 TFLOP/s, under the
// power cap; alone 1138, 1195); 10007 rows of 24 (5 empty) of 3328 x 8192 in e4m3 197
// us (2770 TFLOP/s), of 19 188 us; 12 rows of 12 of 2048 x 8192 39 us (5.2 TB/s of
// weights).

#include <cuda_bf16.h>

#include "launch.cuh"
#include "ptx.cuh"

namespace {

using namespace dgl;

constexpr int kTileRows = 256;
constexpr int kMaxExperts = 1024;
constexpr int kStages = 6;
constexpr uint32_t kStageQ = (kTileRows / 2) * kRowBytes;
constexpr uint32_t kStage = kStageP + kStageQ;
constexpr uint32_t kTableBytes = 3 * (kMaxExperts + 2) * 4;
constexpr uint32_t kSmem = kStages * kStage + kEpiWarps * kStoreBuf + kTableBytes + 256 + 1024;
constexpr uint32_t kTmemCols = 2 * kTileRows;
constexpr int64_t kSlot = (int64_t)cut_slot_floats(kTileRows);
constexpr int kTailRows = 64; // rows of a K block in the gradient
constexpr int kBand = 8;      // row tiles of a band (4: 3 % slower on 16384 rows of 8 experts, 16: 1 %)

struct Args {
  CUtensorMap p;           // 3-d: (K or features, features or K, expert)
  CUtensorMap q[4];        // rows: boxes of 128, 64, 32 and 16 rows; gradient: the first, of 64 columns x 64 rows
  CUtensorMap p_tail, q_tail;  // gradient: each group's last rows, padded with zeros
  const int32_t* ends;
  int experts, T;
  int feats, rows, red;    // output features; gradient: output rows; forward: reduction length
  void* out;
  const float *sa, *sb;
  int64_t sa_s, sb_e, sb_n;
  uint32_t idesc;
  Raster raster;
  Divider per_unit;        // by the pairs of the launch
  int may_be_few;          // tiles of 256 rows may leave more than half of the pairs idle
  uint32_t* counters;      // cut tiles
  float* partial;
  Watch watch;
};

struct Tile {
  int e, row0, rows, f0, kblocks, k0, tail;
};

// Rows of a group's tiles: as few tiles as `most` rows allow, of equal height (a
// multiple of 32), because a short tile still loads all of its features.
__device__ __forceinline__ int tile_height(int rows, int nt, int most) {
  return nt > 1 ? ((rows + nt - 1) / nt + 31) / 32 * 32 : most;
}

// The most rows of a tile: 256, or as few (a multiple of 32) as still give every
// tile a pair of its own where tiles of 256 would leave more than half of the
// pairs idle.  (A K block of a tile takes about 256 + rows cycles, its loads', so
// short tiles on more pairs end sooner, but cost more in all.)
__device__ __forceinline__ int most_rows(int tiles, int units) {
  if (2 * tiles > units || tiles == 0) return kTileRows;
  const int share = (int)(__fdividef((float)units, (float)tiles) + 0.01f);
  return max(32, ((int)__fdividef((float)kTileRows, (float)share) + 31) / 32 * 32);
}

// Group starts (start[e], e <= experts; start[experts + 1] = T), the number of
// tiles before each group and the groups' row tiles and their height (shape[e] =
// row tiles << 9 | height), by one warp.  Ends are clamped to [previous end,
// T]; the forward's group `experts` is the rows past the last end.
template <bool GRAD>
__device__ void scan_groups(const Args& p, int* start, int* first, uint32_t* shape, int lane) {
  const int groups = GRAD ? p.experts : p.experts + 1;
  int v = 0, s = 0;  // end and start of group b + lane
  auto chunk = [&](int b, int before) {
    const int e = b + lane;
    v = e < p.experts ? min(max(__ldg(p.ends + e), 0), p.T) : p.T;
    if (lane == 0) v = max(v, before);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = max(v, u);
    }
    s = __shfl_up_sync(0xffffffffu, v, 1);
    if (lane == 0) s = before;
  };
  int most = kTileRows;
  if (!GRAD && p.may_be_few) {
    int count = 0, before = 0;
    for (int b = 0; b < groups; b += 32) {
      chunk(b, before);
      const int rows = b + lane < p.experts ? v - s : 0;
      count += __reduce_add_sync(0xffffffffu, (unsigned)((rows + kTileRows - 1) / kTileRows));
      before = __shfl_sync(0xffffffffu, v, 31);
    }
    const int units = gridDim.x >> 1;
    most = most_rows(min(count, units) * min(p.raster.nf, units), units);
  }
  int end = 0, tiles = 0;
  if (lane == 0) start[0] = first[0] = 0;
  for (int b = 0; b < groups; b += 32) {
    const int e = b + lane;
    if (!p.may_be_few || groups > 32) chunk(b, end);  // (else the one chunk is still there)
    const int rows = GRAD ? p.rows : v - s, nt = (rows + most - 1) / most;
    int t = e < groups ? nt * p.raster.nf : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += u;
    }
    t += tiles;
    if (e < groups)
      start[e + 1] = v, first[e + 1] = t,
      shape[e] = (uint32_t)nt << 9 | (uint32_t)(GRAD ? kTileRows : tile_height(rows, nt, most));
    end = __shfl_sync(0xffffffffu, v, 31);
    tiles = __shfl_sync(0xffffffffu, t, 31);
  }
}

// Tile t of the list; `e`: a cursor that only moves forward.
template <bool GRAD, bool F8>
__device__ __forceinline__ Tile tile_at(const Args& p, const int* start, const int* first, const uint32_t* shape, int t,
                                        int& e) {
  while (t >= first[e + 1]) ++e;
  const int len = start[e + 1] - start[e], rows = GRAD ? p.rows : len;
  const int high = (int)(shape[e] & 511u);
  int f, r;
  raster_at(p.raster, t - first[e], (int)(shape[e] >> 9), r, f);
  Tile tl;
  tl.e = e;
  tl.rows = min(high, rows - r * high);
  tl.f0 = f * kPairFeats;
  if (GRAD) {
    tl.row0 = r * high;
    tl.k0 = start[e];
    tl.kblocks = (len + kTailRows - 1) / kTailRows;
    tl.tail = len % kTailRows;
  } else {
    constexpr int kb = F8 ? 128 : 64;
    tl.row0 = start[e] + r * high;
    tl.k0 = 0;
    tl.kblocks = e < p.experts ? (p.red + kb - 1) / kb : 0;  // rows past the last group: zeros
    tl.tail = 0;
  }
  return tl;
}

// Accumulator columns of a tile: its rows rounded up to what a pair's MMA takes
// (the gradient's operand boxes are whole).
template <bool GRAD>
__device__ __forceinline__ int columns(const Tile& t) {
  return GRAD ? kTileRows : (t.rows + 31) / 32 * 32;
}

// A factor of D whose product with another such one is 0 or a normal number.
__device__ __forceinline__ bool plain_scale(float s) {
  return s == 0.f || (fabsf(s) >= 0x1p-60f && fabsf(s) <= 0x1p60f);
}
// v[i] times lane i's s and this lane's sb, whose product may be out of range
// where the result is not: the exponents last, in two steps.  (A call of its own,
// for the registers of the ordinary path.)
static __device__ __noinline__ void scale_apart(float* v, float s, float sb) {
  int es, eb;
  const float ms = frexpf(s, &es), mb = frexpf(sb, &eb);
  for (int i = 0; i < 32; ++i) {
    const float m = __shfl_sync(0xffffffffu, ms, i) * mb;
    const int e = __shfl_sync(0xffffffffu, es, i) + eb, a = min(max(e, -126), 127), b = min(max(e - a, -126), 127);
    v[i] = v[i] * m * __uint_as_float((uint32_t)(a + 127) << 23) * __uint_as_float((uint32_t)(b + 127) << 23);
  }
}

template <bool F8, bool PMN, bool GRAD, bool OUT32>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    grouped_kernel(const __grid_constant__ Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* store_buf = smem + kStages * kStage;
  int* start = reinterpret_cast<int*>(store_buf + kEpiWarps * kStoreBuf);
  int* first = start + kMaxExperts + 2;
  uint32_t* shape = reinterpret_cast<uint32_t*>(first + kMaxExperts + 2);
  uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(start) + kTableBytes);
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages, tempty = tfull + 16;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 4);
  // after the barriers of the stages and accumulators: ten words, then the ring's barriers
  volatile uint32_t* s_last = s_tmem + 1;
  volatile uint32_t* s_go = s_tmem + 2;  // [2]
  volatile int* s_next = reinterpret_cast<volatile int*>(s_tmem + 4);  // [2]
  const Ring ring{smem_u32(bars + 2 * kStages + 10), smem_u32(bars + 2 * kStages + 10 + kRing),
                  reinterpret_cast<volatile int*>(s_tmem + 6)};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t half = cluster_ctarank();
  const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;

  let_next_start();
  if (threadIdx.x < 5) prefetch_map(threadIdx.x == 4 ? &p.p : &p.q[GRAD ? 0 : threadIdx.x]);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(tfull + 8 * i, 1), mbar_init(tempty + 8 * i, 2 * kEpiWarps);
    for (int i = 0; i < kRing; ++i) mbar_init(ring.full + 8 * i, 1), mbar_init(ring.empty + 8 * i, kRingReaders);
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(smem_u32(s_tmem), kTmemCols);
  wait_for_previous();
  if (warp == 2) scan_groups<GRAD>(p, start, first, shape, lane);
  fence_before();
  __syncwarp();
  cluster_sync();
  fence_after();
  const uint32_t tmem = *s_tmem;
  // the tiles with work, then (forward) those of the rows past the last group
  const int real = first[p.experts], total = first[GRAD ? p.experts : p.experts + 1];
  constexpr int kb_red = F8 ? 128 : 64;
  Cut cut{0, 1, 0};
  if (!GRAD) {
    cut = cut_of(real, units, p.per_unit, (p.red + kb_red - 1) / kb_red,
                 (float)start[p.experts] * (float)p.raster.nf);
  }
  const bool draw = (GRAD ? p.T / kTailRows / p.experts : (p.red + kb_red - 1) / kb_red) >= kDrawBlocks;
  const uint32_t base = smem_u32(smem);

  if (warp == 0) {
    // -------------------------------------------------------------- producer
    uint32_t stage = 0, phase = 0;
    int e = 0;
    bool ok = true;
    Item w;
    Feed feed(cut, unit, units, total, draw);
    // the even CTA: lane 0 holds the next draw; the tile after the one being loaded is passed on once its loads have begun
    const uint32_t wrap = (uint32_t)(feed.rest + units - 1);
    uint32_t drawn = 0, passed = 0;
    int ahead = -1;  // a tile passed on and not begun
    if (half == 0 && lane == 0 && !feed.none()) drawn = atomicInc(p.counters + kDrawCounter, wrap);
    auto pass = [&]() {
      const uint32_t s = passed % kRing;
      if (!(ok = mbar_wait_warp(p.watch, ring.empty + 8 * s, ((passed / kRing) & 1) ^ 1, 0x600u | s))) return;
      const uint32_t d = __shfl_sync(0xffffffffu, drawn, 0);
      ahead = d < (uint32_t)feed.rest ? cut.tiles + units + (int)d : total;
      if (lane == 0) {
        ring_pass(ring, s, ahead);
        if (ahead < total) drawn = atomicInc(p.counters + kDrawCounter, wrap);
      }
      __syncwarp();
      ++passed;
    };
    while (ok) {
      if (!feed.own(w)) {
        if (feed.none()) break;
        int t = ahead;
        if (half != 0) {
          if (lane == 0) t = feed.read(p.watch, ring);
          t = __shfl_sync(0xffffffffu, t, 0);
          ++feed.n;
        }
        ahead = -1;
        if (!feed.take(t, w)) break;
      }
      const Tile tl = tile_at<GRAD, F8>(p, start, first, shape, w.tile, e);
      const int kb1 = GRAD ? tl.kblocks : min(w.kb1, tl.kblocks);
      const int n = columns<GRAD>(tl), mine = n / 2;  // this CTA's share of the rows operand
      const int f = tl.f0 + (int)half * kLanes, q0 = tl.row0 + (int)half * mine;
      for (int kb = w.kb0; kb < kb1; ++kb) {
        if (!(ok = mbar_wait_warp(p.watch, empty + 8 * stage, phase ^ 1, 0x100u | stage))) break;
        const uint32_t fb = mapa(full + 8 * stage, 0);
        const uint32_t sp = base + stage * kStage, sq = sp + kStageP;
        if (elect_one()) {
          if (half == 0) mbar_expect(full + 8 * stage, 2 * (kStageP + (uint32_t)mine * kRowBytes));
          if constexpr (GRAD) {
            // 64 columns x 64 rows per box, MN-major; a group's last rows come
            // from their zero-padded copy, so no other group's rows enter
            const bool tail = tl.tail != 0 && kb == tl.kblocks - 1;
            const CUtensorMap* pm = tail ? &p.p_tail : &p.p;
            const CUtensorMap* qm = tail ? &p.q_tail : &p.q[0];
            const int y = tl.k0 + kb * kTailRows;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              tma_3d(sp + i * (kStageP / 2), pm, fb, f + i * 64, tail ? 0 : y, tail ? tl.e : 0);
              tma_2d(sq + i * (kStageQ / 2), qm, fb, q0 + i * 64, tail ? tl.e * kTailRows : y);
            }
          } else {
            const int x = kb * (F8 ? 128 : 64);
            if constexpr (PMN) {
              tma_3d(sp, &p.p, fb, f, x, tl.e);
              tma_3d(sp + kStageP / 2, &p.p, fb, f + 64, x, tl.e);
            } else {
              tma_3d(sp, &p.p, fb, x, f, tl.e);
            }
            // a share of up to 128 rows, in boxes as large as they come (many small ones load at half the rate)
            if (mine == kTileRows / 2) {
              tma_2d(sq, &p.q[0], fb, x, q0);
            } else {
              int i = 0;
#pragma unroll
              for (int b = 1, r = 64; b < 4; ++b, r /= 2)
                if (mine & r) tma_2d(sq + i * kRowBytes, &p.q[b], fb, x, q0 + i), i += r;
            }
          }
        }
        __syncwarp();
        if (++stage == kStages) stage = 0, phase ^= 1;
        if (half == 0 && ahead < 0 && !feed.none()) {
          pass();
          if (!ok) break;
        }
      }
      if (ok && half == 0 && ahead < 0 && !feed.none()) pass();  // (a tile without K blocks)
    }
  } else if (warp == 1) {
    if (half == 0) {
      // ----------------------------------------------------------------- MMA
      uint32_t stage = 0, phase = 0, it = 0;
      int e = 0;
      bool ok = true;
      Item w;
      Feed feed(cut, unit, units, total, draw);
      for (; ok; ++it) {
        if (!feed.own(w)) {
          if (feed.none()) break;
          int t = -1;
          if (lane == 0) t = feed.read(p.watch, ring);
          ++feed.n;
          if (!feed.take(__shfl_sync(0xffffffffu, t, 0), w)) break;
        }
        const Tile tl = tile_at<GRAD, F8>(p, start, first, shape, w.tile, e);
        const int kb1 = GRAD ? tl.kblocks : min(w.kb1, tl.kblocks);
        const uint32_t idesc = p.idesc | idesc_columns((uint32_t)columns<GRAD>(tl));
        const uint32_t buf = it & 1;
        if (!(ok = mbar_wait_warp(p.watch, tempty + 8 * buf, ((it >> 1) & 1) ^ 1, 0x200u | buf))) break;
        fence_after();
        const uint32_t d = tmem + buf * kTileRows;
        for (int kb = w.kb0; kb < kb1; ++kb) {
          if (!(ok = mbar_wait_warp(p.watch, full + 8 * stage, phase, 0x300u | stage))) break;
          fence_after();
          const uint32_t sp = base + stage * kStage, sq = sp + kStageP;
          const uint64_t pd = PMN ? desc_mn_major(sp, kStageP / 2) : desc_k_major(sp);
          const uint64_t qd = GRAD ? desc_mn_major(sq, kStageQ / 2) : desc_k_major(sq);
          // per instruction: 32 bytes along a K-major row, or 16 rows of 128 bytes
          constexpr uint64_t p_step = PMN ? 16 * kRowBytes / 16 : 2, q_step = GRAD ? 16 * kRowBytes / 16 : 2;
          const int subs = GRAD && tl.tail != 0 && kb == tl.kblocks - 1 ? (tl.tail + 15) / 16 : 4;
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              if (!GRAD || s < subs) mma_pair<F8>(d, pd + s * p_step, qd + s * q_step, idesc, kb != w.kb0 || s != 0);
            commit_pair(empty + 8 * stage);
          }
          __syncwarp();
          if (++stage == kStages) stage = 0, phase ^= 1;
        }
        if (ok && elect_one()) commit_pair(tfull + 8 * buf);
        __syncwarp();
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue
    const int q = warp & 3;  // the TMEM lanes that this warp may read
    const int odd_steps = (warp - 2) >> 2;
    uint8_t* box = store_buf + (warp - 2) * kStoreBuf;
    uint32_t it = 0;
    int e = 0;
    Item w;
    Feed feed(cut, unit, units, total, draw);
    for (;; ++it) {
      if (!feed.own(w)) {
        if (feed.none()) break;
        // one thread reads for all the warps, which must agree
        if (threadIdx.x == 64) s_next[feed.n & 1] = feed.read(p.watch, ring);
        epilogue_sync();
        const int t = s_next[feed.n & 1];
        ++feed.n;
        if (t < 0) settle();
        if (!feed.take(t, w)) break;
      }
      const Tile tl = tile_at<GRAD, F8>(p, start, first, shape, w.tile, e);
      const uint32_t buf = it & 1;
      const int f0 = tl.f0 + (int)half * kLanes + q * 32;  // this warp's first feature
      const int feats_ok = min(32, p.feats - f0);
      const int64_t row0 = (int64_t)tl.row0 + (GRAD ? (int64_t)tl.e * p.rows : 0);
      // the scales of this lane's feature and of its rows of each step, fetched while the tile is computed
      float sb = 1.f, sa[kTileRows / kChunk / 2];
      if (!GRAD) {
        if (p.sb && lane < feats_ok && tl.e < p.experts)
          sb = __ldg(p.sb + tl.e * p.sb_e + (int64_t)(f0 + lane) * p.sb_n);
#pragma unroll
        for (int i = 0; i < kTileRows / kChunk / 2; ++i) {
          const int r = (2 * i + odd_steps) * kChunk + lane;
          sa[i] = p.sa && r < tl.rows ? __ldg(p.sa + (row0 + r) * p.sa_s) : 1.f;
        }
      }
      bool plain = true;
      if (!GRAD && (p.sa || p.sb)) {
        plain = plain_scale(sb);
#pragma unroll
        for (int i = 0; i < kTileRows / kChunk / 2; ++i) plain = plain && plain_scale(sa[i]);
        plain = __all_sync(0xffffffffu, plain) != 0;
      }
      if (!epilogue_wait(p.watch, tfull, it, s_go)) break;
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
      if (!GRAD && w.tile < cut.tiles && (ways = cut_ways(cut, w.tile)) > 1) {
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
        } else if (tl.kblocks > 0) {
          read(c, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
        if (ways == 1 && c + 2 >= nch) release();
        const int rows_ok = min(kChunk, tl.rows - c * kChunk);
        const int64_t r0 = row0 + c * kChunk;
        if (!GRAD && (p.sa || p.sb) && tl.kblocks > 0) {
          float s = sa[0];
#pragma unroll
          for (int i = 1; i < kTileRows / kChunk / 2; ++i) s = c / 2 == i ? sa[i] : s;
          if (plain) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= __shfl_sync(0xffffffffu, s, i) * sb;
          } else {
            float u[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = v[i];
            scale_apart(u, s, sb);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = u[i];
          }
        }
        const int64_t at = r0 * p.feats + f0;
        if constexpr (OUT32)
          store_box_f32(static_cast<float*>(p.out) + at, p.feats, rows_ok, feats_ok, lane, v);
        else
          store_box_bf16(static_cast<__nv_bfloat16*>(p.out) + at, p.feats, rows_ok, feats_ok, lane, v, box);
      }
    }
  }
  fence_before();
  __syncwarp();
  cluster_sync();  // both CTAs are done with each other's barriers and shared memory
  fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_free(tmem, kTmemCols);
  }
}

// The gradient's last rows of each group (its row count modulo 64), copied to
// [expert][64][columns] with zeros up to the next multiple of 16 rows.
__global__ void __launch_bounds__(256) grouped_tail_kernel(const int32_t* ends, int T, const __nv_bfloat16* a,
                                                           int64_t ld_a, int64_t ka, __nv_bfloat16* a_tail,
                                                           const __nv_bfloat16* d, int64_t ld_d, int64_t kd,
                                                           __nv_bfloat16* d_tail) {
  __shared__ int s_from[8], s_to[8];
  begin_kernel();
  const int e = blockIdx.y;
  int from = 0, to = 0;  // this group's clamped start and end: the largest ends before and up to it
  for (int i = threadIdx.x; i <= e; i += blockDim.x) {
    const int v = min(max(__ldg(ends + i), 0), T);
    to = max(to, v);
    if (i < e) from = max(from, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    from = max(from, __shfl_xor_sync(0xffffffffu, from, o));
    to = max(to, __shfl_xor_sync(0xffffffffu, to, o));
  }
  if ((threadIdx.x & 31) == 0) s_from[threadIdx.x >> 5] = from, s_to[threadIdx.x >> 5] = to;
  __syncthreads();
  for (int i = 0; i < 8; ++i) from = max(from, s_from[i]), to = max(to, s_to[i]);
  const int tail = (to - from) % kTailRows;
  if (tail == 0) return;
  const int padded = (tail + 15) / 16 * 16;
  const int64_t t0 = to - tail, va = ka / 8, vd = kd / 8, n = padded * (va + vd);
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const bool of_a = i < padded * va;
    const int64_t j = of_a ? i : i - padded * va, per = of_a ? va : vd, r = j / per, c = j - r * per;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (r < tail)
      u = *reinterpret_cast<const uint4*>((of_a ? a + (t0 + r) * ld_a : d + (t0 + r) * ld_d) + c * 8);
    *reinterpret_cast<uint4*>((of_a ? a_tail + ((int64_t)e * kTailRows + r) * ka
                                    : d_tail + ((int64_t)e * kTailRows + r) * kd) + c * 8) = u;
  }
}

template <bool F8, bool PMN, bool GRAD, bool OUT32>
int run(Args& p, int64_t most_tiles, cudaStream_t s) {
  auto* kernel = grouped_kernel<F8, PMN, GRAD, OUT32>;
  int sms = 0;
  if (int rc = sm_count(&sms)) return rc;
  DGL_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem));
  // the forward's tiles may be cut along K, so it takes every SM pair
  const int64_t units = GRAD && most_tiles < sms / 2 ? most_tiles : sms / 2;
  if (!GRAD) {  // whatever the groups are
    const int64_t bytes = (int64_t)(p.T < p.experts ? p.T : p.experts) * p.feats * p.red * (F8 ? 1 : 2);
    p.may_be_few = p.T > 32 && 2 * (int64_t)p.raster.nf * ((p.T + kTileRows - 1) / kTileRows) <= units && bytes <= kSharedBytes;
  }
  p.per_unit = divider_of(units > 1 ? units : 2);  // (a single pair has the gradient's one tile, and divides nothing)
  return dgl::launch(kernel, dim3((unsigned)(2 * units)), dim3(kThreads), kSmem, s, p);
}

uint32_t format_of(int type) { return type == DG_TYPE_BF16 ? 1u : type == DG_TYPE_E5M2 ? 1u : 0u; }

// A size rounded up to whole tiles or K blocks, and their first coordinates, fit 32 bits.
constexpr int64_t kMaxSize = INT32_MAX - 255;

int check_sizes(int64_t T, int64_t N, int64_t K, int experts) {
  if (T < 0 || N < 0 || K < 0 || T > kMaxSize || N > kMaxSize || K > kMaxSize)
    return fail(DG_ERR_ARG, "T %lld, N %lld, K %lld out of range", (long long)T, (long long)N, (long long)K);
  if (experts < 1 || experts > kMaxExperts) return fail(DG_ERR_ARG, "experts (%d) must be 1 to %d", experts, kMaxExperts);
  return DG_OK;
}

Watch watch_of(void* status) {
  return Watch{static_cast<unsigned long long*>(status), next_tag(), 4000000000ull};
}

}  // namespace

extern "C" size_t dg_layer_products_workspace(void) {
  int sms = 0;
  if (sm_count(&sms) != DG_OK) return 0;
  return cut_bytes(sms / 2, kTileRows);
}

extern "C" int dg_layer_grouped_matmul(const void* A, int64_t ld_a, int a_type, const void* B, int64_t ld_b,
                                       int64_t ld_e, int b_type, int b_n_major, const int32_t* ends, int experts,
                                       const float* scale_a, int64_t sa, const float* scale_b, int64_t sb_e,
                                       int64_t sb_n, void* D, int d_type, int64_t T, int64_t N, int64_t K,
                                       void* workspace, void* status, void* stream) {
  if (int rc = check_sizes(T, N, K, experts)) return rc;
  const bool f8 = is_fp8(a_type) && is_fp8(b_type);
  if (!f8 && (a_type != DG_TYPE_BF16 || b_type != DG_TYPE_BF16))
    return fail(DG_ERR_ARG, "A and B are both bf16 or both 8-bit (types %d, %d)", a_type, b_type);
  if (f8 && b_n_major) return fail(DG_ERR_ARG, "an 8-bit B must be contiguous along K");
  if (d_type != DG_TYPE_BF16 && d_type != DG_TYPE_F32) return fail(DG_ERR_ARG, "D is bf16 or fp32 (got type %d)", d_type);
  const int64_t esz = f8 ? 1 : 2;
  if (N % 8 || K * esz % 16) return fail(DG_ERR_SHAPE, "N %% 8 and K %% %d must be 0 (N %lld, K %lld)", f8 ? 16 : 8, (long long)N, (long long)K);
  if (T == 0 || N == 0) return DG_OK;
  if (!D || !ends || !status) return fail(DG_ERR_ARG, "D, ends and status must not be null");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) {
    DGL_CUDA(cudaMemsetAsync(D, 0, (size_t)T * N * (d_type == DG_TYPE_F32 ? 4 : 2), s));
    return DG_OK;
  }
  if (!A || !B || !workspace) return fail(DG_ERR_ARG, "A, B and workspace must not be null");
  const int64_t inner = b_n_major ? N : K;
  if (!aligned16(A) || !aligned16(B) || !aligned16(D) || !aligned16(workspace) || ld_a * esz % 16 || ld_b * esz % 16 ||
      (experts > 1 && ld_e * esz % 16))
    return fail(DG_ERR_ARG, "A, B, D, the workspace and the pitches must be multiples of 16 bytes");
  if (ld_a < K || ld_b < inner || (experts > 1 && ld_e <= 0)) return fail(DG_ERR_ARG, "a pitch is shorter than its rows");
  Args p{};
  const int64_t pd[3] = {inner, b_n_major ? K : N, experts}, ps[2] = {ld_b, experts > 1 ? ld_e : ld_b * pd[1]};
  const int64_t qd[2] = {K, T}, qs[1] = {ld_a};
  if (int rc = encode_map(&p.p, B, (int)esz, 3, pd, ps, b_n_major ? 64 : kLanes)) return rc;
  for (int b = 0; b < 4; ++b)
    if (int rc = encode_map(&p.q[b], A, (int)esz, 2, qd, qs, (kTileRows / 2) >> b)) return rc;
  p.ends = ends, p.experts = experts, p.T = (int)T, p.feats = (int)N, p.rows = 0, p.red = (int)K, p.out = D;
  p.sa = scale_a, p.sb = scale_b, p.sa_s = sa, p.sb_e = sb_e, p.sb_n = sb_n;
  p.raster = raster_of(N, kBand);
  p.idesc = idesc_of(format_of(b_type), format_of(a_type), b_n_major != 0, false);
  p.watch = watch_of(status);
  p.counters = static_cast<uint32_t*>(workspace);
  p.partial = reinterpret_cast<float*>(p.counters + kCutCounters);
  const int64_t most = (T / kTileRows + experts + 1) * ((N + kPairFeats - 1) / kPairFeats);
  if (most > INT32_MAX) return fail(DG_ERR_ARG, "T x N is too large (%lld tiles)", (long long)most);
  const bool f32 = d_type == DG_TYPE_F32;
  if (f8) return f32 ? run<true, false, false, true>(p, most, s) : run<true, false, false, false>(p, most, s);
  if (b_n_major) return f32 ? run<false, true, false, true>(p, most, s) : run<false, true, false, false>(p, most, s);
  return f32 ? run<false, false, false, true>(p, most, s) : run<false, false, false, false>(p, most, s);
}

extern "C" size_t dg_layer_grouped_grad_workspace(int experts, int64_t N, int64_t K) {
  if (experts < 1 || N <= 0 || K <= 0) return 256;
  return (size_t)experts * kTailRows * (size_t)(N + K) * 2 + 256;
}

extern "C" int dg_layer_grouped_weight_grad(const void* dD, int64_t ld_d, const void* A, int64_t ld_a,
                                            const int32_t* ends, int experts, void* dB, int d_type, int64_t T,
                                            int64_t N, int64_t K, void* workspace, void* products_workspace, void* status, void* stream) {
  if (int rc = check_sizes(T, N, K, experts)) return rc;
  if (d_type != DG_TYPE_BF16 && d_type != DG_TYPE_F32) return fail(DG_ERR_ARG, "dB is bf16 or fp32 (got type %d)", d_type);
  if (N % 8 || K % 8) return fail(DG_ERR_SHAPE, "N %% 8 and K %% 8 must be 0 (N %lld, K %lld)", (long long)N, (long long)K);
  if (N == 0 || K == 0) return DG_OK;
  if (!dB) return fail(DG_ERR_ARG, "dB must not be null");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = d_type == DG_TYPE_F32;
  if (T == 0) {
    DGL_CUDA(cudaMemsetAsync(dB, 0, (size_t)experts * N * K * (f32 ? 4 : 2), s));
    return DG_OK;
  }
  if (!dD || !A || !ends || !workspace || !products_workspace || !status) return fail(DG_ERR_ARG, "a required pointer is null");
  if (!aligned16(dD) || !aligned16(A) || !aligned16(dB) || !aligned16(workspace) || !aligned16(products_workspace) || ld_d % 8 || ld_a % 8)
    return fail(DG_ERR_ARG, "dD, A, dB, their pitches and the workspaces must be multiples of 16 bytes");
  if (ld_d < N || ld_a < K) return fail(DG_ERR_ARG, "a pitch is shorter than its rows");
  const int64_t tiles = (int64_t)experts * ((N + kTileRows - 1) / kTileRows) * ((K + kPairFeats - 1) / kPairFeats);
  if (tiles > INT32_MAX) return fail(DG_ERR_ARG, "experts x N x K is too large (%lld tiles)", (long long)tiles);
  __nv_bfloat16* a_tail = static_cast<__nv_bfloat16*>(workspace);
  __nv_bfloat16* d_tail = a_tail + (int64_t)experts * kTailRows * K;
  Args p{};
  const int64_t pd[3] = {K, T, 1}, ps[2] = {ld_a, ld_a * T}, ptd[3] = {K, kTailRows, experts}, pts[2] = {K, K * kTailRows};
  const int64_t qd[2] = {N, T}, qs[1] = {ld_d}, qtd[2] = {N, (int64_t)experts * kTailRows}, qts[1] = {N};
  if (int rc = encode_map(&p.p, A, 2, 3, pd, ps, 64)) return rc;
  if (int rc = encode_map(&p.q[0], dD, 2, 2, qd, qs, 64)) return rc;
  if (int rc = encode_map(&p.p_tail, a_tail, 2, 3, ptd, pts, 64)) return rc;
  if (int rc = encode_map(&p.q_tail, d_tail, 2, 2, qtd, qts, 64)) return rc;
  p.ends = ends, p.experts = experts, p.T = (int)T, p.feats = (int)K, p.rows = (int)N, p.red = 0, p.out = dB;
  p.raster = raster_of(K, kBand);
  p.counters = static_cast<uint32_t*>(products_workspace);
  p.idesc = idesc_of(1, 1, true, true);
  p.watch = watch_of(status);
  const int64_t vecs = 64 * (N + K) / 8;
  // a vector per thread, but no more than a thousand blocks in all (most groups' tails are short)
  const int64_t most_x = 1024 / experts > 8 ? 1024 / experts : 8, want_x = (vecs + 255) / 256;
  const unsigned gx = (unsigned)(want_x < most_x ? want_x : most_x);
  if (int rc = dgl::launch(grouped_tail_kernel, dim3(gx, experts), dim3(256), 0, s, ends, (int)T,
                           static_cast<const __nv_bfloat16*>(A), ld_a, K, a_tail, static_cast<const __nv_bfloat16*>(dD),
                           ld_d, N, d_tail))
    return rc;
  return f32 ? run<false, true, true, true>(p, tiles, s) : run<false, true, true, false>(p, tiles, s);
}

extern "C" size_t dg_layer_grouped_grad8_workspace(int64_t T, int experts, int64_t N, int64_t K) {
  if (T <= 0 || N <= 0 || K <= 0) return 256;
  return dg_layer_grouped_grad_workspace(experts, N, K) + (size_t)T * (size_t)K * 2;
}

// From rows kept in 8-bit blocks.  The scales differ from row to row, along which
// the product sums, and both of its operands have one type: so the values go through
// the workspace in bf16 first (8192 x 8192: 33 us, beside 165 us of the product for
// 8 experts of 2048).
extern "C" int dg_layer_grouped_weight_grad8(const void* dD, int64_t ld_d, const void* values, int type, const float* scales,
                                             int64_t s_row, int64_t s_block, const int32_t* ends, int experts, void* dB, int n_major,
                                             int d_type, int64_t T, int64_t N, int64_t K, void* workspace,
                                             void* products_workspace, void* status, void* stream) {
  if (int rc = check_sizes(T, N, K, experts)) return rc;
  if (!is_fp8(type)) return fail(DG_ERR_ARG, "8-bit blocks hold e4m3 or e5m2 (got type %d)", type);
  if (K % 16) return fail(DG_ERR_SHAPE, "K %% 16 must be 0 (got %lld)", (long long)K);
  if (d_type != DG_TYPE_BF16 && d_type != DG_TYPE_F32) return fail(DG_ERR_ARG, "dB is bf16 or fp32 (got type %d)", d_type);
  if (N % 8) return fail(DG_ERR_SHAPE, "N %% 8 must be 0 (got %lld)", (long long)N);
  if (T > 0 && N > 0 && K > 0) {
    if (!dD || !values || !scales || !ends || !dB || !workspace || !products_workspace || !status)
      return fail(DG_ERR_ARG, "a required pointer is null");
    if (!aligned16(dD) || !aligned16(values) || !aligned16(dB) || !aligned16(workspace) || !aligned16(products_workspace) || ld_d % 8)
      return fail(DG_ERR_ARG, "dD, its pitch, the values, dB and the workspaces must be multiples of 16 bytes");
    if (ld_d < N) return fail(DG_ERR_ARG, "a pitch is shorter than its rows");
    if (int rc = dg_layer_block8_dequantize(values, type, scales, s_row, s_block, 1, workspace, DG_TYPE_BF16, T, K, stream)) return rc;
  }
  void* rest = workspace ? static_cast<uint8_t*>(workspace) + (size_t)T * (size_t)K * 2 : nullptr;
  if (n_major)  // the gradient's transpose: the other operand's columns are the contiguous ones
    return dg_layer_grouped_weight_grad(workspace, K, dD, ld_d, ends, experts, dB, d_type, T, K, N, rest, products_workspace, status,
                                        stream);
  return dg_layer_grouped_weight_grad(dD, ld_d, workspace, K, ends, experts, dB, d_type, T, N, K, rest, products_workspace, status,
                                      stream);
}
