// ptx.cuh -- PTX wrappers of the matrix-product kernels behind
// include/dg_layer.h (CTA pairs: tcgen05 cta_group::2, TMA into a pair,
// mbarriers), their bounded waits and the epilogue's stores.
//
// The kernels compute D^T: the dimension that is contiguous in memory (the
// output features) lies on the accumulator's 128 x 2 lanes, the output's rows
// on its columns.  A column count is a run-time field of the instruction
// descriptor, so a ragged group of rows costs its own rows (rounded up to 32)
// and not a whole tile, and a handful of rows still fills the tensor core's M.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

namespace dgl {

constexpr int kEpiWarps = 8;          // two for each quarter of the lanes
constexpr int kThreads = 64 + 32 * kEpiWarps;  // producer warp, MMA warp, epilogue warps
constexpr int kLanes = 128;           // output features per CTA (accumulator lanes)
constexpr int kPairFeats = 2 * kLanes;
constexpr uint32_t kRowBytes = 128;   // one operand row of a K block (the swizzle span)
constexpr uint32_t kStageP = kLanes * kRowBytes;
constexpr int kChunk = 32;            // output rows (accumulator columns) per epilogue step
constexpr int kPairPitch = 36;        // words from one row pair of a box to the next (bank-conflict free)
constexpr uint32_t kStoreBuf = kChunk / 2 * kPairPitch * 4;  // one warp's 32 x 32 bf16 box

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One lane of a converged warp.  The loading and the issuing warp run their
// loops with all lanes and let the elected one act: the compiler then keeps
// descriptors and addresses in uniform registers, where the asynchronous
// instructions take them from.  (With the loop inside a one-lane branch each
// such instruction took 58-70 cycles to issue, which bounded the 4-bit product
// and short reductions.)
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok));
  return ok != 0;
}

// ----------------------------------------------------------------- mbarriers

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Arrive on a barrier of either CTA.  The release is of this CTA's scope: what it
// orders here are reads of tensor memory, complete by then (tcgen05.wait::ld),
// not writes that the other CTA reads.  A release of the cluster's scope waits
// for all of the thread's global stores, which held each accumulator for the
// time that the tile before took to reach memory (7000 cycles a tile).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Pipeline waits are bounded: after `limit_ns` the waiter records the wait in
// the caller's status word, tagged with the launch's epoch, and every role of
// every CTA of the launch that waits from then on gives up too.
struct Watch {
  unsigned long long* status;
  uint32_t epoch;
  uint64_t limit_ns;
};
__device__ __forceinline__ bool gave_up(const Watch& w) {
  unsigned long long v;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(w.status) : "memory");
  return (uint32_t)(v >> 32) == w.epoch;
}
static __device__ __noinline__ bool mbar_wait_slow(const Watch& w, uint32_t bar, uint32_t parity, uint32_t what) {
  const uint64_t t0 = globaltimer();
  for (uint32_t n = 1;; ++n) {
    if (mbar_try(bar, parity)) return true;
    if ((n & 255u) == 0) {
      if (gave_up(w)) return false;
      if (globaltimer() - t0 > w.limit_ns) {
        atomicExch(w.status, ((unsigned long long)w.epoch << 32) | what);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool mbar_wait(const Watch& w, uint32_t bar, uint32_t parity, uint32_t what) {
  if (mbar_try(bar, parity)) return true;
  return mbar_wait_slow(w, bar, parity, what);
}
// The same by a whole warp, which agrees on the outcome: a lane that gave up must
// not leave the others at the next warp-wide instruction.
__device__ __forceinline__ bool mbar_wait_warp(const Watch& w, uint32_t bar, uint32_t parity, uint32_t what) {
  bool ok = mbar_try(bar, parity);
  if (__any_sync(0xffffffffu, !ok)) ok = __all_sync(0xffffffffu, ok || mbar_wait_slow(w, bar, parity, what)) != 0;
  return ok;
}
// Before a launch that gave up ends, its copies and MMAs in flight land.
static __device__ __noinline__ void settle() {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < 20000000ull) __nanosleep(1000);
}

// ----------------------------------------------------------------------- TMA

// Loads into this CTA's shared memory that complete on a barrier of either CTA
// of the pair (here: the even CTA's).
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y,
                                       int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// ------------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D (both CTAs' accumulators) = P Q [+ D]; bf16 (K = 16) or 8-bit (K = 32) operands.
template <bool F8>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t pdesc, uint64_t qdesc, uint32_t idesc, uint32_t acc) {
  if constexpr (F8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(pdesc), "l"(qdesc), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(pdesc), "l"(qdesc), "r"(idesc), "r"(acc)
        : "memory");
}
// One arrival on the barrier at this offset in both CTAs of the pair once the
// issuing thread's earlier tcgen05 operations are complete.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// 32 lanes x 32 columns: thread i of the warp gets columns 0..31 of lane i.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Shared-memory descriptors of operand tiles that TMA wrote with the 128-byte
// swizzle: version 1 (bit 46), swizzle code 2 (bits 61-63), offsets in 16-byte
// units.  K-major: rows of 128 bytes along K, groups of 8 rows 1024 bytes apart
// (stride offset).  MN-major: rows of 64 values along M (or N), one row per k;
// groups of 8 k 1024 bytes apart (stride offset), the next 64 values
// `next_bytes` further (leading offset).
__device__ __forceinline__ uint64_t desc_k_major(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t addr, uint32_t next_bytes) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(next_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: fp32 accumulator (bits 4-5), P and Q formats (bits
// 7-9, 10-12), MN-major flags (bits 15, 16), columns / 8 (bit 17), lanes / 16 (bit 24).
__host__ __device__ constexpr uint32_t idesc_of(uint32_t p_fmt, uint32_t q_fmt, bool p_mn, bool q_mn) {
  return (1u << 4) | (p_fmt << 7) | (q_fmt << 10) | ((p_mn ? 1u : 0u) << 15) | ((q_mn ? 1u : 0u) << 16) |
         ((uint32_t)(kPairFeats >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_columns(uint32_t n) { return (n >> 3) << 17; }

// ------------------------------------------------------------- order of tiles

// Order of a matrix's tiles: bands of up to 16 row tiles swept feature tile by
// feature tile, so that the tiles in flight share operands in L2.  The divisions
// by a band's tiles and by its width are multiplications (the decoding stands
// before the first load of a tile, and a division took a third of a
// microsecond): m = floor(2^(31 + s) / d) + 1 with s = ceil(log2 d) gives exact
// quotients below 2^31, and 2^32 / w rounded up those by w <= 16 below 2^28.
struct Divider {  // by 2 <= d < 2^31
  uint32_t mul, shift;
  __device__ __forceinline__ int of(int n) const { return (int)(__umulhi((uint32_t)n, mul) >> shift); }
};
inline Divider divider_of(uint64_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return Divider{(uint32_t)((1ull << (31 + s)) / d + 1), s - 1};
}
struct Raster {
  Divider per_band;
  uint32_t width[17];
  int nf, band;  // feature tiles, row tiles of a band
};
inline Raster raster_of(int64_t feats, int band) {
  Raster r;
  r.nf = (int)((feats + kPairFeats - 1) / kPairFeats);
  r.band = band;
  r.per_band = divider_of((uint64_t)band * r.nf);
  r.width[0] = r.width[1] = 0;
  for (uint64_t w = 2; w <= 16; ++w) r.width[w] = (uint32_t)(((1ull << 32) + w - 1) / w);
  return r;
}
__device__ __forceinline__ void raster_at(const Raster& o, int tile, int row_tiles, int& row, int& feat) {
  const int band = o.per_band.of(tile), in = tile - band * o.band * o.nf;
  const int wide = min(o.band, row_tiles - band * o.band);
  feat = wide == 1 ? in : (int)__umulhi((uint32_t)in, o.width[wide]);
  row = band * o.band + in - feat * wide;
}

// The epilogue warps: warp w reads lane quarter w % 4, and of its tile's steps of
// 32 rows those of its half (the first four warps the even ones).  Eight warps
// rather than four: a step is a chain of latencies (tensor memory, shared
// memory, stores), and four left stores of short reductions at 2.4 TB/s.
//
// They decide together whether a tile's accumulator
// arrived (one thread waits; `go`: two words of shared memory, by turns), so
// that none is left at a barrier by one that gave up.
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory"); }
__device__ __forceinline__ bool epilogue_wait(const Watch& w, uint32_t tfull, uint32_t it, volatile uint32_t* go) {
  const uint32_t buf = it & 1;
  if (threadIdx.x == 64) go[buf] = mbar_wait(w, tfull + 8 * buf, (it >> 1) & 1, 0x400u | buf) ? 1u : 0u;
  epilogue_sync();
  if (go[buf] == 0) {
    settle();
    return false;
  }
  fence_after();
  return true;
}

// --------------------------------------------------------------- split tiles

// The tiles of a list walked by `units` CTA pairs.  Where the last round of
// tiles would leave many pairs idle, the list's first `cut` tiles (fewer than
// the pairs) are cut along K into equal shares of K blocks instead, one
// contiguous range of shares to a pair, and the rest is dealt out whole.  A
// pair's range meets at most two tiles.  The pairs of one cut tile leave fp32
// partial accumulators in the workspace and count themselves in; the last one
// adds them in the order of K (the same bits every time) and stores the tile.
// No pair waits for another.
constexpr int kMinShare = 8;   // K blocks
constexpr int kJoin = 3;       // partials whose loads are in flight at once
struct Cut {
  int tiles, kblocks, share;
};
// Few tall tiles are made shorter, so that more pairs take part, only where their
// features fit the L2 (64 MB of its 129): tiles that share features read them
// from DRAM once while they run side by side, and cut tiles do not.
constexpr int64_t kSharedBytes = 64000000;
// `all_rows`: of all the tiles together.  Leaving and joining partials costs about 4 us
// for up to 64 rows and 2.2 us for each further step of 32 rows and three
// partials (measured), a K block 0.2 us: so cutting pays for short tiles, as of
// a decoding step, and for tall ones with a long K and few of them.
// `per_unit`: division by the pairs.
constexpr int kShortCost = 20;  // K blocks
__device__ __forceinline__ Cut cut_of(int total, int units, const Divider& per_unit, int kblocks, float all_rows) {
  // (a K so long that the products below would pass 32 bits is left whole)
  if (kblocks <= kMinShare + kShortCost || kblocks > (1 << 20)) return Cut{0, kblocks, 0};
  Cut c{total - per_unit.of(total) * units, kblocks, 0};
  if (c.tiles == 0) return Cut{0, kblocks, 0};
  const float rows = __fdividef(all_rows, (float)total);
  c.share = max(kMinShare, per_unit.of(c.tiles * kblocks + units - 1));
  const float ways = __fdividef((float)kblocks, (float)c.share) + 1.f, steps = rows * (1.f / kChunk);
  const float cost = steps <= 2.f ? (float)kShortCost : 11.f * steps * ((ways + 2.f) * (1.f / kJoin) + 1.f) * 0.5f;
  return (float)(kblocks - c.share) > cost ? c : Cut{0, kblocks, 0};
}
// How many pairs share tile t of the cut ones, the first of them, and the
// workspace slot of the j-th pair's partial.
__device__ __forceinline__ int cut_first(const Cut& c, int t) { return t * c.kblocks / c.share; }
__device__ __forceinline__ int cut_ways(const Cut& c, int t) {
  return ((t + 1) * c.kblocks - 1) / c.share - cut_first(c, t) + 1;
}
__device__ __forceinline__ int cut_slot(const Cut& c, int t, int unit) {
  return 2 * unit + (unit * c.share / c.kblocks < t ? 1 : 0);
}

struct Item {
  int tile, kb0, kb1;
};
struct Walk {
  int pos, end, next, total, units, kblocks;
  __device__ __forceinline__ Walk(const Cut& c, int unit, int units_, int total_)
      : pos(min(unit * c.share, c.tiles * c.kblocks)), end(min(pos + c.share, c.tiles * c.kblocks)), next(c.tiles + unit),
        total(total_), units(units_), kblocks(c.kblocks) {}
  __device__ __forceinline__ bool get(Item& it) {
    if (pos < end) {
      it.tile = pos / kblocks;
      it.kb0 = pos - it.tile * kblocks;
      it.kb1 = min(kblocks, it.kb0 + end - pos);
      pos += it.kb1 - it.kb0;
      return true;
    }
    it.tile = next;
    it.kb0 = 0;
    it.kb1 = kblocks;
    next += units;
    return it.tile < total;
  }
};

// The whole tiles of a ragged list, dealt out as pairs become free (their costs
// differ: dealing them in turn left pairs idle for 4 to 7 % of the time).  Each
// pair starts with its own shares and one tile of its own; further tiles (`rest`
// of them; where there are none, nothing is drawn) come from a counter in the
// workspace, which the even CTA's loading warp draws from ahead of its need and
// passes on through a ring of slots in both CTAs' shared memory to the other
// loading warp, the issuing warp and the epilogues.  Every pair draws until it
// draws past the end, so the counter wraps back to 0 with the last draw of the
// launch.
constexpr int kDrawBlocks = 16;  // K blocks of a tile (on average) from which on drawing pays: it costs 0.3 us a tile
constexpr int kRing = 4;
constexpr int kRingReaders = 4;  // the issuing warp, the odd CTA's loading warp, two epilogues
struct Ring {
  uint32_t full, empty;  // barriers
  volatile int* slot;    // [kRing]
};
// A tile into slot s of both CTAs' rings (by one thread of the even CTA): the
// store itself completes the barrier's phase, so nothing waits for other stores.
__device__ __forceinline__ void ring_pass(const Ring& r, uint32_t s, int tile) {
  const uint32_t at = smem_u32((const void*)(r.slot + s));
#pragma unroll
  for (uint32_t c = 0; c < 2; ++c) {
    const uint32_t bar = mapa(r.full + 8 * s, c);
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(4) : "memory");
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(mapa(at, c)), "r"(tile),
                 "r"(bar)
                 : "memory");
  }
}
struct Feed {
  Walk walk;
  bool first = true;  // the pair's own whole tile is still to come
  int n = 0;          // tiles taken from the ring
  int rest;           // tiles that are drawn
  bool draw;
  __device__ __forceinline__ Feed(const Cut& c, int unit, int units, int total, bool draw_)
      : walk(c, unit, units, total), rest(draw_ ? max(0, total - c.tiles - units) : 0), draw(draw_) {}
  // Shares and the first whole tile (every one in turn, where none are drawn);
  // false: the ring's turn, or (none) the end.
  __device__ __forceinline__ bool own(Item& it) {
    if (!draw || walk.pos < walk.end) return walk.get(it);
    if (!first) return false;
    first = false;
    return walk.get(it);
  }
  __device__ __forceinline__ bool none() const { return rest == 0; }
  __device__ __forceinline__ bool take(int tile, Item& it) {
    it.tile = tile;
    it.kb0 = 0;
    it.kb1 = walk.kblocks;
    return tile >= 0 && tile < walk.total;
  }
  // One thread's wait for the next tile of the ring: -1 if it gave up.
  __device__ __forceinline__ int read(const Watch& w, const Ring& r) {
    const uint32_t s = n % kRing;
    if (!mbar_wait(w, r.full + 8 * s, (n / kRing) & 1, 0x500u | s)) return -1;
    const int t = r.slot[s];
    if (t >= 0) mbar_arrive_cluster(mapa(r.empty + 8 * s, 0));  // (always: the branch has the read complete before it)
    return t;
  }
};

// Workspace of the cut tiles: a counter for each (tile, half), which wraps back
// to 0 with its last pair, then slots of [half][column][lane].
constexpr int kCutCounters = 2 * 256;  // the last one is the tiles' counter
constexpr int kDrawCounter = kCutCounters - 1;
__host__ __device__ constexpr size_t cut_slot_floats(int columns) { return (size_t)2 * columns * kLanes; }
__host__ __device__ constexpr size_t cut_bytes(int units, int columns) {
  return kCutCounters * 4 + (size_t)2 * units * cut_slot_floats(columns) * 4;
}

// A warp's 32 x 32 box of a partial accumulator to its slot.
__device__ __forceinline__ void store_partial(float* slot, int column, int lane_of, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) __stcg(slot + (int64_t)(column + i) * kLanes + lane_of, v[i]);
}
// The sum of `ways` partials, in their order; slot(j): the j-th one's.
template <class Slot>
__device__ __forceinline__ void join_partials(int ways, Slot slot, int column, int lane_of, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 1
  for (int j = 0; j < ways; j += kJoin) {
    float u[kJoin][32];
#pragma unroll
    for (int k = 0; k < kJoin; ++k) {
      const float* s = slot(min(j + k, ways - 1)) + (int64_t)column * kLanes + lane_of;
#pragma unroll
      for (int i = 0; i < 32; ++i) u[k][i] = j + k < ways ? __ldcg(s + i * kLanes) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kJoin; ++k)
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += u[k][i];
  }
}
// After every epilogue thread of this half has stored its partial: whether this
// pair is the tile's last.  `flag`: a word of shared memory.
__device__ __forceinline__ bool cut_last(uint32_t* counter, int ways, volatile uint32_t* flag) {
  __threadfence();
  epilogue_sync();
  if (threadIdx.x == 64) *flag = atomicInc(counter, (uint32_t)ways - 1) == (uint32_t)ways - 1 ? 1u : 0u;
  epilogue_sync();
  const bool last = *flag != 0;
  if (last) __threadfence();
  return last;
}

// ------------------------------------------------------------ epilogue stores

// A warp's box of 32 features x 32 rows from registers (v[i]: row i, this
// lane's feature) to row-major memory: `d` points at (first row, first feature
// of the warp), `pitch` elements from row to row; rows_ok rows and feats_ok
// features (a multiple of 8) are stored.  bf16 goes through `buf` (kStoreBuf
// bytes of the warp's own) so that each lane stores 16 bytes; fp32 rows are
// whole 128-byte lines as they are.
__device__ __forceinline__ void store_box_f32(float* d, int64_t pitch, int rows_ok, int feats_ok, int lane,
                                              const float (&v)[32]) {
  if (lane < feats_ok) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < rows_ok) d[i * pitch + lane] = v[i];
  }
}
__device__ __forceinline__ void store_box_bf16(__nv_bfloat16* d, int64_t pitch, int rows_ok, int feats_ok, int lane,
                                               const float (&v)[32], uint8_t* buf) {
  // words of two rows' values of one feature go in, eight features of two rows
  // come out and are sorted into the rows
  uint32_t* w = reinterpret_cast<uint32_t*>(buf);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i * kPairPitch + lane] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __syncwarp();
  const int f = (lane & 3) * 8;
  __nv_bfloat16* at = d + (int64_t)(lane >> 2) * 2 * pitch + f;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = (j * 8 + (lane >> 2)) * 2;  // the first of the two rows
    const uint4* s = reinterpret_cast<const uint4*>(w + r / 2 * kPairPitch + f);
    const uint4 a = s[0], b = s[1];
    if (f < feats_ok) {
      __nv_bfloat16* to = at + j * 16 * pitch;
      if (r < rows_ok)
        *reinterpret_cast<uint4*>(to) = make_uint4(__byte_perm(a.x, a.y, 0x5410), __byte_perm(a.z, a.w, 0x5410),
                                                   __byte_perm(b.x, b.y, 0x5410), __byte_perm(b.z, b.w, 0x5410));
      if (r + 1 < rows_ok)
        *reinterpret_cast<uint4*>(to + pitch) = make_uint4(__byte_perm(a.x, a.y, 0x7632), __byte_perm(a.z, a.w, 0x7632),
                                                           __byte_perm(b.x, b.y, 0x7632), __byte_perm(b.z, b.w, 0x7632));
    }
  }
  __syncwarp();  // the box may be overwritten
}

}  // namespace dgl
