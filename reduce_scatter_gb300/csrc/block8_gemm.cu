// block8_gemm.cu -- product of two 8-bit tensors with an fp32 scale for each
// block of 128 (dg_layer_block8_matmul).
//
//   D[m, n] = sum over K blocks j of sa[m, j] sb[n, j] sum_{k in j} a[m, k] b[n, k]
//
// The tensor cores sum one K block of 128 at a time into one of two fp32
// accumulators (256 x 256 of a CTA pair, half of tensor memory each); eight warps
// read it, multiply it by the block's scales and add it to the running sums,
// which stay in their registers (32 rows x 128 columns a warp, 128 sums a
// thread), while the tensor cores fill the other one.  Rows lie on the
// accumulator's lanes here, so that a thread's sums share their row's scale, and
// a warp's 128 columns the scale of b's 128 x 128 block: one factor per thread
// and K block, and no operand but the accumulator itself.
//
// b with a scale for each row (1 x 128) costs a product more per sum, and the scales'
// way into the registers: loads from shared memory and from tensor memory share the
// way back, and a row a thread would read 128 column scales a K block (8192^3: 1233
// us).  There tensor memory is read so that a thread has four rows of 32 columns (16
// lanes at a time): a quarter of the scales, which asynchronous copies bring into a
// ring of four K blocks in shared memory (745 us).
//
// Bound by the tensor cores' and the summing warps' share of tensor and shared
// memory: 8192^3 427 us (2.6 PFLOP/s); the products alone 303, without the sums'
// arithmetic 303, with half of it 390.  To fp32 657 us with the same loop: it is
// sensitive to where the compiler keeps the sums (see the stores' wait below).
//
// Warp 0 loads (TMA, 128-byte swizzle), warp 1 issues the MMAs (even CTA of the
// pair), warps 2-9 add up and store.  Either operand may lie with its other
// dimension contiguous (an MN-major operand), as the gradients need it: then its
// blocks are 128 x 128.

#include <cuda_bf16.h>

#include "block8_few.h"
#include "launch.cuh"
#include "pairs.cuh"
#include "ptx.cuh"

namespace {

using namespace dgl;

constexpr int kTile = 256;    // rows and columns
constexpr int kStages = 5;
constexpr int kBlockK = 128;
constexpr uint32_t kStage = 2 * kStageP;          // 128 rows of each operand
constexpr uint32_t kBox = 32 * 128;               // 32 rows x 128 bytes of output
constexpr uint32_t kSmem = kStages * kStage + kEpiWarps * 2 * kBox + 256 + 1024;
constexpr uint32_t kTmemCols = 2 * kTile;
constexpr int64_t kSlot = (int64_t)cut_slot_floats(kTile);
constexpr int kBand = 8;
constexpr int kAhead = 3;     // K blocks by which the column scales are ahead (a power of two less one)

struct Args {
  CUtensorMap a, b, d;     // boxes of 128 bytes x 128 rows; of 128 bytes x 32 rows
  int rows, cols, kblocks, row_tiles;
  int a_mn, b_mn;          // the operand's rows are K's (contiguous along M or N)
  // scale of row m, K block j: sa[(m >> a_shift) * sa_m + j * sa_k]
  const float *sa, *sb;
  int64_t sa_m, sa_k, sb_n, sb_k;
  int a_shift, b_shift;
  int cols_next;           // b's scales of neighbouring columns lie next to each other, in whole vectors of 16 bytes
  uint32_t idesc;
  Raster raster;
  Divider per_unit;
  uint32_t* counters;
  float* partial;
  Watch watch;
};

__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t src, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// COLS: b has a scale for each row (1 x 128).
template <bool COLS, bool OUT32>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1) block8_kernel(const __grid_constant__ Args p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* boxes = smem + kStages * kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(boxes + kEpiWarps * 2 * kBox);
  const uint32_t full = smem_u32(bars), empty = full + 8 * kStages, tfull = empty + 8 * kStages, tempty = tfull + 16;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * kStages + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t half = cluster_ctarank();
  const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;
  let_next_start();
  if (threadIdx.x < 3) prefetch_map(threadIdx.x == 0 ? &p.a : threadIdx.x == 1 ? &p.b : &p.d);
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
  // (leaving and joining a tile's sums costs about 20 of its K blocks, which are slow ones)
  const Cut cut = cut_of(total, units, p.per_unit, p.kblocks, (float)kChunk * (float)total);

  if (warp == 0) {
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    Item w;
    for (Walk walk(cut, unit, units, total); ok && walk.get(w);) {
      int r, c;
      raster_at(p.raster, w.tile, p.row_tiles, r, c);
      const int m0 = r * kTile + (int)half * kLanes, n0 = c * kTile + (int)half * kLanes;
      for (int kb = w.kb0; kb < w.kb1; ++kb) {
        if (!(ok = mbar_wait_warp(p.watch, empty + 8 * stage, phase ^ 1, 0x100u | stage))) break;
        const uint32_t fb = mapa(full + 8 * stage, 0);
        const uint32_t sp = base + stage * kStage;
        if (elect_one()) {
          if (half == 0) mbar_expect(full + 8 * stage, 2 * kStage);
          const int k = kb * kBlockK;
          tma_2d(sp, &p.a, fb, p.a_mn ? m0 : k, p.a_mn ? k : m0);
          tma_2d(sp + kStageP, &p.b, fb, p.b_mn ? n0 : k, p.b_mn ? k : n0);
        }
        __syncwarp();
        if (++stage == kStages) stage = 0, phase ^= 1;
      }
    }
  } else if (warp == 1) {
    if (half == 0) {
      uint32_t stage = 0, phase = 0, it = 0;
      bool ok = true;
      Item w;
      // from one instruction (K = 32) to the next: 32 bytes of a row, or 32 rows
      const uint64_t a_step = p.a_mn ? 32 * kRowBytes / 16 : 2, b_step = p.b_mn ? 32 * kRowBytes / 16 : 2;
      for (Walk walk(cut, unit, units, total); ok && walk.get(w);) {
        for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
          const uint32_t buf = it & 1;
          if (!(ok = mbar_wait_warp(p.watch, full + 8 * stage, phase, 0x300u | stage))) break;
          if (!(ok = mbar_wait_warp(p.watch, tempty + 8 * buf, ((it >> 1) & 1) ^ 1, 0x200u | buf))) break;
          fence_after();
          const uint32_t sp = base + stage * kStage;
          const uint64_t ad = desc_k_major(sp), bd = desc_k_major(sp + kStageP);  // (MN-major: one swizzle span wide, the same fields)
          const uint32_t d = tmem + buf * kTile;
          if (elect_one()) {
#pragma unroll
            for (uint32_t s = 0; s < 4; ++s) mma_pair<true>(d, ad + s * a_step, bd + s * b_step, p.idesc, s != 0);
            commit_pair(tfull + 8 * buf);
            commit_pair(empty + 8 * stage);
          }
          __syncwarp();
          if (++stage == kStages) stage = 0, phase ^= 1;
        }
      }
    }
  } else {
    const int q = warp & 3;            // the lanes that this warp may read
    const int side = (warp - 2) >> 2;  // its half of the columns
    const uint32_t box = smem_u32(boxes) + (uint32_t)(warp - 2) * 2 * kBox;
    const uint32_t col_table = box + kBox;  // COLS: the 128 column scales of kAhead + 1 K blocks by turns, in the second box
    uint32_t it = 0;
    bool ok = true;
    Item w;
    for (Walk walk(cut, unit, units, total); ok && walk.get(w);) {
      int r, c;
      raster_at(p.raster, w.tile, p.row_tiles, r, c);
      const int m0 = r * kTile + (int)half * kLanes + q * 32, n0 = c * kTile + side * 128;  // this warp's first row and column
      const bool mine = m0 < p.rows && n0 < p.cols;
      const float* sa = p.sa + (int64_t)(min(m0 + lane, p.rows - 1) >> p.a_shift) * p.sa_m;
      const float* sb = p.sb + (int64_t)(min(n0, p.cols - 1) >> p.b_shift) * p.sb_n;
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      float a_next = __ldg(sa + w.kb0 * p.sa_k), b_next = COLS ? 0.f : __ldg(sb + w.kb0 * p.sb_k);
      // (copied past the registers, which the sums fill)
      auto fetch_cols = [&](int kb) {
        if (kb < w.kb1) {
          const uint32_t to = col_table + (uint32_t)(kb & kAhead) * 512;
          if (p.cols_next) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + lane * 16),
                         "l"(p.sb + min(n0 + 4 * lane, p.cols - 4) + kb * p.sb_k)
                         : "memory");
          } else {
#pragma unroll 1
            for (int i = lane; i < 128; i += 32)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + i * 4),
                           "l"(p.sb + min(n0 + i, p.cols - 1) * p.sb_n + kb * p.sb_k)
                           : "memory");
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      if constexpr (COLS) {
        if (lane == 0) stores_read<0>();  // the last tile's stores have left the box
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch_cols(w.kb0 + i);
      }
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
        const uint32_t buf = it & 1;
        const float s = COLS ? a_next : a_next * b_next;
        const uint64_t s2 = pair_of(s, s);
        const uint32_t table = col_table + (uint32_t)(kb & kAhead) * 512 + (lane & 3) * 8;  // (this thread's first columns)
        uint64_t rows[2][2];  // COLS: the scales of the four rows that a thread reads
        const int kn = min(kb + 1, w.kb1 - 1);
        a_next = __ldg(sa + kn * p.sa_k);
        if constexpr (COLS) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
          __syncwarp();  // every lane's part is there, and the table that is written next has been read
          fetch_cols(kb + kAhead);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float r = __shfl_sync(0xffffffffu, s, 8 * i + (lane >> 2));
            rows[i >> 1][i & 1] = pair_of(r, r);
          }
        } else {
          b_next = __ldg(sb + kn * p.sb_k);
        }
        if (!(ok = mbar_wait_warp(p.watch, tfull + 8 * buf, (it >> 1) & 1, 0x400u | buf))) break;
        fence_after();
        if (mine) {
          const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + buf * kTile + side * 128;
          if constexpr (COLS) {
            // steps of 16 columns, their lower and upper 16 rows
            uint64_t cs[2];
            uint32_t u[2][8];
            tmem_ld_rows16(at, u[0]);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if ((j & 1) == 0) {
                asm volatile("ld.shared.b64 %0, [%1];" : "=l"(cs[0]) : "r"(table + j * 32));
                asm volatile("ld.shared.b64 %0, [%1];" : "=l"(cs[1]) : "r"(table + j * 32 + 32));
              }
              uint64_t both[4];  // the products of the scales
#pragma unroll
              for (int i = 0; i < 4; ++i) both[i] = mul2(cs[i >> 1], rows[j & 1][i & 1]);
              tmem_ld_wait(u[j & 1]);
              if (j < 15) tmem_ld_rows16(at + (j + 1) / 2 * 16 + ((uint32_t)((j + 1) & 1) << 20), u[(j + 1) & 1]);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[j * 4 + i] = fma2(pair_of(__uint_as_float(u[j & 1][2 * i]), __uint_as_float(u[j & 1][2 * i + 1])), both[i], acc[j * 4 + i]);
            }
          } else {
            uint32_t u[2][16];
            tmem_ld16(at, u[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              tmem_ld_wait(u[j & 1]);
              if (j < 7) tmem_ld16(at + (j + 1) * 16, u[(j + 1) & 1]);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint64_t f = pair_of(__uint_as_float(u[j & 1][2 * i]), __uint_as_float(u[j & 1][2 * i + 1]));
                acc[j * 8 + i] = fma2(f, s2, acc[j * 8 + i]);
              }
            }
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa(tempty + 8 * buf, 0));
      }
      if (!ok) break;
      if (!mine) continue;
      if constexpr (!COLS) {  // the last tile's stores have left the boxes, which at an edge are an odd number (a count that
                              // goes on over the tiles, in place of the wait: other registers, 8192^3 427 -> 543 us)
        if (lane == 0) stores_read<0>();
        __syncwarp();
      }
      // 32 columns of this warp's box, from v (this lane's row; COLS: four rows and eight columns of it, as they were read)
      auto emit = [&](int c32, const float(&v)[32]) {
        constexpr int per_box = OUT32 ? 1 : 2;  // such steps in 128 bytes
        const int b = c32 / per_box, part = c32 % per_box;
        if (n0 + b * 32 * per_box >= p.cols) return;
        const uint32_t to = box + (uint32_t)(b & 1) * kBox;
        if (part == 0) {
          if (lane == 0) stores_read<1>();  // the store before the last one has left its box
          __syncwarp();
        }
        if constexpr (COLS) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int row = (i & 4) * 4 + (i & 1) * 8 + (lane >> 2), col = part * 32 + (i >> 3) * 16 + (i & 2) * 4 + (lane & 3) * 2;
            const uint32_t bytes = (uint32_t)col * (OUT32 ? 4 : 2), at = to + row * 128 + (((bytes >> 4) ^ (row & 7)) << 4) + (bytes & 15);
            if constexpr (OUT32) {
              asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v[2 * i]), "f"(v[2 * i + 1]) : "memory");
            } else {
              const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(*reinterpret_cast<const uint32_t*>(&h)) : "memory");
            }
          }
        } else {
          const uint32_t row = to + lane * 128;
#pragma unroll
          for (int i = 0; i < (OUT32 ? 8 : 4); ++i) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (OUT32) {
                x[k] = __float_as_uint(v[4 * i + k]);
              } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]);
                x[k] = *reinterpret_cast<const uint32_t*>(&h);
              }
            }
            const uint32_t chunk = (uint32_t)(part * 4 + i) ^ (lane & 7);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + chunk * 16), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                         "r"(x[3])
                         : "memory");
          }
        }
        if (part == per_box - 1) {
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) store_box(&p.d, to, n0 + b * 32 * per_box, m0);
        }
      };
      int ways = 1;
      if (w.tile < cut.tiles && (ways = cut_ways(cut, w.tile)) > 1) {
        const int head = cut_first(cut, w.tile);
        auto slot = [&](int pair) { return p.partial + cut_slot(cut, w.tile, pair) * kSlot + half * (kSlot / 2); };
        float* to = slot(unit);
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          const float2 f = unpair(acc[i]);
          __stcg(to + (int64_t)(side * 128 + 2 * i) * kLanes + q * 32 + lane, f.x);
          __stcg(to + (int64_t)(side * 128 + 2 * i + 1) * kLanes + q * 32 + lane, f.y);
        }
        if (!warp_last(p.counters + 4 * w.tile + 2 * half + side, q, ways, lane)) continue;
#pragma unroll 1
        for (int c32 = 0; c32 < 4; ++c32) {
          float v[32];
          join_partials(ways, [&](int j) { return slot(head + j); }, side * 128 + c32 * 32, q * 32 + lane, v);
          emit(c32, v);
        }
      } else {
#pragma unroll
        for (int c32 = 0; c32 < 4; ++c32) {
          float v[32];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 f = unpair(acc[c32 * 16 + i]);
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
          }
          emit(c32, v);
        }
      }
    }
    if (!ok) settle();
    if (COLS) asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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

template <bool COLS, bool OUT32>
int run(Args& p, cudaStream_t s) {
  int sms = 0;
  if (int rc = sm_count(&sms)) return rc;
  DGL_CUDA(cudaFuncSetAttribute(block8_kernel<COLS, OUT32>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem));
  p.per_unit = divider_of((uint64_t)(sms / 2));
  return dgl::launch(block8_kernel<COLS, OUT32>, dim3((unsigned)(sms / 2 * 2)), dim3(kThreads), kSmem, s, p);
}

constexpr int64_t kMaxSize = INT32_MAX - 255;

// One operand: its map, and the strides of its scales.
int operand(CUtensorMap* map, const void* values, int trans, int64_t outer, int64_t K, int64_t s_row, int64_t s_block,
            int block_rows, int64_t* s_outer, int64_t* s_k, int* shift) {
  const int64_t dims[2] = {trans ? outer : K, trans ? K : outer}, pitch[1] = {dims[0]};
  if (int rc = encode_map(map, values, 1, 2, dims, pitch, 128)) return rc;
  *s_outer = trans ? s_block : s_row;
  *s_k = trans ? s_row : s_block;
  *shift = trans || block_rows == 128 ? 7 : 0;
  return DG_OK;
}

}  // namespace

extern "C" int dg_layer_block8_matmul(const void* a, int a_type, const float* a_scales, int64_t sa_row, int64_t sa_block,
                                      int a_block_rows, int trans_a, const void* b, int b_type, const float* b_scales,
                                      int64_t sb_row, int64_t sb_block, int b_block_rows, int trans_b, void* D, int d_type,
                                      int64_t M, int64_t N, int64_t K, void* workspace, void* status, void* stream) {
  if (M < 0 || N < 0 || K < 0 || M > kMaxSize || N > kMaxSize || K > kMaxSize)
    return fail(DG_ERR_ARG, "M %lld, N %lld, K %lld out of range", (long long)M, (long long)N, (long long)K);
  if (!is_fp8(a_type) || !is_fp8(b_type)) return fail(DG_ERR_ARG, "a and b hold e4m3 or e5m2 (types %d, %d)", a_type, b_type);
  if (d_type != DG_TYPE_BF16 && d_type != DG_TYPE_F32) return fail(DG_ERR_ARG, "D is bf16 or fp32 (got type %d)", d_type);
  if ((a_block_rows != 1 && a_block_rows != 128) || (b_block_rows != 1 && b_block_rows != 128))
    return fail(DG_ERR_ARG, "a block has 1 or 128 rows (got %d, %d)", a_block_rows, b_block_rows);
  if ((trans_a && a_block_rows != 128) || (!trans_b && b_block_rows != 128))
    return fail(DG_ERR_ARG, "an operand whose rows are summed over needs blocks of 128 rows");
  if (N % 8 || (trans_a ? M : K) % 16 || (trans_b ? K : N) % 16)
    return fail(DG_ERR_SHAPE, "N %% 8 and the columns of a and b %% 16 must be 0 (M %lld, N %lld, K %lld)", (long long)M, (long long)N,
                (long long)K);
  if (M == 0 || N == 0) return DG_OK;
  if (!D || !status) return fail(DG_ERR_ARG, "D and status must not be null");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) {
    DGL_CUDA(cudaMemsetAsync(D, 0, (size_t)M * N * (d_type == DG_TYPE_F32 ? 4 : 2), s));
    return DG_OK;
  }
  if (!a || !a_scales || !b || !b_scales || !workspace) return fail(DG_ERR_ARG, "values, scales and the workspace must not be null");
  if (!aligned16(a) || !aligned16(b) || !aligned16(D) || !aligned16(workspace))
    return fail(DG_ERR_ARG, "values, D and the workspace must be 16-byte aligned");
  const int64_t tiles = ((M + kTile - 1) / kTile) * ((N + kTile - 1) / kTile);
  if (tiles > INT32_MAX) return fail(DG_ERR_ARG, "M x N is too large (%lld tiles)", (long long)tiles);
  Args p{};
  const bool f32 = d_type == DG_TYPE_F32;
  if (M <= kFewRows && !trans_a) {  // (8 rows of 8192 x 28672: 62 us here)
    const FewRows f{a, b, a_type, b_type, !trans_b, a_scales, b_scales, sa_row, sa_block, trans_b ? sb_row : sb_block,
                    trans_b ? sb_block : sb_row, a_block_rows == 128 ? 7 : 0, b_block_rows == 128 ? 7 : 0, D, f32, M, N, K, workspace, status};
    return block8_few(f, stream);
  }
  if (int rc = operand(&p.a, a, trans_a, M, K, sa_row, sa_block, a_block_rows, &p.sa_m, &p.sa_k, &p.a_shift)) return rc;
  if (int rc = operand(&p.b, b, !trans_b, N, K, sb_row, sb_block, b_block_rows, &p.sb_n, &p.sb_k, &p.b_shift)) return rc;
  const int64_t dd[2] = {N, M}, dp[1] = {N};
  if (int rc = encode_map(&p.d, D, f32 ? 4 : 2, 2, dd, dp, 32)) return rc;
  p.rows = (int)M, p.cols = (int)N, p.kblocks = (int)((K + kBlockK - 1) / kBlockK), p.row_tiles = (int)((M + kTile - 1) / kTile);
  p.a_mn = trans_a != 0, p.b_mn = trans_b == 0;
  p.sa = a_scales, p.sb = b_scales;
  p.idesc = idesc_of(a_type == DG_TYPE_E5M2, b_type == DG_TYPE_E5M2, p.a_mn != 0, p.b_mn != 0) | idesc_columns(kTile);
  p.raster = raster_of(N, kBand);
  p.counters = static_cast<uint32_t*>(workspace);
  p.partial = reinterpret_cast<float*>(p.counters + kCutCounters);
  p.watch = Watch{static_cast<unsigned long long*>(status), next_tag(), 4000000000ull};
  const bool cols = p.b_shift == 0;
  p.cols_next = cols && p.sb_n == 1 && p.sb_k % 4 == 0 && aligned16(b_scales);
  if (cols) return f32 ? run<true, true>(p, s) : run<true, false>(p, s);
  return f32 ? run<false, true>(p, s) : run<false, false>(p, s);
}
