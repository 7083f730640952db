// layer_common.h -- host helpers shared by the translation units behind
// include/dg_layer.h: error messages, device properties, tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "dg_layer.h"

namespace dgl {

// Record a message for dg_layer_last_error() and return `code`.
int fail(int code, const char* fmt, ...);
int cuda_fail(cudaError_t e, const char* what);

#define DGL_CUDA(call)                                       \
  do {                                                       \
    cudaError_t e_ = (call);                                 \
    if (e_ != cudaSuccess) return dgl::cuda_fail(e_, #call); \
  } while (0)

int sm_count(int* n);

// A tag for the next launch of a product, with which it marks the status word if
// it gives up: never 0, which the word of a device without such a launch holds.
inline uint32_t next_tag(std::atomic<uint32_t>& last) {
  uint32_t tag;
  do tag = last.fetch_add(1, std::memory_order_relaxed) + 1;
  while (tag == 0);
  return tag;
}
uint32_t next_tag();  // of the process's counter

// A tiled tensor map with the 128-byte swizzle over `rank` (2 or 3) dimensions
// of esz-byte elements, innermost first; strides in elements (stride[0] is
// dimension 1's).  The box's inner extent is 128 bytes.
int encode_map(CUtensorMap* map, const void* base, int esz, int rank, const int64_t* dims, const int64_t* strides,
               int box_rows);

// A map over the 4-bit scale layout: (256 words of 4 bytes: the scales of 128
// rows x 256 columns, K blocks, row tiles), boxes of one K block and `box_tiles`
// row tiles.
int encode_scale_map(CUtensorMap* map, const void* base, int64_t kblocks, int64_t row_tiles, int box_tiles);

inline bool is_fp8(int type) { return type == DG_TYPE_E4M3 || type == DG_TYPE_E5M2; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace dgl
