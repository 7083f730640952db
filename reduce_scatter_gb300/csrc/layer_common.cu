// layer_common.cu -- error messages, device properties and tensor maps of the
// calls behind include/dg_layer.h.

#include "layer_common.h"

#include <cstdarg>
#include <cstdio>
#include <mutex>

namespace dgl {
namespace {

thread_local char g_err[512] = "";

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    cudaDriverEntryPointQueryResult q;
    void* f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

}  // namespace

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

int cuda_fail(cudaError_t e, const char* what) { return fail(DG_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e)); }

uint32_t next_tag() {
  static std::atomic<uint32_t> last{0};
  return next_tag(last);
}

int sm_count(int* n) {
  static std::mutex mu;
  static int cached[64] = {};
  int dev = 0;
  DGL_CUDA(cudaGetDevice(&dev));
  if (dev < 64) {
    std::lock_guard<std::mutex> lk(mu);
    if (cached[dev] == 0) DGL_CUDA(cudaDeviceGetAttribute(&cached[dev], cudaDevAttrMultiProcessorCount, dev));
    *n = cached[dev];
    return DG_OK;
  }
  DGL_CUDA(cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev));
  return DG_OK;
}

int encode_map(CUtensorMap* map, const void* base, int esz, int rank, const int64_t* dims, const int64_t* strides,
               int box_rows) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(DG_ERR_UNSUPPORTED, "driver entry point cuTensorMapEncodeTiled not found");
  cuuint64_t d[3], s[2];
  cuuint32_t box[3] = {(cuuint32_t)(128 / esz), (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) d[i] = (cuuint64_t)dims[i];
  for (int i = 0; i + 1 < rank; ++i) s[i] = (cuuint64_t)(strides[i] * esz);
  const CUresult r =
      fn(map, esz == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
             : esz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, (cuuint32_t)rank,
         const_cast<void*>(base), d, s, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(DG_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for %lld x %lld x %lld", (int)r, (long long)dims[0],
                (long long)dims[1], (long long)(rank > 2 ? dims[2] : 1));
  return DG_OK;
}

int encode_scale_map(CUtensorMap* map, const void* base, int64_t kblocks, int64_t row_tiles, int box_tiles) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(DG_ERR_UNSUPPORTED, "driver entry point cuTensorMapEncodeTiled not found");
  const cuuint64_t d[3] = {256, (cuuint64_t)kblocks, (cuuint64_t)row_tiles};
  const cuuint64_t s[2] = {1024, (cuuint64_t)kblocks * 1024};
  const cuuint32_t box[3] = {256, 1, (cuuint32_t)box_tiles}, one[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), d, s, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(DG_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d) for %lld x %lld scale tiles", (int)r, (long long)row_tiles,
                (long long)kblocks);
  return DG_OK;
}

}  // namespace dgl

extern "C" const char* dg_layer_last_error(void) { return dgl::g_err; }

extern "C" int dg_layer_check(void* status, void* stream) {
  if (!status) return dgl::fail(DG_ERR_ARG, "status is null");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  unsigned long long v = 0;
  DGL_CUDA(cudaMemcpyAsync(&v, status, sizeof(v), cudaMemcpyDeviceToHost, s));
  DGL_CUDA(cudaStreamSynchronize(s));
  if (v == 0) return DG_OK;  // (cleared only when read: a launch on another stream may report in between)
  DGL_CUDA(cudaMemsetAsync(status, 0, sizeof(v), s));
  DGL_CUDA(cudaStreamSynchronize(s));
  return dgl::fail(DG_ERR_HANG, "a pipeline wait ran out (wait 0x%llx)", v & 0xffffffffull);
}
