"""The layer operators without a GPU, at the edges: calls whose derivatives
would be lost, sizes beside 2^31, the launches' tags, the status word."""

import os
import subprocess

import pytest
import torch
from torch.autograd import forward_ad

from reduce_scatter_gb300 import dg, layer, ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "reduce_scatter_gb300", "csrc")
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(dg.LIB_PATH) or not os.path.exists(layer.EXT_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return layer.lib()


def compiled(tmp_path, source):
    """Output of a host program over the library's sources."""
    cuda = "/usr/local/cuda/include"
    cpp, exe = tmp_path / "t.cpp", tmp_path / "t"
    cpp.write_text(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", f"-I{ROOT}/include", f"-I{CSRC}", f"-I{cuda}", "-o", str(exe), str(cpp)],
                   check=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.split()


def test_tangents_are_refused(L):
    x, w = torch.ones(4, 64, dtype=BF16), torch.ones(64, dtype=BF16)
    b, ends = torch.ones(2, 64, 32, dtype=BF16), torch.tensor([2, 4], dtype=torch.int32)
    d, scale, rstd = torch.ones(4, 32, dtype=BF16), torch.ones(1), torch.ones(4)
    calls = [(lambda x: ops.add_rms_norm(x, w), x), (lambda w: ops.add_rms_norm(x, w), w),
             (lambda r: ops.add_rms_norm(x, w, residual=r), x.clone()),
             (lambda s: ops.add_rms_norm(x, w, out_dtype=E4M3, scale=s), scale),
             (lambda dy: ops.add_rms_norm_backward(dy, x, w, rstd), x), (lambda h: ops.add_rms_norm_backward(x, h, w, rstd), x),
             (lambda w: ops.add_rms_norm_backward(x, x, w, rstd), w), (lambda r: ops.add_rms_norm_backward(x, x, w, r), rstd),
             (lambda d: ops.add_rms_norm_backward(x, x, w, rstd, d_residual=d), x),
             (lambda a: ops.grouped_matmul(a, b, ends), x), (lambda b: ops.grouped_matmul(x, b, ends), b),
             (lambda s: ops.grouped_matmul(x, b, ends, scale_a=s), scale), (lambda s: ops.grouped_matmul(x, b, ends, scale_b=s), scale),
             (lambda d: ops.grouped_matmul_backward(d, x, b, ends), d), (lambda a: ops.grouped_matmul_backward(d, a, b, ends), x),
             (lambda b: ops.grouped_matmul_backward(d, x, b, ends), b), (lambda x: ops.quantize_mx4(x), x)]
    for i, (call, t) in enumerate(calls):
        with forward_ad.dual_level():
            with pytest.raises(ValueError, match="forward-mode"):
                call(forward_ad.make_dual(t, torch.ones_like(t)))
            with pytest.raises(ValueError, match="CUDA"):   # (a tensor without a tangent: the next check)
                call(t)


def test_gradients_that_would_be_dropped_are_refused(L):
    x, w = torch.ones(4, 64, dtype=BF16), torch.ones(64, dtype=BF16)
    b, ends = torch.ones(2, 64, 32, dtype=BF16), torch.tensor([2, 4], dtype=torch.int32)
    a8, b8 = x.to(E4M3), b.to(E4M3)
    scale = torch.ones(1, requires_grad=True)
    calls = [lambda: ops.quantize_mx4(x.clone().requires_grad_()), lambda: ops.quantize_mx4(x.float().requires_grad_()),
             lambda: ops.add_rms_norm(x, w, out_dtype=E4M3, scale=scale),
             lambda: ops.grouped_matmul(a8, b8, ends, scale_a=scale), lambda: ops.grouped_matmul(a8, b8, ends, scale_b=scale),
             lambda: ops.grouped_matmul(x, b, ends, scale_a=scale), lambda: ops.grouped_matmul(x, b, ends, scale_b=scale)]
    for call in calls:
        with pytest.raises(ValueError, match="no gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call()


def test_a_scale_of_16_bit_rows_is_refused_with_and_without_gradients(L):
    x, w = torch.ones(4, 64, dtype=BF16), torch.ones(64, dtype=BF16)
    for t in (x, x.clone().requires_grad_()):
        for s in (1.0, torch.ones(1)):
            with pytest.raises(ValueError, match="needs a float8 out_dtype"):
                ops.add_rms_norm(t, w, scale=s)


def test_launch_tags_skip_zero(tmp_path):
    # a status word of 0 means that nothing gave up, so no launch is tagged 0
    out = compiled(tmp_path, """
        #include <cstdio>
        #include "layer_common.h"
        int main() {
          std::atomic<uint32_t> last{0xfffffffdu};
          for (int i = 0; i < 4; ++i) std::printf("%u\\n", dgl::next_tag(last));
        }""")
    assert [int(v) for v in out] == [2 ** 32 - 2, 2 ** 32 - 1, 1, 2]


def test_check_loses_no_report(tmp_path):
    # a launch on another stream that gives up just after the word was read must be found by the next check
    out = compiled(tmp_path, """
        #include <cstdio>
        #include <cstring>
        #include "layer_common.cu"
        static unsigned long long word;
        static int late;  // 1: a report lands after the next read of the word
        extern "C" {
        cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, cudaMemcpyKind, cudaStream_t) {
          std::memcpy(d, s, n);
          if (late) word = (7ull << 32) | 0x203, late = 0;
          return cudaSuccess;
        }
        cudaError_t cudaMemsetAsync(void* d, int v, size_t n, cudaStream_t) { std::memset(d, v, n); return cudaSuccess; }
        cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
        const char* cudaGetErrorString(cudaError_t) { return ""; }
        cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
        cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { *v = 152; return cudaSuccess; }
        cudaError_t cudaGetDriverEntryPointByVersion(const char*, void**, unsigned, unsigned long long, cudaDriverEntryPointQueryResult*) {
          return cudaErrorUnknown;
        }
        }
        int main() {
          std::printf("%d\\n", dg_layer_check(&word, nullptr));   // nothing
          late = 1;
          std::printf("%d\\n", dg_layer_check(&word, nullptr));   // nothing when read
          std::printf("%d\\n", dg_layer_check(&word, nullptr));   // the report
          std::printf("%d\\n", dg_layer_check(&word, nullptr));   // cleared
        }""")
    assert [int(v) for v in out] == [dg.OK, dg.OK, dg.ERR_HANG, dg.OK]


@pytest.mark.parametrize("big", [dict(t=2 ** 31 - 1), dict(t=2 ** 31 - 255), dict(n=2 ** 31 - 8), dict(k=2 ** 31 - 128)])
def test_sizes_whose_tiles_pass_32_bits_are_refused(L, big):
    v = dict(t=4, n=64, k=64) | big
    assert L.dg_layer_grouped_matmul(16, v["k"], 0, 16, v["k"], v["k"] * v["n"], 0, 0, 16, 1, None, 0, None, 0, 0, 16, 0, v["t"],
                                     v["n"], v["k"], 256, 16, None) == dg.ERR_ARG
    assert L.dg_layer_grouped_weight_grad(16, v["n"], 16, v["k"], 16, 1, 16, 0, v["t"], v["n"], v["k"], 256, 256, 16,
                                          None) == dg.ERR_ARG
