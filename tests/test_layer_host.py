"""Layer operators on the host (no GPU): refusals and host-side paths beside test_layer."""
import ctypes
import os
import subprocess

import pytest

import mamba_ssd_chunked_02_gb300 as m2
from mamba_ssd_chunked_02_gb300 import build as m2build
from mamba_ssd_chunked_02_gb300 import layer as L

P = 1 << 20       # an aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    m2build.build()
    return m2.load()


def test_turn_selftest_refusals(lib):
    f = L._fn("scan_selftest")

    def status(shape, ptrs=(P,) * 8, space=1 << 40, limit=1000):
        return f(ctypes.addressof(shape), *ptrs, space, limit, None)

    turns = L.ScanShape(40, 400, 1000, 16, 1, m2.BF16, 0)     # 1280 rows of blocks
    assert status(turns, limit=0) == m2.ERR_INVALID_ARG and status(turns, limit=100001) == m2.ERR_INVALID_ARG
    assert status(L.ScanShape(2, 400, 1000, 16, 1, m2.BF16, 0)) == m2.ERR_UNSUPPORTED
    assert status(L.ScanShape(40, 400, 1000, 12, 1, m2.BF16, 0)) == m2.ERR_UNSUPPORTED
    for k in range(7):
        assert status(turns, [None if i == k else P for i in range(8)]) == m2.ERR_INVALID_ARG
    assert status(turns, space=4) == m2.ERR_WORKSPACE


STUBS = """
#include "internal.h"
#include "layer.cuh"
namespace m2 {
static cudaError_t g;
cudaError_t launch_conv_fwd(const ConvArgs&, const void*, const float*, const float*, const void*, const int32_t*, void*,
                            void*, cudaStream_t) { return g; }
cudaError_t launch_conv_step(const ConvArgs&, void*, const void*, const float*, const float*, void*, cudaStream_t) { return g; }
int64_t conv_bwd_slots(const ConvArgs&) { return 0; }
cudaError_t launch_conv_bwd(const ConvArgs&, const void*, const float*, const float*, const void*, const void*, const void*,
                            const int32_t*, void*, float*, float*, void*, float*, cudaStream_t) { return g; }
cudaError_t launch_norm_fwd(const NormArgs&, const void*, const float*, const void*, void*, cudaStream_t) { return g; }
int64_t norm_bwd_slots(const NormArgs&) { return 0; }
cudaError_t launch_norm_bwd(const NormArgs&, const void*, const float*, const void*, const void*, void*, void*, float*,
                            float*, cudaStream_t) { return g; }
size_t scan_fwd_workspace(const ScanArgs&) { return 0; }
bool scan_fwd_turns(const ScanArgs&) { return true; }
cudaError_t launch_scan_fwd(const ScanArgs&, const void*, const void*, const float*, const void*, const void*, const float*,
                            const void*, const float*, const float*, const int32_t*, void*, float*, void*, cudaStream_t,
                            uint64_t) { return g; }
cudaError_t launch_scan_step(const ScanArgs&, float*, const void*, const void*, const float*, const void*, const void*,
                             const float*, const void*, const float*, void*, cudaStream_t) { return g; }
size_t scan_bwd_workspace(const ScanArgs&) { return 0; }
cudaError_t launch_scan_bwd(const ScanArgs&, const void*, const void*, const float*, const void*, const void*, const float*,
                            const void*, const float*, const float*, const void*, const float*, const int32_t*,
                            const ScanGrads&, void*, cudaStream_t) { return g; }
}
extern "C" __attribute__((visibility("default"))) void set_error(int e) { m2::g = static_cast<cudaError_t>(e); }
"""


def test_a_cuda_error_is_not_an_unsupported_shape(tmp_path):
    """The checks over launchers that fail as CUDA does: an invalid value at a launch is an error
    of the call, not a shape the library refuses."""
    src, out = tmp_path / "stubs.cu", tmp_path / "api.so"
    src.write_text(STUBS)
    r = subprocess.run([m2build.nvcc(), *m2build.NVCC_FLAGS, "-shared", "-cudart", "static", "-o", str(out), str(src),
                        os.path.join(m2build.CSRC, "layer_api.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    api = ctypes.CDLL(str(out))
    sh = L.NormShape(2, 4, 8, 1, 1e-5, m2.BF16, 0)
    args = [ctypes.c_void_p(v) for v in (ctypes.addressof(sh), None, P, None, None, P, None)]
    for error in (0, 1, 2, 700, 801):       # 1: cudaErrorInvalidValue
        api.set_error(error)
        assert api.mamba2_norm_fwd(*args) == (m2.ERR_CUDA if error else m2.OK), error


def test_too_large_a_grid_is_unsupported(lib):
    """The launchers' own limits, which nothing was launched for."""
    for name, sh, ptrs, space in (("conv_fwd", L.ConvShape(1 << 24, 1 << 12, 4096, 4, m2.BF16, 0), 7, False),
                                  ("conv_bwd", L.ConvShape(1 << 24, 1 << 12, 4096, 4, m2.BF16, 0), 11, True),
                                  ("norm_fwd", L.NormShape(1 << 24, 1 << 12, 16, 1, 1e-5, m2.BF16, 0), 4, False),
                                  ("norm_bwd", L.NormShape(1 << 24, 1 << 12, 16, 1, 1e-5, m2.BF16, 0), 7, True),
                                  ("scan_fwd", L.ScanShape(1 << 24, 1 << 6, 8192, 16, 1, m2.BF16, 0), 12, True),
                                  ("scan_bwd", L.ScanShape(1 << 24, 1 << 12, 64, 16, 1, m2.BF16, 0), 21, True)):
        tail = [P, 1 << 62, None] if space else [None]
        assert L._fn(name)(ctypes.addressof(sh), None, *[P] * ptrs, *tail) == m2.ERR_UNSUPPORTED, name


def test_overlapping_output_rows_are_refused_at_any_stride(lib):
    """2^25 sequences of two tokens, rows of 8 elements one element apart: the extent of the
    sequences passes 64 bits."""
    far = 1 << 39
    st = L._strides2(16, 8, far, 1)
    sh = L.ConvShape(1 << 25, 2, 8, 4, m2.BF16, 0)
    assert L._fn("conv_fwd")(ctypes.addressof(sh), ctypes.addressof(st), *[P] * 7, None) == m2.ERR_INVALID_ARG
    st = L._strides2(16, 8, 1, far)       # the same with the two dimensions' parts exchanged
    sh = L.ConvShape(2, 1 << 25, 8, 4, m2.BF16, 0)
    assert L._fn("conv_fwd")(ctypes.addressof(sh), ctypes.addressof(st), *[P] * 7, None) == m2.ERR_INVALID_ARG


def test_workspace_sizes_are_public(lib):
    conv, norm = m2.ConvShape(2, 64, 8, 4, m2.BF16, 0), m2.NormShape(2, 64, 8, 1, 1e-5, m2.BF16, 0)
    scan = m2.ScanShape(2, 64, 8, 16, 1, m2.BF16, 0)
    assert m2.conv_bwd_workspace_size(conv) >= 2 * 8 * 5 * 4      # a slot a sequence at least
    assert m2.scan_bwd_workspace_size(scan) > 2 * 8 * 8 * 16 * 4  # a state every 8 tokens
    assert m2.norm_bwd_workspace_size(m2.NormShape(0, 64, 8, 1, 1e-5, m2.BF16, 0)) == 0
    assert m2.norm_bwd_workspace_size(norm) % (8 * 4) == 0
