"""A device on which the kernels of the FP8 expert operators cannot be set up: those calls fail,
every other call works as it did before they were there.

The ABI layer (csrc/api.cu) is linked against a fake CUDA runtime and fake kernels, whose set-up
fails on request; nothing here reaches a GPU.
"""

import ctypes
import os
import subprocess

import pytest

from moe_decode_router_gb300 import build as B
from moe_decode_router_gb300 import flint_moe as F

KERNELS = r"""
#include "flint_internal.h"
using namespace flint;
static int fail_group, fail_gemm, launches;
extern "C" {
void fake_reset(int r, int g) { fail_group = r; fail_gemm = g; launches = 0; }
int fake_launches() { return launches; }
}
namespace flint {
static cudaError_t launched() { ++launches; return cudaSuccess; }
cudaError_t decode_kernels_init(int) { return cudaSuccess; }
cudaError_t fused_kernels_init(int) { return cudaSuccess; }
cudaError_t dense_kernels_init() { return cudaSuccess; }
cudaError_t medium_kernels_init() { return cudaSuccess; }
cudaError_t prefill_kernels_init(int) { return cudaSuccess; }
cudaError_t route_kernels_init(int* most) { *most = 16; return fail_group ? cudaErrorInvalidValue : cudaSuccess; }
cudaError_t block_gemm_kernels_init() { return fail_gemm ? cudaErrorInvalidConfiguration : cudaSuccess; }
DecodeWs carve_decode_ws(void*, int) { return {}; }
FusedWs carve_fused_ws(void*) { return {}; }
MediumWs carve_medium_ws(void*) { return {}; }
size_t prefill_ws_bytes(int) { return 256; }
size_t dense_packed_bytes(int N, int K) { return (size_t)N * K * 9 / 16; }
cudaError_t launch_pack(int, const void*, const uint8_t*, const void*, const uint8_t*, void*, cudaStream_t) { return launched(); }
cudaError_t launch_pack_dense(const uint8_t*, const uint8_t*, int, int, void*, cudaStream_t) { return launched(); }
cudaError_t launch_dense_gemv(const void*, int, int, float, const void*, int, void*, int, unsigned*, cudaStream_t) { return launched(); }
cudaError_t launch_prefill(const LayerArgs&, const void*, int, float, void*, int32_t*, float*, void*, int, unsigned*, cudaStream_t) { return launched(); }
cudaError_t launch_decode_chain(int, const LayerArgs&, const void*, const void*, int, float, void*, void*, void*, int32_t*, float*, const DecodeWs&, int, unsigned*, cudaStream_t, bool) { return launched(); }
cudaError_t launch_fused_stack(const LayerArgs*, int, const void*, int, float, void*, void*, int32_t*, float*, const FusedWs&, int, unsigned*, long long, cudaStream_t) { return launched(); }
cudaError_t launch_medium_chain(const LayerArgs&, const void*, const LayerArgs*, int, float, void*, int32_t*, float*, const MediumWs&, int, unsigned*, cudaStream_t, bool) { return launched(); }
cudaError_t launch_route(const RouteSpec&, const void*, bool, long long, int, const float*, int32_t*, float*, cudaStream_t) { return launched(); }
cudaError_t launch_group_pairs(const int32_t*, int, int, int32_t*, int32_t*, int32_t*, int, cudaStream_t) { return launched(); }
cudaError_t launch_quantize_rows(const void*, bool, long long, int, int, bool, const int32_t*, int, long long, void*, float*, cudaStream_t) { return launched(); }
cudaError_t launch_combine(const void*, bool, long long, const int32_t*, const float*, int, int, int, const void*, void*, cudaStream_t) { return launched(); }
cudaError_t launch_block_gemm(const void*, const float*, int, const void*, const float*, int, const int32_t*, int, int, void*, bool, int, unsigned*, cudaStream_t) { return launched(); }
}
"""
RUNTIME = r"""
#include <cuda_runtime_api.h>
static unsigned word;
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaSetDevice(int) { return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() { return cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void** p, const void*) { *p = &word; return cudaSuccess; }
cudaError_t cudaStreamCreateWithFlags(cudaStream_t* s, unsigned) { *s = nullptr; return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) { *s = cudaStreamCaptureStatusNone; return cudaSuccess; }
cudaError_t cudaStreamBeginCapture(cudaStream_t, cudaStreamCaptureMode) { return cudaErrorUnknown; }
cudaError_t cudaStreamEndCapture(cudaStream_t, cudaGraph_t*) { return cudaErrorUnknown; }
cudaError_t cudaGraphDestroy(cudaGraph_t) { return cudaSuccess; }
cudaError_t cudaGraphExecDestroy(cudaGraphExec_t) { return cudaSuccess; }
cudaError_t cudaGraphInstantiate(cudaGraphExec_t*, cudaGraph_t, unsigned long long) { return cudaErrorUnknown; }
cudaError_t cudaGraphLaunch(cudaGraphExec_t, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t cudaMemcpy(void*, const void*, size_t, cudaMemcpyKind) { return cudaSuccess; }
cudaError_t cudaMemcpyAsync(void*, const void*, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaMemset(void*, int, size_t) { return cudaSuccess; }
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
}
"""


@pytest.fixture(scope="module")
def faked(tmp_path_factory):
    """Loads a fresh copy of the ABI layer over the fakes: each copy has set up no device yet."""
    d = tmp_path_factory.mktemp("fake")
    kernels, runtime, api, lib = d / "kernels.cu", d / "runtime.cpp", d / "api.o", d / "libfake.so"
    kernels.write_text(KERNELS)
    runtime.write_text(RUNTIME)
    flags = [*B.ARCH, "-std=c++17", "-Xcompiler", "-fPIC", "-I", B.INCLUDE, "-I", B.CSRC]
    nvcc = B.nvcc_path()
    subprocess.run([nvcc, *flags, "-c", os.path.join(B.CSRC, "api.cu"), "-o", api], check=True)
    subprocess.run([nvcc, *flags, "-cudart", "none", "-shared", "-Xlinker", "-Bsymbolic", kernels, runtime, api, "-o", lib],
                   check=True)
    n = [0]

    def load(fail_group, fail_gemm):
        n[0] += 1
        copy = d / f"libfake{n[0]}.so"
        copy.write_bytes(lib.read_bytes())
        L = ctypes.CDLL(str(copy))
        for name, (res, args) in F._SIGS.items():
            getattr(L, name).restype, getattr(L, name).argtypes = res, args
        L.fake_reset(fail_group, fail_gemm)
        return L

    return load


def addr(i):
    return 0x7F0000000000 + (i << 36)  # checked by the host code, never read


def old_calls(L):
    dims = F.Dims(F.HIDDEN, F.N_EXPERTS, F.N_SHARED, F.INTER, F.TOP_K, F.W_NVFP4, 1e-6)
    layer = F.Layer(addr(0), addr(1), addr(2), addr(3))
    ws = 1 << 30
    return [
        L.flint_moe_decode_layer(dims, layer, addr(4), 2, addr(5), None, None, addr(6), ws, None),
        L.flint_moe_prefill_layer(dims, layer, addr(4), 100, addr(5), None, None, addr(6), ws, None),
        L.flint_moe_dense_gemv(addr(0), 256, 256, 1.0, addr(1), 1, addr(2), None),
    ]


def new_calls(L):
    r = F.Routing(64, 4, 0, 1, 1, 0, 1, 1.0)
    return [
        L.flint_moe_route(r, addr(0), 0, 64, 4, None, addr(1), addr(2), None),
        L.flint_moe_group_pairs(addr(0), 16, 64, addr(1), addr(2), addr(3), None),
        L.flint_moe_quantize_rows(addr(0), 0, 128, 4, 128, 0, None, 0, 4, addr(1), addr(2), None),
        L.flint_moe_block_gemm(addr(0), addr(1), 4, addr(2), addr(3), 1, None, 128, 128, addr(4), 0, None),
        L.flint_moe_combine(addr(0), 0, 4, addr(1), addr(2), 4, 1, 128, None, addr(3), None),
    ]


def test_all_set_up(faked):
    L = faked(0, 0)
    assert old_calls(L) == [0] * 3 and new_calls(L) == [0] * 5 and L.fake_launches() == 8


@pytest.mark.parametrize("fail_group,fail_gemm", [(1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("new_first", [False, True])
def test_expert_operators_not_set_up(faked, fail_group, fail_gemm, new_first):
    """The calls whose kernels are not there say so, whichever call came first."""
    L = faked(fail_group, fail_gemm)
    bad = F.FLINT_MOE_ERR_CUDA
    want = [0, bad if fail_group else 0, 0, bad if fail_gemm else 0, 0]
    if new_first:
        assert new_calls(L) == want
    assert old_calls(L) == [0] * 3
    assert new_calls(L) == want
    assert L.fake_launches() == 3 + (2 if new_first else 1) * want.count(0)
