"""A device on which the tensor-core kernels of the linear, gated and integer products cannot be
set up: the products say so, quantising rows works, and no call is made on the way.

csrc/linear_api.cu is linked against fakes of the library's set-up, of the kernels and of the
runtime; nothing here reaches a GPU.
"""

import ctypes
import os
import subprocess

import pytest

from moe_decode_router_gb300 import build as B
from moe_decode_router_gb300 import flint_moe as F

FAKES = r"""
#include "flint_internal.h"
using namespace flint;
static int library_fails, kernels_fail, launches, inits, few;
extern "C" {
void fake_reset(int a, int b, int c) { library_fails = a; kernels_fail = b; few = c; launches = inits = 0; }
int fake_launches() { return launches; }
int fake_inits() { return inits; }
}
namespace flint {
static cudaError_t launched(int n) { launches += n; return cudaSuccess; }
int device_info(int* sms, unsigned** err) { *sms = 152; *err = nullptr; return library_fails ? -4 : 0; }
cudaError_t pair_gemm_kernels_init(int* ks) { ++inits; *ks = 4; return kernels_fail ? cudaErrorInvalidConfiguration : cudaSuccess; }
bool few_rows_take(const ProductArgs&, bool, const PairDevice&) { return few != 0; }
cudaError_t launch_few_rows(const ProductArgs&, bool, cudaStream_t) { return launched(1); }
cudaError_t launch_pair_forward(const ProductArgs&, bool, const PairDevice&, cudaStream_t) { return launched(100); }
cudaError_t launch_pair_backward(const GradArgs&, const PairDevice&, cudaStream_t) { return launched(100); }
cudaError_t launch_gate_backward(const void*, const void*, const int32_t*, int, int, int, int, void*, cudaStream_t) { return launched(1); }
cudaError_t launch_integer_rows(const void*, bool, long long, int, int, const int32_t*, int, int, void*, float*, cudaStream_t) { return launched(1); }
}
"""

RUNTIME = r"""
#include <cuda_runtime_api.h>
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
}
"""


@pytest.fixture(scope="module")
def faked(tmp_path_factory):
    """Loads a fresh copy of the entry points over the fakes: each copy has set up no device yet."""
    d = tmp_path_factory.mktemp("fake")
    fakes, runtime, lib = d / "fakes.cu", d / "runtime.cpp", d / "libfake.so"
    fakes.write_text(FAKES)
    runtime.write_text(RUNTIME)
    subprocess.run([B.nvcc_path(), *B.ARCH, "-std=c++17", "-Xcompiler", "-fPIC", "-I", B.INCLUDE, "-I", B.CSRC, "-cudart", "none",
                    "-shared", "-Xlinker", "-Bsymbolic", fakes, runtime, os.path.join(B.CSRC, "linear_api.cu"), "-o", lib], check=True)
    n = [0]

    def load(library_fails=0, kernels_fail=0, few=0):
        n[0] += 1
        copy = d / f"libfake{n[0]}.so"
        copy.write_bytes(lib.read_bytes())
        L = ctypes.CDLL(str(copy))
        for name, (res, args) in F._LINEAR_SIGS.items():
            getattr(L, name).restype, getattr(L, name).argtypes = res, args
        L.fake_reset(library_fails, kernels_fail, few)
        return L

    return load


def addr(i):
    return 0x7F0000000000 + (i << 36)  # checked by the host code, never read


def products(L):
    return [
        L.flint_moe_linear(addr(0), 64, addr(1), 1, None, 128, 128, addr(2), 0, None),
        L.flint_moe_gated_linear(addr(0), 64, addr(1), 1, None, 128, 128, 1, addr(2), addr(3), None),
        L.flint_moe_integer_gemm(addr(0), addr(1), 64, addr(2), addr(3), 1, None, 128, 128, 0, addr(4), 0, None),
        L.flint_moe_linear_backward(addr(0), addr(1), 64, addr(2), 1, None, 128, 128, addr(3), addr(4), 0, None),
        L.flint_moe_gated_linear_backward(addr(0), addr(1), addr(2), 64, addr(3), 1, None, 128, 128, 1, addr(4), None, None, 0, None),
    ]


def rows(L):
    return L.flint_moe_integer_quantize_rows(addr(0), 0, 128, 4, 128, None, 0, 4, addr(1), addr(2), None)


@pytest.mark.parametrize("few,launches", [(0, 100 * 3 + 100 + 1 + 1), (1, 3 + 100 + 1 + 1)])
def test_all_set_up_once(faked, few, launches):
    L = faked(few=few)
    assert products(L) == [0] * 5 and rows(L) == 0
    assert L.fake_launches() == launches and L.fake_inits() == 1  # the gated gradient without dx and dw: one pass


@pytest.mark.parametrize("rows_first", [False, True])
def test_kernels_not_set_up(faked, rows_first):
    L = faked(kernels_fail=1)
    if rows_first:
        assert rows(L) == 0
    assert products(L) == [F.FLINT_MOE_ERR_CUDA] * 5
    assert rows(L) == 0
    assert products(L) == [F.FLINT_MOE_ERR_CUDA] * 5
    assert L.fake_launches() == (2 if rows_first else 1) and L.fake_inits() == 1


def test_library_not_set_up(faked):
    L = faked(library_fails=1)
    assert products(L) == [F.FLINT_MOE_ERR_CUDA] * 5 and rows(L) == F.FLINT_MOE_ERR_CUDA
    assert L.fake_launches() == 0 and L.fake_inits() == 0
