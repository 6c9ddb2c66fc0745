"""A set-up of the tensor-core kernels that fails: one that may pass is tried again by the next
call, one that cannot is not, and the products of few rows need none of it.  What the library's
set-up throws is a status of every call.

csrc/linear_api.cu is linked against fakes of the library's set-up, of the kernels and of the
runtime; nothing here reaches a GPU.
"""

import ctypes
import os
import subprocess
import sys

import pytest

from moe_decode_router_gb300 import build as B
from moe_decode_router_gb300 import flint_moe as F
from test_linear_setup import RUNTIME, products, rows

FAKES = r"""
#include "flint_internal.h"
using namespace flint;
#include <new>
static int error, failures, few, inits, launches;
extern "C" {
void fake_set(int e, int n, int f) { error = e; failures = n; few = f; }
int fake_inits() { return inits; }
int fake_launches() { return launches; }
}
namespace flint {
static cudaError_t launched(int n) { launches += n; return cudaSuccess; }
int device_info(int* sms, unsigned** err) {
  if (error < 0) throw std::bad_alloc();
  *sms = 152;
  *err = nullptr;
  return 0;
}
cudaError_t pair_gemm_kernels_init(int* ks) {
  ++inits;
  *ks = 4;  // whatever is left behind by a set-up that fails
  return failures-- > 0 ? (cudaError_t)error : cudaSuccess;
}
bool few_rows_take(const ProductArgs&, bool, const PairDevice&) { return few != 0; }
cudaError_t launch_few_rows(const ProductArgs&, bool, cudaStream_t) { return launched(1); }
cudaError_t launch_pair_forward(const ProductArgs&, bool, const PairDevice&, cudaStream_t) { return launched(100); }
cudaError_t launch_pair_backward(const GradArgs&, const PairDevice&, cudaStream_t) { return launched(100); }
cudaError_t launch_gate_backward(const void*, const void*, const int32_t*, int, int, int, int, void*, cudaStream_t) { return launched(1); }
cudaError_t launch_integer_rows(const void*, bool, long long, int, int, const int32_t*, int, int, void*, float*, cudaStream_t) { return launched(1); }
}
"""

OUT_OF_MEMORY, LAUNCH_OUT_OF_RESOURCES = 2, 701
INVALID_VALUE, INVALID_CONFIGURATION, NO_KERNEL_IMAGE, NOT_SUPPORTED = 1, 9, 209, 801
BAD = F.FLINT_MOE_ERR_CUDA


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

    def load(error, failures, few=0):
        n[0] += 1
        copy = d / f"libfake{n[0]}.so"
        copy.write_bytes(lib.read_bytes())
        L = ctypes.CDLL(str(copy))
        for name, (res, args) in F._LINEAR_SIGS.items():
            getattr(L, name).restype, getattr(L, name).argtypes = res, args
        L.fake_set(error, failures, few)
        return L

    return load


@pytest.mark.parametrize("error", [OUT_OF_MEMORY, LAUNCH_OUT_OF_RESOURCES])
def test_a_failure_that_passes(faked, error):
    L = faked(error, 2)
    assert products(L) == [BAD, BAD, 0, 0, 0] and L.fake_inits() == 3
    assert products(L) == [0] * 5 and L.fake_inits() == 3 and rows(L) == 0


@pytest.mark.parametrize("error", [INVALID_VALUE, INVALID_CONFIGURATION, NO_KERNEL_IMAGE, NOT_SUPPORTED])
def test_a_failure_that_lasts(faked, error):
    L = faked(error, 1)
    assert products(L) == [BAD] * 5 and products(L) == [BAD] * 5
    assert L.fake_inits() == 1 and L.fake_launches() == 0


@pytest.mark.parametrize("error", [OUT_OF_MEMORY, NOT_SUPPORTED])
def test_few_rows_go_ahead(faked, error):
    L = faked(error, 1 << 20, few=1)
    assert products(L) == [0, 0, 0, BAD, BAD] and L.fake_launches() == 3
    L.fake_set(error, 1 << 20, 0)
    assert products(L) == [BAD] * 5 and L.fake_launches() == 3


THROWS = """
import sys
sys.path[:0] = [%r, %r]
import ctypes
from moe_decode_router_gb300 import flint_moe as F
from test_linear_setup import products, rows
L = ctypes.CDLL(%r)
for name, (res, args) in F._LINEAR_SIGS.items():
    getattr(L, name).restype, getattr(L, name).argtypes = res, args
L.fake_set(-1, 0, 0)
assert products(L) == [F.FLINT_MOE_ERR_CUDA] * 5 and rows(L) == F.FLINT_MOE_ERR_CUDA
L.fake_set(0, 0, 0)
assert products(L) == [0] * 5 and rows(L) == 0
"""


def test_no_exception_leaves_a_call(faked):
    """In a process of its own: an exception at a C entry would end it."""
    here = os.path.dirname(os.path.abspath(__file__))
    L = faked(0, 0)
    r = subprocess.run([sys.executable, "-c", THROWS % (os.path.dirname(here), here, L._name)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
