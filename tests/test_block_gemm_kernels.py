"""The block-scaled product, kernel by kernel: shapes that the library's choice sends to each of
them (asserted from the choice itself), with the group lengths, widths and types where each can
go wrong.  References and tolerances as in test_expert_ops.py.
"""

import os

import numpy as np
import pytest
import torch

import expert_ops_reference as R
from moe_decode_router_gb300 import build as _build
from moe_decode_router_gb300 import flint_moe as F
from test_expert_ops import check_product, dev, f64, gen, gpu, make_product

FEW_SPLIT, FEW, WIDE_IN_4, WIDE_IN_2, WIDE, TALL = range(6)
BOTH = pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])


def kernel_of(M, N, K, E=1, grouped=False, sms=None):
    if sms is None:
        sms = torch.cuda.get_device_properties(0).multi_processor_count
    return F.load_library().flint_block_gemm_kernel(M, N, K, E, int(grouped), sms)


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def run(kernel, out, counts, N, K, behind=0, ins=None):
    """The product of groups of `counts` rows (one number: dense), `behind` rows that belong to no
    group, and a row on either side of y that must stay; returns y."""
    d = dev()
    dense = isinstance(counts, int)
    E, M = (1, counts) if dense else (len(counts), sum(counts) + behind)
    assert kernel_of(M, N, K, E, not dense) == kernel
    a, sa, b, sb = ins if ins is not None else make_product(M, N, K, E, M + N + K, d)
    off = None if dense else offsets_of(counts)
    before = torch.randn(M + 2, N, generator=gen(1)).to(out).to(d)
    guard = before.clone()
    y = guard[1:-1]
    F.block_gemm(a, sa, b, sb, y, offsets=None if dense else torch.from_numpy(off).to(d))
    torch.cuda.synchronize()
    assert F.device_error() == 0
    assert torch.equal(guard[0], before[0]) and torch.equal(guard[-1], before[-1])
    if behind:
        assert torch.equal(y[M - behind:], before[1:-1][M - behind:])
    if ins is None:
        check_product(y, a, sa, b, sb, off, before[1:-1])
        again = before.clone()
        F.block_gemm(a, sa, b, sb, again[1:-1], offsets=None if dense else torch.from_numpy(off).to(d))
        torch.cuda.synchronize()
        assert torch.equal(guard, again)
    return y


def test_every_kernel_is_chosen():
    """On 152 SMs, by the cases below."""
    assert kernel_of(8, 520, 272, 1024, True, 152) == FEW_SPLIT
    assert kernel_of(16, 4096, 2048, sms=152) == FEW_SPLIT
    assert kernel_of(100, 264, 400, 1024, True, 152) == FEW
    assert kernel_of(32, 4096, 2048, sms=152) == WIDE_IN_4
    assert kernel_of(100, 4096, 4096, sms=152) == WIDE_IN_2
    assert kernel_of(256, 4096, 2048, sms=152) == WIDE
    assert kernel_of(8191, 4096, 4096, sms=152) == TALL
    assert kernel_of(49152, 1024, 2048, 256, True, 152) == TALL


def test_no_copy_goes_to_several_blocks():
    """Operands are copied into the memory of the block that asks for them and nowhere else, as any
    caller's weights may lie in another GPU's memory."""
    word = "multi" + "cast"
    for name in sorted(os.listdir(_build.CSRC)):
        with open(os.path.join(_build.CSRC, name)) as f:
            assert word not in f.read().lower(), name


# ------------------------------------------------------------------ long groups

LONG = [1, 127, 128, 129, 0, 255, 256, 257, 40, 0, 512]


@gpu
@BOTH
@pytest.mark.parametrize("M,N,K", [(2050, 1288, 656), (2311, 1032, 1040), (2200, 776, 272), (2304, 1024, 128),
                                   (2433, 1160, 16)])
def test_tall_dense(out, M, N, K):
    """Odd and even numbers of weight tiles, last tiles of 2, 7, 24, 0 and 129 rows, one K block and
    a K block that ends early."""
    run(TALL, out, M, N, K)


@gpu
@BOTH
@pytest.mark.parametrize("N,K", [(1032, 400), (1280, 1040), (1416, 656), (1288, 144)])
@pytest.mark.parametrize("behind", [0, 5])
@pytest.mark.parametrize("order", ["ascending", "reversed"])
def test_tall_grouped(out, N, K, behind, order):
    """Groups around the tiles' 128 and 256 rows, empty ones, and one that ends where a ends."""
    run(TALL, out, LONG if order == "ascending" else LONG[::-1], N, K, behind)


@gpu
@BOTH
@pytest.mark.parametrize("counts", [[700], [0, 0, 2000], [2000, 0], [90] * 20, [300, 1] * 8])
def test_tall_few_groups(out, counts):
    run(TALL, out, counts, 1800, 272)


@gpu
def test_tall_all_groups_empty():
    """No unit at all: y stays as it was."""
    d = dev()
    M, N = 2000, 1032
    assert kernel_of(M, N, 128, 3, True) == TALL
    a, sa, b, sb = make_product(M, N, 128, 3, 1, d)
    y = torch.full((M, N), 3.0, device=d)
    F.block_gemm(a, sa, b, sb, y, offsets=torch.zeros(4, dtype=torch.int32, device=d))
    torch.cuda.synchronize()
    assert F.device_error() == 0 and bool((y == 3.0).all())


# ------------------------------------------------------------------ 33 to 128 rows


@gpu
@BOTH
@pytest.mark.parametrize("counts,N,K", [
    ([17, 0, 9, 8, 1] + [0] * 59, 136, 272), ([0] * 63 + [40], 264, 1040), ([128] + [0] * 127, 128, 400),
    ([1] * 33, 520, 16), ([0, 25, 0, 16, 7, 24] + [0] * 66, 1000, 656)])
@pytest.mark.parametrize("behind", [0, 5])
def test_few_rows_of_many_experts(out, counts, N, K, behind):
    """Runs of more than eight rows of one expert; rows behind the last group stay."""
    if sum(counts) + behind > len(counts) or sum(counts) + behind > 128:
        behind = 0
    run(FEW, out, counts, N, K, behind)


# ------------------------------------------------------------------ 1,024 experts


@gpu
@BOTH
@pytest.mark.parametrize("kernel,M,N,K", [(FEW_SPLIT, 8, 520, 272), (FEW, 100, 264, 400), (WIDE_IN_4, 9, 128, 1040),
                                          (WIDE_IN_2, 20, 264, 1552), (WIDE, 300, 264, 272), (TALL, 40000, 136, 144)])
def test_most_experts(kernel, out, M, N, K):
    """As many experts as are allowed, most of them without rows or with a few."""
    counts = np.bincount(np.random.default_rng(M).integers(0, 1024, M), minlength=1024)
    run(kernel, out, [int(c) for c in counts], N, K)


# ------------------------------------------------------------------ exact sums and NaN, every kernel

KERNELS = [(FEW_SPLIT, [3, 0, 5], 264, 656), (FEW, [17, 0, 23] + [0] * 40, 264, 656), (WIDE_IN_4, [30, 0, 31], 264, 1040),
           (WIDE_IN_2, [70, 0, 61], 1160, 1552), (WIDE, [70, 0, 61], 264, 656), (TALL, [1000, 0, 100, 303], 1160, 656)]


@gpu
@pytest.mark.parametrize("kernel,counts,N,K", KERNELS)
def test_exact_integers(kernel, counts, N, K):
    """Small integers and power-of-two scales: every sum is exact, in any order."""
    d = dev()
    E, M, kb, nb = len(counts), sum(counts), -(-K // 128), -(-N // 128)
    g = gen(kernel)
    a = torch.randint(-2, 3, (M, K), generator=g).float().to(torch.float8_e4m3fn).to(d)
    b = torch.randint(-2, 3, (E, N, K), generator=g).float().to(torch.float8_e4m3fn).to(d)
    sa = torch.exp2(torch.randint(-1, 2, (kb, M), generator=g).float()).to(d)
    sb = torch.exp2(torch.randint(-1, 2, (E, nb, kb), generator=g).float()).to(d)
    y = run(kernel, torch.float32, counts, N, K, ins=(a, sa, b, sb))
    assert np.array_equal(f64(y), R.gemm(f64(a), f64(sa), f64(b), f64(sb), offsets_of(counts))[0])


@gpu
@BOTH
@pytest.mark.parametrize("kernel,counts,N,K", KERNELS)
def test_nan_stays_in_its_row(kernel, out, counts, N, K):
    """A NaN code or an infinite scale of a row, and a NaN code of one expert's weights, reach
    nothing else."""
    d = dev()
    E, M = len(counts), sum(counts)
    a, sa, b, sb = make_product(M, N, K, E, 3, d)
    lo, hi = offsets_of(counts)[2:4]  # the rows of expert 2
    a.view(torch.uint8)[1, K - 1] = 0x7F
    sa[0, 0] = float("inf")
    b.view(torch.uint8)[2, N - 3, 9] = 0x7F
    y = run(kernel, out, counts, N, K, ins=(a, sa, b, sb)).cpu()
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[0]).any()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[:2] = True
    bad[lo:hi, N - 3] = True
    assert torch.isnan(y[lo:hi, N - 3]).all()
    assert torch.isfinite(y[~bad]).all()
