"""Long sums of the linear products and their gradients: how far an fp32 output may be off does
not grow with the length as a sum in the tensor cores alone would.

Tolerances.  An MMA adds 16 products to its accumulator and cuts the sum: by 2^-22 of the running
magnitude (the sum's last bit, and as much for the terms that it was lined up with).  An
accumulator begins anew after at most 512 products (1,024 in some shapes of the few-row kernel): 32
MMAs, or 64 whose running sum is half of theirs on average.  What it held is added to an fp32 sum
with a rounding of 2^-24, or to those of other warps.  No kernel adds fewer than 128 products at a time.
  terms of one sign   the running sum never passes the result: 32 2^-22 and (n / 128 + 8) 2^-24 of it.
                      One accumulator over n products loses n / 16 cuts of a sum that is half the result
                      on average: 2^-13 of 2^14 products, 2^-10 of 2^17.
  normal terms        a cut is taken for 2^-24 of the running sum, towards zero: 32 of them 2^-19.6
                      of the 2-norm; the roundings, of either sign, 2^-25 sqrt(n / 128) / 2.  Together
                      below 2^-19 for up to 2^17 products.
"""

import pytest
import torch

import linear_reference as R
from moe_decode_router_gb300 import flint_moe as F
from test_linear_ops import BF16, dev, done, groups, half_step, near, rand

gpu = pytest.mark.gpu


def positive(seed, *shape):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    return torch.rand(shape, generator=g, device=dev()).to(torch.bfloat16)


def one_sign(n):
    return 32 * 2.0 ** -22 + (n / 128 + 8) * 2.0 ** -24


def off_by(got, want):
    """(largest error relative to the value, error of the 2-norm)"""
    e = (got.double() - want).abs()
    return float((e / want.abs()).max()), float(e.norm() / want.norm())


# rows of each expert (one: dense), N: the few-row kernel's shapes and the pairs
LONG = [([1], 32), ([8], 48), ([3, 0, 5], 32), ([9, 30, 1] + [3] * 9, 32), ([6] * 24, 48), ([300], 64), ([200, 300], 32)]


@gpu
@pytest.mark.parametrize("K", [4096, 16384, 131072])
@pytest.mark.parametrize("counts,N", LONG)
def test_linear_in_fp32(counts, N, K):
    M, E, offsets = sum(counts), len(counts), groups(counts)
    y = torch.empty(M, N, device=dev())
    x, w = positive(1, M, K), positive(2, E, N, K)
    F.linear(x, w, y, offsets=offsets)
    done()
    assert off_by(y, R.product(x, w, offsets)[0])[0] <= one_sign(K)
    x, w = rand(1, M, K), rand(2, E, N, K)
    F.linear(x, w, y, offsets=offsets)
    done()
    assert off_by(y, R.product(x, w, offsets)[0])[1] <= 2.0 ** -19


@gpu
@pytest.mark.parametrize("counts", [[131072], [16384, 0, 100000, 5]])
def test_weight_gradient_in_fp32(counts):
    M, E, N, K, offsets = sum(counts), len(counts), 64, 48, groups(counts)
    w, dw = rand(1, E, N, K), torch.empty(E, N, K, device=dev())
    dy, x = positive(2, M, N), positive(3, M, K)
    F.linear_backward(dy, x, w, dw=dw, offsets=offsets)
    done()
    live = [e for e, c in enumerate(counts) if c]
    assert off_by(dw[live], R.weight_gradient(dy, x, E, offsets)[0][live])[0] <= one_sign(max(counts))
    dy, x = rand(2, M, N), rand(3, M, K)
    F.linear_backward(dy, x, w, dw=dw, offsets=offsets)
    done()
    assert off_by(dw[live], R.weight_gradient(dy, x, E, offsets)[0][live])[1] <= 2.0 ** -19


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("M", [(1 << 17) + 3, (1 << 22) + 5])
def test_weight_gradient_of_many_rows(M, grouped, out):
    """Terms of one sign: one accumulator over 2^22 of them would be off by 2 %, several times the
    rounding to bf16."""
    N, K, d = 64, 48, dev()
    offsets = torch.tensor([0, 0, M], dtype=torch.int32, device=d) if grouped else None
    dy, x, w = positive(2, M, N), positive(3, M, K), rand(1, 2 if grouped else 1, N, K)
    dw, dx = torch.empty(w.shape, dtype=out, device=d), torch.empty_like(x)
    F.linear_backward(dy, x, w, dx=dx, dw=dw, offsets=offsets)
    done()
    want = sum(a.double().T @ b.double() for a, b in zip(dy.split(1 << 18), x.split(1 << 18)))
    # half a step of the type beside the sum's own error; the fp32 sum has M / 512 parts
    tol = (BF16 if out == torch.bfloat16 else 0.0) + 1.01 * (32 * 2.0 ** -22 + (M / 512 + 8) * 2.0 ** -24)
    assert off_by(dw[-1], want)[0] <= tol
    assert not grouped or not bool(dw[0].any())
    ref, mag = R.input_gradient(dy[-100:], w[-1:])
    near(dx[-100:], ref, (N + 2) * 2.0 ** -23 * mag + half_step(dx, ref))


@gpu
@pytest.mark.parametrize("K", [880, 896, 1040, 1792])
@pytest.mark.parametrize("counts", [[3], [300], [150, 0, 151], [2] * 30])
def test_integer_sums_keep_their_last_bit(counts, K):
    """Sums of large odd products, up to 2^23.7 in 896 of K, which fp32 holds to the last bit."""
    M, E, N, offsets, d = sum(counts), len(counts), 64, groups(counts), dev()
    g = torch.Generator(device=d)
    g.manual_seed(K)
    a = torch.randint(100, 128, (M, K), dtype=torch.int8, generator=g, device=d)
    b = torch.randint(100, 128, (E, N, K), dtype=torch.int8, generator=g, device=d)
    a[1::3] *= -1
    b[:, ::2, K // 2:] *= torch.randint(0, 2, (E, N // 2, K - K // 2), dtype=torch.int8, generator=g, device=d)
    y, ones = torch.empty(M, N, device=d), torch.ones(max(M, E * N), device=d)
    F.integer_gemm(a, ones[:M].contiguous(), b, ones[:E * N].reshape(E, N).contiguous(), y, offsets=offsets)
    done()
    want = R.integer_sums(a, b, offsets)
    assert K > 896 or float(want.abs().max()) < 2 ** 24
    assert torch.equal(y, want.float())
