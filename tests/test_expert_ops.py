"""Routing, grouping, quantisation, block-scaled product and combine of FP8 expert
layers against 64-bit references, through the Python binding and the C ABI.

Tolerances, derived from the number formats:
  routing weights   expf within 2 units (2^-22), the rounding of its argument (up to
                    |x| 2^-24 for |x| < 40), sums and quotients of at most 16 + 1024 / 32
                    roundings: below 2^-17 relative.
  quantisation      scale: one rounding of the block's largest magnitude, 2^-23; a code
                    is the rounding of a quotient that is off by at most 2^-22 of itself,
                    so it lies within half an E4M3 step plus 2^-22 of the exact quotient.
                    With the gated activation the row itself is off by (8 + |gate|) 2^-22.
  product           a block's 128 exact products are added by the tensor cores with at
                    most 2^-23 of the running magnitude lost an addition, then scaled and
                    added with two roundings: at most (128 + 2 + K / 128) 2^-23 of the sum of magnitudes.
  combine           at most k + 1 fp32 roundings of the sum of magnitudes.
  bf16 outputs      half a step more, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import expert_ops_reference as R
from moe_decode_router_gb300 import flint_moe as F

gpu = pytest.mark.gpu
BF16 = 2.0 ** -8


def dev():
    F.load_library()
    return torch.device("cuda:0")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ routing


def run_route(logits, top_k, **kw):
    T = logits.shape[0]
    ids = torch.full((T, top_k), -7, dtype=torch.int32, device=logits.device)
    w = torch.full((T, top_k), float("nan"), device=logits.device)
    F.route(logits, ids, w, **kw)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), f64(w)


f64 = R.f64


def check_route(logits, top_k, bias=None, softmax=False, n_groups=1, top_groups=1, top2=False, renorm=True, scale=1.0):
    ids, w = run_route(logits, top_k, bias=bias, score=F.SCORE_SOFTMAX if softmax else F.SCORE_SIGMOID,
                       n_groups=n_groups, top_groups=top_groups, group_score=F.GROUP_TOP2 if top2 else F.GROUP_MAX,
                       renormalise=renorm, scale=scale)
    rid, rw = R.route(f64(logits), top_k, None if bias is None else f64(bias), softmax, n_groups, top_groups, top2,
                      renorm, scale)
    assert np.array_equal(ids, rid)
    assert np.all(np.abs(w - rw) <= 2.0 ** -17 * np.abs(rw) + 1e-37)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 6), (8, 256, 6), (5, 33, 3), (301, 64, 16), (67, 1000, 8),
                                   (2, 1024, 16), (130, 160, 6), (9, 8, 8)])
def test_route(dtype, softmax, T, E, k):
    d = dev()
    x = torch.randn(T, E, generator=gen(T + E)).to(dtype).to(d)
    check_route(x, k, softmax=softmax, renorm=(T % 2 == 0), scale=2.5)
    check_route(x, k, softmax=softmax, bias=(0.05 * torch.randn(E, generator=gen(1))).to(d))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("E,G,top,k", [(256, 8, 4, 8), (64, 32, 3, 6), (96, 4, 1, 5), (160, 8, 3, 6), (1024, 16, 2, 16),
                                       (32, 32, 8, 8)])
def test_route_groups(dtype, bias, top2, E, G, top, k):
    d = dev()
    x = torch.randn(200, E, generator=gen(E + G)).to(dtype).to(d)
    b = (0.1 * torch.randn(E, generator=gen(2))).to(d) if bias else None
    for softmax in (False, True):
        check_route(x, k, bias=b, softmax=softmax, n_groups=G, top_groups=top, top2=top2)


@gpu
def test_route_close_scores():
    """Scores a few fp32 units apart, equal ones, and saturated ones: decided as real numbers."""
    d = dev()
    E = 64
    x = torch.zeros(6, E)
    x[0] = 1.0 + torch.arange(E).flip(0) * 2.0 ** -23           # neighbours in fp32
    x[1] = 1.0                                                  # all equal: lowest indices
    x[2] = 12.0 + torch.arange(E) * 2.0 ** -20                  # sigmoid near 1
    x[3] = -80.0 - torch.arange(E) * 0.25                       # tiny scores
    x[4] = torch.where(torch.arange(E) % 2 == 0, 0.0, -0.0)     # two zeros, one value
    x[5] = 1.0 + (torch.arange(E) % 7) * 2.0 ** -22
    x = x.to(d)
    for bias in (None, torch.zeros(E), (torch.arange(E) % 3) * 2.0 ** -24):
        b = None if bias is None else bias.to(d)
        for softmax in (False, True):
            check_route(x, 8, bias=b, softmax=softmax)
            check_route(x, 8, bias=b, softmax=softmax, n_groups=8, top_groups=3, top2=True)
            check_route(x, 8, bias=b, softmax=softmax, n_groups=8, top_groups=3)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_route_masked(dtype):
    """-inf and NaN are never chosen; a row without candidates gives -1 and 0; the type's
    lowest value is a logit like any other; +inf scores 1."""
    d = dev()
    E = 40
    x = torch.randn(7, E, generator=gen(3))
    x[0] = -float("inf")
    x[1] = float("nan")
    x[2, 3:] = -float("inf")
    x[3, ::2] = float("nan")
    x[4] = torch.finfo(dtype).min
    x[5, 7] = float("inf")
    x[5, 9] = float("inf")
    x[6, 5:] = torch.finfo(dtype).min
    x = x.to(dtype).to(d)
    for softmax in (False, True):
        for kw in (dict(), dict(n_groups=4, top_groups=2), dict(n_groups=4, top_groups=2, top2=True)):
            check_route(x, 6, softmax=softmax, **kw)
    ids, w = run_route(x, 6)
    assert np.all(ids[:2] == -1) and np.all(w[:2] == 0)
    assert list(ids[2]) [3:] == [-1, -1, -1] and np.all(w[2, 3:] == 0)


@gpu
@pytest.mark.parametrize("softmax", [False, True])
def test_route_masked_with_bias(softmax):
    """The same with keys that a bias decides: infinite and NaN biases, and logits so low or
    high that the score is 0 or 1."""
    d = dev()
    E = 48
    x = torch.randn(9, E, generator=gen(11))
    x[0] = -float("inf")
    x[1, ::3] = -float("inf")
    x[2, 5:] = float("nan")
    x[3] = torch.finfo(torch.float32).min
    x[4, 7], x[4, 9] = float("inf"), float("inf")
    x[5] = -200.0
    x[6] = 60.0
    x[7] = 0.5
    b = 0.1 * torch.randn(E, generator=gen(12))
    for case in range(3):
        if case == 1:
            b[3], b[4] = -float("inf"), float("nan")
        if case == 2:
            b[20], b[33] = float("inf"), float("inf")
        for kw in (dict(), dict(n_groups=6, top_groups=2), dict(n_groups=6, top_groups=2, top2=True)):
            check_route(x.to(d), 6, bias=b.to(d), softmax=softmax, **kw)


@gpu
def test_route_strided_rows():
    d = dev()
    big = torch.randn(50, 300, generator=gen(4)).to(d)
    check_route(big[:, 8:8 + 203], 5)
    check_route(big[:, :259].to(torch.bfloat16), 5)
    check_route(big.to(torch.bfloat16)[::3, :259], 5)


# ------------------------------------------------------------------ grouping


@gpu
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 6, 256), (64, 6, 256), (1000, 3, 7), (5003, 8, 1024), (8192, 6, 256),
                                   (70001, 2, 300), (33, 1, 2)])
def test_group_pairs(T, k, E):
    d = dev()
    ids = torch.randint(-2, E + 2, (T, k), generator=gen(T), dtype=torch.int32).to(d)
    if T == 1000:
        ids[:] = 3  # one expert takes all
    offsets = torch.full((E + 1,), -9, dtype=torch.int32, device=d)
    order = torch.full((T * k,), -9, dtype=torch.int32, device=d)
    pos = torch.full((T, k), -9, dtype=torch.int32, device=d)
    F.group_pairs(ids, offsets, order, pos)
    torch.cuda.synchronize()
    ro, rr, rp = R.group(ids.cpu().numpy(), E)
    assert np.array_equal(offsets.cpu().numpy(), ro)
    assert np.array_equal(order.cpu().numpy(), rr)
    assert np.array_equal(pos.cpu().numpy().reshape(-1), rp)


@gpu
def test_group_pairs_none_left():
    d = dev()
    ids = torch.full((37, 2), -1, dtype=torch.int32, device=d)
    offsets, order = torch.empty(5, dtype=torch.int32, device=d), torch.empty(74, dtype=torch.int32, device=d)
    pos = torch.empty(37, 2, dtype=torch.int32, device=d)
    F.group_pairs(ids, offsets, order, pos)
    torch.cuda.synchronize()
    assert not offsets.any() and (order == -1).all() and (pos == -1).all()


# ------------------------------------------------------------------ quantisation


def silu_mul(x):
    g, u = np.split(x, 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def check_codes(q, scales, x, slack):
    """q, scales of the rows x [rows][K]; slack: relative error of the rows' values, [rows][K]."""
    _, rs, v = R.quantise_values(x)
    kb = rs.shape[0]
    worst = np.stack([slack[:, b * 128:(b + 1) * 128].max(1) for b in range(kb)])
    assert np.all(np.abs(scales - rs) <= (2.0 ** -23 + worst) * rs)
    rel = 2.0 ** -22 + slack + np.repeat(worst.T, 128, axis=1)[:, :x.shape[1]]
    assert np.all(np.abs(q - v) <= R.e4m3_step(v) / 2 + rel * np.abs(v))


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("rows,K,pad", [(1, 16, 0), (3, 128, 8), (7, 144, 0), (129, 2048, 0), (1000, 512, 16),
                                        (2, 8208, 0)])
def test_quantize_rows(dtype, silu, rows, K, pad):
    d = dev()
    cols = 2 * K if silu else K
    x = (3 * torch.randn(rows, cols + pad, generator=gen(rows + K))).to(dtype).to(d)[:, :cols]
    q = torch.empty(rows, K, dtype=torch.float8_e4m3fn, device=d)
    s = torch.empty(-(-K // 128), rows, device=d)
    F.quantize_rows(x, q, s, silu_mul=silu)
    torch.cuda.synchronize()
    v = f64(x)
    slack = np.zeros((rows, K))
    if silu:
        slack = (8 + np.abs(v[:, :K])) * 2.0 ** -22
        v = silu_mul(v)
    check_codes(f64(q), f64(s), v, slack)


@gpu
def test_quantize_rows_to_places():
    """Every row goes to all of its places; places of no row keep their bytes; places out of
    range are skipped."""
    d = dev()
    rows, K, k, places = 50, 272, 3, 200
    x = torch.randn(rows, K, generator=gen(9)).to(torch.bfloat16).to(d)
    perm = torch.randperm(places, generator=gen(10))[:rows * k].to(torch.int32).reshape(rows, k)
    perm[3, 1], perm[4] = -1, -1
    perm[5, 2] = places
    q = torch.full((places, K), 0x55, dtype=torch.uint8, device=d)
    s = torch.full((3, places), -5.0, device=d)
    F.quantize_rows(x, q.view(torch.float8_e4m3fn), s, pos=perm.to(d))
    plain_q = torch.empty(rows, K, dtype=torch.float8_e4m3fn, device=d)
    plain_s = torch.empty(3, rows, device=d)
    F.quantize_rows(x, plain_q, plain_s)
    torch.cuda.synchronize()
    want_q, want_s = torch.full((places, K), 0x55, dtype=torch.uint8), torch.full((3, places), -5.0)
    for t in range(rows):
        for j in range(k):
            if 0 <= perm[t, j] < places:
                want_q[perm[t, j]] = plain_q[t].view(torch.uint8).cpu()
                want_s[:, perm[t, j]] = plain_s[:, t].cpu()
    assert torch.equal(q.cpu(), want_q) and torch.equal(s.cpu(), want_s)


@gpu
def test_quantize_rows_edge_values():
    d = dev()
    x = torch.zeros(6, 256)
    x[1, :128] = 1e-38
    x[2] = 3e38
    x[3, 5] = float("nan")
    x[4, 200] = -float("inf")
    x[5] = torch.linspace(-1, 1, 256)
    q = torch.empty(6, 256, dtype=torch.float8_e4m3fn, device=d)
    s = torch.empty(2, 6, device=d)
    F.quantize_rows(x.to(d), q, s)
    torch.cuda.synchronize()
    v, sc = f64(q), f64(s)
    assert np.all(v[0] == 0) and np.all(sc[:, 0] == np.float32(R.FLOOR) / np.float32(448))
    assert np.all(v[1] == 0)
    assert np.all(v[2] == 448) and np.allclose(sc[:, 2] * 448, 3e38, rtol=1e-6)
    assert not np.isfinite(sc[0, 3]) and np.isfinite(sc[1, 3]) and np.all(v[3, 128:] == 0)
    assert np.isfinite(sc[0, 4]) and not np.isfinite(sc[1, 4])
    check_codes(v[5:], sc[:, 5:], f64(x[5:]), np.zeros((1, 256)))


# ------------------------------------------------------------------ product


def make_product(M, N, K, E, seed, d):
    g = gen(seed)
    a = (100 * torch.randn(M, K, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn).to(d)
    b = (100 * torch.randn(E, N, K, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn).to(d)
    sa = (0.01 * torch.exp(torch.randn(-(-K // 128), M, generator=g))).to(d)
    sb = (0.01 * torch.exp(torch.randn(E, -(-N // 128), -(-K // 128), generator=g))).to(d)
    return a, sa, b, sb


def check_product(y, a, sa, b, sb, offsets=None, before=None):
    ry, mag = R.gemm(f64(a), f64(sa), f64(b), f64(sb), offsets)
    got = f64(y)
    live = ~np.isnan(ry)
    K = a.shape[1]
    tol = (130 + K / 128) * 2.0 ** -23 * mag + (BF16 * np.abs(ry) if y.dtype == torch.bfloat16 else 0)
    assert np.all(np.abs(got - ry)[live] <= tol[live])
    if before is not None:
        assert np.array_equal(got[~live], f64(before)[~live])


SHAPES = [(1, 8, 16), (1, 4096, 2048), (3, 136, 144), (8, 128, 128), (9, 264, 1552), (17, 520, 272), (64, 1024, 512),
          (65, 392, 2064), (100, 128, 1040), (128, 256, 256), (129, 264, 400), (255, 640, 128), (256, 512, 1024),
          (257, 1032, 528), (1000, 776, 640)]


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_block_gemm_dense(out, M, N, K):
    d = dev()
    a, sa, b, sb = make_product(M, N, K, 1, M + N + K, d)
    y = torch.full((M, N), float("nan"), dtype=out, device=d)
    F.block_gemm(a, sa, b, sb, y)
    torch.cuda.synchronize()
    assert F.device_error() == 0
    check_product(y, a, sa, b, sb)
    y2 = torch.full_like(y, 7.0)
    F.block_gemm(a, sa, b, sb, y2)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 128, 128), ([0, 0, 5, 0], 136, 272), ([1, 2, 3, 0, 9, 17], 264, 400), ([0, 300, 0, 1, 255, 256, 257], 384, 256),
    ([8] * 40, 256, 528), ([513, 0, 31], 520, 1040), ([0] * 30 + [1] + [0] * 33, 1024, 2048), ([2] * 200, 128, 144),
    ([64, 65, 63, 1, 0, 128, 129], 264, 640)])
@pytest.mark.parametrize("behind", [0, 5])
def test_block_gemm_grouped(out, counts, N, K, behind):
    """Ragged and empty groups; rows of y behind the last group stay as they were."""
    d = dev()
    E, M = len(counts), sum(counts) + behind
    a, sa, b, sb = make_product(M, N, K, E, M + N, d)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    before = torch.randn(M, N, generator=gen(1)).to(out)
    y = before.to(d)
    F.block_gemm(a, sa, b, sb, y, offsets=torch.from_numpy(offsets).to(d))
    torch.cuda.synchronize()
    assert F.device_error() == 0
    check_product(y, a, sa, b, sb, offsets, before)


@gpu
def test_block_gemm_all_groups_empty():
    d = dev()
    a, sa, b, sb = make_product(300, 128, 128, 3, 1, d)
    y = torch.full((300, 128), 3.0, device=d)
    F.block_gemm(a, sa, b, sb, y, offsets=torch.zeros(4, dtype=torch.int32, device=d))
    torch.cuda.synchronize()
    assert (y == 3.0).all()


@gpu
@pytest.mark.parametrize("M", [2, 200])
def test_block_gemm_exact_integers(M):
    """Small integers and power-of-two scales: every sum is exact, in any order."""
    d = dev()
    N, K, g = 264, 656, gen(5)
    a = torch.randint(-2, 3, (M, K), generator=g).float().to(torch.float8_e4m3fn).to(d)
    b = torch.randint(-2, 3, (2, N, K), generator=g).float().to(torch.float8_e4m3fn).to(d)
    sa = torch.exp2(torch.randint(-1, 2, (6, M), generator=g).float()).to(d)
    sb = torch.exp2(torch.randint(-1, 2, (2, 3, 6), generator=g).float()).to(d)
    y = torch.empty(M, N, device=d)
    off = np.array([0, M // 2, M], np.int32)
    F.block_gemm(a, sa, b, sb, y, offsets=torch.from_numpy(off).to(d))
    torch.cuda.synchronize()
    assert np.array_equal(f64(y), R.gemm(f64(a), f64(sa), f64(b), f64(sb), off)[0])


@gpu
@pytest.mark.parametrize("M", [3, 300])
def test_block_gemm_nan_stays_in_its_row(M):
    """A NaN code or scale of one row, or of another group's weights, reaches no other row."""
    d = dev()
    a, sa, b, sb = make_product(M, 256, 384, 2, 3, d)
    off = np.array([0, M - 1, M], np.int32)
    a.view(torch.uint8)[1, 200] = 0x7F
    sa[0, 0] = float("inf")
    b.view(torch.uint8)[1, 7, 9] = 0x7F
    y = torch.empty(M, 256, device=d)
    F.block_gemm(a, sa, b, sb, y, offsets=torch.from_numpy(off).to(d))
    torch.cuda.synchronize()
    got = y.cpu()
    assert torch.isnan(got[1]).all() and not torch.isfinite(got[0]).any()
    assert torch.isfinite(got[2:M - 1]).all() if M > 3 else True
    nan = torch.isnan(got[M - 1])
    assert nan[7] and nan.sum() == 1


# ------------------------------------------------------------------ combine


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("T,k,N", [(1, 1, 8), (8, 6, 2048), (33, 16, 264), (700, 6, 1032)])
def test_combine(dtype, shared, T, k, N):
    d = dev()
    g = gen(T + N)
    rows = torch.randn(T * k, N, generator=g).to(dtype).to(d)
    pos = torch.randperm(T * k, generator=g).to(torch.int32).reshape(T, k)
    pos[torch.rand(T, k, generator=g) < 0.2] = -1
    if T > 8:
        pos[5], pos[6, 0] = -1, T * k
    w = torch.rand(T, k, generator=g).to(d)
    sh = torch.randn(T, N, generator=g).to(torch.bfloat16).to(d) if shared else None
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device=d)
    F.combine(rows, pos.to(d), w, y, shared=sh)
    torch.cuda.synchronize()
    ry, mag = R.combine(f64(rows), pos.numpy(), f64(w), None if sh is None else f64(sh))
    assert np.all(np.abs(f64(y) - ry) <= (k + 2) * 2.0 ** -24 * mag + BF16 * np.abs(ry))


@gpu
def test_combine_skips_what_pos_does_not_name():
    """Rows that no place names may hold NaN."""
    d = dev()
    rows = torch.full((10, 16), float("nan"), dtype=torch.bfloat16, device=d)
    rows[4] = 2.0
    y = torch.empty(2, 16, dtype=torch.bfloat16, device=d)
    F.combine(rows, torch.tensor([[4, -1], [-1, -1]], dtype=torch.int32, device=d), torch.full((2, 2), 0.5, device=d), y)
    torch.cuda.synchronize()
    assert (y[0] == 1.0).all() and (y[1] == 0.0).all()


# ------------------------------------------------------------------ beyond 32 bits


@gpu
def test_offsets_beyond_32_bits():
    """Outputs and inputs of more than 2^31 elements: the last rows against the reference."""
    d = dev()
    rows, wide, n = 70016, 32768, 5
    assert rows * wide > 2 ** 31
    a, sa, b, sb = make_product(rows, wide, 16, 1, 3, d)
    y = torch.empty(rows, wide, dtype=torch.bfloat16, device=d)
    F.block_gemm(a, sa, b, sb, y)
    torch.cuda.synchronize()
    assert F.device_error() == 0
    check_product(y[-n:], a[-n:], sa[:, -n:], b, sb)
    q = torch.empty(rows, wide, dtype=torch.float8_e4m3fn, device=d)
    s = torch.empty(wide // 128, rows, device=d)
    F.quantize_rows(y, q, s)
    torch.cuda.synchronize()
    check_codes(f64(q[-n:]), f64(s[:, -n:]), f64(y[-n:]), np.zeros((n, wide)))
    pos = torch.tensor([[rows - 1, 0], [rows - 2, -1]], dtype=torch.int32, device=d)
    w, out = torch.tensor([[0.5, 2.0], [1.0, 1.0]], device=d), torch.empty(2, wide, dtype=torch.bfloat16, device=d)
    F.combine(y, pos, w, out)
    torch.cuda.synchronize()
    ends = f64(torch.stack([y[0], y[-2], y[-1]]))
    ry, mag = R.combine(ends, np.array([[2, 0], [1, -1]]), f64(w))
    assert np.all(np.abs(f64(out) - ry) <= 4 * 2.0 ** -24 * mag + BF16 * np.abs(ry))


@gpu
def test_route_rows_beyond_32_bits():
    """Rows so far apart that the last one starts beyond 2^31 elements."""
    d = dev()
    T, stride = 5, 1 << 29
    big = torch.empty(T * stride, dtype=torch.bfloat16, device=d)
    x = big.as_strided((T, 256), (stride, 1))
    x.copy_(torch.randn(T, 256, generator=gen(2)).to(torch.bfloat16))
    check_route(x, 6)


@gpu
@pytest.mark.parametrize("M,E", [(64, 16), (2000, 16), (6000, 16)])
def test_block_gemm_on_two_streams(M, E):
    """Calls that overlap on two streams give what each gives alone."""
    d = dev()
    N, K = 520, 656
    counts = np.bincount(np.arange(M) * 7 % 13 % E, minlength=E)
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(d)
    ins = [make_product(M, N, K, E, s, d) for s in (1, 2)]
    alone = [torch.empty(M, N, device=d) for _ in ins]
    for i, y in zip(ins, alone):
        F.block_gemm(*i, y, offsets=off)
    torch.cuda.synchronize()
    ys = [torch.full((M, N), float("nan"), device=d) for _ in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, i, y in zip(streams, ins, ys):
            F.block_gemm(*i, y, offsets=off, stream=st)
    torch.cuda.synchronize()
    assert F.device_error() == 0
    for y, z in zip(ys, alone):
        assert torch.equal(y, z)
    check_product(alone[0], *ins[0], off.cpu().numpy())


# ------------------------------------------------------------------ the run of them


class ExpertLayer:
    """An FP8 expert layer of the five operators, buffers included."""

    def __init__(self, T, H, I, E, k, d, seed=0, groups=(1, 1)):
        g = gen(seed)
        self.E, self.k, self.groups, P = E, k, groups, T * k

        def weight(n, kk):
            w = (100 * torch.randn(E, n, kk, generator=g)).clamp(-448, 448).to(torch.float8_e4m3fn).to(d)
            return w, (1e-3 * torch.exp(0.3 * torch.randn(E, -(-n // 128), -(-kk // 128), generator=g))).to(d)

        self.gu, self.gu_s = weight(2 * I, H)
        self.dn, self.dn_s = weight(H, I)
        self.bias = (0.05 * torch.randn(E, generator=g)).to(d)
        i32 = dict(dtype=torch.int32, device=d)
        f8 = dict(dtype=torch.float8_e4m3fn, device=d)
        self.ids, self.w = torch.empty(T, k, **i32), torch.empty(T, k, device=d)
        self.offsets, self.order, self.pos = torch.empty(E + 1, **i32), torch.empty(P, **i32), torch.empty(T, k, **i32)
        self.xq, self.xs = torch.zeros(P, H, **f8), torch.zeros(-(-H // 128), P, device=d)
        self.hq, self.hs = torch.zeros(P, I, **f8), torch.zeros(-(-I // 128), P, device=d)
        self.g = torch.zeros(P, 2 * I, dtype=torch.bfloat16, device=d)
        self.o = torch.zeros(P, H, dtype=torch.bfloat16, device=d)
        self.y = torch.zeros(T, H, dtype=torch.bfloat16, device=d)

    def run(self, logits, x, shared=None):
        F.route(logits, self.ids, self.w, bias=self.bias, n_groups=self.groups[0], top_groups=self.groups[1],
                group_score=F.GROUP_TOP2, scale=2.0)
        F.group_pairs(self.ids, self.offsets, self.order, self.pos)
        F.quantize_rows(x, self.xq, self.xs, pos=self.pos)
        F.block_gemm(self.xq, self.xs, self.gu, self.gu_s, self.g, offsets=self.offsets)
        F.quantize_rows(self.g, self.hq, self.hs, silu_mul=True)
        F.block_gemm(self.hq, self.hs, self.dn, self.dn_s, self.o, offsets=self.offsets)
        F.combine(self.o, self.pos, self.w, self.y, shared=shared)
        return self.y


def layer_inputs(T, H, E, seed, d):
    g = gen(seed)
    return (torch.randn(T, E, generator=g).to(d), torch.randn(T, H, generator=g).to(torch.bfloat16).to(d),
            torch.randn(T, H, generator=g).to(torch.bfloat16).to(d))


def check_layer_run(L, logits, x, shared, groups):
    """Every step against its reference on the inputs that the step before it left."""
    rid, rw = R.route(f64(logits), L.k, f64(L.bias), False, groups[0], groups[1], True, True, 2.0)
    assert np.array_equal(L.ids.cpu().numpy(), rid)
    ro, rr, rp = R.group(rid, L.E)
    n = int(ro[-1])
    assert np.array_equal(L.offsets.cpu().numpy(), ro) and np.array_equal(L.pos.cpu().numpy().reshape(-1), rp)
    xs = f64(x)[rr[:n] // L.k]
    check_codes(f64(L.xq)[:n], f64(L.xs)[:, :n], xs, np.zeros_like(xs))
    check_product(L.g[:n], L.xq[:n], L.xs[:, :n], L.gu, L.gu_s, ro)
    v = f64(L.g)[:n]
    check_codes(f64(L.hq)[:n], f64(L.hs)[:, :n], silu_mul(v), (8 + np.abs(v[:, :v.shape[1] // 2])) * 2.0 ** -22)
    check_product(L.o[:n], L.hq[:n], L.hs[:, :n], L.dn, L.dn_s, ro)
    ry, mag = R.combine(f64(L.o), rp.reshape(rid.shape), f64(L.w), f64(shared))
    assert np.all(np.abs(f64(L.y) - ry) <= (L.k + 2) * 2.0 ** -24 * mag + BF16 * np.abs(ry))


@gpu
@pytest.mark.parametrize("T,H,I,E,k,groups", [(1, 256, 128, 16, 4, (4, 2)), (8, 512, 192, 64, 6, (8, 3)),
                                              (301, 272, 144, 24, 3, (1, 1)), (900, 256, 128, 4, 2, (1, 1))])
def test_layer_of_the_five(T, H, I, E, k, groups):
    d = dev()
    L = ExpertLayer(T, H, I, E, k, d, groups=groups)
    logits, x, shared = layer_inputs(T, H, E, 5, d)
    if T > 100:
        logits[50] = -float("inf")  # a padded token
    L.run(logits, x, shared)
    torch.cuda.synchronize()
    assert F.device_error() == 0
    check_layer_run(L, logits, x, shared, groups)


@gpu
@pytest.mark.parametrize("T", [4, 200])
def test_layer_captured_on_a_side_stream(T):
    """Captured once on a stream of its own, replayed with new inputs; two captured layers
    and an eager one do not disturb each other."""
    d = dev()
    H, I, E, k = 256, 128, 12, 3
    layers = [ExpertLayer(T, H, I, E, k, d, seed=s) for s in (0, 1)]
    ins = [layer_inputs(T, H, E, 7 + s, d) for s in (0, 1)]
    layers[0].run(*ins[0])
    torch.cuda.synchronize()
    graphs, st = [], torch.cuda.Stream()
    for L, i in zip(layers, ins):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            L.run(*i)
        graphs.append(gr)
    eager = ExpertLayer(T, H, I, E, k, d, seed=2)
    new = layer_inputs(T, H, E, 99, d)
    for i in ins:
        for a, b in zip(i, new):
            a.copy_(b)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    graphs[0].replay()
    with torch.cuda.stream(other):
        graphs[1].replay()
        eager.run(*new)
    torch.cuda.synchronize()
    assert F.device_error() == 0
    for L in layers + [eager]:
        check_layer_run(L, *new, (1, 1))


# ------------------------------------------------------------------ refusals


FAKE = 0x7F0000000000
G = 1 << 36
no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake device addresses")
INV, UNS = F.FLINT_MOE_ERR_INVALID_ARG, F.FLINT_MOE_ERR_UNSUPPORTED


def addr(i):
    return FAKE + i * G


@no_gpu_only
def test_route_refusals():
    import ctypes
    lib = F.load_library()

    def call(E=256, k=6, score=0, G=1, top=1, gs=0, scale=1.0, logits=addr(0), kind=0, stride=None, T=4, bias=None,
             ids=addr(1), w=addr(2)):
        r = F.Routing(E, k, score, G, top, gs, 1, scale)
        return lib.flint_moe_route(ctypes.byref(r), logits, kind, E if stride is None else stride, T, bias, ids, w, None)

    assert lib.flint_moe_route(None, addr(0), 0, 256, 4, None, addr(1), addr(2), None) == INV
    for kw in (dict(E=0), dict(k=0), dict(T=0), dict(G=0), dict(top=0), dict(E=250, G=8, top=2), dict(top=2),
               dict(E=8, k=9), dict(E=64, G=8, top=1, k=9), dict(scale=float("nan")), dict(stride=255),
               dict(logits=None), dict(ids=None), dict(w=None), dict(logits=addr(0) + 8), dict(bias=addr(3) + 4),
               dict(ids=addr(0) + 512), dict(w=addr(1) + 32), dict(bias=addr(2))):
        assert call(**kw) == INV, kw
    for kw in (dict(kind=2), dict(score=2), dict(gs=2), dict(E=1025), dict(k=17), dict(E=66, G=33, top=2),
               dict(T=(1 << 20) + 1)):
        assert call(**kw) == UNS, kw


@no_gpu_only
def test_group_pairs_refusals():
    lib = F.load_library()

    def call(ids=addr(0), n=48, E=256, off=addr(1), order=addr(2), pos=addr(3)):
        return lib.flint_moe_group_pairs(ids, n, E, off, order, pos, None)

    for kw in (dict(n=0), dict(E=0), dict(ids=None), dict(off=None), dict(order=None), dict(pos=None),
               dict(ids=addr(0) + 4), dict(pos=addr(2) + 16), dict(order=addr(0) + 64), dict(off=addr(3) - 1024)):
        assert call(**kw) == INV, kw
    assert call(n=(1 << 24) + 1) == UNS and call(E=1025) == UNS


@no_gpu_only
def test_quantize_rows_refusals():
    lib = F.load_library()

    def call(x=addr(0), kind=0, stride=2048, rows=8, K=2048, silu=0, pos=None, k=0, places=8, q=addr(1), s=addr(2)):
        return lib.flint_moe_quantize_rows(x, kind, stride, rows, K, silu, pos, k, places, q, s, None)

    for kw in (dict(rows=0), dict(K=0), dict(places=0), dict(places=9), dict(stride=2032), dict(silu=1),
               dict(pos=addr(3)), dict(x=None), dict(q=None), dict(s=None), dict(x=addr(0) + 8), dict(q=addr(1) + 8),
               dict(q=addr(0) + 64), dict(s=addr(1) + 2048), dict(pos=addr(2), k=6, places=48)):
        assert call(**kw) == INV, kw
    for kw in (dict(kind=2), dict(K=2040), dict(stride=2052), dict(K=1 << 18, stride=1 << 18),
               dict(pos=addr(3), k=17, places=8 * 17), dict(rows=(1 << 24) + 1, places=(1 << 24) + 1)):
        assert call(**kw) == UNS, kw


@no_gpu_only
def test_block_gemm_refusals():
    lib = F.load_library()

    def call(a=addr(0), sa=addr(1), M=16, b=addr(2), sb=addr(3), E=4, off=addr(4), N=256, K=512, y=addr(5), kind=0):
        return lib.flint_moe_block_gemm(a, sa, M, b, sb, E, off, N, K, y, kind, None)

    for kw in (dict(M=0), dict(N=0), dict(K=0), dict(E=0), dict(off=None), dict(a=None), dict(sa=None), dict(b=None),
               dict(sb=None), dict(y=None), dict(a=addr(0) + 8), dict(off=addr(4) + 4), dict(y=addr(0) + 512),
               dict(y=addr(2) + 4096), dict(y=addr(4)), dict(y=addr(1) + 16), dict(y=addr(3) + 16)):
        assert call(**kw) == INV, kw
    for kw in (dict(kind=2), dict(N=252), dict(K=520), dict(E=1025), dict(N=(1 << 17) + 8), dict(K=(1 << 17) + 16),
               dict(M=(1 << 24) + 1)):
        assert call(**kw) == UNS, kw


@no_gpu_only
def test_combine_refusals():
    lib = F.load_library()

    def call(rows=addr(0), kind=0, n=48, pos=addr(1), w=addr(2), T=8, k=6, N=2048, shared=None, y=addr(3)):
        return lib.flint_moe_combine(rows, kind, n, pos, w, T, k, N, shared, y, None)

    for kw in (dict(n=0), dict(T=0), dict(k=0), dict(N=0), dict(rows=None), dict(pos=None), dict(w=None), dict(y=None),
               dict(y=addr(0) + 4096), dict(shared=addr(3)), dict(y=addr(1)), dict(y=addr(2)), dict(shared=addr(4) + 8)):
        assert call(**kw) == INV, kw
    for kw in (dict(kind=3), dict(N=2044), dict(k=17), dict(T=(1 << 20) + 1), dict(n=(1 << 24) + 1),
               dict(N=(1 << 17) + 8)):
        assert call(**kw) == UNS, kw


def test_binding_refuses_what_it_can_see():
    """Wrong types, shapes and devices raise before a pointer is taken."""
    z = torch.zeros
    ids, w = z(4, 6, dtype=torch.int32), z(4, 6)
    with pytest.raises(TypeError, match="logits"):
        F.route([1.0], ids, w)
    with pytest.raises(ValueError, match="logits: dtype"):
        F.route(z(4, 64, dtype=torch.float64), ids, w)
    with pytest.raises(ValueError, match="logits: shape"):
        F.route(z(64), ids, w)
    with pytest.raises(ValueError, match="elements of a row"):
        F.route(z(64, 4).t(), ids, w)
    with pytest.raises(ValueError, match="current CUDA device"):
        F.route(z(4, 64), ids, w)
    with pytest.raises(ValueError, match="ids"):
        F.group_pairs(ids.long(), z(9, dtype=torch.int32), z(24, dtype=torch.int32), ids)
    with pytest.raises(TypeError, match="q: expected"):
        F.quantize_rows(z(4, 256), None, z(2, 4))
    with pytest.raises(ValueError, match="x: shape"):
        F.quantize_rows(z(4, 256), z(4, 128, dtype=torch.float8_e4m3fn), z(1, 4))
    with pytest.raises(ValueError, match="b: expected"):
        F.block_gemm(None, None, z(128, 128), None, None)
    with pytest.raises(ValueError, match="y: shape"):
        F.block_gemm(None, None, z(1, 128, 128), None, z(4, 64))
    with pytest.raises(ValueError, match="rows: shape"):
        F.combine(z(4, 64), ids, w, z(4, 128, dtype=torch.bfloat16))


@gpu
def test_binding_refuses_tensors_without_storage():
    """A tensor of the right kind that has no memory raises, from every call, and the
    interpreter goes on."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    d = dev()
    with FakeTensorMode():
        def e(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device=d)

        i32, bf, f8 = torch.int32, torch.bfloat16, torch.float8_e4m3fn
        ids, w = e(4, 6, dtype=i32), e(4, 6)
        calls = [
            lambda: F.route(e(4, 64), ids, w),
            lambda: F.group_pairs(ids, e(65, dtype=i32), e(24, dtype=i32), e(4, 6, dtype=i32)),
            lambda: F.quantize_rows(e(4, 256, dtype=bf), e(4, 256, dtype=f8), e(2, 4)),
            lambda: F.block_gemm(e(4, 256, dtype=f8), e(2, 4), e(1, 128, 256, dtype=f8), e(1, 1, 2), e(4, 128, dtype=bf)),
            lambda: F.combine(e(24, 128, dtype=bf), ids, w, e(4, 128, dtype=bf)),
        ]
        for f in calls:
            with pytest.raises(RuntimeError):
                f()
    x = torch.ones(2, 64, device=d)
    F.route(x, torch.empty(2, 6, dtype=i32, device=d), torch.empty(2, 6, device=d))
    torch.cuda.synchronize()


def test_binding_refuses_counts_beyond_31_bits():
    """What the C ABI's ints cannot hold raises; cut to 32 bits it would be a small count."""
    n = (1 << 32) + 4

    def m(*shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="meta")

    i32, f8 = torch.int32, torch.float8_e4m3fn
    ids, w = torch.zeros(4, 6, dtype=i32), torch.zeros(4, 6)
    for kw in (dict(score=1 << 32), dict(n_groups=n), dict(top_groups=n), dict(group_score=-(1 << 32))):
        with pytest.raises(ValueError, match="31 bits"):
            F.route(torch.zeros(4, 64), ids, w, **kw)
    with pytest.raises(ValueError, match="logits: .*31 bits"):
        F.route(m(n, 64), m(n, 6, dtype=i32), m(n, 6))
    with pytest.raises(ValueError, match="ids, offsets: .*31 bits"):
        F.group_pairs(m(n, dtype=i32), m(9, dtype=i32), m(n, dtype=i32), m(n, dtype=i32))
    with pytest.raises(ValueError, match="q: .*31 bits"):
        F.quantize_rows(m(4, 128), m(n, 128, dtype=f8), m(1, n))
    with pytest.raises(ValueError, match="x: .*31 bits"):
        F.quantize_rows(m(n, 128), m(4, 128, dtype=f8), m(1, 4))
    with pytest.raises(ValueError, match="b: .*31 bits"):
        F.block_gemm(m(4, 128, dtype=f8), m(1, 4), m(n, 128, 128, dtype=f8), m(n, 1, 1), m(4, 128))
    with pytest.raises(ValueError, match="y: .*31 bits"):
        F.block_gemm(m(n, 128, dtype=f8), m(1, n), m(1, 128, 128, dtype=f8), m(1, 1, 1), m(n, 128))
    with pytest.raises(ValueError, match="rows: .*31 bits"):
        F.combine(m(n, 128), ids, w, torch.zeros(4, 128, dtype=torch.bfloat16))


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(16, 7168, 144), (16, 7176, 144), (41, 2568, 400), (60, 1792, 272), (70, 1640, 272),
                                   (130, 1032, 1552), (193, 520, 272), (215, 8, 1040)])
def test_block_gemm_dense_passes(out, M, N, K):
    """Dense products on either side of what passes of eight rows take."""
    d = dev()
    a, sa, b, sb = make_product(M, N, K, 1, M + N + K, d)
    guard = torch.full((M + 2, N), 7.0, dtype=out, device=d)
    y = guard[1:-1]
    F.block_gemm(a, sa, b, sb, y)
    torch.cuda.synchronize()
    assert F.device_error() == 0
    assert bool((guard[0] == 7).all()) and bool((guard[-1] == 7).all())
    check_product(y, a, sa, b, sb)


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,N,K", [
    ([70], 1640, 1040),   # 9 blocks: three CTAs of three and one of none
    ([130], 1032, 1552),  # 13 blocks
    ([41], 2600, 1536),
    ([64], 4096, 1024),   # 8 blocks
    ([100], 2568, 2064),  # 17 blocks between two CTAs
    ([8], 8192, 4112),
    ([0, 33, 0, 37], 520, 1168),
    ([5, 0, 65, 30], 1032, 1552),
])
def test_block_gemm_split_sums(out, counts, N, K):
    """Products with too few units for the SMs, whose K blocks several blocks share; rows
    behind and between stay as they were, and a second call gives the same bits."""
    d = dev()
    E, M = len(counts), sum(counts)
    behind = 3 if E > 1 else 0
    a, sa, b, sb = make_product(M + behind, N, K, E, M + N + K, d)
    offsets = None if E == 1 else torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=d)
    before = torch.randn(M + behind + 2, N, generator=gen(5)).to(out).to(d)
    ys = []
    for _ in range(2):
        guard = before.clone()
        F.block_gemm(a, sa, b, sb, guard[1:-1], offsets=offsets)
        torch.cuda.synchronize()
        assert F.device_error() == 0
        assert torch.equal(guard[0], before[0]) and torch.equal(guard[-1], before[-1])
        ys.append(guard[1:-1])
    check_product(ys[0], a, sa, b, sb, None if offsets is None else offsets.cpu().numpy(), before[1:-1])
    assert torch.equal(ys[0], ys[1])


@gpu
def test_block_gemm_split_sums_at_once():
    """Captured and replayed on two streams at a time, each with its own inputs."""
    d = dev()
    ins = [make_product(48, 2048, 2560, 1, i, d) for i in range(2)]
    want = [torch.empty(48, 2048, device=d) for _ in ins]
    got = [torch.zeros(48, 2048, device=d) for _ in ins]
    for i, y in zip(ins, want):
        F.block_gemm(*i, y)
    torch.cuda.synchronize()
    streams, graphs = [torch.cuda.Stream() for _ in ins], []
    for st, i, y in zip(streams, ins, got):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(8):
                F.block_gemm(*i, y)
        graphs.append(g)
    for _ in range(5):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert F.device_error() == 0
    for y, w in zip(got, want):
        assert torch.equal(y, w)
