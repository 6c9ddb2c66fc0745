"""Linear, gated and integer products, their gradients, and rows to 8-bit integers, against
64-bit references, through the Python binding.

Tolerances, derived from the number formats:
  product       K exact products, each addition losing at most 2^-23 of the running magnitude:
                (K + 2) 2^-23 of the sum of magnitudes; bf16 outputs half a step more, 2^-8 of
                the value.  Gradients the same, over N or the expert's rows.
  activation    g * sigmoid(v): expf and the quotient within (8 + 2 |v|) 2^-22 of the value,
                the inner polynomial's four roundings within that; below v = -87 it may be 0.
                Both slopes stay below 1.13, which carries a sum's error to the output.
  slope         p + g p q v' with each factor as above: (16 + 4 |v|) 2^-22 of the terms' magnitudes.
  integers      sums are exact; the two scales and their product are three roundings, 2^-22.
  codes         exact: the whole number next to the quotient by the stored scale.
"""

import math

import pytest
import torch

import linear_reference as R
from moe_decode_router_gb300 import flint_moe as F

gpu = pytest.mark.gpu
BF16 = 2.0 ** -8
ACTS = {"silu": F.ACT_SILU, "gelu": F.ACT_GELU}
TINY = 1e-36


def dev():
    F.load_library()
    return torch.device("cuda:0")


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rand(seed, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=gen(seed))).to(torch.bfloat16).to(dev())


def codes(seed, *shape):
    return torch.randint(-128, 128, shape, generator=gen(seed), dtype=torch.int8).to(dev())


def groups(counts):
    """offsets of groups of so many rows, or None for one dense group."""
    if len(counts) == 1:
        return None
    edge = [0]
    for c in counts:
        edge.append(edge[-1] + c)
    return torch.tensor(edge, dtype=torch.int32, device=dev())


def done():
    torch.cuda.synchronize()
    assert F.device_error() == 0


def half_step(t, y):
    return BF16 * y.abs() if t.dtype == torch.bfloat16 else 0.0


def near(got, want, tol, before=None):
    """Within the tolerance where there is a value, as before where the reference has none."""
    live = ~torch.isnan(want)
    off = (got.double() - want).abs()
    bad = live & ~(off <= tol)
    assert not bool(bad.any()), (int(bad.sum()), float((off / tol)[bad].max()), bad.nonzero()[:4].tolist())
    if before is not None:
        assert torch.equal(got[~live], before[~live])


def framed(shape, dtype, seed=5):
    """An output of random values with a guard row on either side: (whole, inner, before)."""
    whole = torch.randn(shape[0] + 2, *shape[1:], generator=gen(seed)).to(dtype).to(dev())
    return whole, whole[1:-1], whole.clone()


def unframed(whole, before):
    assert torch.equal(whole[0], before[0]) and torch.equal(whole[-1], before[-1])


# rows of each expert (one: dense), N (of gated products I = N / 2), K
SHAPES = [
    ([1], 32, 16), ([1], 8192, 2048), ([3], 160, 144), ([8], 1024, 2048), ([9], 224, 1552), ([17], 544, 272),
    ([64], 1024, 512), ([65], 416, 2064), ([100], 128, 1040), ([128], 256, 256), ([129], 288, 400), ([255], 640, 128),
    ([256], 512, 1024), ([257], 1056, 528), ([700], 800, 640), ([1031], 256, 336),
    ([0, 1, 0, 2], 96, 80), ([1] * 8, 128, 256), ([8, 0, 9, 7, 1], 160, 208), ([33, 64, 0, 65], 320, 272),
    ([0, 0, 130, 3], 544, 144), ([300, 1, 40, 511], 288, 400), ([5] * 40, 224, 96), ([0, 1000, 0], 128, 1040),
]
SHAPES_8 = [([5], 8, 16), ([130], 1032, 96), ([20, 0, 70], 136, 272)]  # N a multiple of 8 alone


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,N,K", SHAPES + SHAPES_8)
def test_linear(out, counts, N, K):
    E, behind = len(counts), 3 if len(counts) > 1 else 0
    M, offsets = sum(counts) + behind, groups(counts)
    x, w = rand(M + N, M, K), rand(K, E, N, K, scale=0.1)
    if behind:
        x[-behind:] = math.nan
    whole, y, before = framed((M, N), out)
    F.linear(x, w, y, offsets=offsets)
    done()
    unframed(whole, before)
    ref, mag = R.product(x, w, offsets)
    near(y, ref, (K + 2) * 2.0 ** -23 * mag + half_step(y, ref), before[1:-1])


def check_gated(h, g, u, g_off, u_off, act):
    """h against act(g) * u of sums that are off by no more than g_off and u_off."""
    a, v = R.activation(g, act), R.inner(g, act)[0]
    want = a * u
    tol = 1.13 * g_off * (u.abs() + u_off) + a.abs() * u_off + (8 + 2 * v.abs()) * 2.0 ** -22 * want.abs() + TINY * (1 + u.abs())
    return want, tol + half_step(h, want.abs() + tol)


@gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_gated_linear(act, keep, counts, N, K):
    E, behind = len(counts), 3 if len(counts) > 1 else 0
    M, offsets, I = sum(counts) + behind, groups(counts), N // 2
    x, w = rand(M + N, M, K), rand(K, E, N, K, scale=2 / math.sqrt(K))
    if behind:
        x[-behind:] = math.nan
    whole, h, before = framed((M, I), torch.bfloat16)
    kept_whole, gu, kept_before = framed((M, N), torch.bfloat16)
    F.gated_linear(x, w, h, gu=gu if keep else None, offsets=offsets, act=ACTS[act])
    done()
    unframed(whole, before)
    sums, mag = R.product(x, w, offsets)
    off = (K + 2) * 2.0 ** -23 * mag
    near(h, *check_gated(h, sums[:, :I], sums[:, I:], off[:, :I], off[:, I:], act), before[1:-1])
    if keep:
        unframed(kept_whole, kept_before)
        near(gu, sums, off + half_step(gu, sums.abs() + off), kept_before[1:-1])
    else:
        assert torch.equal(kept_whole, kept_before)


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("which", ["both", "dx", "dw"])
@pytest.mark.parametrize("counts,N,K", SHAPES + SHAPES_8)
def test_linear_backward(out, which, counts, N, K):
    E, behind = len(counts), 3 if len(counts) > 1 else 0
    M, offsets = sum(counts) + behind, groups(counts)
    dy, x, w = rand(M, M, N), rand(M + N, M, K), rand(K, E, N, K, scale=0.1)
    if behind:
        x[-behind:] = math.nan
        dy[-behind:] = math.inf
    whole, dx, before = framed((M, K), torch.bfloat16)
    w_whole, dw, w_before = framed((E, N, K), out)
    F.linear_backward(dy, x, w, dx=None if which == "dw" else dx, dw=None if which == "dx" else dw, offsets=offsets)
    done()
    unframed(whole, before)
    unframed(w_whole, w_before)
    if which != "dw":
        ref, mag = R.input_gradient(dy, w, offsets)
        near(dx, ref, (N + 2) * 2.0 ** -23 * mag + half_step(dx, ref), before[1:-1])
    else:
        assert torch.equal(whole, before)
    if which != "dx":
        ref, mag = R.weight_gradient(dy, x, E, offsets)
        near(dw, ref, (max(counts) + 2) * 2.0 ** -23 * mag + half_step(dw, ref))
    else:
        assert torch.equal(w_whole, w_before)


def check_gate_backward(dgu, dh, gu, act, before=None, live=None):
    I = dh.shape[1]
    g, u, d = gu[:, :I].double(), gu[:, I:].double(), dh.double()
    s, terms = R.slope(g, act)
    v, a = R.inner(g, act)[0].abs(), R.activation(g, act)
    want = torch.cat([d * u * s, d * a], 1)
    tol = torch.cat([(d * u).abs() * ((16 + 4 * v) * 2.0 ** -22 * terms + TINY), d.abs() * ((8 + 2 * v) * 2.0 ** -22 * a.abs() + TINY)], 1)
    if live is not None:
        want[live:] = math.nan
    near(dgu, want, tol + half_step(dgu, want.abs() + tol) + TINY, before)


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("counts,N,K", SHAPES)
def test_gated_linear_backward(out, act, counts, N, K):
    E, behind = len(counts), 3 if len(counts) > 1 else 0
    M, offsets, I = sum(counts) + behind, groups(counts), N // 2
    dh, gu = rand(M, M, I), rand(M + 1, M, N, scale=2.0)
    x, w = rand(M + N, M, K), rand(K, E, N, K, scale=0.1)
    if behind:
        for t in (dh, gu, x):
            t[-behind:] = math.nan
    d_whole, dgu, d_before = framed((M, N), torch.bfloat16)
    whole, dx, before = framed((M, K), torch.bfloat16)
    w_whole, dw, w_before = framed((E, N, K), out)
    F.gated_linear_backward(dh, gu, x, w, dgu, dx=dx, dw=dw, offsets=offsets, act=ACTS[act])
    done()
    for a, b in ((d_whole, d_before), (whole, before), (w_whole, w_before)):
        unframed(a, b)
    check_gate_backward(dgu, dh, gu, act, d_before[1:-1], M - behind)
    if behind:
        dgu[-behind:] = 0
    ref, mag = R.input_gradient(dgu, w, offsets)
    near(dx, ref, (N + 2) * 2.0 ** -23 * mag + half_step(dx, ref), before[1:-1])
    ref, mag = R.weight_gradient(dgu, x, E, offsets)
    near(dw, ref, (max(counts) + 2) * 2.0 ** -23 * mag + half_step(dw, ref))


@gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gate_backward_values(act):
    """Gates from the type's lowest to its highest: finite slopes that end at 0 and 1."""
    d = dev()
    g = torch.cat([torch.linspace(-100, 100, 4001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e4, -1e4, 1e19, -1e19, 3e38, -3e38])])
    g = torch.cat([g, torch.zeros(-g.numel() % 16)]).to(torch.bfloat16).to(d)[None]
    I = g.shape[1]
    gu = torch.cat([g, torch.full_like(g, 0.5)], 1)
    dh, dgu = torch.full_like(g, 2.0), torch.empty_like(gu)
    x, w = rand(1, 1, 16), rand(2, 1, 2 * I, 16)
    F.gated_linear_backward(dh, gu, x, w, dgu, act=ACTS[act])
    done()
    got, real = dgu.double(), g.double()
    assert bool(torch.isfinite(got[:, :I]).all())
    near_zero = real.abs() <= 100
    s, terms = R.slope(real.clamp(-100, 100), act)
    v = R.inner(real.clamp(-100, 100), act)[0].abs()
    off = (got[:, :I] - s).abs()
    tol = (16 + 4 * v.clamp(max=90)) * 2.0 ** -22 * terms + 1e-30
    assert bool((off <= tol + BF16 * (s.abs() + tol))[near_zero].all())
    assert bool((got[:, :I][real > 50] == 1).all()) and bool((got[:, :I][real < -200] == 0).all())
    twice = (2 * real).to(torch.bfloat16).double()  # the type's largest, doubled, is its infinity
    assert bool((got[:, I:][real > 50] == twice[real > 50]).all()) and bool((got[:, I:][real < -200] == 0).all())


@gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_against_differences(act):
    """The change of sum(dh * h) along a direction of x and of w, by central differences in 64
    bits.  The kernel rounds dgu to bf16 and the gradients once more: 2^-8 of the magnitudes each."""
    counts, N, K = [70, 0, 33], 96, 80
    M, offsets, I, E = sum(counts), groups(counts), N // 2, len(counts)
    x, w = rand(1, M, K), rand(2, E, N, K, scale=0.2)
    h, gu = torch.empty(M, I, dtype=torch.bfloat16, device=dev()), torch.empty(M, N, dtype=torch.bfloat16, device=dev())
    dh = rand(3, M, I)
    F.gated_linear(x, w, h, gu=gu, offsets=offsets, act=ACTS[act])
    dgu, dx, dw = torch.empty_like(gu), torch.empty_like(x), torch.empty(E, N, K, device=dev())
    F.gated_linear_backward(dh, gu, x, w, dgu, dx=dx, dw=dw, offsets=offsets, act=ACTS[act])
    done()
    along_x, along_w = rand(4, M, K), rand(5, E, N, K)

    def loss(step, change):
        s = gu.double() + step * change
        return float((dh.double() * R.activation(s[:, :I], act) * s[:, I:]).sum())

    for change, grad, along, mag in (
            (R.product(along_x, w, offsets)[0], dx, along_x, R.input_gradient(dgu.abs(), w.abs(), offsets)[0]),
            (R.product(x, along_w, offsets)[0], dw, along_w, R.weight_gradient(dgu.abs(), x.abs(), E, offsets)[0])):
        eps = 1e-4
        want = (loss(eps, change) - loss(-eps, change)) / (2 * eps)
        got = float((grad.double() * along.double()).sum())
        assert abs(got - want) <= 2.1 * BF16 * float((mag * along.double().abs()).sum())


# ------------------------------------------------------------------ integers


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("counts,N,K", SHAPES + SHAPES_8)
def test_integer_gemm(out, act, counts, N, K):
    if act != "none" and N % 32:
        pytest.skip("a gated matrix has a multiple of 32 rows")
    E, behind = len(counts), 3 if len(counts) > 1 else 0
    M, offsets = sum(counts) + behind, groups(counts)
    a, b = codes(M + N, M, K), codes(K, E, N, K)
    sa = torch.exp(torch.randn(M, generator=gen(1))).to(dev()) / 128
    sb = torch.exp(torch.randn(E, N, generator=gen(2))).to(dev()) / (64 * math.sqrt(K))
    if behind:
        sa[-behind:] = math.nan
    width = N if act == "none" else N // 2
    whole, y, before = framed((M, width), out)
    F.integer_gemm(a, sa, b, sb, y, offsets=offsets, act=ACTS.get(act, F.ACT_NONE))
    done()
    unframed(whole, before)
    sums, scale = R.integer_sums(a, b, offsets), torch.full((M, N), math.nan, dtype=torch.float64, device=dev())
    for e, at in enumerate(R.by_expert(offsets, M, E)):
        scale[at] = sa[at].double()[:, None] * sb[e].double()
    v = sums * scale
    off = 2.0 ** -22 * v.abs()
    if act == "none":
        near(y, v, off + half_step(y, v.abs() + off), before[1:-1])
    else:
        near(y, *check_gated(y, v[:, :width], v[:, width:], off[:, :width], off[:, width:], act), before[1:-1])


@gpu
@pytest.mark.parametrize("K", [16, 1024, 1040, 4096, 131056])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_integer_sums_are_exact(M, K):
    """The largest sums there are, and sums whose last bit an fp32 accumulator would lose."""
    d, N = dev(), 64
    a = torch.full((M, K), -128, dtype=torch.int8)
    b = torch.full((1, N, K), -128, dtype=torch.int8)
    b[0, 1] = 127
    b[0, 2, ::2] = 127
    b[0, 3, 0] = -127
    b[0, 4, -1] = 1
    b[0, 5:] = torch.randint(-128, 128, (N - 5, K), generator=gen(K), dtype=torch.int8)
    a[M // 2, K // 2:] = 1
    a[M - 1] = torch.randint(-128, 128, (K,), generator=gen(M), dtype=torch.int8)
    a, b = a.to(d), b.to(d)
    y, ones = torch.empty(M, N, device=d), torch.ones(max(M, N), device=d)
    F.integer_gemm(a, ones[:M], b, ones[None, :N].contiguous(), y)
    done()
    want = R.integer_sums(a, b)
    assert torch.equal(y, want.float())


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,K,pad", [(1, 16, 0), (3, 128, 8), (7, 144, 0), (129, 2048, 0), (1000, 512, 16),
                                        (5, 2064, 0), (2, 16400, 8), (3, 131072, 0), (1025, 1040, 0), (33, 1024, 8),
                                        (1030, 1808, 0), (70, 4096, 0), (3, 8208, 0), (9, 5136, 16)])
def test_integer_quantize_rows(dtype, rows, K, pad):
    x = (3 * torch.randn(rows, K + pad, generator=gen(rows + K))).to(dtype).to(dev())[:, :K]
    q_whole, q, q_before = framed((rows, K), torch.int8)
    s = torch.empty(rows, device=dev())
    F.integer_quantize_rows(x, q, s)
    done()
    unframed(q_whole, q_before)
    want, scale = R.integer_rows(x)
    assert torch.equal(s, scale) and torch.equal(q.double(), want)


@gpu
def test_integer_quantize_rows_ties():
    """Quotients that are the middle of two codes, and their neighbours in the type."""
    d, K = dev(), 512
    half = torch.arange(-126.5, 127, 1.0)
    x = torch.zeros(12, K)
    for r, (top, dtype) in enumerate([(127.0, torch.bfloat16), (127.0, torch.float32), (254.0, torch.float32),
                                      (127.0 * 2.0 ** -20, torch.float32), (1.0, torch.float32), (0.3, torch.float32)]):
        v = (half * (top / 127)).float()
        x[2 * r, :254], x[2 * r, 300] = v, top
        x[2 * r + 1, :254], x[2 * r + 1, 300] = torch.nextafter(v, torch.tensor(math.inf)), top
    for dtype in (torch.float32, torch.bfloat16):
        t = x.to(dtype).to(d)
        q, s = torch.empty(12, K, dtype=torch.int8, device=d), torch.empty(12, device=d)
        F.integer_quantize_rows(t, q, s)
        done()
        want, scale = R.integer_rows(t)
        assert torch.equal(s, scale) and torch.equal(q.double(), want)


@gpu
@pytest.mark.parametrize("K", [272, 4112])
def test_integer_quantize_rows_to_places(K):
    """Every row goes to all of its places; places of no row keep their bytes; places out of
    range are skipped."""
    d, rows, k, places = dev(), 50, 3, 200
    x = rand(9, rows, K)
    perm = torch.randperm(places, generator=gen(10))[:rows * k].to(torch.int32).reshape(rows, k)
    perm[3, 1], perm[4] = -1, -1
    perm[5, 2] = places
    q, s = torch.full((places, K), 0x55, dtype=torch.int8, device=d), torch.full((places,), -5.0, device=d)
    F.integer_quantize_rows(x, q, s, pos=perm.to(d))
    done()
    plain_q, plain_s = R.integer_rows(x)
    want_q, want_s = torch.full((places, K), 0x55, dtype=torch.float64, device=d), torch.full((places,), -5.0, device=d)
    for t in range(rows):
        for p in perm[t].tolist():
            if 0 <= p < places:
                want_q[p], want_s[p] = plain_q[t], plain_s[t]
    assert torch.equal(q.double(), want_q) and torch.equal(s, want_s)


@gpu
@pytest.mark.parametrize("K", [256, 2304])
def test_integer_quantize_rows_edge_values(K):
    d = dev()
    x = torch.zeros(6, K)
    x[1, :128] = 1e-38
    x[2], x[2, 7] = 3e38, -3e38
    x[3, 5] = math.nan
    x[4, 200], x[4, 3] = -math.inf, 2.0
    x[5] = torch.linspace(-1, 1, K)
    q, s = torch.full((6, K), 9, dtype=torch.int8, device=d), torch.empty(6, device=d)
    F.integer_quantize_rows(x.to(d), q, s)
    done()
    assert not bool(torch.isfinite(s[3:5]).any()) and not bool(q[3:5].any())
    fine = [0, 1, 2, 5]
    want, scale = R.integer_rows(x[fine].to(d))
    assert torch.equal(s[fine], scale) and torch.equal(q[fine].double(), want)
    assert bool((q[2] != 0).all()) and not bool(q[:2].any())


# ------------------------------------------------------------------ values that are not finite


@gpu
def test_not_finite_values_stay_with_their_rows():
    """Infinities and NaN of one row reach that row's outputs and its expert's gradient alone,
    in tiles that rows of several experts share."""
    counts, N, K = [37, 70, 5, 141], 96, 80
    M, offsets, E = sum(counts), groups(counts), len(counts)
    x, w, dy = rand(1, M, K), rand(2, E, N, K, scale=0.2), rand(3, M, N)

    def run(x, dy):
        y, dx, dw = (torch.empty(s, device=dev(), dtype=torch.bfloat16) for s in ((M, N), (M, K), (E, N, K)))
        h, gu = torch.empty(M, N // 2, device=dev(), dtype=torch.bfloat16), torch.empty_like(y)
        F.linear(x, w, y, offsets=offsets)
        F.linear_backward(dy, x, w, dx=dx, dw=dw, offsets=offsets)
        F.gated_linear(x, w, h, gu=gu, offsets=offsets)
        done()
        return y, dx, dw, h, gu

    good = run(x, dy)
    for row, e in ((36, 0), (37, 1), (106, 1), (107, 2), (112, 3), (252, 3)):
        for bad in (math.nan, math.inf):
            x2, dy2 = x.clone(), dy.clone()
            x2[row, 3], dy2[row, 5] = bad, bad
            y, dx, dw, h, gu = run(x2, dy2)
            rest = torch.arange(M, device=dev()) != row
            for a, b in ((y, good[0]), (dx, good[1]), (h, good[3]), (gu, good[4])):
                assert torch.equal(a[rest], b[rest]) and not bool(torch.isfinite(a[row]).all())
            for i in range(E):
                assert torch.equal(dw[i], good[2][i]) == (i != e)


# ------------------------------------------------------------------ together


def layer(T, k, E, K, I, seed):
    """A layer's tensors and its routing: (x, gate_up, down, w, offsets, order, pos)."""
    d = dev()
    x, gate_up = rand(seed, T, K), rand(seed + 1, E, 2 * I, K, scale=1.5 / math.sqrt(K))
    down, logits = rand(seed + 2, E, K, I, scale=1.5 / math.sqrt(I)), rand(seed + 3, T, E)
    i32 = dict(dtype=torch.int32, device=d)
    ids, w = torch.empty(T, k, **i32), torch.empty(T, k, device=d)
    offsets, order, pos = torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T, k, **i32)
    F.route(logits, ids, w)
    F.group_pairs(ids, offsets, order, pos)
    return x, gate_up, down, w, offsets, order, pos


@gpu
@pytest.mark.parametrize("T,k,E,K,I", [(3, 2, 8, 256, 64), (200, 3, 8, 272, 96), (64, 6, 32, 512, 128)])
def test_expert_layer_in_integers(T, k, E, K, I):
    """Routed, quantised, both products and combined, step by step against 64 bits on the codes
    that each step left."""
    d = dev()
    x, gate_up, down, w, offsets, order, pos = layer(T, k, E, K, I, T)
    P, bf = T * k, torch.bfloat16

    def quantised(m):
        q, s = torch.empty(m.shape, dtype=torch.int8, device=d), torch.empty(m.shape[:-1], device=d)
        F.integer_quantize_rows(m.reshape(-1, m.shape[-1]), q.view(-1, m.shape[-1]), s.view(-1))
        return q, s

    (gq, gs), (dq, ds) = quantised(gate_up), quantised(down)
    xq, xs = torch.empty(P, K, dtype=torch.int8, device=d), torch.empty(P, device=d)
    h, y, out = (torch.empty(P, n, dtype=bf, device=d) for n in (I, K, K))
    out = torch.empty(T, K, dtype=bf, device=d)
    F.integer_quantize_rows(x, xq, xs, pos=pos)
    F.integer_gemm(xq, xs, gq, gs, h, offsets=offsets, act=F.ACT_SILU)
    hq, hs = quantised(h)
    F.integer_gemm(hq, hs, dq, ds, y, offsets=offsets)
    F.combine(y, pos, w, out)
    done()
    want_q, want_s = R.integer_rows(x[order.long() // k])
    assert torch.equal(xq.double(), want_q) and torch.equal(xs, want_s)

    def exact(q, s, bq, bs):
        v = R.integer_sums(q, bq, offsets) * s.double()[:, None]
        for e, at in enumerate(R.by_expert(offsets, P, E)):
            v[at] *= bs[e].double()
        return v

    v = exact(xq, xs, gq, gs)
    off = 2.0 ** -22 * v.abs()
    near(h, *check_gated(h, v[:, :I], v[:, I:], off[:, :I], off[:, I:], "silu"))
    v = exact(hq, hs, dq, ds)
    near(y, v, (2.0 ** -22 + BF16) * v.abs())
    # and the whole against the layer in 64 bits: codes are off by half of 1/127 of the row's largest
    s, _ = R.product(x[order.long() // k], gate_up, offsets)
    full, _ = R.product(R.activation(s[:, :I], "silu") * s[:, I:], down, offsets)
    ref = torch.zeros(T, K, dtype=torch.float64, device=d)
    for j in range(k):
        ref += w[:, j].double()[:, None] * full[pos[:, j].long()]
    assert float((out.double() - ref).norm() / ref.norm()) < 0.05


@gpu
def test_expert_layer_trained():
    """Forward and backward of a layer of experts, each step against 64 bits on what it was given."""
    T, k, E, K, I = 150, 3, 8, 272, 96
    d, bf = dev(), torch.bfloat16
    x, gate_up, down, w, offsets, order, pos = layer(T, k, E, K, I, 1)
    P = T * k
    xp = x[order.long() // k].contiguous()
    h, gu, y = (torch.empty(P, n, dtype=bf, device=d) for n in (I, 2 * I, K))
    F.gated_linear(xp, gate_up, h, gu=gu, offsets=offsets)
    F.linear(h, down, y, offsets=offsets)
    dy = rand(7, P, K)
    dh, dgu, dxp = torch.empty_like(h), torch.empty_like(gu), torch.empty_like(xp)
    d_down, d_gate_up = torch.empty(down.shape, device=d), torch.empty(gate_up.shape, device=d)
    F.linear_backward(dy, h, down, dx=dh, dw=d_down, offsets=offsets)
    F.gated_linear_backward(dh, gu, xp, gate_up, dgu, dx=dxp, dw=d_gate_up, offsets=offsets)
    done()
    for got, (ref, mag), n in ((gu, R.product(xp, gate_up, offsets), K), (y, R.product(h, down, offsets), I),
                               (dh, R.input_gradient(dy, down, offsets), K), (dxp, R.input_gradient(dgu, gate_up, offsets), 2 * I),
                               (d_down, R.weight_gradient(dy, h, E, offsets), P), (d_gate_up, R.weight_gradient(dgu, xp, E, offsets), P)):
        off = (n + 2) * 2.0 ** -23 * mag
        near(got, ref, off + half_step(got, ref.abs() + off))
    check_gate_backward(dgu, dh, gu, "silu")


# ------------------------------------------------------------------ streams, graphs, order


def every_call(seed):
    """(buffers that are written, a function that makes every call once)."""
    d, bf = dev(), torch.bfloat16
    counts = [40, 0, 300, 17]
    offsets, M, E, N, K = groups(counts), sum(counts), len(counts), 160, 144
    x, w, dy, dh = rand(seed, M, K), rand(seed + 1, E, N, K, scale=0.2), rand(seed + 2, M, N), rand(seed + 3, M, N // 2)
    b, sb = codes(seed + 4, E, N, K), torch.rand(E, N, generator=gen(seed)).to(d)
    o = dict(y=(M, N), h=(M, N // 2), gu=(M, N), dx=(M, K), dw=(E, N, K), dgu=(M, N), dx2=(M, K), dw2=(E, N, K), z=(M, N // 2))
    o = {n: torch.zeros(s, dtype=bf, device=d) for n, s in o.items()}
    o["q"], o["s"] = torch.zeros(M, K, dtype=torch.int8, device=d), torch.zeros(M, device=d)

    def run(stream=None):
        F.linear(x, w, o["y"], offsets=offsets, stream=stream)
        F.gated_linear(x, w, o["h"], gu=o["gu"], offsets=offsets, act=F.ACT_GELU, stream=stream)
        F.linear_backward(dy, x, w, dx=o["dx"], dw=o["dw"], offsets=offsets, stream=stream)
        F.gated_linear_backward(dh, o["gu"], x, w, o["dgu"], dx=o["dx2"], dw=o["dw2"], offsets=offsets, act=F.ACT_GELU,
                                stream=stream)
        F.integer_quantize_rows(x, o["q"], o["s"], stream=stream)
        F.integer_gemm(o["q"], o["s"], b, sb, o["z"], offsets=offsets, act=F.ACT_SILU, stream=stream)

    return o, run


@gpu
def test_repeated_calls_give_the_same_bits():
    o, run = every_call(1)
    run()
    done()
    first = {n: t.clone() for n, t in o.items()}
    for t in o.values():
        t.zero_()
    run()
    done()
    for n in o:
        assert torch.equal(o[n], first[n]), n


@gpu
def test_two_streams_and_captured_graphs_at_once():
    sets = [every_call(s) for s in (1, 100)]
    for _, run in sets:
        run()
    done()
    want = [{n: t.clone() for n, t in o.items()} for o, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    graphs = []
    for st, (_, run) in zip(streams, sets):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            run()
        graphs.append(g)
    for o, _ in sets:
        for t in o.values():
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(4):
        for st, g, (_, run) in zip(streams, graphs, sets):
            with torch.cuda.stream(st):
                g.replay()
            run(stream=st)
    done()
    for (o, _), w in zip(sets, want):
        for n in o:
            assert torch.equal(o[n], w[n]), n


@gpu
def test_both_marshallings_make_the_same_calls(monkeypatch):
    assert not isinstance(F._FAST, F._NotLoaded)
    o, run = every_call(3)
    run()
    done()
    first = {n: t.clone() for n, t in o.items()}
    for t in o.values():
        t.zero_()
    monkeypatch.setattr(F, "_FAST", F._NotLoaded())
    run(stream=torch.cuda.current_stream())
    done()
    for n in o:
        assert torch.equal(o[n], first[n]), n


@gpu
@pytest.mark.parametrize("op", ["linear", "gated", "integer"])
def test_offsets_beyond_32_bits(op):
    """Rows whose elements lie past 2^31 and 2^32 bytes."""
    d = dev()
    K, N, tail = 16384, 64, 5
    M = (1 << 31) // K + 300
    x = torch.zeros(M, K, dtype=torch.int8 if op == "integer" else torch.bfloat16, device=d)
    w = codes(2, 1, N, K) if op == "integer" else rand(2, 1, N, K, scale=0.05)
    x[-tail:] = codes(1, tail, K) if op == "integer" else rand(1, tail, K)
    y = torch.full((M, N if op != "gated" else N // 2), 7.0, dtype=torch.bfloat16, device=d)
    if op == "linear":
        F.linear(x, w, y)
    elif op == "gated":
        F.gated_linear(x, w, y)
    else:
        F.integer_gemm(x, torch.ones(M, device=d), w, torch.ones(1, N, device=d), y)
    done()
    assert not bool(y[:-tail].any())
    ref, mag = R.product(x[-tail:], w)
    if op == "gated":
        off = (K + 2) * 2.0 ** -23 * mag
        near(y[-tail:], *check_gated(y, ref[:, :N // 2], ref[:, N // 2:], off[:, :N // 2], off[:, N // 2:], "silu"))
    else:
        near(y[-tail:], ref, (K + 2) * 2.0 ** -23 * mag + half_step(y, ref))


# ------------------------------------------------------------------ refusals

INV, UNS = F.FLINT_MOE_ERR_INVALID_ARG, F.FLINT_MOE_ERR_UNSUPPORTED
no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="passes fake device addresses")


def addr(i):
    return 0x7F0000000000 + (i << 36)  # checked by the host code, never read


WIDE = 1 << 17
SHAPE_INVALID = (dict(M=0), dict(N=0), dict(K=0), dict(E=0), dict(off=None), dict(M=-1), dict(off=addr(9) + 4))
SHAPE_UNSUPPORTED = (dict(K=520), dict(E=1025), dict(K=WIDE + 16), dict(M=(1 << 24) + 1))


@no_gpu_only
def test_linear_refusals():
    lib = F.load_library()

    def call(x=addr(0), M=16, w=addr(1), E=4, off=addr(9), N=256, K=512, y=addr(2), kind=0):
        return lib.flint_moe_linear(x, M, w, E, off, N, K, y, kind, None)

    for kw in (*SHAPE_INVALID, dict(x=None), dict(w=None), dict(y=None), dict(x=addr(0) + 8), dict(w=addr(1) + 2),
               dict(y=addr(2) + 4), dict(y=addr(0) + 512), dict(y=addr(1) + 4096), dict(y=addr(9))):
        assert call(**kw) == INV, kw
    for kw in (*SHAPE_UNSUPPORTED, dict(N=252), dict(N=WIDE + 8), dict(kind=2), dict(kind=-1)):
        assert call(**kw) == UNS, kw


@no_gpu_only
def test_gated_linear_refusals():
    lib = F.load_library()

    def call(x=addr(0), M=16, w=addr(1), E=4, off=addr(9), N=256, K=512, act=1, h=addr(2), gu=addr(3)):
        return lib.flint_moe_gated_linear(x, M, w, E, off, N, K, act, h, gu, None)

    for kw in (*SHAPE_INVALID, dict(x=None), dict(w=None), dict(h=None), dict(gu=addr(3) + 8), dict(gu=addr(2)),
               dict(h=addr(0)), dict(gu=addr(1) + 64), dict(h=addr(9)), dict(N=-16)):
        assert call(**kw) == INV, kw
    for kw in (*SHAPE_UNSUPPORTED, dict(N=264), dict(N=WIDE // 2 + 16), dict(N=1 << 30), dict(act=0), dict(act=3)):
        assert call(**kw) == UNS, kw


@no_gpu_only
def test_backward_refusals():
    lib = F.load_library()

    def call(dy=addr(0), x=addr(1), M=16, w=addr(2), E=4, off=addr(9), N=256, K=512, dx=addr(3), dw=addr(4), kind=0):
        return lib.flint_moe_linear_backward(dy, x, M, w, E, off, N, K, dx, dw, kind, None)

    for kw in (*SHAPE_INVALID, dict(dy=None), dict(x=None), dict(w=None), dict(dx=None, dw=None), dict(dx=addr(3) + 8),
               dict(dw=addr(4) + 8), dict(dx=addr(4)), dict(dx=addr(0)), dict(dw=addr(2)), dict(dw=addr(1) + 512)):
        assert call(**kw) == INV, kw
    for kw in (*SHAPE_UNSUPPORTED, dict(N=252), dict(kind=2)):
        assert call(**kw) == UNS, kw

    def gated(dh=addr(0), gu=addr(1), x=addr(2), M=16, w=addr(3), E=4, off=addr(9), N=256, K=512, act=1, dgu=addr(4),
              dx=addr(5), dw=addr(6), kind=0):
        return lib.flint_moe_gated_linear_backward(dh, gu, x, M, w, E, off, N, K, act, dgu, dx, dw, kind, None)

    for kw in (*SHAPE_INVALID, dict(dh=None), dict(gu=None), dict(x=None), dict(w=None), dict(dgu=None),
               dict(dgu=addr(1)), dict(dx=addr(4) + 64), dict(dw=addr(5)), dict(dx=addr(2)), dict(dgu=addr(0) + 16)):
        assert gated(**kw) == INV, kw
    for kw in (*SHAPE_UNSUPPORTED, dict(N=264), dict(kind=2), dict(act=0), dict(act=-1)):
        assert gated(**kw) == UNS, kw


@no_gpu_only
def test_integer_refusals():
    lib = F.load_library()

    def call(a=addr(0), sa=addr(1), M=16, b=addr(2), sb=addr(3), E=4, off=addr(9), N=256, K=512, act=0, y=addr(4), kind=0):
        return lib.flint_moe_integer_gemm(a, sa, M, b, sb, E, off, N, K, act, y, kind, None)

    for kw in (*SHAPE_INVALID, dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(y=None),
               dict(sa=addr(1) + 4), dict(y=addr(0) + 512), dict(y=addr(1)), dict(y=addr(2) + 16), dict(y=addr(3))):
        assert call(**kw) == INV, kw
    for kw in (*SHAPE_UNSUPPORTED, dict(N=252), dict(N=264, act=1), dict(K=WIDE), dict(act=3), dict(kind=2)):
        assert call(**kw) == UNS, kw

    def rows(x=addr(0), kind=0, stride=2048, rows=8, K=2048, pos=None, k=0, places=8, q=addr(1), s=addr(2)):
        return lib.flint_moe_integer_quantize_rows(x, kind, stride, rows, K, pos, k, places, q, s, None)

    for kw in (dict(rows=0), dict(K=0), dict(places=0), dict(places=9), dict(stride=2032), dict(pos=addr(3)),
               dict(x=None), dict(q=None), dict(s=None), dict(x=addr(0) + 8), dict(q=addr(0) + 64), dict(s=addr(1) + 2048),
               dict(pos=addr(2), k=6, places=48)):
        assert rows(**kw) == INV, kw
    for kw in (dict(kind=2), dict(K=2040), dict(stride=2052), dict(K=1 << 18, stride=1 << 18),
               dict(pos=addr(3), k=17, places=8 * 17), dict(rows=(1 << 24) + 1, places=(1 << 24) + 1)):
        assert rows(**kw) == UNS, kw


def test_binding_refuses_what_it_can_see():
    z, bf, i8 = torch.zeros, torch.bfloat16, torch.int8
    x, w, y = z(4, 64, dtype=bf), z(2, 32, 64, dtype=bf), z(4, 32, dtype=bf)
    with pytest.raises(TypeError, match="x: expected"):
        F.linear(None, w, y)
    with pytest.raises(ValueError, match=r"w: expected \[experts\]"):
        F.linear(x, w[0], y)
    with pytest.raises(ValueError, match="w: dtype"):
        F.linear(x, w.float(), y)
    with pytest.raises(ValueError, match="w: must be contiguous"):
        F.linear(x, w.transpose(1, 2), y)
    with pytest.raises(ValueError, match="w: must be on the current CUDA device"):
        F.linear(x, w, y)
    with pytest.raises(ValueError, match=r"w: expected \[experts\]\[2I\]"):
        F.gated_linear(x, z(1, 33, 64, dtype=bf), y)
    with pytest.raises(TypeError, match="w: expected"):
        F.linear_backward(y, x, None, dx=x)
    with pytest.raises(TypeError, match="dh: expected"):
        F.gated_linear_backward(None, y, x, w, y)
    with pytest.raises(ValueError, match="b: dtype"):
        F.integer_gemm(z(4, 64, dtype=i8), z(4), w, z(2, 32), y)
    with pytest.raises(ValueError, match="x: shape"):
        F.integer_quantize_rows(x, z(4, 32, dtype=i8), z(4))
    with pytest.raises(ValueError, match="x: dtype"):
        F.integer_quantize_rows(x.half(), z(4, 64, dtype=i8), z(4))


def test_binding_refuses_counts_beyond_31_bits():
    n = (1 << 32) + 4

    def m(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")

    with pytest.raises(ValueError, match="x: .*31 bits"):
        F.linear(m(n, 64), m(1, 32, 64), m(n, 32))
    with pytest.raises(ValueError, match="w: .*31 bits"):
        F.gated_linear(m(4, 64), m(n, 32, 64), m(4, 16))
    with pytest.raises(ValueError, match="dy: .*31 bits"):
        F.linear_backward(m(n, 32), m(n, 64), m(1, 32, 64), dx=m(n, 64))
    with pytest.raises(ValueError, match="q: .*31 bits"):
        F.integer_quantize_rows(m(4, 64), m(n, 64, dtype=torch.int8), m(n, dtype=torch.float32))
    with pytest.raises(ValueError, match="a: .*31 bits"):
        F.integer_gemm(m(n, 64, dtype=torch.int8), None, None, None, None)


@gpu
def test_binding_refuses_on_the_gpu():
    d, bf = dev(), torch.bfloat16
    x, w, y = rand(1, 4, 64), rand(2, 2, 32, 64), torch.empty(4, 32, dtype=bf, device=d)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=d)
    for f in (lambda: F.linear(x, w, y[:3], offsets=off), lambda: F.linear(x, w, y.half(), offsets=off),
              lambda: F.linear(x, w, y, offsets=off[:2]), lambda: F.linear(x, w, y, offsets=off.long()),
              lambda: F.linear(x[:, ::2], w, y, offsets=off), lambda: F.gated_linear(x, w, y, offsets=off),
              lambda: F.gated_linear(x, w, y[:, :16].contiguous(), gu=y[:3], offsets=off),
              lambda: F.linear_backward(y, x, w, dw=w.half(), offsets=off)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: F.linear(x, w, y), lambda: F.linear_backward(y, x, w, offsets=off),
              lambda: F.gated_linear(x, w, y[:, :16].contiguous(), offsets=off, act=F.ACT_NONE),
              lambda: F.linear_backward(y, x, w, dx=x, offsets=off)):
        with pytest.raises(F.FlintMoeError):
            f()
    F.linear(x, w, y, offsets=off)
    done()
