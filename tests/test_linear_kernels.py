"""Every kernel and plan of the linear, gated and integer products: which one a product takes,
and each of them against the 64-bit references, with the tolerances of test_linear_ops.py."""

import math
import pathlib
import subprocess
import sys

import pytest
import torch

import linear_reference as R
from moe_decode_router_gb300 import flint_moe as F
from test_linear_ops import check_gated, codes, dev, done, framed, gen, groups, half_step, near, rand, unframed

gpu = pytest.mark.gpu
FORWARD, INTEGERS, DX, DW, BOTH = range(5)


def plan(what, M, N, K, sms=None):
    """0 for the few-row kernel, else (pairs that share a contraction, tile of rows, tile of dw)."""
    if sms is None:
        sms = torch.cuda.get_device_properties(0).multi_processor_count
    v = F.load_library().flint_linear_plan(what, M, N, K, sms)
    return (v // 1000000, v // 1000 % 1000, v % 1000) if v else 0


def test_every_plan_is_chosen():
    """On 152 SMs, by the cases below and the measured crossings."""
    assert plan(FORWARD, 8, 8192, 2048, 152) == 0 and plan(INTEGERS, 8, 64, 16, 152) == 0
    assert plan(FORWARD, 24, 2048, 2048, 152) == 0 and plan(FORWARD, 64, 2048, 2048, 152)[0] == 4
    assert plan(INTEGERS, 64, 2048, 2048, 152) == 0 and plan(INTEGERS, 128, 2048, 2048, 152)[0] == 4
    assert plan(FORWARD, 64, 4096, 4096, 152)[0] == 2 and plan(INTEGERS, 96, 4096, 4096, 152)[0] == 2
    assert plan(FORWARD, 64, 8192, 2048, 152)[0] == 1
    assert plan(FORWARD, 8191, 4096, 4096, 152)[:2] == (1, 256) and plan(INTEGERS, 8191, 4096, 4096, 152)[:2] == (1, 256)
    assert plan(DX, 16, 8192, 2048, 152)[0] == 4 and plan(DX, 200, 4096, 4096, 152)[0] == 2
    assert plan(DW, 8192, 512, 512, 152)[0] == 4 and plan(DW, 4096, 1024, 1024, 152)[0] == 2
    assert plan(DW, 4096, 2048, 512, 152)[0] == 2 and plan(DW, 4096, 4096, 4096, 152)[0] == 1
    assert plan(BOTH, 4095, 2048, 1408, 152)[0] == 1


def twice(call, outs):
    """Runs a call two times on outputs of its own and asserts the same bits; returns the first."""
    got = []
    for _ in range(2):
        fresh = [framed(s, t) for s, t in outs]
        call(*(f[1] for f in fresh))
        done()
        for whole, _, before in fresh:
            unframed(whole, before)
        got.append([f[1] for f in fresh])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    return got[0]


# what, rows, N, K, pairs that share a contraction
SHARED = [(FORWARD, 256, 1032, 1552, 4), (FORWARD, 70, 2048, 2064, 4), (FORWARD, 300, 416, 4112, 4), (FORWARD, 129, 4104, 4096, 2),
          (FORWARD, 700, 1032, 2064, 2), (FORWARD, 256, 1032, 1040, 1), (FORWARD, 90, 8192, 2064, 1), (FORWARD, 1000, 1056, 272, 1)]


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("what,M,N,K,ks", SHARED)
def test_dense_forward(out, what, M, N, K, ks):
    assert plan(what, M, N, K)[0] == ks
    x, w = rand(M + N, M, K), rand(K, 1, N, K, scale=0.1)
    y, = twice(lambda y: F.linear(x, w, y), [((M, N), out)])
    ref, mag = R.product(x, w)
    near(y, ref, (K + 2) * 2.0 ** -23 * mag + half_step(y, ref))


@gpu
@pytest.mark.parametrize("what,M,N,K,ks", [(w, M, N // 32 * 32, K, ks) for w, M, N, K, ks in SHARED])
def test_dense_gated(what, M, N, K, ks):
    assert plan(what, M, N, K)[0] == ks
    x, w, I = rand(M + N, M, K), rand(K, 1, N, K, scale=2 / math.sqrt(K)), N // 2
    h, gu = twice(lambda h, gu: F.gated_linear(x, w, h, gu=gu, act=F.ACT_GELU), [((M, I), torch.bfloat16), ((M, N), torch.bfloat16)])
    sums, mag = R.product(x, w)
    off = (K + 2) * 2.0 ** -23 * mag
    near(h, *check_gated(h, sums[:, :I], sums[:, I:], off[:, :I], off[:, I:], "gelu"))
    near(gu, sums, off + half_step(gu, sums.abs() + off))


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("M,N,K,ks", [(300, 1024, 1552, 4), (200, 1056, 4112, 4), (130, 4096, 4096, 2), (800, 1056, 2576, 2),
                                      (100, 8192, 2064, 1), (1000, 1056, 272, 1)])
def test_dense_integers(out, act, M, N, K, ks):
    assert plan(INTEGERS, M, N, K)[0] == ks
    a, b = codes(M + N, M, K), codes(K, 1, N, K)
    sa = torch.exp(torch.randn(M, generator=gen(1))).to(dev()) / 128
    sb = torch.exp(torch.randn(1, N, generator=gen(2))).to(dev()) / (64 * math.sqrt(K))
    width = N if act == "none" else N // 2
    y, = twice(lambda y: F.integer_gemm(a, sa, b, sb, y, act=F.ACT_NONE if act == "none" else F.ACT_SILU), [((M, width), out)])
    v = R.integer_sums(a, b) * (sa.double()[:, None] * sb[0].double())
    off = 2.0 ** -22 * v.abs()
    if act == "none":
        near(y, v, off + half_step(y, v.abs() + off))
    else:
        near(y, *check_gated(y, v[:, :width], v[:, width:], off[:, :width], off[:, width:], act))


@gpu
@pytest.mark.parametrize("M,N,K,ks", [(300, 1024, 8208, 4), (800, 1056, 4112, 2), (2100, 2048, 4112, 1)])
def test_integer_sums_small_and_large(M, N, K, ks):
    """Sums that stay below 2^21, pass it in the first or in a later segment, or return, side by side."""
    d = dev()
    assert plan(INTEGERS, M, N, K)[0] == ks
    level = torch.tensor([3, 18, -18, 40, 127, -128, 18], dtype=torch.int8)
    a = level[torch.arange(M) // 64 % 7][:, None].repeat(1, K)
    a[64 * 6:64 * 7, K // 2:] *= -1
    a[::5] = torch.randint(-128, 128, (len(a[::5]), K), generator=gen(M), dtype=torch.int8)
    b = torch.randint(0, 128, (1, N, K), generator=gen(N), dtype=torch.int8)
    b[0, ::3] = torch.randint(-128, 128, (len(b[0, ::3]), K), generator=gen(K), dtype=torch.int8)
    b[0, 40:44] = -128
    a, b = a.to(d), b.to(d)
    y, ones = torch.empty(M, N, device=d), torch.ones(max(M, N), device=d)
    F.integer_gemm(a, ones[:M], b, ones[None, :N].contiguous(), y)
    done()
    assert torch.equal(y, R.integer_sums(a, b).float())


@gpu
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("what,M,N,K,ks", [
    (DX, 30, 4096, 1040, 4), (DX, 200, 4104, 2048, 4), (DX, 200, 4104, 4112, 2), (DX, 700, 520, 2064, 1),
    (DW, 4001, 520, 528, 4), (DW, 2047, 1024, 1040, 2), (DW, 4001, 2056, 528, 2), (DW, 1500, 2056, 2064, 1),
    (BOTH, 500, 1032, 528, None), (BOTH, 40, 4104, 1040, None), (BOTH, 3001, 1416, 1040, None)])
def test_dense_gradients(out, what, M, N, K, ks):
    if ks is not None:
        assert plan(what, M, N, K)[0] == ks
    dy, x, w = rand(M, M, N), rand(M + N, M, K), rand(K, 1, N, K, scale=0.1)
    dx, dw = twice(lambda dx, dw: F.linear_backward(dy, x, w, dx=None if what == DW else dx, dw=None if what == DX else dw),
                   [((M, K), torch.bfloat16), ((1, N, K), out)])
    if what != DW:
        ref, mag = R.input_gradient(dy, w)
        near(dx, ref, (N + 2) * 2.0 ** -23 * mag + half_step(dx, ref))
    if what != DX:
        ref, mag = R.weight_gradient(dy, x, 1)
        near(dw, ref, (M + 2) * 2.0 ** -23 * mag + half_step(dw, ref))


@gpu
@pytest.mark.parametrize("E,high,N,K", [(70, 9, 544, 272), (70, 90, 1056, 528), (70, 600, 544, 1040), (1024, 24, 96, 80)])
def test_many_groups(E, high, N, K):
    """Groups of 0 to `high` rows: several units a pair, every length of a last step, and the
    few-row kernel by experts."""
    counts = torch.randint(0, high + 1, (E,), generator=gen(high)).tolist()
    counts[3] = counts[E - 1] = 0
    M, offsets, I = sum(counts), groups(counts), N // 2
    x, w, dy, dh = rand(1, M, K), rand(2, E, N, K, scale=2 / math.sqrt(K)), rand(3, M, N), rand(4, M, I)
    bf = torch.bfloat16
    y, h, gu, dx, dw = twice(lambda y, h, gu, dx, dw: (
        F.linear(x, w, y, offsets=offsets), F.gated_linear(x, w, h, gu=gu, offsets=offsets),
        F.linear_backward(dy, x, w, dx=dx, dw=dw, offsets=offsets)),
        [((M, N), bf), ((M, I), bf), ((M, N), bf), ((M, K), bf), ((E, N, K), bf)])
    sums, mag = R.product(x, w, offsets)
    off = (K + 2) * 2.0 ** -23 * mag
    near(y, sums, off + half_step(y, sums.abs() + off))
    near(gu, sums, off + half_step(gu, sums.abs() + off))
    near(h, *check_gated(h, sums[:, :I], sums[:, I:], off[:, :I], off[:, I:], "silu"))
    ref, mag = R.input_gradient(dy, w, offsets)
    near(dx, ref, (N + 2) * 2.0 ** -23 * mag + half_step(dx, ref))
    ref, mag = R.weight_gradient(dy, x, E, offsets)
    near(dw, ref, (high + 2) * 2.0 ** -23 * mag + half_step(dw, ref))
    a, b = codes(5, M, K), codes(6, E, N, K)
    z, = twice(lambda z: F.integer_gemm(a, torch.ones(M, device=dev()), b, torch.ones(E, N, device=dev()), z, offsets=offsets),
               [((M, N), torch.float32)])
    assert torch.equal(z, R.integer_sums(a, b, offsets).float())


@gpu
def test_captured_shared_contractions_at_once():
    """Captured and replayed on two streams at a time, each with its own inputs."""
    M, N, K = 100, 2048, 2064
    assert plan(FORWARD, M, N, K)[0] == 4
    ins = [(rand(i, M, K), rand(i + 9, 1, N, K, scale=0.1), rand(i + 5, M, N)) for i in range(2)]
    outs = [[torch.zeros(M, N, device=dev()), torch.zeros(M, K, dtype=torch.bfloat16, device=dev()), torch.zeros(1, N, K, device=dev())]
            for _ in ins]

    def run(i, o):
        F.linear(i[0], i[1], o[0])
        F.linear_backward(i[2], i[0], i[1], dx=o[1], dw=o[2])

    for i, o in zip(ins, outs):
        run(i, o)
    done()
    want = [[t.clone() for t in o] for o in outs]
    streams, graphs = [torch.cuda.Stream() for _ in ins], []
    for st, i, o in zip(streams, ins, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(6):
                run(i, o)
        graphs.append(g)
        for t in o:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
    done()
    for o, w in zip(outs, want):
        for a, b in zip(o, w):
            assert torch.equal(a, b)


FIRST_CALL_CAPTURED = """
import torch
from moe_decode_router_gb300 import flint_moe as F
d = torch.device("cuda:0")
bf = dict(device=d, dtype=torch.bfloat16)
F.load_library()
ids = torch.tensor([[0], [1], [1], [0]], dtype=torch.int32, device=d)
offsets, order, pos = (torch.empty(s, dtype=torch.int32, device=d) for s in (3, 4, (4, 1)))
F.group_pairs(ids, offsets, order, pos)  # sets up the library
x, w, dy = torch.randn(300, 256, **bf), torch.randn(1, 512, 256, **bf), torch.randn(300, 512, **bf)
outs = [torch.zeros(300, 512, **bf), torch.zeros(300, 256, **bf), torch.zeros(1, 512, 256, **bf),
        torch.zeros(300, 256, **bf), torch.zeros(2, 512, **bf), torch.zeros(300, 256, dtype=torch.int8, device=d),
        torch.zeros(300, device=d)]


def run():
    F.linear(x, w, outs[0])
    F.linear_backward(dy, x, w, outs[1], outs[2])
    F.gated_linear(x, w, outs[3])
    F.linear(x[:2], w, outs[4])
    F.integer_quantize_rows(x, outs[5], outs[6])


g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
assert not any(bool(o.any()) for o in outs)
g.replay()
torch.cuda.synchronize()
got = [o.clone() for o in outs]
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) and bool(a.any()) for a, b in zip(got, outs)) and F.device_error() == 0
"""


@gpu
def test_first_products_may_be_captured():
    """Once any call has set up the library, the first call of every product may be on a capturing stream."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], capture_output=True, text=True, timeout=300,
                       cwd=pathlib.Path(__file__).resolve().parents[1])
    assert r.returncode == 0, r.stderr
