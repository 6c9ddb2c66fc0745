"""The largest counts that the linear, gated and integer products take, one at a time, with the
tolerances of test_linear_ops.py."""

import pytest
import torch

import linear_reference as R
from moe_decode_router_gb300 import flint_moe as F
from test_linear_ops import check_gate_backward, check_gated, dev, done, half_step, near

gpu = pytest.mark.gpu
WIDE, ROWS = 1 << 17, 1 << 24
BF = torch.bfloat16


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    return torch.empty(shape, dtype=BF, device=dev()).normal_(generator=g).mul_(scale)


def codes(seed, *shape):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    return torch.randint(-128, 128, shape, dtype=torch.int8, generator=g, device=dev())


def empty(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device=dev())


def by_parts(n, parts=16):
    return torch.arange(n, device=dev()).chunk(parts)


def grouped(M, cuts):
    """Offsets of len(cuts) + 1 groups, or None and one."""
    return (None, [slice(0, M)]) if cuts is None else (
        torch.tensor([0, *cuts, M], dtype=torch.int32, device=dev()), [slice(a, b) for a, b in zip([0, *cuts], [*cuts, M])])


# many rows of little, dense and by expert; and a matrix that is as wide, or as deep, as may be
MANY = [(ROWS, 32, 16, None), (ROWS - 7, 32, 16, (1, ROWS // 3, ROWS // 3))]
WIDEST = [(3, WIDE, 16, None), (200, WIDE, 32, None), (70, WIDE, 16, (3, 40)), (3, 32, WIDE - 16, None), (200, 32, WIDE - 16, None),
          (90, 32, WIDE - 16, (30, 30))]


@gpu
@pytest.mark.parametrize("M,N,K,cuts", MANY + WIDEST)
def test_forward(M, N, K, cuts):
    offsets, at = grouped(M, cuts)
    E, I = len(at), N // 2
    x, w = normal(1, M, K), normal(2, E, N, K, scale=2 * K ** -0.5)
    y, h, gu = empty(M, N), empty(M, I), empty(M, N)
    F.linear(x, w, y, offsets=offsets)
    F.gated_linear(x, w, h, gu=gu, offsets=offsets)
    done()
    for e, rows in enumerate(at):
        for part in by_parts(rows.stop - rows.start) if rows.stop - rows.start > 1000 else [torch.arange(rows.stop - rows.start, device=dev())]:
            r = part + rows.start
            s, mag = R.product(x[r], w[e:e + 1])
            off = (K + 2) * 2.0 ** -23 * mag
            near(y[r], s, off + half_step(y, s.abs() + off))
            near(gu[r], s, off + half_step(gu, s.abs() + off))
            near(h[r], *check_gated(h, s[:, :I], s[:, I:], off[:, :I], off[:, I:], "silu"))


@gpu
@pytest.mark.parametrize("M,N,K,cuts", MANY + WIDEST)
def test_integers(M, N, K, cuts):
    offsets, at = grouped(M, cuts)
    E = len(at)
    a, b = codes(1, M, K), codes(2, E, N, K)
    sa, sb = torch.rand(M, device=dev()) + 0.1, torch.rand(E, N, device=dev()) + 0.1
    y = empty(M, N, dtype=torch.float32)
    F.integer_gemm(a, sa, b, sb, y, offsets=offsets)
    done()
    for e, rows in enumerate(at):
        for part in by_parts(rows.stop - rows.start) if rows.stop - rows.start > 1000 else [torch.arange(rows.stop - rows.start, device=dev())]:
            r = part + rows.start
            v = R.integer_sums(a[r], b[e:e + 1]) * (sa[r].double()[:, None] * sb[e].double())
            near(y[r], v, 2.0 ** -22 * v.abs())


@gpu
@pytest.mark.parametrize("M,N,K,cuts", [(ROWS, 32, 16, None), (200, WIDE, 16, None), (70, WIDE, 16, (3, 40)), (200, 32, WIDE, None),
                                        (90, 32, WIDE, (30, 30))])
def test_gradients(M, N, K, cuts):
    offsets, at = grouped(M, cuts)
    E, I = len(at), N // 2
    dh, gu, x, w = normal(1, M, I), normal(2, M, N), normal(3, M, K), normal(4, E, N, K, scale=0.1)
    dgu, dx, dw = empty(M, N), empty(M, K), empty(E, N, K, dtype=torch.float32)
    F.gated_linear_backward(dh, gu, x, w, dgu, dx=dx, dw=dw, offsets=offsets)
    done()
    for e, rows in enumerate(at):
        n = rows.stop - rows.start
        want, mag = torch.zeros(N, K, dtype=torch.float64, device=dev()), torch.zeros(N, K, dtype=torch.float64, device=dev())
        for part in by_parts(n) if n > 1000 else [torch.arange(n, device=dev())]:
            r = part + rows.start
            check_gate_backward(dgu[r], dh[r], gu[r], "silu")
            ref, m = R.input_gradient(dgu[r], w[e:e + 1])
            near(dx[r], ref, (N + 2) * 2.0 ** -23 * m + half_step(dx, ref))
            d, m = R.weight_gradient(dgu[r], x[r], 1)
            want += d[0]
            mag += m[0]
        near(dw[e], want, (n + 2) * 2.0 ** -23 * mag)


@gpu
@pytest.mark.parametrize("rows,K,k", [(ROWS, 16, 0), (ROWS // 16, 16, 16), (3, WIDE, 2)])
def test_rows_to_integers(rows, K, k):
    places = rows * max(1, k)
    x, q, s = normal(1, rows, K), torch.empty(places, K, dtype=torch.int8, device=dev()), torch.empty(places, device=dev())
    pos = torch.randperm(places, device=dev()).to(torch.int32).reshape(rows, k) if k else None
    F.integer_quantize_rows(x, q, s, pos=pos)
    done()
    for r in by_parts(rows) if rows > 1000 else [torch.arange(rows, device=dev())]:
        want, scale = R.integer_rows(x[r])
        for j in range(max(1, k)):
            p = r if pos is None else pos[r, j].long()
            assert torch.equal(s[p], scale) and torch.equal(q[p].double(), want)
