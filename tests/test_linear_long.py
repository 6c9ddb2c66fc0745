"""Products that last longer than one bounded wait of a kernel may."""

import pytest
import torch

import linear_reference as R
from moe_decode_router_gb300 import flint_moe as F
from test_linear_ops import BF16, dev, done, near

gpu = pytest.mark.gpu


@gpu
def test_gradients_behind_a_second_of_others():
    """dx alone takes some 2.9e9 cycles here, a wait 2e9 at most, and the last step of every unit of
    dw, behind dx, holds rows that do not exist (100,001 is no multiple of 16)."""
    d, (M, N, K) = dev(), (100001, 131064, 131056)
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("needs 200 GB of device memory")
    g = torch.Generator(device=d)
    g.manual_seed(1)
    dy, x, w = (torch.empty(s, dtype=torch.bfloat16, device=d).normal_(generator=g) for s in ((M, N), (M, K), (1, N, K)))
    dx, dw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    F.linear_backward(dy, x, w, dx=dx, dw=dw)
    done()
    # rows of dx and of dw, of first, middle and last tiles, in parts of the contracted dimension
    for got, length, a, b in ((dx, M, dy, w[0]), (dw[0], N, dy.T, x)):
        rows = torch.tensor([0, 255, 256, length // 2, length - 2, length - 1], device=d)
        want = torch.zeros(len(rows), K, dtype=torch.float64, device=d)
        mag = want.clone()
        for at in torch.arange(b.shape[0], device=d).split(8192):
            part, m = R.product(a[rows][:, at], b[at].T[None])
            want += part
            mag += m
        near(got[rows], want, (b.shape[0] + 2) * 2.0 ** -23 * mag + BF16 * want.abs())
        assert not bool((got == 7.0).all(1).any())  # no row was left as it was
    del dy, x, w, dx, dw
    torch.cuda.empty_cache()
