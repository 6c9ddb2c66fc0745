"""The linear, gated and integer products, their gradients and the quantisation of rows to
8-bit integers in 64 bits, written from their definitions."""

import math

import torch

FLOOR = 2.0 ** -96


def by_expert(offsets, M, E):
    edge = [0, M] if offsets is None else [int(o) for o in offsets]
    return [slice(edge[e], edge[e + 1]) for e in range(E)]


def product(x, w, offsets=None):
    """(y, sum of the magnitudes of its terms), both [M][N]; rows of no expert are NaN."""
    x, w = x.double(), w.double()
    y = torch.full((x.shape[0], w.shape[1]), math.nan, dtype=torch.float64, device=x.device)
    mag = y.clone()
    for e, at in enumerate(by_expert(offsets, x.shape[0], w.shape[0])):
        y[at] = x[at] @ w[e].T
        mag[at] = x[at].abs() @ w[e].abs().T
    return y, mag


def input_gradient(dy, w, offsets=None):
    return product(dy, w.transpose(1, 2), offsets)


def weight_gradient(dy, x, E, offsets=None):
    dy, x = dy.double(), x.double()
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64, device=x.device)
    mag = dw.clone()
    for e, at in enumerate(by_expert(offsets, x.shape[0], E)):
        dw[e] = dy[at].T @ x[at]
        mag[e] = dy[at].abs().T @ x[at].abs()
    return dw, mag


def inner(g, act):
    """v of g * sigmoid(v), and dv/dg."""
    if act == "silu":
        return g, torch.ones_like(g)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (g + 0.044715 * g ** 3), c * (1 + 0.134145 * g ** 2)


def activation(g, act):
    return g * torch.sigmoid(inner(g, act)[0])


def slope(g, act):
    """The derivative of the activation, and the sum of its terms' magnitudes."""
    v, dv = inner(g, act)
    p, q = torch.sigmoid(v), torch.sigmoid(-v)
    bend = g * p * q * dv
    return p + bend, p + bend.abs()


def integer_rows(x):
    """codes [rows][K] and fp32 scales [rows] of finite rows."""
    top = x.double().abs().amax(1).clamp(min=FLOOR)
    scale = (top * torch.tensor(1 / 127, dtype=torch.float32).double()).float()  # a product of two fp32 is exact in 64 bits
    z = x.double() / scale.double()[:, None]
    q = torch.floor(z)
    rest = z - q
    q += ((rest > 0.5) | ((rest == 0.5) & (q % 2 != 0))).double()
    return q, scale


def integer_sums(a, b, offsets=None):
    """Exact sums [M][N]: 64-bit floats hold them all (at most 2^31)."""
    return product(a, b, offsets)[0]
