"""Cases, inputs and plain forms of the operators of an expert's feed-forward block beside the FP8 ones: its gated projections
and its linear product in bf16, forward and backward, dense or grouped by expert, and for serving the same products in 8-bit
integers with one scale for each row (token) and each output (channel), with the quantisation of rows that goes before them.

A pair is one (token, choice) entry of the routing; "expert order" is all pairs sorted by expert.  offsets [E + 1] give every
expert its rows.  A gated matrix is [E][2 I][K]: rows 0 .. I - 1 the gate's, I .. 2 I - 1 the other factor's.
"""

import math

import torch

own = False

DEV = "cuda"
FLOOR = 2.0 ** -96  # smallest row maximum that a scale is made for
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases


def listed():
    return [
        # A 64-request decode step: each token's row, quantised to the places of its six experts.
        dict(name="quantise decode", op="quantise", rows=64, K=2048, top_k=6, E=256, dtype="bf16", pad=0),
        # The same for a prompt.
        dict(name="quantise prompt", op="quantise", rows=8191, K=2048, top_k=6, E=256, dtype="bf16", pad=0),
        # 64 requests through their experts' gate and up projections in 8 bits: some 200 experts with a row or two each.
        dict(name="int8 experts decode", op="int8", M=64, N=1024, K=2048, E=256, top_k=6, act="silu", out="bf16"),
        # A prompt (an odd number of rows) through a dense 8-bit projection: bound by the tensor cores.
        dict(name="int8 prompt", op="int8", M=8191, N=4096, K=4096, E=0, top_k=0, act="none", out="fp32"),
        # 8 requests through the shared expert's gate and up projections: the smallest call, all latency.
        dict(name="gated decode", op="gated", M=8, I=512, K=2048, E=0, top_k=0, act="silu", keep=False),
        # A prompt or training batch through a dense model's gated projections, which are kept for the gradient.
        dict(name="gated batch", op="gated", M=8191, I=5632, K=2048, E=0, top_k=0, act="gelu", keep=True),
        # Training the experts: gradients of the gated projections of 49,152 pairs.
        dict(name="gated backward, experts", op="gated backward", M=8192, I=512, K=2048, E=256, top_k=6, act="silu"),
        # A smaller dense block's, at an odd number of rows.
        dict(name="gated backward, dense", op="gated backward", M=2047, I=1408, K=1024, E=0, top_k=0, act="gelu"),
        # One token through a dense projection: bound by the weights' bytes.
        dict(name="linear decode", op="linear", M=1, N=8192, K=2048, E=0, top_k=0, out="bf16"),
        # A prompt through its experts' down projections: ragged groups of about 192 rows.
        dict(name="linear prompt, experts", op="linear", M=8192, N=2048, K=512, E=256, top_k=6, out="bf16"),
        # Training the experts: gradients of those.
        dict(name="linear backward, experts", op="linear backward", M=8192, N=2048, K=512, E=256, top_k=6, out="bf16"),
        # A dense down projection's, weight gradients in fp32 for a sum over several batches.
        dict(name="linear backward, dense", op="linear backward", M=4095, N=2048, K=1408, E=0, top_k=0, out="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantise", "int8", "int8", "gated", "gated", "gated backward", "linear", "linear backward"])
    if op == "quantise":
        return dict(op=op, rows=_log(rng, 1, 8192), K=16 * rng.randint(8, 128), top_k=rng.choice([0, 2, 6]),
                    E=rng.randint(8, 256), dtype=rng.choice(["bf16", "fp32"]), pad=rng.choice([0, 8]))
    back = op.endswith("backward")
    dense = rng.random() < 0.5
    E = 0 if dense else _log(rng, 4, 256)
    top_k = 0 if dense else rng.randint(1, min(6, E))
    M = _log(rng, 1, 4096 if back or not dense else 8191)
    # a gated matrix has 2 I rows: as many as another's N
    I, K = 16 * rng.randint(4, 110 if dense else 32), 16 * rng.randint(8, 250 if dense else 128)
    N = 8 * rng.randint(16, 440 if dense else 128)
    c = dict(op=op, M=M, K=K, E=E, top_k=top_k)
    if op == "int8":
        act = rng.choice(["none", "silu", "gelu"])
        return dict(c, N=N if act == "none" else 2 * I, act=act, out=rng.choice(["bf16", "fp32"]))
    if op == "gated":
        return dict(c, I=I, act=rng.choice(["silu", "gelu"]), keep=rng.random() < 0.5)
    if op == "gated backward":
        return dict(c, I=I, act=rng.choice(["silu", "gelu"]))
    return dict(c, N=N, out=rng.choice(["bf16", "fp32"]))


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _choices(g, T, E, top_k):
    """Expert ids [T][top_k] of tokens whose router prefers some experts a little."""
    z = torch.randn(T, E, generator=g, device=DEV) + 0.3 * torch.randn(E, generator=g, device=DEV)
    return torch.topk(z, top_k, dim=1).indices.to(torch.int32)


def _places(ids, E):
    """offsets [E + 1] and pos [T][top_k] of expert order."""
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=DEV)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0).to(torch.int32)
    return offsets, pos.to(torch.int32).reshape(ids.shape)


def _randn(g, shape, scale):
    """bf16 normal values, a matrix at a time."""
    t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for e in range(shape[0]) if len(shape) == 3 else [slice(None)]:
        t[e] = scale * torch.randn(t[e].shape, generator=g, device=DEV)
    return t


def _codes(g, shape):
    t = torch.empty(shape, dtype=torch.int8, device=DEV)
    for e in range(shape[0]) if len(shape) == 3 else [slice(None)]:
        t[e] = (32.0 * torch.randn(t[e].shape, generator=g, device=DEV)).round_().clamp_(-127, 127).to(torch.int8)
    return t


def prepare(case, seed):
    g, op, K = _gen(seed), case["op"], case["K"]
    s = dict(case=case)
    if op == "quantise":
        R, k = case["rows"], case["top_k"]
        x = torch.randn(R, K + case["pad"], generator=g, device=DEV)
        x *= torch.exp(torch.randn(K + case["pad"], generator=g, device=DEV))  # channels of unlike size
        s["x"] = x.to(DTYPES[case["dtype"]])[:, :K]
        s["pos"] = _places(_choices(g, R, case["E"], k), case["E"])[1] if k else None
        s["q"] = torch.empty(R * max(1, k), K, dtype=torch.int8, device=DEV)
        s["scales"] = torch.empty(R * max(1, k), dtype=torch.float32, device=DEV)
        return s
    M, E, k = case["M"], case["E"], case["top_k"]
    G, rows = max(1, E), M * k if E else M
    N = 2 * case["I"] if op.startswith("gated") else case["N"]
    s["offsets"] = None
    if E:
        s["offsets"] = _places(_choices(g, M, E, k), E)[0]
        n = torch.diff(s["offsets"].long())
        live = torch.nonzero(n).reshape(-1)  # the plain form's plan: live experts and their rows, padded to the longest group
        at = torch.arange(int(n.max()), device=DEV)
        s["live"], s["have"] = live, at < n[live, None]
        s["rows"] = torch.where(s["have"], s["offsets"][:-1].long()[live, None] + at, 0)
    if op == "int8":
        s["a"], s["b"] = _codes(g, (rows, K)), _codes(g, (G, N, K))
        s["a_scales"] = 0.02 * torch.exp(0.5 * torch.randn(rows, generator=g, device=DEV))
        s["b_scales"] = 0.05 / math.sqrt(K) * torch.exp(0.5 * torch.randn(G, N, generator=g, device=DEV))
        s["y"] = torch.empty(rows, N if case["act"] == "none" else N // 2, dtype=DTYPES[case["out"]], device=DEV)
        return s
    s["x"], s["w"] = _randn(g, (rows, K), 1.0), _randn(g, (G, N, K), 1.5 / math.sqrt(K))
    if op == "gated":
        s["h"] = torch.empty(rows, N // 2, dtype=torch.bfloat16, device=DEV)
        s["gu"] = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV) if case["keep"] else None
    elif op == "linear":
        s["y"] = torch.empty(rows, N, dtype=DTYPES[case["out"]], device=DEV)
    else:
        s["dx"] = torch.empty(rows, K, dtype=torch.bfloat16, device=DEV)
        s["dw"] = torch.empty(G, N, K, dtype=DTYPES[case.get("out", "bf16")], device=DEV)
        if op == "gated backward":
            s["dh"], s["gu"] = _randn(g, (rows, N // 2), 0.01), _randn(g, (rows, N), 1.5)
            s["dgu"] = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
        else:
            s["dy"] = _randn(g, (rows, N), 0.01)
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def _own(s):
    from moe_decode_router_gb300 import flint_moe as F

    c = s["case"]
    act = {"none": F.ACT_NONE, "silu": F.ACT_SILU, "gelu": F.ACT_GELU}[c.get("act", "none")]
    if c["op"] == "quantise":
        F.integer_quantize_rows(s["x"], s["q"], s["scales"], pos=s["pos"])
        return s["q"], s["scales"]
    if c["op"] == "int8":
        F.integer_gemm(s["a"], s["a_scales"], s["b"], s["b_scales"], s["y"], offsets=s["offsets"], act=act)
        return s["y"]
    if c["op"] == "gated":
        F.gated_linear(s["x"], s["w"], s["h"], gu=s["gu"], offsets=s["offsets"], act=act)
        return (s["h"], s["gu"]) if c["keep"] else s["h"]
    if c["op"] == "linear":
        F.linear(s["x"], s["w"], s["y"], offsets=s["offsets"])
        return s["y"]
    if c["op"] == "linear backward":
        F.linear_backward(s["dy"], s["x"], s["w"], dx=s["dx"], dw=s["dw"], offsets=s["offsets"])
        return s["dx"], s["dw"]
    F.gated_linear_backward(s["dh"], s["gu"], s["x"], s["w"], s["dgu"], dx=s["dx"], dw=s["dw"], offsets=s["offsets"], act=act)
    return s["dgu"], s["dx"], s["dw"]


def _plain_quantise(s):
    x = s["x"].float()
    scale = x.abs().amax(1).clamp(min=FLOOR) / 127
    # the nearest whole number of the exact quotient, ties to even: next to a border 32 bits lose it
    q = torch.round(x.double() / scale.double()[:, None]).to(torch.int8)
    if s["pos"] is None:
        return q, scale
    k, at = s["pos"].shape[1], s["pos"].reshape(-1).long()
    out, sc = torch.empty_like(s["q"]), torch.empty_like(s["scales"])
    out[at] = q.repeat_interleave(k, 0)
    sc[at] = scale.repeat_interleave(k)
    return out, sc


def _times(s, x, w):
    """x [rows][K] times each row's expert's w [experts][N][K], transposed, in fp32."""
    if s["offsets"] is None:
        return torch.matmul(x.float(), w[0].float().T)
    y = torch.bmm(x[s["rows"]].float(), w[s["live"]].float().transpose(1, 2))
    return y[s["have"]]


def _back(s, dy):
    """Gradients of x and w of _times, from dy [rows][N]."""
    x, w = s["x"], s["w"]
    if s["offsets"] is None:
        return torch.matmul(dy, w[0].float()), torch.matmul(dy.T, x.float())[None]
    live, have, rows = s["live"], s["have"], s["rows"]
    d = dy[rows] * have[:, :, None]
    dx = torch.bmm(d, w[live].float())[have]
    dw = torch.zeros(w.shape, dtype=torch.float32, device=w.device)
    dw[live] = torch.bmm(d.transpose(1, 2), x[rows].float())
    return dx, dw


def _act(g, name):
    """The activation, and its derivative."""
    if name == "silu":
        t = 1 / (1 + torch.exp(-g))
        return g * t, t * (1 + g * (1 - t))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _plain_int8(s):
    y = _times(s, s["a"], s["b"]) * s["a_scales"][:, None]
    if s["offsets"] is None:
        y *= s["b_scales"]
    else:
        n = torch.diff(s["offsets"].long())
        y *= s["b_scales"].repeat_interleave(n, 0)
    if s["case"]["act"] != "none":
        gate, up = y.chunk(2, 1)
        y = _act(gate, s["case"]["act"])[0] * up
    return y.to(s["y"].dtype)


def _plain_gated(s):
    gu = _times(s, s["x"], s["w"])
    gate, up = gu.chunk(2, 1)
    h = (_act(gate, s["case"]["act"])[0] * up).to(torch.bfloat16)
    return (h, gu.to(torch.bfloat16)) if s["case"]["keep"] else h


def _plain_gated_backward(s):
    gate, up = s["gu"].float().chunk(2, 1)
    a, slope = _act(gate, s["case"]["act"])
    dh = s["dh"].float()
    dgu = torch.cat([dh * up * slope, dh * a], 1)
    dx, dw = _back(s, dgu)
    return dgu.to(torch.bfloat16), dx.to(torch.bfloat16), dw.to(torch.bfloat16)


def _plain_linear(s):
    return _times(s, s["x"], s["w"]).to(s["y"].dtype)


def _plain_linear_backward(s):
    dx, dw = _back(s, s["dy"].float())
    return dx.to(torch.bfloat16), dw.to(s["dw"].dtype)


_PLAIN = {"quantise": _plain_quantise, "int8": _plain_int8, "gated": _plain_gated, "gated backward": _plain_gated_backward,
          "linear": _plain_linear, "linear backward": _plain_linear_backward}


# ------------------------------------------------------------------ work


def work(case):
    """Bytes and operations of one pass; an expert's weights count where rows are expected to reach it."""
    op, K, size = case["op"], case["K"], {"bf16": 2, "fp32": 4}
    if op == "quantise":
        R, k = case["rows"], case["top_k"]
        return dict(bytes=R * K * size[case["dtype"]] + 4 * R * k + R * max(1, k) * (K + 4), flops=R * K * 3)
    M, E, k = case["M"], case["E"], case["top_k"]
    rows = M * k if E else M
    live = min(E, rows) if E and rows >= 8 * E else E * (1 - (1 - k / E) ** M) if E else 1
    edge = 4 * (E + 1) if E else 0
    N = 2 * case["I"] if op.startswith("gated") else case["N"]
    product = 2 * rows * N * K
    if op == "int8":
        out = N if case["act"] == "none" else N // 2
        return dict(bytes=rows * (K + 4 + out * size[case["out"]]) + live * N * (K + 4) + edge, flops=product)
    read = 2 * (rows * K + live * N * K) + edge
    if op == "gated":
        return dict(bytes=read + rows * N * (3 if case["keep"] else 1), flops=product)
    if op == "linear":
        return dict(bytes=read + rows * N * size[case["out"]], flops=product)
    grads = 2 * rows * K + max(1, E) * N * K * size[case.get("out", "bf16")]
    return dict(bytes=read + grads + rows * N * (2 if op == "linear backward" else 5), flops=2 * product)


# ------------------------------------------------------------------ 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        return _exact_quantise(s)
    N = 2 * case["I"] if op.startswith("gated") else case["N"]
    rows = (s["a"] if op == "int8" else s["x"]).shape[0]
    if 2 * rows * N * case["K"] > 1e12:
        return None
    edge = [0, rows] if s["offsets"] is None else s["offsets"].tolist()
    parts = [_EXACT[op](s, e, slice(edge[e], edge[e + 1])) for e in range(len(edge) - 1)]
    if not op.endswith("backward"):
        whole = tuple(torch.cat(p) for p in zip(*parts))
        return whole if op == "gated" and case["keep"] else whole[0]
    by = list(zip(*parts))
    return tuple(torch.cat(p) for p in by[:-1]) + (torch.stack(by[-1]),)


def _exact_quantise(s):
    x = s["x"].double()
    top = torch.clamp(torch.linalg.vector_norm(x, ord=math.inf, dim=1), min=FLOOR)
    step = (top / 127).float().double()  # codes count the scale that is stored
    z = x / step[:, None]
    q = torch.floor(z)
    rest = z - q
    q = torch.where((rest > 0.5) | ((rest == 0.5) & (q % 2 != 0)), q + 1, q).to(torch.int8)
    scale = top / 127
    if s["pos"] is not None:
        k = s["pos"].shape[1]
        src = torch.empty(x.shape[0] * k, dtype=torch.long, device=DEV)
        src[s["pos"].reshape(-1).long()] = torch.arange(x.shape[0] * k, device=DEV) // k
        q, scale = q[src], scale[src]
    return q, scale


def _sigmoid_form(z, act):
    """Both activations are z * sigmoid(v): v is z itself, or 2 sqrt(2 / pi) (z + 0.044715 z^3).  Returns the value and the derivative."""
    if act == "silu":
        v, dv = z, torch.ones_like(z)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        v, dv = c * z * (1 + 0.044715 * z ** 2), c * (1 + 0.134145 * z ** 2)
    p = torch.sigmoid(v)
    return z * p, p + z * p * torch.sigmoid(-v) * dv


def _exact_int8(s, e, at):
    act = s["case"]["act"]
    y = (s["a"][at].double() * s["a_scales"][at].double()[:, None]) @ (s["b"][e].double() * s["b_scales"][e].double()[:, None]).T
    half = y.shape[1] // 2
    return (y if act == "none" else _sigmoid_form(y[:, :half], act)[0] * y[:, half:],)


def _exact_gated(s, e, at):
    y = s["x"][at].double() @ s["w"][e].double().T
    half = y.shape[1] // 2
    return _sigmoid_form(y[:, :half], s["case"]["act"])[0] * y[:, half:], y


def _exact_linear(s, e, at):
    return (s["x"][at].double() @ s["w"][e].double().T,)


def _exact_linear_backward(s, e, at):
    d = s["dy"][at].double()
    return d @ s["w"][e].double(), d.T @ s["x"][at].double()


def _exact_gated_backward(s, e, at):
    half = s["case"]["I"]
    value, slope = _sigmoid_form(s["gu"][at, :half].double(), s["case"]["act"])
    d = s["dh"][at].double()
    dgu = torch.empty_like(s["gu"][at], dtype=torch.float64)
    dgu[:, :half] = d * s["gu"][at, half:].double() * slope
    dgu[:, half:] = d * value
    return dgu, dgu @ s["w"][e].double(), dgu.T @ s["x"][at].double()


_EXACT = {"int8": _exact_int8, "gated": _exact_gated, "linear": _exact_linear, "linear backward": _exact_linear_backward,
          "gated backward": _exact_gated_backward}
