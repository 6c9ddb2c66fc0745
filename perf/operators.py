"""Cases, inputs and plain forms of the operators of a mixture-of-experts layer with 8-bit weights: routing to experts, grouping
pairs of token and expert, quantising rows in blocks of 128, the block-scaled matrix product (dense and grouped), and the
weighted combine.

A pair is one (token, choice) entry of the routing; "expert order" is all pairs sorted by expert, pairs of one expert in
ascending order.  Scales of quantised rows are stored block by block, [K / 128][rows]; those of weights [experts][N / 128][K / 128].
"""

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
FLOOR = 2.0 ** -96  # smallest block maximum that a scale is made for
DEV = "cuda"


# ------------------------------------------------------------------ cases


def listed():
    return [
        # One decode step of 8 requests: the smallest routing call, all latency.
        dict(name="route decode", op="route", T=8, E=256, top_k=6, score="sigmoid", bias=False, groups=1, top_groups=1,
             group_score="max", renorm=True, scale=1.0, dtype="bf16", masked=0.0),
        # A prompt routed within device groups, with the bias that balances the experts' load.
        dict(name="route prompt, groups", op="route", T=8191, E=256, top_k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_score="top2", renorm=True, scale=2.5, dtype="fp32", masked=0.0),
        # The pairs of a 64-request decode step.
        dict(name="group decode", op="group", T=64, E=256, top_k=6, dropped=0.0),
        # The pairs of an 8,192-token prompt, some dropped as padding.
        dict(name="group prompt", op="group", T=8192, E=256, top_k=6, dropped=0.03),
        # A prompt's activations, quantised once and written to the places of their six experts.
        dict(name="quantise prompt, scatter", op="quantise", rows=8192, K=2048, top_k=6, E=256, silu=False, dtype="bf16",
             pad=0),
        # The pairs' gate and up projections of that prompt: the activation and its quantisation in one pass.
        dict(name="quantise gated prompt", op="quantise", rows=49152, K=512, top_k=0, E=0, silu=True, dtype="bf16", pad=0),
        # One token through a dense projection: bound by the weights' bytes.
        dict(name="product decode", op="product", M=1, N=4096, K=2048, E=0, top_k=0, out="bf16"),
        # A prompt (an odd number of rows) through a dense projection: bound by the tensor cores.
        dict(name="product prompt", op="product", M=8191, N=4096, K=4096, E=0, top_k=0, out="bf16"),
        # 8 requests through their 6 experts: some 45 experts with a row or two each.
        dict(name="experts decode", op="product", M=8, N=1024, K=2048, E=256, top_k=6, out="bf16"),
        # A prompt through its experts' gate and up projections: ragged groups of about 192 rows.
        dict(name="experts prompt", op="product", M=8192, N=1024, K=2048, E=256, top_k=6, out="bf16"),
        # The experts' outputs of 8 requests, weighted and summed with the shared expert's.
        dict(name="combine decode", op="combine", T=8, N=2048, top_k=6, shared=True, dtype="bf16", dropped=0.0),
        # The same for a prompt.
        dict(name="combine prompt", op="combine", T=8192, N=2048, top_k=6, shared=True, dtype="bf16", dropped=0.03),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "group", "quantise", "product", "product", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(1, 16 // groups), 512 // groups)
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, top_groups * (E // groups)))
        return dict(op=op, T=_log(rng, 1, 8192), E=E, top_k=top_k, score=rng.choice(["sigmoid", "softmax"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, group_score=rng.choice(["max", "top2"]),
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["bf16", "fp32"]),
                    masked=rng.choice([0.0, 0.0, 0.1]))
    if op == "group":
        E = rng.randint(8, 512)
        return dict(op=op, T=_log(rng, 1, 8192), E=E, top_k=rng.randint(1, 8), dropped=rng.choice([0.0, 0.05]))
    if op == "quantise":
        if rng.random() < 0.5:
            return dict(op=op, rows=_log(rng, 1, 32768), K=16 * rng.randint(8, 128), top_k=0, E=0, silu=True,
                        dtype=rng.choice(["bf16", "fp32"]), pad=rng.choice([0, 8]))
        return dict(op=op, rows=_log(rng, 1, 8192), K=16 * rng.randint(8, 160), top_k=rng.choice([0, 2, 6]), E=rng.randint(8, 256),
                    silu=False, dtype=rng.choice(["bf16", "fp32"]), pad=rng.choice([0, 8]))
    if op == "combine":
        return dict(op=op, T=_log(rng, 1, 8192), N=8 * rng.randint(16, 256), top_k=rng.randint(1, 8), shared=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp32"]), dropped=rng.choice([0.0, 0.05]))
    out = rng.choice(["bf16", "fp32"])
    if rng.random() < 0.5:
        return dict(op=op, M=_log(rng, 1, 8192), N=8 * rng.randint(16, 500), K=16 * rng.randint(8, 250), E=0, top_k=0, out=out)
    E = _log(rng, 4, 256)
    return dict(op=op, M=_log(rng, 1, 4096), N=8 * rng.randint(16, 128), K=16 * rng.randint(8, 128), E=E,
                top_k=rng.randint(1, min(6, E)), out=out)


# ------------------------------------------------------------------ inputs

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _choices(g, T, E, top_k, dropped=0.0):
    """Expert ids [T][top_k] of tokens whose router prefers some experts a little."""
    z = torch.randn(T, E, generator=g, device=DEV) + 0.3 * torch.randn(E, generator=g, device=DEV)
    ids = torch.topk(z, top_k, dim=1).indices.to(torch.int32)
    if dropped:
        ids[torch.rand(T, generator=g, device=DEV) < dropped] = -1  # padded tokens
    return ids


def _places(ids, E):
    """offsets [E + 1] and pos [T][top_k] of expert order."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=DEV)
    pos = torch.where(flat < 0, -1, pos).to(torch.int32).reshape(ids.shape)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(torch.bincount(key, minlength=E + 1)[:E], 0).to(torch.int32)
    return offsets, pos


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op == "route":
        T, E, k = case["T"], case["E"], case["top_k"]
        z = torch.randn(T, E, generator=g, device=DEV)
        if case["masked"]:  # experts that a deployment has taken out for some tokens
            z[torch.rand(T, E, generator=g, device=DEV) < case["masked"]] = -math.inf
        s["logits"] = z.to(DTYPES[case["dtype"]])
        s["bias"] = 0.05 * torch.randn(E, generator=g, device=DEV) if case["bias"] else None
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
        s["w"] = torch.empty(T, k, dtype=torch.float32, device=DEV)
    elif op == "group":
        T, E, k = case["T"], case["E"], case["top_k"]
        s["ids"] = _choices(g, T, E, k, case["dropped"])
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
        s["order"] = torch.empty(T * k, dtype=torch.int32, device=DEV)
        s["pos"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
    elif op == "quantise":
        R, K, k = case["rows"], case["K"], case["top_k"]
        cols = 2 * K if case["silu"] else K
        x = torch.randn(R, cols + case["pad"], generator=g, device=DEV)
        x *= torch.exp(torch.randn(cols + case["pad"], generator=g, device=DEV))  # channels of unlike size
        s["x"] = x.to(DTYPES[case["dtype"]])[:, :cols]
        s["pos"] = _places(_choices(g, R, case["E"], k), case["E"])[1] if k else None
        out_rows = R * max(1, k)
        s["q"] = torch.empty(out_rows, K, dtype=torch.float8_e4m3fn, device=DEV)
        s["scales"] = torch.empty(-(-K // BLOCK), out_rows, dtype=torch.float32, device=DEV)
    elif op == "product":
        M, N, K, E, k = case["M"], case["N"], case["K"], case["E"], case["top_k"]
        G, kb, nb = max(1, E), -(-K // BLOCK), -(-N // BLOCK)
        rows = M * k if E else M
        s["a"] = (100.0 * torch.randn(rows, K, generator=g, device=DEV)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["a_scales"] = 0.005 * torch.exp(0.5 * torch.randn(kb, rows, generator=g, device=DEV))
        b = torch.empty(G, N, K, dtype=torch.float8_e4m3fn, device=DEV)
        for e in range(0, G, 64):
            b[e : e + 64] = (100.0 * torch.randn(min(64, G - e), N, K, generator=g, device=DEV)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        s["b"] = b
        s["b_scales"] = 0.0002 * torch.exp(0.5 * torch.randn(G, nb, kb, generator=g, device=DEV))
        s["offsets"] = None
        if E:
            s["offsets"] = _places(_choices(g, M, E, k), E)[0]
            n = torch.diff(s["offsets"].long())
            live = torch.nonzero(n).reshape(-1)  # the plain form's plan: live experts and their rows, padded to the longest group
            at = torch.arange(int(n.max()), device=DEV)
            s["live"], s["have"] = live, at < n[live, None]
            s["rows"] = torch.where(s["have"], s["offsets"][:-1].long()[live, None] + at, 0)
        s["y"] = torch.empty(rows, N, dtype=DTYPES[case["out"]], device=DEV)
    else:
        T, N, k = case["T"], case["N"], case["top_k"]
        ids = _choices(g, T, 64, k, case["dropped"])
        s["pos"] = _places(ids, 64)[1]
        s["rows"] = torch.randn(T * k, N, generator=g, device=DEV).to(DTYPES[case["dtype"]])
        s["w"] = torch.rand(T, k, generator=g, device=DEV)
        s["shared"] = torch.randn(T, N, generator=g, device=DEV).to(torch.bfloat16) if case["shared"] else None
        s["y"] = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    return s


# ------------------------------------------------------------------ one pass


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def _own(s):
    from moe_decode_router_gb300 import flint_moe as F

    c = s["case"]
    if c["op"] == "route":
        F.route(s["logits"], s["ids"], s["w"], bias=s["bias"],
                score=F.SCORE_SIGMOID if c["score"] == "sigmoid" else F.SCORE_SOFTMAX,
                n_groups=c["groups"], top_groups=c["top_groups"],
                group_score=F.GROUP_MAX if c["group_score"] == "max" else F.GROUP_TOP2,
                renormalise=c["renorm"], scale=c["scale"])
        return s["ids"], s["w"]
    if c["op"] == "group":
        F.group_pairs(s["ids"], s["offsets"], s["order"], s["pos"])
        return s["offsets"], s["order"], s["pos"]
    if c["op"] == "quantise":
        F.quantize_rows(s["x"], s["q"], s["scales"], pos=s["pos"], silu_mul=c["silu"])
        return s["q"], s["scales"]
    if c["op"] == "product":
        F.block_gemm(s["a"], s["a_scales"], s["b"], s["b_scales"], s["y"], offsets=s["offsets"])
        return s["y"]
    F.combine(s["rows"], s["pos"], s["w"], s["y"], shared=s["shared"])
    return s["y"]


def _plain_route(s):
    c = s["case"]
    T, E, G = c["T"], c["E"], c["groups"]
    z = s["logits"].double()  # neighbouring scores decide what is selected
    fine = z > -math.inf  # false for a masked logit, and for NaN
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-z))
    else:
        top = torch.where(fine, z, -math.inf).max(1, keepdim=True).values
        u = torch.where(fine, torch.exp(torch.where(z == top, 0.0, z - top)), 0.0)
        score = u / u.sum(1, keepdim=True)
    key = z if s["bias"] is None else score + s["bias"].double()  # both scores grow with the logit
    key = torch.where(fine, key, -math.inf)
    if G > 1:
        if c["group_score"] == "max":
            gs = key.reshape(T, G, -1).max(2).values
        else:
            v = score if s["bias"] is None else key
            two = torch.where(fine, v, -math.inf).reshape(T, G, -1).sort(dim=2, descending=True).values[:, :, :2]
            gs = torch.where(two[:, :, :1] > -math.inf, torch.where(two > -math.inf, two, 0.0).sum(2, keepdim=True), -math.inf)[:, :, 0]
        rank = gs.sort(dim=1, descending=True, stable=True).indices.sort(dim=1).indices
        key = torch.where((rank < c["top_groups"]).repeat_interleave(E // G, 1), key, -math.inf)
    best = key.sort(dim=1, descending=True, stable=True)
    ids, there = best.indices[:, : c["top_k"]], best.values[:, : c["top_k"]] > -math.inf
    w = torch.where(there, score.gather(1, ids), 0.0)
    if c["renorm"]:
        w = torch.where(there, w / w.sum(1, keepdim=True), 0.0)
    return torch.where(there, ids, -1).to(torch.int32), (w * c["scale"]).float()


def _plain_group(s):
    ids, E = s["ids"].reshape(-1).long(), s["case"]["E"]
    key = torch.where(ids < 0, E, ids)
    by = key.sort(stable=True)
    offsets = torch.searchsorted(by.values, torch.arange(E + 1, device=ids.device)).to(torch.int32)
    order = torch.where(by.values < E, by.indices, -1).to(torch.int32)
    pos = torch.where(ids < 0, -1, by.indices.sort().indices).to(torch.int32)
    return offsets, order, pos.reshape(s["ids"].shape)


def _plain_quantise(s):
    c = s["case"]
    R, K = c["rows"], c["K"]
    x = s["x"].float()
    if c["silu"]:
        gate, up = x[:, :K], x[:, K:]
        x = gate / (1 + torch.exp(-gate)) * up
    kb = -(-K // BLOCK)
    x = torch.nn.functional.pad(x, (0, kb * BLOCK - K)).reshape(R, kb, BLOCK)
    top = x.abs().amax(2).clamp(min=FLOOR)
    q = (x * (E4M3_MAX / top)[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).reshape(R, kb * BLOCK)[:, :K]
    scales = (top / E4M3_MAX).T
    if s["pos"] is None:
        return q.contiguous(), scales.contiguous()
    k = s["pos"].shape[1]
    at = s["pos"].reshape(-1).long()
    out, sc = torch.empty(R * k, K, dtype=torch.uint8, device=x.device), torch.empty(kb, R * k, device=x.device)
    out[at] = q.contiguous().view(torch.uint8).repeat_interleave(k, 0)
    sc[:, at] = scales.repeat_interleave(k, 1)
    return out.view(torch.float8_e4m3fn), sc


def _plain_product(s):
    c = s["case"]
    K, N = c["K"], c["N"]
    a = s["a"].float() * s["a_scales"].T.repeat_interleave(BLOCK, 1)[:, :K]
    if s["offsets"] is None:
        b = s["b"][0].float() * s["b_scales"][0].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
        return torch.matmul(a, b.T).to(s["y"].dtype)
    live = s["live"]
    b = s["b"].view(torch.uint8)[live].view(torch.float8_e4m3fn).float()
    b *= s["b_scales"][live].repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]
    y = torch.bmm(a[s["rows"]], b.transpose(1, 2))
    return y[s["have"]].to(s["y"].dtype)


def _plain_combine(s):
    pos = s["pos"].long()
    v = s["rows"][pos.clamp(min=0)].float() * torch.where(pos < 0, 0.0, s["w"])[:, :, None]
    y = v.sum(1)
    return (y if s["shared"] is None else y + s["shared"].float()).to(torch.bfloat16)


_PLAIN = dict(route=_plain_route, group=_plain_group, quantise=_plain_quantise, product=_plain_product, combine=_plain_combine)


# ------------------------------------------------------------------ work


def work(case):
    """Bytes and operations of one pass; an expert's weights count where rows are expected to reach it."""
    op, size = case["op"], {"bf16": 2, "fp32": 4}
    if op == "route":
        T, E, k = case["T"], case["E"], case["top_k"]
        return dict(bytes=T * E * size[case["dtype"]] + (4 * E if case["bias"] else 0) + T * k * 8, flops=T * E * 4)
    if op == "group":
        P = case["T"] * case["top_k"]
        return dict(bytes=12 * P + 4 * (case["E"] + 1), flops=P)
    if op == "quantise":
        R, K, k = case["rows"], case["K"], case["top_k"]
        cols, out = (2 * K if case["silu"] else K), R * max(1, k)
        return dict(bytes=R * cols * size[case["dtype"]] + 4 * R * k + out * (K + 4 * -(-K // BLOCK)), flops=R * cols * 4)
    if op == "product":
        M, N, K, E, k = case["M"], case["N"], case["K"], case["E"], case["top_k"]
        rows = M * k if E else M
        live = min(E, rows) if E and rows >= 8 * E else E * (1 - (1 - k / E) ** M) if E else 1
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        return dict(bytes=rows * (K + 4 * kb + N * size[case["out"]]) + live * (N * K + 4 * nb * kb) + 4 * (E + 1 if E else 0),
                    flops=2 * rows * N * K)
    T, N, k = case["T"], case["N"], case["top_k"]
    rows = T * k * (1 - case["dropped"])
    return dict(bytes=rows * N * size[case["dtype"]] + 8 * T * k + T * N * (4 if case["shared"] else 2), flops=2 * rows * N)


# ------------------------------------------------------------------ 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "group":
        return _exact_group(s)
    if op == "quantise":
        return _exact_quantise(s)
    if op == "product":
        return _exact_product(s)
    pos, w = s["pos"], s["w"].double()
    y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device=DEV)
    for j in range(case["top_k"]):
        on = torch.nonzero(pos[:, j] >= 0).reshape(-1)
        y[on] += w[on, j, None] * s["rows"][pos[on, j].long()].double()
    return y if s["shared"] is None else y + s["shared"].double()


def _exact_route(s):
    """Row by row, choice by choice, as the definition reads."""
    import numpy as np

    c = s["case"]
    z = s["logits"].double().cpu().numpy()
    bias = None if s["bias"] is None else s["bias"].double().cpu().numpy()
    T, E, k, G = c["T"], c["E"], c["top_k"], c["groups"]
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        open_ = np.flatnonzero(z[t] > -np.inf)
        if not open_.size:
            continue
        score = np.zeros(E)
        if c["score"] == "sigmoid":
            score[open_] = 1 / (1 + np.exp(-z[t, open_]))
        else:
            e = np.exp(z[t, open_] - z[t, open_].max())
            score[open_] = e / e.sum()
        key = np.full(E, -np.inf)
        key[open_] = z[t, open_] if bias is None else score[open_] + bias[open_]
        if G > 1:
            gs = np.full(G, -np.inf)
            for q in range(G):
                mine = open_[(open_ >= q * (E // G)) & (open_ < (q + 1) * (E // G))]
                if mine.size:
                    v = key[mine] if c["group_score"] == "max" or bias is not None else score[mine]
                    gs[q] = v.max() if c["group_score"] == "max" else np.sort(v)[-2:].sum()
            out = np.argsort(-gs, kind="stable")[c["top_groups"]:]
            for q in out:
                key[q * (E // G) : (q + 1) * (E // G)] = -np.inf
        best = np.argsort(-key, kind="stable")[:k]
        best = best[key[best] > -np.inf]
        v = score[best]
        ids[t, : best.size] = best
        w[t, : best.size] = c["scale"] * (v / v.sum() if c["renorm"] else v)
    return ids, w


def _exact_group(s):
    import numpy as np

    ids = s["ids"].cpu().numpy().reshape(-1)
    E, offsets, order, pos = s["case"]["E"], [0], np.full(ids.size, -1, np.int32), np.full(ids.size, -1, np.int32)
    for e in range(E):
        mine = np.flatnonzero(ids == e)
        order[offsets[-1] : offsets[-1] + mine.size] = mine
        pos[mine] = offsets[-1] + np.arange(mine.size)
        offsets.append(offsets[-1] + mine.size)
    return np.array(offsets, np.int32), order, pos.reshape(tuple(s["ids"].shape))


def _exact_quantise(s):
    c = s["case"]
    K, k = c["K"], c["top_k"]
    x = s["x"].double()
    if c["silu"]:
        x = torch.sigmoid(x[:, :K]) * x[:, :K] * x[:, K:]
    q, sc = torch.empty_like(x), []
    for b in range(0, K, BLOCK):
        v = x[:, b : b + BLOCK]
        step = v.abs().max(1).values.clamp(min=FLOOR) / E4M3_MAX
        v = v / step[:, None]
        # e4m3: three bits behind the leading one, and steps of 2^-9 below 2^-6
        unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        q[:, b : b + BLOCK] = torch.round(v / unit) * unit
        sc.append(step)
    sc = torch.stack(sc)
    if k:
        src = torch.empty(q.shape[0] * k, dtype=torch.long, device=DEV)
        src[s["pos"].reshape(-1).long()] = torch.arange(q.shape[0] * k, device=DEV) // k
        q, sc = q[src], sc[:, src]
    return q, sc


def _exact_product(s):
    c = s["case"]
    rows, K, N = s["a"].shape[0], c["K"], c["N"]
    if 2 * rows * N * K > 1e12:
        return None
    y = torch.zeros(rows, N, dtype=torch.float64, device=DEV)
    edge = [0, rows] if s["offsets"] is None else s["offsets"].tolist()
    kb = torch.arange(K, device=DEV) // BLOCK
    nb = torch.arange(N, device=DEV) // BLOCK
    for e in range(len(edge) - 1):
        lo, hi = edge[e], edge[e + 1]
        if lo == hi:
            continue
        a = s["a"][lo:hi].double() * s["a_scales"].double()[kb, lo:hi].T
        b = s["b"][e].double() * s["b_scales"][e].double()[nb][:, kb]
        y[lo:hi] = a @ b.T
    return y
