"""Measured cases of the expert operators: the norm in front of the routing, the
FP8 block product, and the experts' gated feed-forward between a dispatch and
its combine (low-latency cells and dispatched rows, with the backward pass).

``own`` selects the framework's kernels; otherwise ``run`` computes the same in
elementary torch operations, in 32 bits, rounded once at the end.
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
BLOCK = 128
FP8_MAX = 448.0
AMAX_FLOOR = 1e-4


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step: residual, norm, 8-bit rows for the next product
        {"name": "norm_token", "kind": "norm", "T": 1, "H": 7168, "residual": True, "fp8": True},
        # a prefill batch in front of the router, the dispatch and a shared expert
        {"name": "norm_prefill", "kind": "norm", "T": 8192, "H": 7168, "residual": True, "fp8": True},
        # the training batch's norm, backwards
        {"name": "norm_backward", "kind": "norm_backward", "T": 4096, "H": 7168, "residual": True},
        # one token through a dense 8-bit projection: the weight is read once
        {"name": "product_token", "kind": "product", "M": 1, "N": 7168, "K": 2048},
        # a ragged chunk of tokens, a width that ends inside a scale block
        {"name": "product_ragged", "kind": "product", "M": 333, "N": 1000, "K": 1152},
        # a full prefill batch through a gate and up projection
        {"name": "product_prefill", "kind": "product", "M": 8192, "N": 4096, "K": 7168},
        # the low-latency decode batch: 256 experts, four rows each, FP8 weights
        {"name": "decode_fp8", "kind": "cells", "T": 128, "H": 7168, "I": 2048, "E": 256, "R": 32, "K": 8,
         "S": 128, "fp8": True, "mask": 0.0},
        # a single token on bf16 weights
        {"name": "decode_token", "kind": "cells", "T": 1, "H": 2048, "I": 768, "E": 64, "R": 8, "K": 8,
         "S": 16, "fp8": False, "mask": 0.0},
        # a large low-latency batch: about 128 rows for each expert
        {"name": "cells_large_fp8", "kind": "cells", "T": 1024, "H": 7168, "I": 2048, "E": 64, "R": 32, "K": 8,
         "S": 1024, "fp8": True, "mask": 0.0},
        # the experts of a dispatched batch, inference
        {"name": "experts_forward", "kind": "experts", "T": 4096, "H": 7168, "I": 2048, "E": 32, "R": 8, "K": 8,
         "mask": 0.0, "step": False},
        # the same as a training step: outputs and every gradient
        {"name": "experts_step", "kind": "experts", "T": 4096, "H": 7168, "I": 2048, "E": 32, "R": 8, "K": 8,
         "mask": 0.0, "step": True},
        # a small ragged batch with masked slots, some experts nearly empty
        {"name": "experts_step_ragged", "kind": "experts", "T": 601, "H": 256, "I": 352, "E": 64, "R": 16, "K": 6,
         "mask": 0.1, "step": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _steps(rng, lo, hi, step):
    return max(lo, min(hi, _log(rng, lo, hi) // step * step))


def draw(rng):
    kind = rng.choice(["norm", "norm_backward", "product", "cells", "cells", "experts", "experts"])
    if kind == "norm":
        return {"kind": kind, "T": _log(rng, 1, 8192), "H": _steps(rng, 128, 7168, 128),
                "residual": rng.random() < 0.7, "fp8": rng.random() < 0.7}
    if kind == "norm_backward":
        return {"kind": kind, "T": _log(rng, 1, 4096), "H": _steps(rng, 64, 7168, 8),
                "residual": rng.random() < 0.5}
    if kind == "product":
        return {"kind": kind, "M": _log(rng, 1, 8192), "N": _steps(rng, 64, 7168, 8),
                "K": _steps(rng, 128, 4096, 128)}
    ranks = rng.choice([1, 2, 4, 8, 16, 32])
    local = rng.choice([1, 2, 3, 4])
    experts = ranks * local
    k = rng.randint(1, min(8, experts))
    mask = rng.choice([0.0, 0.05, 0.3])
    if kind == "cells":
        fp8 = rng.random() < 0.6
        tokens = _log(rng, 1, 1024)
        return {"kind": kind, "T": tokens, "H": _steps(rng, 128, 4096, 128),
                "I": _steps(rng, 128, 2048, 128) if fp8 else _steps(rng, 64, 2048, 8),
                "E": experts, "R": ranks, "K": k, "S": tokens + rng.choice([0, 1, 17]), "fp8": fp8, "mask": mask}
    return {"kind": kind, "T": _log(rng, 1, 4096), "H": _steps(rng, 64, 4096, 8), "I": _steps(rng, 64, 2048, 8),
            "E": experts, "R": ranks, "K": k, "mask": mask, "step": rng.random() < 0.6}


# --------------------------------------------------------------- inputs

def _normal(gen, shape, scale=1.0, dtype=torch.bfloat16):
    """A normal tensor, made a slab at a time so that no fp32 copy of a large one is held."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    step = 1 << 28
    for a in range(0, flat.numel(), step):
        n = min(step, flat.numel() - a)
        flat[a:a + n] = torch.randn(n, generator=gen, device="cuda") * scale
    return out


def _rows_fp8(gen, shape):
    """Rows as an FP8 dispatch or norm leaves them: codes and a scale for each 128 elements."""
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    rows, width = codes.view(-1, shape[-1]), shape[-1]
    scales = torch.empty((rows.shape[0], width // BLOCK), device="cuda")
    step = max(1, (1 << 27) // width)
    for a in range(0, rows.shape[0], step):
        v = torch.randn((min(step, rows.shape[0] - a), width // BLOCK, BLOCK), generator=gen, device="cuda")
        amax = v.abs().amax(-1, keepdim=True).clamp_min(AMAX_FLOOR)
        rows[a:a + step] = (v * (FP8_MAX / amax)).to(torch.float8_e4m3fn).view(-1, width)
        scales[a:a + step] = (amax / FP8_MAX).squeeze(-1)
    return codes, scales.view(*shape[:-1], width // BLOCK)


def _weight_fp8(gen, count, n, k):
    """count weights [n, k] in e4m3 with one fp32 scale for each 128 x 128 block."""
    nb, kb = -(-n // BLOCK), k // BLOCK
    codes = torch.empty((count, n, k), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((count, nb, kb), device="cuda")
    for e in range(count):
        v = torch.zeros((nb * BLOCK, k), device="cuda")
        v[:n] = torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)
        v = v.view(nb, BLOCK, kb, BLOCK)
        amax = v.abs().amax((1, 3), keepdim=True).clamp_min(AMAX_FLOOR)
        codes[e] = (v * (FP8_MAX / amax)).to(torch.float8_e4m3fn).reshape(nb * BLOCK, k)[:n]
        scales[e] = (amax / FP8_MAX).view(nb, kb)
    return codes, scales


def _routing(gen, case):
    """Distinct uniform experts for every token, some slots masked with -1, and softmax weights."""
    T, E, K = case["T"], case["E"], case["K"]
    topk = torch.rand((T, E), generator=gen, device="cuda").argsort(1)[:, :K].contiguous()
    drop = torch.rand((T, K), generator=gen, device="cuda") < case["mask"]
    drop[0, 0] = False  # a batch routes something
    topk = torch.where(drop, -1, topk)
    weights = torch.softmax(torch.randn((T, K), generator=gen, device="cuda"), 1)
    return topk, weights


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind = case["kind"]
    if kind == "norm":
        T, H = case["T"], case["H"]
        return {"case": case, "x": _normal(gen, (T, H)),
                "residual": _normal(gen, (T, H), 2.0) if case["residual"] else None,
                "weight": (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(torch.bfloat16)}
    if kind == "norm_backward":
        T, H = case["T"], case["H"]
        h = _normal(gen, (T, H), 2.0)
        return {"case": case, "dout": _normal(gen, (T, H)), "h": h,
                "weight": (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(torch.bfloat16),
                "rstd": torch.rsqrt(h.double().square().mean(1) + EPS).float(),
                "dresidual": _normal(gen, (T, H)) if case["residual"] else None}
    if kind == "product":
        codes, scales = _weight_fp8(gen, 1, case["N"], case["K"])
        return {"case": case, "a": _rows_fp8(gen, (case["M"], case["K"])), "w": (codes[0], scales[0])}
    H, I, E, R, K = case["H"], case["I"], case["E"], case["R"], case["K"]
    local = E // R
    topk, weights = _routing(gen, case)
    if kind == "cells":
        S = case["S"]
        state = {"case": case}
        # pairs of an expert take its slots in (token, slot) order
        hit = torch.nn.functional.one_hot(topk.reshape(-1) + 1, E + 1)[:, 1:]
        place = (hit.cumsum(0) - 1).gather(1, topk.reshape(-1, 1).clamp_min(0)).view_as(topk)
        state["slot"] = torch.where(topk >= 0, place, -1).int()
        state["count"] = hit.sum(0).view(R, local).t().contiguous().int()
        state["src"] = torch.full((local, R, S), -1, dtype=torch.int32, device="cuda")
        cells = (local, R, S, H)
        if case["fp8"]:
            state["packed"] = _rows_fp8(gen, cells)
            state["w13"], state["w2"] = _weight_fp8(gen, E, 2 * I, H), _weight_fp8(gen, E, H, I)
        else:
            state["packed"] = _normal(gen, cells)
            state["w13"] = _normal(gen, (E, 2 * I, H), 1 / math.sqrt(H))
            state["w2"] = _normal(gen, (E, H, I), 1 / math.sqrt(I))
        state["out"] = torch.zeros(cells, dtype=torch.bfloat16, device="cuda")
        return state
    # what a dispatch leaves in worst-case buffers (no host sync): each token once for each rank,
    # rows ordered by (rank, token), then rows of an earlier batch that the prefix leaves out
    rank = torch.where(topk >= 0, topk // local, -1)
    member = torch.nn.functional.one_hot(rank + 1, R + 1)[:, :, 1:].amax(1)
    row_rank, row_token = member.t().nonzero(as_tuple=True)
    mine = rank[row_token] == row_rank[:, None]
    ids = torch.where(mine, topk[row_token] - (row_rank * local)[:, None], -1)
    rows, used = case["T"] * min(K, R), len(row_token)
    x = _normal(gen, (rows, H))
    x[:used] = _normal(gen, (case["T"], H))[row_token]
    stale = torch.randint(-1, local, (rows, K), generator=gen, device="cuda")
    stale[:used] = ids
    held = torch.rand((rows, K), generator=gen, device="cuda")
    held[:used] = torch.where(mine, weights[row_token], 0.0)
    state = {"case": case, "x": x, "ids": stale, "weights": held,
             "prefix": member.sum(0).cumsum(0).int(),
             "w13": _normal(gen, (E, 2 * I, H), 1 / math.sqrt(H)),
             "w2": _normal(gen, (E, H, I), 1 / math.sqrt(I)),
             # rows that the fullest expert holds: the padding of the plain form
             "most": int(torch.bincount(topk[topk >= 0], minlength=E).max()) if bool((topk >= 0).any()) else 1}
    if case["step"]:
        state["dy"] = _normal(gen, (rows, H), 0.1)
    return state


# ------------------------------------------------------------ plain forms

def _blocks(v):
    return v.view(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK)


def _quantised(v):
    """(codes, scales) of rows of values: amax of 128, its floor, e4m3 to nearest."""
    b = _blocks(v)
    amax = b.abs().amax(-1, keepdim=True).clamp_min(AMAX_FLOOR)
    return (b * (FP8_MAX / amax)).to(torch.float8_e4m3fn).view(v.shape), (amax / FP8_MAX).squeeze(-1)


def _values(rows):
    codes, scales = rows
    return (_blocks(codes.float()) * scales[..., None]).view(codes.shape)


def _weight_values(w):
    codes, scales = w
    n = codes.shape[-2]
    wide = scales.repeat_interleave(BLOCK, -2)[..., :n, :]
    return (_blocks(codes.float()) * wide[..., None]).view(codes.shape)


def _plain_norm(s):
    v = s["x"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    rstd = torch.rsqrt(v.square().mean(1) + EPS)
    y = v * rstd[:, None] * s["weight"].float()
    fp8 = _quantised(y) if s["case"]["fp8"] else None
    return y.to(torch.bfloat16), fp8, v.to(torch.bfloat16) if s["residual"] is not None else None, rstd


def _plain_norm_backward(s):
    dout, rstd = s["dout"].float(), s["rstd"][:, None]
    a = dout * s["weight"].float()
    xh = s["h"].float() * rstd
    dx = rstd * (a - xh * (a * xh).mean(1, keepdim=True))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return dx.to(torch.bfloat16), (dout * xh).sum(0)


def _gated(gu):
    g, u = gu.chunk(2, -1)
    return g * torch.sigmoid(g) * u


def _plain_cells(s):
    c = s["case"]
    local, R, S, H = s["out"].shape
    x = _values(s["packed"]) if c["fp8"] else s["packed"].float()
    x = x.transpose(0, 1).reshape(c["E"], S, H)  # expert e sits at cell block (e % local, e // local)
    w13, w2 = (_weight_values(s[n]) if c["fp8"] else s[n].float() for n in ("w13", "w2"))
    act = _gated(torch.bmm(x, w13.transpose(1, 2)))
    del w13
    if c["fp8"]:
        act = _values(_quantised(act))
    z = torch.bmm(act, w2.transpose(1, 2)).view(R, local, S, H).transpose(0, 1)
    used = torch.arange(S, device="cuda") < s["count"][..., None]
    return torch.where(used[..., None], z, 0.0).to(torch.bfloat16)


def _plain_experts(s):
    c = s["case"]
    E, R, most = c["E"], c["R"], s["most"]
    N, K = s["ids"].shape
    H = c["H"]
    # every (row, slot) pair sorted by expert, padded to the fullest expert's rows
    rank = torch.searchsorted(s["prefix"], torch.arange(N, dtype=torch.int32, device="cuda"), right=True)
    key = torch.where((s["ids"] >= 0) & (rank < R)[:, None], rank[:, None] * (E // R) + s["ids"], E).view(-1)
    order = key.argsort(stable=True)
    first = (key[None, :] < torch.arange(E + 1, device="cuda")[:, None]).sum(1)
    place = torch.arange(N * K, device="cuda") - first[key[order]]
    table = torch.full((E * most + 1,), N * K, device="cuda")
    table[torch.where(key[order] < E, key[order] * most + place, E * most)] = order
    table = table[:-1]
    live = table < N * K
    row = torch.where(live, table // K, 0)
    weight = torch.where(live, s["weights"].view(-1)[table.clamp_max(N * K - 1)], 0.0)[:, None]
    keep = live[:, None].float()
    x = (s["x"][row].float() * keep).view(E, most, H)
    w13, w2 = s["w13"].float(), s["w2"].float()
    gu = torch.bmm(x, w13.transpose(1, 2))
    act = _gated(gu)
    z = torch.bmm(act, w2.transpose(1, 2)).view(-1, H) * weight
    y = torch.zeros((N, H), device="cuda").index_add_(0, row, z).to(torch.bfloat16)
    if not c["step"]:
        return y
    dy = (s["dy"][row].float() * keep).view(E, most, H)
    d = torch.bmm(dy, w2)
    dweight = torch.zeros(N * K + 1, device="cuda")
    dweight[table] = (act * d).sum(-1).view(-1)
    da = d * weight.view(E, most, 1)
    g, u = gu.chunk(2, -1)
    sig = torch.sigmoid(g)
    dgu = torch.cat((da * u * sig * (1 + g * (1 - sig)), da * g * sig), -1)
    dw2 = torch.bmm(dy.transpose(1, 2), act * weight.view(E, most, 1)).to(torch.bfloat16)
    dw13 = torch.bmm(dgu.transpose(1, 2), x).to(torch.bfloat16)
    dx = torch.bmm(dgu, w13).view(-1, H)
    dx = torch.zeros((N, H), device="cuda").index_add_(0, row, dx * keep).to(torch.bfloat16)
    return y, dx, dweight[:-1].view(N, K), dw13, dw2


# ------------------------------------------------------------------- run

def _run_own(s):
    import combine_get_dispatch_05_amd as ep
    c = s["case"]
    if c["kind"] == "norm":
        return ep.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], use_fp8=c["fp8"])
    if c["kind"] == "norm_backward":
        return ep.rms_norm_backward(s["dout"], s["h"], s["weight"], s["rstd"], dresidual=s["dresidual"])
    if c["kind"] == "product":
        return ep.fp8_product(s["a"], s["w"])
    buf = ep.Buffer(c["R"], c["E"])
    if c["kind"] == "cells":
        handle = ep.LowLatencyHandle(s["src"], s["slot"], c["S"], c["E"], c["H"])
        return buf.low_latency_expert_ffn(s["packed"], s["count"], handle, s["w13"], s["w2"], out=s["out"])
    rows = buf.expert_rows(s["ids"], s["prefix"], num_tokens=c["T"])
    y, saved = buf.expert_ffn(s["x"], rows, s["weights"], s["w13"], s["w2"], save=c["step"])
    if not c["step"]:
        return y
    return (y, *buf.expert_ffn_backward(s["dy"], s["x"], rows, s["weights"], s["w13"], s["w2"], saved))


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "product": _plain_product,
            "cells": _plain_cells, "experts": _plain_experts}[state["case"]["kind"]](state)


def _plain_product(s):
    return (_values(s["a"]) @ _weight_values(s["w"]).t()).to(torch.bfloat16)


# ------------------------------------------------------------------ work

def work(case):
    kind = case["kind"]
    if kind == "norm":
        n = case["T"] * case["H"]
        fp8 = n + n // 32 if case["fp8"] else 0
        return {"bytes": n * (8 if case["residual"] else 4) + fp8 + 4 * case["T"] + 2 * case["H"],
                "flops": n * (8 if case["fp8"] else 5)}
    if kind == "norm_backward":
        n = case["T"] * case["H"]
        return {"bytes": n * (8 if case["residual"] else 6) + 4 * case["T"] + 6 * case["H"], "flops": n * 10}
    if kind == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * 33 // 32 + N * K + -(-N // BLOCK) * (K // BLOCK) * 4 + 2 * M * N,
                "flops": 2 * M * N * K}
    H, I, E = case["H"], case["I"], case["E"]
    pairs = case["T"] * case["K"] * (1 - case["mask"])
    reached = E * (1 - (1 - (1 - case["mask"]) * case["K"] / E) ** case["T"])
    flops = 6 * pairs * H * I
    if kind == "cells":
        size = 1 if case["fp8"] else 2
        return {"bytes": int(3 * H * I * size * reached + pairs * H * (size + 2)), "flops": int(flops)}
    ranks = case["R"]
    rows = case["T"] * ranks * (1 - (1 - (1 - case["mask"]) * case["K"] / E) ** (E // ranks))
    held = case["T"] * min(case["K"], ranks)  # rows of the worst-case buffers: outputs are whole
    nbytes = 6 * H * I * reached + 2 * rows * H + 2 * held * H + rows * case["K"] * 12
    if case["step"]:
        nbytes += 6 * H * I * E + 2 * rows * H + 2 * held * H + held * case["K"] * 4
        flops *= 3
    return {"bytes": int(nbytes), "flops": int(flops)}


# ----------------------------------------------------------------- exact

def _exact_round(v):
    """Rows of 128-blocks as the values their 8-bit codes stand for, and codes and scales."""
    shape = v.shape
    b = v.reshape(*shape[:-1], -1, BLOCK)
    amax = torch.clamp(b.abs().max(dim=-1, keepdim=True).values, min=AMAX_FLOOR)
    t = b / amax * FP8_MAX
    # e4m3: three mantissa bits, the smallest step 2^-9
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(t.abs().clamp_min(1e-30))), min=-6.0) - 3.0)
    codes = torch.clamp(torch.round(t / step) * step, -FP8_MAX, FP8_MAX)
    scale = amax / FP8_MAX
    return codes.reshape(shape), scale.squeeze(-1), (codes * scale).reshape(shape)


def _exact_weight(w, e):
    codes, scales = w
    v = codes[e].double()
    up = scales[e].double().repeat_interleave(BLOCK, 0)[:v.shape[0]].repeat_interleave(BLOCK, 1)
    return v * up


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "norm":
        v = s["x"].double()
        if case["residual"]:
            v = v + s["residual"].double()
        rstd = 1 / torch.sqrt((v * v).sum(1) / case["H"] + EPS)
        y = v * rstd.unsqueeze(1) * s["weight"].double()
        fp8 = None
        if case["fp8"]:
            codes, scale, _ = _exact_round(y)
            fp8 = (codes, scale)
        return y, fp8, v if case["residual"] else None, rstd
    if kind == "norm_backward":
        h, w, d, r = s["h"].double(), s["weight"].double(), s["dout"].double(), s["rstd"].double().unsqueeze(1)
        inner = (d * w * h).sum(1, keepdim=True)
        dx = r * d * w - r ** 3 * h * inner / case["H"]
        if case["residual"]:
            dx = dx + s["dresidual"].double()
        return dx, (d * h * r).sum(0)
    if kind == "product":
        codes, scales = s["a"]
        a = codes.double() * scales.double().repeat_interleave(BLOCK, 1)
        w = _exact_weight((s["w"][0][None], s["w"][1][None]), 0)
        return a @ w.t()
    E, R = case["E"], case["R"]
    local = E // R
    if kind == "cells":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        for e in range(E):
            le, r = e % local, e // local
            n = int(s["count"][le, r])
            if n == 0:
                continue
            if case["fp8"]:
                x = s["packed"][0][le, r, :n].double() * s["packed"][1][le, r, :n].double().repeat_interleave(BLOCK, 1)
                w13, w2 = _exact_weight(s["w13"], e), _exact_weight(s["w2"], e)
            else:
                x, w13, w2 = s["packed"][le, r, :n].double(), s["w13"][e].double(), s["w2"][e].double()
            g, u = x @ w13[:case["I"]].t(), x @ w13[case["I"]:].t()
            act = g / (1 + torch.exp(-g)) * u
            if case["fp8"]:
                act = _exact_round(act)[2]
            out[le, r, :n] = act @ w2.t()
        return out
    N, K = s["ids"].shape
    I, H = case["I"], case["H"]
    start = [0] + s["prefix"].tolist()
    y = torch.zeros((N, H), dtype=torch.float64, device="cuda")
    grads = case["step"]
    if grads:
        dx = torch.zeros_like(y)
        dweights = torch.zeros((N, K), dtype=torch.float64, device="cuda")
        dw13 = torch.zeros((E, 2 * I, H), dtype=torch.float64, device="cuda")
        dw2 = torch.zeros((E, H, I), dtype=torch.float64, device="cuda")
    for e in range(E):
        a, b = start[e // local], start[e // local + 1]
        row, slot = (s["ids"][a:b] == e % local).nonzero(as_tuple=True)
        if row.numel() == 0:
            continue
        row = row + a
        x, p = s["x"][row].double(), s["weights"][row, slot].double().unsqueeze(1)
        wg, wu, w2 = s["w13"][e, :I].double(), s["w13"][e, I:].double(), s["w2"][e].double()
        g, u = x @ wg.t(), x @ wu.t()
        sig = 1 / (1 + torch.exp(-g))
        act = g * sig * u
        y.index_add_(0, row, p * (act @ w2.t()))
        if not grads:
            continue
        dy = s["dy"][row].double()
        dact = dy @ w2
        dweights[row, slot] = (dact * act).sum(1)
        dact = dact * p
        du = dact * g * sig
        dg = dact * u * (sig + g * sig * (1 - sig))
        dw2[e] = (p * dy).t() @ act
        dw13[e, :I], dw13[e, I:] = dg.t() @ x, du.t() @ x
        dx.index_add_(0, row, dg @ wg + du @ wu)
    return (y, dx, dweights, dw13, dw2) if grads else y
