"""Measured cases of the operators around the experts: the router with its gradient,
the whole mixture-of-experts layer for a few tokens, and the low-rank adapters of many
requests beside a shared projection, with their gradients.

``own`` selects the framework's kernels; otherwise ``run`` computes the same in
elementary torch operations, in 32 bits (the router's comparisons in 64), rounded once
at the end.
"""

from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
FP8_MAX = 448.0
AMAX_FLOOR = 1e-4
WEIGHT_FLOOR = 1e-20  # beside the sum that sigmoid weights are divided by


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding token through a sigmoid router with groups and a balancing bias
        {"name": "route_token", "kind": "route", "T": 1, "E": 256, "R": 32, "K": 8, "score": "sigmoid", "bias": True,
         "G": 8, "g": 4, "norm": True, "bf16": False, "mask": 0.0, "step": False},
        # the same router on a prefill batch
        {"name": "route_prefill", "kind": "route", "T": 8192, "E": 256, "R": 32, "K": 8, "score": "sigmoid",
         "bias": True, "G": 8, "g": 4, "norm": True, "bf16": False, "mask": 0.0, "step": False},
        # a training batch: weights, the balancing loss's sums, and the gradient of both
        {"name": "route_step", "kind": "route", "T": 4096, "E": 256, "R": 64, "K": 8, "score": "softmax",
         "bias": False, "G": 1, "g": 1, "norm": True, "bf16": False, "mask": 0.0, "step": True},
        # a ragged batch of bf16 logits (full of ties) with experts masked here and there
        {"name": "route_step_ragged", "kind": "route", "T": 601, "E": 288, "R": 144, "K": 6, "score": "softmax",
         "bias": False, "G": 1, "g": 1, "norm": False, "bf16": True, "mask": 0.1, "step": True},
        # one token through a small bf16 layer: what a decode step waits for
        {"name": "layer_token", "kind": "layer", "T": 1, "H": 2048, "I": 768, "E": 64, "K": 8, "score": "softmax",
         "bias": False, "G": 1, "g": 1, "fp8": False, "residual": True},
        # one token through a large layer with FP8 weights
        {"name": "layer_token_fp8", "kind": "layer", "T": 1, "H": 7168, "I": 2048, "E": 256, "K": 8,
         "score": "sigmoid", "bias": True, "G": 8, "g": 4, "fp8": True, "residual": True},
        # a handful of odd sizes in bf16
        {"name": "layer_few", "kind": "layer", "T": 13, "H": 1000, "I": 520, "E": 24, "K": 3, "score": "softmax",
         "bias": False, "G": 1, "g": 1, "fp8": False, "residual": False},
        # a small decode batch that reaches nearly every expert
        {"name": "layer_batch_fp8", "kind": "layer", "T": 32, "H": 7168, "I": 2048, "E": 64, "K": 8,
         "score": "sigmoid", "bias": True, "G": 8, "g": 4, "fp8": True, "residual": True},
        # one token's adapter on a projection's output
        {"name": "adapter_token", "kind": "adapter", "T": 1, "K": 7168, "N": 2048, "r": 16, "L": 8, "runs": False,
         "none": 0.0, "step": False},
        # a decode batch, nearly every request with an adapter of its own, some with none
        {"name": "adapter_decode", "kind": "adapter", "T": 128, "K": 7168, "N": 4096, "r": 16, "L": 64, "runs": False,
         "none": 0.1, "step": False},
        # prefill: long runs of tokens that share an adapter
        {"name": "adapter_prefill", "kind": "adapter", "T": 8192, "K": 7168, "N": 7168, "r": 64, "L": 16,
         "runs": True, "none": 0.1, "step": False},
        # a training step of several adapters at once: outputs and every gradient
        {"name": "adapter_step", "kind": "adapter", "T": 4096, "K": 7168, "N": 4096, "r": 32, "L": 8, "runs": True,
         "none": 0.0, "step": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _steps(rng, lo, hi, step):
    return max(lo, min(hi, _log(rng, lo, hi) // step * step))


def _router(rng, E, K):
    """A scoring rule for E experts, K of them chosen."""
    groups = rng.choice([n for n in (1, 1, 2, 4, 8) if E % n == 0])
    chosen = rng.randint(-(-K * groups // E), groups) if groups > 1 else 1
    return {"score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "G": groups, "g": chosen}


def draw(rng):
    kind = rng.choice(["route", "route", "layer", "layer", "adapter", "adapter"])
    if kind == "adapter":
        return {"kind": kind, "T": _log(rng, 1, 4096), "K": _steps(rng, 64, 7168, 8), "N": _steps(rng, 64, 7168, 8),
                "r": rng.choice([8, 16, 24, 32, 64, 128]), "L": _log(rng, 1, 32), "runs": rng.random() < 0.5,
                "none": rng.choice([0.0, 0.1, 0.6]), "step": rng.random() < 0.5}
    ranks = rng.choice([1, 2, 4, 8, 16, 32])
    E = ranks * rng.choice([1, 2, 3, 4, 8])
    if kind == "layer":
        E = min(E, 64)
    K = rng.randint(1, min(8, E))
    case = {"kind": kind, "E": E, "K": K, **_router(rng, E, K)}
    if kind == "route":
        return {**case, "T": _log(rng, 1, 8192), "R": ranks, "norm": rng.random() < 0.6, "bf16": rng.random() < 0.4,
                "mask": rng.choice([0.0, 0.0, 0.1, 0.8]), "step": rng.random() < 0.6}
    fp8 = rng.random() < 0.5
    return {**case, "T": _log(rng, 1, 64), "H": _steps(rng, 128, 4096, 128 if fp8 else 8),
            "I": _steps(rng, 128, 2048, 128) if fp8 else _steps(rng, 64, 1024, 8), "fp8": fp8, "residual": rng.random() < 0.5}


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


def _weight_fp8(gen, count, n, k):
    """count weights [n, k] in e4m3 with one fp32 scale for each 128 x 128 block."""
    nb, kb = n // BLOCK, k // BLOCK
    codes = torch.empty((count, n, k), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((count, nb, kb), device="cuda")
    for e in range(count):
        v = torch.randn((nb, BLOCK, kb, BLOCK), generator=gen, device="cuda") / math.sqrt(k)
        amax = v.abs().amax((1, 3), keepdim=True).clamp_min(AMAX_FLOOR)
        codes[e] = (v * (FP8_MAX / amax)).to(torch.float8_e4m3fn).view(n, k)
        scales[e] = (amax / FP8_MAX).view(nb, kb)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    kind, T = case["kind"], case["T"]
    if kind == "adapter":
        L, r, K, N = case["L"], case["r"], case["K"], case["N"]
        parts = 3 * L if case["runs"] else T  # runs: a batch of sequences, each with one adapter or none
        none = torch.rand(parts, generator=gen, device="cuda") < case["none"]
        ids = torch.randint(0, L, (parts,), generator=gen, device="cuda")
        part = torch.arange(T, device="cuda") * parts // T
        ids, none = ids[part], none[part]
        state = {"case": case, "x": _normal(gen, (T, K)), "ids": torch.where(none, -1, ids),
                 "down": _normal(gen, (L, r, K), 1 / math.sqrt(K)), "up": _normal(gen, (L, N, r), 1 / math.sqrt(r)),
                 "scales": 0.5 + torch.rand(L, generator=gen, device="cuda"), "base": _normal(gen, (T, N))}
        if case["step"]:
            state["dy"], state["dx_base"] = _normal(gen, (T, N), 0.1), _normal(gen, (T, K), 0.1)
        return state
    E = case["E"]
    # a bias as balancing leaves it: of the size of the scores' own differences
    bias = 0.1 * torch.randn(E, generator=gen, device="cuda") if case["bias"] else None
    if kind == "route":
        logits = torch.randn((T, E), generator=gen, device="cuda") * 1.5
        logits[torch.rand((T, E), generator=gen, device="cuda") < case["mask"]] = -math.inf
        state = {"case": case, "logits": logits.to(torch.bfloat16) if case["bf16"] else logits, "bias": bias}
        if case["step"]:
            state["dweights"] = torch.randn((T, case["K"]), generator=gen, device="cuda")
            state["dsums"] = 0.1 * torch.randn(E, generator=gen, device="cuda")
        return state
    H, I = case["H"], case["I"]
    state = {"case": case, "bias": bias, "x": _normal(gen, (T, H)),
             "w_router": _normal(gen, (E, H), 1.5 / math.sqrt(H)),
             "residual": _normal(gen, (T, H), 2.0) if case["residual"] else None}
    if case["fp8"]:
        state["w13"], state["w2"] = _weight_fp8(gen, E, 2 * I, H), _weight_fp8(gen, E, H, I)
    else:
        state["w13"] = _normal(gen, (E, 2 * I, H), 1 / math.sqrt(H))
        state["w2"] = _normal(gen, (E, H, I), 1 / math.sqrt(I))
    return state


# ------------------------------------------------------------ plain forms

def _scale_of(case):
    return 2.5 if case["score"] == "sigmoid" else 1.0


def _plain_chosen(case, logits, bias):
    """The chosen experts [T, K] of fp32 logits, -1 where there are too few."""
    T, E = logits.shape
    # both scores grow with the logit, so without a bias the logits are compared
    key = logits.double()
    if bias is not None:
        key = torch.sigmoid(key) if case["score"] == "sigmoid" else torch.softmax(key, 1)
        key = key + bias.double()
    key = torch.where(logits > -math.inf, key, -math.inf)
    if case["G"] > 1:
        parts = key.view(T, case["G"], -1).sort(dim=2, descending=True).values
        best = parts[:, :, 0]
        if bias is not None and parts.shape[2] > 1:
            second = parts[:, :, 1]
            best = best + torch.where(second > -math.inf, second, 0.0)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :case["g"]]
        keep = torch.zeros((T, case["G"]), device="cuda").scatter_(1, order, 1.0) > 0
        key = torch.where(keep.repeat_interleave(E // case["G"], 1), key, -math.inf)
    value, index = key.sort(dim=1, descending=True, stable=True)
    return torch.where(value[:, :case["K"]] > -math.inf, index[:, :case["K"]], -1)


def _plain_weights(case, logits, chosen, norm):
    """(weights [T, K], scores [T, E], shares of the chosen [T, K]) of fp32 logits."""
    live = chosen >= 0
    picked = logits.gather(1, chosen.clamp_min(0))
    if case["score"] == "softmax":
        score = torch.softmax(logits, 1).nan_to_num(0.0)  # no score in a row that is masked whole
        one = torch.where(live, score.gather(1, chosen.clamp_min(0)), 0.0)
        # normalised: the softmax of the chosen alone
        share = torch.softmax(torch.where(live, picked, -math.inf), 1).nan_to_num(0.0)
    else:
        score = torch.sigmoid(logits)
        one = torch.where(live, score.gather(1, chosen.clamp_min(0)), 0.0)
        share = one / (one.sum(1, keepdim=True) + WEIGHT_FLOOR)
    return (share if norm else one) * _scale_of(case), score, share


def _plain_route(s):
    case, logits = s["case"], s["logits"].float()
    chosen = _plain_chosen(case, logits, s["bias"])
    weights, score, share = _plain_weights(case, logits, chosen, case["norm"])
    if not case["step"]:
        return chosen, weights
    soft = case["score"] == "softmax"
    total = score.sum(1, keepdim=True)
    p = score if soft else (score / total).nan_to_num(0.0)
    sums = p.sum(0)
    slot = chosen.clamp_min(0)
    dw = torch.where(chosen >= 0, s["dweights"], 0.0) * _scale_of(case)
    dp = s["dsums"].expand_as(p)
    if soft:
        dscore = dp if case["norm"] else dp.scatter_add(1, slot, dw)
        dlogits = score * (dscore - (dscore * score).sum(1, keepdim=True))
        if case["norm"]:
            dlogits = dlogits.scatter_add(1, slot, share * (dw - (dw * share).sum(1, keepdim=True)))
    else:
        dscore = torch.where(total > 0, (dp - (dp * p).sum(1, keepdim=True)) / total, 0.0)
        if case["norm"]:
            one = torch.where(chosen >= 0, score.gather(1, slot), 0.0)
            dw = (dw - (dw * share).sum(1, keepdim=True)) / (one.sum(1, keepdim=True) + WEIGHT_FLOOR)
        dscore = dscore.scatter_add(1, slot, torch.where(chosen >= 0, dw, 0.0))
        dlogits = dscore * score * (1 - score)
    return chosen, weights, sums, dlogits.to(s["logits"].dtype)


def _weight_values(w, pick=None):
    """fp32 weights, of the picked experts where some are picked."""
    if not isinstance(w, tuple):
        return (w if pick is None else w[pick]).float()
    codes, scales = w if pick is None else (w[0][pick], w[1][pick])
    v = codes.float().view(-1, codes.shape[1] // BLOCK, BLOCK, codes.shape[2] // BLOCK, BLOCK)
    return (v * scales[:, :, None, :, None]).view(codes.shape)


def _plain_layer(s):
    case, x = s["case"], s["x"].float()
    T, H = x.shape
    E, K, I = case["E"], case["K"], case["I"]
    logits = (s["x"].double() @ s["w_router"].double().t()).float()
    chosen = _plain_chosen(case, logits, s["bias"])
    weights = _plain_weights(case, logits, chosen, True)[0]
    if T * K < E:  # fewer products than experts: those that are chosen, one by one
        pick = chosen.reshape(-1).clamp_min(0)
        g, u = torch.bmm(_weight_values(s["w13"], pick), x.repeat_interleave(K, 0)[:, :, None]).chunk(2, 1)
        z = torch.bmm(_weight_values(s["w2"], pick), g * torch.sigmoid(g) * u).view(T, K, H)
        y = (z * weights[:, :, None]).sum(1)
    else:
        gu = (x @ _weight_values(s["w13"]).view(-1, H).t()).view(T, E, 2 * I)
        g, u = gu.chunk(2, 2)
        dense = torch.zeros((T, E), device="cuda").scatter_add_(1, chosen.clamp_min(0), weights)
        act = (g * torch.sigmoid(g) * u * dense[:, :, None]).transpose(0, 1).contiguous()
        y = torch.bmm(act, _weight_values(s["w2"]).transpose(1, 2)).sum(0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16), chosen, weights


def _plain_adapter(s):
    case = s["case"]
    T, L, r, K, N = case["T"], case["L"], case["r"], case["K"], case["N"]
    x, down = s["x"].float(), s["down"].float().view(L * r, K)
    up = s["up"].float().transpose(1, 2).reshape(L * r, N)
    mine = (s["ids"][:, None] == torch.arange(L, device="cuda")).float() * s["scales"]
    mine = mine.repeat_interleave(r, 1)
    hidden = (x @ down.t()) * mine
    out = (s["base"].float() + hidden @ up).to(torch.bfloat16)
    if not case["step"]:
        return out
    dy = s["dy"].float()
    dhidden = (dy @ up.t()) * mine
    dx = (s["dx_base"].float() + dhidden @ down).to(torch.bfloat16)
    ddown = (dhidden.t() @ x).view(L, r, K).to(torch.bfloat16)
    dup = (dy.t() @ hidden).view(N, L, r).transpose(0, 1).contiguous().to(torch.bfloat16)
    return out, dx, ddown, dup


# ------------------------------------------------------------------- run

def _run_own(s):
    import combine_get_dispatch_05_amd as ep
    case = s["case"]
    if case["kind"] == "adapter":
        out, hidden = ep.adapter_product(s["x"], s["ids"], s["down"], s["up"], s["scales"], base=s["base"],
                                         save=case["step"])
        if not case["step"]:
            return out
        return (out, *ep.adapter_product_backward(s["dy"], s["x"], s["ids"], s["down"], s["up"], s["scales"], hidden,
                                                  dx_base=s["dx_base"]))
    rule = ep.Router(case["K"], score=case["score"], num_groups=case["G"], topk_groups=case["g"],
                     normalize=case.get("norm", True), scale=_scale_of(case))
    if case["kind"] == "layer":
        buf = ep.Buffer(1, case["E"])
        return buf.low_latency_moe(s["x"], s["w_router"], rule, s["w13"], s["w2"], bias=s["bias"],
                                   residual=s["residual"])
    buf = ep.Buffer(case["R"], case["E"])
    chosen, weights, sums = buf.route(s["logits"], rule, bias=s["bias"], score_sums=case["step"])
    if not case["step"]:
        return chosen, weights
    return chosen, weights, sums, buf.route_backward(s["dweights"], s["logits"], chosen, rule,
                                                     dscore_sums=s["dsums"])


def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "layer": _plain_layer, "adapter": _plain_adapter}[state["case"]["kind"]](state)


# ------------------------------------------------------------------ work

def work(case):
    kind, T = case["kind"], case["T"]
    if kind == "route":
        n = T * case["E"]
        size = 2 if case["bf16"] else 4
        nbytes, flops = n * size + T * case["K"] * 12, n * 6
        if case["step"]:  # the logits are read once for the choice and its gradient
            nbytes, flops = nbytes + n * size + T * case["K"] * 4 + case["E"] * 8, 3 * flops
        return {"bytes": nbytes, "flops": flops}
    if kind == "layer":
        H, I, E, K = case["H"], case["I"], case["E"], case["K"]
        reached = E * (1 - (1 - K / E) ** T)
        size = 1 + 4 / BLOCK ** 2 if case["fp8"] else 2
        return {"bytes": int(3 * H * I * size * reached + 2 * E * H + T * H * (6 if case["residual"] else 4)
                             + T * K * 12),
                "flops": 6 * T * K * H * I + 2 * T * E * H}
    r, K, N, L = case["r"], case["K"], case["N"], case["L"]
    reached = L * (1 - (1 - (1 - case["none"]) / L) ** T)
    nbytes = 2 * T * K + 4 * T * N + 8 * T + 2 * r * (K + N) * reached
    flops = 2 * T * (1 - case["none"]) * r * (K + N)
    if case["step"]:
        nbytes += 2 * T * N + 4 * T * K + 2 * L * r * (K + N)
        flops *= 3
    return {"bytes": int(nbytes), "flops": int(flops)}


# ----------------------------------------------------------------- exact

def _exact_route(case, logits, bias):
    """Chosen experts and scores from the definition; logits fp64 of the given values."""
    score = 1 / (1 + torch.exp(-logits))
    if case["score"] == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True).clamp_min(-1e300))
        score = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    key = logits if bias is None else score + bias.double()
    key = key.masked_fill(logits == -math.inf, -math.inf)
    T, E = key.shape
    if case["G"] > 1:
        size = E // case["G"]
        rank = []
        for n in range(case["G"]):
            top = key[:, n * size:(n + 1) * size].topk(min(2, size)).values
            two = top[:, 1] if bias is not None and size > 1 else torch.zeros_like(top[:, 0])
            rank.append(top[:, 0] + two.masked_fill(two == -math.inf, 0.0))
        rank = torch.stack(rank, 1)
        for n in range(case["G"]):
            ahead = (rank > rank[:, n:n + 1]).sum(1) + (rank[:, :n] == rank[:, n:n + 1]).sum(1)
            key[:, n * size:(n + 1) * size].masked_fill_((ahead >= case["g"])[:, None], -math.inf)
    chosen = torch.full((T, case["K"]), -1, device="cuda")
    for k in range(case["K"]):
        big = key.amax(1, keepdim=True)
        first = torch.where(key == big, torch.arange(E, device="cuda"), E).amin(1)
        chosen[:, k] = torch.where(big[:, 0] > -math.inf, first, -1)
        key = key.scatter(1, first[:, None], -math.inf)
    return chosen, score


def _exact_weights(case, score, chosen, norm):
    w = score.gather(1, chosen.clamp_min(0)).masked_fill(chosen < 0, 0.0)
    if norm:
        w = w / (w.sum(1, keepdim=True) + (WEIGHT_FLOOR if case["score"] == "sigmoid" else 0.0)).clamp_min(1e-300)
    return w * _scale_of(case)


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "route":
        logits = s["logits"].double()
        chosen, score = _exact_route(case, logits, s["bias"])
        if not case["step"]:
            return chosen, _exact_weights(case, score, chosen, case["norm"])
        x = logits.detach().clone()
        dead = x == -math.inf
        x = x.masked_fill(dead, 0.0).requires_grad_()
        if case["score"] == "softmax":
            score = torch.softmax(x.masked_fill(dead & ~dead.all(1, keepdim=True), -math.inf), 1)
            score = score.masked_fill(dead, 0.0)
            p = score
        else:
            score = torch.sigmoid(x).masked_fill(dead, 0.0)
            p = score / score.sum(1, keepdim=True).clamp_min(1e-300)
        weights = _exact_weights(case, score, chosen, case["norm"])
        live = (chosen >= 0).double()
        loss = (weights * live * s["dweights"].double()).sum() + (p.sum(0) * s["dsums"].double()).sum()
        loss.backward()
        return chosen, weights.detach(), p.detach().sum(0), x.grad
    if kind == "layer":
        x, T, I = s["x"].double(), case["T"], case["I"]
        logits = (x @ s["w_router"].double().t()).float().double()
        chosen, score = _exact_route(case, logits, s["bias"])
        weights = _exact_weights(case, score, chosen, True)
        y = s["residual"].double() if case["residual"] else torch.zeros((T, case["H"]), dtype=torch.float64, device="cuda")
        y = y.clone()

        def value(w, e):
            if not case["fp8"]:
                return w[e].double()
            return w[0][e].double() * w[1][e].double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)

        for e in sorted(set(chosen[chosen >= 0].tolist())):
            t, k = (chosen == e).nonzero(as_tuple=True)
            gu = x[t] @ value(s["w13"], e).t()
            act = gu[:, :I] / (1 + torch.exp(-gu[:, :I])) * gu[:, I:]
            y.index_add_(0, t, weights[t, k][:, None] * (act @ value(s["w2"], e).t()))
        return y, chosen, weights
    out = s["base"].double().clone()
    step = case["step"]
    if step:
        dx = s["dx_base"].double().clone()
        ddown, dup = torch.zeros_like(s["down"], dtype=torch.float64), torch.zeros_like(s["up"], dtype=torch.float64)
    for a in range(case["L"]):
        t = (s["ids"] == a).nonzero()[:, 0]
        x, A, B, c = s["x"][t].double(), s["down"][a].double(), s["up"][a].double(), s["scales"][a].double()
        h = x @ A.t()
        out[t] += c * (h @ B.t())
        if step:
            dy = s["dy"][t].double()
            dh = c * (dy @ B)
            dx[t] += dh @ A
            ddown[a], dup[a] = dh.t() @ x, c * (dy.t() @ h)
    return (out, dx, ddown, dup) if step else out
