"""The router against its definition in 64 bits: choices bit for bit (ties, gaps far
below fp32 rounding, masks, values that are not finite), weights, score sums and gradients.

Bounds: the roundings a value goes through at their worst, U = 2^-24 each.  An exponential
of x is off by |x| U from rounding x and by 2 U of its own; sums over a row are trees
of at most 40 terms deep (a wave's 6 levels, its 8 registers, a block's 4 waves)."""

from __future__ import annotations

import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402
from combine_get_dispatch_05_amd import abi  # noqa: E402

BF, U = 2.0 ** -8, 2.0 ** -24
INF = math.inf


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def scores(l, soft):
    """fp64 scores; rows that are masked whole have none."""
    if not soft:
        return torch.sigmoid(l)
    dead = (l == -INF).all(1, keepdim=True)
    return torch.softmax(l.masked_fill(dead, 0.0), 1).masked_fill(dead, 0.0)


def choose(l, r, bias=None, masked=()):
    """The definition, one expert at a time, on fp64 logits."""
    T, E = l.shape
    key = l.clone() if bias is None else scores(l, r.score == "softmax") + bias.double()
    off = (l == -INF) | l.isnan() | key.isnan()
    for e in masked:
        off[:, e] = True
    key[off] = -INF
    if r.num_groups > 1:
        size = E // r.num_groups
        by = key.view(T, r.num_groups, size)
        best = by.amax(2)
        if bias is not None and size > 1:
            second = by.topk(2, 2).values[..., 1]
            best = best + second.masked_fill(second == -INF, 0.0)
        order = best.sort(dim=1, descending=True, stable=True).indices[:, :r.topk_groups]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order, True)
        key = by.masked_fill(~keep[..., None], -INF).view(T, E)
    v, i = key.sort(dim=1, descending=True, stable=True)
    if r.num_topk > E:
        pad = r.num_topk - E
        v, i = torch.nn.functional.pad(v, (0, pad), value=-INF), torch.nn.functional.pad(i, (0, pad))
    v, i = v[:, :r.num_topk], i[:, :r.num_topk]
    return torch.where(v > -INF, i, -1)


def weigh(s, idx, r, l):
    one = s.gather(1, idx.clamp_min(0)).masked_fill(idx < 0, 0.0)
    if r.normalize and r.score == "softmax":
        p = torch.softmax(l.gather(1, idx.clamp_min(0)).masked_fill(idx < 0, -INF), 1)
        one = p.nan_to_num(0.0)
    elif r.normalize:
        one = one / (one.sum(1, keepdim=True) + 1e-20)
    return one * r.scale


def span(l):
    f = l[l.isfinite()]
    return float(f.max() - f.min()) if f.numel() else 0.0


def close(got, ref, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - tol
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} out, by up to {worst:.3g}"


def check(l, r, ranks=1, bias=None, masked_ranks=(), seed=0):
    """Choice, weights, sums and gradients of logits l (as given)."""
    T, E = l.shape
    buf = epm.Buffer(ranks, E)
    for rank in masked_ranks:
        buf.low_latency_update_mask_buffer(rank, True)
    ld, soft = l.double(), r.score == "softmax"
    masked = [e for e in range(E) if e // (E // ranks) in masked_ranks]
    idx, w, sums = buf.route(l, r, bias=bias, score_sums=True)
    ref = choose(ld, r, bias, masked)
    assert torch.equal(idx, ref), f"{int((idx != ref).any(1).sum())} of {T} tokens"
    s = scores(ld, soft)
    rel = (64 + 2 * span(ld)) * U
    wr = weigh(s, ref, r, ld)
    tiny = 2.0 ** -120  # where a share is below the normal numbers
    close(w, wr, wr.abs() * rel + tiny, "weights")
    total = s.sum(1, keepdim=True)
    p = s if soft else torch.where(total > 0, s / total, 0.0)
    close(sums, p.sum(0), p.sum(0) * (rel + (T + 16) * U) + tiny * (T + 1), "sums")
    plain = buf.route(l, r, bias=bias)
    assert torch.equal(plain[0], idx) and torch.equal(plain[1], w) and plain[2] is None
    # gradients, from the formulas
    g = gen(seed + 1)
    dw = torch.randn((T, r.num_topk), generator=g, device="cuda")
    for q in (None, torch.randn(E, generator=g, device="cuda")):
        dl = buf.route_backward(dw, l, idx, r, dscore_sums=q)
        assert dl.dtype == l.dtype and dl.shape == l.shape
        live = ref >= 0
        c = dw.double().masked_fill(~live, 0.0) * r.scale
        slot = ref.clamp_min(0)
        share = weigh(s, ref, epm.Router(r.num_topk, score=r.score), ld)
        qd = torch.zeros(E, dtype=torch.float64, device="cuda") if q is None else q.double()
        qd = qd.expand(T, E)
        one = s.gather(1, slot).masked_fill(~live, 0.0)
        if soft:
            ds, mag = qd, qd.abs()
            if not r.normalize:
                ds, mag = ds.scatter_add(1, slot, c), mag.scatter_add(1, slot, c.abs())
            refl = s * (ds - (ds * s).sum(1, keepdim=True))
            mag = s * (mag + (mag * s).sum(1, keepdim=True))
            if r.normalize:
                refl = refl.scatter_add(1, slot, share * (c - (c * share).sum(1, keepdim=True)))
                mag = mag.scatter_add(1, slot, share * (c.abs() + (c.abs() * share).sum(1, keepdim=True)))
        else:
            inv = torch.where(total > 0, 1 / total, 0.0)
            ds = (qd - (qd * p).sum(1, keepdim=True)) * inv
            mag = (qd.abs() + (qd.abs() * p).sum(1, keepdim=True)) * inv
            cc, cm = c, c.abs()
            if r.normalize:
                of = one.sum(1, keepdim=True) + 1e-20
                cc, cm = (c - (c * share).sum(1, keepdim=True)) / of, (c.abs() + (c.abs() * share).sum(1, keepdim=True)) / of
                cc, cm = cc.masked_fill(~live, 0.0), cm.masked_fill(~live, 0.0)
            ds, mag = ds.scatter_add(1, slot, cc), mag.scatter_add(1, slot, cm)
            refl = ds * s * (1 - s)
            mag = mag * s  # 1 - s is taken of a rounded s: its error is U of 1
        half = BF if l.dtype == torch.bfloat16 else U
        close(dl, refl, refl.abs() * half + mag * 2 * rel + tiny, f"dlogits, sums {q is not None}")
    return idx, w


CASES = [  # T, E, ranks, router, bias, bf16, mask
    (1, 1, 1, epm.Router(1), False, False, 0.0),
    (5, 3, 1, epm.Router(3, score="sigmoid"), True, False, 0.0),
    (33, 8, 4, epm.Router(2, normalize=False), False, True, 0.0),
    (7, 63, 3, epm.Router(5), False, False, 0.2),
    (9, 65, 5, epm.Router(6, score="sigmoid", normalize=False, scale=2.5), True, False, 0.0),
    (130, 128, 8, epm.Router(4, num_groups=4, topk_groups=2), False, True, 0.1),
    (1, 256, 32, epm.Router(8, score="sigmoid", num_groups=8, topk_groups=4, scale=2.5), True, False, 0.0),
    (2051, 256, 32, epm.Router(8, score="sigmoid", num_groups=8, topk_groups=4, scale=2.5), True, False, 0.0),
    (1025, 256, 64, epm.Router(8), False, False, 0.0),
    (601, 288, 144, epm.Router(6, normalize=False), True, True, 0.1),
    (65, 320, 4, epm.Router(8, num_groups=5, topk_groups=3), True, False, 0.7),
    (40, 384, 2, epm.Router(64, num_groups=64, topk_groups=9), False, False, 0.0),  # 54 left for 64 slots
    (300, 512, 512, epm.Router(64, score="sigmoid"), True, False, 0.0),
    (3, 512, 1, epm.Router(1, num_groups=2, topk_groups=1, score="sigmoid", normalize=False), False, False, 0.0),
    (70, 520, 8, epm.Router(8, num_groups=8, topk_groups=3), True, False, 0.1),  # a block a token
    (3, 8192, 512, epm.Router(64, score="sigmoid", num_groups=64, topk_groups=10), True, True, 0.0),
    (2, 1000, 1, epm.Router(9, normalize=False), False, False, 0.99),
    (6, 4, 4, epm.Router(7), False, False, 0.3),  # more slots than experts
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_route(case):
    T, E, ranks, r, with_bias, bf16, mask = CASES[case]
    g = gen(100 + case)
    l = torch.randn((T, E), generator=g, device="cuda") * 2
    l[torch.rand((T, E), generator=g, device="cuda") < mask] = -INF
    bias = torch.randn(E, generator=g, device="cuda") * 0.3 if with_bias else None
    check(l.to(torch.bfloat16) if bf16 else l, r, ranks, bias, seed=case)


@pytest.mark.parametrize("E", [24, 256, 600])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_ranks_ties_and_empty_rows(E, score, with_bias):
    g = gen(E)
    r = epm.Router(6, score=score, num_groups=4, topk_groups=2, scale=1.5)
    l = (torch.randint(-2, 3, (50, E), generator=g, device="cuda") * 0.5)  # ties everywhere
    l[7] = -INF
    l[8, 1:] = -INF
    l[9] = 3.0
    l[10, :E // 2] = -INF
    bias = torch.randint(-1, 2, (E,), generator=g, device="cuda") * 0.25 if with_bias else None
    idx, w = check(l, r, 8, bias, masked_ranks=(0, 5))
    assert (idx[7] == -1).all() and (w[7] == 0).all()  # nothing to choose
    assert (idx[8] == -1).all()  # its one expert sits on a masked rank
    everyone = epm.Buffer(8, E)
    for rank in range(8):
        everyone.low_latency_update_mask_buffer(rank, True)
    idx, w, _ = everyone.route(l, r, bias=bias)
    assert (idx == -1).all() and (w == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [2, 70, 700])
def test_gaps_far_below_fp32_are_decided(E, score):
    """Two experts ahead of all others, whose keys are equal in fp32 and differ in 64 bits."""
    g = gen(3)
    T = 400
    l = torch.full((T, E), -9.0, device="cuda")
    a = 4 + torch.rand(T, generator=g, device="cuda") * 4
    b = a.clone()
    for _ in range(2):  # two steps of fp32 away: scores 1e-8 to 1e-10 apart
        b = torch.where(torch.rand(T, generator=g, device="cuda") < 0.5, torch.nextafter(b, b + 1), b)
    flip = torch.rand(T, generator=g, device="cuda") < 0.5
    l[:, 0], l[:, E - 1] = torch.where(flip, b, a), torch.where(flip, a, b)
    bias = torch.full((E,), 0.25, device="cuda")
    r = epm.Router(1, score=score)
    idx, _, _ = epm.Buffer(1, E).route(l, r, bias=bias)
    assert torch.equal(idx, choose(l.double(), r, bias))
    assert 0 < int((idx == E - 1).sum()) < T
    if E % 2 == 0:  # the same gap between two groups
        r = epm.Router(1, score=score, num_groups=2, topk_groups=1)
        idx, _, _ = epm.Buffer(1, E).route(l, r, bias=bias)
        assert torch.equal(idx, choose(l.double(), r, bias))


@pytest.mark.parametrize("E", [40, 640])
def test_values_that_are_not_finite(E):
    l = torch.zeros((4, E), device="cuda")
    l[0, 3] = math.nan
    l[1, 5] = INF
    l[2, 2], l[2, 4] = 200.0, -200.0
    buf = epm.Buffer(1, E)
    for r in (epm.Router(3, score="sigmoid"), epm.Router(3, score="sigmoid", num_groups=4, topk_groups=4)):
        idx, w, _ = buf.route(l, r)
        assert idx.tolist() == [[0, 1, 2], [5, 0, 1], [2, 0, 1], [0, 1, 2]]
        assert torch.allclose(w[1], torch.tensor([0.5, 0.25, 0.25], device="cuda"))
        assert torch.allclose(w[0], torch.full((3,), 1 / 3, device="cuda"))
    idx, w, _ = buf.route(l, epm.Router(3, normalize=False))
    assert idx.tolist() == [[0, 1, 2], [5, 0, 1], [2, 0, 1], [0, 1, 2]]
    assert w[0].isnan().all() and w[1].isnan().any() and w[2, 0] == 1 and (w[3] == 1 / E).all()
    # a bias that is not finite: NaN keys are not chosen, +inf goes first
    bias = torch.zeros(E, device="cuda")
    bias[0], bias[7], bias[1] = math.nan, INF, -INF
    idx, _, _ = buf.route(l[3:], epm.Router(3, score="sigmoid"), bias=bias)
    assert idx.tolist() == [[7, 2, 3]]


def test_no_tokens_and_refusals():
    buf, r = epm.Buffer(2, 8), epm.Router(2)
    idx, w, sums = buf.route(torch.zeros((0, 8), device="cuda"), r, score_sums=True)
    assert idx.shape == (0, 2) and w.shape == (0, 2) and (sums == 0).all()
    assert buf.route_backward(w, torch.zeros((0, 8), device="cuda"), idx, r).shape == (0, 8)
    l = torch.zeros((4, 8), device="cuda")
    idx, w, _ = buf.route(l, r)
    for bad in (lambda: buf.route(l[:, :4], r), lambda: buf.route(l.t(), r),
                lambda: buf.route(l, r, bias=torch.zeros(7, device="cuda")),
                lambda: buf.route(l, epm.Router(2, score="relu")),
                lambda: buf.route_backward(w[:3], l, idx, r), lambda: buf.route_backward(w, l, idx[:3], r),
                lambda: buf.route_backward(w, l, idx, r, dscore_sums=w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (epm.Router(0), epm.Router(65), epm.Router(2, num_groups=3), epm.Router(2, num_groups=2, topk_groups=3)):
        with pytest.raises(abi.EpError):
            buf.route(l, bad)
    with pytest.raises(TypeError):
        buf.route_backward(w, l, idx.int(), r)
    # ids that name no expert, and one expert twice
    odd = torch.tensor([[-5, 99], [1, 1], [0, 1 << 40], [3, -1]], device="cuda")
    dl = buf.route_backward(torch.ones_like(w), l, odd, epm.Router(2, score="sigmoid", normalize=False))
    want = torch.zeros((4, 8), device="cuda")
    want[1, 1], want[2, 0], want[3, 3] = 0.5, 0.25, 0.25
    assert torch.equal(dl, want)


def test_gradient_against_differences():
    """The loss itself in 64 bits, moved along a direction."""
    T, E = 20, 32
    g = gen(9)
    l = torch.randn((T, E), generator=g, device="cuda")
    dw = torch.randn((T, 4), generator=g, device="cuda")
    q = torch.randn(E, generator=g, device="cuda")
    d = torch.randn((T, E), generator=g, device="cuda", dtype=torch.float64)
    for score in ("softmax", "sigmoid"):
        for normalize in (True, False):
            r = epm.Router(4, score=score, normalize=normalize, scale=1.5)
            buf = epm.Buffer(1, E)
            idx, _, _ = buf.route(l, r, score_sums=True)
            dl = buf.route_backward(dw, l, idx, r, dscore_sums=q).double()

            def loss(x):
                s = scores(x, score == "softmax")
                return (weigh(s, idx, r, x) * dw).sum() + ((s / s.sum(1, keepdim=True)).sum(0) * q).sum()
            h = 1e-5
            slope = (loss(l.double() + h * d) - loss(l.double() - h * d)) / (2 * h)
            assert abs(float((dl * d).sum() - slope)) < 1e-4 * float((dl * d).abs().sum())
