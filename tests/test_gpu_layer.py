"""The mixture-of-experts layer for a few tokens against its definition in 64 bits.

Bounds, per element: sums of n terms 2 (n + 8) U of the summed magnitudes (matrix instructions need
not round to nearest inside), the activation's rounding (to bf16, half a step of 2^-8, beside FP8 weights; to the
sum of two such values beside bf16 ones) and the result's.  The FP8 products are exact here (codes
widened to bf16), so the same bounds hold."""

from __future__ import annotations

import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402
from combine_get_dispatch_05_amd import abi  # noqa: E402
from test_gpu_experts import fp8_weight, weight_value  # noqa: E402
from test_gpu_router import choose, gen, scores, weigh  # noqa: E402

BF, U = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


def normal(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def made(T, H, I, E, fp8=False, f32=False, seed=0):
    g = gen(seed)
    x = normal(g, (T, H))
    wr = torch.randn((E, H), generator=g, device="cuda") * 1.5 / math.sqrt(H)
    wr = wr if f32 else wr.to(torch.bfloat16)
    if fp8:
        w13, w2 = fp8_weight(g, (E, 2 * I, H)), fp8_weight(g, (E, H, I))
    else:
        w13, w2 = normal(g, (E, 2 * I, H), 1 / math.sqrt(H)), normal(g, (E, H, I), 1 / math.sqrt(I))
    return x, wr, w13, w2


def reference(x, wr, r, w13, w2, bias=None, residual=None, masked=()):
    """(y, bound, idx, weights)"""
    T, H = x.shape
    l = (x.double() @ wr.double().t()).float().double()
    idx = choose(l, r, bias, masked)
    wt = weigh(scores(l, r.score == "softmax"), idx, r, l)
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    if residual is not None:
        y += residual.double()
    err = y.abs() * U
    value = (lambda w, e: weight_value((w[0][e], w[1][e]))) if isinstance(w13, tuple) else (lambda w, e: w[e].double())
    for e in sorted(set(idx[idx >= 0].tolist())):
        t, k = (idx == e).nonzero(as_tuple=True)
        a, b = value(w13, e), value(w2, e)
        I = b.shape[1]
        xe, p = x[t].double(), wt[t, k][:, None]
        gu, mag = xe @ a.t(), xe.abs() @ a.abs().t() * (2 * (H + 8) * U)
        g, u = gu[:, :I], gu[:, I:]
        s = torch.sigmoid(g)
        act = g * s * u
        kept = BF if isinstance(w13, tuple) else BF * BF
        ea = 1.1 * mag[:, :I] * (u.abs() + mag[:, I:]) + (g * s).abs() * mag[:, I:] + act.abs() * (kept + 16 * U)
        y.index_add_(0, t, p * (act @ b.t()))
        most = (act.abs() + ea) @ b.abs().t()
        err.index_add_(0, t, p * (ea @ b.abs().t() + most * (2 * (I + 8) * U + 200 * U)))
    return y, err + y.abs() * (BF + (r.num_topk + 4) * U) + 2.0 ** -120, idx, wt


def check(x, wr, r, w13, w2, ranks=1, masked_ranks=(), **kw):
    E = wr.shape[0]
    buf = epm.Buffer(ranks, E)
    for rank in masked_ranks:
        buf.low_latency_update_mask_buffer(rank, True)
    y, idx, wt = buf.low_latency_moe(x, wr, r, w13, w2, **kw)
    masked = [e for e in range(E) if e // (E // ranks) in masked_ranks]
    ref, bound, ridx, rwt = reference(x, wr, r, w13, w2, masked=masked, **kw)
    assert torch.equal(idx, ridx)
    assert ((wt - rwt).abs() <= rwt * 200 * U + 2.0 ** -120).all()
    assert torch.isfinite(y).all()
    over = (y.double() - ref).abs() - bound
    assert float(over.max()) <= 0, f"{int((over > 0).sum())} of {over.numel()} out, by up to {float(over.max()):.3g}"
    return y, idx, wt


SIGMOID = dict(score="sigmoid", num_groups=4, topk_groups=2, scale=2.5)
SHAPES = [  # T, H, I, E, router, bias, fp8, fp32 router, residual
    (1, 8, 8, 1, epm.Router(1), False, False, False, False),
    (1, 2048, 768, 64, epm.Router(8), False, False, False, True),
    (2, 200, 24, 5, epm.Router(3), True, False, True, False),
    (3, 1000, 520, 24, epm.Router(3), False, False, False, False),
    (7, 136, 72, 8, epm.Router(8), False, False, False, True),  # every expert has every token
    (8, 512, 128, 32, epm.Router(4, **SIGMOID), True, False, False, False),
    (9, 264, 264, 6, epm.Router(2), False, False, True, True),
    (17, 72, 1032, 3, epm.Router(1), False, False, False, False),
    (33, 128, 64, 2, epm.Router(2), False, False, False, True),  # 33 rows an expert
    (64, 320, 160, 4, epm.Router(3), True, False, False, False),  # 48
    (64, 256, 96, 1, epm.Router(1), False, False, False, True),  # 64
    (64, 2048, 256, 512, epm.Router(10), False, False, False, True),
    (64, 64, 16, 320, epm.Router(64), False, False, False, False),  # 4096 pairs
    (1, 128, 128, 4, epm.Router(2), False, True, False, False),
    (1, 7168, 2048, 16, epm.Router(8, **SIGMOID), True, True, False, True),
    (5, 384, 1152, 12, epm.Router(4, normalize=False), False, True, True, True),
    (20, 1280, 256, 8, epm.Router(2), True, True, False, False),
    (64, 512, 384, 2, epm.Router(2), False, True, False, True),
    (40, 256, 128, 130, epm.Router(6), False, True, False, False),
    (1, 256, 64, 200, epm.Router(8, **SIGMOID), True, False, False, False),
    (1, 128, 40, 512, epm.Router(64), False, False, True, True),
    (6, 256, 64, 132, epm.Router(4, **SIGMOID), True, False, False, True),
    (8, 128, 64, 512, epm.Router(10), False, False, False, False),
    (4, 256, 128, 300, epm.Router(12), True, True, False, True),
    (8, 192, 320, 100, epm.Router(4), False, False, False, False),  # 320 blocks of the gate
    (8, 192, 256, 100, epm.Router(4), False, False, False, False),  # 256
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_layer(case):
    T, H, I, E, r, with_bias, fp8, f32, res = SHAPES[case]
    x, wr, w13, w2 = made(T, H, I, E, fp8, f32, case)
    g = gen(1000 + case)
    bias = torch.randn(E, generator=g, device="cuda") * 0.2 if with_bias else None
    check(x, wr, r, w13, w2, bias=bias, residual=normal(g, (T, H), 2.0) if res else None)


def test_a_token_alone_and_in_any_batch_takes_the_same_experts():
    x, wr, w13, w2 = made(64, 1024, 64, 48, seed=5)
    wr[7] = wr[30]  # two experts that every token likes equally: the lower one goes first
    r = epm.Router(6, score="sigmoid")
    buf = epm.Buffer(1, 48)
    _, idx, wt = buf.low_latency_moe(x, wr, r, w13, w2)
    for T in (1, 2, 7, 8, 9, 33):
        _, i, w = buf.low_latency_moe(x[:T].contiguous(), wr, r, w13, w2)
        assert torch.equal(i, idx[:T]) and torch.equal(w, wt[:T]), T
    for row in idx.tolist():
        assert (30 not in row) or row.index(7) < row.index(30)


def test_masked_ranks_and_tokens_with_nothing():
    x, wr, w13, w2 = made(10, 256, 64, 16, seed=6)
    res = normal(gen(3), (10, 256))
    check(x, wr, epm.Router(4), w13, w2, ranks=8, masked_ranks=(0, 3), residual=res)
    buf = epm.Buffer(8, 16)
    for rank in range(8):
        buf.low_latency_update_mask_buffer(rank, True)
    for residual in (res, None):  # no expert at all: the residual alone
        y, idx, wt = buf.low_latency_moe(x, wr, epm.Router(4), w13, w2, residual=residual)
        assert (idx == -1).all() and (wt == 0).all()
        assert torch.equal(y, res if residual is not None else torch.zeros_like(y))
    # a token whose logits are NaN gets no expert and disturbs nobody
    good = epm.Buffer(1, 16).low_latency_moe(x, wr, epm.Router(4), w13, w2, residual=res)
    bad = x.clone()
    bad[3] = math.nan
    y, idx, wt = epm.Buffer(1, 16).low_latency_moe(bad, wr, epm.Router(4), w13, w2, residual=res)
    assert (idx[3] == -1).all() and torch.equal(y[3], res[3])
    rest = [t for t in range(10) if t != 3]
    assert torch.equal(idx[rest], good[1][rest])
    assert (y[rest].float() - good[0][rest].float()).abs().max() < 0.1


def test_experts_that_nobody_chose_may_hold_anything():
    x, wr, w13, w2 = made(4, 256, 64, 16, seed=7)
    buf, r = epm.Buffer(1, 16), epm.Router(2)
    y, idx, _ = buf.low_latency_moe(x, wr, r, w13, w2)
    unused = [e for e in range(16) if e not in set(idx.flatten().tolist())]
    assert unused
    w13[unused], w2[unused] = math.nan, math.inf
    again, _, _ = buf.low_latency_moe(x, wr, r, w13, w2)
    assert torch.equal(y, again)


@pytest.mark.parametrize("T", [1, 5, 12])
def test_an_activation_past_the_largest_number_is_infinite_and_alone(T):
    x, wr, w13, w2 = made(T, 256, 64, 16, seed=8)
    wr[:, 0] = 0
    w13[:], w13[:, 0, 0], w13[:, 64, 0] = 0, 1, 1  # act is (x0 silu(x0), 0, 0, ..)
    w2[:, :128, 0], w2[:, 128:, 0] = 1, -1
    buf, r = epm.Buffer(1, 16), epm.Router(2, normalize=True)
    x[:, 0] = 2.0 ** 10
    one, idx, _ = buf.low_latency_moe(x, wr, r, w13, w2)
    x[T - 1, 0] = 2.0 ** 70
    y, again, _ = buf.low_latency_moe(x, wr, r, w13, w2)
    assert torch.equal(idx, again) and torch.equal(y[:T - 1], one[:T - 1])
    want = torch.full((256,), math.inf, device="cuda", dtype=torch.bfloat16)
    want[128:] = -math.inf
    assert torch.equal(y[T - 1], want)


def test_refusals_and_no_tokens():
    x, wr, w13, w2 = made(4, 256, 64, 8)
    buf, r = epm.Buffer(1, 8), epm.Router(2)
    y, idx, wt = buf.low_latency_moe(x[:0], wr, r, w13, w2)
    assert y.shape == (0, 256) and idx.shape == (0, 2) and wt.shape == (0, 2)
    for bad in (lambda: buf.low_latency_moe(x, wr[:4], r, w13, w2), lambda: buf.low_latency_moe(x, wr, r, w13[:4], w2),
                lambda: buf.low_latency_moe(x, wr, r, w13, w2[:, :, :32]),
                lambda: buf.low_latency_moe(x, wr, r, w13, w2, residual=x[:2]),
                lambda: buf.low_latency_moe(x, wr, r, w13, w2, bias=torch.zeros(4, device="cuda")),
                lambda: buf.low_latency_moe(x.t(), wr, r, w13, w2)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        buf.low_latency_moe(x, wr, r, fp8_weight(gen(0), (8, 128, 256)), w2)
    with pytest.raises(abi.EpError, match="needs more"):
        buf.low_latency_moe(torch.zeros((65, 256), dtype=torch.bfloat16, device="cuda"), wr, r, w13, w2)
    with pytest.raises(abi.EpError):
        buf.low_latency_moe(x, wr, epm.Router(0), w13, w2)
