"""The router where a choice or a gradient hangs on what fp32 drops, against its definition in 64 bits."""

from __future__ import annotations

import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402
from test_gpu_router import choose, close, gen, weigh  # noqa: E402

U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


def cancelling(E, groups, size):
    """A bias of +size and -size on the first two experts of every second group, whose sum is then small and
    whose keys are not; of none on the first two of the others."""
    bias = torch.full((groups, E // groups), -3 * size, device="cuda")  # so that those two are a group's best
    bias[:, :2] = 0
    bias[::2, 0], bias[::2, 1] = size, -size
    return bias.view(E)


@pytest.mark.parametrize("size", [256.0, 1000.0, 1e5, 1e6])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,kept", [(4, 2, 1), (24, 8, 3), (256, 4, 2), (512, 64, 20), (1024, 4, 2)])
def test_biases_that_cancel_inside_a_group(E, groups, kept, score, size):
    g = gen(E)
    T = 4000
    # scores of neighbouring groups some 2^-24 of the biases apart
    l = 0.3 + torch.randn((T, E), generator=g, device="cuda") * size * 1e-6
    r = epm.Router(kept, score=score, num_groups=groups, topk_groups=kept)
    bias = cancelling(E, groups, size)
    want = choose(l.double(), r, bias)
    idx, _, _ = epm.Buffer(1, E).route(l, r, bias=bias)
    assert torch.equal(idx, want), f"{int((idx != want).any(1).sum())} of {T} tokens"


@pytest.mark.parametrize("T", [1, 5, 64])
def test_the_layer_with_biases_that_cancel_inside_a_group(T):
    E, H, I = 4, 64, 8
    g = gen(T)
    r = epm.Router(1, score="sigmoid", num_groups=2, topk_groups=1)
    wr = torch.zeros((E, H), device="cuda")
    wr[:, 0] = 0.3
    wr[:, 1:] = torch.randn((E, H - 1), generator=g, device="cuda") * 0.0125
    w13 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros((E, H, I), dtype=torch.bfloat16, device="cuda")
    bias, buf = cancelling(E, 2, 1e5), epm.Buffer(1, E)
    for _ in range(1000 // T):
        x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
        x[:, 0] = 1
        want = choose((x.double() @ wr.double().t()).float().double(), r, bias)
        _, idx, _ = buf.low_latency_moe(x, wr, r, w13, w2, bias=bias)
        assert torch.equal(idx, want)


@pytest.mark.parametrize("E", [12, 128, 512, 600])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("with_sums", [False, True])
def test_sigmoid_gradient_of_large_logits(E, normalize, with_sums):
    """s (1 - s) keeps its digits on both sides.  The slope of a logit is exact but for its exponential (2 U), a sum, a
    square and a quotient (5 U with what the sum's rounding does in the square); a choice's part of ds is a product, normalised a difference of
    the slot's own gradient and the mean over 6 slots, over their sum; the sums' part one of a mean over E."""
    g = gen(E)
    T, K = 30, 6
    l = torch.tensor([-80.0, -30, -17, -16, -10, 0, 10, 16, 17, 20, 30, 80], device="cuda").repeat(T, -(-E // 12))[:, :E]
    l = (l + torch.rand((T, E), generator=g, device="cuda")).gather(1, torch.rand((T, E), generator=g, device="cuda").argsort(1))
    r = epm.Router(K, score="sigmoid", normalize=normalize, scale=1.5)
    buf = epm.Buffer(1, E)
    idx = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :K].contiguous()  # any experts, not the largest alone
    dw = torch.randn((T, K), generator=g, device="cuda")
    q = torch.randn(E, generator=g, device="cuda") if with_sums else None
    dl = buf.route_backward(dw, l, idx, r, dscore_sums=q)
    ld = l.double()
    s = torch.sigmoid(ld)
    slope = s * torch.sigmoid(-ld)
    c = dw.double() * r.scale
    mag = c.abs()
    if normalize:
        share = weigh(s, idx, epm.Router(K, score="sigmoid"), ld)
        of = s.gather(1, idx).sum(1, keepdim=True) + 1e-20
        c, mag = (c - (c * share).sum(1, keepdim=True)) / of, (mag + (mag * share).sum(1, keepdim=True)) / of
    ds = torch.zeros_like(ld).scatter_add(1, idx, c)
    mag = torch.zeros_like(ld).scatter_add(1, idx, mag)
    if with_sums:
        total, p = s.sum(1, keepdim=True), s / s.sum(1, keepdim=True)
        ds = ds + (q.double() - (q.double() * p).sum(1, keepdim=True)) / total
        mag = mag + (q.double().abs() + (q.double().abs() * p).sum(1, keepdim=True)) / total
    # (sums over a row: at most 40 terms deep)
    rel = 16 * U if not (normalize or with_sums) else 128 * U
    close(dl, ds * slope, mag * slope * rel + 2.0 ** -120, "dlogits")
    if not (normalize or with_sums):
        got = dl.gather(1, idx)[(dw.abs() > 0.01) & (l.gather(1, idx).abs() < 60)]
        assert (got != 0).all()


@pytest.mark.parametrize("E", [40, 640])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_softmax_rows_that_are_not_finite(E, bad):
    """Scores that are NaN are no keys beside a bias; weights of the chosen alone do not see a NaN that is not chosen."""
    l = torch.arange(E, device="cuda").flip(0).float().repeat(2, 1) / E
    l[0, 5] = bad
    buf, none = epm.Buffer(1, E), torch.zeros(E, device="cuda")
    for normalize in (False, True):
        r = epm.Router(3, normalize=normalize)
        idx, w, sums = buf.route(l, r, bias=none, score_sums=True)
        assert (idx[0] == -1).all() and (w[0] == 0).all() and idx[1].tolist() == [0, 1, 2]
        assert sums.isnan().all()
        idx, w, sums = buf.route(l, r, score_sums=True)
        assert idx.tolist() == [[5, 0, 1] if bad == math.inf else [0, 1, 2], [0, 1, 2]] and sums.isnan().all()
        assert w[1].isfinite().all()
        if bad == math.inf or not normalize:
            assert w[0].isnan().all()
        else:
            assert torch.equal(w[0], w[1])


@pytest.mark.parametrize("E", [40, 640])
def test_sigmoid_rows_with_a_nan_leave_the_others_choice_and_weights(E):
    l = torch.zeros((2, E), device="cuda")
    l[0, 1] = math.nan
    buf, r = epm.Buffer(1, E), epm.Router(2, score="sigmoid", normalize=False)
    for bias in (None, torch.zeros(E, device="cuda")):
        idx, w, sums = buf.route(l, r, bias=bias, score_sums=True)
        assert idx.tolist() == [[0, 2], [0, 1]] and (w == 0.5).all() and sums.isnan().all()


def centred(p, v):
    """p_i sum_j p_j (v_i - v_j) for weights p whose sum is one, and the magnitudes: no difference from a mean, so that it keeps
    its digits where one weight is nearly one."""
    d = v[:, :, None] - v[:, None, :]
    m = (v.abs()[:, :, None] + v.abs()[:, None, :]) * (1 - torch.eye(v.shape[1], dtype=v.dtype, device=v.device))
    return p * (d * p[:, None, :]).sum(2), p * (m * p[:, None, :]).sum(2)


@pytest.mark.parametrize("E", [12, 128, 512, 600])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("with_sums", [False, True])
def test_gradient_where_one_expert_is_nearly_everything(E, score, normalize, with_sums):
    """One logit some 16 to 30 past all others: what is left of its gradient is of the others' size.  Scores are off by
    (64 + 2 span) U, sums over a row are at most 40 terms deep; a difference is off by what its two sides are, here taken
    without the part that they have in common."""
    g = gen(E)
    T, K, soft = 40, 5, score == "softmax"
    l = torch.randn((T, E), generator=g, device="cuda")
    top = torch.randint(0, E, (T, 1), generator=g, device="cuda")
    gap = 16 + 14 * torch.rand((T, 1), generator=g, device="cuda")
    l = (l if soft else l - gap - 8).scatter(1, top, gap if soft else torch.randn((T, 1), generator=g, device="cuda") - 4)
    buf, r = epm.Buffer(1, E), epm.Router(K, score=score, normalize=normalize, scale=1.5)
    idx, _, _ = buf.route(l, r)
    assert (idx[:, :1] == top).all()
    dw = torch.randn((T, K), generator=g, device="cuda")
    q = torch.randn(E, generator=g, device="cuda") if with_sums else None
    dl = buf.route_backward(dw, l, idx, r, dscore_sums=q)
    ld = l.double()
    s = torch.softmax(ld, 1) if soft else torch.sigmoid(ld)
    p = s / s.sum(1, keepdim=True)
    c = dw.double() * r.scale
    qd = q.double().expand(T, E) if with_sums else torch.zeros((T, E), dtype=torch.float64, device="cuda")
    one = s.gather(1, idx)
    share = one / one.sum(1, keepdim=True)
    if soft:
        ref, mag = centred(p, qd if normalize else qd.scatter_add(1, idx, c))
        if normalize:
            a, m = centred(share, c)
            ref, mag = ref.scatter_add(1, idx, a), mag.scatter_add(1, idx, m)
    else:
        a, m = centred(p, qd)  # p (q - sum q p): over p and the sum of the scores, which is over s
        ref, mag = a / s, m / s
        a, m = c, c.abs()
        if normalize:  # (beside the sum of the chosen, 1e-20 leaves that much of each c)
            of = one.sum(1, keepdim=True) + 1e-20
            a, m = centred(share, c)
            a, m = (a / share + c * (1e-20 / of)) / of, (m / share + c.abs() * (1e-20 / of)) / of
        slope = s * torch.sigmoid(-ld)
        ref, mag = ref.scatter_add(1, idx, a) * slope, mag.scatter_add(1, idx, m) * slope
    rel = (64 + 2 * float(l.max() - l.min())) * U
    close(dl, ref, mag * 2 * rel + 2.0 ** -120, "dlogits")


@pytest.mark.parametrize("E", [48, 384, 960])
@pytest.mark.parametrize("low", [torch.finfo(torch.float32).min, -3e38])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_barred_experts_come_before_those_that_cannot_be_chosen(E, low, score):
    """A bias near the lowest number bars experts; two of a group sum to less than fp32 holds.  Groups on masked ranks have
    no expert at all and come after them, wherever they lie."""
    g = gen(E)
    l = torch.randn((300, E), generator=g, device="cuda")
    bias = torch.zeros(E, device="cuda")
    size = E // 24
    for group in (2, 3, 7, 8, 9, 15, 20):
        bias[group * size:(group + 1) * size] = low
    masked = [0, 1, 4, 5, 6, 10, 11, 16, 17, 18, 21, 22, 23]  # groups, which are ranks here; 12, 13, 14 and 19 are as usual
    off = [e for e in range(E) if e // size in masked]
    buf = epm.Buffer(24, E)
    for rank in masked:
        buf.low_latency_update_mask_buffer(rank, True)
    for kept in (3, 5, 8, 11, 13):
        r = epm.Router(min(64, 12 * size), score=score, num_groups=24, topk_groups=kept)
        idx, _, _ = buf.route(l, r, bias=bias)
        assert torch.equal(idx, choose(l.double(), r, bias, off)), kept
