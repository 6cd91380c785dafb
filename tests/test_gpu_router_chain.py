"""The router, the few-token layer and the adapters in use: a training step from logits to their
gradient, a decode step beside the operations it replaces, captured graphs, streams, tensors past 4 GB."""

from __future__ import annotations

import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402
from test_gpu_adapter import check as check_adapter, made as made_adapter  # noqa: E402
from test_gpu_experts import fp8_rows, fp8_weight  # noqa: E402
from test_gpu_layer import check as check_layer, made as made_layer, reference  # noqa: E402
from test_gpu_router import choose, gen, scores, weigh  # noqa: E402

BF, U = 2.0 ** -8, 2.0 ** -24
SIGMOID = epm.Router(4, score="sigmoid", num_groups=4, topk_groups=2, scale=2.5)


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


def normal(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_training_step_from_logits_to_their_gradient(score):
    """route, dispatch, experts, combine and all the way back: the weights' gradient that arrives at the router is the
    definition's, and so is the logits'."""
    T, H, I, E, R, K = 97, 128, 64, 16, 4, 3
    g = gen(11)
    x, w13, w2 = normal(g, (T, H)), normal(g, (E, 2 * I, H), 1 / math.sqrt(H)), normal(g, (E, H, I), 1 / math.sqrt(I))
    logits, dout = torch.randn((T, E), generator=g, device="cuda"), normal(g, (T, H))
    r = epm.Router(K, score=score, scale=1.5)
    buf = epm.Buffer(R, E)
    idx, weights, _ = buf.route(logits, r)
    recv, rti, rtw, _, handle, _ = buf.dispatch(x, idx, weights)
    rows = buf.expert_rows(rti, handle)
    y, saved = buf.expert_ffn(recv, rows, rtw, w13, w2, save=True)
    out, back, _ = buf.combine(y, handle, rtw)
    assert torch.equal(back, weights)  # every slot's weight came round once
    dy, _, _, _, _, _ = buf.dispatch(dout, handle=handle)
    dx, drw, _, _ = buf.expert_ffn_backward(dy, recv, rows, rtw, w13, w2, saved)
    _, dweights, _ = buf.combine(dx, handle, drw)
    dlogits = buf.route_backward(dweights, logits, idx, r)
    handle.free()

    f64 = dict(dtype=torch.float64, device="cuda")
    dw, dw_err, ref_out, out_err = torch.zeros((T, K), **f64), torch.zeros((T, K), **f64), torch.zeros((T, H), **f64), \
        torch.zeros((T, H), **f64)
    sum_err = lambda n: 2 * (n + 8) * U  # noqa: E731
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        a, b, xe, de = w13[e].double(), w2[e].double(), x[t].double(), dout[t].double()
        gu, mag = xe @ a.t(), xe.abs() @ a.abs().t() * sum_err(H)
        sig = torch.sigmoid(gu[:, :I])
        act = gu[:, :I] * sig * gu[:, I:]
        ea = 1.1 * mag[:, :I] * (gu[:, I:].abs() + mag[:, I:]) + (gu[:, :I] * sig).abs() * mag[:, I:] + act.abs() * 16 * U
        d, ed = de @ b, de.abs() @ b.abs() * sum_err(H)
        dw[t, k] = (act * d).sum(1)
        dw_err[t, k] = (ea * d.abs() + (act.abs() + ea) * (ed + sum_err(I) * (d.abs() + ed))).sum(1)
        p = weights[t, k].double()[:, None]
        er = ea + BF * (act.abs() + ea)
        ref_out.index_add_(0, t, p * (act @ b.t()))
        out_err.index_add_(0, t, p * (er @ b.abs().t() + sum_err(I) * ((act.abs() + er) @ b.abs().t())))
    # each rank's row is rounded, and their sum
    assert ((out.double() - ref_out).abs() <= out_err * (1 + 3 * BF) + 2 * BF * out_err + BF * ref_out.abs() * 2 + 0.02).all()
    assert ((dweights.double() - dw).abs() <= dw_err).all()
    s = scores(logits.double(), score == "softmax")
    share = weigh(s, idx, epm.Router(K, score=score), logits.double())
    one = s.gather(1, idx)
    c, ec = dw * r.scale, dw_err * r.scale
    inner, ei = (c * share).sum(1, keepdim=True), (ec * share).sum(1, keepdim=True)
    if score == "softmax":
        ref = torch.zeros((T, E), **f64).scatter_add(1, idx, share * (c - inner))
        err = torch.zeros((T, E), **f64).scatter_add(1, idx, share * (ec + ei + 100 * U * (c.abs() + inner.abs())))
    else:
        of = one.sum(1, keepdim=True)
        ref = torch.zeros((T, E), **f64).scatter_add(1, idx, (c - inner) / of * one * (1 - one))
        err = torch.zeros((T, E), **f64).scatter_add(1, idx, (ec + ei + 100 * U * (c.abs() + (c * share).abs().sum(1, keepdim=True))) / of * one)
    assert ((dlogits.double() - ref).abs() <= err + 2.0 ** -100).all()


@pytest.mark.parametrize("T", [1, 3, 29])
def test_decode_step_beside_the_operations_it_replaces(T):
    """Norm, an FP8 projection with adapters beside it, norm, and the layer; the layer's experts are those of route,
    its rows those of dispatch, experts and combine within their roundings."""
    H, I, E, R, L, rank = 512, 256, 16, 4, 5, 16
    g = gen(T)
    hidden, residual, wn = normal(g, (T, H)), normal(g, (T, H)), normal(g, (H,))
    _, pair, residual, _ = epm.rms_norm(hidden, wn, 1e-6, residual=residual, use_fp8=True)
    proj = fp8_weight(g, (H, H))
    base = epm.fp8_product(pair, proj)
    x16, _, _, _ = epm.rms_norm(residual, wn, 1e-6)
    ids = torch.randint(-1, L, (T,), generator=g, device="cuda")
    _, down, up, scales, _, dy, dxb = made_adapter(T, H, H, rank, L)
    out = check_adapter(ids, x16, down, up, scales, base, dy, dxb)[0]
    normed, _, residual, _ = epm.rms_norm(out, wn, 1e-6, residual=residual)
    _, wr, w13, w2 = made_layer(T, H, I, E, seed=T)
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    y, idx, wt = check_layer(normed, wr, SIGMOID, w13, w2, bias=bias, residual=residual)
    buf = epm.Buffer(R, E)
    logits = (normed.double() @ wr.double().t()).float()
    idx2, wt2, _ = buf.route(logits, SIGMOID, bias=bias)
    assert torch.equal(idx, idx2) and ((wt - wt2).abs() <= 100 * U * wt2).all()
    packed, count, handle, _, _ = buf.low_latency_dispatch(normed, idx2, T)
    # (cells that hold no row are left as they are: zeros, so that the largest cell is a used one)
    cells = buf.low_latency_expert_ffn(packed, count, handle, w13, w2, out=torch.zeros_like(packed))
    combined, _, _ = buf.low_latency_combine(cells, idx2, wt2, handle)
    ref, bound, _, _ = reference(normed, wr, SIGMOID, w13, w2, bias=bias)
    # the cells are rounded to bf16 before they are weighted, the sum once more
    slack = bound + BF * ref.abs() + BF * (wt2.double().sum(1, keepdim=True) * cells.double().abs().max())
    assert ((combined.double() - ref).abs() <= slack).all()
    assert ((y.double() - residual.double() - combined.double()).abs() <= slack + bound + BF * y.double().abs()).all()


def test_captured_graphs_replay_with_new_inputs():
    """Every operation and both backward passes in two graphs that are replayed in turn, with eager work between."""
    T, H, I, E, K, N, rank, L = 9, 256, 128, 32, 4, 264, 24, 6
    buf = epm.Buffer(4, E)
    r = epm.Router(K, score="sigmoid", num_groups=4, topk_groups=2)
    x, wr, w13, w2 = made_layer(T, H, I, E, seed=1)
    one = x[:1].clone()
    big = normal(gen(5), (700, H))
    ids, big_ids = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.zeros(700, dtype=torch.int64, device="cuda")
    _, down, up, scales, _, _, _ = made_adapter(1, H, N, rank, L)
    dy, bias = normal(gen(6), (700, N)), torch.zeros(E, device="cuda")
    logits, dw, q = torch.zeros((700, E), device="cuda"), torch.zeros((700, K), device="cuda"), torch.zeros(E, device="cuda")

    def layer():
        return [*buf.low_latency_moe(x, wr, r, w13, w2, bias=bias, residual=x),
                *buf.low_latency_moe(one, wr, r, w13, w2, bias=bias), epm.adapter_product(x, ids, down, up, scales)[0]]

    def step():
        idx, wt, sums = buf.route(logits, r, bias=bias, score_sums=True)
        out, hidden = epm.adapter_product(big, big_ids, down, up, scales, save=True)
        return [idx, wt, sums, buf.route_backward(dw, logits, idx, r, dscore_sums=q), out,
                *epm.adapter_product_backward(dy, big, big_ids, down, up, scales, hidden)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(), step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for f in (layer, step):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = f()
        graphs.append((graph, held, f))
    for n in range(4):
        g = gen(100 + n)
        x.copy_(normal(g, (T, H)))
        one.copy_(normal(g, (1, H)))
        big.copy_(normal(g, (700, H)))
        dy.copy_(normal(g, (700, N)))
        for t in (logits, dw, q, bias):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        ids.copy_(torch.randint(-1, L, (T,), generator=g, device="cuda"))
        big_ids.copy_(torch.randint(-1, L, (700,), generator=g, device="cuda"))
        wants = [f() for _, _, f in graphs]
        for graph, _, _ in graphs if n % 2 else graphs[::-1]:
            graph.replay()
        for (_, held, f), want in zip(graphs, wants):
            assert len(held) == len(want)
            for i, (a, b) in enumerate(zip(held, want)):
                assert torch.equal(a, b), (f.__name__, n, i)
        torch.cuda.synchronize()


def test_streams_at_once_and_run_to_run():
    """Four streams, each with its own inputs, interleaved call by call: the same bits as alone."""
    T, H, I, E, N, rank, L = 40, 512, 128, 24, 256, 32, 4
    r = epm.Router(3)
    buf = epm.Buffer(2, E)
    _, wr, w13, w2 = made_layer(1, H, I, E, seed=2)
    _, down, up, scales, _, _, _ = made_adapter(1, H, N, rank, L)
    xs = [normal(gen(20 + i), (T, H)) for i in range(4)]
    big = [normal(gen(40 + i), (1200, H)) for i in range(4)]
    ids = [torch.randint(-1, L, (1200,), generator=gen(60 + i), device="cuda") for i in range(4)]

    def run(i):
        y, idx, wt = buf.low_latency_moe(xs[i], wr, r, w13, w2)
        out, hidden = epm.adapter_product(big[i], ids[i], down, up, scales, save=True)
        grads = epm.adapter_product_backward(out, big[i], ids[i], down, up, scales, hidden)
        logits = big[i][:, :E].float().contiguous()
        return [y, idx, wt, out, *grads, *buf.route(logits, r, score_sums=True)]

    alone = [run(i) for i in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [None] * 4
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = run(i)
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_offsets_past_four_gigabytes():
    # logits: the last tokens of 2^23 rows of 512
    T, E = (1 << 23) + 5, 512
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    tail = normal(gen(1), (300, E))
    logits[-300:] = tail
    buf, r = epm.Buffer(1, E), epm.Router(4)
    idx, wt, _ = buf.route(logits, r)
    a, b, _ = buf.route(tail, r)
    assert torch.equal(idx[-300:], a) and torch.equal(wt[-300:], b)
    assert (idx[:-300] == torch.arange(4, device="cuda")).all()
    dw = torch.zeros((T, 4), device="cuda")
    dw[-300:] = torch.randn((300, 4), generator=gen(2), device="cuda")
    dl = buf.route_backward(dw, logits, idx, r)
    assert torch.equal(dl[-300:], buf.route_backward(dw[-300:].contiguous(), tail, a, r))
    assert (dl[:1000] == 0).all()
    del logits, idx, wt, dw, dl
    torch.cuda.empty_cache()
    # tokens of an adapter behind 4 GB of others, and an adapter behind 4 GB of others
    T, K, N, rank, L = 300000, 8192, 64, 128, 2200
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    x[-40:] = normal(gen(3), (40, K))
    ids = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    ids[-40:] = torch.tensor([L - 1, 0], device="cuda").repeat(20)
    down = torch.zeros((L, rank, K), dtype=torch.bfloat16, device="cuda")
    up = torch.zeros((L, N, rank), dtype=torch.bfloat16, device="cuda")
    for a in (0, L - 1):
        down[a], up[a] = normal(gen(4 + a), (rank, K), 0.01), normal(gen(5 + a), (N, rank), 0.1)
    scales, dy = torch.ones(L, device="cuda"), torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    dy[-40:] = normal(gen(6), (40, N))
    out, hidden = epm.adapter_product(x, ids, down, up, scales, save=True)
    dx, ddown, dup = epm.adapter_product_backward(dy, x, ids, down, up, scales, hidden)
    few = (x[-40:].contiguous(), (ids[-40:] > 0).long(), down[[0, L - 1]].contiguous(), up[[0, L - 1]].contiguous(),
           scales[:2].contiguous())
    want, wh = epm.adapter_product(*few, save=True)
    tol = lambda v: 4 * BF * v.abs().max()  # noqa: E731  (the same sums, split another way)
    assert (out[-40:].float() - want.float()).abs().max() <= tol(want.float()) and (out[:-40] == 0).all()
    wx, wd, wu = epm.adapter_product_backward(dy[-40:].contiguous(), *few, wh)
    for got, ref in ((dx[-40:], wx), (ddown[[0, L - 1]], wd), (dup[[0, L - 1]], wu)):
        assert (got.float() - ref.float()).abs().max() <= tol(ref.float())
    assert (dx[:1000] == 0).all() and (ddown[1:L - 1:97] == 0).all()
    del x, down, dx, ddown, out
    torch.cuda.empty_cache()
    # an expert behind 4 GB of others
    H, I, E = 7168, 2048, 80
    w13 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros((E, H, I), dtype=torch.bfloat16, device="cuda")
    for e in (0, E - 1):
        w13[e], w2[e] = normal(gen(7 + e), (2 * I, H), 0.01), normal(gen(8 + e), (H, I), 0.02)
    bias = torch.zeros(E, device="cuda")
    bias[[0, E - 1]] = torch.tensor([2.0, 3.0], device="cuda")
    for T in (1, 3):
        check_layer(normal(gen(9), (T, H)), normal(gen(10), (E, H), 0.01), epm.Router(2, score="sigmoid"), w13, w2, bias=bias)
