"""Calls at the ends of what the expert operations document: the most slots, the widest
rows, no rows at all, experts named twice past their cells, a handle's rows inside a
captured graph, and two captured graphs at work at once.  References and bounds are
those of test_gpu_experts.py."""

from __future__ import annotations

import sys

import pytest
import torch

import test_gpu_experts as base
from test_gpu_experts import dispatched, experts_ref, close, gen, normal, routing
from test_gpu_experts_chain import _capture, _flat, _noise, _replays

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


# 64 slots a token, in all ranks and with one expert several times; rows and inner
# widths of 2^20, with K split and in tiles
@pytest.mark.parametrize("T,H,I,E,R,K,mask,dup", [
    (5, 72, 40, 64, 2, 64, 0.2, False), (9, 72, 40, 64, 8, 64, 0.0, True), (40, 64, 72, 2, 1, 64, 0.1, True),
    (3, 1 << 20, 8, 4, 2, 2, 0.0, False), (3, 8, 1 << 20, 4, 2, 2, 0.0, False), (70, 1 << 20, 8, 1, 1, 1, 0.0, False)])
def test_expert_ffn_and_gradients(T, H, I, E, R, K, mask, dup):
    base.test_expert_ffn_and_gradients(T, H, I, E, R, K, mask, dup)


@pytest.mark.parametrize("M,N,K", [(3, 8, 1 << 20), (20, 72, 1 << 20)])
def test_fp8_product_of_a_long_sum(M, N, K):
    base.test_fp8_product(M, N, K)


def test_no_rows():
    """A dispatch that sent nothing: empty rows, zero gradients of the weights."""
    T, H, I, E, R, K = 7, 64, 40, 6, 3, 2
    g = gen(1)
    buf = epm.Buffer(R, E)
    topk = torch.full((T, K), -1, dtype=torch.int64, device="cuda")
    recv, ids, tw, _, h, _ = buf.dispatch(normal(g, (T, H)), topk, torch.zeros((T, K), device="cuda"))
    assert recv.shape == (0, H)
    rows = buf.expert_rows(ids, h)
    assert (rows.expert_offsets == 0).all() and rows.row_pair.shape == (0, K)
    w13, w2 = normal(g, (E, 2 * I, H)), normal(g, (E, H, I))
    y, saved = buf.expert_ffn(recv, rows, tw, w13, w2, save=True)
    assert y.shape == (0, H) and saved.shape == (0, 2 * I)
    dx, dtw, dw13, dw2 = buf.expert_ffn_backward(y, recv, rows, tw, w13, w2, saved)
    assert dx.shape == (0, H) and dtw.shape == (0, K)
    assert dw13.shape == w13.shape and (dw13 == 0).all() and dw2.shape == w2.shape and (dw2 == 0).all()
    h.free()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T,K", [(2, 3), (40, 4), (300, 2)])
def test_experts_named_twice_past_their_cells(T, K, fp8):
    """Counts above the slots of a cell block: its slots are computed, nothing past them."""
    E, R, H, I, S = 4, 2, 256, 128, T
    g = gen(T)
    topk = torch.full((T, K), 2, dtype=torch.int64, device="cuda")
    topk[0, 0] = 1
    buf = epm.Buffer(R, E)
    x = normal(g, (T, H))
    packed, count, hdl, _, _ = buf.low_latency_dispatch(x, topk, S, use_fp8=fp8)
    assert int(count.max()) == T * K - 1 > S
    if fp8:
        w13, w2 = base.fp8_weight(g, (E, 2 * I, H)), base.fp8_weight(g, (E, H, I))
    else:
        w13, w2 = normal(g, (E, 2 * I, H), H ** -0.5), normal(g, (E, H, I), I ** -0.5)
    shape = (E // R, R, S, H)
    guarded = torch.full((E * S + 64, H), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guarded[32:-32].view(shape)
    buf.low_latency_expert_ffn(packed, count, hdl, w13, w2, out=out)
    assert (guarded[:32] == 7.0).all() and (guarded[-32:] == 7.0).all()
    used = torch.arange(S, device="cuda") < count[..., None]
    assert (out[~used] == 7.0).all()
    # expert 2's cells against 64 bits
    if fp8:
        cells, v13, v2 = base.rows_value((packed[0][0, 1], packed[1][0, 1])), base.weight_value(w13), base.weight_value(w2)
    else:
        cells, v13, v2 = packed[0, 1].double(), w13.double(), w2.double()
    _, _, _, act, _, _, eact = base.ffn_ref(cells, v13[2], v2[2], fp8=fp8)
    if fp8:  # half a step of the activation's code: 2^-4 of it, or of the block's least
        least = act.view(S, -1, 128).abs().amax(-1, keepdim=True).clamp_min(1e-4) / 448 * 2.0 ** -10
        kept = torch.maximum((act.abs() + eact) * 2.0 ** -4, least.expand(-1, -1, 128).reshape(act.shape) * 1.01)
    else:
        kept = act.abs() * base.BF * 1.01
    ref = act @ v2[2].t()
    tol = (eact + kept) @ v2[2].abs().t() + base.sum_err(I) * (act.abs() @ v2[2].abs().t()) * 1.1
    if fp8:
        tol = tol + base.fp8_sum_err(act, v2[2]) * 1.1
    close(out[0, 1], ref, tol * 1.01 + ref.abs() * base.BF * 1.01 + base.TINY)


def test_handles_rows_in_a_graph():
    """expert_rows reads the handle's layout on the stream, without a host sync: it can be captured."""
    T, H, I, E, R, K = 150, 128, 136, 8, 2, 3
    g = gen(4)
    buf, h, _, x, ids, tw = dispatched(g, T, H, E, R, K, 0.2, False)
    w13, w2 = normal(g, (E, 2 * I, H), 0.1), normal(g, (E, H, I), 0.1)

    def step():
        rows = buf.expert_rows(ids, h)
        y, saved = buf.expert_ffn(x, rows, tw, w13, w2, save=True)
        return y, buf.expert_ffn_backward(y, x, rows, tw, w13, w2, saved)
    _replays(*_capture(step), step, lambda i: x.copy_(normal(g, x.shape)))
    h.free()


def test_two_graphs_at_once():
    """Two captured steps replayed side by side on two streams, again and again: each
    gives its eager result."""
    E, R, K, H, I = 16, 4, 3, 256, 136
    steps = []
    for T in (90, 400):
        g = gen(T)
        topk, w = routing(g, T, E, K, 0.1)
        buf = epm.Buffer(R, E)
        x = normal(g, (T, H))
        recv, ids, tw, _, h, _ = buf.dispatch(x, topk, w)
        prefix = h.layout().rank_prefix_matrix.clone()
        h.free()
        w13, w2 = normal(g, (E, 2 * I, H), 0.06), normal(g, (E, H, I), 0.06)

        def step(T=T, x=x, recv=recv, ids=ids, tw=tw, prefix=prefix, w13=w13, w2=w2, topk=topk, buf=buf):
            rows = buf.expert_rows(ids, prefix, num_tokens=T)
            y, saved = buf.expert_ffn(recv, rows, tw, w13, w2, save=True)
            packed, count, hdl, _, _ = buf.low_latency_dispatch(x, topk, T)
            z = torch.zeros_like(packed)
            buf.low_latency_expert_ffn(packed, count, hdl, w13, w2, out=z)
            return y, buf.expert_ffn_backward(y, recv, rows, tw, w13, w2, saved), z
        steps.append((step, *_capture(step)))
    want = [[t.clone() for t in _flat(step())] for step, _, _ in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for i in range(5):
        for _, _, out in steps:
            for t in _flat(out):
                t.view(torch.uint8).fill_(0x5A)
        _noise()
        for s, (_, graph, _) in zip(streams, steps):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for j, (_, _, out) in enumerate(steps):
            for k, (a, b) in enumerate(zip(_flat(out), want[j])):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (i, j, k)


def test_rows_without_the_number_of_tokens():
    """A bare prefix leaves room for every slot of every row; the results are the same."""
    T, H, I, E, R, K = 60, 72, 40, 8, 4, 5
    g = gen(6)
    buf, h, prefix, x, ids, tw = dispatched(g, T, H, E, R, K, 0.1, False, extra=11)
    w13, w2 = normal(g, (E, 2 * I, H), H ** -0.5), normal(g, (E, H, I), I ** -0.5)
    dy = normal(g, x.shape)
    refs = experts_ref(x, ids, tw, prefix, E, R, w13, w2, dy)
    rows = buf.expert_rows(ids, prefix)
    assert rows.pair_row.shape == (x.shape[0] * K,)
    y, saved = buf.expert_ffn(x, rows, tw, w13, w2, save=True)
    grads = buf.expert_ffn_backward(dy, x, rows, tw, w13, w2, saved)
    for name, got, (ref, tol) in zip(("y", "dx", "dtopk_weights", "dw13", "dw2"), (y, *grads), refs):
        close(got, ref, tol, name)
    h.free()
