"""The expert operations as they are used: a training step from dispatch to
combine and back, a decode step from the norm to the combine, captured graphs,
other streams, tensors past 4 GB, and what the binding turns down on a GPU.

The bounds are those of test_gpu_experts.py, carried through the sums that
follow (n * 2^-24 of the summed magnitudes and one rounding to bf16)."""

from __future__ import annotations

import ctypes
import sys

import pytest
import torch

from test_gpu_experts import (BF, TINY, U, close, dispatched, experts_ref, ffn_ref, fp8_rows, fp8_weight, gen,
                              normal, routing, rows_value, sum_err, weight_value)

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402
from combine_get_dispatch_05_amd import abi  # noqa: E402


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


def to_tokens(values, src, T):
    return torch.zeros((T, values.shape[1]), dtype=torch.float64, device="cuda").index_add_(0, src, values)


@pytest.mark.parametrize("T,H,I,E,R,K,mask,dup", [(90, 128, 72, 16, 4, 5, 0.2, False),
                                                  (260, 64, 136, 6, 2, 3, 0.0, True)])
def test_training_step_from_dispatch_to_combine(T, H, I, E, R, K, mask, dup):
    g = gen(T)
    topk, w = routing(g, T, E, K, mask, dup)
    buf = epm.Buffer(R, E)
    x = normal(g, (T, H))
    w13, w2 = normal(g, (E, 2 * I, H), H ** -0.5), normal(g, (E, H, I), I ** -0.5)
    dout = normal(g, (T, H))
    # forward and backward, the dispatch's cached handle carrying the gradient
    recv, ids, tw, _, h, _ = buf.dispatch(x, topk, w)
    rows = buf.expert_rows(ids, h)
    y, saved = buf.expert_ffn(recv, rows, tw, w13, w2, save=True)
    out, _, _ = buf.combine(y, h)
    dy = buf.dispatch(dout, handle=h)[0]
    dxr, dtw, dw13, dw2 = buf.expert_ffn_backward(dy, recv, rows, tw, w13, w2, saved)
    dx, dw, _ = buf.combine(dxr, h, dtw)
    # the dense definition in fp64, its gradients by autograd
    x64, w64, a64, b64 = (t.double().requires_grad_() for t in (x, w, w13, w2))
    dense = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, k = (topk == e).nonzero(as_tuple=True)
        z = x64[t]
        act = torch.nn.functional.silu(z @ a64[e, :I].t()) * (z @ a64[e, I:].t())
        dense = dense.index_add(0, t, w64[t, k, None] * (act @ b64[e].t()))
    dense.backward(dout.double())
    # bounds from the rows, carried through the combine
    prefix = h.layout().rank_prefix_matrix
    src = h.layout().recv_src_idx.long()
    (yr, ey), (dxr64, edx), (dwr, edw), (r13, e13), (r2, e2) = experts_ref(recv, ids, tw, prefix, E, R, w13, w2, dy)

    def combined(v, err):
        mag = to_tokens(v.abs(), src, T)
        return to_tokens(err, src, T) * 1.01 + (R + 1) * U * mag * 1.01 + to_tokens(v, src, T).abs() * BF * 1.01 + TINY
    tiny = 1e-9  # fp64 against fp64
    close(to_tokens(yr, src, T), dense.detach(), tiny * (1 + dense.detach().abs()), "the row form is the dense one")
    close(out, dense.detach(), combined(yr, ey), "out")
    close(dx, x64.grad, combined(dxr64, edx), "dx")
    close(dw, w64.grad, to_tokens(edw, src, T) + TINY, "dweights")
    close(dw13, a64.grad, e13, "dw13")
    close(dw2, b64.grad, e2, "dw2")
    # gradients against differences of the dense form, along one direction of each input
    def loss(xx, ww, aa, bb):
        s = 0.0
        for e in range(E):
            t, k = (topk == e).nonzero(as_tuple=True)
            z = xx[t]
            act = torch.nn.functional.silu(z @ aa[e, :I].t()) * (z @ aa[e, I:].t())
            s = s + (ww[t, k, None] * (act @ bb[e].t()) * dout.double()[t]).sum()
        return s
    base = [t.detach() for t in (x64, w64, a64, b64)]
    for i, (grad, tol) in enumerate(((dx, combined(dxr64, edx)), (dw, to_tokens(edw, src, T) + TINY), (dw13, e13),
                                     (dw2, e2))):
        v = torch.randn(base[i].shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-5
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + step * v, base[i] - step * v
        num = (loss(*up) - loss(*down)) / (2 * step)
        # the gradient's own bound along v; the differences' error stays far below it
        slack = (tol * v.abs()).sum() + 1e-5 * (grad.double().abs() * v.abs()).sum()
        assert abs(float(num - (grad.double() * v).sum())) <= float(slack), i
    h.free()


def test_masked_rank_gets_no_part_in_a_step():
    T, H, I, E, R, K = 40, 64, 32, 8, 4, 3
    g = gen(5)
    topk, w = routing(g, T, E, K, 0.0)
    buf = epm.Buffer(R, E)
    buf.low_latency_update_mask_buffer(2, True)
    x = normal(g, (T, H))
    w13, w2 = normal(g, (E, 2 * I, H), 0.1), normal(g, (E, H, I), 0.1)
    recv, ids, tw, _, h, _ = buf.dispatch(x, topk, w)
    rows = buf.expert_rows(ids, h)
    off = rows.expert_offsets.tolist()
    assert off[4] == off[5] == off[6]  # rank 2 holds experts 4 and 5
    y, saved = buf.expert_ffn(recv, rows, tw, w13, w2, save=True)
    _, _, dw13, dw2 = buf.expert_ffn_backward(y, recv, rows, tw, w13, w2, saved)
    assert (dw13[4:6] == 0).all() and (dw2[4:6] == 0).all() and (dw13[0] != 0).any()
    packed, count, hdl, _, _ = buf.low_latency_dispatch(x, topk, T)
    out = torch.full_like(packed, 3.0)
    buf.low_latency_expert_ffn(packed, count, hdl, w13, w2, out=out)
    assert (out[:, 2] == 3.0).all() and (out[:, 0] != 3.0).any()
    h.free()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_step_from_norm_to_combine(fp8):
    T, H, I, E, R, K, S = 24, 256, 128, 16, 4, 4, 32
    g = gen(77)
    topk, w = routing(g, T, E, K, 0.1)
    buf = epm.Buffer(R, E)
    x, res, nw = normal(g, (T, H)), normal(g, (T, H), 2.0), normal(g, (H,))
    out, rows8, _, _ = epm.rms_norm(x, nw, residual=res, use_fp8=True)
    packed, count, hdl, _, _ = buf.low_latency_dispatch(out, topk, S, use_fp8=fp8)
    if fp8:
        w13, w2 = fp8_weight(g, (E, 2 * I, H)), fp8_weight(g, (E, H, I))
        v13, v2, cells = weight_value(w13), weight_value(w2), rows_value(packed)
    else:
        w13, w2 = normal(g, (E, 2 * I, H), H ** -0.5), normal(g, (E, H, I), I ** -0.5)
        v13, v2, cells = w13.double(), w2.double(), packed.double()
    z = buf.low_latency_expert_ffn(packed, count, hdl, w13, w2)
    y, _, _ = buf.low_latency_combine(z, topk, w, hdl)
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    tol, mag = torch.zeros_like(ref), torch.zeros_like(ref)
    for e in range(E):
        t, k = (topk == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        le, r = e % (E // R), e // (E // R)
        xs = cells[le, r, hdl.topk_slot[t, k].long()]
        _, _, _, act, _, _, eact = ffn_ref(xs, v13[e], v2[e], fp8=fp8)
        if fp8:  # the activation's codes: half a step, 2^-4 of the value or of the block's least
            least = (act.view(len(t), -1, 128).abs().amax(-1, keepdim=True).clamp_min(1e-4) / 448 * 2.0 ** -10)
            eq = torch.maximum((act.abs() + eact) * 2.0 ** -4, least.expand(-1, -1, 128).reshape(act.shape) * 1.01)
        else:
            eq = act.abs() * BF * 1.01
        p = w[t, k].double()[:, None]
        zz = act @ v2[e].t()
        ez = (eact + eq) @ v2[e].abs().t() + sum_err(I) * (act.abs() @ v2[e].abs().t()) * 1.1 + zz.abs() * BF * 1.01
        if fp8:
            ez = ez + 7 * 2.0 ** -13 * 1.1 * (act.abs().view(len(t), -1, 8).amax(-1) @ v2[e].abs().view(H, -1, 8).amax(-1).t())
        ref.index_add_(0, t, p * zz)
        tol.index_add_(0, t, p * ez * 1.01)
        mag.index_add_(0, t, (p * zz).abs())
    close(y, ref, tol + (K + 1) * U * mag + ref.abs() * BF * 1.01 + TINY)
    # a dense expert on the norm's own 8-bit rows joins through the normal combine's bias
    shared = fp8_weight(g, (H, H))
    dense = epm.fp8_product(rows8, shared)
    recv, ids, tw, _, h, _ = buf.dispatch(out, topk, w)
    plain, _, _ = buf.combine(recv, h)
    both, _, _ = buf.combine(recv, h, bias=dense)
    want = to_tokens(recv.double(), h.layout().recv_src_idx.long(), T) + dense.double()
    size = to_tokens(recv.double().abs(), h.layout().recv_src_idx.long(), T) + dense.double().abs()
    close(both, want, want.abs() * BF * 1.01 + (R + 2) * U * size + TINY)
    assert not torch.equal(plain, both)
    h.free()


def _noise():
    a = torch.randn(1 << 20, device="cuda")
    (a * 2 + 1).sum().item()
    torch.cuda.synchronize()


def _capture(step):
    step()  # once eagerly before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    torch.cuda.synchronize()
    return g, out


def _flat(v):
    return [t for x in v for t in _flat(x)] if isinstance(v, (tuple, list)) else [] if v is None else [v]


def _replays(g, out, step, change):
    """Every replay, with new inputs and the program's own work between, against the eager step."""
    for i in range(4):
        change(i)
        _noise()
        for t in _flat(out):
            t.view(torch.uint8).fill_(0x5A)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in _flat(out)]
        want = _flat(step())
        assert len(got) == len(want)
        for j, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (i, j)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_decode_step_graph(fp8):
    T, H, I, E, R, K, S = 96, 256, 256, 16, 4, 4, 96
    g = gen(8)
    buf = epm.Buffer(R, E)
    x, res, nw = normal(g, (T, H)), normal(g, (T, H)), normal(g, (H,))
    topk, w = routing(g, T, E, K, 0.1)
    if fp8:
        w13, w2 = fp8_weight(g, (E, 2 * I, H)), fp8_weight(g, (E, H, I))
    else:
        w13, w2 = normal(g, (E, 2 * I, H), 0.06), normal(g, (E, H, I), 0.06)

    def step():
        out, rows, r, _ = epm.rms_norm(x, nw, residual=res, use_fp8=True)
        packed, count, hdl, _, _ = buf.low_latency_dispatch(out, topk, S, use_fp8=fp8)
        z = buf.low_latency_expert_ffn(packed, count, hdl, w13, w2)
        return buf.low_latency_combine(z, topk, w, hdl)[0], r, rows

    def change(i):
        x.copy_(normal(g, (T, H)))
        t = routing(g, T, E, K, 0.1)[0]
        if i % 2:
            t[:, 0] = 3  # one expert holds every token: past the few-rows kernel
            t[:, 1:] = torch.where(t[:, 1:] == 3, -1, t[:, 1:])
        topk.copy_(t)
    _replays(*_capture(step), step, change)


def test_training_step_graph():
    T, H, I, E, R, K = 200, 128, 136, 8, 2, 4
    g = gen(21)
    buf = epm.Buffer(R, E)
    _, h, prefix, x, ids, tw = dispatched(g, T, H, E, R, K, 0.2, False)
    N = x.shape[0]
    prefix, tw = prefix.clone(), tw.clone()
    x, ids = x.clone(), ids.clone()
    h.free()
    w13, w2 = normal(g, (E, 2 * I, H), 0.1), normal(g, (E, H, I), 0.1)
    dy, nw = normal(g, (N, H)), normal(g, (H,))

    def step():
        v, _, _, rstd = epm.rms_norm(x, nw)
        rows = buf.expert_rows(ids, prefix, num_tokens=T)
        y, saved = buf.expert_ffn(v, rows, tw, w13, w2, save=True)
        dv, dtw, dw13, dw2 = buf.expert_ffn_backward(dy, v, rows, tw, w13, w2, saved)
        return y, epm.rms_norm_backward(dv, x, nw, rstd), dtw, dw13, dw2

    def change(i):
        x.copy_(normal(g, (N, H)))
        perm = torch.randint(-1, E // R, ids.shape, generator=g, device="cuda")
        perm[torch.rand(ids.shape, generator=g, device="cuda") < 0.5] = -1
        # no more pairs than the batch has slots
        keep = (perm >= 0).view(-1).cumsum(0).view(ids.shape) <= T * K
        ids.copy_(torch.where(keep, perm, -1))
        prefix.copy_(torch.tensor([N // 2 - i, N - 3 * i], dtype=torch.int32, device="cuda"))
    _replays(*_capture(step), step, change)


def test_streams():
    """On another stream, and on two at once: the same bits as on the default one."""
    T, H, I, E, R, K = 150, 256, 128, 8, 4, 3
    g = gen(31)
    topk, w = routing(g, T, E, K, 0.1)
    buf = epm.Buffer(R, E)
    x, nw = normal(g, (T, H)), normal(g, (H,))
    w13, w2 = normal(g, (E, 2 * I, H), 0.06), normal(g, (E, H, I), 0.06)
    q13, q2 = fp8_weight(g, (E, 2 * I, H)), fp8_weight(g, (E, H, I))
    a, b = fp8_rows(g, (T, H)), fp8_weight(g, (512, H))
    recv, ids, tw, _, h, _ = buf.dispatch(x, topk, w)
    packed, count, hdl, _, _ = buf.low_latency_dispatch(x, topk, T)
    p8, c8, h8, _, _ = buf.low_latency_dispatch(x, topk, T, use_fp8=True)
    zero = torch.zeros_like(packed)

    def work():
        rows = buf.expert_rows(ids, h.layout().rank_prefix_matrix, num_tokens=T)
        y, saved = buf.expert_ffn(recv, rows, tw, w13, w2, save=True)
        n = int(rows.expert_offsets[-1])
        z, z8 = zero.clone(), zero.clone()
        buf.low_latency_expert_ffn(packed, count, hdl, w13, w2, out=z)
        buf.low_latency_expert_ffn(p8, c8, h8, q13, q2, out=z8)
        return _flat((y, saved[:n], buf.expert_ffn_backward(y, recv, rows, tw, w13, w2, saved),
                      epm.rms_norm(x, nw, use_fp8=True), epm.fp8_product(a, b), z, z8))
    torch.cuda.synchronize()
    want = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(work())
    torch.cuda.synchronize()
    for run in got:
        for i, (p, q) in enumerate(zip(run, want)):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8)), i
    h.free()


def test_cells_past_four_gigabytes():
    """The last expert of cells of 7.5 GB, in bf16: its rows are at offsets past 2^32 bytes."""
    E, R, S, H, I, T, K = 128, 4, 4096, 7168, 64, 2, 1
    g = gen(13)
    packed = torch.empty((E // R, R, S, H), dtype=torch.bfloat16, device="cuda")
    packed[-1, -1, :2] = normal(g, (2, H))
    count = torch.zeros((E // R, R), dtype=torch.int32, device="cuda")
    count[-1, -1] = 2
    w13, w2 = normal(g, (E, 2 * I, H), H ** -0.5), normal(g, (E, H, I), I ** -0.5)
    hdl = epm.LowLatencyHandle(torch.empty(0, device="cuda"), torch.zeros((T, K), dtype=torch.int32, device="cuda"), S, E, H)
    out = epm.Buffer(R, E).low_latency_expert_ffn(packed, count, hdl, w13, w2)
    x, W2 = packed[-1, -1, :2].double(), w2[E - 1].double()
    _, _, _, act, _, _, eact = ffn_ref(x, w13[E - 1].double(), W2)
    ref = act @ W2.t()
    tol = (eact + act.abs() * BF * 1.01) @ W2.abs().t() + sum_err(I) * (act.abs() @ W2.abs().t())
    close(out[-1, -1, :2], ref, tol * 1.01 + ref.abs() * BF * 1.01 + TINY)


def test_norm_past_two_to_the_32_elements():
    T, H = 600_000, 7168  # 4.3e9 elements
    x = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    x[-1] = 3.0
    x[-2, ::2] = 0.0
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    out, (q, sc), _, rstd = epm.rms_norm(x, w, 0.0, use_fp8=True)
    assert (out[-1] == 1).all() and (out[0] == 1).all() and (out[T // 2] == 1).all()
    close(rstd[-3:], torch.tensor([1.0, 2 ** 0.5, 1 / 3], dtype=torch.float64, device="cuda"),
          torch.full((3,), (H + 16) * U * 2, dtype=torch.float64, device="cuda"))
    assert (q[-1].float() == 448).all() and (q[-2, ::2].float() == 0).all() and (q[-2, 1::2].float() == 448).all()
    del x, out, q, sc


def test_residual_in_place_through_the_abi():
    """residual_out may be the residual's or x's own memory, on short rows and on long."""
    for T, H in ((5, 640), (3, 40960)):
        g = gen(H)
        x, r, w = normal(g, (T, H)), normal(g, (T, H)), normal(g, (H,))
        want, _, res, rstd = epm.rms_norm(x, w, residual=r)
        for into in ("x", "r"):
            a, b = x.clone(), r.clone()
            out, s = torch.empty_like(x), torch.empty_like(rstd)
            abi.check(abi.lib().ep_rms_norm(T, H, 1e-6, abi.ptr(a), abi.ptr(b), abi.ptr(w),
                                            abi.ptr(a if into == "x" else b), abi.ptr(out), None, None, abi.ptr(s),
                                            abi.current_stream()), "ep_rms_norm")
            assert torch.equal(out, want) and torch.equal(s, rstd)
            assert torch.equal(a if into == "x" else b, res)


def test_grouping_of_ids_that_no_dispatch_wrote():
    """A prefix that is none, ids out of range, more pairs than the capacity: nothing
    is written outside its buffer, and what fits is in order."""
    E, R, K, N, T = 8, 4, 4, 50, 6
    g = gen(2)
    ids = torch.randint(-3, 9, (N, K), generator=g, device="cuda")
    prefix = torch.tensor([50, -7, 99, 20], dtype=torch.int32, device="cuda")
    buf = epm.Buffer(R, E)
    d = abi.dims(T, 8, K, E, R)
    cap = T * K
    guard = -77
    i32 = dict(dtype=torch.int32, device="cuda")
    bufs = [torch.full((n + 64,), guard, **i32) for n in (E, E + 1, cap, cap, N * K)]
    P = [ctypes.c_void_p(t.data_ptr() + 128) for t in bufs]  # 32 words in
    abi.check(abi.lib().ep_expert_rows(ctypes.byref(d), abi.ptr(prefix), abi.ptr(ids), N, cap, *P,
                                       abi.current_stream()), "ep_expert_rows")
    torch.cuda.synchronize()
    for t in bufs:
        assert (t[:32] == guard).all() and (t[-32:] == guard).all()
    off = bufs[1][32:32 + E + 1].tolist()
    assert off == sorted(off) and off[0] == 0 and off[-1] == cap
    rows = buf.expert_rows(ids, prefix, num_tokens=T)
    x = normal(g, (N, 64))
    w13, w2 = normal(g, (E, 64, 64)), normal(g, (E, 64, 32))
    y, saved = buf.expert_ffn(x, rows, torch.rand((N, K), generator=g, device="cuda"), w13, w2, save=True)
    assert torch.isfinite(y).all()


def test_refusals_on_device_tensors():
    bf = torch.bfloat16
    buf = epm.Buffer(2, 4)
    x = torch.zeros((4, 256), dtype=bf, device="cuda")
    w = torch.ones(256, dtype=bf, device="cuda")
    with pytest.raises(ValueError, match="weight must have shape"):
        epm.rms_norm(x, w[:128])
    with pytest.raises(ValueError, match="contiguous"):
        epm.rms_norm(x.t().contiguous().t(), w)
    with pytest.raises(ValueError, match="residual must have"):
        epm.rms_norm(x, w, residual=x[:2])
    with pytest.raises(ValueError, match="whole 128"):
        epm.rms_norm(x[:, :64].contiguous(), w[:64].contiguous(), use_fp8=True)
    with pytest.raises(ValueError, match="nothing to return"):
        epm.rms_norm(x, w, bf16_out=False)
    with pytest.raises(epm.abi.EpError, match="invalid argument"):
        epm.rms_norm(x, w, eps=-1.0)
    odd = torch.zeros(4 * 256 + 8, dtype=bf, device="cuda")[4:4 + 1024].view(4, 256)  # 8 bytes off
    with pytest.raises(epm.abi.EpError, match="alignment"):
        epm.rms_norm(odd, w)
    with pytest.raises(ValueError, match="device tensor"):
        epm.rms_norm(x, w.cpu())
    with pytest.raises(ValueError, match="rstd must have"):
        epm.rms_norm_backward(x, x, w, torch.zeros(3, device="cuda"))
    q = torch.zeros((4, 256), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.zeros((4, 2), device="cuda")
    wq, wsc = torch.zeros((136, 256), dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros((2, 2), device="cuda")
    assert epm.fp8_product((q, sc), (wq, wsc)).shape == (4, 136)
    assert epm.fp8_product((q.view(torch.uint8), sc), (wq, wsc)).shape == (4, 136)
    with pytest.raises(ValueError, match="w scales must have"):
        epm.fp8_product((q, sc), (wq, wsc[:1]))
    with pytest.raises(ValueError, match="w codes must have"):
        epm.fp8_product((q[:, :128].contiguous(), sc[:, :1].contiguous()), (wq, wsc))
    with pytest.raises(epm.abi.EpError, match="alignment"):
        epm.fp8_product((q, sc), (wq[:132].contiguous(), wsc))  # 132 columns: rows of 264 bytes
    topk = torch.zeros((4, 1), dtype=torch.int64, device="cuda")
    packed, count, hdl, _, _ = buf.low_latency_dispatch(x, topk, 4)
    w13, w2 = torch.zeros((4, 64, 256), dtype=bf, device="cuda"), torch.zeros((4, 256, 32), dtype=bf, device="cuda")
    with pytest.raises(ValueError, match="w13 must have shape"):
        buf.low_latency_expert_ffn(packed, count, hdl, w13[:, :62].contiguous(), w2)
    with pytest.raises(ValueError, match="out must have"):
        buf.low_latency_expert_ffn(packed, count, hdl, w13, w2, out=packed[:1])
    with pytest.raises(ValueError, match="another number of experts"):
        epm.Buffer(2, 8).low_latency_expert_ffn(packed, torch.zeros((4, 2), dtype=torch.int32, device="cuda"), hdl,
                                                w13, w2)
    recv, ids, tw, _, h, _ = buf.dispatch(x, topk, torch.ones((4, 1), device="cuda"))
    rows = buf.expert_rows(ids, h)
    with pytest.raises(ValueError, match="topk_weights must have"):
        buf.expert_ffn(recv, rows, tw[:2], w13, w2)
    with pytest.raises(ValueError, match="row_pair must have"):
        buf.expert_ffn(recv[:2], rows, tw, w13, w2)
    with pytest.raises(ValueError, match="saved must have"):
        buf.expert_ffn_backward(recv, recv, rows, tw, w13, w2, torch.zeros((1, 64), device="cuda"))
    with pytest.raises(ValueError, match="other experts or ranks"):
        epm.Buffer(1, 4).expert_rows(ids, h)
    with pytest.raises(ValueError, match="rank_prefix_matrix must have"):
        buf.expert_rows(ids, torch.zeros(3, dtype=torch.int32, device="cuda"))
    h.free()
