"""The experts' gate at the ends of its range: infinite, and finite but so large that
its exponent's argument overflows, in every kernel that forms an activation."""

from __future__ import annotations

import sys

import pytest
import torch

from test_gpu_experts import BF, TINY, ffn_ref, gen, normal, sum_err

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


# the gate of row 0 (row 1 has its negative), from products that are powers of two:
# exact in any order of the sum
GATES = {"inf": (2.0 ** 100, 2.0 ** 100, float("inf")), "2^127 and a half": (1.5 * 2.0 ** 63, 2.0 ** 64, 1.5 * 2.0 ** 127)}


def inputs(T, H, I, E, gate):
    """Rows 0 and 1 of every expert meet the large gate in channel 0, whose u is 1;
    w2's channel 0 is 2^-100."""
    xv, wv, _ = GATES[gate]
    g = gen(T + H)
    x, w13, w2 = normal(g, (T, H)), normal(g, (E, 2 * I, H), H ** -0.5), normal(g, (E, H, I), I ** -0.5)
    x[:, :2] = 0
    w13[:, :, :2] = 0
    x[0, 0], x[1, 0], x[:2, 1] = xv, -xv, 1.0
    w13[:, 0], w13[:, I] = 0, 0
    w13[:, 0, 0], w13[:, I, 1] = wv, 1.0
    w2[:, :, 0] = 2.0 ** -100
    return x, w13, w2


def rest_of(x, w13, w2, e):
    """fp64 outputs of expert e without channel 0, and their bound."""
    I = w2.shape[2]
    others = torch.cat((w13[e, 1:I], w13[e, I + 1:])).double()
    W2 = w2[e, :, 1:].double()
    _, _, _, act, _, _, eact = ffn_ref(x.double(), others, W2)
    ref = act @ W2.t()
    tol = ((eact + act.abs() * BF * 1.01) @ W2.abs().t() + sum_err(I) * (act.abs() @ W2.abs().t())) * 1.01
    return ref, tol + ref.abs() * BF * 1.01 + TINY


# rows of an expert and widths that take: K split, 64-row tiles, 256-row tiles
SHAPES = [(4, 64, 72, 2), (70, 264, 136, 4), (300, 256, 2056, 16)]


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T,H,I,E", SHAPES)
def test_large_gate(T, H, I, E, gate):
    x, w13, w2 = inputs(T, H, I, E, gate)
    value = GATES[gate][2]
    buf = epm.Buffer(1, E)
    ids = torch.arange(E, device="cuda").repeat(T, 1)  # every row to every expert
    packed, count, hdl, _, _ = buf.low_latency_dispatch(x, ids, T)
    cells = buf.low_latency_expert_ffn(packed, count, hdl, w13, w2)
    rows = buf.expert_rows(ids, torch.tensor([T], dtype=torch.int32, device="cuda"))
    weights = torch.ones((T, E), device="cuda") / E
    y, saved = buf.expert_ffn(x, rows, weights, w13, w2, save=True)
    for e in (0, E - 1):
        got = cells[e, 0].double()
        if value == float("inf"):
            assert (got[0] == float("inf")).all() and got[1].isnan().all()  # silu(-inf) = -inf * 0
        else:
            # 1.5 * 2^27, to bf16's half step; the other channels' part is below 2^10
            assert ((got[0] - value * 2.0 ** -100).abs() <= value * 2.0 ** -100 * BF + 2.0 ** 10).all()
            ref, tol = rest_of(x[1:2], w13, w2, e)
            assert ((got[1:2] - ref).abs() <= tol).all()
        assert got[2:].isfinite().all()
    assert y[2:].isfinite().all()
    if value == float("inf"):
        assert (y[0] == float("inf")).all() and y[1].isnan().all()
        return
    assert y[:2].isfinite().all()
    dy = torch.zeros_like(x)
    dy[:2] = 2.0 ** -100  # d of channel 0 is H 2^-200 = 0, of the others below 2^-90
    dx, dtw, dw13, dw2 = buf.expert_ffn_backward(dy, x, rows, weights, w13, w2, saved)
    for t in (dx, dtw, dw13, dw2):
        assert t.isfinite().all()
    # channel 0 of dW2 is dy of row 0 times its weighted activation
    want = 2.0 ** -100 * value / E
    assert ((dw2[:, :, 0].double() - want).abs() <= want * 2 * BF * 1.01).all()


@pytest.mark.parametrize("T,H,I,E", SHAPES)
def test_gate_that_is_not_a_number(T, H, I, E):
    """Its row is NaN in the outputs and in its own gradient, every other row as it was."""
    g = gen(T)
    x, w13, w2 = normal(g, (T, H)), normal(g, (E, 2 * I, H), H ** -0.5), normal(g, (E, H, I), I ** -0.5)
    buf = epm.Buffer(1, E)
    ids = torch.arange(E, device="cuda").repeat(T, 1)
    rows = buf.expert_rows(ids, torch.tensor([T], dtype=torch.int32, device="cuda"))
    weights = torch.rand((T, E), generator=g, device="cuda")
    dy = normal(g, x.shape)

    def run():
        packed, count, hdl, _, _ = buf.low_latency_dispatch(x, ids, T)
        cells = buf.low_latency_expert_ffn(packed, count, hdl, w13, w2)
        y, saved = buf.expert_ffn(x, rows, weights, w13, w2, save=True)
        dx, dtw, dw13, dw2 = buf.expert_ffn_backward(dy, x, rows, weights, w13, w2, saved)
        return cells[:, 0], y[None], dx[None], dtw[None, :, :], dw13, dw2
    want = run()
    x[1, 3] = float("nan")
    got = run()
    others = torch.arange(T, device="cuda") != 1
    for a, b in zip(got[:4], want[:4]):
        assert a[:, 1].isnan().all() and torch.equal(a[:, others], b[:, others]) and b.isfinite().all()
    assert got[4].isnan().all() and got[5].isnan().all()  # sums over all rows


# K split, 64-row tiles of few activations and of many, 256-row tiles
@pytest.mark.parametrize("T,H,I,E", [(4, 128, 128, 2), (70, 128, 128, 4), (70, 256, 1024, 4), (300, 256, 2048, 16)])
def test_large_gate_fp8(T, H, I, E):
    """Row 0's first block holds an activation of 1.5 * 2^127, whose code is 448 and whose
    scale follows it; the others of that block are then zero."""
    one, one_and_half = 0x38, 0x3C  # e4m3
    g = gen(T)
    buf = epm.Buffer(1, E)
    codes = torch.randn((E, 1, T, H), generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.full((E, 1, T, H // 128), 2.0 ** -4, device="cuda")
    q13 = torch.randn((E, 2 * I, H), generator=g, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    s13 = torch.full((E, 2 * I // 128, H // 128), 2.0 ** -4, device="cuda")
    q2 = torch.full((E, H, I), one, dtype=torch.uint8, device="cuda")
    s2 = torch.full((E, H // 128, I // 128), 2.0 ** -100, device="cuda")
    codes[..., :2] = 0
    q13[:, :, :128] = 0  # in the first block of K only channel 0 meets anything,
    q13[:, 0] = 0        # and channel 0 nothing past it
    q13[:, I] = 0
    codes[:, :, 0, 0], codes[:, :, 0, 1] = one_and_half, one
    q13[:, 0, 0], q13[:, I, 1] = one, one
    scales[:, :, 0, 0], s13[:, 0, 0] = 2.0 ** 63, 2.0 ** 64  # g = 1.5 * 2^127
    s13[:, I // 128, 0] = 2.0 ** -63                         # u = 1
    count = torch.full((E, 1), T, dtype=torch.int32, device="cuda")
    hdl = epm.LowLatencyHandle(torch.empty(0, device="cuda"), torch.zeros((T, E), dtype=torch.int32, device="cuda"),
                               T, E, H)
    out = buf.low_latency_expert_ffn((codes, scales), count, hdl, (q13, s13), (q2, s2))
    assert out.isfinite().all()
    # times w2, 2^-100; two roundings of the scale, one to bf16; the other blocks add below 2^-80
    want = 1.5 * 2.0 ** 27
    assert ((out[:, 0, 0].double() - want).abs() <= want * (BF + 2.0 ** -20)).all()
