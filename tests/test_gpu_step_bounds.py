"""The output of a training step from logits through dispatch, experts and combine, within its roundings alone."""

from __future__ import annotations

import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402
from test_gpu_router import close, gen  # noqa: E402

BF, U = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


def normal(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,H,I,E,R,K", [(97, 128, 64, 16, 4, 3), (33, 256, 96, 24, 8, 6)])
def test_output_of_a_step_within_its_roundings(score, T, H, I, E, R, K):
    """Sums of n terms are off by 2 (n + 8) U of the summed magnitudes; the activation is rounded to bf16, the
    row that a rank sends back (the weighted sum over its experts) too, and the sum of the ranks' rows."""
    g = gen(T)
    x, w13, w2 = normal(g, (T, H)), normal(g, (E, 2 * I, H), 1 / math.sqrt(H)), normal(g, (E, H, I), 1 / math.sqrt(I))
    logits, r, buf = torch.randn((T, E), generator=g, device="cuda"), epm.Router(K, score=score, scale=1.5), epm.Buffer(R, E)
    idx, weights, _ = buf.route(logits, r)
    recv, rti, rtw, _, handle, _ = buf.dispatch(x, idx, weights)
    y = buf.expert_ffn(recv, buf.expert_rows(rti, handle), rtw, w13, w2, save=True)[0]
    out, _, _ = buf.combine(y, handle, rtw)
    handle.free()
    f64 = dict(dtype=torch.float64, device="cuda")
    rows, err = torch.zeros((R, T, H), **f64), torch.zeros((R, T, H), **f64)
    sum_err = lambda n: 2 * (n + 8) * U  # noqa: E731
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        a, b, xe = w13[e].double(), w2[e].double(), x[t].double()
        gu, mag = xe @ a.t(), xe.abs() @ a.abs().t() * sum_err(H)
        sig = torch.sigmoid(gu[:, :I])
        act = gu[:, :I] * sig * gu[:, I:]
        ea = 1.1 * mag[:, :I] * (gu[:, I:].abs() + mag[:, I:]) + (gu[:, :I] * sig).abs() * mag[:, I:] + act.abs() * 16 * U
        ea = ea + BF * (act.abs() + ea)
        p = weights[t, k].double()[:, None]
        most = (act.abs() + ea) @ b.abs().t()
        rows[e // (E // R)].index_add_(0, t, p * (act @ b.t()))
        # (the weight and the sum over a rank's experts: K + 2 roundings)
        err[e // (E // R)].index_add_(0, t, p * (ea @ b.abs().t() + (sum_err(I) + (K + 2) * U) * most))
    err = err + BF * (rows.abs() + err)
    ref, bound = rows.sum(0), err.sum(0) + R * U * (rows.abs() + err).sum(0)
    close(out, ref, bound + BF * (ref.abs() + bound), "out")
