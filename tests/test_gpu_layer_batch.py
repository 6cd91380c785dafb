"""The layer for a few tokens: a token's experts and weights are the same bits alone and in any batch, also where
its logits hang on the order of their sums."""

from __future__ import annotations

import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402
from test_gpu_router import gen  # noqa: E402


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("E,H", [(48, 1024), (130, 72), (512, 2056)])
def test_experts_whose_logits_hang_on_the_order_of_a_sum(E, H, f32):
    g = gen(E)
    # pairs of v and -v anywhere in a row: what is left of the sum is its roundings
    v = torch.randn((E, H // 2), generator=g, device="cuda") * 2.0 ** (torch.rand((E, H // 2), generator=g, device="cuda") * 70)
    if not f32:
        v = v.to(torch.bfloat16)
    wr = torch.cat([v, -v], 1)
    wr = wr.gather(1, torch.rand((E, H), generator=g, device="cuda").argsort(1)).contiguous()
    x = (1 + torch.arange(64, device="cuda")[:, None] / 64).to(torch.bfloat16).repeat(1, H).contiguous()
    w13 = torch.zeros((E, 16, H), dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros((E, H, 8), dtype=torch.bfloat16, device="cuda")
    buf, r = epm.Buffer(1, E), epm.Router(4, score="sigmoid")
    _, idx, wt = buf.low_latency_moe(x, wr, r, w13, w2)
    assert (idx >= 0).all()
    for T in (1, 2, 8, 9, 16, 17, 33, 50):
        for t0 in (0, 64 - T):
            _, i, w = buf.low_latency_moe(x[t0:t0 + T].contiguous(), wr, r, w13, w2)
            assert torch.equal(i, idx[t0:t0 + T]) and torch.equal(w, wt[t0:t0 + T]), (T, t0)


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,H,I", [(40, 256, 8), (100, 8192, 8), (100, 264, 1032), (300, 16392, 8)])
def test_weights_are_the_same_bits_wherever_the_choice_is_made(E, H, I, score, normalize):
    """In the gate's blocks (one token; up to eight where those are few) or in a launch of its own."""
    g = gen(E + H)
    x = torch.randn((64, H), generator=g, device="cuda").to(torch.bfloat16)
    wr = torch.randn((E, H), generator=g, device="cuda") * 2 / H ** 0.5
    w13 = torch.zeros((E, 2 * I, H), dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros((E, H, I), dtype=torch.bfloat16, device="cuda")
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    buf, r = epm.Buffer(1, E), epm.Router(3, score=score, num_groups=4, topk_groups=2, normalize=normalize)
    _, idx, wt = buf.low_latency_moe(x, wr, r, w13, w2, bias=bias)
    for T in (1, 2, 3, 8, 9, 20):
        for t0 in (0, 30, 64 - T):
            _, i, w = buf.low_latency_moe(x[t0:t0 + T].contiguous(), wr, r, w13, w2, bias=bias)
            assert torch.equal(i, idx[t0:t0 + T]) and torch.equal(w, wt[t0:t0 + T]), (T, t0)
