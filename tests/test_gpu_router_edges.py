"""The router where a choice or a gradient hangs on what fp32 drops, against its definition in 64 bits."""

from __future__ import annotations

import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402
from test_gpu_router import choose, gen  # noqa: E402


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
