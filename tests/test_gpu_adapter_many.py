"""Many adapters at once: gradients in more blocks than one dimension of a launch holds."""

from __future__ import annotations

import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

from test_gpu_adapter import check, gen, made  # noqa: E402


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


def test_gradients_of_more_than_four_million_blocks():
    T, K, N, r, L = 40, 1 << 17, (1 << 17) + 64, 8, 1024
    assert L * (K // 64 + N // 64) > 1 << 22
    x, down, up, scales, base, dy, dxb = made(T, K, N, r, L)
    ids = torch.randint(-1, L, (T,), generator=gen(1), device="cuda")
    ids[0], ids[1], ids[2:5] = 0, L - 1, L - 1
    check(ids, x, down, up, scales, base, dy, dxb)
    del down, up
    torch.cuda.empty_cache()
