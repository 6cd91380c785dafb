"""The backward pass takes every size that the forward pass takes and a card can hold, without a GPU: what is
refused for its size is known before the workspace is looked at."""

from __future__ import annotations

import pytest

from combine_get_dispatch_05_amd import abi
from test_adapter_cpu import A, CAP, INV, L, call, dims

GOOD = {"d": None, **{p: A for p in ("dy", "x", "ids", "down", "up", "scales", "hidden", "dx_base", "dx", "ddown", "dup")},
        "work": A, "size": 0, "stream": None}


@pytest.mark.parametrize("size", [(16, 28672, 8192, 16, 8192), (16, 16384, 16448, 8, 8192), (16, 1 << 20, 1 << 20, 8, 4096),
                                  (16, 8, 1 << 20, 8, 8191)])
def test_many_wide_adapters_are_taken(size):
    assert L.ep_adapter_workspace(dims(*size), 1) > 0
    assert call(L.ep_adapter_product_backward, GOOD, d=dims(*size)) == CAP  # (the workspace of 0 bytes, not the size)


@pytest.mark.parametrize("size", [(16, 1 << 20, 1 << 20, 8, 4097), (16, 1 << 20, 8, 8, 8192)])
def test_more_than_a_card_holds_is_refused(size):
    tokens, wide, out, rank, adapters = size
    assert 4 * adapters * rank * (wide + out) >= 270e9  # bytes of the weights and their gradients
    assert call(L.ep_adapter_product_backward, GOOD, d=dims(*size)) == INV == abi.EP_ERR_INVALID
