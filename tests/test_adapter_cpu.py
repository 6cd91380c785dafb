"""The adapters' refusals, without a GPU."""

from __future__ import annotations

import ctypes

import pytest
import torch

import combine_get_dispatch_05_amd as epm
from combine_get_dispatch_05_amd import abi
from test_router_cpu import A, ALIGN, CAP, INV, M2, M4, call

L = abi.lib()
M8 = ctypes.c_void_p(0x10008)
M128 = ctypes.c_void_p(0x10080)


def dims(*a):
    return ctypes.byref(abi.AdapterDims(*a))


@pytest.mark.parametrize("back", [False, True], ids=["forward", "backward"])
def test_adapter_rules(back):
    n = L.ep_adapter_workspace(dims(32, 256, 128, 16, 4), int(back))
    assert n >= 6 * 4 + 32 * 4 + 32 * 16 * 4
    if back:
        f, small = L.ep_adapter_product_backward, {"ids": M4, "scales": M2}
        ptrs = ["dy", "x", "ids", "down", "up", "scales", "hidden", "dx_base", "dx", "ddown", "dup"]
        free = {"dx_base"}
    else:
        f, small = L.ep_adapter_product, {"ids": M4, "scales": M2}
        ptrs, free = ["x", "ids", "down", "up", "scales", "base", "out", "hidden"], {"base", "hidden"}
    good = {"d": dims(32, 256, 128, 16, 4), **{p: A for p in ptrs}, "work": A, "size": n, "stream": None}
    for p in ptrs:
        if p not in free:
            assert call(f, good, **{p: None}) == INV, p
        assert call(f, good, **{p: small.get(p, M8)}) == ALIGN, p
    assert call(f, good, work=None) == INV
    assert call(f, good, work=M128) == ALIGN
    assert call(f, good, d=None) == INV
    for bad, code in (((-1, 256, 128, 16, 4), INV), (((1 << 24) + 1, 256, 128, 16, 4), INV), ((4, 0, 128, 16, 4), INV),
                      ((4, 256, 0, 16, 4), INV), ((4, 256, 128, 0, 4), INV), ((4, 256, 128, 136, 4), INV),
                      ((4, 256, 128, 16, 0), INV), ((4, 256, 128, 16, 8193), INV), ((4, (1 << 20) + 8, 128, 16, 4), INV),
                      ((4, 256, (1 << 20) + 8, 16, 4), INV), ((4, 252, 128, 16, 4), ALIGN), ((4, 256, 124, 16, 4), ALIGN),
                      ((4, 256, 128, 12, 4), ALIGN)):
        assert call(f, good, d=dims(*bad)) == code, bad
        assert L.ep_adapter_workspace(dims(*bad), int(back)) == 0
    assert L.ep_adapter_workspace(None, int(back)) == 0
    assert call(f, good, size=n - 1) == CAP
    if back:  # more blocks than a launch holds
        assert call(f, good, d=dims(16, 1 << 20, 1 << 20, 8, 8192)) == INV
    else:
        assert call(f, good, d=dims(0, 256, 128, 16, 4)) == abi.EP_OK  # nothing to do


def test_workspace_holds_what_the_launches_write():
    """Offsets, order, the rank's parts of every split, and dh of a backward pass."""
    for T, K, N, r, ad in ((1, 8, 8, 8, 1), (1, 7168, 2048, 16, 8), (128, 7168, 4096, 16, 64), (8192, 7168, 7168, 64, 16),
                           (1 << 24, 1 << 20, 8, 128, 8192), (3, 1 << 20, 1 << 20, 128, 8192)):
        for back in (0, 1):
            n = L.ep_adapter_workspace(dims(T, K, N, r, ad), back)
            if not back and T <= 16 and r <= 64 and r * K <= 1 << 17:  # one launch
                assert n == 0
                continue
            padded = 16 if r <= 16 else 32 if r <= 32 else 64 if r <= 64 else 128
            height = 64 if r <= 64 else 32
            tiles = T // height + min(ad + 1, T)
            steps = -(-(N if back else K) // 64)
            splits = max(1, min(512 // tiles, -(-steps // 4)))
            assert n >= (ad + 2) * 4 + T * 4 + splits * T * padded * 4 + back * T * r * 4


def test_binding_refuses_before_the_library():
    bf = torch.bfloat16
    x, ids = torch.zeros((4, 16), dtype=bf), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="x must be"):
        epm.adapter_product(x.float(), ids, x, x, x)
    with pytest.raises(ValueError, match="x must be"):
        epm.adapter_product(x, ids, x, x, x)  # not on the device
