"""The few-token layer's refusals, without a GPU."""

from __future__ import annotations

import ctypes

import pytest
import torch

import combine_get_dispatch_05_amd as epm
from combine_get_dispatch_05_amd import abi
from test_router_cpu import A, ALIGN, BAD_RULES, CAP, INV, M2, M4, call, dims, rule

L = abi.lib()
M128 = ctypes.c_void_p(0x10080)
M8 = ctypes.c_void_p(0x10008)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_low_latency_moe_rules(fp8):
    n = L.ep_ll_moe_workspace(dims(16, 256, 2, 8, 4), 128)
    assert n >= 16 * 8 * 4 + 32 * 8 + 32 * 128 * 2
    scale = A if fp8 else None
    good = dict(d=dims(16, 256, 2, 8, 4), inter=128, rule=rule(), x=A, wr=A, f32=0, bias=A, mask=A, w13=A, s13=scale,
                w2=A, s2=scale, res=A, idx=A, w=A, y=A, work=A, size=n, stream=None)
    f = L.ep_ll_moe
    for bad in ((-1, 256, 2, 8, 4), (4, 0, 2, 8, 4), (4, 256, 0, 8, 4), (4, 256, 65, 128, 4), (4, 256, 2, 10, 4),
                (4, 256, 2, 16384, 4), (4, (1 << 20) + 128, 2, 8, 4)):
        assert call(f, good, d=dims(*bad)) == INV, bad
    for bad in BAD_RULES:
        assert call(f, good, rule=rule(**bad)) == INV, bad
    for p in ("d", "rule", "x", "wr", "w13", "w2", "idx", "w", "y", "work"):
        assert call(f, good, **{p: None}) == INV, p
    assert call(f, good, s13=None if fp8 else A) == INV
    for p in ("x", "wr", "w13", "w2", "res", "y"):
        assert call(f, good, **{p: M8}) == ALIGN, p
    for bad in (dict(idx=M4), dict(w=M2), dict(bias=M2), dict(mask=M2), dict(work=M128),
                dict(d=dims(16, 192 if fp8 else 12, 2, 8, 4)), dict(inter=192 if fp8 else 12)):
        assert call(f, good, **bad) == ALIGN, bad
    if fp8:
        assert call(f, good, s13=M2) == ALIGN and call(f, good, s2=M2) == ALIGN
    assert call(f, good, d=dims(65, 256, 2, 8, 4)) == abi.EP_ERR_TOO_LARGE
    assert call(f, good, d=dims(4, 256, 2, 516, 4)) == abi.EP_ERR_TOO_LARGE
    assert call(f, good, size=n - 1) == CAP
    assert call(f, good, d=dims(0, 256, 2, 8, 4)) == abi.EP_OK  # nothing to do
    assert L.ep_ll_moe_workspace(dims(65, 256, 2, 8, 4), 128) == 0
    assert L.ep_ll_moe_workspace(dims(4, 256, 2, 516, 4), 128) == 0
    assert L.ep_ll_moe_workspace(None, 128) == 0


def test_binding_refuses_before_the_library():
    buf, r = epm.Buffer(2, 8), epm.Router(2)
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="x must be"):
        buf.low_latency_moe(x.float(), x, r, x, x)
    with pytest.raises(ValueError, match="x must be"):
        buf.low_latency_moe(x, x, r, x, x)  # not on the device
