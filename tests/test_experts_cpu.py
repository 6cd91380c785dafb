"""The expert operations' refusals, without a GPU: the C ABI turns bad arguments
down before any device call, and the binding turns down tensors of another type,
shape or place."""

from __future__ import annotations

import ctypes

import pytest
import torch

import combine_get_dispatch_05_amd as epm
from combine_get_dispatch_05_amd import abi

L = abi.lib()
A = ctypes.c_void_p(0x10000)    # an aligned address that is never followed
M8 = ctypes.c_void_p(0x10008)   # 8-byte aligned
M4 = ctypes.c_void_p(0x10004)
M2 = ctypes.c_void_p(0x10002)
INV, ALIGN, CAP = abi.EP_ERR_INVALID, abi.EP_ERR_ALIGN, abi.EP_ERR_CAPACITY


def call(fn, good, **bad):
    """fn with the named good arguments, some replaced."""
    assert not set(bad) - set(good), bad
    return fn(*{**good, **bad}.values())


def test_rms_norm_rules():
    good = dict(T=4, H=256, eps=1e-6, x=A, residual=A, weight=A, residual_out=A, out=A, q=A, scale=A, rstd=A,
                stream=None)
    f = L.ep_rms_norm
    for bad in (dict(T=-1), dict(T=(1 << 24) + 1), dict(H=0), dict(H=(1 << 20) + 8), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(weight=None),
                dict(residual=None), dict(out=None, q=None, scale=None), dict(scale=None), dict(q=None)):
        assert call(f, good, **bad) == INV, bad
    for bad in (dict(H=12), dict(H=192), dict(x=M8), dict(residual=M8), dict(weight=M8), dict(residual_out=M8),
                dict(out=M8), dict(q=M4), dict(scale=M2), dict(rstd=M2)):
        assert call(f, good, **bad) == ALIGN, bad
    assert call(f, good, T=0, H=192) == ALIGN


def test_rms_norm_backward_rules():
    n = L.ep_rms_norm_backward_workspace(4, 256)
    assert n == 4 * 256 * 4
    assert L.ep_rms_norm_backward_workspace(0, 256) == 0
    assert L.ep_rms_norm_backward_workspace(4, 12) == 0
    assert L.ep_rms_norm_backward_workspace(1 << 24, 1 << 20) >= (1 << 20) * 4  # fits size_t
    good = dict(T=4, H=256, dout=A, h=A, weight=A, rstd=A, dresidual=A, dx=A, dweight=A, work=A, size=n, stream=None)
    f = L.ep_rms_norm_backward
    for bad in (dict(T=-1), dict(H=0), dict(dout=None), dict(h=None), dict(weight=None), dict(rstd=None),
                dict(dx=None), dict(dweight=None), dict(work=None)):
        assert call(f, good, **bad) == INV, bad
    for bad in (dict(H=12), dict(dout=M8), dict(h=M8), dict(weight=M8), dict(dresidual=M8), dict(dx=M8),
                dict(work=M8), dict(rstd=M2), dict(dweight=M2)):
        assert call(f, good, **bad) == ALIGN, bad
    assert call(f, good, size=n - 1) == CAP


def test_fp8_product_rules():
    good = dict(m=4, n=64, k=256, aq=A, asc=A, wq=A, wsc=A, out=A, stream=None)
    f = L.ep_fp8_product
    for bad in (dict(m=-1), dict(m=(1 << 24) + 1), dict(n=0), dict(k=0), dict(k=(1 << 20) + 128),
                dict(n=(1 << 20) + 8), dict(aq=None), dict(asc=None), dict(wq=None), dict(wsc=None),
                dict(out=None), dict(m=1 << 24, n=1 << 20)):
        assert call(f, good, **bad) == INV, bad
    for bad in (dict(k=192), dict(n=12), dict(aq=M8), dict(wq=M8), dict(out=M8), dict(asc=M2), dict(wsc=M2)):
        assert call(f, good, **bad) == ALIGN, bad
    assert call(f, good, m=0) == abi.EP_OK


def bad_dims():
    """(dims, code): T, H, K, E, R"""
    return [((-1, 256, 2, 8, 4), INV), ((4, 0, 2, 8, 4), INV), ((4, 12, 2, 8, 4), ALIGN), ((4, 256, 0, 8, 4), INV),
            ((4, 256, 65, 128, 4), INV), ((4, 256, 2, 10, 4), INV), ((4, 256, 2, 1024, 1024), INV),
            ((4, 256, 2, 16384, 4), INV)]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_low_latency_expert_ffn_rules(fp8):
    d = abi.dims(16, 256, 2, 8, 4)
    head = dict(d=ctypes.byref(d), slots=16, inter=128)
    if fp8:
        f = L.ep_ll_expert_ffn_fp8
        ptrs = ["q", "sc", "count", "w13", "s13", "w2", "s2", "aq", "asc", "out"]
        small = {"sc", "count", "s13", "s2", "asc"}
    else:
        f = L.ep_ll_expert_ffn
        ptrs = ["x", "count", "w13", "w2", "act", "out"]
        small = {"count"}
    good = {**head, **{p: A for p in ptrs}, "stream": None}
    for p in ptrs:
        assert call(f, good, **{p: None}) == INV, p
        assert call(f, good, **{p: M2 if p in small else M8}) == ALIGN, p
    assert call(f, good, d=None) == INV
    assert call(f, good, slots=0) == INV
    assert call(f, good, slots=5000) == INV
    assert call(f, good, slots=15) == CAP  # fewer slots than tokens
    assert call(f, good, inter=0) == INV
    assert call(f, good, inter=(1 << 20) + 128) == INV
    assert call(f, good, inter=12 if not fp8 else 64) == ALIGN
    if fp8:
        assert call(f, good, d=ctypes.byref(abi.dims(16, 192, 2, 8, 4))) == ALIGN
    for dims, code in bad_dims():
        assert call(f, good, d=ctypes.byref(abi.dims(*dims))) == code, dims
    assert call(f, good, d=ctypes.byref(abi.dims(0, 256, 2, 8, 4))) == abi.EP_OK  # nothing to do


def test_expert_rows_rules():
    d = abi.dims(16, 8, 2, 8, 4)
    good = dict(d=ctypes.byref(d), prefix=A, ids=A, rows=20, cap=32, counts=A, offsets=A, pair_row=A, pair_slot=A,
                row_pair=A, stream=None)
    f = L.ep_expert_rows
    for p in ("prefix", "ids", "counts", "offsets", "pair_row", "pair_slot", "row_pair"):
        assert call(f, good, **{p: None}) == INV, p
        assert call(f, good, **{p: M4 if p == "ids" else M2}) == ALIGN, p
    for bad in (dict(d=None), dict(rows=-1), dict(cap=-1), dict(rows=1 << 30), dict(rows=1 << 62),
                dict(cap=1 << 31)):
        assert call(f, good, **bad) == INV, bad
    assert call(f, good, cap=31) == CAP
    assert call(f, good, rows=3, cap=5) == CAP
    for dims, code in bad_dims():
        assert call(f, good, d=ctypes.byref(abi.dims(*dims))) == code, dims


@pytest.mark.parametrize("back", [False, True], ids=["forward", "backward"])
def test_expert_ffn_rules(back):
    d = abi.dims(0, 256, 2, 8, 4)

    def groups(**kw):
        v = {**dict(rows=20, cap=32, off=0x10000, pr=0x10000, ps=0x10000, rp=0x10000), **kw}
        return ctypes.byref(abi.ExpertGroups(*v.values()))

    if back:
        f = L.ep_expert_ffn_backward
        ptrs = ["dy", "x", "tw", "w13", "w2", "gu", "dgu", "act", "terms", "parts", "dx", "dtw", "dw13", "dw2"]
        small, free = {"tw", "dtw", "parts"}, set()
    else:
        f = L.ep_expert_ffn
        ptrs = ["x", "tw", "w13", "w2", "act", "gu", "terms", "y"]
        small, free = {"tw"}, {"gu"}
    good = {"d": ctypes.byref(d), "inter": 64, "g": groups(), **{p: A for p in ptrs}, "stream": None}
    for p in ptrs:
        if p not in free:
            assert call(f, good, **{p: None}) == INV, p
        assert call(f, good, **{p: M2 if p in small else M8}) == ALIGN, p
    for g, code in ((None, INV), (groups(rows=-1), INV), (groups(cap=-1), INV), (groups(off=None), INV),
                    (groups(pr=None), INV), (groups(ps=None), INV), (groups(rp=None), INV),
                    (groups(rows=1 << 31), INV), (groups(cap=1 << 31), INV), (groups(off=0x10002), ALIGN),
                    (groups(rp=0x10002), ALIGN)):
        assert call(f, good, g=g) == code
    assert call(f, good, inter=0) == INV
    assert call(f, good, inter=12) == ALIGN
    for dims, code in bad_dims():
        assert call(f, good, d=ctypes.byref(abi.dims(*dims))) == code, dims
    # more blocks than a launch holds
    assert call(f, good, d=ctypes.byref(abi.dims(0, 1 << 20, 2, 8192, 4)), inter=1 << 20) == INV


def test_binding_refuses_before_the_library():
    bf, buf = torch.bfloat16, epm.Buffer(2, 4)
    x = torch.zeros((4, 256), dtype=bf)
    w = torch.zeros(256, dtype=bf)
    with pytest.raises(ValueError, match="device tensor"):
        epm.rms_norm(x, w)
    with pytest.raises(TypeError, match="x must be"):
        epm.rms_norm(x.float(), w)
    with pytest.raises(TypeError, match="pair"):
        epm.fp8_product(x, (x, x))
    with pytest.raises(TypeError, match="codes must be"):
        epm.fp8_product((x, x), (x, x))
    with pytest.raises(TypeError, match="recv_topk_idx must be"):
        buf.expert_rows(torch.zeros((4, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError, match="packed_count must be"):
        buf.low_latency_expert_ffn(x, torch.zeros((2, 2)), None, None, None)
