"""The router's refusals, without a GPU: the C ABI turns bad arguments down before any
device call, and the binding turns down tensors of another type, shape or place."""

from __future__ import annotations

import copy
import ctypes
import dataclasses
import pickle

import pytest
import torch

import combine_get_dispatch_05_amd as epm
from combine_get_dispatch_05_amd import abi

L = abi.lib()
A = ctypes.c_void_p(0x10000)  # an aligned address that is never followed
M4 = ctypes.c_void_p(0x10004)
M2 = ctypes.c_void_p(0x10002)
M1 = ctypes.c_void_p(0x10001)
INV, ALIGN, CAP = abi.EP_ERR_INVALID, abi.EP_ERR_ALIGN, abi.EP_ERR_CAPACITY


def call(fn, good, **bad):
    assert not set(bad) - set(good), bad
    return fn(*{**good, **bad}.values())


def dims(*a):
    return ctypes.byref(abi.dims(*a))


def rule(score=0, groups=1, kept=1, normalize=1, scale=1.0):
    return ctypes.byref(abi.RouterRule(score, groups, kept, normalize, scale))


BAD_DIMS = [(-1, 8, 2, 8, 4), ((1 << 24) + 1, 8, 2, 8, 4), (4, 8, 0, 8, 4), (4, 8, 65, 128, 4), (4, 8, 2, 10, 4),
            (4, 8, 2, 1024, 1024), (4, 8, 2, 16384, 4), (4, 8, 2, 0, 1)]
BAD_RULES = [dict(score=2), dict(score=-1), dict(groups=0), dict(groups=3), dict(groups=2, kept=3), dict(kept=0),
             dict(scale=float("inf")), dict(scale=float("nan"))]


def test_route_rules():
    n = L.ep_route_workspace(dims(16, 8, 2, 8, 4))
    assert n > 0 and n % (8 * 4) == 0
    assert L.ep_route_workspace(dims(0, 8, 2, 8, 4)) == 0
    assert L.ep_route_workspace(None) == 0
    assert L.ep_route_workspace(dims(1 << 24, 8, 2, 8192, 4)) <= 512 * 8192 * 4
    good = dict(d=dims(16, 8, 2, 8, 4), rule=rule(), logits=A, bf16=0, bias=A, mask=A, idx=A, w=A, sums=A, work=A,
                size=n, stream=None)
    f = L.ep_route
    for bad in BAD_DIMS:
        assert call(f, good, d=dims(*bad)) == INV, bad
    for bad in BAD_RULES:
        assert call(f, good, rule=rule(**bad)) == INV, bad
    assert call(f, good, rule=rule(groups=65), d=dims(16, 8, 2, 130, 1)) == INV  # too many groups
    for bad in (dict(d=None), dict(rule=None), dict(logits=None), dict(idx=None), dict(w=None), dict(work=None)):
        assert call(f, good, **bad) == INV, bad
    for bad in (dict(logits=M2), dict(logits=M1, bf16=1), dict(bias=M2), dict(mask=M2), dict(idx=M4), dict(w=M2),
                dict(sums=M2), dict(work=M2)):
        assert call(f, good, **bad) == ALIGN, bad
    assert call(f, good, size=n - 1) == CAP


def test_route_backward_rules():
    good = dict(d=dims(16, 8, 2, 8, 4), rule=rule(), dw=A, logits=A, bf16=0, idx=A, dsums=A, dlogits=A, stream=None)
    f = L.ep_route_backward
    for bad in BAD_DIMS:
        assert call(f, good, d=dims(*bad)) == INV, bad
    for bad in BAD_RULES:
        assert call(f, good, rule=rule(**bad)) == INV, bad
    for bad in (dict(d=None), dict(rule=None), dict(dw=None), dict(logits=None), dict(idx=None), dict(dlogits=None)):
        assert call(f, good, **bad) == INV, bad
    for bad in (dict(dw=M2), dict(logits=M2), dict(logits=M1, bf16=1), dict(idx=M4), dict(dsums=M2), dict(dlogits=M2)):
        assert call(f, good, **bad) == ALIGN, bad
    assert call(f, good, d=dims(0, 8, 2, 8, 4)) == abi.EP_OK  # nothing to do


def test_binding_refuses_before_the_library():
    buf, r = epm.Buffer(2, 8), epm.Router(2)
    with pytest.raises(TypeError, match="logits must be"):
        buf.route(torch.zeros((4, 8), dtype=torch.float64), r)
    with pytest.raises(ValueError, match="logits must"):
        buf.route(torch.zeros((4, 8)), r)  # not on the device
    with pytest.raises(ValueError, match="score must be"):
        epm.Router(2, score="tanh")


def test_a_router_is_copied_pickled_and_compared_by_what_it_says():
    r = epm.Router(6, score="sigmoid", num_groups=8, topk_groups=4, normalize=False, scale=2.5)
    for other in (copy.copy(r), copy.deepcopy({"r": r})["r"], pickle.loads(pickle.dumps(r)), dataclasses.replace(r)):
        assert other == r and hash(other) == hash(r)
        raw = other._raw._obj
        assert (raw.score, raw.num_groups, raw.topk_groups, raw.normalize, raw.scale) == (1, 8, 4, 0, 2.5)


def test_counts_past_32_bits_do_not_wrap():
    for wrong in (dict(num_topk=2 ** 32 + 8), dict(num_topk=8, num_groups=2 ** 32 + 1),
                  dict(num_topk=8, topk_groups=-2 ** 40)):
        with pytest.raises(ValueError, match="32 bits"):
            epm.Router(**wrong)
