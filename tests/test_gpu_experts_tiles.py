"""The kernels of large batches: tiles of 256 rows in bf16 and FP8 at each height
their last tiles are computed at, launches of more tiles than compute units, and
batches of more experts than a block has threads.  References and bounds are those
of test_gpu_experts.py; the launch log says which tiles a call took, so that a
change of the rules cannot take these shapes elsewhere unseen."""

from __future__ import annotations

import ctypes
import re
import sys

import pytest
import torch

import test_gpu_experts as base

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


@pytest.fixture
def heights(monkeypatch, capfd):
    """The heights of the tiles launched so far, by the launch's name."""
    monkeypatch.setenv("EP_LOG", "1")

    def read():
        found = {}
        for what, bm in re.findall(r"^\[ep\] ([^:]*): .* tile=(\d+)x", capfd.readouterr().err, re.M):
            found.setdefault(what, set()).add(int(bm))
        return found
    return read


# rows of an expert: last tiles of up to 64, 128, 192 and 256 rows, none, and alone
SIZES = [300, 340, 400, 470, 256, 512, 30, 200, 129, 0, 258, 600]
T, E, R, K = sum(SIZES), 2 * len(SIZES), 4, 2


def sized(monkeypatch):
    """Every token goes to an even and to an odd expert, of which there are these many rows each."""
    def routing(g, tokens, experts, k, mask, dup=False):
        assert (tokens, experts, k) == (T, E, K)
        n = torch.tensor(SIZES, device="cuda")
        half = torch.arange(E // 2, device="cuda").repeat_interleave(n)
        halves = [half[torch.randperm(T, generator=g, device="cuda")] for _ in range(K)]
        topk = torch.stack((2 * halves[0], 2 * halves[1] + 1), 1).contiguous()
        return topk, torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1)
    monkeypatch.setattr(base, "routing", routing)


# H, I and the heights of the gated, the down, the gate's backward and the dx product:
# whole steps of K, one step with a tail and many columns, two steps and many columns
WIDTHS = [(1280, 1024, (256, 256, 256, 256)), (72, 2056, (256, 64, 256, 64)), (2056, 40, (64, 256, 64, 256))]


@pytest.mark.parametrize("H,I,want", WIDTHS)
def test_expert_ffn_and_gradients(monkeypatch, heights, H, I, want):
    sized(monkeypatch)
    base.test_expert_ffn_and_gradients(T, H, I, E, R, K, 0.0, False)
    names = ("expert_ffn gated", "expert_ffn down", "expert_ffn gate backward", "expert_ffn dx")
    assert heights() == {n: {h} for n, h in zip(names, want)}


@pytest.mark.parametrize("H,I,want", WIDTHS)
def test_low_latency_expert_ffn(monkeypatch, heights, H, I, want):
    sized(monkeypatch)
    base.test_low_latency_expert_ffn(T, H, I, E, R, K, 0.0)
    assert heights() == {"ll_expert_ffn gated": {want[0]}, "ll_expert_ffn down": {want[1]}}


@pytest.mark.parametrize("H,I,want", [(1280, 1024, (256, 256)), (128, 2048, (256, 64)), (2048, 128, (64, 256)),
                                      (768, 384, (256, 256))])
def test_low_latency_expert_ffn_fp8(monkeypatch, heights, H, I, want):
    """Every code of a large batch is held to its own bound, the 8-bit instruction's alignment in it."""
    sized(monkeypatch)
    base.test_low_latency_expert_ffn_fp8(T, H, I, E, R, K, 0.0)
    assert heights() == {"ll_expert_ffn_fp8 gated tiles": {want[0]}, "ll_expert_ffn_fp8 down tiles": {want[1]}}


# the last row tile at each height, columns that end inside a tile and inside a scale
# block, one to ten steps of K, one row tile of many columns
@pytest.mark.parametrize("M,N,K", [(8229, 1536, 128), (8292, 1536, 256), (8342, 1544, 384), (8406, 1608, 1280),
                                   (70, 33000, 256), (256, 33000, 128)])
def test_fp8_product(heights, M, N, K):
    base.test_fp8_product(M, N, K)
    assert heights() == {"fp8_product": {256}}


# rows of an expert: 20 on average, in tiles of 64 rows; fewer pairs than experts, K split
@pytest.mark.parametrize("tokens,experts,k,tile", [(3000, 600, 4, {64}), (20, 1200, 4, None)])
def test_more_experts_than_threads(heights, tokens, experts, k, tile):
    base.test_expert_ffn_and_gradients(tokens, 64, 64, experts, 8, k, 0.1, False)
    assert heights().get("expert_ffn gated") == tile
    base.test_low_latency_expert_ffn(tokens, 64, 64, experts, 8, k, 0.1)
    assert heights().get("ll_expert_ffn gated") == tile
    base.test_low_latency_expert_ffn_fp8(tokens, 128, 128, experts, 8, k, 0.1)
    assert heights().get("ll_expert_ffn_fp8 gated tiles") == tile


def quantised(buf, topk, x, w13, w2):
    """Slots, codes and scales of the activation, and the outputs of an FP8 batch."""
    tokens, H = x.shape
    S, I, abi = tokens, w2[0].shape[2], base.abi
    (q, sc), count, hdl, _, _ = buf.low_latency_dispatch(x, topk, S, use_fp8=True)
    shape = q.shape[:3]
    aq = torch.zeros((*shape, I), dtype=torch.uint8, device="cuda")
    asc = torch.zeros((*shape, I // 128), device="cuda")
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    d = abi.dims(tokens, H, topk.shape[1], buf.num_experts, buf.num_ranks)
    abi.check(abi.lib().ep_ll_expert_ffn_fp8(
        ctypes.byref(d), S, I, *[abi.ptr(t) for t in (q, sc, count, *w13, *w2, aq, asc, out)],
        abi.current_stream()), "ep_ll_expert_ffn_fp8")
    return hdl.topk_slot.long(), aq.view(torch.float8_e4m3fn), asc, q, sc


def test_fp8_codes_of_a_token_in_a_small_and_a_large_batch(heights):
    """The gated products of few activations are fp32 sums, those of many are the 8-bit
    instruction's: in each batch a token's codes are those of a value within its sum's
    bound of the exact activation."""
    few, tokens, experts, ranks, k, H, I = 6, 600, 8, 4, 3, 2048, 1024
    g = base.gen(11)
    topk, _ = base.routing(g, tokens, experts, k, 0.0)
    x = base.normal(g, (tokens, H))
    w13, w2 = base.fp8_weight(g, (experts, 2 * I, H)), base.fp8_weight(g, (experts, H, I))
    v13, v2 = base.weight_value(w13), base.weight_value(w2)
    buf = base.epm.Buffer(ranks, experts)
    small = quantised(buf, topk[:few].contiguous(), x[:few].contiguous(), w13, w2)
    assert heights() == {}  # K split
    large = quantised(buf, topk, x, w13, w2)
    assert "ll_expert_ffn_fp8 gated tiles" in heights()
    epr = experts // ranks
    for t in range(few):
        for j in range(k):
            e = int(topk[t, j])
            le, r = e % epr, e // epr
            values, bounds = [], []
            for (slot, codes, scales, q, sc), fp8 in ((small, False), (large, True)):
                at = (le, r, int(slot[t, j]))
                row = base.rows_value((q[at][None], sc[at][None]))
                _, _, _, act, _, _, eact = base.ffn_ref(row, v13[e], v2[e], fp8=fp8)
                s = scales[at].double().repeat_interleave(128)[None]
                value = codes[at].double()[None] * s
                # half a step, the sum's own error, and the code's two fp32 roundings
                tol = torch.maximum((act.abs() + eact) * 2.0 ** -4, s * 2.0 ** -10) + eact + 8 * base.U * act.abs()
                base.close(value, act, tol, f"token {t}, expert {e}, {'large' if fp8 else 'small'} batch")
                values.append(value)
                bounds.append(tol)
            base.close(values[0], values[1], bounds[0] + bounds[1], "between the batches")
