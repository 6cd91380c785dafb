"""The products of few rows or few tiles at the borders between their kernels: K
split over a block's waves, tiles of 64 rows, and batches whose groups take
different ones.  References and bounds are those of test_gpu_experts.py."""

from __future__ import annotations

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


# M: one, two and four row tiles, a block for each 64 rows, as many blocks as
# compute units and one run more; N: inside one block, more blocks than compute units
@pytest.mark.parametrize("M,N,K", [(2, 8, 128), (16, 72, 1408), (17, 1000, 256), (32, 64, 4096), (33, 72, 1152),
                                   (64, 7168, 128), (129, 40, 640), (700, 512, 384), (4090, 200, 256),
                                   (4100, 200, 256), (16384, 64, 128), (3, 66000, 128), (5, 66000, 128),
                                   (40, 66000, 256)])
def test_fp8_product(M, N, K):
    base.test_fp8_product(M, N, K)


def skewed(monkeypatch):
    """Expert 5 gets a slot of every token, the other slots go elsewhere."""
    plain = base.routing

    def routing(g, T, E, K, mask, dup=False):
        topk, w = plain(g, T, E, K, mask, dup)
        topk = torch.where(topk == 5, 6, topk)
        topk[:, 0] = 5
        return topk, w
    monkeypatch.setattr(base, "routing", routing)


# rows of a group on average: 1, 2, 12, 24, 48, 4 of many, past 64
CELLS = [(5, 264, 72, 16, 4, 4, 0.0), (16, 1024, 128, 64, 8, 8, 0.1), (12, 328, 200, 2, 1, 2, 0.0),
         (24, 72, 136, 2, 1, 2, 0.0), (48, 520, 64, 2, 2, 2, 0.0), (64, 1024, 512, 64, 4, 4, 0.0),
         (70, 264, 136, 3, 3, 2, 0.1)]


@pytest.mark.parametrize("T,H,I,E,R,K,mask", CELLS)
def test_low_latency_expert_ffn(T, H, I, E, R, K, mask):
    base.test_low_latency_expert_ffn(T, H, I, E, R, K, mask)


# the crowded expert's rows in one block's runs, in several blocks, and in tiles (past 16 runs)
@pytest.mark.parametrize("T,H,I,E,R,K", [(60, 200, 72, 64, 8, 2), (100, 136, 200, 64, 8, 2), (64, 1024, 512, 64, 4, 4),
                                         (300, 72, 64, 128, 8, 2), (90, 64, 40, 8, 2, 2)])
def test_low_latency_expert_ffn_skewed(monkeypatch, T, H, I, E, R, K):
    skewed(monkeypatch)
    base.test_low_latency_expert_ffn(T, H, I, E, R, K, 0.0)


FP8_CELLS = [(5, 256, 128, 16, 4, 4, 0.0), (16, 1024, 128, 64, 8, 8, 0.1), (12, 384, 256, 2, 1, 2, 0.0),
             (24, 128, 128, 2, 1, 2, 0.0), (48, 512, 128, 2, 2, 2, 0.0), (64, 1024, 512, 64, 4, 4, 0.0),
             (150, 256, 1024, 4, 2, 2, 0.1)]


@pytest.mark.parametrize("T,H,I,E,R,K,mask", FP8_CELLS)
def test_low_latency_expert_ffn_fp8(T, H, I, E, R, K, mask):
    base.test_low_latency_expert_ffn_fp8(T, H, I, E, R, K, mask)


@pytest.mark.parametrize("T,H,I,E,R,K", [(60, 256, 128, 64, 8, 2), (100, 128, 256, 64, 8, 2), (64, 1024, 512, 64, 4, 4),
                                         (300, 128, 128, 128, 8, 2), (20, 128, 128, 8, 2, 2),
                                         (60, 128, 128, 8, 2, 2)])
def test_low_latency_expert_ffn_fp8_skewed(monkeypatch, T, H, I, E, R, K):
    skewed(monkeypatch)
    base.test_low_latency_expert_ffn_fp8(T, H, I, E, R, K, 0.0)


@pytest.mark.parametrize("T,H,I,E,R,K", [(6, 256, 128, 1, 1, 1), (24, 128, 128, 2, 1, 1), (40, 1408, 256, 4, 2, 2),
                                         (64, 1024, 384, 64, 4, 4)])
def test_fp8_activations_of_small_batches_keep_their_codes(monkeypatch, T, H, I, E, R, K):
    """Few activations (below 2^17): the gated products are fp32 sums of exact
    terms, so codes and scales hold without the 8-bit instruction's own error."""
    plain = base.ffn_ref
    monkeypatch.setattr(base, "ffn_ref", lambda x, w13, w2, fp8=False: plain(x, w13, w2))
    base.test_low_latency_expert_ffn_fp8(T, H, I, E, R, K, 0.0)


@pytest.mark.parametrize("M,N,K", [(12, 200, 384), (40, 200, 384), (300, 200, 384), (5000, 520, 256)])
def test_not_finite_row_of_a_product_stays_alone(M, N, K):
    g = base.gen(M)
    (q, sc), w = base.fp8_rows(g, (M, K)), base.fp8_weight(g, (N, K))
    want = base.epm.fp8_product((q, sc), w)
    sc = sc.clone()
    sc[M // 3] = float("nan")
    sc[M - 1, 0] = float("inf")
    got = base.epm.fp8_product((q, sc), w)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[M // 3] = keep[M - 1] = False
    assert torch.equal(got[keep], want[keep])
    assert got[M // 3].isnan().all() and not got[M - 1].isfinite().any()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T,E,R,K", [(6, 8, 4, 2), (60, 4, 2, 2), (200, 3, 1, 2)])
def test_unused_cells_and_experts_may_hold_anything(T, E, R, K, fp8):
    g = base.gen(T)
    H, I = 256, 128
    topk, _ = base.routing(g, T, E, K, 0.1)
    topk = torch.where(topk == 1, -1, topk)  # expert 1 has no row
    buf = base.epm.Buffer(R, E)
    packed, count, h, _, _ = buf.low_latency_dispatch(base.normal(g, (T, H)), topk, T + 2, use_fp8=fp8)
    if fp8:
        w13, w2 = base.fp8_weight(g, (E, 2 * I, H)), base.fp8_weight(g, (E, H, I))
        cells, weights = packed[1], (w13[1], w2[1])
    else:
        w13, w2 = base.normal(g, (E, 2 * I, H), H ** -0.5), base.normal(g, (E, H, I), I ** -0.5)
        cells, weights = packed, (w13, w2)
    unused = torch.arange(T + 2, device="cuda") >= count[..., None]
    outs = []
    for fill in (0.0, float("nan")):
        cells[unused] = fill
        for w in weights:
            w[1] = fill
        out = torch.full((E // R, R, T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
        outs.append(buf.low_latency_expert_ffn(packed, count, h, w13, w2, out=out))
    assert (outs[0][unused] == 7.0).all() and outs[0].isfinite().all()
    assert torch.equal(outs[0], outs[1])


# dispatched rows on the few-rows kernels: rows of an expert 1, 12, 24 and 40 on average,
# many experts, one expert past 64 rows beside small ones, widths that end inside a K step
DISPATCHED = [(3, 200, 72, 16, 4, 4, 0.0, False), (12, 328, 136, 2, 1, 2, 0.0, False),
              (24, 72, 200, 2, 2, 2, 0.1, False), (40, 136, 64, 3, 3, 3, 0.0, False),
              (64, 1024, 512, 64, 4, 4, 0.0, False), (100, 136, 200, 64, 8, 2, 0.0, True),
              (300, 72, 64, 128, 8, 2, 0.0, True)]


@pytest.mark.parametrize("T,H,I,E,R,K,mask,skew", DISPATCHED)
def test_expert_ffn_and_gradients(monkeypatch, T, H, I, E, R, K, mask, skew):
    if skew:
        skewed(monkeypatch)
    base.test_expert_ffn_and_gradients(T, H, I, E, R, K, mask, False)
