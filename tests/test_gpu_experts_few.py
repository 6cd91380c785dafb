"""The products of few rows or few tiles at the borders between their kernels: K
split over a block's waves, wide blocks, tiles of 64 rows, and batches whose groups
take different ones.  References and bounds are those of test_gpu_experts.py."""

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
# compute units and one run more; N: inside one block, wide enough for wide blocks
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


# rows of a group on average: 1, 2, 12, 24, 48; wide blocks (64 experts x 4); past 64 rows
CELLS = [(5, 264, 72, 16, 4, 4, 0.0), (16, 1024, 128, 64, 8, 8, 0.1), (12, 328, 200, 2, 1, 2, 0.0),
         (24, 72, 136, 2, 1, 2, 0.0), (48, 520, 64, 2, 2, 2, 0.0), (64, 1024, 512, 64, 4, 4, 0.0),
         (70, 264, 136, 3, 3, 2, 0.1)]


@pytest.mark.parametrize("T,H,I,E,R,K,mask", CELLS)
def test_low_latency_expert_ffn(T, H, I, E, R, K, mask):
    base.test_low_latency_expert_ffn(T, H, I, E, R, K, mask)


@pytest.mark.parametrize("T,H,I,E,R,K", [(60, 200, 72, 64, 8, 2), (100, 136, 200, 64, 8, 2), (64, 1024, 512, 64, 4, 4)])
def test_low_latency_expert_ffn_skewed(monkeypatch, T, H, I, E, R, K):
    skewed(monkeypatch)
    base.test_low_latency_expert_ffn(T, H, I, E, R, K, 0.0)


FP8_CELLS = [(5, 256, 128, 16, 4, 4, 0.0), (16, 1024, 128, 64, 8, 8, 0.1), (12, 384, 256, 2, 1, 2, 0.0),
             (24, 128, 128, 2, 1, 2, 0.0), (48, 512, 128, 2, 2, 2, 0.0), (64, 1024, 512, 64, 4, 4, 0.0),
             (150, 256, 1024, 4, 2, 2, 0.1)]


@pytest.mark.parametrize("T,H,I,E,R,K,mask", FP8_CELLS)
def test_low_latency_expert_ffn_fp8(T, H, I, E, R, K, mask):
    base.test_low_latency_expert_ffn_fp8(T, H, I, E, R, K, mask)


@pytest.mark.parametrize("T,H,I,E,R,K", [(60, 256, 128, 64, 8, 2), (100, 128, 256, 64, 8, 2), (64, 1024, 512, 64, 4, 4)])
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
