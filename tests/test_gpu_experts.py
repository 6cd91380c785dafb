"""The expert operations against their formulas in 64 bits: the norm with its
gradients, the FP8 block product, rows grouped by expert, the gated feed-forward
with its gradients, and the low-latency cells.

Every bound is the sum of the roundings a result goes through, taken at their
worst: half a step for each value kept in fewer bits (bf16 2^-8 of the value,
e4m3 2^-4 or half its smallest step), and n * 2^-24 of the summed magnitudes for
an fp32 sum of n terms (twice that for the matrix instructions, whose inner
adds need not round to nearest).  The FP8 matrix instructions add the products
of each eight neighbouring k after aligning them to the largest: fp8_sum_err."""

from __future__ import annotations

import ctypes
import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402
from combine_get_dispatch_05_amd import abi  # noqa: E402

BF, U = 2.0 ** -8, 2.0 ** -24
TINY = 2.0 ** -60


@pytest.fixture(autouse=True)
def _announce(request):
    sys.__stderr__.write(f"\n[gpu-test] {request.node.nodeid}\n")
    sys.__stderr__.flush()
    yield
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def close(got, ref, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - tol
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} out, by up to {worst:.3g}"


def sum_err(n):
    """Relative error bound of an n-term fp32 matrix sum, of the summed magnitudes."""
    return 2 * (n + 8) * U


def fp8_sum_err(a, w):
    """What the FP8 matrix instruction's alignment can lose in a @ w.t(), besides sum_err.

    It adds the products of eight neighbouring k after shifting them to the exponent
    of the largest, 2^E, and drops what falls below 2^(E - 13): next to a product of
    2^16 one of 2^3 is kept whole and one of 2^2 is lost, both ways round in sign
    (test_fp8_product_alignment).  So each of the other seven products of an eight loses
    less than 2^-13 of the eight's largest, which is at most max|a| max|w| over it."""
    def most(v):
        return v.abs().unflatten(-1, (-1, 8)).amax(-1)
    return 7 * 2.0 ** -13 * (most(a) @ most(w).t())


def quantise(v):
    """fp64 rows in the FP8 dispatch's format: codes (as values) and scales."""
    b = v.reshape(*v.shape[:-1], -1, 128)
    amax = b.abs().amax(-1, keepdim=True).clamp_min(1e-4)
    t = (b * (448.0 / amax)).float().to(torch.float8_e4m3fn)
    return t.view(v.shape), (amax / 448.0).squeeze(-1).float()


def fp8_rows(g, shape, scale=1.0):
    return quantise(torch.randn(shape, generator=g, device="cuda", dtype=torch.float64) * scale)


def fp8_weight(g, shape):
    """[.., N, K] weight with one scale per 128 x 128 block (N may end inside one)."""
    *lead, N, K = shape
    nb, kb = -(-N // 128), K // 128
    w = torch.zeros((*lead, nb * 128, K), device="cuda")
    w[..., :N, :] = torch.randn((*lead, N, K), generator=g, device="cuda") / math.sqrt(K)
    b = w.view(*lead, nb, 128, kb, 128)
    amax = b.abs().amax((-3, -1), keepdim=True).clamp_min(1e-4)
    codes = (b * (448.0 / amax)).to(torch.float8_e4m3fn).view(*lead, nb * 128, K)
    scales = (amax / 448.0).view(*lead, nb, kb)
    return codes[..., :N, :].contiguous(), scales.contiguous()


def rows_value(pair):
    q, s = pair
    return q.double() * s.double().repeat_interleave(128, -1)


def weight_value(pair):
    q, s = pair
    return q.double() * s.double().repeat_interleave(128, -1).repeat_interleave(128, -2)[..., :q.shape[-2], :]


# ------------------------------------------------------------------- norm

NORM_SHAPES = [(1, 8), (1, 128), (3, 512), (1, 7168), (130, 640), (5, 2056), (1030, 1280), (2, 7176),
               (1100, 7168), (3, 16384), (2, 40960)]


@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_rms_norm(T, H, residual):
    g = gen(T * 7 + H)
    x, w = normal(g, (T, H)), normal(g, (H,))
    r = normal(g, (T, H), 3.0) if residual else None
    fp8 = H % 128 == 0
    out, pair, res, rstd = epm.rms_norm(x, w, 1e-5, residual=r, use_fp8=fp8)
    s = x.double() + (r.double() if residual else 0)
    ref_rstd = 1 / torch.sqrt((s * s).mean(1) + 1e-5)
    y = s * ref_rstd[:, None] * w.double()
    rel = (H + 16) * U  # the sum of squares, its root and the three products
    close(rstd, ref_rstd, ref_rstd * rel, "rstd")
    close(out, y, y.abs() * (BF + 2 * rel) + TINY, "out")
    if residual:
        close(res, s, s.abs() * (BF + U), "residual_out")
    else:
        assert res is None
    if not fp8:
        assert pair is None
        return
    amax = y.view(T, -1, 128).abs().amax(-1).clamp_min(1e-4)
    close(pair[1], amax / 448, amax / 448 * (rel + 4 * U), "scales")
    t = y.view(T, -1, 128) * (448 / amax)[..., None]
    close(pair[0].view(t.shape), t, (t.abs() * 2.0 ** -4).clamp_min(2.0 ** -10) + 3 * rel * t.abs(), "codes")


def test_rms_norm_zero_rows_floor_and_not_finite():
    H = 256
    x = torch.zeros((4, H), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    x[1] = 2.0 ** -70  # far below the block floor of 1e-4
    x[2, 5] = float("inf")
    x[3, 200] = float("nan")
    out, (q, sc), _, rstd = epm.rms_norm(x, w, 1.0, use_fp8=True)
    assert (out[0] == 0).all() and (q[0].float() == 0).all()
    assert torch.equal(sc[0], torch.full((2,), 1e-4, device="cuda") / 448.0)
    assert rstd[0] == 1.0 and torch.equal(sc[1], sc[0])
    # a row that is not finite says so; the others are as they were
    assert rstd[2] == 0 and out[2, 5].isnan() and (out[2, :5] == 0).all()
    assert rstd[3].isnan() and out[3].isnan().all() and q[3].float().isnan().all()
    # zeros and no eps: the formula's 0 * inf
    assert epm.rms_norm(x[:1], w, 0.0)[0].isnan().all()
    empty = epm.rms_norm(x[:0], w, use_fp8=True)
    assert empty[0].shape == (0, H) and empty[1][1].shape == (0, 2) and empty[3].shape == (0,)


def test_rms_norm_codes_follow_the_dispatch_format():
    """Rows that bf16 holds exactly give the dispatch's own codes and scales."""
    T, H = 16, 512
    g = gen(3)
    x = normal(g, (T, H))
    x[:, 0] = 1.0
    # a norm with rstd exactly 1: mean(x^2) + eps = 1 is not to be had, so the
    # norm's own bf16 output is sent through the dispatch and its codes compared
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    out, (q, sc), _, _ = epm.rms_norm(x, w, use_fp8=True)
    buf = epm.Buffer(1, 1)
    topk = torch.zeros((T, 1), dtype=torch.int64, device="cuda")
    (dq, dsc), _, _, _, _ = buf.low_latency_dispatch(out, topk, T, use_fp8=True)
    a = rows_value((q, sc)).view(T, -1, 128)
    b = rows_value((dq[0, 0], dsc[0, 0])).view(T, -1, 128)
    amax = b.abs().amax(-1, keepdim=True)
    # each is within half a code step of its own row, the rows within a bf16 half step
    step = torch.maximum(b.abs() * 2.0 ** -4, amax * 2.0 ** -10 / 448)
    close(a, b, 2.2 * step + b.abs() * BF * 1.1)


@pytest.mark.parametrize("dres", [False, True], ids=["plain", "dresidual"])
@pytest.mark.parametrize("T,H", [(1, 8), (7, 512), (600, 328), (33, 2048), (1030, 1280), (520, 7168), (3, 9000),
                                 (700, 20000)])
def test_rms_norm_backward(T, H, dres):
    g = gen(T + H)
    h, dout, w = normal(g, (T, H), 2.0), normal(g, (T, H)), normal(g, (H,))
    r = normal(g, (T, H)) if dres else None
    rstd = (1 / torch.sqrt((h.double() ** 2).mean(1) + 1e-6)).float()
    dx, dw = epm.rms_norm_backward(dout, h, w, rstd, dresidual=r)
    R, hd, a = rstd.double()[:, None], h.double(), dout.double() * w.double()
    inner = (a * hd).sum(1, keepdim=True)
    mag = (a * hd).abs().sum(1, keepdim=True)
    ref = R * a - R ** 3 * hd * inner / H + (r.double() if dres else 0)
    err = (H + 16) * U * R ** 3 * hd.abs() * mag / H + 8 * U * (R * a.abs() + R ** 3 * hd.abs() * inner.abs() / H)
    close(dx, ref, ref.abs() * (BF + U) + 2 * err + TINY, "dx")
    xh = hd * R
    close(dw, (dout.double() * xh).sum(0), (T + 8) * U * (dout.double() * xh).abs().sum(0) + TINY, "dweight")
    # against differences of the norm's own formula in 64 bits, along a direction
    if T <= 33:
        v = torch.randn((T, H), generator=g, device="cuda", dtype=torch.float64)

        def loss(z):
            return (z / torch.sqrt((z * z).mean(1, keepdim=True) + 1e-6) * w.double() * dout.double()).sum()
        num = (loss(hd + 1e-5 * v) - loss(hd - 1e-5 * v)) / 2e-5
        got = ((dx.double() - (r.double() if dres else 0)) * v).sum()
        # dx's own bound along v, and the differences' truncation and cancellation
        tol = ((ref.abs() * (BF + U) + 2 * err) * v.abs()).sum() + 1e-6 * (R * a * v).abs().sum()
        assert abs(float(num - got)) <= float(tol)


def test_rms_norm_backward_without_tokens():
    z = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    dx, dw = epm.rms_norm_backward(z, z, torch.ones(64, dtype=torch.bfloat16, device="cuda"),
                                   torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros(64, device="cuda"))


# ---------------------------------------------------------------- product

@pytest.mark.parametrize("M,N,K", [(1, 8, 128), (1, 4096, 1024), (15, 200, 384), (16, 128, 128), (17, 136, 256),
                                   (64, 520, 2176), (65, 264, 640), (200, 1000, 1152), (333, 328, 256),
                                   (1025, 512, 384)])
def test_fp8_product(M, N, K):
    g = gen(M + N + K)
    a, w = fp8_rows(g, (M, K)), fp8_weight(g, (N, K))
    av, wv = rows_value(a), weight_value(w)
    ref, mag = av @ wv.t(), av.abs() @ wv.abs().t()
    out = epm.fp8_product(a, w)
    assert out.dtype == torch.bfloat16 and out.shape == (M, N)
    close(out, ref, ref.abs() * BF * 1.01 + (sum_err(K) * mag + fp8_sum_err(av, wv)) * 1.01)


def test_fp8_product_alignment():
    """The alignment that fp8_sum_err allows for, and no more than it: beside 2^16 in
    the same eight a term of 2^3 arrives whole and one of 2^2 may not; in another
    eight every power of two arrives."""
    K, terms = 128, [(k, e) for k in (1, 7, 8, 9, 64, 127) for e in (9, 6, 3, 2)]
    a = torch.zeros((len(terms), K), device="cuda")
    w = torch.zeros((8, K), device="cuda")
    w[:, :] = 2.0
    w[:, 0] = 256.0
    a[:, 0] = 256.0
    for i, (k, e) in enumerate(terms):
        a[i, k] = 2.0 ** (e - 1)
    one = torch.ones((1, 1), device="cuda")
    # 2^16 is taken off again by a second block, so that bf16 shows the rest exactly
    a = torch.cat([a, torch.zeros_like(a)], 1)
    a[:, K] = -256.0
    w = torch.cat([w, w], 1)
    out = epm.fp8_product((a.to(torch.float8_e4m3fn), one.expand(len(terms), 2).contiguous()),
                          (w.to(torch.float8_e4m3fn), one.expand(1, 2).contiguous()))
    for i, (k, e) in enumerate(terms):
        if k >= 8 or e >= 3:
            assert (out[i] == 2.0 ** e).all(), (k, e, out[i])
        else:
            assert ((out[i] == 2.0 ** e) | (out[i] == 0)).all(), (k, e, out[i])


def test_fp8_product_scales_and_not_finite():
    M, N, K = 40, 136, 256
    g = gen(9)
    a, w = fp8_rows(g, (M, K)), fp8_weight(g, (N, K))
    a[1][3, 1] = float("inf")       # row 3: infinite, or NaN where the block's sum is zero
    a[0].view(torch.uint8)[5, 7] = 0x7F  # row 5: a NaN code
    w[0].view(torch.uint8)[9, 200] = 0xFF  # column 9: a NaN code
    out = epm.fp8_product(a, w)
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[3], want[5], want[:, 9] = True, True, True
    assert torch.equal(bad, want)
    assert epm.fp8_product((a[0][:0], a[1][:0]), w).shape == (0, N)


# --------------------------------------------------- experts' feed-forward

def ffn_ref(x, w13, w2, fp8=False):
    """fp64 g, u, sigmoid(g) and act of one expert, and the bounds of the kernel's g, u and act."""
    I = w2.shape[1]
    H = x.shape[1]
    g, u = x @ w13[:I].t(), x @ w13[I:].t()
    eg = sum_err(H) * (x.abs() @ w13[:I].abs().t())
    eu = sum_err(H) * (x.abs() @ w13[I:].abs().t())
    if fp8:
        eg, eu = eg + fp8_sum_err(x, w13[:I]), eu + fp8_sum_err(x, w13[I:])
    s = torch.sigmoid(g)
    act = g * s * u
    # |silu'| <= 1.1, and the function itself to a few units
    eact = 1.1 * eg * (u.abs() + eu) + (g * s).abs() * eu + 8 * U * act.abs()
    return g, u, s, act, eg, eu, eact


def routing(g, T, E, K, mask, dup=False):
    if dup:
        topk = torch.randint(0, E, (T, K), generator=g, device="cuda")
    else:
        topk = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :K].contiguous()
    drop = torch.rand((T, K), generator=g, device="cuda") < mask
    return torch.where(drop, -1, topk), torch.softmax(torch.randn((T, K), generator=g, device="cuda"), 1)


GROUP_SHAPES = [(1, 4, 2, 2, 0.0, False), (40, 16, 4, 4, 0.3, False), (300, 24, 24, 5, 0.1, True),
                (257, 8, 1, 3, 0.5, False), (600, 64, 16, 6, 0.1, False), (5, 6, 3, 2, 1.0, False)]


@pytest.mark.parametrize("T,E,R,K,mask,dup", GROUP_SHAPES)
def test_expert_rows(T, E, R, K, mask, dup):
    g = gen(T + E)
    topk, w = routing(g, T, E, K, mask, dup)
    buf = epm.Buffer(R, E)
    x = normal(g, (T, 8))
    recv, ids, _, counts, h, _ = buf.dispatch(x, topk, w)
    rows = buf.expert_rows(ids, h)
    N = recv.shape[0]
    prefix = h.layout().rank_prefix_matrix.tolist()
    want = [[] for _ in range(E)]
    per_row = [0] * N
    for r in range(R):
        for i in range(prefix[r - 1] if r else 0, prefix[r]):
            for k, v in enumerate(ids[i].tolist()):
                if v >= 0:
                    want[r * (E // R) + v].append((i, k))
                    per_row[i] += 1
    off = rows.expert_offsets.tolist()
    flat = [p for e in range(E) for p in want[e]]
    assert off == [sum(len(want[j]) for j in range(e)) for e in range(E + 1)]
    n = off[-1]
    pr, ps = rows.pair_row[:n].tolist(), rows.pair_slot[:n].tolist()
    assert [p & 0x7FFFFFFF for p in pr] == [i for i, _ in flat]
    assert ps == [i * K + k for i, k in flat]
    assert [p < 0 for p in pr] == [per_row[i] == 1 for i, _ in flat]
    back = torch.full((N, K), -1, dtype=torch.int32)
    for p, (i, k) in enumerate(flat):
        back[i, k] = p
    assert torch.equal(rows.row_pair.cpu(), back)
    # the same through the prefix, in buffers that hold rows past the last segment
    extra = torch.cat([ids, torch.zeros((9, K), dtype=torch.int64, device="cuda")])
    pad = buf.expert_rows(extra, h.layout().rank_prefix_matrix, num_tokens=T)
    assert torch.equal(pad.expert_offsets, rows.expert_offsets)
    assert torch.equal(pad.pair_slot[:n], rows.pair_slot[:n])
    assert torch.equal(pad.row_pair[:N], rows.row_pair) and (pad.row_pair[N:] == -1).all()
    h.free()


def dispatched(g, T, H, E, R, K, mask, dup, extra=0):
    """A dispatch, its rows in buffers with extra stale rows behind the last segment."""
    topk, w = routing(g, T, E, K, mask, dup)
    buf = epm.Buffer(R, E)
    recv, ids, tw, _, h, _ = buf.dispatch(normal(g, (T, H)), topk, w)
    prefix = h.layout().rank_prefix_matrix
    if extra:
        recv = torch.cat([recv, torch.full((extra, H), float("nan"), dtype=torch.bfloat16, device="cuda")])
        ids = torch.cat([ids, torch.zeros((extra, K), dtype=torch.int64, device="cuda")])
        tw = torch.cat([tw, torch.full((extra, K), float("nan"), device="cuda")])
    return buf, h, prefix, recv, ids, tw


def experts_ref(x, ids, tw, prefix, E, R, w13, w2, dy=None):
    """fp64 outputs and bounds over all rows, from the definition."""
    N, H = x.shape
    I = w2.shape[2]
    epr = E // R
    z = dict(device="cuda", dtype=torch.float64)
    y, ey, ymag = torch.zeros((N, H), **z), torch.zeros((N, H), **z), torch.zeros((N, H), **z)
    dx, edx, dxmag = torch.zeros_like(y), torch.zeros_like(y), torch.zeros_like(y)
    dw, edw = torch.zeros(ids.shape, **z), torch.zeros(ids.shape, **z)
    dw13, e13 = torch.zeros(w13.shape, **z), torch.zeros(w13.shape, **z)
    dw2, e2 = torch.zeros(w2.shape, **z), torch.zeros(w2.shape, **z)
    start = [0] + prefix.tolist()
    for e in range(E):
        a, b = start[e // epr], start[e // epr + 1]
        row, slot = (ids[a:b] == e % epr).nonzero(as_tuple=True)
        if not len(row):
            continue
        row = row + a
        xe, p = x[row].double(), tw[row, slot].double()[:, None]
        W13, W2 = w13[e].double(), w2[e].double()
        gg, u, s, act, eg, eu, eact = ffn_ref(xe, W13, W2)
        kact = eact + act.abs() * BF * 1.01  # the activation as bf16
        zz = act @ W2.t()
        ez = kact @ W2.abs().t() + sum_err(I) * (act.abs() @ W2.abs().t())
        y.index_add_(0, row, p * zz)
        ey.index_add_(0, row, p.abs() * (ez * 1.01 + 2 * U * zz.abs()))
        ymag.index_add_(0, row, (p * zz).abs())
        if dy is None:
            continue
        d0 = dy[row].double()
        d, dmag = d0 @ W2, d0.abs() @ W2.abs()
        ed = sum_err(H) * dmag
        dw[row, slot] = (act * d).sum(1)
        edw[row, slot] = (eact * d.abs() + act.abs() * ed).sum(1) * 1.01 + sum_err(I) * (act * d).abs().sum(1)
        silu, dsilu = gg * s, s * (1 + gg * (1 - s))
        du, dg = p * d * silu, p * d * u * dsilu
        # |silu'| <= 1.1, |silu''| <= 0.5
        edu = p.abs() * (ed * silu.abs() + d.abs() * 1.1 * eg) * 1.01 + du.abs() * (BF * 1.01 + 8 * U)
        edg = (p.abs() * (ed * (u * dsilu).abs() + d.abs() * 1.1 * eu + (d * u).abs() * 0.5 * eg) * 1.01
               + p.abs() * (d * u).abs() * 8 * U + dg.abs() * BF * 1.01)
        dgu, edgu = torch.cat((dg, du), 1), torch.cat((edg, edu), 1)
        t, tm = dgu @ W13, dgu.abs() @ W13.abs()
        dx.index_add_(0, row, t)
        dxmag.index_add_(0, row, t.abs())
        edx.index_add_(0, row, edgu @ W13.abs() + sum_err(2 * I) * tm)
        n = len(row)
        dw13[e] = dgu.t() @ xe
        e13[e] = edgu.t() @ xe.abs() + sum_err(n) * (dgu.abs().t() @ xe.abs())
        wa = p * act
        ewa = p.abs() * eact + wa.abs() * (BF * 1.01 + 4 * U)
        dw2[e] = d0.t() @ wa
        e2[e] = d0.abs().t() @ ewa + sum_err(n) * (d0.abs().t() @ wa.abs())
    K = ids.shape[1]
    ey = ey + y.abs() * BF * 1.01 + (K + 1) * U * ymag + TINY
    edx = edx * 1.01 + dx.abs() * BF * 1.01 + (K + 1) * U * dxmag + TINY
    e13 = e13 * 1.01 + dw13.abs() * BF * 1.01 + TINY
    e2 = e2 * 1.01 + dw2.abs() * BF * 1.01 + TINY
    return (y, ey), (dx, edx), (dw, edw + TINY), (dw13, e13), (dw2, e2)


FFN_SHAPES = [  # T, H, I, E, R, K, mask, dup
    (1, 8, 8, 4, 2, 2, 0.0, False),
    (3, 128, 64, 8, 8, 4, 0.0, False),
    (50, 72, 40, 6, 3, 3, 0.4, True),
    (200, 256, 352, 16, 4, 6, 0.1, False),
    (300, 200, 136, 2, 1, 2, 0.0, False),
    (700, 320, 264, 4, 2, 2, 0.0, False),
    (20, 64, 24, 96, 32, 2, 0.3, False),
    (6, 64, 64, 4, 2, 2, 1.0, False),
]


@pytest.mark.parametrize("T,H,I,E,R,K,mask,dup", FFN_SHAPES)
def test_expert_ffn_and_gradients(T, H, I, E, R, K, mask, dup):
    g = gen(T + H + I)
    buf, h, prefix, x, ids, tw = dispatched(g, T, H, E, R, K, mask, dup, extra=5)
    w13, w2 = normal(g, (E, 2 * I, H), H ** -0.5), normal(g, (E, H, I), I ** -0.5)
    rows = buf.expert_rows(ids, prefix, num_tokens=T)
    y, none = buf.expert_ffn(x, rows, tw, w13, w2)
    assert none is None
    dy = normal(g, x.shape)
    y2, saved = buf.expert_ffn(x, rows, tw, w13, w2, save=True)
    assert torch.equal(y, y2)
    dx, dw, dw13, dw2 = buf.expert_ffn_backward(dy, x, rows, tw, w13, w2, saved)
    refs = experts_ref(x, ids, tw, prefix, E, R, w13, w2, dy)
    for name, got, (ref, tol) in zip(("y", "dx", "dtopk_weights", "dw13", "dw2"), (y, dx, dw, dw13, dw2), refs):
        close(got, ref, tol, name)
    # a row or an expert without pairs is exactly zero, whatever stale values its row holds
    none = (rows.row_pair < 0).all(1)
    assert (y[none] == 0).all() and (dx[none] == 0).all()
    assert (dw[rows.row_pair < 0] == 0).all()
    empty = rows.expert_offsets.diff() == 0
    assert (dw13[empty] == 0).all() and (dw2[empty] == 0).all()
    # the same bits again
    again = buf.expert_ffn_backward(dy, x, rows, tw, w13, w2, saved)
    for a, b in zip((dx, dw, dw13, dw2), again):
        assert torch.equal(a, b)
    h.free()


@pytest.mark.parametrize("T,H,I,E,R,K,mask", [(1, 128, 64, 8, 4, 4, 0.0), (40, 200, 72, 6, 3, 3, 0.2),
                                              (64, 256, 136, 4, 4, 2, 0.0), (500, 136, 264, 3, 1, 2, 0.0),
                                              (9, 64, 32, 8, 2, 2, 1.0)])
def test_low_latency_expert_ffn(T, H, I, E, R, K, mask):
    g = gen(T + H)
    topk, _ = routing(g, T, E, K, mask)
    buf = epm.Buffer(R, E)
    S = T + 3
    packed, count, hdl, _, _ = buf.low_latency_dispatch(normal(g, (T, H)), topk, S)
    w13, w2 = normal(g, (E, 2 * I, H), H ** -0.5), normal(g, (E, H, I), I ** -0.5)
    out = torch.full(packed.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got = buf.low_latency_expert_ffn(packed, count, hdl, w13, w2, out=out)
    assert got is out
    epr = E // R
    for e in range(E):
        le, r = e % epr, e // epr
        n = int(count[le, r])
        assert (out[le, r, n:] == 7.0).all(), "unused cells are left alone"
        if n == 0:
            continue
        x, W2 = packed[le, r, :n].double(), w2[e].double()
        _, _, _, act, _, _, eact = ffn_ref(x, w13[e].double(), W2)
        ref = act @ W2.t()
        tol = ((eact + act.abs() * BF * 1.01) @ W2.abs().t() + sum_err(I) * (act.abs() @ W2.abs().t())) * 1.01
        close(out[le, r, :n], ref, tol + ref.abs() * BF * 1.01 + TINY, f"expert {e}")


@pytest.mark.parametrize("T,H,I,E,R,K,mask", [(1, 128, 128, 8, 4, 4, 0.0), (40, 256, 384, 6, 3, 3, 0.2),
                                              (100, 384, 128, 4, 2, 2, 0.0), (500, 256, 256, 3, 1, 2, 0.0),
                                              (90, 256, 256, 64, 8, 2, 0.0), (9, 128, 128, 8, 2, 2, 1.0)])
def test_low_latency_expert_ffn_fp8(T, H, I, E, R, K, mask):
    """Through the C ABI, whose workspaces show the quantised activation: its codes
    and scales against the formula, then the output against those very codes."""
    g = gen(T + I)
    topk, _ = routing(g, T, E, K, mask)
    if T == 90:
        topk[:, 0] = 5  # one expert holds every token, the others a few
    buf = epm.Buffer(R, E)
    S = T + 3
    (q, sc), count, hdl, _, _ = buf.low_latency_dispatch(normal(g, (T, H)), topk, S, use_fp8=True)
    w13, w2 = fp8_weight(g, (E, 2 * I, H)), fp8_weight(g, (E, H, I))
    epr = E // R
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    aq = torch.zeros((epr, R, S, I), dtype=torch.uint8, device="cuda")
    asc = torch.zeros((epr, R, S, I // 128), device="cuda")
    P = abi.ptr
    d = abi.dims(T, H, K, E, R)
    abi.check(abi.lib().ep_ll_expert_ffn_fp8(
        ctypes.byref(d), S, I, P(q), P(sc), P(count), P(w13[0]), P(w13[1]), P(w2[0]), P(w2[1]), P(aq), P(asc),
        P(out), abi.current_stream()), "ep_ll_expert_ffn_fp8")
    W13v, W2v = weight_value(w13), weight_value(w2)
    for e in range(E):
        le, r = e % epr, e // epr
        n = int(count[le, r])
        assert (out[le, r, n:] == 7.0).all(), "unused cells are left alone"
        if n == 0:
            continue
        x, W2 = rows_value((q[le, r, :n], sc[le, r, :n])), W2v[e]
        _, _, _, act, _, _, eact = ffn_ref(x, W13v[e], W2, fp8=True)
        b, eb = act.view(n, -1, 128), eact.view(n, -1, 128)
        amax, eamax = b.abs().amax(-1).clamp_min(1e-4), eb.amax(-1)
        s = asc[le, r, :n].double()
        close(s, amax / 448, eamax / 448 + amax / 448 * 4 * U, f"scales of expert {e}")
        codes = aq[le, r, :n].view(torch.float8_e4m3fn).double().view(b.shape)
        t = b / s[..., None]
        # half a step of the code, the kernel's own error in steps, and its two roundings
        et = eb / s[..., None] + 8 * U * t.abs()
        close(codes, t, (t.abs() + et).mul(2.0 ** -4).clamp_min(2.0 ** -10) + et, f"codes of expert {e}")
        a = (codes * s[..., None]).view(n, I)
        ref = a @ W2.t()
        err = sum_err(I) * (a.abs() @ W2.abs().t()) + fp8_sum_err(a, W2)
        close(out[le, r, :n], ref, ref.abs() * BF * 1.01 + err * 1.01 + TINY, f"expert {e}")
    # the binding gives the same bits
    hold = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(buf.low_latency_expert_ffn((q, sc), count, hdl, w13, w2, out=hold), out)
