"""Low-rank adapters and their gradients against the formulas in 64 bits.

Bounds, per element: fp32 sums of n terms 2 (n + 8) U of the summed magnitudes, half a bf16 step (2^-8) for
every result and its square for h and dh, which are sums of two bf16 values, and what an error of h or dh gives behind
its second product."""

from __future__ import annotations

import math
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

import combine_get_dispatch_05_amd as epm  # noqa: E402
from combine_get_dispatch_05_amd import abi  # noqa: E402

BF, U = 2.0 ** -8, 2.0 ** -24
TINY = 2.0 ** -100


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


def close(got, ref, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - tol
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: {int((over > 0).sum())} of {over.numel()} out, by up to {worst:.3g}"


def err(n):
    return 2 * (n + 8) * U


def made(T, K, N, r, L, seed=0):
    g = gen(seed)
    return (normal(g, (T, K)), normal(g, (L, r, K), 1 / math.sqrt(K)), normal(g, (L, N, r), 1 / math.sqrt(r)),
            0.5 + torch.rand(L, generator=g, device="cuda"), normal(g, (T, N)), normal(g, (T, N)), normal(g, (T, K)))


def check(ids, x, down, up, scales, base, dy, dx_base):
    T, K = x.shape
    L, r = down.shape[:2]
    N = up.shape[1]
    out, hidden = epm.adapter_product(x, ids, down, up, scales, base=base, save=True)
    same, none = epm.adapter_product(x, ids, down, up, scales, base=base)
    assert none is None and torch.equal(same, out)
    dx, ddown, dup = epm.adapter_product_backward(dy, x, ids, down, up, scales, hidden, dx_base=dx_base)
    f64 = dict(dtype=torch.float64, device="cuda")
    ro = base.double().clone() if base is not None else torch.zeros((T, N), **f64)
    rx = dx_base.double().clone() if dx_base is not None else torch.zeros((T, K), **f64)
    eo, ex = ro.abs() * U, rx.abs() * U
    rh, eh, es = (torch.zeros((T, r), **f64) for _ in range(3))
    for a in range(L):
        t = (ids == a).nonzero()[:, 0]
        c, A, B = scales[a].double(), down[a].double(), up[a].double()
        xa, ya = x[t].double(), dy[t].double()
        h, eh_ = c * (xa @ A.t()), c * (xa.abs() @ A.abs().t()) * (err(K) + 2 * U)
        es[t] = eh_ * (1 + BF)
        eh_ = eh_ + BF * (h.abs() + eh_)
        rh[t], eh[t] = h, eh_
        ro[t] += h @ B.t()
        e2 = es[t] + BF * BF * h.abs()  # (as the sum of two values; 2 r products)
        eo[t] += (e2 + err(2 * r) * (h.abs() + e2) * (1 + BF)) @ B.abs().t()
        dh, ed = c * (ya @ B), c * (ya.abs() @ B.abs()) * (err(N) + 2 * U)
        ed = ed * (1 + BF) + BF * BF * dh.abs()
        rx[t] += dh @ A
        ex[t] += (ed + err(2 * r) * (dh.abs() + ed) * (1 + BF)) @ A.abs()
        kept = hidden[0, t].double() + hidden[1, t].double()
        rd, ref = dh.t() @ xa, ya.t() @ kept
        close(ddown[a], rd, rd.abs() * BF + (ed + err(len(t)) * (dh.abs() + ed)).t() @ xa.abs() * (1 + BF) + TINY, f"ddown {a}")
        close(dup[a], ref, ref.abs() * BF + err(len(t)) * (ya.abs().t() @ hidden[:, t].double().abs().sum(0)) + TINY, f"dup {a}")
    close(hidden[0], rh, eh + TINY, "hidden")
    # the two together are h to 2^-16 of it, besides its sums
    close(hidden[0].double() + hidden[1].double(), rh, es + BF * BF * rh.abs() + TINY, "hidden as a sum")
    close(out, ro, ro.abs() * BF + eo * (1 + BF) + TINY, "out")
    close(dx, rx, rx.abs() * BF + ex * (1 + BF) + TINY, "dx")
    return out, hidden, dx, ddown, dup


SHAPES = [  # T, K, N, r, L, share without an adapter
    (1, 8, 8, 8, 1, 0.0), (1, 7168, 2048, 16, 8, 0.0), (2, 64, 72, 24, 3, 0.5), (15, 200, 136, 16, 2, 0.1),
    (16, 128, 64, 32, 1, 0.0), (17, 136, 320, 32, 1, 0.0), (63, 72, 1000, 64, 4, 0.2), (64, 512, 256, 64, 1, 0.0),
    (65, 1024, 264, 40, 1, 0.0), (128, 2048, 512, 16, 64, 0.1), (130, 264, 520, 128, 5, 0.1), (33, 64, 64, 104, 1, 0.0),
    (600, 640, 1032, 8, 70, 0.1), (700, 520, 328, 72, 2, 0.6), (1500, 256, 512, 64, 7, 0.0), (2100, 128, 136, 16, 200, 0.3),
    (5000, 64, 64, 32, 3, 0.05), (300, 4096, 64, 128, 2, 0.0), (40, 8, 2048, 8, 4, 0.2),
    (256, 264, 200, 128, 1, 0.0), (256, 64, 128, 32, 127, 0.3), (257, 64, 128, 16, 2, 0.0), (200, 64, 136, 24, 128, 0.3),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_adapter(case):
    T, K, N, r, L, none = SHAPES[case]
    g = gen(50 + case)
    ids = torch.randint(0, L, (T,), generator=g, device="cuda")
    ids[torch.rand(T, generator=g, device="cuda") < none] = -1
    x, down, up, scales, base, dy, dxb = made(T, K, N, r, L, case)
    check(ids, x, down, up, scales, base if case % 3 else None, dy, dxb if case % 4 else None)


def test_runs_one_adapter_and_none():
    x, down, up, scales, base, dy, dxb = made(1000, 192, 200, 16, 6)
    runs = torch.arange(1000, device="cuda") * 6 // 1000
    check(runs, x, down, up, scales, base, dy, dxb)
    check(torch.full((1000,), 4, device="cuda"), x, down, up, scales, base, dy, dxb)
    # ids that name no adapter, of every kind: the base alone, and no gradients
    odd = torch.tensor([-1, 6, 1 << 40, -(1 << 50)], device="cuda").repeat(250)
    out, hidden, dx, ddown, dup = check(odd, x, down, up, scales, base, dy, dxb)
    assert torch.equal(out, base) and torch.equal(dx, dxb)
    assert (hidden == 0).all() and (ddown == 0).all() and (dup == 0).all()
    out, _ = epm.adapter_product(x, odd, down, up, scales)
    assert (out == 0).all()


@pytest.mark.parametrize("T", [12, 200])
def test_ids_that_name_no_adapter_among_few_tokens(T):
    x, down, up, scales, base, dy, dxb = made(T, 192, 200, 16, 6)
    odd = torch.tensor([-1, 6, 1 << 40, -(1 << 50)], device="cuda").repeat(T // 4)
    out, hidden, dx, ddown, dup = check(odd, x, down, up, scales, base, dy, dxb)
    assert torch.equal(out, base) and torch.equal(dx, dxb)
    assert (hidden == 0).all() and (ddown == 0).all() and (dup == 0).all()
    odd[::3] = 5
    check(odd, x, down, up, scales, base, dy, dxb)


def test_rows_and_adapters_that_are_not_finite_stay_alone():
    T, K, N, r, L = 200, 136, 264, 24, 5
    g = gen(8)
    x, down, up, scales, base, dy, dxb = made(T, K, N, r, L)
    ids = torch.randint(0, L - 1, (T,), generator=g, device="cuda")
    args = (ids, x, down, up, scales)
    good, hid = epm.adapter_product(x, ids, down, up, scales, base=base, save=True)
    back = epm.adapter_product_backward(dy, x, ids, down, up, scales, hid, dx_base=dxb)
    bad_down, bad_up, bad_scales = down.clone(), up.clone(), scales.clone()
    bad_down[L - 1], bad_up[L - 1], bad_scales[L - 1] = math.nan, math.inf, math.nan  # nobody's
    out, hid2 = epm.adapter_product(x, ids, bad_down, bad_up, bad_scales, base=base, save=True)
    assert torch.equal(out, good) and torch.equal(hid, hid2)
    again = epm.adapter_product_backward(dy, x, ids, bad_down, bad_up, bad_scales, hid, dx_base=dxb)
    assert all(torch.equal(a, b) for a, b in zip(back, again))
    t = int((ids == 2).nonzero()[0])
    bad = x.clone()
    bad[t, 5] = math.nan
    out, _ = epm.adapter_product(bad, ids, down, up, scales, base=base)
    rest = [i for i in range(T) if i != t]
    assert out[t].isnan().all() and torch.equal(out[rest], good[rest])
    ids2 = ids.clone()
    ids2[t] = -1  # without an adapter its row is not looked at
    bad_dy = dy.clone()
    bad_dy[t] = math.nan
    out, hid2 = epm.adapter_product(bad, ids2, down, up, scales, base=base, save=True)
    assert torch.equal(out[t], base[t])
    dx, ddown, dup = epm.adapter_product_backward(bad_dy, bad, ids2, down, up, scales, hid2, dx_base=dxb)
    assert torch.isfinite(ddown).all() and torch.isfinite(dup).all() and torch.equal(dx[t], dxb[t])


def test_no_tokens_and_refusals():
    x, down, up, scales, base, dy, dxb = made(6, 64, 72, 16, 3)
    ids = torch.zeros(6, dtype=torch.int64, device="cuda")
    out, hidden = epm.adapter_product(x[:0], ids[:0], down, up, scales, base=base[:0], save=True)
    assert out.shape == (0, 72) and hidden.shape == (2, 0, 16)
    dx, ddown, dup = epm.adapter_product_backward(dy[:0], x[:0], ids[:0], down, up, scales, hidden)
    assert dx.shape == (0, 64) and (ddown == 0).all() and (dup == 0).all()
    out, hidden = epm.adapter_product(x, ids, down, up, scales, save=True)
    back = epm.adapter_product_backward
    for bad in (lambda: epm.adapter_product(x, ids[:5], down, up, scales),
                lambda: epm.adapter_product(x, ids, down[:, :, :32], up, scales),
                lambda: epm.adapter_product(x, ids, down, up[:2], scales),
                lambda: epm.adapter_product(x, ids, down, up[:, :, :8], scales),
                lambda: epm.adapter_product(x, ids, down, up, scales[:2]),
                lambda: epm.adapter_product(x, ids, down, up, scales, base=x),
                lambda: epm.adapter_product(x.t(), ids, down, up, scales),
                lambda: back(x, x, ids, down, up, scales, hidden), lambda: back(dy, x, ids, down, up, scales, hidden[0]),
                lambda: back(dy, x, ids, down, up, scales, hidden, dx_base=dy)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        epm.adapter_product(x, ids.int(), down, up, scales)
    with pytest.raises(abi.EpError):  # a rank past 128
        epm.adapter_product(x, ids, torch.zeros((3, 136, 64), dtype=torch.bfloat16, device="cuda"),
                            torch.zeros((3, 72, 136), dtype=torch.bfloat16, device="cuda"), scales)


def test_in_place_through_the_library():
    """out over base and dx over dx_base, which the ABI allows."""
    import ctypes
    T, K, N, r, L = 90, 128, 136, 16, 3
    x, down, up, scales, base, dy, dxb = made(T, K, N, r, L)
    ids = torch.randint(-1, L, (T,), generator=gen(2), device="cuda")
    out, hidden = epm.adapter_product(x, ids, down, up, scales, base=base, save=True)
    dx, ddown, dup = epm.adapter_product_backward(dy, x, ids, down, up, scales, hidden, dx_base=dxb)
    d = abi.AdapterDims(T, K, N, r, L)
    p = abi.address
    for back in (0, 1):
        n = abi.lib().ep_adapter_workspace(ctypes.byref(d), back)
        work = torch.empty(n, dtype=torch.uint8, device="cuda")
        s = abi.current_stream()
        if back:
            abi.check(abi.lib().ep_adapter_product_backward(
                ctypes.byref(d), p(dy), p(x), p(ids), p(down), p(up), p(scales), p(hidden), p(dxb), p(dxb), p(ddown), p(dup),
                p(work), n, s), "backward")
        else:
            abi.check(abi.lib().ep_adapter_product(ctypes.byref(d), p(x), p(ids), p(down), p(up), p(scales), p(base),
                                                   p(base), None, p(work), n, s), "forward")
    assert torch.equal(base, out) and torch.equal(dxb, dx)


def test_gradient_against_differences():
    """The loss sum(out * dy) in 64 bits, moved along a direction of x, down and up."""
    T, K, N, r, L = 24, 64, 48, 8, 3
    x, down, up, scales, base, dy, _ = made(T, K, N, r, L)
    ids = torch.randint(0, L, (T,), generator=gen(4), device="cuda")
    _, hidden = epm.adapter_product(x, ids, down, up, scales, save=True)
    grads = epm.adapter_product_backward(dy, x, ids, down, up, scales, hidden)

    def loss(v):
        xx, dd, uu = v
        h = torch.bmm(dd[ids], xx[:, :, None])[:, :, 0] * scales.double()[ids][:, None]
        return (torch.bmm(uu[ids], h[:, :, None])[:, :, 0] * dy.double()).sum()

    at = [v.double() for v in (x, down, up)]
    # an element is off by half a step of its own and of each dh (or h) that it sums
    mine = torch.nn.functional.one_hot(ids, L).double()
    dh = torch.bmm(up.double()[ids].transpose(1, 2).contiguous(), dy.double()[:, :, None])[:, :, 0].abs()
    dh = dh * scales.double()[ids][:, None]
    mags = [torch.bmm(dh[:, None, :], down.double()[ids].abs())[:, 0],
            torch.stack([(dh * m[:, None]).t() @ x.double().abs() for m in mine.t()]),
            torch.stack([(dy.double().abs() * m[:, None]).t() @ hidden[0].double().abs() for m in mine.t()])]
    for i, g in enumerate(grads):
        d = torch.randn(g.shape, generator=gen(30 + i), device="cuda", dtype=torch.float64)
        step = 1e-4

        def moved(h):
            return loss([v + h * d if j == i else v for j, v in enumerate(at)])
        slope = (moved(step) - moved(-step)) / (2 * step)
        assert abs(float((g.double() * d).sum() - slope)) <= BF * float(((g.double().abs() + mags[i]) * d.abs()).sum())
