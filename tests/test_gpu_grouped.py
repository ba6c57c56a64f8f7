"""The products grouped by expert and their gradients on the GPU against their 64-bit definitions.

Operands are exact and so is every product of two of them in fp32 (16 or 22 bits).  A sum of n terms is off by at most one
unit in the last place, 2^-23, of the sum of the absolute products per addition, whichever way the matrix units round:
2^-23 (n + 2) of it bounds the whole.  The result adds its own rounding.  8-bit sums are exact; turning one to fp32 and
the two scales round three times, 2^-24 each (and 1 + 2^-20 for the products of these).
"""
import numpy as np
import pytest
import torch

import grouped_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0**-23


def _q():
    import quantized_routed_moe_router_amd as q
    return q


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def half(a, kind):
    """A tensor of that type on the GPU, and its values."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DT[kind])
    return t.cuda(), t.double().numpy()


def host(t):
    return t.double().cpu().numpy()


def check(got, want, mag, terms, kind):
    err = np.abs(host(got) - want)
    bound = U * (terms + 2) * mag + R.HALF_STEP[kind] * np.abs(want) * (1 + 2.0**-7) + R.TINY[kind]
    assert got.shape == want.shape and (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())


#       T, E, k, N, K
SIZES = [(1, 1, 1, 1, 8), (1, 8, 2, 16, 16), (3, 4, 2, 17, 24), (1, 256, 8, 64, 512), (16, 300, 4, 40, 64), (37, 5, 3, 100, 72),
         (64, 512, 4, 33, 128), (130, 4, 1, 129, 136), (300, 3, 2, 260, 320), (700, 7, 3, 131, 1000), (2000, 2, 2, 384, 200),
         (1000, 2, 1, 700, 96), (513, 1, 1, 513, 2056), (90, 2, 2, 64, 4096), (1500, 40, 4, 72, 192)]


def case(T, E, k, N, K, kind, seed=0, pad=0, skew=0.5):
    rng = np.random.default_rng(T * 7 + E + seed)
    x, xv = half(rng.standard_normal((T, K + pad)), kind)
    w, wv = half(0.1 * rng.standard_normal((E, N, K)), kind)
    offsets, perm = R.routing(T, E, k, rng, skew)
    return x[:, :K], xv[:, :K], w, wv, offsets, perm


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("T,E,k,N,K", SIZES)
def test_product(kind, T, E, k, N, K):
    q = _q()
    x, xv, w, wv, offsets, perm = case(T, E, k, N, K, kind, pad=8 if T % 2 else 0)
    want, mag = R.matmul(xv, wv, offsets, R.rows_of(perm, k, T, T * k))
    for out in ("f32", kind):
        y = q.grouped_matmul(x, w, dev(offsets), dev(perm), k, y_dtype=DT[out])
        assert y.dtype == DT[out]
        check(y, want, mag, K, out)
        assert torch.equal(y, q.grouped_matmul(x, w, dev(offsets), dev(perm), k, y_dtype=DT[out]))
    # rows in order already
    rows = R.rows_of(perm, k, T, T * k)
    y2 = q.grouped_matmul(x[torch.from_numpy(rows).cuda()].contiguous(), w, dev(offsets))
    assert torch.equal(y2, q.grouped_matmul(x, w, dev(offsets), dev(perm), k))


@pytest.mark.parametrize("T,E,k,N,K", [s for s in SIZES if s[4] % 16 == 0])
def test_int8_product(T, E, k, N, K):
    q = _q()
    rng = np.random.default_rng(T + E)
    offsets, perm = R.routing(T, E, k, rng, 0.5)
    xc, wc = rng.integers(-127, 128, (T, K)).astype(np.int8), rng.integers(-128, 128, (E, N, K)).astype(np.int8)
    xs, ws = (rng.random(T) + 0.1).astype(np.float32), (rng.random((E, N)) + 0.1).astype(np.float32)
    rows = R.rows_of(perm, k, T, T * k)
    sums, _ = R.matmul(xc.astype(np.float64), wc.astype(np.float64), offsets, rows)
    per = np.concatenate([np.repeat(ws[e][None], offsets[e + 1] - offsets[e], 0) for e in range(E)]).astype(np.float64)
    want = sums * xs.astype(np.float64)[rows][:, None] * per
    for out in DT:
        y = q.grouped_matmul(dev(xc), dev(wc), dev(offsets), dev(perm), k, x_scales=dev(xs), w_scales=dev(ws), y_dtype=DT[out])
        err = np.abs(host(y) - want)
        big = np.abs(want) > 65504 if out == "f16" else np.zeros_like(want, dtype=bool)
        assert (err[~big] <= (3 * 2.0**-24 * (1 + 2.0**-20) + (R.HALF_STEP[out] * (1 + 2.0**-7) if out != "f32" else 0)) * np.abs(want[~big])
                + R.TINY[out]).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("T,E,k,N,K", [(T, E, k, (N + 7) // 8 * 8, K) for T, E, k, N, K in SIZES])
def test_gradients(kind, T, E, k, N, K):
    q = _q()
    x, xv, w, wv, offsets, perm = case(T, E, k, N, K, kind, pad=8 if T % 2 else 0)
    dy, dyv = half(np.random.default_rng(5).standard_normal((T * k, N + 8)), kind)
    dy, dyv = dy[:, :N], dyv[:, :N]
    rows = R.rows_of(perm, k, T, T * k)
    wx, ww, mx, mw = R.backward(dyv, xv, wv, offsets, rows)
    dx, dw = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), k)
    assert dx.dtype == dw.dtype == DT[kind]
    check(dx, wx, mx, N + k, kind)
    check(dw, ww, mw, T, kind)
    none, dw32 = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), k, need_dx=False, dw_dtype=torch.float32)
    assert none is None
    check(dw32, ww, mw, T, "f32")
    again, none = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), k, need_dw=False)
    assert none is None and torch.equal(again, dx)
    # rows in order already: a gradient of its own for every position
    xs, xsv = x[torch.from_numpy(rows).cuda()].contiguous(), xv[rows]
    wx, ww, mx, mw = R.backward(dyv, xsv, wv, offsets, np.arange(T * k))
    dx, dw2 = q.grouped_matmul_backward(dy, xs, w, dev(offsets))
    check(dx, wx, mx, N, kind)
    assert torch.equal(dw, dw2)


def test_gradients_are_the_differences():
    """Central differences of sum(dy * y) in 64 bits along random directions of x and w."""
    q = _q()
    T, E, k, N, K = 40, 4, 2, 24, 32
    x, xv, w, wv, offsets, perm = case(T, E, k, N, K, "f16")
    dy, dyv = half(np.random.default_rng(1).standard_normal((T * k, N)), "f16")
    dx, dw = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), k, dw_dtype=torch.float32)
    rng, rows, h = np.random.default_rng(2), R.rows_of(perm, k, T, T * k), 2.0**-10
    for _ in range(4):
        ux, uw = rng.standard_normal(xv.shape), rng.standard_normal(wv.shape)
        up, down = (R.matmul(xv + s * h * ux, wv, offsets, rows)[0] for s in (1, -1))
        want = ((up - down) * dyv).sum() / (2 * h)  # linear in x: exact but for 64-bit roundings
        _, _, mx, mw = R.backward(dyv, xv, wv, offsets, rows)
        bound = (np.abs(ux) * (mx * (U * (N + k + 2) + 2.0**-11) + R.TINY["f16"])).sum()
        assert abs((host(dx) * ux).sum() - want) <= bound
        up, down = (R.matmul(xv, wv + s * h * uw, offsets, rows)[0] for s in (1, -1))
        want = ((up - down) * dyv).sum() / (2 * h)
        assert abs((host(dw) * uw).sum() - want) <= (np.abs(uw) * mw).sum() * U * (T + 2)


@pytest.mark.parametrize("T", [9, 700])
def test_positions_of_no_expert_and_unnamed_rows(T):
    """Offsets that begin behind the first position and end before the last, experts without rows, entries of the
    permutation that name no row: zeros come out and no gradient goes in; absent assignments add nothing."""
    q = _q()
    E, k, N, K = 6, 2, 136, 72
    x, xv, w, wv, _, _ = case(T, E, k, N, K, "bf16")
    rng = np.random.default_rng(3)
    perm = rng.permutation(T * k).astype(np.int32)[:T * k - 3]
    P = perm.size
    perm[[2, P // 2]] = [-1, T * k]
    perm[1] = 2**31 - 1
    a, b = 4, P - 3
    offsets = np.array([a, a, a + (b - a) // 2, a + (b - a) // 2, b - 1, b - 1, b], dtype=np.int32)
    rows = R.rows_of(perm, k, T, P)
    want, mag = R.matmul(xv, wv, offsets, rows)
    y = q.grouped_matmul(x, w, dev(offsets), dev(perm), k)
    check(y, want, mag, K, "bf16")
    assert not host(y)[:a].any() and not host(y)[b:].any()
    dy, dyv = half(rng.standard_normal((P, N)), "bf16")
    wx, ww, mx, mw = R.backward(dyv, xv, wv, offsets, rows)
    dx, dw = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), k)
    check(dx, wx, mx, N + k, "bf16")
    check(dw, ww, mw, P, "bf16")
    assert not host(dw)[[0, 2, 4]].any()
    # all positions of no expert
    none = np.zeros(E + 1, dtype=np.int32)
    assert not host(q.grouped_matmul(x, w, dev(none), dev(perm), k)).any()
    dx, dw = q.grouped_matmul_backward(dy, x, w, dev(none), dev(perm), k)
    assert not host(dx).any() and not host(dw).any()


def test_offsets_are_held_to_the_arrays():
    """Offsets outside 0..P touch nothing outside the arrays: what they say within them is done."""
    q = _q()
    T, E, N, K = 300, 3, 72, 64
    x, xv, w, wv, _, _ = case(T, E, 1, N, K, "bf16")
    held = np.array([0, 100, 300, 300], dtype=np.int32)
    wild = np.array([-7, 100, 2**31 - 1, 2**31 - 1], dtype=np.int32)
    dy = half(np.random.default_rng(1).standard_normal((T, N)), "bf16")[0]
    assert torch.equal(q.grouped_matmul(x, w, dev(wild)), q.grouped_matmul(x, w, dev(held)))
    for a, b in zip(q.grouped_matmul_backward(dy, x, w, dev(wild)), q.grouped_matmul_backward(dy, x, w, dev(held))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,N,K", [(5, 40, 72), (300, 136, 200)])
def test_bad_values_stay_in_their_rows(T, N, K):
    """NaN and infinities of one token, of another expert and behind the rows' and the matrices' ends reach only what they
    belong to."""
    q = _q()
    E, k = 4, 1
    x, xv, w, wv, offsets, perm = case(T, E, k, N, K, "bf16", pad=8, skew=0.0)
    bad = int(perm[0]) // k
    store = x._base if x._base is not None else x
    store[:, K:] = float("nan")
    rows = R.rows_of(perm, k, T, T * k)
    clean = q.grouped_matmul(x, w, dev(offsets), dev(perm), k)
    x2 = store.clone()[:, :K]
    x2[bad] = float("inf")
    y = q.grouped_matmul(x2, w, dev(offsets), dev(perm), k)
    of = rows == bad
    assert not np.isfinite(host(y)[of]).any() and torch.equal(y[torch.from_numpy(~of).cuda()], clean[torch.from_numpy(~of).cuda()])
    big = half(np.random.default_rng(1).standard_normal((T * k, N + 8)), "bf16")[0]
    big[:, N:] = float("nan")
    dy = big[:, :N]
    dx0, dw0 = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), k)
    assert torch.isfinite(dx0).all() and torch.isfinite(dw0).all()
    p = int(offsets[1])  # the first position of expert 1
    big[p, 3] = float("nan")
    dx, dw = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), k)
    e = int(np.searchsorted(offsets, p, side="right") - 1)
    t = int(perm[p]) // k
    assert torch.isnan(dx[t]).all() and torch.isnan(dw[e, 3]).all()
    dx[t], dw[e, 3] = dx0[t], dw0[e, 3]
    assert torch.equal(dx, dx0) and torch.equal(dw, dw0)


def test_no_positions_and_no_tokens():
    q = _q()
    w = torch.ones(3, 16, 32, dtype=torch.bfloat16, device="cuda")
    offsets, perm = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    for T in (0, 5):
        x = torch.ones(T, 32, dtype=torch.bfloat16, device="cuda")
        y = q.grouped_matmul(x, w, offsets, perm, 2)
        assert y.shape == (0, 16)
        dx, dw = q.grouped_matmul_backward(y, x, w, offsets, perm, 2)
        assert dx.shape == (T, 32) and dw.shape == w.shape and not dx.any() and not dw.any()


def test_an_assignment_that_stands_twice():
    """The product takes it twice; dx counts its last position, dw both."""
    q = _q()
    x, xv, w, wv, _, _ = case(4, 2, 1, 16, 32, "bf16")
    perm, offsets = np.array([1, 1, 3, 1], dtype=np.int32), np.array([0, 2, 4], dtype=np.int32)
    rows = R.rows_of(perm, 1, 4, 4)
    want, mag = R.matmul(xv, wv, offsets, rows)
    check(q.grouped_matmul(x, w, dev(offsets), dev(perm)), want, mag, 32, "bf16")
    dy, dyv = half(np.random.default_rng(1).standard_normal((4, 16)), "bf16")
    dx, dw = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm))
    _, ww, _, mw = R.backward(dyv, xv, wv, offsets, rows)
    check(dw, ww, mw, 4, "bf16")
    once = np.zeros_like(xv)
    once[3], once[1] = dyv[2] @ wv[1], dyv[3] @ wv[1]
    check(dx, once, np.abs(once) + 1, 16 * 16, "bf16")


def test_streams_graphs_and_two_calls_at_once():
    """On a side stream, two calls side by side, and captured with both gradients: replays on new inputs give the eager
    results, with eager work between them."""
    q = _q()
    T, E, k, N, K = 200, 6, 2, 136, 128
    x, _, w, _, offsets, perm = case(T, E, k, N, K, "bf16")
    dy = half(np.random.default_rng(1).standard_normal((T * k, N)), "bf16")[0]
    o, p = dev(offsets), dev(perm)
    want = q.grouped_matmul(x, w, o, p, k)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(5):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                outs.append((q.grouped_matmul(x, w, o, p, k), *q.grouped_matmul_backward(dy, x, w, o, p, k)))
    torch.cuda.synchronize()
    eager = q.grouped_matmul_backward(dy, x, w, o, p, k)
    assert all(torch.equal(y, want) and torch.equal(a, eager[0]) and torch.equal(b, eager[1]) for y, a, b in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = q.grouped_matmul(x, w, o, p, k)
        dx, dw = q.grouped_matmul_backward(dy, x, w, o, p, k)
    for i in range(4):
        x.copy_(half(np.random.default_rng(i).standard_normal((T, K)), "bf16")[0])
        off, per = R.routing(T, E, k, np.random.default_rng(i), 0.5, unused=(i,))
        o.copy_(dev(off))
        p.copy_(dev(per))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw)]
        fresh = (q.grouped_matmul(x, w, o, p, k), *q.grouped_matmul_backward(dy, x, w, o, p, k))
        assert all(torch.equal(a, b) for a, b in zip(got, fresh))
