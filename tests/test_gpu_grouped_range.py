"""The products grouped by expert over the rest of their range: rows, weights and results beyond 32-bit offsets, every
height of a tile and every number of its rows, many experts with few rows and few with many, unnamed rows in long sums,
subnormal operands, types of the results; training steps and 8-bit calls on the C ABI.  Bounds as in test_gpu_grouped.
"""
import ctypes

import numpy as np
import pytest
import torch

import grouped_ref as R
from test_gpu_grouped import DT, _q, case, check, dev, half, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "int8"])
@pytest.mark.parametrize("P", [6, 700])
def test_gathered_rows_beyond_32_bit_offsets(dtype, P):
    """5.2 GB of rows of a wider buffer, of which the permutation names the first, the last and some between."""
    q = _q()
    T, step, N, K, E, k = (40000, 65536, 72, 192, 3, 1) if dtype == "bf16" else (40000, 131072, 72, 192, 3, 1)
    store = torch.zeros(T, step, dtype=DT.get(dtype, torch.int8), device="cuda")
    rng = np.random.default_rng(P)
    rows = np.sort(rng.choice(T, P - 2, replace=False))
    rows = rng.permutation(np.concatenate([[0], rows, [T - 1]])).astype(np.int32)
    offsets = np.array([0, P // 3, P // 3, P], dtype=np.int32)
    vals = rng.integers(-20, 21, (P, K)) / 4.0
    at = torch.from_numpy(rows.astype(np.int64)).cuda()
    w = rng.integers(-20, 21, (E, N, K)) / (4.0 if dtype == "bf16" else 1.0)
    if dtype == "int8":
        vals *= 4
        store[at, :K] = torch.from_numpy(vals).to(torch.int8).cuda()
        last = {int(r): i for i, r in enumerate(rows)}
        vals = np.stack([vals[last[int(r)]] for r in rows])
        y = q.grouped_matmul(store[:, :K], torch.from_numpy(w).to(torch.int8).cuda(), dev(offsets), dev(rows), k,
                             x_scales=torch.ones(T, device="cuda"), w_scales=torch.ones(E, N, device="cuda"), y_dtype=torch.float32)
        want, _ = R.matmul(vals, w, offsets, np.arange(P))
        assert np.array_equal(host(y), want)  # integers below 2^24
        return
    store[at, :K] = torch.from_numpy(vals).to(torch.bfloat16).cuda()
    last = {int(r): i for i, r in enumerate(rows)}
    vals = np.stack([vals[last[int(r)]] for r in rows])
    wt = torch.from_numpy(w).to(torch.bfloat16).cuda()
    want, _ = R.matmul(vals, w, offsets, np.arange(P))
    y = q.grouped_matmul(store[:, :K], wt, dev(offsets), dev(rows), k, y_dtype=torch.float32)
    assert np.array_equal(host(y), want)  # sixteenths below 2^24 of them
    dy = rng.integers(-20, 21, (P, N)) / 4.0
    _, dw = q.grouped_matmul_backward(torch.from_numpy(dy).to(torch.bfloat16).cuda(), store[:, :K], wt, dev(offsets), dev(rows), k,
                                      need_dx=False, dw_dtype=torch.float32)
    _, ww, _, _ = R.backward(dy, vals, w, offsets, np.arange(P))
    assert np.array_equal(host(dw), ww)


def test_rows_in_order_and_their_gradients_beyond_32_bit_offsets():
    """Rows of x, dy and results 4.6 GB long, one expert over nearly all of them: rows at both ends are not zero."""
    q = _q()
    P, N, K = 150000, 72, 64
    xs = torch.zeros(P, 16384, dtype=torch.bfloat16, device="cuda")
    ds = torch.zeros(P, 16384, dtype=torch.bfloat16, device="cuda")
    x, dy = xs[:, :K], ds[:, :N]
    rng = np.random.default_rng(0)
    live = np.array([0, 1, 3, 70000, 131071, 131072, 140000, P - 2, P - 1])
    xv, dv = rng.integers(-8, 9, (live.size, K)) / 4.0, rng.integers(-8, 9, (live.size, N)) / 4.0
    at = torch.from_numpy(live).cuda()
    xs[at, :K] = torch.from_numpy(xv).to(torch.bfloat16).cuda()
    ds[at, :N] = torch.from_numpy(dv).to(torch.bfloat16).cuda()
    w = rng.integers(-8, 9, (2, N, K)) / 4.0
    wt = torch.from_numpy(w).to(torch.bfloat16).cuda()
    offsets = torch.tensor([0, 2, P], dtype=torch.int32, device="cuda")
    e = (live >= 2).astype(int)
    y = q.grouped_matmul(x, wt, offsets, y_dtype=torch.float32)
    assert np.array_equal(host(y[at]), np.stack([w[e[i]] @ xv[i] for i in range(live.size)]))
    assert int((y != 0).any(1).sum()) <= live.size
    dx, dw = q.grouped_matmul_backward(dy, x, wt, offsets, dw_dtype=torch.float32)
    want = torch.from_numpy(np.stack([dv[i] @ w[e[i]] for i in range(live.size)])).to(torch.bfloat16)
    assert torch.equal(dx[at].cpu(), want) and int((dx != 0).any(1).sum()) <= live.size
    assert np.array_equal(host(dw), np.stack([sum(np.outer(dv[i], xv[i]) for i in range(live.size) if e[i] == j) for j in range(2)]))


def test_weights_and_results_beyond_32_bit_offsets():
    q = _q()
    E, N, K = 34, 65536, 1024  # 4.6 GB of weights
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(0)
    wl = rng.integers(-8, 9, (2, K)) / 4.0
    w[E - 1, 0], w[E - 1, N - 1] = (torch.from_numpy(v).to(torch.bfloat16).cuda() for v in wl)
    for T in (20, 300):
        xv = rng.integers(-8, 9, (T, K)) / 4.0
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[E] = T
        y = q.grouped_matmul(torch.from_numpy(xv).to(torch.bfloat16).cuda(), w, offsets, y_dtype=torch.float32)
        assert np.array_equal(host(y[:, [0, N - 1]]), xv @ wl.T) and not y[:, 1:N - 1].any()
        dv = rng.integers(-8, 9, (T, 2)) / 4.0
        dy = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
        dy[:, 0], dy[:, N - 1] = (torch.from_numpy(dv[:, i]).to(torch.bfloat16).cuda() for i in (0, 1))
        dx, _ = q.grouped_matmul_backward(dy, torch.from_numpy(xv).to(torch.bfloat16).cuda(), w, offsets, need_dw=False)
        assert torch.equal(dx.cpu(), torch.from_numpy(dv @ wl).to(torch.bfloat16))
    _, dw = q.grouped_matmul_backward(dy, torch.from_numpy(xv).to(torch.bfloat16).cuda(), w, offsets, need_dx=False)
    assert torch.equal(dw[E - 1, [0, N - 1]].cpu(), torch.from_numpy(dv.T @ xv).to(torch.bfloat16)) and not dw[:E - 1].any()
    del w, dw
    P, N, K = 36000, 65536, 64  # 4.7 GB of results
    x, wt = torch.zeros(P, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, N, K, dtype=torch.bfloat16, device="cuda")
    x[P - 1], wt[0, N - 1] = 2, 3
    y = q.grouped_matmul(x, wt, torch.tensor([0, P], dtype=torch.int32, device="cuda"))
    assert float(y[P - 1, N - 1]) == 6 * K and int(torch.count_nonzero(y[-2:])) == 1 and not y[0].any()


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 143, 159, 160, 161, 175, 176, 177, 191, 192, 193,
                                  223, 224, 225, 255, 256, 257, 383, 500])
def test_every_number_of_rows_in_a_tile(rows):
    """One expert with this many rows between two others, in the form of many results (tiles of 256 columns) and of few."""
    q = _q()
    for E, N, K, others in ((3, 300, 72, 5), (3, 8192, 40, 4200), (3, 8192, 24, 60)):
        counts = [others, rows, others // 2]
        P = sum(counts)
        offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        rng = np.random.default_rng(rows)
        x, w = rng.integers(-4, 5, (P, K)).astype(np.float32), rng.integers(-4, 5, (E, N, K)).astype(np.float32)
        y = q.grouped_matmul(dev(x).bfloat16(), dev(w).bfloat16(), dev(offsets), y_dtype=torch.float32)
        a, b = offsets[1], offsets[2]
        for e in range(E):
            lo, hi = (offsets[e], offsets[e + 1]) if e == 1 else (offsets[e], min(offsets[e + 1], offsets[e] + 300))
            assert torch.equal(y[lo:hi], torch.from_numpy(x[lo:hi]).cuda() @ torch.from_numpy(w[e]).cuda().t())
        dy = rng.integers(-2, 3, (P, N)).astype(np.float32)
        dx, dw = q.grouped_matmul_backward(dev(dy).bfloat16(), dev(x).bfloat16(), dev(w).bfloat16(), dev(offsets), dw_dtype=torch.float32) if N % 8 == 0 else (None, None)
        if dx is not None:
            assert torch.equal(dx[a:b], (torch.from_numpy(dy[a:b]).cuda() @ torch.from_numpy(w[1]).cuda()).bfloat16())
            assert torch.equal(dw[1], torch.from_numpy(dy[a:b]).cuda().t() @ torch.from_numpy(x[a:b]).cuda())


@pytest.mark.parametrize("T,E,k,N,K", [(64, 512, 8, 24, 64), (4096, 512, 2, 40, 48), (1 << 15, 9, 1, 16, 32), (300, 64, 16, 24, 40), (300, 65, 15, 24, 40),
                                       (9000, 3, 2, 2064, 48)])
def test_many_experts_and_many_rows(T, E, k, N, K):
    q = _q()
    x, xv, w, wv, offsets, perm = case(T, E, k, N, K, "f16", skew=1.0)
    rows = R.rows_of(perm, k, T, T * k)
    want, mag = R.matmul(xv, wv, offsets, rows)
    check(q.grouped_matmul(x, w, dev(offsets), dev(perm), k), want, mag, K, "f16")
    dy, dyv = half(0.1 * np.random.default_rng(5).standard_normal((T * k, N)), "f16")
    wx, ww, mx, mw = R.backward(dyv, xv, wv, offsets, rows)
    dx, dw = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), k, dw_dtype=torch.bfloat16)
    check(dx, wx, mx, N + k, "f16")
    check(dw, ww, mw, T, "bf16")


@pytest.mark.parametrize("P", [12, 900])
def test_unnamed_rows_in_long_sums(P):
    q = _q()
    T, E, k, N, K = 50, 4, 2, 2048, 2056
    x, xv, w, wv, _, _ = case(T, E, k, N, K, "bf16")
    rng = np.random.default_rng(P)
    perm = rng.integers(-3, T * k + 3, P).astype(np.int32)
    offsets = np.sort(np.concatenate([[0, P], rng.integers(0, P + 1, E - 1)])).astype(np.int32)
    rows = R.rows_of(perm, k, T, P)
    want, mag = R.matmul(xv, wv, offsets, rows)
    y = q.grouped_matmul(x, w, dev(offsets), dev(perm), k)
    check(y, want, mag, K, "bf16")
    assert not host(y)[rows < 0].any() and (rows < 0).any()
    dy, dyv = half(rng.standard_normal((P, N)), "bf16")
    _, ww, _, mw = R.backward(dyv, xv, wv, offsets, rows)
    _, dw = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), k, need_dx=False)
    check(dw, ww, mw, P, "bf16")


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("T", [4, 200])
def test_subnormal_operands(kind, T):
    """Products of the smallest values with large ones count in full."""
    q = _q()
    tiny, big = (2.0**-133, 2.0**120) if kind == "bf16" else (2.0**-24, 2.0**12)
    x = torch.full((T, 64), tiny, dtype=DT[kind], device="cuda")
    w = torch.full((1, 16, 64), big, dtype=DT[kind], device="cuda")
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    assert (q.grouped_matmul(x, w, offsets, y_dtype=torch.float32) == 64 * tiny * big).all()
    dy = torch.full((T, 16), big, dtype=DT[kind], device="cuda")
    dx, dw = q.grouped_matmul_backward(dy, x, torch.full_like(w, tiny), offsets, dw_dtype=torch.float32)
    assert (dx.float() == 16 * tiny * big).all() and (dw == T * tiny * big).all()


def test_no_tokens_behind_positions():
    q = _q()
    x, w = torch.zeros(0, 32, dtype=torch.bfloat16, device="cuda"), torch.ones(2, 16, 32, dtype=torch.bfloat16, device="cuda")
    perm, offsets = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    y = q.grouped_matmul(x, w, offsets, perm, 2)
    assert y.shape == (5, 16) and not y.any()
    dx, dw = q.grouped_matmul_backward(torch.ones_like(y), x, w, offsets, perm, 2)
    assert dx.shape == (0, 32) and not dw.any()


def test_results_of_the_c_abi_stay_in_their_rows():
    """Rows of results further apart than they are long: what lies between and around them stays as it was."""
    q = _q()
    B = q.binding
    for T, N, K, gap in ((9, 40, 64, 3), (300, 136, 72, 8), (300, 2041, 72, 1)):
        x, xv, w, wv, offsets, perm = case(T, 4, 2, N, K, "bf16")
        P = 2 * T
        store = torch.full((P + 2, N + gap), 7.0, device="cuda")
        d = B.make_grouped_dims(N, K, 4, 2, P, T, y_dtype=B.DS4MOE_F32)
        out = store[1:]
        if out.data_ptr() % 16:
            out = torch.full((P + 1, N + gap), 7.0, device="cuda")
        B.ds4moe_grouped_matmul(d, out, N + gap, x, K, None, w, None, dev(offsets), dev(perm))
        torch.cuda.synchronize()
        assert torch.equal(out[:P, :N], q.grouped_matmul(x, w, dev(offsets), dev(perm), 2, y_dtype=torch.float32))
        assert (out[:P, N:] == 7).all() and (out[P:] == 7).all()
        a = torch.randn(T, K, device="cuda").bfloat16()
        wc, ws = q.int8_quantize(torch.randn(N, K, device="cuda"))
        out.fill_(7)
        n = B.ds4moe_int8_workspace_bytes(T, K, B.DS4MOE_BF16)
        space = torch.empty(n, dtype=torch.uint8, device="cuda")
        B.ds4moe_int8_matmul(out, B.DS4MOE_F32, N + gap, a, None, B.DS4MOE_BF16, K, wc, ws, T, N, K, space, n)
        torch.cuda.synchronize()
        assert torch.equal(out[:T, :N], q.int8_matmul(a, wc, ws, y_dtype=torch.float32)) and (out[:T, N:] == 7).all() and (out[T:] == 7).all()


def test_a_training_step_of_routed_experts():
    """Gate, grouped up product, activation, grouped down product, weighted sum, and the whole of it backwards by the
    framework's gradients, against autograd in 64 bits on the same choice.  Steps hold fp16 values, 2^-11 each, and there
    are fewer than eight of them on any path: 2^-8 of the sums of absolute values along the paths bounds the result."""
    q = _q()
    T, E, k, H, I = 60, 8, 2, 128, 96
    rng = np.random.default_rng(0)
    x, xv = half(rng.standard_normal((T, H)), "f16")
    wu, uv = half(0.1 * rng.standard_normal((E, I, H)), "f16")
    wd, dv = half(0.1 * rng.standard_normal((E, H, I)), "f16")
    logits = torch.from_numpy(rng.standard_normal((T, E))).float().cuda()
    gy, gv = half(rng.standard_normal((T, H)), "f16")
    gate = q.Gate(E, k, score="sigmoid")
    r = gate.forward(logits)
    o, p = r["offsets"], r["perm"]
    a = q.grouped_matmul(x, wu, o, p, k)
    h = torch.relu(a)
    z = q.grouped_matmul(h, wd, o)
    pl = p.long()
    weight = r["topk_w"].reshape(-1)[pl]
    y = torch.zeros(T, H, device="cuda").index_add_(0, pl // k, z.float() * weight[:, None])
    # backwards
    dz = (gy.float()[pl // k] * weight[:, None]).half()
    d_weight = torch.empty(T * k, device="cuda")
    d_weight[pl] = (gy.float()[pl // k] * z.float()).sum(1)
    dh, dwd = q.grouped_matmul_backward(dz, h, wd, o)
    dx, dwu = q.grouped_matmul_backward(dh * (a > 0), x, wu, o, p, k)
    dl = gate.backward(logits, r["topk_idx"], d_weight.view(T, k))

    X, U, D, L = (torch.from_numpy(v).requires_grad_(True) for v in (xv, uv, dv, logits.double().cpu().numpy()))
    idx = r["topk_idx"].long().cpu()
    s = torch.sigmoid(L).gather(1, idx)
    s = s / s.sum(1, keepdim=True)
    act = (torch.bmm(U[idx].reshape(T * k, I, H), X.repeat_interleave(k, 0)[:, :, None])[:, :, 0])
    on = torch.from_numpy(host(a) > 0)[torch.argsort(pl.cpu())]  # the same side of the bend
    out = torch.bmm(D[idx].reshape(T * k, H, I), (act * on)[:, :, None])[:, :, 0].view(T, k, H)
    Y = (out * s[:, :, None]).sum(1)
    gX, gU, gD, gL = torch.autograd.grad((Y * torch.from_numpy(gv)).sum(), (X, U, D, L))
    with torch.no_grad():
        A = [v.abs() for v in (X, U, D, torch.from_numpy(gv))]
        hs = torch.bmm(A[1][idx].reshape(T * k, I, H), A[0].repeat_interleave(k, 0)[:, :, None])[:, :, 0]
        zs = torch.bmm(A[2][idx].reshape(T * k, H, I), hs[:, :, None])[:, :, 0]
        dzs = A[3].repeat_interleave(k, 0) * s.reshape(-1, 1)
        dhs = torch.bmm(A[2][idx].reshape(T * k, H, I).transpose(1, 2).contiguous(), dzs[:, :, None])[:, :, 0]
        dxs = torch.bmm(A[1][idx].reshape(T * k, I, H).transpose(1, 2).contiguous(), dhs[:, :, None])[:, :, 0].view(T, k, H).sum(1)
        flat = idx.reshape(-1)
        dws = torch.zeros(E, H, I, dtype=torch.float64).index_add_(0, flat, dzs[:, :, None] * hs[:, None, :])
        dus = torch.zeros(E, I, H, dtype=torch.float64).index_add_(0, flat, dhs[:, :, None] * A[0].repeat_interleave(k, 0)[:, None, :])
        dls = 2 * (A[3].repeat_interleave(k, 0) * zs).sum(1).view(T, k).sum(1, keepdim=True)
    for got, want, mag in ((y, Y.detach(), (zs.view(T, k, H) * s[:, :, None]).sum(1)), (dx, gX, dxs), (dwd, gD, dws), (dwu, gU, dus), (dl, gL, dls)):
        assert (np.abs(host(got) - want.detach().numpy()) <= 2.0**-8 * mag.detach().numpy() + 1e-6).all()


def test_gradients_of_rows_whose_last_stage_ends_beyond_32_bit_offsets():
    """513 rows within 2^32 bytes, 544 of which (whole stages of 32) are not: what lies at the buffer's start, where their
    offsets would come out again, adds nothing."""
    q = _q()
    P, step, N, K = 513, 8372128 // 2, 72, 64
    rng = np.random.default_rng(0)
    xs, ds = (torch.full((P * step,), 3.0, dtype=torch.bfloat16, device="cuda").view(P, step) for _ in range(2))
    xv, dv = rng.integers(-8, 9, (P, K)) / 4.0, rng.integers(-8, 9, (P, N)) / 4.0
    xs[:, :K], ds[:, :N] = torch.from_numpy(xv).to(torch.bfloat16).cuda(), torch.from_numpy(dv).to(torch.bfloat16).cuda()
    w = torch.zeros(1, N, K, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    rows = rng.permutation(P).astype(np.int32)
    for perm, order in ((None, np.arange(P)), (dev(rows), rows)):
        _, dw = q.grouped_matmul_backward(ds[:, :N], xs[:, :K], w, offsets, perm, need_dx=False, dw_dtype=torch.float32)
        assert np.array_equal(host(dw)[0], dv.T @ xv[order])  # sixteenths below 2^24 of them


def test_weights_gradients_of_many_experts_with_middling_rows():
    """Large tiles of experts whose sums are a few stages long, from one to a dozen: each of them ends in another part of
    the loop."""
    q = _q()
    E, N, K = 512, 264, 264
    rng = np.random.default_rng(5)
    rows = np.arange(E) % 400
    offsets = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    P = int(offsets[-1])
    perm = rng.permutation(P).astype(np.int32)
    x, xv = half(rng.integers(-8, 9, (P, K)) / 4.0, "bf16")
    dy, dv = half(rng.integers(-8, 9, (P, N)) / 4.0, "bf16")
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    for at, order in ((dev(perm), perm), (None, np.arange(P))):
        for _ in range(2):
            _, dw = q.grouped_matmul_backward(dy, x, w, dev(offsets), at, need_dx=False, dw_dtype=torch.float32)
            got = dw.cpu().numpy()
            for e in range(E):
                p = slice(offsets[e], offsets[e + 1])
                assert np.array_equal(got[e], dv[p].T @ xv[order[p]]), (e, rows[e])  # sixteenths below 2^24 of them
