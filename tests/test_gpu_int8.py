"""The 8-bit integer operators on the GPU against their 64-bit definitions.

Codes and scales are exact (the nearest integer to the exact quotient, ties to even), and so are dequantised values but
for one rounding.  A product's sum of integers is exact; turning it to fp32 and the two scales round three times, 2^-24
each, and a bf16 or fp16 result once more.
"""
import numpy as np
import pytest
import torch

import grouped_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _q():
    import quantized_routed_moe_router_amd as q
    return q


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def same(got, want):
    return np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 16, 0), (5, 31, 2), (16, 1001, 24), (70, 256, 0), (33, 257, 7), (9, 2048, 8), (7, 2049, 0),
                                           (4, 4096, 0), (3, 16384, 0), (2, 16400, 16), (3, 40001, 3), (1000, 48, 0), (300, 4095, 1)])
def test_quantize_is_the_definition(dtype, rows, cols, pad):
    q = _q()
    rng = np.random.default_rng(rows * cols)
    x = rng.standard_normal((rows, cols + pad)) * np.exp2(rng.integers(-10, 6, (rows, 1)))
    x = torch.from_numpy(x).to(DT[dtype]).cuda()[:, :cols]
    codes, scales = q.int8_quantize(x)
    rc, rs = R.quantize(x.double().cpu().numpy())
    assert same(scales.cpu().numpy(), rs) and same(codes.cpu().numpy(), rc)
    values = rc.astype(np.float32) * rs[:, None]
    for out in DT:
        got = q.int8_dequantize(codes, scales, cols, DT[out])
        assert got.dtype == DT[out] and torch.equal(got.cpu(), torch.from_numpy(values[:, :cols]).to(DT[out]))


def test_quantize_borders():
    """Quotients at and next to every half integer, in units from the subnormals to the largest: the scale of a row is its
    first value's, 127 units."""
    q = _q()
    rows = []
    for unit in (1.0, 0.75, 2.0**-126, 2.0**-140, 2.0**-149, 2.0**-70 * 1.37, 2.0**120 * 1.1, 1e-30, 3.3e-9):
        u = np.float64(np.float32(unit))
        half = (np.arange(-127, 127) + 0.5) * u
        near = np.concatenate([half, half * (1 + 2.0**-23), half * (1 - 2.0**-23), np.arange(-127, 128) * u])
        with np.errstate(over="ignore"):
            rows.append(np.concatenate([[127 * u], near]).astype(np.float32))
    x = np.stack(rows)
    codes, scales = q.int8_quantize(dev(x))
    rc, rs = R.quantize(x)
    assert same(scales.cpu().numpy(), rs) and same(codes.cpu().numpy(), rc)
    # random rows of few bits, where ties are frequent
    x = (np.random.default_rng(0).integers(-254, 255, (200, 777)) / 2).astype(np.float32)
    x[:, 0] = 127
    codes, scales = q.int8_quantize(dev(x))
    rc, rs = R.quantize(x)
    assert same(scales.cpu().numpy(), rs) and same(codes.cpu().numpy(), rc)


def test_quantize_specials():
    """Zeros, signed zeros, the smallest and the largest values, NaN and infinities: only their own rows are touched."""
    q = _q()
    fmax, tiny = float(np.finfo(np.float32).max), float(np.float32(2.0**-149))
    x = np.ones((9, 50), dtype=np.float32)
    x[1], x[2], x[3], x[4] = 0, -0.0, tiny, fmax
    x[5, 17], x[6, 17], x[7, 49] = np.nan, np.inf, -np.inf
    x[8] = np.linspace(-fmax, fmax, 50)
    codes, scales = q.int8_quantize(dev(x))
    rc, rs = R.quantize(x)
    assert np.isnan(rs).sum() == 3 and rs[3] == np.float32(tiny)
    assert same(scales.cpu().numpy(), rs) and same(codes.cpu().numpy(), rc)
    got = q.int8_dequantize(codes, scales, 50).cpu().numpy()
    assert np.isnan(got[5:8]).all() and np.isfinite(got[[0, 1, 2, 3, 4, 8]]).all()
    assert q.int8_quantize(torch.empty(0, 64, device="cuda"))[0].shape == (0, 64)
    c, s = q.int8_quantize(torch.empty(3, 0, device="cuda"))
    assert c.shape == (3, 0) and not s.any()


PRODUCTS = [(1, 16, 16), (1, 512, 4096), (2, 17, 96), (3, 1, 32), (15, 33, 160), (16, 64, 128), (17, 100, 1056), (37, 1001, 2064), (64, 128, 256),
            (65, 129, 288), (128, 256, 512), (130, 500, 96), (200, 80, 4128), (257, 272, 640), (513, 384, 384), (600, 3000, 48), (1030, 1100, 272)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(M, N, K):
    q = _q()
    rng = np.random.default_rng(M + N + K)
    a, w = rng.integers(-128, 128, (M, K + 16)).astype(np.int8), rng.integers(-128, 128, (N, K)).astype(np.int8)
    sa, sw = (rng.random(M) + 0.1).astype(np.float32) / 127, (rng.random(N) + 0.1).astype(np.float32) / 127
    want = (a[:, :K].astype(np.float64) @ w.astype(np.float64).T) * sa.astype(np.float64)[:, None] * sw.astype(np.float64)
    at = dev(a)[:, :K]
    for out in DT:
        y = q.int8_matmul(at, dev(w), dev(sw), dev(sa), y_dtype=DT[out])
        assert y.shape == (M, N) and y.dtype == DT[out]
        err = np.abs(y.double().cpu().numpy() - want)
        bound = (3 * 2.0**-24 * (1 + 2.0**-20) + (R.HALF_STEP[out] * (1 + 2.0**-7) if out != "f32" else 0)) * np.abs(want) + R.TINY[out]
        assert (err <= bound).all(), float((err / bound).max())
        assert torch.equal(y, q.int8_matmul(at.contiguous(), dev(w), dev(sw), dev(sa), y_dtype=DT[out]))


def test_the_largest_sums_are_exact():
    """131056 products of -128 by -128: 2147221504, next to the end of 32 bits."""
    q = _q()
    K = 131056
    for M in (1, 40, 130):
        a, w = torch.full((M, K), -128, dtype=torch.int8, device="cuda"), torch.full((20, K), -128, dtype=torch.int8, device="cuda")
        one = torch.ones(M, device="cuda"), torch.ones(20, device="cuda")
        y = q.int8_matmul(a, w, one[1], one[0], y_dtype=torch.float32)
        assert (y == float(np.float32(K * 16384))).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (1, 512, 4096), (1, 100, 4095), (3, 33, 1001), (5, 20, 16384), (16, 64, 1000), (17, 100, 1056), (40, 65, 2049),
                                   (130, 140, 300), (2, 20, 40001)])
def test_product_quantises_its_activations(dtype, M, N, K):
    """The same bits as of the two calls, at any length and step of the rows."""
    q = _q()
    rng = np.random.default_rng(M * N + K)
    a = torch.from_numpy(rng.standard_normal((M, K + M % 3))).to(DT[dtype]).cuda()[:, :K]
    if M > 2:
        a[1] = 0
        a[2, K // 2] = float("inf")
    w, sw = q.int8_quantize(torch.from_numpy(rng.standard_normal((N, K))).float().cuda())
    codes, sa = q.int8_quantize(a)
    for out in DT:
        y = q.int8_matmul(a, w, sw, y_dtype=DT[out])
        want = q.int8_matmul(codes, w, sw, sa, y_dtype=DT[out])
        assert torch.equal(torch.nan_to_num(y, nan=7.5), torch.nan_to_num(want, nan=7.5))
        if M > 2:
            assert torch.isnan(y[2]).all() and not torch.isnan(y[3:]).any() and not y[1].any()


def test_product_in_a_graph_and_on_a_side_stream():
    q = _q()
    a = torch.randn(9, 200, device="cuda").bfloat16()
    w, sw = q.int8_quantize(torch.randn(70, 200, device="cuda"))
    want = q.int8_matmul(a, w, sw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        side = q.int8_matmul(a, w, sw)
    s.synchronize()
    assert torch.equal(side, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = q.int8_matmul(a, w, sw)
        back = q.int8_dequantize(*q.int8_quantize(a), 200)
    for i in range(4):
        a.copy_(torch.randn(9, 200, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        got, codes = y.clone(), back.clone()
        assert torch.equal(got, q.int8_matmul(a, w, sw)) and torch.equal(codes, q.int8_dequantize(*q.int8_quantize(a), 200))
    assert q.int8_matmul(a[:0], w, sw).shape == (0, 70) and q.int8_matmul(a, w[:0], sw[:0]).shape == (9, 0)


def test_routed_experts_of_8_bits_run_together():
    """Gate, quantised tokens, grouped gate and up products, SwiGLU, quantised again, grouped down product, weighted sum:
    against the same steps in 64 bits on the codes that the calls made."""
    q = _q()
    T, E, k, H, I = 50, 12, 3, 256, 96
    g = torch.Generator().manual_seed(0)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    logits = torch.randn(T, E, generator=g).cuda()
    up, down = 0.05 * torch.randn(E, 2 * I, H, generator=g).cuda(), 0.1 * torch.randn(E, H, I, generator=g).cuda()
    uc, us = q.int8_quantize(up.view(-1, H))
    dc, ds = q.int8_quantize(down.view(-1, I))
    uc, us, dc, ds = uc.view(E, 2 * I, H), us.view(E, 2 * I), dc.view(E, H, I), ds.view(E, H)
    r = q.Gate(E, k).forward(logits)
    xc, xs = q.int8_quantize(x)
    h = q.grouped_matmul(xc, uc, r["offsets"], r["perm"], k, x_scales=xs, w_scales=us, y_dtype=torch.float32)
    h = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
    hc, hs = q.int8_quantize(h)
    y = q.grouped_matmul(hc, dc, r["offsets"], x_scales=hs, w_scales=ds, y_dtype=torch.float32)
    perm = r["perm"].long()
    out = torch.empty_like(y).index_copy_(0, perm, y).view(T, k, H)
    out = (out * r["topk_w"][:, :, None]).sum(1)
    # 64 bits
    idx, tw = r["topk_idx"].cpu().numpy(), r["topk_w"].cpu().double().numpy()
    val = lambda c, s: c.cpu().double().numpy() * s.cpu().double().numpy()[..., None]
    xv, uv, dv, hv = val(xc, xs), val(uc, us), val(dc, ds), val(hc, hs)
    want, mag, pos = np.zeros((T, H)), np.zeros((T, H)), np.empty(T * k, dtype=np.int64)
    pos[perm.cpu().numpy()] = np.arange(T * k)
    for t in range(T):
        for j in range(k):
            e, p = idx[t, j], pos[t * k + j]
            a = uv[e] @ xv[t]
            act = a[:I] / (1 + np.exp(-a[:I])) * a[I:]
            # the 8-bit intermediate is within half a step, and a little more for the fp32 steps before it
            assert (np.abs(hv[p] - act) <= 0.51 * float(hs[p])).all()
            v = tw[t, j] * (dv[e] @ hv[p])
            want[t] += v
            mag[t] += np.abs(v)
    assert (np.abs(out.cpu().double().numpy() - want) <= 2.0**-20 * mag).all()


@pytest.mark.parametrize("rows,cols", [(9001, 40), (65549, 250), (4103, 300), (9000, 264), (2050, 4097), (70000, 272)])
def test_more_rows_than_workgroups_go_round(rows, cols):
    q = _q()
    x = (np.random.default_rng(rows).standard_normal((rows, cols)) * 3).astype(np.float32)
    codes, scales = q.int8_quantize(dev(x))
    rc, rs = R.quantize(x)
    assert same(scales.cpu().numpy(), rs) and same(codes.cpu().numpy(), rc)
    got = q.int8_dequantize(codes, scales, cols)
    assert np.array_equal(got.cpu().numpy(), (rc.astype(np.float32) * rs[:, None])[:, :cols])


@pytest.mark.parametrize("M,K", [(1, 65520), (1, 65521), (2, 32752), (15, 4336), (16, 4080), (16, 4081), (9, 7200)])
def test_rows_up_to_the_size_of_a_workgroups_memory(M, K):
    """The longest rows that are quantised in the product's own launch, and the shortest that are not: the same bits as of
    two calls."""
    q = _q()
    rng = np.random.default_rng(K)
    a = dev(rng.standard_normal((M, K)).astype(np.float32))
    w, sw = q.int8_quantize(dev(rng.standard_normal((33, K)).astype(np.float32)))
    codes, sa = q.int8_quantize(a)
    assert torch.equal(q.int8_matmul(a, w, sw, y_dtype=torch.float32), q.int8_matmul(codes, w, sw, sa, y_dtype=torch.float32))
