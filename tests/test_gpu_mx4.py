"""The 4-bit microscaled operators on the GPU against their 64-bit definitions.

Quantised codes and scales are exact, and so are dequantised values.  Products:
operands are exact, every product is exact in fp32 or nearly so and the fp32
sum of K terms is off by at most K 2^-24 of sum |a w| (any order); 2^-24 * (K + 2)
bounds it per element, and bf16 results add 2^-8 of their value.  Experts: the
gate and up sums as above, an ulp or three of the SwiGLU, the intermediate's
rounding (2^-9 in bf16, none to speak of in three terms), carried through the
down sums with their absolute values; the bound is evaluated in 64 bits from
the same inputs.
"""
import numpy as np
import pytest
import torch

import mx4_ref as R

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 2.0**-24


def _q():
    import quantized_routed_moe_router_amd as q
    return q


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def matrix(rows, cols, seed, sigma=0.02):
    return R.quantize(sigma * np.random.default_rng(seed).standard_normal((rows, cols)))


# ------------------------------------------------------------------ quantise
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 32, 0), (3, 1, 0), (5, 31, 2), (4, 33, 0), (16, 1000, 24), (7, 64, 3), (130, 96, 0), (2, 4100, 4)])
def test_quantize_is_the_definition(dtype, rows, cols, pad):
    q = _q()
    rng = np.random.default_rng(rows * cols)
    x = rng.standard_normal((rows, cols + pad)) * np.exp2(rng.integers(-20, 20, (rows, cols + pad)))
    x = torch.from_numpy(x.astype(np.float32)).cuda().to(DT[dtype])[:, :cols]
    codes, scales = q.mx4_quantize(x)
    rc, rs = R.quantize(x.float().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    v = R.values(rc, rs)[:, :cols]
    for out in ("f32", "bf16"):
        got = q.mx4_dequantize(codes, scales, cols, DT[out])
        assert np.array_equal(got.float().cpu().numpy().astype(np.float64), v)


def test_quantize_ties_edges_and_specials():
    """Every midpoint and its neighbours, saturation, subnormal blocks, the largest value, zeros, signed zeros, NaN and
    infinities (a block with one of them is NaN as a whole, its neighbours are not)."""
    q = _q()
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.99])
    near = np.concatenate([mid, mid * (1 + 2.0**-23), mid * (1 - 2.0**-23), [4.0, 0.0]])[:32]
    near[31] = 4.0
    tiny = float(np.float32(2.0**-149))
    blocks = [near, -near, near * 2.0**-120, np.full(32, tiny), np.linspace(0, 1, 32) * 2.0**-126, np.zeros(32), -np.zeros(32),
              np.full(32, R.FMAX), np.linspace(-R.FMAX, R.FMAX, 32), np.ones(32)]
    for bad in (np.nan, np.inf, -np.inf):
        b = np.ones(32)
        b[17] = bad
        blocks += [b, np.ones(32)]
    x = np.concatenate(blocks).astype(np.float32)[None]
    codes, scales = q.mx4_quantize(dev(x))
    rc, rs = R.quantize(x)
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)
    got = q.mx4_dequantize(codes, scales).cpu().numpy().astype(np.float64)
    want = R.values(rc, rs)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(want).sum() == 96
    assert np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_every_code_and_scale():
    q = _q()
    codes = np.tile(np.arange(256, dtype=np.uint8), 16).reshape(256, 16)
    scales = np.arange(256, dtype=np.uint8)[:, None]
    want = R.values(codes, scales)
    with np.errstate(over="ignore"):
        want = want.astype(np.float32).astype(np.float64)
    got = q.mx4_dequantize(dev(codes), dev(scales)).cpu().numpy().astype(np.float64)
    assert np.array_equal(got, want, equal_nan=True)
    assert q.mx4_quantize(torch.empty(0, 64, device="cuda"))[0].shape == (0, 32)


# ------------------------------------------------------------------ product
def product_case(M, N, K, kind, seed, pad=0):
    rng = np.random.default_rng(seed)
    w = matrix(N, K, seed)
    if kind == "mx4":
        a = R.quantize(rng.standard_normal((M, K)))
        return (dev(a[0]), dev(a[1])), R.values(*a), w
    x = R.bf16(rng.standard_normal((M, K + pad)).astype(np.float32))
    return (torch.from_numpy(x).cuda().to(torch.bfloat16)[:, :K], None), x[:, :K].astype(np.float64), w


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("M,N,K", [
    (1, 16, 32), (1, 512, 4096), (2, 17, 96), (3, 1, 32), (15, 33, 160), (16, 64, 128), (17, 100, 1056), (37, 1000, 2080),
    (64, 128, 256), (65, 129, 288), (128, 256, 512), (130, 500, 96), (200, 80, 4128), (257, 272, 640), (513, 384, 384),
    (513, 3000, 96), (1600, 4096, 96), (1600, 4096, 128), (2048, 3100, 256), (2047, 3101, 640),
    (2048, 3100, 768), (600, 384, 768)])
def test_product(kind, M, N, K):
    q = _q()
    (a, sa), av, w = product_case(M, N, K, kind, M + N + K, pad=8 if M % 2 else 0)
    wv = R.values(*w)
    want, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    for dtype in ("f32", "bf16"):
        y = q.mx4_matmul(a, dev(w[0]), dev(w[1]), sa, DT[dtype])
        assert y.shape == (M, N) and y.dtype == DT[dtype]
        err = np.abs(y.double().cpu().numpy() - want)
        bound = EPS * (K + 2) * mag + (2.0**-8 * np.abs(want) if dtype == "bf16" else 0)
        assert (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())
        assert torch.equal(y, q.mx4_matmul(a, dev(w[0]), dev(w[1]), sa, DT[dtype]))


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_product_of_every_scale(kind, M):
    """Weights whose blocks' scales span 2^-60 .. 2^60, with NaN scales: only the rows that hold one are NaN."""
    q = _q()
    rng = np.random.default_rng(5)
    N, K = 48, 256
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = rng.integers(67, 188, (N, K // 32), dtype=np.uint8)
    scales[7, 3] = 255
    (a, sa), av, _ = product_case(M, N, K, kind, 1)
    wv = R.values(codes, scales)
    want, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    y = q.mx4_matmul(a, dev(codes), dev(scales), sa, torch.float32).double().cpu().numpy()
    assert np.isnan(y[:, 7]).all() and np.isfinite(np.delete(y, 7, axis=1)).all()
    live = [n for n in range(N) if n != 7]
    assert (np.abs(y - want)[:, live] <= EPS * (K + 2) * mag[:, live]).all()


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("M", [2, 100])
def test_product_of_strange_rows_stays_in_its_rows(kind, M):
    """A NaN row of activations reaches its own results alone; rows of a wider result are left as they are."""
    q = _q()
    B = q.binding
    N, K = 70, 96
    (a, sa), av, w = product_case(M, N, K, kind, 3)
    if kind == "bf16":
        a = a.clone()
        a[1] = float("nan")
    else:
        sa = sa.clone()
        sa[1] = 255
    wide = torch.full((M, N + 11), 7.0, device="cuda")
    wc, ws = dev(w[0]), dev(w[1])
    B.ds4moe_mx4_matmul(wide, B.DS4MOE_F32, N + 11, a, sa, B.DS4MOE_BF16 if sa is None else B.DS4MOE_MX4, K, wc, ws, M, N, K)
    y = wide.double().cpu().numpy()
    assert (y[:, N:] == 7).all() and np.isnan(y[1, :N]).all()
    rows = [m for m in range(M) if m != 1]
    wv = R.values(*w)
    assert (np.abs(y[rows, :N] - av[rows] @ wv.T) <= EPS * (K + 2) * (np.abs(av[rows]) @ np.abs(wv).T)).all()


def test_rows_that_overlap_are_refused():
    """A row repeated by a stride of 0 is not a matrix of rows that lie apart."""
    q = _q()
    w = matrix(32, 64, 0)
    x = torch.ones(1, 64, dtype=torch.bfloat16, device="cuda").expand(4, 64)
    for call in (lambda: q.mx4_quantize(x), lambda: q.mx4_matmul(x, dev(w[0]), dev(w[1])), lambda: q.Gate(64, 2).forward(x),
                 lambda: q.mx4_quantize(torch.ones(64, 4, device="cuda").t())):
        with pytest.raises(ValueError):
            call()


def test_product_without_rows():
    q = _q()
    w = matrix(32, 64, 0)
    assert q.mx4_matmul(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), dev(w[0]), dev(w[1])).shape == (0, 32)


# ------------------------------------------------------------------ experts
def experts_case(T, H, I, E, k, seed, skew=0.0):
    rng = np.random.default_rng(seed)
    x = R.bf16(rng.standard_normal((T, H)).astype(np.float32))
    ws = [[matrix(r, c, seed + 7 * e + n, 0.05) for e in range(E)] for n, (r, c) in enumerate(((I, H), (I, H), (H, I)))]
    ws = [(np.stack([m[0] for m in w]), np.stack([m[1] for m in w])) for w in ws]
    logits = rng.standard_normal((T, E)) - skew * np.arange(E)
    idx, w, _ = R.gate(logits, None, k, "softmax")
    return x, ws, idx, w.astype(np.float32)


def routing_of(idx, w, E):
    c, o, p = R.permutation(idx, E)
    d = {"topk_idx": idx, "counts": c, "offsets": o, "perm": p}
    return {**{n: dev(v.astype(np.int32)) for n, v in d.items()}, "topk_w": dev(w)}


def experts_bound(x, idx, w, vals, bf16_y):
    """The 64-bit result and how far a call may be off it, element by element."""
    gv, uv, dv = vals
    x = x.astype(np.float64)
    H, I = x.shape[1], gv.shape[1]
    y, b = np.zeros((x.shape[0], dv.shape[1])), np.zeros((x.shape[0], dv.shape[1]))
    for t in range(x.shape[0]):
        for e, a in zip(idx[t], w[t].astype(np.float64)):
            if not 0 <= e < gv.shape[0]:
                continue
            g, u = gv[e] @ x[t], uv[e] @ x[t]
            eg, eu = (EPS * (H + 2) * (np.abs(m[e]) @ np.abs(x[t])) for m in (gv, uv))
            s = g / (1 + np.exp(-g))
            h = s * u
            # |silu'| <= 1.1; the SwiGLU itself in fp32: 8 ulp
            eh = 1.1 * eg * (np.abs(u) + eu) + (np.abs(s)) * eu + 8 * 2 * EPS * np.abs(h)
            eh = eh + (2.0**-9 if bf16_y else 2.0**-23) * (np.abs(h) + eh)
            y[t] += a * (dv[e] @ h)
            m = np.abs(dv[e]) @ np.abs(h)
            b[t] += abs(a) * (np.abs(dv[e]) @ eh + EPS * (3 * I + 2) * m) + 20 * EPS * np.abs(a * (dv[e] @ h))
    return y, b + (2.0**-8 * np.abs(y) if bf16_y else 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I,E,k,skew", [
    (1, 256, 128, 8, 2, 0.0), (1, 32, 32, 1, 1, 0.0), (2, 96, 160, 5, 3, 0.0), (7, 1024, 352, 6, 4, 0.5), (16, 320, 64, 16, 4, 0.0),
    (33, 160, 96, 3, 2, 1.0), (70, 512, 256, 9, 2, 0.4), (150, 256, 288, 4, 3, 1.0), (300, 128, 128, 40, 4, 0.1),
    (520, 96, 96, 2, 1, 1.0),
    # few tokens of many experts; experts of more than four of them; rows longer than one pass holds
    (8, 256, 128, 16, 2, 0.0), (16, 512, 256, 32, 2, 0.0), (12, 1024, 352, 64, 4, 0.1), (16, 256, 128, 64, 4, 1.0),
    (16, 8224, 96, 64, 2, 0.2), (1, 8224, 64, 8, 2, 0.0), (3, 9216, 32, 4, 2, 0.0), (1, 64, 2080, 4, 2, 0.0),
    (1, 32, 8192, 4, 2, 0.0), (4, 64, 2080, 6, 3, 0.0), (6, 32, 4128, 16, 2, 0.0),
    # tiles of 256 weight rows
    (200, 1024, 512, 64, 4, 0.0), (230, 1056, 544, 64, 4, 0.3)])
def test_experts(dtype, T, H, I, E, k, skew):
    q = _q()
    x, ws, idx, w = experts_case(T, H, I, E, k, T + H, skew)
    want, bound = experts_bound(x, idx, w, [R.values(*m) for m in ws], dtype == "bf16")
    ex = q.Mx4Experts(H, I, E, k, *[tuple(dev(v) for v in m) for m in ws], y_dtype=DT[dtype])
    xt, r = torch.from_numpy(x).cuda().to(torch.bfloat16), routing_of(idx, w, E)
    y = ex.forward(xt, r)
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= bound).all(), float((err / np.maximum(bound, 1e-300)).max())
    assert torch.equal(y, ex.forward(xt, r))
    # rows of a wider buffer
    wide = torch.zeros(T, H + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, :H] = xt
    assert torch.equal(y, ex.forward(wide[:, :H], r))
    # a token alone goes through other kernels: within the same bound
    one = ex.forward(xt[T // 2:T // 2 + 1], routing_of(idx[T // 2:T // 2 + 1], w[T // 2:T // 2 + 1], E))
    assert (np.abs(one.double().cpu().numpy()[0] - want[T // 2]) <= bound[T // 2]).all()


def test_experts_of_no_tokens_and_of_indices_out_of_range():
    q = _q()
    x, ws, idx, w = experts_case(4, 64, 64, 4, 2, 0)
    ex = q.Mx4Experts(64, 64, 4, 2, *[tuple(dev(v) for v in m) for m in ws], y_dtype=torch.float32)
    assert ex.forward(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), routing_of(idx[:0], w[:0], 4)).shape == (0, 64)
    r = routing_of(idx, w, 4)
    bad = idx.copy()
    bad[1, 0], bad[2, 1] = -1, 99
    r["topk_idx"] = dev(bad.astype(np.int32))
    y = ex.forward(torch.from_numpy(x).cuda().to(torch.bfloat16), r).double().cpu().numpy()
    want, bound = experts_bound(x, bad, w, [R.values(*m) for m in ws], False)
    # an expert's range is opened by its first assignment: tokens whose experts' ranges are whole are right
    first = {int(e): int(np.flatnonzero(idx.reshape(-1) == e)[0]) for e in np.unique(idx)}
    whole = [t for t in range(4) if all(bad.reshape(-1)[first[int(e)]] == e for e in idx[t])]
    assert np.isfinite(y[whole]).all()
    assert (np.abs(y - want)[whole] <= bound[whole]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_too_far_apart_for_32_bits(dtype):
    """Tokens that span more than 2^32 bytes of their buffer."""
    q = _q()
    T, H, I, E, k = 140, 96, 64, 4, 2
    x, ws, idx, w = experts_case(T, H, I, E, k, 1)
    buf = torch.empty(T, 2**24, dtype=torch.bfloat16, device="cuda")
    far = buf[:, :H]
    far.copy_(torch.from_numpy(x))
    ex = q.Mx4Experts(H, I, E, k, *[tuple(dev(v) for v in m) for m in ws], y_dtype=DT[dtype])
    r = routing_of(idx, w, E)
    assert torch.equal(ex.forward(far, r), ex.forward(far.contiguous(), r))
    wc, sc = dev(ws[0][0][0]), dev(ws[0][1][0])
    assert torch.equal(q.mx4_matmul(far, wc, sc, y_dtype=DT[dtype]), q.mx4_matmul(far.contiguous(), wc, sc, y_dtype=DT[dtype]))
    del far, buf
    farther = torch.empty(70, 2**24 + 8, dtype=torch.bfloat16, device="cuda")[:, :H]
    farther.copy_(torch.from_numpy(x[:70]))
    got, want = (q.mx4_matmul(a, wc, sc, y_dtype=torch.float32) for a in (farther, farther.contiguous()))
    mag = np.abs(x[:70].astype(np.float64)) @ np.abs(R.values(ws[0][0][0], ws[0][1][0])).T
    assert (np.abs((got - want).double().cpu().numpy()) <= 2 * EPS * (H + 2) * mag).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 3, 12, 60])
def test_index_out_of_range_adds_nothing_to_its_token(dtype, T):
    q = _q()
    H, I, E, k = 96, 64, 16, 2
    x, ws, idx, w = experts_case(T, H, I, E, k, T)
    r = routing_of(idx, w, E)
    bad = idx.copy()
    bad[::3, 0], bad[1::5, 1] = -1, E
    r["topk_idx"] = dev(bad.astype(np.int32))
    ex = q.Mx4Experts(H, I, E, k, *[tuple(dev(v) for v in m) for m in ws], y_dtype=DT[dtype])
    y = ex.forward(torch.from_numpy(x).cuda().to(torch.bfloat16), r).double().cpu().numpy()
    want, bound = experts_bound(x, bad, w, [R.values(*m) for m in ws], dtype == "bf16")
    assert (np.abs(y - want) <= bound).all()


def test_experts_beyond_32_bit_offsets():
    """A gate matrix whose last experts' codes lie past 2^31 bytes."""
    q = _q()
    H, I, E, k, T = 4096, 4096, 300, 1, 2
    g = torch.Generator(device="cuda").manual_seed(0)
    code = [torch.randint(0, 256, (E, r, c // 2), dtype=torch.uint8, device="cuda", generator=g) for r, c in ((I, H), (I, H), (H, I))]
    assert code[0].numel() > 2**31
    scale = [torch.full((E, r, c // 32), 120, dtype=torch.uint8, device="cuda") for r, c in ((I, H), (I, H), (H, I))]
    idx, w = np.array([[299], [281]]), np.array([[1.0], [0.5]], np.float32)
    x = R.bf16(np.random.default_rng(0).standard_normal((T, H)).astype(np.float32))
    ex = q.Mx4Experts(H, I, E, k, *zip(code, scale), y_dtype=torch.float32)
    y = ex.forward(torch.from_numpy(x).cuda().to(torch.bfloat16), routing_of(idx, w, E)).double().cpu().numpy()
    for t in range(T):
        e = int(idx[t, 0])
        vals = [R.values(c[e:e + 1].cpu().numpy(), s[e:e + 1].cpu().numpy()) for c, s in zip(code, scale)]
        want, bound = experts_bound(x[t:t + 1], np.zeros((1, 1), int), w[t:t + 1], vals, False)
        assert (np.abs(y[t] - want[0]) <= bound[0]).all()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("T", [1, 9, 100])
def test_layer_runs_gate_and_experts_together(T):
    """Router, gate and experts as one layer, against the 64-bit composition on the layer's own logits."""
    q = _q()
    H, I, E, k = 256, 64, 16, 4
    x, ws, _, _ = experts_case(T, H, I, E, k, 3)
    rng = np.random.default_rng(1)
    router, bias = (0.1 * rng.standard_normal((E, H))).astype(np.float32), (0.05 * rng.standard_normal(E)).astype(np.float32)
    layer = q.Mx4Layer(dev(router), q.Gate(E, k, "sigmoid", 4, 2, 2, scale=2.5),
                       q.Mx4Experts(H, I, E, k, *[tuple(dev(v) for v in m) for m in ws], y_dtype=torch.float32), dev(bias))
    xt = torch.from_numpy(x).cuda().to(torch.bfloat16)
    l = layer.logits(xt).double().cpu().numpy()
    want_l = x.astype(np.float64) @ router.astype(np.float64).T
    assert np.array_equal(l.astype(np.float32), want_l.astype(np.float32))
    idx, w, gaps = R.gate(l, bias, k, "sigmoid", 4, 2, 2, True, 2.5)
    y = layer.forward(xt).double().cpu().numpy()
    want, bound = experts_bound(x, idx, w, [R.values(*m) for m in ws], False)
    sure = gaps > 1e-5
    assert sure.mean() > 0.9
    # the weights' own error, 3e-6, on top of the experts'
    assert (np.abs(y - want)[sure] <= (bound + 3e-6 * np.abs(want).max(axis=1, keepdims=True) * k)[sure]).all()


def test_layer_in_a_graph_and_on_another_stream():
    q = _q()
    T, H, I, E, k = 5, 256, 64, 8, 2
    x, ws, _, _ = experts_case(T, H, I, E, k, 4)
    router = (0.1 * np.random.default_rng(1).standard_normal((E, H))).astype(np.float32)
    layer = q.Mx4Layer(dev(router), q.Gate(E, k, "softmax"), q.Mx4Experts(H, I, E, k, *[tuple(dev(v) for v in m) for m in ws]))
    xt = torch.from_numpy(x).cuda().to(torch.bfloat16)
    want = layer.forward(xt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = layer.forward(xt)
    s.synchronize()
    assert torch.equal(want, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer.forward(xt)
    for sign in (1.0, -1.0, 0.5):
        new = torch.from_numpy(x).cuda().to(torch.bfloat16) * sign
        xt.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, layer.forward(new))
