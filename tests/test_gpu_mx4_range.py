"""The 4-bit microscaled operators over the rest of their range: the SwiGLU intermediate's bits in every form of the
experts, the streaming kernels over more than one step, scale bytes at both ends.

Bounds as in test_gpu_mx4, evaluated in 64 bits element by element; the intermediate's rounding is that of its terms: two
bf16 roundings, each of 2^-8 of what it rounds, leave 2^-16 of a value, three 2^-24.
"""
import numpy as np
import pytest
import torch

import mx4_ref as R
from test_gpu_mx4 import DT, EPS, _q, dev, experts_case, routing_of

pytestmark = pytest.mark.gpu


def experts_bound(x, idx, w, vals, dtype):
    """The 64-bit result and how far a call may be off it."""
    gv, uv, dv = vals
    terms, rest = (2, 2.0**-16) if dtype == "bf16" else (3, 2.0**-23)
    x = x.astype(np.float64)
    H, I = x.shape[1], gv.shape[1]
    y, b = np.zeros((x.shape[0], dv.shape[1])), np.zeros((x.shape[0], dv.shape[1]))
    for t in range(x.shape[0]):
        for e, a in zip(idx[t], w[t].astype(np.float64)):
            g, u = gv[e] @ x[t], uv[e] @ x[t]
            eg, eu = (EPS * (H + 2) * (np.abs(m[e]) @ np.abs(x[t])) for m in (gv, uv))
            s = g / (1 + np.exp(-g))
            h = s * u
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 8 * 2 * EPS * np.abs(h)
            eh = eh + rest * (np.abs(h) + eh)
            y[t] += a * (dv[e] @ h)
            m = np.abs(dv[e]) @ np.abs(h)
            b[t] += abs(a) * (np.abs(dv[e]) @ eh + EPS * (terms * I + 2) * m) + 20 * EPS * np.abs(a * (dv[e] @ h))
    return y, b + (2.0**-8 * (np.abs(y) + b) if dtype == "bf16" else 0)


def check_experts(dtype, x, ws, idx, w):
    q = _q()
    (E, I), H, k = ws[0][0].shape[:2], x.shape[1], idx.shape[1]
    want, bound = experts_bound(x, idx, w, [R.values(*m) for m in ws], dtype)
    ex = q.Mx4Experts(H, I, E, k, *[tuple(dev(v) for v in m) for m in ws], y_dtype=DT[dtype])
    xt, r = torch.from_numpy(x).cuda().to(torch.bfloat16), routing_of(idx, w, E)
    y = ex.forward(xt, r)
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= bound).all(), (float((err / np.maximum(bound, 1e-300)).max()), float((err > bound).mean()))
    assert torch.equal(y, ex.forward(xt, r))


@pytest.mark.parametrize("T,H,I,E,k", [
    (3, 64, 64, 4, 2), (12, 64, 64, 16, 2), (20, 64, 64, 2, 1), (70, 64, 96, 3, 2), (120, 96, 32, 4, 2), (300, 32, 128, 2, 1),
    (200, 1024, 64, 64, 4)])
def test_intermediate_holds_16_bits_however_many_tokens(T, H, I, E, k):
    """Short sums, so that a rounding of the intermediate to 8 bits is far above what the bound leaves to them."""
    check_experts("bf16", *experts_case(T, H, I, E, k, T + I))


# few tokens: rows of more than one step of the streaming kernels (gate and up 4096 columns a step, down 1024), with and
# without whole loads of scales, up to the most LDS that they stage
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I,E,k", [
    (16, 256, 2048, 64, 4), (16, 256, 1024, 64, 4), (8, 128, 1056, 32, 2), (8, 128, 1408, 32, 2), (8, 64, 4096, 32, 2),
    (6, 96, 2080, 24, 2), (5, 64, 2688, 12, 2),
    (1, 4128, 64, 8, 2), (8, 4128, 64, 12, 2), (1, 8192, 32, 4, 2), (8, 8192, 64, 12, 2), (9, 5120, 96, 12, 2), (4, 4608, 32, 12, 3),
    (7, 7168, 64, 12, 2), (16, 6176, 32, 16, 2)])
def test_streams_of_more_than_one_step(dtype, T, H, I, E, k):
    check_experts(dtype, *experts_case(T, H, I, E, k, T + H + I))


# ------------------------------------------------------------------ scale bytes at both ends
LOW, HIGH = (0, 1, 2, 30, 60), (190, 220, 250, 253, 254)


@pytest.mark.parametrize("kind", ["bf16", "mx4"])
@pytest.mark.parametrize("ends", ["low", "high"])
@pytest.mark.parametrize("M,N,K", [(1, 60, 96), (20, 60, 512), (60, 60, 256), (100, 60, 288), (300, 60, 512), (700, 1000, 128)])
def test_product_of_the_lowest_and_highest_scales(kind, ends, M, N, K):
    """Rows of blocks of one scale byte each, the other operand as far from 1 the other way: subnormal bf16 operands below
    2^-126 are exact.  Weights beyond bf16 (from 2^128 on) are infinities against bf16 activations and values against
    4-bit ones."""
    q = _q()
    rng = np.random.default_rng(M + N)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    codes[1::2] &= 0xBB  # magnitudes of 0 to 1.5: in range with any scale
    scales = np.array(LOW if ends == "low" else HIGH, np.uint8)[np.arange(N) // 2 % 5][:, None].repeat(K // 32, 1)
    a = rng.standard_normal((M, K))
    shift = 100 if ends == "low" else -100
    if kind == "mx4":
        ac, asc = R.quantize(a)
        asc = (asc.astype(int) + shift).astype(np.uint8)
        at, sa, av = dev(ac), dev(asc), R.values(ac, asc)
    else:
        av = np.ldexp(R.bf16(a.astype(np.float32)).astype(np.float64), shift)
        at, sa = torch.from_numpy(av).cuda().to(torch.bfloat16), None
    wv = R.values(codes, scales)
    y = q.mx4_matmul(at, dev(codes), dev(scales), sa, torch.float32).double().cpu().numpy()
    inf = np.abs(wv) >= 2.0**128
    rows = ~inf.any(axis=1) if kind == "bf16" else np.ones(N, bool)
    assert rows[1::2].all() and (ends == "low" or kind == "mx4" or not rows.all())
    want, mag = av @ wv[rows].T, np.abs(av) @ np.abs(wv[rows]).T
    err = np.abs(y[:, rows] - want)
    assert (err <= EPS * (K + 2) * mag).all(), float((err / np.maximum(EPS * (K + 2) * mag, 1e-300)).max())
    with np.errstate(invalid="ignore"):
        beyond = av @ np.where(inf, np.sign(wv) * np.inf, wv)[~rows].T
    assert np.array_equal(y[:, ~rows], beyond, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2, 9, 60])
def test_experts_of_the_lowest_scales(dtype, T):
    """Down weights about 2^-127 (subnormal in bf16) against an intermediate about 2^95 (the up projection's scales)."""
    H, I, E, k = 96, 64, 16, 2
    x, ws, idx, w = experts_case(T, H, I, E, k, T)
    ws[1] = (ws[1][0], (ws[1][1].astype(int) + 95).astype(np.uint8))
    ws[2] = (ws[2][0], np.random.default_rng(T).integers(0, 4, ws[2][1].shape).astype(np.uint8))
    check_experts(dtype, x, ws, idx, w)
