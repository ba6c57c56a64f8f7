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
