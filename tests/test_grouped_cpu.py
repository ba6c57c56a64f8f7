"""The 8-bit integer operators and the products grouped by expert without a GPU: what the C ABI refuses (fake addresses,
never read: every call returns before a launch), and what the torch entry points check before they call it."""
import ctypes

import numpy as np
import pytest
import torch

import grouped_ref as R
import quantized_routed_moe_router_amd as q
from quantized_routed_moe_router_amd import binding as B
from test_mx4_entry_cpu import Tensor

I8, I32, BF16, F16, F32 = torch.int8, torch.int32, torch.bfloat16, torch.float16, torch.float32
NULL, SHAPE, DTYPE, ALIGN, WS, UNSUP = (B.DS4MOE_ERR_NULL, B.DS4MOE_ERR_SHAPE, B.DS4MOE_ERR_DTYPE, B.DS4MOE_ERR_ALIGN,
                                        B.DS4MOE_ERR_WORKSPACE, B.DS4MOE_ERR_UNSUPPORTED)
A = 1 << 20  # an aligned address


def dims(**kw):
    d = dict(dtype=B.DS4MOE_BF16, y_dtype=B.DS4MOE_BF16, n_experts=4, top_k=2, rows=20, tokens=10, N=64, K=128)
    d.update(kw)
    return ctypes.byref(B.GroupedDims(**d))


def forward(d=None, ldy=64, ldx=128, xs=None, ws=None, **kw):
    p = {"y": A, "x": A, "w": A, "offsets": A, "perm": A, **kw}
    return B.lib().ds4moe_grouped_matmul(d if d is not None else dims(), p["y"], ldy, p["x"], ldx, xs, p["w"], ws, p["offsets"],
                                         p["perm"], None)


def dx(d=None, lddx=128, lddy=64, ws=A, n=1 << 40, **kw):
    p = {"dx": A, "dy": A, "w": A, "offsets": A, "perm": A, **kw}
    return B.lib().ds4moe_grouped_dx(d if d is not None else dims(), p["dx"], lddx, p["dy"], lddy, p["w"], p["offsets"], p["perm"], ws, n,
                                     None)


def dw(d=None, lddy=64, ldx=128, **kw):
    p = {"dw": A, "dy": A, "x": A, "offsets": A, "perm": A, **kw}
    return B.lib().ds4moe_grouped_dw(d if d is not None else dims(), p["dw"], p["dy"], lddy, p["x"], ldx, p["offsets"], p["perm"], None)


BAD_DIMS = [(dict(dtype=0), DTYPE), (dict(dtype=2), DTYPE), (dict(dtype=5), DTYPE), (dict(y_dtype=2), DTYPE), (dict(y_dtype=4), DTYPE),
            (dict(n_experts=0), SHAPE), (dict(n_experts=513), SHAPE), (dict(top_k=0), SHAPE), (dict(top_k=17), SHAPE), (dict(rows=-1), SHAPE),
            (dict(rows=(1 << 24) + 1), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 24) + 1), SHAPE), (dict(N=0), SHAPE),
            (dict(N=65544), SHAPE), (dict(K=0), SHAPE), (dict(K=65544), SHAPE), (dict(K=100), SHAPE), (dict(rows=1 << 24, N=65536), SHAPE),
            (dict(rows=1 << 24, K=65536), SHAPE), (dict(n_experts=512, N=65536, K=65536), SHAPE)]


@pytest.mark.parametrize("bad,status", BAD_DIMS)
def test_sizes_are_refused(bad, status):
    d = dims(**bad)
    big = dict(ldy=1 << 17, ldx=1 << 17)
    assert forward(d, **big) == status
    assert dx(d, lddx=1 << 17, lddy=1 << 17) == status
    assert dw(d, lddy=1 << 17, ldx=1 << 17) == status
    assert B.lib().ds4moe_grouped_workspace_bytes(d) == 0


def test_arguments_are_refused():
    assert forward(ctypes.POINTER(B.GroupedDims)()) == NULL
    for n in ("y", "x", "w", "offsets"):
        assert forward(**{n: None}) == NULL
    for n in ("dx", "dy", "w", "offsets"):
        assert dx(**{n: None}) == NULL
    for n in ("dw", "dy", "x", "offsets"):
        assert dw(**{n: None}) == NULL
    for n in ("y", "x", "w"):
        assert forward(**{n: A + 8}) == ALIGN
    for n in ("dx", "dy", "w"):
        assert dx(**{n: A + 8}) == ALIGN
    for n in ("dw", "dy", "x"):
        assert dw(**{n: A + 8}) == ALIGN
    for f in (forward, dx, dw):
        assert f(offsets=A + 2) == ALIGN and f(perm=A + 2) == ALIGN
    assert [forward(ldy=63), forward(ldx=127), forward(ldx=132), forward(ldx=(1 << 40) + 8), forward(ldy=(1 << 40) + 8)] == [SHAPE] * 5
    assert [dx(lddx=127), dx(lddy=63), dx(lddy=68), dw(lddy=68), dw(ldx=132)] == [SHAPE] * 5
    assert [forward(perm=None), dw(perm=None), dx(perm=None), dx(dims(rows=9), perm=None)] == [SHAPE] * 4
    # scales with 8-bit integers and only with them
    i8 = dims(dtype=B.DS4MOE_I8)
    assert [forward(i8), forward(i8, xs=A), forward(i8, ws=A), forward(xs=A), forward(ws=A)] == [NULL] * 5
    assert forward(i8, xs=A + 2, ws=A) == ALIGN and forward(dims(dtype=B.DS4MOE_I8, K=120), xs=A, ws=A) == SHAPE
    assert dx(i8) == UNSUP and dw(i8) == UNSUP
    assert [dx(dims(N=60), lddy=64), dw(dims(N=60), lddy=64)] == [SHAPE] * 2
    # workspace: only with a permutation
    need = B.lib().ds4moe_grouped_workspace_bytes(dims())
    assert need >= 4 * 20 * 128 + 4 * 20
    assert [dx(ws=None), dx(n=need - 1), dx(ws=A + 16)] == [WS, WS, ALIGN]
    # nothing to do
    assert forward(dims(rows=0), y=None, x=None, w=None, offsets=None, perm=None) == B.DS4MOE_OK
    assert dx(dims(rows=0, tokens=0), dx=None, dy=None, w=None, offsets=None, perm=None) == B.DS4MOE_OK


def test_int8_arguments_are_refused():
    L = B.lib()
    quant = lambda codes=A, scales=A, src=A, t=0, rows=3, cols=40, ld=40: L.ds4moe_int8_quantize(codes, scales, src, t, rows, cols, ld, None)
    back = lambda dst=A, t=0, ld=40, codes=A, scales=A, rows=3, cols=40: L.ds4moe_int8_dequantize(dst, t, ld, codes, scales, rows, cols, None)
    for f in (quant, back):
        assert [f(t=2), f(t=4), f(t=-1)] == [DTYPE] * 3
        assert [f(rows=-1), f(cols=-1), f(cols=1 << 31, ld=1 << 31), f(ld=39), f(rows=(1 << 40) + 1)] == [SHAPE] * 5
        assert [f(codes=None), f(scales=None), f(codes=A + 8), f(scales=A + 2)] == [NULL, NULL, ALIGN, ALIGN]
        assert f(rows=0, codes=None) == f(cols=0, codes=None) == B.DS4MOE_OK
    assert [quant(src=None), quant(src=A + 2), back(dst=None), back(dst=A + 1, t=1)] == [NULL, ALIGN, NULL, ALIGN]
    ws = L.ds4moe_int8_workspace_bytes

    def mul(y=A, yt=1, ldy=64, a=A, sa=A, at=4, lda=32, w=A, sw=A, M=5, N=64, K=32, space=A, n=1 << 30):
        return L.ds4moe_int8_matmul(y, yt, ldy, a, sa, at, lda, w, sw, M, N, K, space, n, None)
    assert [mul(yt=2), mul(yt=4), mul(at=2), mul(at=5)] == [DTYPE] * 4
    assert [mul(M=-1), mul(N=-1), mul(M=(1 << 24) + 1, lda=64), mul(K=0), mul(K=131072, lda=131072), mul(K=24, lda=32), mul(lda=40), mul(lda=16),
            mul(ldy=63), mul(M=1 << 20, N=1 << 20, ldy=1 << 20)] == [SHAPE] * 10
    assert [mul(y=None), mul(a=None), mul(w=None), mul(sw=None), mul(sa=None), mul(at=1)] == [NULL] * 6
    assert [mul(y=A + 8), mul(a=A + 8), mul(w=A + 8), mul(sa=A + 1), mul(sw=A + 1), mul(at=1, sa=None, a=A + 1)] == [ALIGN] * 6
    real = dict(at=1, sa=None, K=31, lda=31)
    need = ws(5, 31, 1)
    assert need >= 5 * 32 + 20 and [mul(**real, space=None), mul(**real, n=need - 1), mul(**real, space=A + 16)] == [WS, WS, ALIGN]
    assert mul(M=0, y=None) == mul(N=0, ldy=0, y=None) == B.DS4MOE_OK
    assert [ws(-1, 32, 1), ws(1, 0, 1), ws(1, 131072, 1), ws(1, 32, 2)] == [0] * 4 and ws(1 << 20, 32, 4) == 256
    assert all(ws(m, 999, 1) <= ws(m + 1, 999, 1) for m in range(200))


def grouped(x=None, w=None, o=None, p="perm", k=2, **kw):
    return q.grouped_matmul(x or Tensor((10, 128), BF16), w or Tensor((4, 64, 128), BF16), o or Tensor((5,), I32),
                            Tensor((20,), I32) if p == "perm" else p, k, **kw)


def backward(dy=None, x=None, w=None, o=None, p="perm", k=2, **kw):
    return q.grouped_matmul_backward(dy or Tensor((20, 64), BF16), x or Tensor((10, 128), BF16), w or Tensor((4, 64, 128), BF16),
                                     o or Tensor((5,), I32), Tensor((20,), I32) if p == "perm" else p, k, **kw)


def test_entry_points_refuse():
    x8, w8 = Tensor((10, 128), I8), Tensor((4, 64, 128), I8)
    scales = dict(x_scales=Tensor((10,), F32), w_scales=Tensor((4, 64), F32))
    calls = {
        "columns": [lambda: grouped(Tensor((10, 120), BF16)), lambda: backward(x=Tensor((10, 120), BF16)),
                    lambda: q.int8_matmul(Tensor((3, 40), BF16), Tensor((8, 64), I8), Tensor((8,), F32)),
                    lambda: q.int8_matmul(Tensor((3, 40), I8), Tensor((8, 48), I8), Tensor((8,), F32), Tensor((3,), F32))],
        "offsets": [lambda: grouped(o=Tensor((4,), I32)), lambda: grouped(o=Tensor((5,), torch.int64))],
        "perm": [lambda: grouped(p=Tensor((20,), torch.int64)), lambda: grouped(p=Tensor((10, 2), I32))],
        "without a permutation": [lambda: grouped(p=None)],
        "w: contiguous": [lambda: grouped(w=Tensor((4, 64, 128), F16)), lambda: grouped(w=Tensor((64, 128), BF16)), lambda: grouped(w=w8),
                          lambda: backward(w=w8)],
        "unsupported type": [lambda: backward(Tensor((20, 64), F32)), lambda: backward(x=x8), lambda: grouped(Tensor((10, 128), I32)),
                             lambda: q.int8_quantize(x8), lambda: q.int8_matmul(x8, Tensor((8, 128), I8), Tensor((8,), F32)),
                             lambda: q.int8_matmul(Tensor((3, 128), BF16), Tensor((8, 128), I8), Tensor((8,), F32), Tensor((3,), F32))],
        "dy:": [lambda: backward(Tensor((19, 64), BF16)), lambda: backward(Tensor((20, 64), F16))],
        "multiple of 8": [lambda: backward(Tensor((20, 60), BF16), w=Tensor((4, 60, 128), BF16))],
        "want x_scales": [lambda: grouped(x8, w8), lambda: grouped(x8, w8, x_scales=scales["x_scales"])],
        "without scales": [lambda: grouped(**scales), lambda: grouped(Tensor((10, 128), F32), Tensor((4, 64, 128), F32))],
        "scales: shape": [lambda: grouped(x8, w8, x_scales=Tensor((20,), F32), w_scales=scales["w_scales"]),
                          lambda: grouped(x8, w8, x_scales=scales["x_scales"], w_scales=Tensor((64,), F32)),
                          lambda: q.int8_dequantize(Tensor((3, 32), I8), Tensor((4,), F32))],
        "is wanted, not": [lambda: grouped(y_dtype=I8), lambda: backward(dw_dtype=I32), lambda: q.int8_dequantize(Tensor((3, 32), I8), Tensor((3,), F32), dtype=I8),
                           lambda: q.int8_matmul(Tensor((3, 64), BF16), Tensor((8, 64), I8), Tensor((8,), F32), y_dtype=I8)],
        "blocks of 16": [lambda: q.int8_dequantize(Tensor((3, 40), I8), Tensor((3,), F32)), lambda: q.int8_dequantize(Tensor((3, 48), I8), Tensor((3,), F32), 30),
                         lambda: q.int8_matmul(Tensor((3, 40), BF16), Tensor((8, 40), I8), Tensor((8,), F32))],
        "cuda:1": [lambda: grouped(o=Tensor((5,), I32, 1)), lambda: grouped(p=Tensor((20,), I32, 1)), lambda: grouped(Tensor((10, 128), BF16, 1)),
                   lambda: grouped(x8, w8, x_scales=Tensor((10,), F32, 1), w_scales=scales["w_scales"]),
                   lambda: grouped(x8, w8, x_scales=scales["x_scales"], w_scales=Tensor((4, 64), F32, 1)),
                   lambda: backward(Tensor((20, 64), BF16, 1)), lambda: backward(x=Tensor((10, 128), BF16, 1)), lambda: backward(o=Tensor((5,), I32, 1)),
                   lambda: q.int8_dequantize(Tensor((3, 32), I8), Tensor((3,), F32, 1)),
                   lambda: q.int8_matmul(Tensor((3, 64), BF16, 1), Tensor((8, 64), I8), Tensor((8,), F32)),
                   lambda: q.int8_matmul(Tensor((3, 64), BF16), Tensor((8, 64), I8), Tensor((8,), F32, 1)),
                   lambda: q.int8_matmul(Tensor((3, 64), I8), Tensor((8, 64), I8), Tensor((8,), F32), Tensor((3,), F32, 1))],
    }
    for match, group in calls.items():
        for i, call in enumerate(group):
            with pytest.raises(ValueError, match=match):
                call()
                pytest.fail(f"{match} {i}")


def test_a_gradient_that_would_be_lost_is_refused():
    def asks(shape, dtype):
        t = Tensor(shape, dtype)
        t.requires_grad = True
        return t
    calls = [lambda: grouped(asks((10, 128), BF16)), lambda: grouped(w=asks((4, 64, 128), BF16)), lambda: q.int8_quantize(asks((3, 64), BF16)),
             lambda: q.int8_matmul(asks((3, 64), BF16), Tensor((8, 64), I8), Tensor((8,), F32))]
    for call in calls:
        with pytest.raises(ValueError, match="asks for a gradient"):
            call()
    with torch.no_grad(), pytest.raises(ValueError, match="columns"):
        grouped(asks((10, 120), BF16))
    with pytest.raises(ValueError, match="dy:"):  # the gradient itself may have operands that ask for one
        backward(Tensor((19, 64), BF16), asks((10, 128), BF16), asks((4, 64, 128), BF16))


def test_the_definitions():
    """The 64-bit forms against loops, and against differences."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((7, 21))
    x[3] = 0
    codes, s = R.quantize(x)
    assert codes.shape == (7, 32) and not codes[:, 21:].any() and not codes[3].any() and s[3] == 0
    assert (np.abs(codes[:, :21] * s[:, None].astype(np.float64) - x) <= s[:, None] * (0.5 + 1e-6)).all()
    T, E, k, N, K = 6, 5, 2, 4, 3
    offsets, perm = R.routing(T, E, k, rng, 0.0, unused=(2,))
    assert offsets[2] == offsets[3] and sorted(perm) == list(range(T * k))
    xv, w, dy = rng.standard_normal((T, K)), rng.standard_normal((E, N, K)), rng.standard_normal((T * k, N))
    rows = R.rows_of(perm, k, T, T * k)
    y, _ = R.matmul(xv, w, offsets, rows)
    for p in range(T * k):
        e = np.searchsorted(offsets, p, side="right") - 1
        assert np.allclose(y[p], w[e] @ xv[perm[p] // k])
    dxv, dwv, _, _ = R.backward(dy, xv, w, offsets, rows)
    for i in np.ndindex(T, K):
        d = np.zeros_like(xv)
        d[i] = 1
        assert np.isclose(dxv[i], (R.matmul(d, w, offsets, rows)[0] * dy).sum())
    for i in np.ndindex(E, N, K):
        d = np.zeros_like(w)
        d[i] = 1
        assert np.isclose(dwv[i], (R.matmul(xv, d, offsets, rows)[0] * dy).sum())
