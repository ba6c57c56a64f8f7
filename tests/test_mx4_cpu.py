"""The expert gate and the 4-bit microscaled operators without a GPU: what
they refuse, on the host and before anything is launched (fake, never
dereferenced addresses), and the 64-bit implementations that the GPU tests go
by, against hand-made values."""
import ctypes

import numpy as np
import pytest
import torch

import mx4_ref as R
import quantized_routed_moe_router_amd as q
from quantized_routed_moe_router_amd import binding as B

P = ctypes.c_void_p


def p(n):
    return P(n)


# ------------------------------------------------------------------ gate
def gate_call(g=None, logits=p(256), ld=256, bias=None, T=4, out=None, ws=p(512), ws_bytes=1 << 30):
    g = g if g is not None else gating()
    out = out if out is not None else routing()
    return B.lib().ds4moe_gate(ctypes.byref(g), logits, ld, bias, T, ctypes.byref(out), ws, ws_bytes, None)


def gating(E=256, k=8, G=1, top=1, rank=1, score=1, renorm=1, dtype=0, scale=1.0):
    return B.Gating(E, k, G, top, rank, score, renorm, dtype, scale)


def routing(**kw):
    f = dict(topk_idx=64, topk_w=64, counts=64, offsets=64, perm=64)
    f.update(kw)
    return B.make_routing(**f)


@pytest.mark.parametrize("bad,status", [
    (dict(E=0), 2), (dict(E=513), 2), (dict(k=0), 2), (dict(k=17), 2), (dict(E=4), 2), (dict(G=3), 2), (dict(G=0), 2), (dict(G=128), 2),
    (dict(G=8, top=0), 2), (dict(G=8, top=9), 2), (dict(G=64, top=1), 2), (dict(rank=0), 2), (dict(rank=3), 2), (dict(score=3), 2),
    (dict(score=-1), 2), (dict(renorm=2), 2), (dict(dtype=2), 3), (dict(scale=float("nan")), 2), (dict(scale=float("inf")), 2)])
def test_bad_gates_are_refused(bad, status):
    g = gating(**bad)
    assert gate_call(g, T=0) == status
    assert B.ds4moe_gate_workspace_bytes(g, 1) == 0
    assert B.lib().ds4moe_gate_backward(ctypes.byref(g), p(64), 600, None, p(64), p(64), 0, p(64), 600, None) == status


def test_gate_argument_errors():
    assert gate_call(T=0) == 0
    assert gate_call(T=-1) == 2 and gate_call(T=(1 << 20) + 1) == 2 and gate_call(ld=255) == 2
    assert gate_call(logits=None) == 1 and gate_call(logits=p(2)) == 4 and gate_call(bias=p(2)) == 4
    assert gate_call(out=routing(perm=None)) == 1 and gate_call(out=routing(counts=None)) == 1
    assert gate_call(out=routing(offsets=None)) == 1 and gate_call(out=routing(logits=64)) == 6
    for n in ("topk_idx", "topk_w", "counts", "offsets", "perm"):
        assert gate_call(out=routing(**{n: 66})) == 4
    assert gate_call(ws=None) == 5 and gate_call(ws=p(128)) == 4
    n = B.ds4moe_gate_workspace_bytes(gating(), 4)
    assert n > 0 and gate_call(ws_bytes=n - 1) == 5
    L, g = B.lib(), gating()
    assert L.ds4moe_gate(None, p(64), 256, None, 4, ctypes.byref(routing()), p(256), 1 << 30, None) == 1
    assert L.ds4moe_gate(ctypes.byref(g), p(64), 256, None, 4, None, p(256), 1 << 30, None) == 1

    def back(logits=p(64), ld=256, bias=None, idx=p(64), dw=p(64), T=4, dl=p(64), ldd=256):
        return L.ds4moe_gate_backward(ctypes.byref(g), logits, ld, bias, idx, dw, T, dl, ldd, None)

    assert back(T=0) == 0 and back(T=-1) == 2 and back(ld=8) == 2 and back(ldd=255) == 2
    assert back(logits=None) == back(idx=None) == back(dw=None) == back(dl=None) == 1
    assert back(logits=p(2)) == back(idx=p(2)) == back(dw=p(2)) == back(dl=p(2)) == back(bias=p(2)) == 4


def test_gate_workspace_grows_with_the_tokens():
    for g in (gating(), gating(E=512, k=16), gating(E=8, k=2)):
        sizes = [B.ds4moe_gate_workspace_bytes(g, T) for T in (0, 1, 63, 64, 65, 4095, 4096, 4097, 8192, 8193, 16385, 1 << 20)]
        assert all(sizes) and sizes == sorted(sizes)
    assert B.ds4moe_gate_workspace_bytes(gating(), -1) == 0 == B.ds4moe_gate_workspace_bytes(gating(), (1 << 20) + 1)
    assert B.lib().ds4moe_gate_workspace_bytes(None, 4) == 0


# ------------------------------------------------------------------ 4-bit values
def test_quantize_argument_errors():
    L = B.lib()

    def quant(c=p(64), s=p(64), x=p(64), d=0, rows=4, cols=64, ld=64):
        return L.ds4moe_mx4_quantize(c, s, x, d, rows, cols, ld, None)

    def dequant(x=p(64), d=0, ld=64, c=p(64), s=p(64), rows=4, cols=64):
        return L.ds4moe_mx4_dequantize(x, d, ld, c, s, rows, cols, None)

    for f in (quant, dequant):
        assert f(rows=0) == 0 and f(cols=0) == 0
        assert f(rows=-1) == f(cols=-1) == f(ld=63) == f(cols=1 << 31, ld=1 << 31) == 2
        assert f(d=2) == 3
        assert f(c=None) == f(s=None) == f(x=None) == 1
        assert f(c=p(68)) == 4 and f(x=p(66)) == 4 and f(x=p(65), d=1) == 4


def test_matmul_argument_errors():
    L = B.lib()

    def mm(y=p(64), yd=0, ldy=48, a=p(64), sa=None, ad=1, lda=64, w=p(64), sw=p(64), M=4, N=48, K=64):
        return L.ds4moe_mx4_matmul(y, yd, ldy, a, sa, ad, lda, w, sw, M, N, K, None)

    assert mm(M=0) == 0 and mm(N=0) == 0
    assert mm(M=-1) == mm(N=-1) == mm(K=0) == mm(K=33) == mm(K=1 << 25) == mm(M=1 << 25) == mm(ldy=47) == 2
    assert mm(lda=63) == mm(lda=68) == mm(lda=56) == 2 and mm(ad=2, sa=p(64), lda=72) == 2
    assert mm(yd=2) == mm(ad=0) == mm(ad=3) == 3
    assert mm(y=None) == mm(a=None) == mm(w=None) == mm(sw=None) == mm(sa=p(64)) == mm(ad=2) == 1
    assert mm(y=p(72)) == mm(a=p(72)) == mm(w=p(72)) == 4


@pytest.mark.parametrize("bad,status", [
    (dict(H=0), 2), (dict(H=48), 2), (dict(H=65568), 2), (dict(I=16), 2), (dict(I=65568), 2), (dict(E=0), 2), (dict(E=513), 2),
    (dict(k=0), 2), (dict(k=17, E=32), 2), (dict(k=9, E=8), 2), (dict(y=2), 3)])
def test_bad_experts_are_refused(bad, status):
    d = dict(H=64, I=32, E=8, k=2, y=1)
    d.update(bad)
    dims = B.make_mx4_dims(d["H"], d["I"], d["E"], d["k"], d["y"])
    assert B.ds4moe_mx4_workspace_bytes(dims, 1) == 0
    w = B.make_mx4_weights(*[64] * 6)
    assert B.lib().ds4moe_mx4_experts(ctypes.byref(dims), ctypes.byref(w), p(64), 65568, 0, ctypes.byref(routing()), p(64), p(256),
                                      1 << 40, None) == status


def test_experts_argument_errors():
    dims, L = B.make_mx4_dims(64, 32, 8, 2), B.lib()

    def ex(w=None, x=p(64), ldx=64, T=4, r=None, y=p(64), ws=p(256), n=1 << 40):
        w, r = w or B.make_mx4_weights(*[64] * 6), r or routing()
        return L.ds4moe_mx4_experts(ctypes.byref(dims), ctypes.byref(w), x, ldx, T, ctypes.byref(r), y, ws, n, None)

    assert ex(T=0) == 0 and ex(T=-1) == ex(ldx=63) == ex(ldx=68) == ex(T=(1 << 20) + 1) == 2
    for i in range(6):
        a = [64] * 6
        a[i] = None
        assert ex(w=B.make_mx4_weights(*a)) == 1
        if i % 2 == 0:
            a[i] = 72
            assert ex(w=B.make_mx4_weights(*a)) == 4
    for n in ("topk_idx", "topk_w", "counts", "offsets", "perm"):
        assert ex(r=routing(**{n: None})) == 1 and ex(r=routing(**{n: 66})) == 4
    assert ex(x=None) == ex(y=None) == 1 and ex(x=p(72)) == ex(y=p(72)) == ex(ws=p(128)) == 4
    assert ex(ws=None) == 5 and ex(n=B.ds4moe_mx4_workspace_bytes(dims, 4) - 1) == 5
    sizes = [B.ds4moe_mx4_workspace_bytes(dims, T) for T in (0, 1, 16, 17, 64, 65, 1000, 1 << 20)]
    assert all(sizes) and sizes == sorted(sizes)
    assert L.ds4moe_mx4_experts(ctypes.byref(dims), None, p(64), 64, 4, ctypes.byref(routing()), p(64), p(256), 1 << 40, None) == 1
    assert L.ds4moe_mx4_experts(None, None, p(64), 64, 4, None, p(64), p(256), 1 << 40, None) == 1


def test_python_entry_points_refuse_what_does_not_fit():
    x = torch.zeros(4, 64)
    for call in (lambda: q.Gate(8, 9), lambda: q.Gate(8, 2, "relu"), lambda: q.Gate(9, 2, n_groups=2), lambda: q.Gate(8, 2).forward(x),
                 lambda: q.mx4_quantize(x), lambda: q.mx4_dequantize(x, x), lambda: q.mx4_matmul(x, x, x),
                 lambda: q.Mx4Experts(48, 32, 8, 2, (x, x), (x, x), (x, x)),
                 lambda: q.Mx4Experts(64, 32, 8, 2, (x, x), (x, x), (x, x), y_dtype=torch.float16)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the plain implementations
def test_reference_quantiser_on_hand_made_blocks():
    x = np.zeros((1, 64))
    x[0, :8] = [4.0, -0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]     # scale 1; every midpoint goes to its even neighbour
    x[0, 32:35] = [7.9, 0.76, -6.1]
    c, s = R.quantize(x)
    assert s.tolist() == [[127, 127]]
    v = R.values(c, s)[0]
    assert v[:8].tolist() == [4.0, -0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0] and v[32:35].tolist() == [6.0, 1.0, -6.0]
    assert c[0, :4].tolist() == [0x86, 0x22, 0x44, 0x66]
    assert R.quantize(np.full((1, 32), 3.0))[1][0, 0] == 126 and R.quantize(np.zeros((1, 5)))[1][0, 0] == 0
    assert R.quantize(np.array([[np.inf] + [1.0] * 31]))[1][0, 0] == 255


def test_reference_gate_on_hand_made_rows():
    l = np.array([[0.0, 2.0, 1.0, 3.0]])
    idx, w, _ = R.gate(l, None, 2, "softmax")
    assert idx.tolist() == [[3, 1]]
    np.testing.assert_allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))]], rtol=1e-14)
    idx, w, _ = R.gate(l, np.array([1.0, 0, 0, 0]), 2, "sigmoid", renorm=False, scale=2.0)
    assert idx.tolist() == [[0, 3]]
    np.testing.assert_allclose(w, [[1.0, 2 / (1 + np.exp(-3))]], rtol=1e-14)
    assert R.gate(l, None, 2, "sigmoid", 2, 1, 1)[0].tolist() == [[3, 2]]
    assert R.gate(np.array([[5.0, -5, 3, 3]]), None, 2, "sigmoid", 2, 1, 2)[0].tolist() == [[2, 3]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(0)
    l, dw, h = rng.standard_normal((3, 8)), rng.standard_normal((3, 3)), 1e-6
    idx = R.gate(l, None, 3, score, renorm=renorm)[0]
    g = R.gate_gradient(l, None, idx, dw, score, renorm, 2.0)

    def f(x):
        s = np.take_along_axis(R.scores(x, score), idx, axis=1)
        return (2.0 * (s / s.sum(axis=1, keepdims=True) if renorm else s) * dw).sum()

    for t in range(3):
        for e in range(8):
            d = np.zeros_like(l)
            d[t, e] = h
            assert abs(g[t, e] - (f(l + d) - f(l - d)) / (2 * h)) < 1e-8


def test_reference_experts_of_one_expert_are_a_dense_ffn():
    rng = np.random.default_rng(1)
    g, u, d = rng.standard_normal((1, 6, 4)), rng.standard_normal((1, 6, 4)), rng.standard_normal((1, 4, 6))
    x = rng.standard_normal((5, 4))
    y = R.experts(x, np.zeros((5, 1), int), np.ones((5, 1)), g, u, d)
    z = torch.from_numpy(x @ g[0].T)
    want = (torch.nn.functional.silu(z).numpy() * (x @ u[0].T)) @ d[0].T
    np.testing.assert_allclose(y, want, rtol=1e-12)
