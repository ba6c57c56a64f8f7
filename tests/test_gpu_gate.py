"""The expert gate on the GPU against its 64-bit formulas.

Weights: every step is fp32 (exponentials to an ulp or two, differences of
logits of up to 16, a sum of at most 16 scores, one quotient, one product):
(16 + 8) * 2 * 2^-24 < 3e-6 relative, which is also the bound of the sqrt(softplus)
form.  Choices hang on fp32 keys with a bias (a score's error over the key):
rows with two keys nearer than 1e-5 are left out of the comparison of indices.
Gradients: sums of k products of such values, 1e-5 of the row's largest
magnitude of what is summed; bf16 adds one rounding, 2^-8.
"""
import numpy as np
import pytest
import torch

import mx4_ref as R

pytestmark = pytest.mark.gpu

TOL = 3e-6
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _q():
    import quantized_routed_moe_router_amd as q
    return q


def make(T, E, seed, dtype, pad=0, spread=1.3):
    rng = np.random.default_rng(seed)
    l = (spread * rng.standard_normal((T, E + pad))).astype(np.float32)
    t = torch.from_numpy(l).cuda().to(DT[dtype])[:, :E]
    return t, t.float().cpu().numpy().astype(np.float64), (0.1 * rng.standard_normal(E)).astype(np.float32)


def check(out, ref, E, label, kept=None):
    idx, w, gaps = ref
    sure = gaps > 1e-5
    assert sure.mean() > 0.8
    gi, gw = out["topk_idx"].cpu().numpy(), out["topk_w"].cpu().numpy()
    assert np.array_equal(gi[sure], idx[sure]), label
    np.testing.assert_allclose(gw[sure], w[sure], rtol=TOL, atol=1e-37, err_msg=label)
    counts, offsets, perm = R.permutation(gi, E)
    assert np.array_equal(out["counts"].cpu().numpy(), counts), label
    assert np.array_equal(out["offsets"].cpu().numpy(), offsets), label
    assert np.array_equal(out["perm"].cpu().numpy(), perm), label


@pytest.mark.parametrize("score", ["sigmoid", "softmax", "sqrt_softplus"])
@pytest.mark.parametrize("T,E,k,G,top,rank", [
    (1, 256, 8, 8, 4, 2), (3, 8, 2, 1, 1, 1), (17, 60, 4, 1, 1, 1), (64, 64, 6, 4, 2, 1), (65, 128, 8, 1, 1, 2),
    (130, 160, 6, 8, 3, 2), (33, 384, 8, 1, 1, 1), (40, 512, 16, 16, 4, 2), (5, 1, 1, 1, 1, 1), (9, 63, 16, 3, 2, 1),
    (6, 64, 3, 64, 5, 2), (300, 256, 8, 2, 1, 1), (7, 65, 5, 13, 4, 2)])
def test_gate_matches_the_formulas(score, T, E, k, G, top, rank):
    q = _q()
    for dtype in ("f32", "bf16"):
        for use_bias, renorm, scale in ((True, True, 2.5), (False, False, 1.0), (False, True, 1.0), (True, False, 0.5)):
            t, l, bias = make(T, E, 7 * T + E, dtype)
            g = q.Gate(E, k, score, G, top, rank, renorm, scale)
            out = g.forward(t, torch.from_numpy(bias).cuda() if use_bias else None)
            ref = R.gate(l, bias if use_bias else None, k, score, G, top, rank, renorm, scale)
            check(out, ref, E, f"{score} {dtype} bias={use_bias} renorm={renorm}")


@pytest.mark.parametrize("T", [1000, 4097, 20000])
def test_gate_many_tokens(T):
    """Several chunk sizes of the permutation, the last chunk not full."""
    q = _q()
    E, k = (96, 4) if T < 10000 else (24, 3)
    t, l, bias = make(T, E, T, "f32")
    out = q.Gate(E, k, "sigmoid", 4, 2, 2).forward(t, torch.from_numpy(bias).cuda())
    check(out, R.gate(l, bias, k, "sigmoid", 4, 2, 2), E, str(T))


def test_gate_rows_apart_and_repeatable():
    q = _q()
    t, l, bias = make(50, 61, 5, "bf16", pad=8)
    assert t.stride(0) == 69
    g, b = q.Gate(61, 5, "softmax", renorm=False), torch.from_numpy(bias).cuda()
    a, c = g.forward(t, b), g.forward(t.contiguous(), b)
    check(a, R.gate(l, bias, 5, "softmax", renorm=False), 61, "rows apart")
    for n in a:
        assert torch.equal(a[n], c[n])
        assert torch.equal(a[n], g.forward(t, b)[n])


def test_ties_go_to_the_lower_expert_and_group():
    q = _q()
    l = torch.zeros(3, 64, device="cuda")
    l[1, 40:44] = 1.0
    for score in ("sigmoid", "softmax", "sqrt_softplus"):
        out = q.Gate(64, 6, score, 8, 2, 2).forward(l, torch.zeros(64, device="cuda"))
        assert out["topk_idx"].tolist() == [[0, 1, 2, 3, 4, 5], [40, 41, 42, 43, 0, 1], [0, 1, 2, 3, 4, 5]]
        np.testing.assert_allclose(out["topk_w"][0].cpu().numpy(), 1 / 6, rtol=TOL)


@pytest.mark.parametrize("score", ["sigmoid", "softmax", "sqrt_softplus"])
@pytest.mark.parametrize("G,top,rank", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
@pytest.mark.parametrize("renorm", [True, False])
def test_masks_infinities_and_extremes(score, G, top, rank, renorm):
    """Rows with every expert masked, fewer than k left, one left in a group, NaN, the largest and lowest values, +inf,
    and biases that mask: indices stay valid and distinct, weights finite, masked experts at weight 0."""
    q = _q()
    E, k = 16, 4
    rng = np.random.default_rng(3)
    l = rng.standard_normal((12, E)).astype(np.float32)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, :] = -np.inf
    l[2, 5] = 0.3
    l[3, ::2] = np.nan
    l[4, 3] = np.inf
    l[5, [2, 9]] = np.inf
    l[6] = -R.FMAX
    l[7] = R.FMAX
    l[8, :] = -R.FMAX
    l[8, 11] = 1.0
    l[9] = -100.0
    l[10, 8:] = -np.inf
    l[11] = np.inf
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    masks = bias.copy()
    masks[[1, 6]] = -np.inf
    masks[12] = np.nan
    for b in (None, bias, masks):
        out = q.Gate(E, k, score, G, top, rank, renorm).forward(
            torch.from_numpy(l).cuda(), None if b is None else torch.from_numpy(b).cuda())
        idx, w, _ = R.gate(l, b, k, score, G, top, rank, renorm)
        gi, gw = out["topk_idx"].cpu().numpy(), out["topk_w"].cpu().numpy()
        assert ((gi >= 0) & (gi < E)).all() and all(len(set(r)) == k for r in gi)
        assert np.isfinite(gw).all()
        skip = [6, 7, 9, 11] if b is not None else []  # scores that meet in one fp32 value: the bias alone orders them
        rows = [t for t in range(12) if t not in skip]
        assert np.array_equal(gi[rows], idx[rows])
        np.testing.assert_allclose(gw[rows], w[rows], rtol=TOL, atol=1e-30)
        assert (gw[0] == 0).all() and (gw[1] == 0).all()


def test_outputs_that_are_not_wanted():
    q = _q()
    B = q.binding
    t, l, _ = make(70, 32, 1, "f32")
    ref = R.gate(l, None, 4, "sigmoid")
    g = B.make_gating(32, 4, score=B.SCORE_SIGMOID)
    n = B.ds4moe_gate_workspace_bytes(g, 70)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    w = torch.empty(70, 4, device="cuda")
    B.ds4moe_gate(g, t, 32, None, 70, B.make_routing(topk_w=w), ws, n)
    np.testing.assert_allclose(w.cpu().numpy(), ref[1], rtol=TOL)
    counts, offsets, perm = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (32, 33, 280))
    B.ds4moe_gate(g, t, 32, None, 70, B.make_routing(counts=counts, offsets=offsets, perm=perm), ws, n)
    c, o, p = R.permutation(ref[0], 32)
    assert np.array_equal(counts.cpu().numpy(), c) and np.array_equal(offsets.cpu().numpy(), o)
    assert np.array_equal(perm.cpu().numpy(), p)
    empty = q.Gate(32, 4).forward(t[:0])
    assert empty["topk_idx"].shape == (0, 4) and empty["counts"].sum() == 0


def test_gate_on_another_stream_and_in_a_graph():
    q = _q()
    t, l, bias = make(200, 48, 9, "f32")
    b, g = torch.from_numpy(bias).cuda(), q.Gate(48, 4, "sigmoid", 4, 2, 2)
    want = g.forward(t, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = g.forward(t, b)
    s.synchronize()
    for n in want:
        assert torch.equal(want[n], got[n])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = g.forward(t, b)
    for seed in (9, 10, 11):
        new = make(200, 48, seed, "f32")[0]
        t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        eager = g.forward(new, b)
        for n in held:
            assert torch.equal(held[n], eager[n])


# ------------------------------------------------------------------ gradient
def grad_scale(l, idx, dw, score, renorm, scale):
    """What the gradient's terms are made of, per row: an error of 1e-5 of it is allowed."""
    return scale * np.abs(dw).sum(axis=1, keepdims=True)


@pytest.mark.parametrize("score", ["sigmoid", "softmax", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (5, 60, 4), (9, 130, 16), (3, 512, 3), (6, 1, 1)])
def test_gradient_matches_the_formula(score, renorm, dtype, T, E, k):
    q = _q()
    t, l, bias = make(T, E, 11 * T + E, dtype, pad=3)
    dw = np.random.default_rng(E).standard_normal((T, k)).astype(np.float32)
    g = q.Gate(E, k, score, renorm=renorm, scale=2.5)
    b = torch.from_numpy(bias).cuda()
    idx = g.forward(t, b)["topk_idx"]
    dl = g.backward(t, idx, torch.from_numpy(dw).cuda(), b)
    assert dl.dtype == t.dtype and dl.is_contiguous()
    ref = R.gate_gradient(l, bias, idx.cpu().numpy(), dw, score, renorm, 2.5)
    err = np.abs(dl.float().cpu().numpy() - ref)
    bound = 1e-5 * grad_scale(l, idx, dw, score, renorm, 2.5) + (2.0**-8 * np.abs(ref) if dtype == "bf16" else 0)
    assert (err <= bound).all(), float((err - bound).max())


@pytest.mark.parametrize("score", ["sigmoid", "softmax", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_matches_differences_of_the_gate(score, renorm):
    """Central differences of the gate's own weights, step 2^-6: their error is the weights' 3e-6 over the step and the
    third derivative times its square (below 0.5 * scale * 2^-12 / 6 * k); 1e-3 holds both."""
    q = _q()
    T, E, k, h = 4, 12, 3, 2.0**-6
    rng = np.random.default_rng(0)
    l = np.stack([rng.permutation(E) * 0.25 - 1.5 for _ in range(T)]).astype(np.float32)  # no two nearer than 0.25
    g = q.Gate(E, k, score, renorm=renorm)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    t = torch.from_numpy(l).cuda()
    first = g.forward(t)
    dl = g.backward(t, first["topk_idx"], torch.from_numpy(dw).cuda()).cpu().numpy()
    for e in range(E):
        f = []
        for s in (h, -h):
            m = l.copy()
            m[:, e] += s
            out = g.forward(torch.from_numpy(m).cuda())
            assert torch.equal(out["topk_idx"], first["topk_idx"])
            f.append((out["topk_w"].double().cpu().numpy() * dw).sum(axis=1))
        np.testing.assert_allclose(dl[:, e], (f[0] - f[1]) / (2 * h), atol=1e-3)


@pytest.mark.parametrize("score", ["sigmoid", "softmax", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_masked_and_extreme_rows(score, renorm):
    q = _q()
    E, k = 16, 4
    rng = np.random.default_rng(3)
    l = rng.standard_normal((7, E)).astype(np.float32)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, :] = -np.inf
    l[2, 5] = 0.3
    l[3] = -60.0 + l[3]
    l[4, 2] = np.inf
    l[5] = 60.0 + l[5]
    l[6, 4:] = np.nan
    bias = np.zeros(E, np.float32)
    bias[[3, 7]] = -np.inf
    dw = rng.standard_normal((7, k)).astype(np.float32)
    t, b = torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda()
    g = q.Gate(E, k, score, renorm=renorm)
    idx = g.forward(t, b)["topk_idx"]
    dl = g.backward(t, idx, torch.from_numpy(dw).cuda(), b).cpu().numpy()
    assert np.isfinite(dl).all()
    assert (dl[0] == 0).all() and (dl[1] == 0).all()
    ref = R.gate_gradient(l, bias, idx.cpu().numpy(), dw, score, renorm, 1.0)
    rows = [2, 3, 5, 6]
    assert (np.abs(dl - ref)[rows] <= 1e-5 * np.abs(dw).sum(axis=1, keepdims=True)[rows]).all()


def test_gradient_leaves_out_indices_out_of_range():
    q = _q()
    t, l, _ = make(2, 8, 0, "f32")
    idx = torch.tensor([[1, -1, 9], [0, 1, 2]], dtype=torch.int32, device="cuda")
    dw = torch.ones(2, 3, device="cuda")
    dl = q.Gate(8, 3, "sigmoid", renorm=False).backward(t, idx, dw).cpu().numpy()
    ref = R.gate_gradient(l, None, idx.cpu().numpy(), dw.cpu().numpy(), "sigmoid", False, 1.0)
    assert np.abs(dl - ref).max() <= 3e-5 and np.count_nonzero(dl[0]) == 1
