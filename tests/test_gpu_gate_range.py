"""The expert gate over the rest of its range: chosen logits far apart, keys far below 1, gradients held element by element.

Weights: 3e-6 relative as in test_gpu_gate, and the rounding of the difference of two logits, which the exponential passes
on: half an ulp, 2^-24 of the difference.  Below 2^-126 fp32 holds a multiple of 2^-149.
"""
import numpy as np
import pytest
import torch

import mx4_ref as R
from test_gpu_gate import DT, TOL, _q, make

pytestmark = pytest.mark.gpu

TINY = 2.0**-126
SCORES = ("sigmoid", "softmax", "sqrt_softplus")

# every expert chosen: the largest above, near and far below 0, the others up to the end of fp32 below it
APART = np.array([
    [-59.0, -100.0, -110.0, -59.5], [0.0, -95.0, -110.0, -150.0], [-10.0, -120.25, -140.0, -97.0], [30.0, -60.0, -70.5, -57.0],
    [-61.0, -100.0, -110.0, -140.0], [-17.5, -18.0, -16.5, -104.0], [-1.0, -16.9, -17.1, -88.0], [-59.9, -89.0, -87.0, -130.75],
    [5.0, -86.5, -87.5, -90.0], [-300.0, -330.0, -380.0, -301.0], [88.0, 0.0, -1.0, -40.0], [-40.0, -200.0, -210.0, -41.0]],
    np.float32)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("use_bias", [True, False])
def test_weights_of_logits_far_apart(score, use_bias):
    q = _q()
    l = np.concatenate([APART, APART[:, ::-1]])
    bias = np.array([0.5, 0.25, 0.125, 0.0], np.float32) if use_bias else None
    out = q.Gate(4, 4, score, scale=2.5).forward(torch.from_numpy(l.copy()).cuda(), None if bias is None else torch.from_numpy(bias).cuda())
    gi, gw = out["topk_idx"].cpu().numpy(), out["topk_w"].double().cpu().numpy()
    assert (np.sort(gi, axis=1) == np.arange(4)).all()
    x = np.take_along_axis(l.astype(np.float64), gi.astype(np.int64), axis=1)
    s = R.log_scores(x, score)
    e = np.exp(s - s.max(axis=1, keepdims=True))
    want = 2.5 * e / e.sum(axis=1, keepdims=True)
    bound = (TOL + 2.0**-24 * np.abs(x - x.max(axis=1, keepdims=True))) * want + 2.5 * TINY
    assert (np.abs(gw - want) <= bound).all(), float((np.abs(gw - want) / bound).max())


# ------------------------------------------------------------------ gradient
def gradient(l, bias, idx, dw, score, renorm, scale):
    """d logits in 64 bits, and the absolute values of what each element is summed from.  Slopes are taken of the scores'
    logarithms, so that nothing cancels where a score is near 0 or 1, and logits that have no part come out as 0."""
    l = R.clean(l)
    T, E = l.shape
    with np.errstate(all="ignore"):
        slope = {"softmax": np.ones_like(l), "sigmoid": 1 / (1 + np.exp(l)),
                 "sqrt_softplus": np.where(l < -40, 0.5, 0.5 / (1 + np.exp(-l)) / np.logaddexp(0.0, l))}[score]
    live = np.take_along_axis(np.isfinite(l) & (np.ones(E, bool) if bias is None else bias > -np.inf), idx, axis=1)
    d = np.zeros((T, E))
    np.put_along_axis(d, idx, np.where(live, dw.astype(np.float64), 0.0), axis=1)
    s = R.scores(l, score)
    if renorm:
        x = np.where(live, R.log_scores(np.take_along_axis(l, idx, axis=1), score), -np.inf)
        e = np.exp(x - np.where(live.any(axis=1), x.max(axis=1), 0.0)[:, None])
        s = np.zeros((T, E))
        np.put_along_axis(s, idx, e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300), axis=1)
    if renorm or score == "softmax":
        g, made = s * slope * (d - (d * s).sum(axis=1, keepdims=True)), s * slope * (np.abs(d) + (np.abs(d) * s).sum(axis=1, keepdims=True))
    else:
        g = s * slope * d
        made = np.abs(g)
    return scale * g, scale * made


def gradient_bound(l, made, scale):
    """1e-5 of the absolute values of what each element is summed from: sums of up to 512 terms in a tree (14 roundings),
    exponentials and quotients of a few ulp, a score good to 3e-6; and the rounding of a difference of two logits."""
    live = np.isfinite(R.clean(l))
    far = np.where(live, R.clean(l), -np.inf).max(axis=1, keepdims=True) - np.where(live, R.clean(l), np.inf)
    return (1e-5 + 2.0**-24 * np.where(live, far, 0.0)) * made + scale * TINY


def check_gradient(t, l, bias, k, score, renorm, scale, seed):
    q = _q()
    T, E = l.shape
    dw = np.random.default_rng(seed).standard_normal((T, k)).astype(np.float32)
    g = q.Gate(E, k, score, renorm=renorm, scale=scale)
    b = None if bias is None else torch.from_numpy(bias).cuda()
    idx = g.forward(t, b)["topk_idx"]
    dl = g.backward(t, idx, torch.from_numpy(dw).cuda(), b)
    ii = idx.cpu().numpy().astype(np.int64)
    ref, made = gradient(l, bias, ii, dw, score, renorm, scale)
    bound = gradient_bound(l, made, scale) + (2.0**-8 * np.abs(ref) if t.dtype == torch.bfloat16 else 0)
    err = np.abs(dl.double().cpu().numpy() - ref)
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_logits_far_apart(score, renorm):
    check_gradient(torch.from_numpy(APART).cuda(), APART, None, 4, score, renorm, 2.5, 1)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,use_bias", [(1, 256, 8, True), (400, 256, 8, False), (9, 130, 16, True), (3, 512, 3, False), (300, 96, 4, True),
                                            (5, 60, 4, False)])
def test_every_element_of_the_gradient(score, renorm, dtype, T, E, k, use_bias):
    """The small gradients of the logits that were not chosen among them, each to 1e-5 of what it is made of."""
    t, l, bias = make(T, E, 3 * T + E, dtype, pad=3)
    check_gradient(t, l, bias if use_bias else None, k, score, renorm, 2.5, E)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("renorm", [True, False])
def test_every_element_of_the_gradient_of_low_and_high_rows(score, renorm):
    rng = np.random.default_rng(2)
    l = (rng.standard_normal((40, 64)) + rng.choice([-60.0, -30.0, -17.0, 17.0, 60.0], (40, 1))).astype(np.float32)
    check_gradient(torch.from_numpy(l).cuda(), l, None, 6, score, renorm, 1.0, 5)


# ------------------------------------------------------------------ selection
@pytest.mark.parametrize("score", SCORES)
def test_selection_tells_keys_apart_that_differ_by_a_millionth(score):
    """Two keys of which one is a score far below 1 and the other a bias, 1e-6 of it above or below: eight ulp, where the
    score's exponential, sum and quotient are off by an ulp each."""
    q = _q()
    g = q.Gate(3, 2, score)
    wrong = []
    for x in np.linspace(-84.0, -18.0, 60).astype(np.float32):
        s = float(R.scores(np.array([[0.0, float(x), -400.0]]), score)[0, 1])
        for sign in (1, -1):
            bias = np.float32(s * (1 + sign * 1e-6))
            t = torch.tensor([[0.0, float(x), -400.0]], device="cuda")
            b = torch.tensor([0.0, 0.0, float(bias)], device="cuda")
            first, second = g.forward(t, b)["topk_idx"][0].tolist()
            assert first == 0
            if second != (2 if float(bias) > s else 1):
                wrong.append((float(x), sign))
    assert not wrong, (len(wrong), wrong[:8])
