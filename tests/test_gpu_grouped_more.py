"""Products grouped by expert on the GPU: the largest results, and what the other files do not ask for.  Bounds as in
test_gpu_grouped."""
import numpy as np
import pytest
import torch

import grouped_ref as R
from test_gpu_grouped import _q, case, check, dev, half, host

pytestmark = pytest.mark.gpu


def test_rows_gradients_of_2_to_the_36_values():
    """128 GiB of gradients of rows in order: as many tiles of four waves had more than 2^31 threads."""
    B = _q().binding
    P, K, N = 1 << 20, 65536, 8
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < P * K * 2 + (4 << 30):
        pytest.skip("the card holds less")
    rng = np.random.default_rng(0)
    dv, w = rng.integers(-4, 5, (P, N)) / 4.0, rng.integers(-4, 5, (1, N, K)) / 4.0
    dy, wt = (torch.from_numpy(v).to(torch.bfloat16).cuda() for v in (dv, w))
    dx = torch.empty(P, K, dtype=torch.bfloat16, device="cuda")
    d = B.make_grouped_dims(N, K, 1, 1, P, P)
    B.ds4moe_grouped_dx(d, dx, K, dy, N, wt, dev(np.array([0, P], dtype=np.int32)), None)
    at = np.unique(np.concatenate([[0, 1, P // 2, P - 64, P - 1], rng.integers(0, P, 40)]))
    got = dx[torch.from_numpy(at).cuda()]
    assert np.array_equal(host(got), dv[at] @ w[0])  # sixteenths below 2^8 of them
    for c in range(0, K, 8192):  # no row was left out: the sums of 128 columns of each
        part = dx[:, c:c + 128].float().sum(1)
        assert torch.equal(part, dy.float() @ wt[0, :, c:c + 128].float().sum(1))
    del dx
    torch.cuda.empty_cache()


def routed(T, E, P, k, style, rng):
    """Entries of a permutation that stand several times, and offsets."""
    if style == "tokens":  # the numbers of tokens, each with several experts: k = 1
        flat = rng.integers(0, E, P)
        offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
        perm = np.sort(rng.integers(0, T, P))[np.argsort(flat, kind="stable")]
    elif style == "one":  # all positions of one assignment
        offsets = np.sort(np.concatenate([[0, P], rng.integers(0, P + 1, E - 1)]))
        perm = np.full(P, T * k // 2)
    elif style == "some":  # distinct ones but for a few, and some that name nothing
        offsets = np.sort(np.concatenate([[0, P], rng.integers(0, P + 1, E - 1)]))
        perm = rng.permutation(T * k)[:P]
        perm[rng.integers(0, P, 3)] = perm[rng.integers(0, P, 3)]
        perm[rng.integers(0, P, 2)] = [-1, T * k]
    elif style == "any":
        offsets = np.sort(np.concatenate([[0, P], rng.integers(0, P + 1, E - 1)]))
        perm = rng.integers(0, T * k, P)
    else:  # "padded": positions of no expert at both ends, all of which name assignment 0
        a, b = P // 7, P - P // 5
        offsets = np.sort(np.concatenate([[a, b], rng.integers(a, b + 1, E - 1)]))
        perm = np.concatenate([np.zeros(a, int), rng.permutation(T * k)[:b - a], np.zeros(P - b, int)])
        perm[a + (b - a) // 2] = 0
    return offsets.astype(np.int32), perm.astype(np.int32)


@pytest.mark.parametrize("T,E,P,k,style", [
    (5, 3, 9, 1, "tokens"), (300, 8, 600, 1, "tokens"), (4000, 8, 8000, 1, "tokens"), (1000, 60, 3711, 1, "tokens"), (64, 4, 1023, 1, "tokens"),
    (64, 4, 1024, 1, "tokens"), (64, 4, 1025, 2, "tokens"), (3, 4, 2049, 1, "one"), (7, 2, 5000, 3, "one"), (1, 6, 6, 1, "one"), (700, 5, 1300, 2, "some"),
    (3000, 5, 9000, 3, "some"), (3, 4, 255, 1, "one"), (3, 4, 256, 1, "one"), (3, 4, 257, 1, "one"), (5, 3, 1280, 1, "tokens"), (2, 3, 1500, 3, "any"),
    (40, 8, 300, 8, "any"), (20, 2, 30, 2, "padded"), (900, 6, 1800, 2, "padded"), (5000, 6, 9001, 2, "padded")])
def test_rows_gradient_of_assignments_that_stand_several_times(T, E, P, k, style):
    """Every position of an expert adds to its token's gradient, in an order that is the same every time; those of no expert
    add nothing and take nothing away."""
    q = _q()
    N, K = 24, 2056 if P < 700 else 1000 if P < 1300 else 40
    x, xv, w, wv, _, _ = case(T, E, 1, N, K, "f16")
    rng = np.random.default_rng(P + T)
    offsets, perm = routed(T, E, P, k, style, rng)
    inside = np.zeros(P, dtype=bool)
    inside[offsets[0]:offsets[-1]] = True
    rows = np.where(inside, R.rows_of(perm, k, T, P), -1)
    assert np.unique(perm[rows >= 0]).size < (rows >= 0).sum() or style == "padded"
    dy, dyv = half(0.1 * rng.standard_normal((P, N)), "f16")
    wx, ww, mx, mw = R.backward(dyv, xv, wv, offsets, rows)
    most = int(np.bincount(rows[rows >= 0], minlength=T).max())
    o, p = dev(offsets), dev(perm)
    dx, dw = q.grouped_matmul_backward(dy, x, w, o, p, k)
    check(dx, wx, mx, N + most, "f16")
    check(dw, ww, mw, P, "f16")
    for _ in range(3):
        assert torch.equal(q.grouped_matmul_backward(dy, x, w, o, p, k, need_dw=False)[0], dx)


def test_rows_gradient_by_tokens_numbers_is_that_of_the_gates_permutation():
    """Top-2 routing by the gate's permutation with k = 2, and by tokens' numbers with k = 1: sums of two, which have no order."""
    q = _q()
    T, E, k, N, K = 500, 8, 2, 64, 136
    x, _, w, _, offsets, perm = case(T, E, k, N, K, "bf16")
    dy = half(np.random.default_rng(1).standard_normal((T * k, N)), "bf16")[0]
    a = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), k)
    b = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm // k), 1)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_gradient_in_a_graph_whose_assignments_change():
    """One captured call, replayed on permutations whose assignments are distinct and on others, in turn."""
    q = _q()
    T, E, k, N, K = 400, 4, 2, 40, 72
    x, _, w, _, offsets, perm = case(T, E, k, N, K, "bf16")
    dy = half(np.random.default_rng(1).standard_normal((T * k, N)), "bf16")[0]
    o, p = dev(offsets), dev(perm)
    q.grouped_matmul_backward(dy, x, w, o, p, k, need_dw=False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dx, _ = q.grouped_matmul_backward(dy, x, w, o, p, k, need_dw=False)
    for i in range(6):
        rng = np.random.default_rng(i)
        p.copy_(dev(perm if i % 2 else rng.integers(-2, T * k + 2, T * k).astype(np.int32)))
        g.replay()
        torch.cuda.synchronize()
        got = dx.clone()
        assert torch.equal(got, q.grouped_matmul_backward(dy, x, w, o, p, k, need_dw=False)[0]), i


def test_rows_gradient_of_repeated_assignments_is_the_difference():
    """Central differences of sum(dy * y) along random directions of x, an assignment standing three times."""
    q = _q()
    T, N, K = 4, 16, 32
    x, xv, w, wv, _, _ = case(T, 2, 1, N, K, "f16")
    perm, offsets = np.array([1, 1, 3, 1], dtype=np.int32), np.array([0, 2, 4], dtype=np.int32)
    rows = R.rows_of(perm, 1, T, 4)
    dy, dyv = half(np.random.default_rng(1).standard_normal((4, N)), "f16")
    dx, _ = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), need_dw=False)
    _, _, mx, _ = R.backward(dyv, xv, wv, offsets, rows)
    rng, h = np.random.default_rng(2), 2.0**-10
    for _ in range(4):
        u = rng.standard_normal(xv.shape)
        up, down = (R.matmul(xv + s * h * u, wv, offsets, rows)[0] for s in (1, -1))
        want = ((up - down) * dyv).sum() / (2 * h)  # linear in x: exact but for 64-bit roundings
        assert abs((host(dx) * u).sum() - want) <= (np.abs(u) * (mx * (2.0**-23 * (N + 5) + 2.0**-11) + R.TINY["f16"])).sum()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("E,N,K,P", [(3, 40, 72, 5), (3, 136, 200, 700), (4, 24, 40, 3000), (512, 264, 264, 20000)])
def test_weights_gradient_of_positions_that_name_nothing(kind, E, N, K, P):
    """NaN and infinities of dy where the permutation names no row: padding, which adds nothing."""
    q = _q()
    T, rng = P, np.random.default_rng(P)
    x, _ = half(rng.standard_normal((T, K)), kind)
    w = torch.zeros(E, N, K, dtype=x.dtype, device="cuda")
    offsets = np.sort(np.concatenate([[0, P], rng.integers(0, P + 1, E - 1)])).astype(np.int32)
    perm = rng.permutation(P).astype(np.int32)
    gone = rng.random(P) < 0.2
    gone[[0, P - 1]] = True
    perm[gone] = rng.choice([-1, T, 2**31 - 1, -2**31], gone.sum())
    dv = 0.1 * rng.standard_normal((P, N))
    dy, _ = half(np.where(gone[:, None], 0, dv), kind)
    bad, _ = half(np.where(gone[:, None], rng.choice([np.nan, np.inf, -np.inf], (P, N)), dv), kind)
    want = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm))
    got = q.grouped_matmul_backward(bad, x, w, dev(offsets), dev(perm))
    assert torch.isfinite(want[1]).all() and torch.equal(got[1], want[1]) and torch.equal(got[0], want[0])


@pytest.mark.parametrize("step", [8372128 // 2, 8388608 // 2])
def test_weights_gradient_of_unnamed_positions_far_apart(step):
    """Rows of dy up to 2^32 bytes from the first, and beyond: NaN in those that name nothing, the last among them."""
    q = _q()
    P, N, K = 513, 72, 64
    rng = np.random.default_rng(0)
    ds = torch.full((P * step,), float("nan"), dtype=torch.bfloat16, device="cuda").view(P, step)
    xv, dv = rng.integers(-8, 9, (P, K)) / 4.0, rng.integers(-8, 9, (P, N)) / 4.0
    perm = rng.permutation(P).astype(np.int32)
    gone = rng.random(P) < 0.3
    gone[[0, P - 2, P - 1]] = True
    perm[gone] = -1
    at = torch.from_numpy(np.nonzero(~gone)[0]).cuda()
    ds[at, :N] = torch.from_numpy(dv[~gone]).to(torch.bfloat16).cuda()
    w = torch.zeros(1, N, K, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    _, dw = q.grouped_matmul_backward(ds[:, :N], torch.from_numpy(xv).to(torch.bfloat16).cuda(), w, offsets, dev(perm), need_dx=False,
                                      dw_dtype=torch.float32)
    assert np.array_equal(host(dw)[0], dv[~gone].T @ xv[perm[~gone]])  # sixteenths below 2^24 of them


@pytest.mark.parametrize("T,k", [(1, 1), (1000, 2)])
def test_tokens_without_positions_of_the_c_abi(T, k):
    """With exactly the workspace that the library asks for: zeros."""
    B = _q().binding
    K, N = 72, 40
    d = B.make_grouped_dims(N, K, 3, k, 0, T)
    n = B.ds4moe_grouped_workspace_bytes(d)
    ws, dx = torch.full((n,), 77, dtype=torch.uint8, device="cuda"), torch.full((T, K), 7.0, dtype=torch.bfloat16, device="cuda")
    w, some = torch.ones(3, N, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    B.ds4moe_grouped_dx(d, dx, K, None, N, w, some, some, ws, n)
    torch.cuda.synchronize()
    assert not dx.any()


def test_rows_gradient_of_more_tokens_than_workgroups():
    """2^20 workgroups add the tokens up and go round: tokens of both rounds that stand several times, some very often."""
    q = _q()
    T, E, N, K = (1 << 20) + 300, 2, 8, 16
    rng = np.random.default_rng(0)
    near = rng.integers(0, 300, 3000)
    perm = np.concatenate([near, near[:1500] + (1 << 20), rng.integers(0, T, 20000), np.full(300, 7), np.full(400, (1 << 20) + 7)]).astype(np.int32)
    rng.shuffle(perm)
    P = perm.size
    offsets = np.array([0, P // 3, P], dtype=np.int32)
    x = torch.zeros(T, K, dtype=torch.float16, device="cuda")
    w, wv = half(rng.integers(-2, 3, (E, N, K)).astype(np.float64), "f16")
    dy, dyv = half(rng.integers(-2, 3, (P, N)).astype(np.float64), "f16")
    dx, _ = q.grouped_matmul_backward(dy, x, w, dev(offsets), dev(perm), need_dw=False)
    want = np.zeros((T, K))
    for e in range(E):
        p = slice(offsets[e], offsets[e + 1])
        np.add.at(want, perm[p], dyv[p] @ wv[e])  # whole numbers: exact in fp32
    assert torch.equal(dx.cpu(), torch.from_numpy(want).half())
