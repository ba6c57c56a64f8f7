"""Every instance that the library's rules choose (csrc/grouped_plan.h), on whole numbers small enough for every sum to be
exact: ragged counts, experts without rows, odd N, sums that end inside a stage.  test_grouped_forms_cpu holds each case to
its instance, so that a changed rule shows there."""
import numpy as np
import pytest
import torch

from test_gpu_grouped import DT, _q, dev

pytestmark = pytest.mark.gpu

#           experts, rows in all, N, K (of 8 bits rounded up to 16), the instance
FORWARD = [(128, 8192, 4104, 72, (8, 128)), (128, 8192, 4099, 72, (8, 128)), (300, 9000, 3777, 136, (8, 128)), (2, 256, 131072 // 2, 40, (4, 0)),
           (4, 8200, 4100, 80, (8, 0)), (3, 4500, 7999, 200, (8, 0)), (40, 2400, 1001, 328, (4, 64)), (5, 3000, 777, 264, (4, 0)), (200, 400, 515, 96, "few")]
#          experts, rows in all, N, K
TURNED = [(512, 30000, 72, 520, (8, 128)), (400, 20000, 136, 776, (8, 128)), (60, 3600, 200, 328, (4, 64)), (6, 5000, 264, 1032, (4, 0))]
WEIGHTS = [(512, 20000, 264, 264, True), (300, 9000, 520, 264, True), (300, 9000, 264, 72, False), (4, 5000, 392, 136, False)]
DENSE = [(8200, 4100, 80, (8, 0)), (100, 400000, 48, (8, 128)), (128, 262400, 144, (8, 128)), (65, 3000, 144, (4, 0)), (64, 999, 144, "few")]


def ragged(E, P, rng):
    """Offsets of P rows: a quarter of the experts have none, one has many."""
    share = rng.random(E) ** 2 * (rng.random(E) > 0.25)
    share[E // 2] = 2
    counts = rng.multinomial(P, share / share.sum())
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def whole(rng, shape, most, kind):
    a = rng.integers(-most, most + 1, shape, dtype=np.int8)
    return torch.from_numpy(a).cuda().to(torch.int8 if kind == "int8" else DT[kind])


def by_expert(offsets):
    return [(e, slice(int(a), int(b))) for e, (a, b) in enumerate(zip(offsets, offsets[1:])) if b > a]


@pytest.mark.parametrize("kind", ["bf16", "f16", "int8"])
@pytest.mark.parametrize("E,P,N,K,form", FORWARD)
def test_product(kind, E, P, N, K, form):
    q = _q()
    rng = np.random.default_rng(E + N)
    K = -(-K // 16) * 16 if kind == "int8" else K
    T = P // 2 + 1
    x, w, offsets = whole(rng, (T, K), 4, kind), whole(rng, (E, N, K), 4, kind), ragged(E, P, rng)
    rows = rng.integers(0, T, P)
    ones = dict(x_scales=torch.ones(T, device="cuda"), w_scales=torch.ones(E, N, device="cuda")) if kind == "int8" else {}
    y = q.grouped_matmul(x, w, dev(offsets), dev(rows.astype(np.int32)), y_dtype=torch.float32, **ones)
    at = torch.from_numpy(rows).cuda()
    for e, p in by_expert(offsets):
        assert torch.equal(y[p], x[at[p]].float() @ w[e].float().t()), (e, p)
    # in order, and in 16 bits: below 2^24 the same sums, rounded
    half = torch.bfloat16 if kind == "int8" else DT[kind]
    more = dict(ones, x_scales=torch.ones(P, device="cuda")) if ones else {}
    assert torch.equal(q.grouped_matmul(x[at].contiguous(), w, dev(offsets), y_dtype=half, **more), y.to(half))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("E,P,N,K,form", TURNED)
def test_gradient_of_the_rows(kind, E, P, N, K, form):
    q = _q()
    rng = np.random.default_rng(E + K)
    dy, w, offsets = whole(rng, (P, N), 2, kind), whole(rng, (E, N, K), 2, kind), ragged(E, P, rng)
    want = torch.zeros(P, K, device="cuda")
    for e, p in by_expert(offsets):
        want[p] = dy[p].float() @ w[e].float()
    x = torch.zeros(P, K, dtype=dy.dtype, device="cuda")
    dx, _ = q.grouped_matmul_backward(dy, x, w, dev(offsets), need_dw=False)
    assert torch.equal(dx, want.to(dx.dtype))
    perm = torch.from_numpy(rng.permutation(P)).cuda()  # two positions a token: one rounding of their sum
    x = x[:(P + 1) // 2]
    dx, _ = q.grouped_matmul_backward(dy, x, w, dev(offsets), perm.int(), 2, need_dw=False)
    both = torch.zeros(2 * x.shape[0], K, device="cuda").index_copy_(0, perm, want).view(-1, 2, K).sum(1)
    assert torch.equal(dx, both.to(dx.dtype))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("E,P,N,K,large", WEIGHTS)
def test_gradient_of_the_weights(kind, E, P, N, K, large):
    q = _q()
    rng = np.random.default_rng(E + K)
    dy, x, offsets = whole(rng, (P, N), 4, kind), whole(rng, (P, K), 4, kind), ragged(E, P, rng)
    w = torch.zeros(E, N, K, dtype=x.dtype, device="cuda")
    perm = torch.from_numpy(rng.permutation(P)).cuda()
    for at in (None, perm):
        _, dw = q.grouped_matmul_backward(dy, x, w, dev(offsets), None if at is None else at.int(), need_dx=False, dw_dtype=torch.float32)
        rows = x if at is None else x[at]
        seen = dict(by_expert(offsets))
        for e in range(E):
            if e in seen:
                assert torch.equal(dw[e], dy[seen[e]].float().t() @ rows[seen[e]].float()), e
            else:
                assert not dw[e].any(), e


@pytest.mark.parametrize("M,N,K,form", DENSE)
def test_dense_product_of_8_bits(M, N, K, form):
    q = _q()
    rng = np.random.default_rng(M)
    a, w = whole(rng, (M, K), 100, "int8"), whole(rng, (N, K), 100, "int8")
    y = q.int8_matmul(a, w, torch.ones(N, device="cuda"), torch.ones(M, device="cuda"), y_dtype=torch.float32)
    assert torch.equal(y, a.float() @ w.float().t())  # below 2^24


def test_fp16_rows_beyond_32_bit_offsets():
    """Gathered from 5.2 GB: the forms by plain addresses, product and weights' gradient."""
    q = _q()
    T, step, N, K, P = 40000, 65536, 136, 72, 900
    store = torch.zeros(T, step, dtype=torch.float16, device="cuda")
    rng = np.random.default_rng(0)
    rows = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, P)]))
    rng.shuffle(rows)
    P = rows.size
    at = torch.from_numpy(rows).cuda()
    store[at, :K] = whole(rng, (P, K), 4, "f16")
    x, w, offsets = store[:, :K], whole(rng, (3, N, K), 4, "f16"), np.array([0, P // 3, P // 3, P], dtype=np.int32)
    dy = whole(rng, (P, N), 4, "f16")
    y = q.grouped_matmul(x, w, dev(offsets), at.int(), y_dtype=torch.float32)
    _, dw = q.grouped_matmul_backward(dy, x, w, dev(offsets), at.int(), need_dx=False, dw_dtype=torch.float32)
    for e, p in by_expert(offsets):
        assert torch.equal(y[p], x[at[p]].float() @ w[e].float().t())
        assert torch.equal(dw[e], dy[p].float().t() @ x[at[p]].float())
    assert not dw[1].any()
