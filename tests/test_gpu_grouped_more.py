"""Products grouped by expert on the GPU: the largest results, and what the other files do not ask for.  Bounds as in
test_gpu_grouped."""
import numpy as np
import pytest
import torch

from test_gpu_grouped import _q, dev, host

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
