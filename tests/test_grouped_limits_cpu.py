"""What the C ABI of the products grouped by expert refuses, each limit by itself: every other argument is one that it
takes, so that only the check in question can refuse (fake addresses, never read: every call returns before a launch)."""
import pytest

from quantized_routed_moe_router_amd import binding as B
from test_grouped_cpu import dims, dw, dx, forward


@pytest.mark.parametrize("T,k", [(1000, 2), (1, 1), (70000, 8)])
def test_workspace_of_no_positions(T, k):
    """Tokens without positions: their places have to be told apart from others' all the same."""
    d = dims(rows=0, tokens=T, top_k=k)
    need = B.lib().ds4moe_grouped_workspace_bytes(d)
    assert need >= 4 * T * k
    assert dx(d, n=need - 1) == B.DS4MOE_ERR_WORKSPACE
    assert B.lib().ds4moe_grouped_workspace_bytes(dims(rows=0, tokens=0)) > 0


FAR = 1 << 17  # a step of results that every row fits
FEW = dict(n_experts=1, rows=8, tokens=8, top_k=1, N=8, K=8)
# sizes at a limit, and the first beyond it
LIMITS = {
    "positions": (dict(FEW, rows=1 << 23), dict(FEW, rows=(1 << 23) + 1)),
    "tokens": (dict(FEW, tokens=1 << 23), dict(FEW, tokens=(1 << 23) + 1)),
    "experts": (dict(FEW, n_experts=512), dict(FEW, n_experts=513)),
    "ranks": (dict(FEW, top_k=16), dict(FEW, top_k=17)),
    "N": (dict(FEW, N=65536), dict(FEW, N=65544)),
    "K": (dict(FEW, K=65536), dict(FEW, K=65544)),
    "P by N": (dict(FEW, rows=1 << 21, N=65536), dict(FEW, rows=(1 << 21) + 1, N=65536)),
    "P by K": (dict(FEW, rows=1 << 21, K=65536), dict(FEW, rows=(1 << 21) + 1, K=65536)),
    "E by N by K": (dict(FEW, n_experts=512, N=4096, K=65536), dict(FEW, n_experts=512, N=4104, K=65536)),
}


@pytest.mark.parametrize("limit", list(LIMITS))
def test_each_limit_of_the_sizes(limit):
    within, beyond = LIMITS[limit]
    assert B.lib().ds4moe_grouped_workspace_bytes(dims(**within)) > 0
    d = dims(**beyond)
    assert B.lib().ds4moe_grouped_workspace_bytes(d) == 0
    assert [forward(d, ldy=FAR, ldx=FAR), dx(d, lddx=FAR, lddy=FAR), dw(d, lddy=FAR, ldx=FAR)] == [B.DS4MOE_ERR_SHAPE] * 3


def test_each_limit_of_the_steps():
    """Operands' rows at most 2^22 values apart, results' at most 2^40, both no closer than they are long."""
    d, far = dims(), 1 << 22
    assert [forward(d, ldx=far + 8), dx(d, lddy=far + 8), dw(d, lddy=far + 8), dw(d, ldx=far + 8)] == [B.DS4MOE_ERR_SHAPE] * 4
    assert [forward(d, ldy=(1 << 40) + 1), dx(d, lddx=(1 << 40) + 1)] == [B.DS4MOE_ERR_SHAPE] * 2
    assert [forward(d, ldx=120), dx(d, lddy=56), dw(d, lddy=56), dw(d, ldx=120), forward(d, ldy=63), dx(d, lddx=127)] == [B.DS4MOE_ERR_SHAPE] * 6
    # values of 16 bits in whole pieces of 16 bytes, of 8 bits too
    assert [forward(d, ldx=132), dx(d, lddy=68), dw(d, lddy=68), dw(d, ldx=132)] == [B.DS4MOE_ERR_SHAPE] * 4
    i8 = dims(dtype=B.DS4MOE_I8)
    A = 1 << 20
    assert [forward(i8, ldx=136, xs=A, ws=A), forward(i8, ldx=far + 16, xs=A, ws=A)] == [B.DS4MOE_ERR_SHAPE] * 2


def test_each_limit_of_the_8_bit_product():
    L, A = B.lib(), 1 << 20
    ws = L.ds4moe_int8_workspace_bytes
    assert ws(1 << 24, 131056, B.DS4MOE_BF16) > 0 and ws((1 << 24) + 1, 16, B.DS4MOE_BF16) == 0 and ws(1, 131057, B.DS4MOE_BF16) == 0

    def mul(ldy=64, lda=64, M=8, N=64, K=64):
        return L.ds4moe_int8_matmul(A, B.DS4MOE_F32, ldy, A, A, B.DS4MOE_I8, lda, A, A, M, N, K, None, 0, None)
    big = 1 << 24
    assert [mul(M=big + 1), mul(N=big + 1, ldy=big + 1), mul(K=131072, lda=131072), mul(M=big, N=8200, ldy=8200), mul(lda=(1 << 22) + 16), mul(lda=48),
            mul(lda=72), mul(ldy=63), mul(ldy=(1 << 40) + 1)] == [B.DS4MOE_ERR_SHAPE] * 9
