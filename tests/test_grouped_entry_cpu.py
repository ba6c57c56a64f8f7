"""What the torch entry points of the 8-bit operators and the grouped products check, without a GPU."""
import pytest
import torch

import quantized_routed_moe_router_amd as q
from test_grouped_cpu import BF16, F32, I8, grouped
from test_mx4_entry_cpu import Tensor


def asks(shape):
    t = Tensor(shape, F32)
    t.requires_grad = True
    return t


CALLS = {
    "dequantize": lambda s: q.int8_dequantize(Tensor((3, 32), I8), s((3,))),
    "matmul, weights' scales": lambda s: q.int8_matmul(Tensor((3, 64), BF16), Tensor((8, 64), I8), s((8,))),
    "matmul, rows' scales": lambda s: q.int8_matmul(Tensor((3, 64), I8), Tensor((8, 64), I8), Tensor((8,), F32), s((3,))),
    "grouped, rows' scales": lambda s: grouped(Tensor((10, 128), I8), Tensor((4, 64, 128), I8), x_scales=s((10,)), w_scales=Tensor((4, 64), F32)),
    "grouped, weights' scales": lambda s: grouped(Tensor((10, 128), I8), Tensor((4, 64, 128), I8), x_scales=Tensor((10,), F32), w_scales=s((4, 64))),
}


@pytest.mark.parametrize("call", list(CALLS))
def test_scales_that_ask_for_a_gradient_are_refused(call, monkeypatch):
    """Learned scales: their gradient would be lost without a word.  Nothing else is refused: without gradients the call goes
    as far as the library's outputs."""
    class Reached(Exception):
        pass

    def empty(*a, **k):
        raise Reached
    monkeypatch.setattr(q.grouped, "_empty", empty)
    with pytest.raises(ValueError, match="asks for a gradient"):
        CALLS[call](asks)
    with torch.no_grad(), pytest.raises(Reached):
        CALLS[call](asks)
    with pytest.raises(Reached):
        CALLS[call](lambda shape: Tensor(shape, F32))
