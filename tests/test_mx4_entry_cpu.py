"""What the torch entry points of the expert gate and the 4-bit operators check before they call the library, without a
GPU: stand-ins for tensors (never read), a stand-in for the library's calls."""
import numpy as np
import pytest
import torch

import quantized_routed_moe_router_amd as q
from quantized_routed_moe_router_amd import mx4

I32, U8, BF16, F32 = torch.int32, torch.uint8, torch.bfloat16, torch.float32


class Tensor:
    """Shape, type and place of a contiguous tensor on a GPU that is not there."""
    is_cuda, requires_grad = True, False

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self.device = tuple(shape), dtype, torch.device("cuda", device)

    def dim(self):
        return len(self.shape)

    def stride(self):
        return tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    def get_device(self):
        return self.device.index


def packed(*shape, device=0, scales_device=None):
    *lead, cols = shape
    return (Tensor((*lead, cols // 2), U8, device),
            Tensor((*lead, cols // 32), U8, device if scales_device is None else scales_device))


def experts(**devices):
    d = {"gate": 0, "up": 0, "down": 0, **devices}
    return q.Mx4Experts(256, 64, 8, 2, packed(8, 64, 256, device=d["gate"]), packed(8, 64, 256, device=d["up"]),
                        packed(8, 256, 64, device=d["down"]))


def routing(T, **devices):
    shapes = {"topk_idx": (T, 2), "topk_w": (T, 2), "counts": (8,), "offsets": (9,), "perm": (2 * T,)}
    return {n: Tensor(s, F32 if n == "topk_w" else I32, devices.get(n, 0)) for n, s in shapes.items()}


def test_tensors_of_two_devices_are_refused():
    gate, x = q.Gate(8, 2), Tensor((4, 256), BF16)
    calls = [
        lambda: gate.forward(Tensor((4, 8), F32), Tensor((8,), F32, 1)),
        lambda: gate.backward(Tensor((4, 8), F32), Tensor((4, 2), I32, 1), Tensor((4, 2), F32)),
        lambda: gate.backward(Tensor((4, 8), F32), Tensor((4, 2), I32), Tensor((4, 2), F32, 1)),
        lambda: q.mx4_dequantize(*packed(4, 64, scales_device=1)),
        lambda: q.mx4_matmul(x, *packed(16, 256, device=1)),
        lambda: q.mx4_matmul(x, *packed(16, 256, scales_device=1)),
        lambda: q.mx4_matmul(packed(4, 256)[0], *packed(16, 256, device=1), a_scales=packed(4, 256)[1]),
        lambda: q.mx4_matmul(packed(4, 256)[0], *packed(16, 256), a_scales=packed(4, 256, device=1)[1]),
        lambda: experts(up=1), lambda: experts(down=1),
        lambda: experts().forward(Tensor((4, 256), BF16, 1), routing(4)),
        *[lambda n=n: experts().forward(x, routing(4, **{n: 1})) for n in routing(4)],
        lambda: q.Mx4Layer(Tensor((8, 256), F32, 1), gate, experts()),
        lambda: q.Mx4Layer(Tensor((8, 256), F32), gate, experts()).logits(Tensor((4, 256), BF16, 1)),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="cuda:1"):
            call()


def test_the_library_is_called_with_the_tensors_device_as_the_current_one(monkeypatch):
    seen = []

    class Device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            seen.append(("on", self.i))

        def __exit__(self, *a):
            seen.append(("off", self.i))

    monkeypatch.setattr(mx4, "_device", lambda: 0)
    monkeypatch.setattr(mx4, "_raw_stream", lambda i: 1000 + i)
    monkeypatch.setattr(torch.cuda, "device", Device)

    def entry(*args):
        seen.append(args)
        return 0

    mx4._call(entry, "x", 0, 1, 2)
    mx4._call(entry, "x", 1, 3)
    assert seen == [(1, 2, 1000), ("on", 1), (3, 1001), ("off", 1)]
    with pytest.raises(q.Ds4MoeError):
        mx4._call(lambda *a: 2, "x", 1)
    assert seen[-1] == ("off", 1)


def test_a_gradient_that_would_be_lost_is_refused():
    def asks(shape, dtype):
        t = Tensor(shape, dtype)
        t.requires_grad = True
        return t

    r = routing(4)
    r["topk_w"] = asks((4, 2), F32)
    calls = [
        lambda: q.Gate(8, 2).forward(asks((4, 8), F32)),
        lambda: q.Gate(8, 2).forward(Tensor((4, 8), F32), asks((8,), F32)),
        lambda: q.mx4_quantize(asks((4, 64), BF16)),
        lambda: q.mx4_matmul(asks((4, 256), BF16), *packed(16, 256)),
        lambda: experts().forward(asks((4, 256), BF16), routing(4)),
        lambda: experts().forward(Tensor((4, 256), BF16), r),
        lambda: q.Mx4Layer(Tensor((8, 256), F32), q.Gate(8, 2), experts()).forward(asks((4, 256), BF16)),
        lambda: q.Mx4Layer(asks((8, 256), F32), q.Gate(8, 2), experts()).forward(Tensor((4, 256), BF16)),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
    with torch.no_grad():  # nothing to lose: the next check speaks
        with pytest.raises(ValueError, match="7 columns"):
            q.Gate(8, 2).forward(asks((4, 7), F32))
    with pytest.raises(ValueError, match="topk_idx"):  # the gradient itself may have logits that ask for one
        q.Gate(8, 2).backward(asks((4, 8), F32), Tensor((4, 3), I32), Tensor((4, 2), F32))


@pytest.mark.parametrize("T,k,E", [(1, 8, 256), (64, 16, 512), (4096, 8, 256), (4096, 16, 512), (4097, 8, 256), (8192, 8, 256), (1 << 17, 4, 16)])
def test_outputs_of_the_gate_keep_little_beside_themselves(monkeypatch, T, k, E):
    """Kept for a backward pass, the choice of many tokens does not keep the workspace, that of few at most 0.7 MB of it."""
    seen = []
    monkeypatch.setattr(mx4, "_empty", lambda *shape, dtype, device: torch.empty(*shape, dtype=dtype))
    monkeypatch.setattr(mx4, "_call", lambda entry, what, dev, *args: seen.append(args))
    gate = q.Gate(E, k)
    out = gate.forward(Tensor((T, E), F32))
    kept = {out[n].untyped_storage().data_ptr(): out[n].untyped_storage().nbytes() for n in out}
    need = sum(out[n].numel() * 4 for n in out)
    assert sum(kept.values()) - need <= (700_000 if T <= 4096 else 0)
    _, _, _, _, _, r, ws, ws_bytes = seen[0]
    r = r._obj
    assert (r.topk_idx, r.perm, r.counts, r.offsets, r.topk_w) == tuple(out[n].data_ptr() for n in ("topk_idx", "perm", "counts", "offsets", "topk_w"))
    # the workspace is its own piece of memory
    spans = sorted([(ws, ws + ws_bytes)] + [(out[n].data_ptr(), out[n].data_ptr() + 4 * out[n].numel()) for n in out])
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
