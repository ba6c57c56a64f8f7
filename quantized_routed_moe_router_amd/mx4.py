"""The expert gate and the 4-bit microscaled (MXFP4) operators on torch tensors.

Plumbing around the C ABI only: shapes, types and devices are checked here,
torch allocates outputs and workspaces (on the current stream, so a workspace
is never shared by calls that overlap), and every step runs in libds4moe.so,
on the device of the call's tensors and its current stream.
Nothing here is recorded by autograd: a tensor that requires a gradient is
refused while gradients are on, and Gate.backward is the gradient that there is.
A matrix in 4-bit form is a pair of uint8 tensors: codes [..., cols/2] and
scales [..., cols/32], rows without gaps.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B

_DTYPES = {torch.float32: B.DS4MOE_F32, torch.bfloat16: B.DS4MOE_BF16}
_BF16 = (torch.bfloat16,)
GATE_JOINT = 2048  # tokens up to which a gate's workspace and its indices are one allocation
_SCORES = {"sqrt_softplus": B.SCORE_SQRT_SOFTPLUS, "sigmoid": B.SCORE_SIGMOID, "softmax": B.SCORE_SOFTMAX}


def _need(ok, what: str) -> None:
    if not ok:
        raise ValueError(what)


# The wrappers run once per layer and token, in the time of a kernel or two:
# addresses go to the library as plain numbers, and a refusal's text is made
# only when there is one.
_raw_stream = torch._C._cuda_getCurrentRawStream
_device = torch._C._cuda_getDevice
_empty = torch.empty
_split = torch.split_with_sizes
_L = B.lib()


def _rows(t: torch.Tensor, what: str, dtypes=_DTYPES) -> int:
    """The distance of the rows of a matrix on the GPU whose columns are adjacent."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{what}: a matrix on the GPU is wanted")
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: unsupported type {t.dtype}")
    rows, cols = t.shape
    d, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{what}: columns have to be adjacent")
    if rows > 1 and d < cols:
        raise ValueError(f"{what}: rows overlap")
    return d if rows > 1 else cols


def _tracked(what: str) -> None:
    """A tensor asks for a gradient: not one that these calls would lose without a word."""
    if torch.is_grad_enabled():
        raise ValueError(f"{what} asks for a gradient, which autograd does not get from this call: detach it, or call "
                         "under torch.no_grad() (Gate.backward gives the gradient of a gate's logits)")


def _elsewhere(t: torch.Tensor, what: str, i: int) -> None:
    raise ValueError(f"{what}: on {t.device}, the call's other tensors on cuda:{i}")


def _flat(t: torch.Tensor, what: str, dtype, shape=None, i=None) -> torch.Tensor:
    """Checked: contiguous, of a type and shape, on a GPU (of index i)."""
    at = t.get_device()
    if t.dtype is not dtype or at < 0 or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous {dtype} tensor on the GPU is wanted")
    if i is not None and at != i:
        _elsewhere(t, what, i)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, not {tuple(shape)}")
    return t


def _packed(codes: torch.Tensor, scales: torch.Tensor, what: str, shape=None, i=None) -> tuple:
    _flat(codes, what, torch.uint8, None if shape is None else (*shape[:-1], shape[-1] // 2), i)
    *rows, n = codes.shape
    if n % 16:
        raise ValueError(f"{what}: whole blocks of 32 are wanted")
    _flat(scales, what + " scales", torch.uint8, (*rows, n // 16), codes.get_device())
    return codes, scales


def _call(entry, what: str, i: int, *args) -> None:
    """A call of the library on the current stream of device i, with that device the current one."""
    if i == _device():
        status = entry(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            status = entry(*args, _raw_stream(i))
    if status:
        raise B.Ds4MoeError(status, what)


class Gate:
    """Scores, groups, top-k and weights of an expert router (ds4moe_gate)."""

    def __init__(self, E: int, k: int, score: str = "sqrt_softplus", n_groups: int = 1, top_groups: int = 1,
                 group_rank: int = 1, renorm: bool = True, scale: float = 1.0):
        _need(score in _SCORES, f"unknown score {score!r}: one of {sorted(_SCORES)}")
        self.E, self.k = E, k
        gatings = {t: B.make_gating(E, k, n_groups, top_groups, group_rank, _SCORES[score], renorm, d, scale)
                   for t, d in _DTYPES.items()}
        _need(B.ds4moe_gate_workspace_bytes(gatings[torch.float32], 1) > 0,
              f"unsupported gate: E={E}, k={k}, {n_groups} groups, {top_groups} kept, rank {group_rank}, scale {scale}")
        self._gating = {t: ctypes.byref(g) for t, g in gatings.items()}

    def _logits(self, logits: torch.Tensor, bias) -> int:
        ld = _rows(logits, "logits")
        if logits.shape[1] != self.E:
            raise ValueError(f"logits: {logits.shape[1]} columns, {self.E} experts")
        if bias is not None:
            _flat(bias, "bias", torch.float32, (self.E,), logits.get_device())
        return ld

    def forward(self, logits: torch.Tensor, bias: torch.Tensor | None = None) -> dict:
        """topk_idx [T,k], topk_w [T,k], counts [E], offsets [E+1] and perm [T*k] of logits [T,E].  All but topk_w are
        parts of one allocation, which holds as long as one of them does."""
        if logits.requires_grad or (bias is not None and bias.requires_grad):
            _tracked("logits or bias")
        ld, g, i = self._logits(logits, bias), self._gating[logits.dtype], logits.get_device()
        T, k, E = logits.shape[0], self.k, self.E
        if T == 0:
            return {n: torch.zeros(s, dtype=torch.float32 if n == "topk_w" else torch.int32, device=i) for n, s in (
                ("topk_idx", (0, k)), ("topk_w", (0, k)), ("counts", E), ("offsets", E + 1), ("perm", 0))}
        # One allocation for the indices; an allocation costs as much as a tenth of a call for one token.  Up to
        # GATE_JOINT tokens the workspace is part of it (first: it wants the alignment): 2048 tokens 13.0 us, 14.2 with
        # one of its own.  Of more tokens the kernels take longer than the call (4096: 14.4 us both ways), and whoever
        # keeps the choice for a backward pass would keep the workspace with it, as much again as the indices.
        n, A = _L.ds4moe_gate_workspace_bytes(g, T), T * k
        w = _empty(T, k, dtype=torch.float32, device=i)
        held = n // 4 if T <= GATE_JOINT else 0
        buf = _empty(held + 2 * A + 2 * E + 1, dtype=torch.int32, device=i)
        _, idx, perm, counts, offsets = _split(buf, (held, A, A, E, E + 1))
        at = buf.data_ptr() + 4 * held
        own = None if held else _empty(n, dtype=torch.uint8, device=i)
        ws = buf.data_ptr() if held else own.data_ptr()
        _call(_L.ds4moe_gate, "gate", i, g, logits.data_ptr(), ld, None if bias is None else bias.data_ptr(), T,
              ctypes.byref(B.Routing(at, w.data_ptr(), at + 8 * A, at + 8 * A + 4 * E, at + 4 * A, None)), ws, n)
        idx = idx.view(T, k)
        return {"topk_idx": idx, "topk_w": w, "counts": counts, "offsets": offsets, "perm": perm}

    def backward(self, logits: torch.Tensor, topk_idx: torch.Tensor, d_topk_w: torch.Tensor,
                 bias: torch.Tensor | None = None) -> torch.Tensor:
        """Gradient of the logits (in their type) from the gradient of topk_w."""
        ld, i = self._logits(logits, bias), logits.get_device()
        T = logits.shape[0]
        _flat(topk_idx, "topk_idx", torch.int32, (T, self.k), i)
        _flat(d_topk_w, "d_topk_w", torch.float32, (T, self.k), i)
        out = _empty(T, self.E, dtype=logits.dtype, device=i)
        _call(_L.ds4moe_gate_backward, "gate_backward", i, self._gating[logits.dtype], logits.data_ptr(), ld,
              None if bias is None else bias.data_ptr(), topk_idx.data_ptr(), d_topk_w.data_ptr(), T, out.data_ptr(),
              self.E)
        return out


def mx4_quantize(x: torch.Tensor) -> tuple:
    """(codes, scales) of a matrix [rows, cols] in fp32 or bf16; columns are filled up with zeros to blocks of 32."""
    if x.requires_grad:
        _tracked("x")
    ld, i = _rows(x, "x"), x.get_device()
    rows, cols = x.shape
    nb = (cols + 31) // 32
    codes = _empty(rows, 16 * nb, dtype=torch.uint8, device=i)
    scales = _empty(rows, nb, dtype=torch.uint8, device=i)
    _call(_L.ds4moe_mx4_quantize, "mx4_quantize", i, codes.data_ptr(), scales.data_ptr(), x.data_ptr(),
          _DTYPES[x.dtype], rows, cols, ld)
    return codes, scales


def mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, cols: int | None = None,
                   dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The values of a 4-bit matrix, the first `cols` of each row (all by default)."""
    _packed(codes, scales, "codes")
    if codes.dim() != 2 or dtype not in _DTYPES:
        raise ValueError(f"a matrix and fp32 or bf16 are wanted, not {dtype}")
    rows, nb = scales.shape
    cols = 32 * nb if cols is None else cols
    if (cols + 31) // 32 != nb:
        raise ValueError(f"{cols} columns are not {nb} blocks")
    i = codes.get_device()
    out = _empty(rows, cols, dtype=dtype, device=i)
    _call(_L.ds4moe_mx4_dequantize, "mx4_dequantize", i, out.data_ptr(), _DTYPES[dtype], cols, codes.data_ptr(),
          scales.data_ptr(), rows, cols)
    return out


def mx4_matmul(a: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, a_scales: torch.Tensor | None = None,
               y_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """a [M,K] times w [N,K]^T: w in 4-bit form, a bf16, or in 4-bit form with a_scales."""
    if a.requires_grad:
        _tracked("a")
    _packed(w, w_scales, "w")
    if w.dim() != 2 or y_dtype not in _DTYPES:
        raise ValueError(f"w: a matrix is wanted, and an fp32 or bf16 result, not {y_dtype}")
    (N, K), i = w.shape, w.get_device()
    K *= 2
    if a_scales is None:
        lda, kind, sa = _rows(a, "a", _BF16), B.DS4MOE_BF16, None
        if a.shape[1] != K:
            raise ValueError(f"a: {a.shape[1]} columns, w has {K}")
        if a.get_device() != i:
            _elsewhere(a, "a", i)
    else:
        _packed(a, a_scales, "a", None, i)
        if a.dim() != 2 or 2 * a.shape[1] != K:
            raise ValueError(f"a: shape {tuple(a.shape)}, w has {K} columns")
        lda, kind, sa = K, B.DS4MOE_MX4, a_scales.data_ptr()
    M = a.shape[0]
    y = _empty(M, N, dtype=y_dtype, device=i)
    _call(_L.ds4moe_mx4_matmul, "mx4_matmul", i, y.data_ptr(), _DTYPES[y_dtype], N, a.data_ptr(), sa, kind, lda,
          w.data_ptr(), w_scales.data_ptr(), M, N, K)
    return y


class Mx4Experts:
    """Routed SwiGLU experts on 4-bit weights: gate, up (codes [E,I,H/2], scales [E,I,H/32]) and down (codes
    [E,H,I/2], scales [E,H,I/32]), which stay where they are."""

    def __init__(self, H: int, I: int, E: int, k: int, gate: tuple, up: tuple, down: tuple,
                 y_dtype: torch.dtype = torch.bfloat16):
        _need(y_dtype in _DTYPES, f"unsupported y_dtype {y_dtype}")
        self.H, self.I, self.E, self.k, self.y_dtype = H, I, E, k, y_dtype
        self.dims = B.make_mx4_dims(H, I, E, k, _DTYPES[y_dtype])
        _need(B.ds4moe_mx4_workspace_bytes(self.dims, 1) > 0, f"unsupported experts: H={H}, I={I}, E={E}, k={k}")
        self.gate = _packed(*gate, "gate", (E, I, H))
        self.device = self.gate[0].device
        self.up = _packed(*up, "up", (E, I, H), self.device.index)
        self.down = _packed(*down, "down", (E, H, I), self.device.index)
        self._dims = ctypes.byref(self.dims)
        self._weights = ctypes.byref(B.make_mx4_weights(*self.gate, *self.up, *self.down))

    def forward(self, x: torch.Tensor, routing: dict) -> torch.Tensor:
        """y [T,H] of bf16 x [T,H]; routing: the dict of Gate.forward or DeviceLayer.route."""
        if x.requires_grad or routing["topk_w"].requires_grad:
            _tracked("x or topk_w")
        ldx, dev = _rows(x, "x", _BF16), self.device
        T, H = x.shape
        if H != self.H:
            raise ValueError(f"x: {H} columns, hidden size {self.H}")
        i = dev.index
        if x.get_device() != i:
            _elsewhere(x, "x", i)
        i32, k, E = torch.int32, self.k, self.E
        r = B.Routing(_flat(routing["topk_idx"], "topk_idx", i32, (T, k), i).data_ptr(),
                      _flat(routing["topk_w"], "topk_w", torch.float32, (T, k), i).data_ptr(),
                      _flat(routing["counts"], "counts", i32, (E,), i).data_ptr(),
                      _flat(routing["offsets"], "offsets", i32, (E + 1,), i).data_ptr(),
                      _flat(routing["perm"], "perm", i32, (T * k,), i).data_ptr(), None)
        n = _L.ds4moe_mx4_workspace_bytes(self._dims, T)
        ws = _empty(n, dtype=torch.uint8, device=dev)
        y = _empty(T, H, dtype=self.y_dtype, device=dev)
        _call(_L.ds4moe_mx4_experts, "mx4_experts", i, self._dims, self._weights, x.data_ptr(), ldx, T,
              ctypes.byref(r), y.data_ptr(), ws.data_ptr(), n)
        return y


class Mx4Layer:
    """A routed layer on 4-bit experts: router logits (accumulated in fp64, as ds4moe_route), gate, experts.  The router
    takes hidden sizes that are multiples of 256 and up to 256 experts; gate and experts go further on their own."""

    def __init__(self, router_w: torch.Tensor, gate: Gate, experts: Mx4Experts, bias: torch.Tensor | None = None):
        _flat(router_w, "router_w", router_w.dtype, (experts.E, experts.H), experts.device.index)
        _need(router_w.dtype in _DTYPES, f"router_w: unsupported type {router_w.dtype}")
        _need((gate.E, gate.k) == (experts.E, experts.k), "gate and experts differ in their numbers of experts or choices")
        self.router_w, self.gate, self.experts, self.bias = router_w, gate, experts, bias
        self._dims = B.make_dims(experts.H, 256, experts.E, 1, 0, B.DS4MOE_BF16, _DTYPES[router_w.dtype])
        _need(B.ds4moe_workspace_bytes(self._dims, 1, B.MODE_ROUTE) > 0,
              f"unsupported router: hidden size {experts.H}, {experts.E} experts")

    def logits(self, x: torch.Tensor) -> torch.Tensor:
        if x.requires_grad or self.router_w.requires_grad:
            _tracked("x or router_w")
        T, dev = x.shape[0], self.experts.device
        _flat(x, "x", torch.bfloat16, (T, self.experts.H), dev.index)
        out = torch.empty((T, self.experts.E), dtype=torch.float32, device=dev)
        n = B.ds4moe_workspace_bytes(self._dims, T, B.MODE_ROUTE)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        w, r = B.make_weights(self.router_w, None, None, None), B.make_routing(logits=out)
        _call(_L.ds4moe_route, "route", dev.index, ctypes.byref(self._dims), ctypes.byref(w), x.data_ptr(), T, ctypes.byref(r),
              ws.data_ptr(), n)
        return out

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return self.experts.forward(x, self.gate.forward(self.logits(x), self.bias))
