"""The expert gate and the 4-bit microscaled (MXFP4) operators on torch tensors.

Plumbing around the C ABI only: shapes and types are checked here, torch
allocates outputs and workspaces (on the current stream, so a workspace is
never shared by calls that overlap), and every step runs in libds4moe.so.
A matrix in 4-bit form is a pair of uint8 tensors: codes [..., cols/2] and
scales [..., cols/32], rows without gaps.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B

_DTYPES = {torch.float32: B.DS4MOE_F32, torch.bfloat16: B.DS4MOE_BF16}
_SCORES = {"sqrt_softplus": B.SCORE_SQRT_SOFTPLUS, "sigmoid": B.SCORE_SIGMOID, "softmax": B.SCORE_SOFTMAX}


def _need(ok, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _rows(t: torch.Tensor, what: str, dtypes=tuple(_DTYPES)) -> int:
    """The distance of the rows of a matrix on the GPU whose columns are adjacent."""
    _need(t.is_cuda and t.dim() == 2, f"{what}: a matrix on the GPU is wanted")
    _need(t.dtype in dtypes, f"{what}: unsupported type {t.dtype}")
    _need(t.stride(1) == 1 or t.shape[1] <= 1, f"{what}: columns have to be adjacent")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _flat(t: torch.Tensor, what: str, dtype, shape=None) -> torch.Tensor:
    _need(t.is_cuda and t.is_contiguous() and t.dtype == dtype, f"{what}: a contiguous {dtype} tensor on the GPU is wanted")
    _need(shape is None or tuple(t.shape) == tuple(shape), f"{what}: shape {tuple(t.shape)}, not {shape}")
    return t


def _packed(codes: torch.Tensor, scales: torch.Tensor, what: str, shape=None) -> tuple:
    _flat(codes, what, torch.uint8, None if shape is None else (*shape[:-1], shape[-1] // 2))
    _flat(scales, what + " scales", torch.uint8, (*codes.shape[:-1], codes.shape[-1] // 16))
    _need(codes.shape[-1] % 16 == 0, f"{what}: whole blocks of 32 are wanted")
    return codes, scales


class Gate:
    """Scores, groups, top-k and weights of an expert router (ds4moe_gate)."""

    def __init__(self, E: int, k: int, score: str = "sqrt_softplus", n_groups: int = 1, top_groups: int = 1,
                 group_rank: int = 1, renorm: bool = True, scale: float = 1.0):
        _need(score in _SCORES, f"unknown score {score!r}: one of {sorted(_SCORES)}")
        self.E, self.k = E, k
        self._gating = {t: B.make_gating(E, k, n_groups, top_groups, group_rank, _SCORES[score], renorm, d, scale)
                        for t, d in _DTYPES.items()}
        _need(B.ds4moe_gate_workspace_bytes(self._gating[torch.float32], 1) > 0,
              f"unsupported gate: E={E}, k={k}, {n_groups} groups, {top_groups} kept, rank {group_rank}, scale {scale}")

    def _logits(self, logits: torch.Tensor, bias) -> int:
        ld = _rows(logits, "logits")
        _need(logits.shape[1] == self.E, f"logits: {logits.shape[1]} columns, {self.E} experts")
        if bias is not None:
            _flat(bias, "bias", torch.float32, (self.E,))
        return ld

    def forward(self, logits: torch.Tensor, bias: torch.Tensor | None = None) -> dict:
        """topk_idx [T,k], topk_w [T,k], counts [E], offsets [E+1] and perm [T*k] of logits [T,E]."""
        ld, g, dev = self._logits(logits, bias), self._gating[logits.dtype], logits.device
        T = logits.shape[0]
        new = torch.zeros if T == 0 else torch.empty
        out = {"topk_idx": new((T, self.k), dtype=torch.int32, device=dev),
               "topk_w": new((T, self.k), dtype=torch.float32, device=dev),
               "counts": new(self.E, dtype=torch.int32, device=dev),
               "offsets": new(self.E + 1, dtype=torch.int32, device=dev),
               "perm": new(T * self.k, dtype=torch.int32, device=dev)}
        n = B.ds4moe_gate_workspace_bytes(g, T)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        B.ds4moe_gate(g, logits, ld, bias, T, B.make_routing(**out), ws, n, torch.cuda.current_stream(dev))
        return out

    def backward(self, logits: torch.Tensor, topk_idx: torch.Tensor, d_topk_w: torch.Tensor,
                 bias: torch.Tensor | None = None) -> torch.Tensor:
        """Gradient of the logits (in their type) from the gradient of topk_w."""
        ld, g, dev = self._logits(logits, bias), self._gating[logits.dtype], logits.device
        T = logits.shape[0]
        _flat(topk_idx, "topk_idx", torch.int32, (T, self.k))
        _flat(d_topk_w, "d_topk_w", torch.float32, (T, self.k))
        out = torch.empty((T, self.E), dtype=logits.dtype, device=dev)
        B.ds4moe_gate_backward(g, logits, ld, bias, topk_idx, d_topk_w, T, out, self.E, torch.cuda.current_stream(dev))
        return out


def mx4_quantize(x: torch.Tensor) -> tuple:
    """(codes, scales) of a matrix [rows, cols] in fp32 or bf16; columns are filled up with zeros to blocks of 32."""
    ld = _rows(x, "x")
    rows, cols = x.shape
    nb = (cols + 31) // 32
    codes = torch.empty((rows, 16 * nb), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, nb), dtype=torch.uint8, device=x.device)
    B.ds4moe_mx4_quantize(codes, scales, x, _DTYPES[x.dtype], rows, cols, max(ld, cols),
                          torch.cuda.current_stream(x.device))
    return codes, scales


def mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, cols: int | None = None,
                   dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The values of a 4-bit matrix, the first `cols` of each row (all by default)."""
    _packed(codes, scales, "codes")
    _need(codes.dim() == 2 and dtype in _DTYPES, f"a matrix and fp32 or bf16 are wanted, not {dtype}")
    rows, nb = scales.shape
    cols = 32 * nb if cols is None else cols
    _need((cols + 31) // 32 == nb, f"{cols} columns are not {nb} blocks")
    out = torch.empty((rows, cols), dtype=dtype, device=codes.device)
    B.ds4moe_mx4_dequantize(out, _DTYPES[dtype], max(cols, 1), codes, scales, rows, cols,
                            torch.cuda.current_stream(codes.device))
    return out


def mx4_matmul(a: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, a_scales: torch.Tensor | None = None,
               y_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """a [M,K] times w [N,K]^T: w in 4-bit form, a bf16, or in 4-bit form with a_scales."""
    _packed(w, w_scales, "w")
    _need(w.dim() == 2 and y_dtype in _DTYPES, f"w: a matrix is wanted, and an fp32 or bf16 result, not {y_dtype}")
    N, K = w.shape[0], 2 * w.shape[1]
    if a_scales is None:
        lda, kind = max(_rows(a, "a", (torch.bfloat16,)), K), B.DS4MOE_BF16
        _need(a.shape[1] == K, f"a: {a.shape[1]} columns, w has {K}")
    else:
        _packed(a, a_scales, "a")
        _need(a.dim() == 2 and 2 * a.shape[1] == K, f"a: shape {tuple(a.shape)}, w has {K} columns")
        lda, kind = K, B.DS4MOE_MX4
    y = torch.empty((a.shape[0], N), dtype=y_dtype, device=a.device)
    B.ds4moe_mx4_matmul(y, _DTYPES[y_dtype], max(N, 1), a, a_scales, kind, lda, w, w_scales, a.shape[0], N, K,
                        torch.cuda.current_stream(a.device))
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
        self.up = _packed(*up, "up", (E, I, H))
        self.down = _packed(*down, "down", (E, H, I))
        self._weights = B.make_mx4_weights(*self.gate, *self.up, *self.down)

    def forward(self, x: torch.Tensor, routing: dict) -> torch.Tensor:
        """y [T,H] of bf16 x [T,H]; routing: the dict of Gate.forward or DeviceLayer.route."""
        ldx = max(_rows(x, "x", (torch.bfloat16,)), self.H)
        T, dev = x.shape[0], x.device
        _need(x.shape[1] == self.H, f"x: {x.shape[1]} columns, hidden size {self.H}")
        r = B.Routing(*(ctypes.c_void_p(_flat(routing[n], n, t, s).data_ptr()) for n, t, s in (
            ("topk_idx", torch.int32, (T, self.k)), ("topk_w", torch.float32, (T, self.k)),
            ("counts", torch.int32, (self.E,)), ("offsets", torch.int32, (self.E + 1,)),
            ("perm", torch.int32, (T * self.k,)))))
        n = B.ds4moe_mx4_workspace_bytes(self.dims, T)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        y = torch.empty((T, self.H), dtype=self.y_dtype, device=dev)
        B.ds4moe_mx4_experts(self.dims, self._weights, x, ldx, T, r, y, ws, n, torch.cuda.current_stream(dev))
        return y


class Mx4Layer:
    """A routed layer on 4-bit experts: router logits (accumulated in fp64, as ds4moe_route), gate, experts."""

    def __init__(self, router_w: torch.Tensor, gate: Gate, experts: Mx4Experts, bias: torch.Tensor | None = None):
        _flat(router_w, "router_w", router_w.dtype, (experts.E, experts.H))
        _need(router_w.dtype in _DTYPES, f"router_w: unsupported type {router_w.dtype}")
        _need((gate.E, gate.k) == (experts.E, experts.k), "gate and experts differ in their numbers of experts or choices")
        self.router_w, self.gate, self.experts, self.bias = router_w, gate, experts, bias
        self._dims = B.make_dims(experts.H, 256, experts.E, 1, 0, B.DS4MOE_BF16, _DTYPES[router_w.dtype])
        _need(B.ds4moe_workspace_bytes(self._dims, 1, B.MODE_ROUTE) > 0,
              f"unsupported router: hidden size {experts.H}, {experts.E} experts")

    def logits(self, x: torch.Tensor) -> torch.Tensor:
        T, dev = x.shape[0], x.device
        _flat(x, "x", torch.bfloat16, (T, self.experts.H))
        out = torch.empty((T, self.experts.E), dtype=torch.float32, device=dev)
        n = B.ds4moe_workspace_bytes(self._dims, T, B.MODE_ROUTE)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
        B.ds4moe_route(self._dims, B.make_weights(self.router_w, None, None, None), x, T, B.make_routing(logits=out),
                       ws, n, torch.cuda.current_stream(dev))
        return out

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return self.experts.forward(x, self.gate.forward(self.logits(x), self.bias))
