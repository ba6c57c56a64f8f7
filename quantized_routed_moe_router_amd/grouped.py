"""8-bit integer operators and products grouped by expert, with their gradients, on torch tensors.

Plumbing around the C ABI only, as for the 4-bit operators: shapes, types and devices are checked here, torch allocates
outputs and workspaces (on the current stream), and every step runs in libds4moe.so, on the device of the call's tensors
and its current stream.
Nothing here is recorded by autograd: a tensor that requires a gradient, the fp32 scales of 8-bit integers too, is
refused while gradients are on.  grouped_matmul_backward is the gradient that there is; it takes operands that require
one, and its results carry none.
A matrix of 8-bit integers is a pair: int8 codes [rows, K16], K16 the columns rounded up to a multiple of 16, and fp32
scales [rows].
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B
from .mx4 import _call, _elsewhere, _empty, _flat, _rows

_L = B.lib()
_REAL = {torch.float32: B.DS4MOE_F32, torch.bfloat16: B.DS4MOE_BF16, torch.float16: B.DS4MOE_F16}
_HALF = {torch.bfloat16: B.DS4MOE_BF16, torch.float16: B.DS4MOE_F16}
_TYPES = {**_REAL, torch.int8: B.DS4MOE_I8}
_INT8 = (torch.int8,)
_byref = ctypes.byref


def _tracked(what: str, instead: str) -> None:
    if torch.is_grad_enabled():
        raise ValueError(f"{what} asks for a gradient, which autograd does not get from this call: detach it, or call "
                         f"under torch.no_grad(){instead}")


def _here(t: torch.Tensor, what: str, i: int) -> None:
    if t.get_device() != i:
        _elsewhere(t, what, i)


def _real(dtype, what: str) -> int:
    if dtype not in _REAL:
        raise ValueError(f"{what}: fp32, bf16 or fp16 is wanted, not {dtype}")
    return _REAL[dtype]


def int8_quantize(x: torch.Tensor) -> tuple:
    """(codes, scales) of a matrix [rows, cols] in fp32, bf16 or fp16: rows' largest magnitude / 127, nearest integers;
    columns are filled up with zeros to a multiple of 16."""
    if x.requires_grad:
        _tracked("x", "")
    ld, i = _rows(x, "x", _REAL), x.get_device()
    rows, cols = x.shape
    codes = _empty(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device=i)
    scales = _empty(rows, dtype=torch.float32, device=i)
    if cols == 0:
        scales.zero_()
    _call(_L.ds4moe_int8_quantize, "int8_quantize", i, codes.data_ptr(), scales.data_ptr(), x.data_ptr(), _REAL[x.dtype],
          rows, cols, ld)
    return codes, scales


def int8_dequantize(codes: torch.Tensor, scales: torch.Tensor, cols: int | None = None,
                    dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The values of a matrix of 8-bit integers, the first `cols` of each row (all by default)."""
    if scales.requires_grad:
        _tracked("scales", "")
    i, kind = codes.get_device(), _real(dtype, "dtype")
    _flat(codes, "codes", torch.int8)
    if codes.dim() != 2 or codes.shape[1] % 16:
        raise ValueError("codes: a matrix of whole blocks of 16 is wanted")
    rows, K = codes.shape
    _flat(scales, "scales", torch.float32, (rows,), i)
    cols = K if cols is None else cols
    if (cols + 15) // 16 * 16 != K:
        raise ValueError(f"{cols} columns are not {K // 16} blocks of 16")
    out = _empty(rows, cols, dtype=dtype, device=i)
    _call(_L.ds4moe_int8_dequantize, "int8_dequantize", i, out.data_ptr(), kind, cols, codes.data_ptr(), scales.data_ptr(),
          rows, cols)
    return out


def int8_matmul(a: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, a_scales: torch.Tensor | None = None,
                y_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """a [M,K] times w [N,K16]^T times both scales: w in 8-bit integers, a too (with a_scales), or in fp32, bf16 or fp16,
    which the call quantises row by row."""
    if a.requires_grad or w_scales.requires_grad or (a_scales is not None and a_scales.requires_grad):
        _tracked("a or a scale", "")
    kind, i = _real(y_dtype, "y_dtype"), w.get_device()
    _flat(w, "w", torch.int8)
    if w.dim() != 2 or w.shape[1] % 16:
        raise ValueError("w: a matrix of whole blocks of 16 columns is wanted")
    N, K16 = w.shape
    _flat(w_scales, "w_scales", torch.float32, (N,), i)
    lda = _rows(a, "a", _REAL if a_scales is None else _INT8)
    M, K = a.shape
    if (K + 15) // 16 * 16 != K16 or (a_scales is not None and K != K16):
        raise ValueError(f"a: {K} columns, w has {K16}")
    _here(a, "a", i)
    if a_scales is None:
        n = _L.ds4moe_int8_workspace_bytes(M, K, _REAL[a.dtype])
        ws = _empty(n, dtype=torch.uint8, device=i)
        sa, space = None, ws.data_ptr()
    else:
        sa, space, n = _flat(a_scales, "a_scales", torch.float32, (M,), i).data_ptr(), None, 0
    y = _empty(M, N, dtype=y_dtype, device=i)
    _call(_L.ds4moe_int8_matmul, "int8_matmul", i, y.data_ptr(), kind, N, a.data_ptr(), sa, _TYPES[a.dtype], lda, w.data_ptr(),
          w_scales.data_ptr(), M, N, K, space, n)
    return y


def _groups(w: torch.Tensor, offsets: torch.Tensor, perm, k: int, tokens: int, types) -> tuple:
    """E, N, K, positions, device and the permutation's address, all checked."""
    i = w.get_device()
    if w.dtype not in types or w.dim() != 3 or i < 0 or not w.is_contiguous():
        raise ValueError("w: contiguous matrices [E, N, K] on the GPU are wanted, in " +
                         ", ".join(str(t)[6:] for t in types))
    E, N, K = w.shape
    _flat(offsets, "offsets", torch.int32, (E + 1,), i)
    if perm is None:
        if k != 1:
            raise ValueError(f"k = {k} without a permutation")
        return E, N, K, tokens, i, None
    _flat(perm, "perm", torch.int32, None, i)
    if perm.dim() != 1:
        raise ValueError("perm: one index per position is wanted")
    return E, N, K, perm.shape[0], i, perm.data_ptr()


def grouped_matmul(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, perm: torch.Tensor | None = None, k: int = 1, *,
                   x_scales: torch.Tensor | None = None, w_scales: torch.Tensor | None = None,
                   y_dtype: torch.dtype | None = None) -> torch.Tensor:
    """y [P,N], y[p] = w[e] x[perm[p] // k] for offsets[e] <= p < offsets[e+1]: x [T,K], w [E,N,K], offsets [E+1] and perm
    [P] as Gate.forward leaves them, perm None for rows that are in order already.  x and w in bf16 or fp16, or both in
    8-bit integers with x_scales [T] and w_scales [E,N].  Positions of no expert come back as zeros.  y_dtype: x's, or
    bf16 of 8-bit integers, by default."""
    if x.requires_grad or w.requires_grad:
        _tracked("x or w", " (grouped_matmul_backward gives the gradients)")
    ldx = _rows(x, "x", _TYPES)
    T = x.shape[0]
    E, N, K, P, i, at = _groups(w, offsets, perm, k, T, (x.dtype,))
    if x.shape[1] != K:
        raise ValueError(f"x: {x.shape[1]} columns, w has {K}")
    _here(x, "x", i)
    if x.dtype is torch.int8:
        if x_scales is None or w_scales is None:
            raise ValueError("8-bit integers want x_scales and w_scales")
        if x_scales.requires_grad or w_scales.requires_grad:
            _tracked("x_scales or w_scales", "")
        sx = _flat(x_scales, "x_scales", torch.float32, (T,), i).data_ptr()
        sw = _flat(w_scales, "w_scales", torch.float32, (E, N), i).data_ptr()
        y_dtype = torch.bfloat16 if y_dtype is None else y_dtype
    else:
        if x.dtype is torch.float32 or x_scales is not None or w_scales is not None:
            raise ValueError("x: bf16 or fp16 without scales is wanted, or 8-bit integers with them")
        sx = sw = None
        y_dtype = x.dtype if y_dtype is None else y_dtype
    kind = _real(y_dtype, "y_dtype")
    y = _empty(P, N, dtype=y_dtype, device=i)
    if P == 0 or T == 0:
        return y.zero_()
    dims = B.GroupedDims(_TYPES[x.dtype], kind, E, k, P, T, N, K)
    _call(_L.ds4moe_grouped_matmul, "grouped_matmul", i, _byref(dims), y.data_ptr(), N, x.data_ptr(), ldx, sx, w.data_ptr(),
          sw, offsets.data_ptr(), at)
    return y


def grouped_matmul_backward(dy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                            perm: torch.Tensor | None = None, k: int = 1, *, need_dx: bool = True, need_dw: bool = True,
                            dw_dtype: torch.dtype | None = None) -> tuple:
    """(dx [T,K] in x's type, dw [E,N,K] in w's or dw_dtype) from dy [P,N], the gradient of grouped_matmul(x, w, offsets,
    perm, k); None in the place of one that is not asked for.  x, w and dy in bf16 or fp16, N a multiple of 8.  A value
    of perm may stand several times (tokens' numbers with k = 1, say): every position of an expert adds to dx."""
    ldy, ldx = _rows(dy, "dy", _HALF), _rows(x, "x", _HALF)
    T = x.shape[0]
    E, N, K, P, i, at = _groups(w, offsets, perm, k, T, (x.dtype,))
    if x.shape[1] != K:
        raise ValueError(f"x: {x.shape[1]} columns, w has {K}")
    if dy.dtype != x.dtype or dy.shape != (P, N):
        raise ValueError(f"dy: {dy.dtype} {tuple(dy.shape)}, not {x.dtype} {(P, N)}")
    if N % 8:
        raise ValueError(f"w: {N} rows, a multiple of 8 is wanted")
    _here(x, "x", i)
    _here(dy, "dy", i)
    dw_dtype = w.dtype if dw_dtype is None else dw_dtype
    kind, half = _real(dw_dtype, "dw_dtype"), _HALF[x.dtype]
    dx = dw = None
    if need_dx:
        dx = _empty(T, K, dtype=x.dtype, device=i)
        if P == 0 or T == 0:
            dx.zero_()
        else:
            dims = B.GroupedDims(half, half, E, k, P, T, N, K)
            n, ws = 0, None
            if perm is not None:
                n = _L.ds4moe_grouped_workspace_bytes(_byref(dims))
                ws = _empty(n, dtype=torch.uint8, device=i)
            _call(_L.ds4moe_grouped_dx, "grouped_dx", i, _byref(dims), dx.data_ptr(), K, dy.data_ptr(), ldy, w.data_ptr(),
                  offsets.data_ptr(), at, None if ws is None else ws.data_ptr(), n)
    if need_dw:
        dw = _empty(E, N, K, dtype=dw_dtype, device=i)
        if P == 0 or T == 0:
            dw.zero_()
        else:
            dims = B.GroupedDims(half, kind, E, k, P, T, N, K)
            _call(_L.ds4moe_grouped_dw, "grouped_dw", i, _byref(dims), dw.data_ptr(), dy.data_ptr(), ldy, x.data_ptr(), ldx,
                  offsets.data_ptr(), at)
    return dx, dw
