"""The products grouped by expert, their gradients and the 8-bit integer operators in 64 bits, from their definitions."""
import numpy as np

HALF_STEP = {"f32": 2.0**-24, "bf16": 2.0**-8, "f16": 2.0**-11}  # a rounding's error, relative
TINY = {"f32": 2.0**-150, "bf16": 2.0**-134, "f16": 2.0**-25}    # and absolute, among the subnormals


def quantize(x):
    """Codes (filled up with zeros to a multiple of 16 columns) and fp32 scales of the rows of a float64 matrix."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    top = np.abs(x).max(axis=1) if cols else np.zeros(rows)
    bad = ~np.isfinite(top)
    s = np.float32(np.where(bad, 0, top) / 127)
    s = np.minimum(s, np.float32(8454659 * 2.0**98))  # 127 of the largest scale stay below infinity
    s[(s == 0) & (top > 0) & ~bad] = np.float32(2.0**-149)
    v = np.where(bad[:, None], 0, x) / np.where(s > 0, s, 1).astype(np.float64)[:, None]
    codes = np.zeros((rows, -(-cols // 16) * 16), dtype=np.int8)
    codes[:, :cols] = np.clip(np.rint(v), -127, 127)
    s[bad] = np.nan
    return codes, s


def rows_of(perm, k, T, P):
    """The rows of x of the positions, -1 for none."""
    if perm is None:
        return np.arange(P)
    t = np.asarray(perm, dtype=np.int64) // k
    return np.where((perm >= 0) & (t < T), t, -1)


def gather(x, rows):
    return np.where(rows[:, None] >= 0, x[np.maximum(rows, 0)], 0.0)


def matmul(x, w, offsets, rows):
    """y and the sums of the absolute products."""
    y = np.zeros((rows.size, w.shape[1]))
    mag = np.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        v = gather(x, rows[a:b])
        y[a:b] = v @ w[e].T
        mag[a:b] = np.abs(v) @ np.abs(w[e]).T
    return y, mag


def backward(dy, x, w, offsets, rows):
    """dx, dw and the sums of the absolute products of both."""
    dx, dw = np.zeros_like(x), np.zeros_like(w)
    mx, mw = np.zeros_like(x), np.zeros_like(w)
    for e in range(w.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        keep = np.nonzero(rows[a:b] >= 0)[0] + a
        np.add.at(dx, rows[keep], dy[keep] @ w[e])
        np.add.at(mx, rows[keep], np.abs(dy[keep]) @ np.abs(w[e]))
        dw[e] = dy[keep].T @ x[rows[keep]]
        mw[e] = np.abs(dy[keep]).T @ np.abs(x[rows[keep]])
    return dx, dw, mx, mw


def routing(T, E, k, rng, skew=0.0, unused=()):
    """offsets and perm of T tokens with k distinct experts each, as the gate leaves them."""
    logits = rng.standard_normal((T, E)) - skew * np.log(1 + np.arange(E))
    logits[:, list(unused)] = -np.inf
    flat = np.argsort(-logits, axis=1, kind="stable")[:, :k].reshape(-1)
    counts = np.bincount(flat, minlength=E)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), np.argsort(flat, kind="stable").astype(np.int32)
