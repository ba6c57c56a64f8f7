"""Plain 64-bit implementations of the expert gate and the 4-bit microscaled
operators, from their formulas (numpy, on the CPU; no code of the package)."""
import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
FMAX = float(np.finfo(np.float32).max)


def bf16(x):
    """fp32 values rounded to bf16 (nearest even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isfinite(x), r, np.float32(x)).reshape(np.shape(x))


# ------------------------------------------------------------------ gate
def clean(l):
    l = np.asarray(l, np.float64)
    return np.where(np.isnan(l), -np.inf, np.minimum(l, FMAX))


def scores(l, score):
    l = clean(l)
    with np.errstate(all="ignore"):
        if score == "softmax":
            m = l.max(axis=-1, keepdims=True)
            e = np.exp(l - np.where(np.isinf(m), 0.0, m))
            s = e.sum(axis=-1, keepdims=True)
            return np.where(s > 0, e / np.where(s > 0, s, 1), 0.0)
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        return np.sqrt(np.logaddexp(0.0, l))


def log_scores(l, score):
    """Logarithms of the scores of some logits of a row, up to a number that they share."""
    with np.errstate(all="ignore"):
        if score == "softmax":
            return l
        if score == "sigmoid":
            return -np.logaddexp(0.0, -l)
        return 0.5 * np.where(l < -40.0, l, np.log(np.logaddexp(0.0, l)))


def gate(logits, bias, k, score, G=1, top_groups=1, rank=1, renorm=True, scale=1.0):
    """topk_idx, topk_w, and the smallest relative distance of two keys or group scores that the choice hangs on."""
    l = clean(logits)
    T, E = l.shape
    s = scores(l, score)
    masked = np.isinf(l)
    key = l.copy()
    if bias is not None:
        b = np.asarray(bias, np.float64)
        masked = masked | np.isnan(b) | (b == -np.inf)
        key = s + np.where(np.isnan(b) | (b == -np.inf), 0.0, b)
    gkey = key if bias is not None or rank == 1 else s
    key = np.where(masked, -np.inf, key)
    gkey = np.where(masked, -np.inf, gkey)
    idx, w, gaps = np.zeros((T, k), np.int64), np.zeros((T, k)), np.full(T, np.inf)
    per = E // G
    for t in range(T):
        stay = np.ones(E, bool)
        if G > 1:
            g = np.sort(gkey[t].reshape(G, per), axis=1)[:, ::-1][:, :rank]
            gs = np.where(np.isinf(g[:, 0]) & (g[:, 0] < 0), -np.inf, np.where(np.isinf(g), 0.0, g).sum(axis=1))
            order = np.argsort(-gs, kind="stable")
            stay = np.isin(np.arange(E) // per, order[:top_groups])
            if top_groups < G:
                a, c = gs[order[top_groups - 1]], gs[order[top_groups]]
                if a != c and np.isfinite(a) and np.isfinite(c):
                    gaps[t] = abs(a - c) / max(abs(a), abs(c))
        cand = np.flatnonzero(stay)
        order = cand[np.lexsort((cand, -key[t][cand]))]
        idx[t] = order[:k]
        v = key[t][order[:k + 1]]
        with np.errstate(all="ignore"):
            d = v[:-1] - v[1:]
            ok = (d != 0) & np.isfinite(v[:-1]) & np.isfinite(v[1:])
            rel = d[ok] / np.maximum(np.abs(v[:-1][ok]), 0.05 if bias is not None else 1e-30)
        if bias is not None and rel.size:
            gaps[t] = min(gaps[t], rel.min())
        live = ~masked[t][idx[t]]
        if renorm:  # quotients of the scores by their logarithms: no score underflows
            x = np.where(live, log_scores(l[t][idx[t]], score), -np.inf)
            if live.any():
                e = np.exp(x - x.max())
                w[t] = e / e.sum()
        else:
            w[t] = np.where(live, s[t][idx[t]], 0.0)
    return idx, scale * w, gaps


def gate_gradient(logits, bias, idx, dw, score, renorm, scale):
    """d logits of sum(dw * w), from the Jacobian of every weight written out."""
    l = clean(logits)
    T, E = l.shape
    k = idx.shape[1]
    s = scores(l, score)
    out = np.zeros((T, E))
    for t in range(T):
        J = np.zeros((E, E))  # d s_a / d l_b
        fin = np.isfinite(l[t])
        if score == "softmax":
            J = np.diag(s[t]) - np.outer(s[t], s[t])
        elif score == "sigmoid":
            J = np.diag(s[t] * (1 - s[t]))
        else:
            lf = np.where(fin, l[t], 0.0)
            with np.errstate(all="ignore"):
                J = np.diag(np.where(fin & (s[t] > 0), 1 / (1 + np.exp(-lf)) / np.where(s[t] > 0, 2 * s[t], 1), 0.0))
        live = np.array([0 <= e < E and fin[e] and not (bias is not None and not bias[e] > -np.inf) for e in idx[t]])
        e = np.where(live, idx[t], 0)
        c = np.where(live, s[t][e], 0.0)
        D = np.zeros((k, E))
        S = c.sum()
        for j in range(k):
            if not live[j] or (renorm and S == 0):
                continue
            if renorm:
                D[j] = J[e[j]] / S - c[j] / S**2 * sum(J[e[i]] for i in range(k) if live[i])
            else:
                D[j] = J[e[j]]
        out[t] = scale * (np.asarray(dw[t], np.float64) @ D)
    return out


def permutation(idx, E):
    flat = idx.reshape(-1)
    counts = np.bincount(flat, minlength=E)
    return counts, np.concatenate([[0], np.cumsum(counts)]), np.argsort(flat, kind="stable")


# ------------------------------------------------------------------ 4-bit values
def quantize(x):
    """codes [rows, 16 nb], scales [rows, nb] of [rows, cols], block by block from the definition."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // 32)
    x = np.concatenate([x, np.zeros((rows, nb * 32 - cols))], axis=1).reshape(rows * nb, 32)
    mid = (GRID[:-1] + GRID[1:]) / 2
    bad = ~np.isfinite(x).all(axis=1)
    v = np.where(bad[:, None], 0.0, np.abs(x))
    top = v.max(axis=1)
    e = np.where(top > 0, np.maximum(-127, np.frexp(top)[1] - 1 - 2), -127)
    u = np.ldexp(v, -e[:, None])
    code = np.searchsorted(mid, u, side="left")            # number of midpoints below u
    code += (code < 7) & (u == mid[np.minimum(code, 6)]) & (code % 2 == 1)
    code = (code + 8 * np.where(bad[:, None], False, np.signbit(x))).astype(np.uint8)
    X = np.where(bad, 255, e + 127).astype(np.uint8)
    return (code[:, ::2] | code[:, 1::2] << 4).reshape(rows, nb * 16), X.reshape(rows, nb)


def values(codes, scales):
    """The 64-bit values of codes [..., 16 nb] and scales [..., nb]."""
    c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def experts(x, idx, w, gate_v, up_v, down_v):
    """The routed SwiGLU experts, token by token."""
    y = np.zeros((x.shape[0], down_v.shape[1]))
    for t in range(x.shape[0]):
        for e, a in zip(idx[t], w[t]):
            if 0 <= e < gate_v.shape[0]:
                g, u = gate_v[e] @ x[t], up_v[e] @ x[t]
                y[t] += float(a) * (down_v[e] @ (g / (1 + np.exp(-g)) * u))
    return y
