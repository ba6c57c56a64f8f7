"""Further operators that perf measures: 8-bit integer quantisation by rows, products with 8-bit integer weights, and products
grouped by expert (16-bit and 8-bit weights) with their gradients.

Each is given in its plain form (elementary torch operations in 32 bits, rounded once at the end) and, where `own` is true, as
the call of this package that a user makes.  `exact` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "int8": 1}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the activations of the long prefill, through 8 bits and back
        {"name": "quantize: 8192 x 4096", "op": "quantize", "rows": 8192, "cols": 4096, "pad": 0, "type": "bf16"},
        # one micro-batch of sessions, rows of a wider buffer, an odd length
        {"name": "quantize: 16 x 1001, rows apart", "op": "quantize", "rows": 16, "cols": 1001, "pad": 24, "type": "f32"},
        # one new token through one projection, its activations quantised on the way: latency
        _product("int8: one token", 1, 2048, 4096, "bf16", "bf16"),
        # a micro-batch of sessions through an odd projection, fp32 results
        _product("int8: 37 tokens, odd", 37, 1001, 2064, "int8", "f32"),
        # a prefill chunk: the matrix cores' rate
        _product("int8: 2048 tokens", 2048, 4096, 4096, "int8", "bf16"),
        # one token through one projection of its 8 of 256 experts: the weights' bytes
        _grouped("grouped: one token", 1, 256, 8, 2048, 4096, "bf16", "bf16", 0.0),
        # a prefill chunk with many experts: about 64 rows each, the weights' bytes
        _grouped("grouped: 2048 tokens, 8 of 256", 2048, 256, 8, 2048, 4096, "bf16", "bf16", 0.0),
        # the long prefill with few experts: the matrix cores' rate
        _grouped("grouped: 8192 tokens, 2 of 8", 8192, 8, 2, 2048, 4096, "bf16", "bf16", 0.0),
        # 8-bit experts, loads as uneven as a router leaves them without a balancing bias
        _grouped("grouped int8: 2048, skewed", 2048, 256, 8, 2048, 4096, "int8", "bf16", 1.0),
        # odd sizes in fp16 with fp32 results
        _grouped("grouped: 1237 tokens, odd, f16", 1237, 60, 3, 1001, 1000, "f16", "f32", 0.75),
        # a training step's gradients: large experts, and many odd ones of which some get no token
        _grouped("gradients: 4096 tokens, 2 of 8", 4096, 8, 2, 2048, 4096, "bf16", "bf16", 0.0, grad=True),
        _grouped("gradients: 1237, odd, skewed", 1237, 60, 3, 488, 1000, "f16", "f16", 1.0, grad=True),
    ]


def _product(name, M, N, K, a, y):
    return {"name": name, "op": "product", "M": M, "N": N, "K": K, "a": a, "y": y}


def _grouped(name, T, E, k, N, K, kind, y, skew, grad=False):
    return {"name": name, "op": "gradients" if grad else "grouped", "T": T, "E": E, "k": k, "N": N, "K": K, "type": kind, "y": y,
            "skew": skew}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "grouped", "grouped", "gradients", "gradients"))
    if op == "quantize":
        cols = _log(rng, 16, 16384)
        rows = max(1, min(_log(rng, 1, 32768), (1 << 25) // cols))
        c = {"op": op, "rows": rows, "cols": cols, "pad": rng.choice((0, 0, rng.randint(1, 40))),
             "type": rng.choice(("f32", "bf16", "f16"))}
    elif op == "product":
        N, K = _log(rng, 16, 8192), 16 * _log(rng, 1, 512)
        M = max(1, min(_log(rng, 1, 8192), int(6e10 / (N * K))))
        c = _product("", M, N, K, rng.choice(("int8", "int8", "bf16", "f16", "f32")), rng.choice(("bf16", "f16", "f32")))
    else:
        grad = op == "gradients"
        N, K = 8 * _log(rng, 8, 512), 16 * _log(rng, 4, 256)
        E = max(1, min(_log(rng, 1, 256), int(2e9 / (N * K)) if not grad else int(2e8 / (N * K))))
        k = rng.randint(1, min(8, E))
        T = max(1, min(_log(rng, 1, 8192), int((6e10 if grad else 1.2e11) / (k * N * K))))
        kind = rng.choice(("bf16", "f16") if grad else ("bf16", "f16", "int8"))
        if not grad:
            N += rng.choice((0, 0, rng.randint(1, 7)))
        c = _grouped("", T, E, k, N, K, kind, kind if grad else rng.choice(("f32", "bf16" if kind == "int8" else kind)),
                     rng.choice((0.0, 0.75, 1.0)), grad)
    c.pop("name", None)
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] == "quantize":
        # activations: normal, with a spread of magnitudes over the channels as after a norm's gain
        x = torch.randn(c["rows"], c["cols"] + c["pad"], generator=g, device=DEV)
        x *= torch.exp(0.5 * torch.randn(c["cols"] + c["pad"], generator=g, device=DEV))
        s["x"] = x.to(TYPES[c["type"]])[:, :c["cols"]]
    elif c["op"] == "product":
        a = torch.randn(c["M"], c["K"], generator=g, device=DEV)
        s["a"], s["a_scales"] = _int8(a) if c["a"] == "int8" else (a.to(TYPES[c["a"]]), None)
        w, scales = _matrices(1, c["N"], c["K"], "int8", g)
        s["w"], s["w_scales"] = w[0], scales[0]
    else:
        T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
        x = torch.randn(T, K, generator=g, device=DEV)
        s["x"], s["x_scales"] = _int8(x) if c["type"] == "int8" else (x.to(TYPES[c["type"]]), None)
        s["w"], s["w_scales"] = _matrices(E, N, K, c["type"], g)
        # what the router leaves: uniform loads, or Zipf(1.1) ones scaled by `skew`
        rank = torch.argsort(torch.rand(E, generator=g, device=DEV)).float() + 1
        logits = torch.randn(T, E, generator=g, device=DEV) - 1.1 * c["skew"] * torch.log(rank)
        flat = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k].reshape(-1)
        counts = torch.bincount(flat, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), torch.cumsum(counts, 0)]).to(torch.int32)
        s["perm"] = torch.sort(flat, stable=True)[1].to(torch.int32)
        s["bounds"] = s["offsets"].tolist()  # on the host, for the plain form's loop over the experts
        if c["op"] == "gradients":
            s["dy"] = torch.randn(T * k, N, generator=g, device=DEV).to(TYPES[c["type"]])
    return s


def _matrices(n, rows, cols, kind, g):
    """n matrices of normal weights (sigma 0.02, the channels' magnitudes spread a little), and the channels' scales of 8-bit ones."""
    w = torch.empty(n, rows, cols, dtype=torch.int8 if kind == "int8" else TYPES[kind], device=DEV)
    scales = torch.empty(n, rows, device=DEV) if kind == "int8" else None
    step = max(1, (1 << 26) // (rows * cols))
    for i in range(0, n, step):
        m = min(step, n - i)
        v = 0.02 * torch.randn(m * rows, cols, generator=g, device=DEV)
        v *= torch.exp(0.3 * torch.randn(m * rows, 1, generator=g, device=DEV))
        if kind == "int8":
            codes, sc = _int8(v)
            w[i:i + m], scales[i:i + m] = codes.view(m, rows, cols), sc.view(m, rows)
        else:
            w[i:i + m] = v.to(w.dtype).view(m, rows, cols)
    return w, scales


# ------------------------------------------------------------------ plain forms
def run(state):
    return OWN[state["case"]["op"]](state) if own else PLAIN[state["case"]["op"]](state)


def _int8(x):
    """Codes and the rows' scales: max / 127 rounded to fp32, and the nearest multiples, ties to even (in 64 bits: next to a
    border an fp32 quotient falls on the wrong side)."""
    x = x.double()
    top = x.abs().amax(1)
    scales = (top / 127).float()
    scales = torch.where((scales == 0) & (top > 0), torch.full_like(scales, 2.0 ** -149), scales)
    unit = torch.where(scales > 0, scales, torch.ones_like(scales)).double()
    return torch.clamp(torch.round(x / unit[:, None]), -127, 127).to(torch.int8), scales


def _quantize_plain(s):
    codes, scales = _int8(s["x"])
    return (codes.float() * scales[:, None]).to(s["x"].dtype)


def _product_plain(s):
    codes, scales = (s["a"], s["a_scales"]) if s["a_scales"] is not None else _int8(s["a"])
    y = codes.float() @ s["w"].float().t()
    return (y * scales[:, None] * s["w_scales"][None, :]).to(TYPES[s["case"]["y"]])


def _rows_of(s):
    return s["perm"].long() // s["case"]["k"]


def _segments(s):
    return [(e, a, b) for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])) if b > a]


def _grouped_plain(s):
    rows = _rows_of(s)
    x = s["x"].float()[rows]
    y = torch.empty(x.shape[0], s["case"]["N"], device=x.device)
    for e, a, b in _segments(s):
        v = x[a:b] @ s["w"][e].float().t()
        y[a:b] = v if s["w_scales"] is None else v * s["x_scales"][rows[a:b], None] * s["w_scales"][e][None, :]
    return y.to(TYPES[s["case"]["y"]])


def _gradients_plain(s):
    rows, k = _rows_of(s), s["case"]["k"]
    x, dy = s["x"].float()[rows], s["dy"].float()
    dx, dw = torch.empty_like(x), torch.zeros(s["w"].shape, device=x.device)
    for e, a, b in _segments(s):
        dx[a:b] = dy[a:b] @ s["w"][e].float()
        dw[e] = dy[a:b].t() @ x[a:b]
    by_choice = torch.empty_like(dx).index_copy_(0, s["perm"].long(), dx)
    return {"dx": by_choice.view(-1, k, dx.shape[1]).sum(1).to(s["x"].dtype), "dw": dw.to(s["w"].dtype)}


PLAIN = {"quantize": _quantize_plain, "product": _product_plain, "grouped": _grouped_plain, "gradients": _gradients_plain}


# ------------------------------------------------------------------ the package's calls
def _quantize_own(s):
    import quantized_routed_moe_router_amd as q
    codes, scales = q.int8_quantize(s["x"])
    return q.int8_dequantize(codes, scales, s["x"].shape[1], s["x"].dtype)


def _product_own(s):
    import quantized_routed_moe_router_amd as q
    return q.int8_matmul(s["a"], s["w"], s["w_scales"], s["a_scales"], y_dtype=TYPES[s["case"]["y"]])


def _grouped_own(s):
    import quantized_routed_moe_router_amd as q
    return q.grouped_matmul(s["x"], s["w"], s["offsets"], s["perm"], s["case"]["k"], x_scales=s["x_scales"], w_scales=s["w_scales"],
                            y_dtype=TYPES[s["case"]["y"]])


def _gradients_own(s):
    import quantized_routed_moe_router_amd as q
    dx, dw = q.grouped_matmul_backward(s["dy"], s["x"], s["w"], s["offsets"], s["perm"], s["case"]["k"])
    return {"dx": dx, "dw": dw}


OWN = {"quantize": _quantize_own, "product": _product_own, "grouped": _grouped_own, "gradients": _gradients_own}


# ------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"]
        return {"bytes": 2 * n * SIZE[c["type"]], "flops": 4 * n}
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K * SIZE[c["a"]] + N * K + 4 * N + M * N * SIZE[c["y"]], "flops": 2 * M * N * K}
    T, E, k, N, K = (c[n] for n in ("T", "E", "k", "N", "K"))
    used = E * (1 - (1 - k / E) ** T)  # distinct experts of even loads
    size = SIZE[c["type"]]
    if c["op"] == "grouped":
        return {"bytes": used * N * K * size + T * K * size + T * k * (N * SIZE[c["y"]] + 4), "flops": 2 * T * k * N * K}
    return {"bytes": ((used + E) * N * K + 2 * T * K + T * k * N) * size + 4 * T * k, "flops": 4 * T * k * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))


def _exact_codes(x):
    """The 8-bit values of a matrix, as multiples of its rows' fp32 scales."""
    x = x.double()
    scale = (x.abs().max(dim=1, keepdim=True)[0] / 127).float().double()
    v = x / scale
    low = torch.floor(v)
    up = (v - low > 0.5) | ((v - low == 0.5) & (low % 2 != 0))
    return low + up.double(), scale


def _exact_quantize(s):
    codes, scale = _exact_codes(s["x"])
    return codes * scale


def _exact_product(s):
    codes, scale = _exact_codes(s["a"]) if s["a_scales"] is None else (s["a"].double(), s["a_scales"].double()[:, None])
    return torch.matmul(codes * scale, (s["w"].double() * s["w_scales"].double()[:, None]).t())


def _exact_matrix(s, e):
    w = s["w"][e].double()
    return w if s["w_scales"] is None else w * s["w_scales"][e].double()[:, None]


def _exact_grouped(s):
    c = s["case"]
    x = s["x"].double() if s["x_scales"] is None else s["x"].double() * s["x_scales"].double()[:, None]
    token = torch.div(s["perm"].long(), c["k"], rounding_mode="floor")
    expert = torch.searchsorted(s["offsets"].long(), torch.arange(token.numel(), device=token.device), right=True) - 1
    y = torch.zeros(token.numel(), c["N"], dtype=torch.float64, device=x.device)
    for e in torch.unique(expert).tolist():
        p = torch.nonzero(expert == e)[:, 0]
        y[p] = x[token[p]] @ _exact_matrix(s, e).t()
    return y


def _exact_gradients(s):
    c = s["case"]
    x, dy = s["x"].double(), s["dy"].double()
    token = torch.div(s["perm"].long(), c["k"], rounding_mode="floor")
    expert = torch.searchsorted(s["offsets"].long(), torch.arange(token.numel(), device=token.device), right=True) - 1
    dx, dw = torch.zeros_like(x), torch.zeros(s["w"].shape, dtype=torch.float64, device=x.device)
    for e in torch.unique(expert).tolist():
        p = torch.nonzero(expert == e)[:, 0]
        dx[token[p]] += dy[p] @ s["w"][e].double()  # an expert's tokens are distinct
        dw[e] = torch.matmul(dy[p].t().contiguous(), x[token[p]])
    return {"dx": dx, "dw": dw}


EXACT = {"quantize": _exact_quantize, "product": _exact_product, "grouped": _exact_grouped, "gradients": _exact_gradients}
