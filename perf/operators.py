"""Cases and plain forms of three operators: products of 8-bit integers with a scale for each token
and each output channel (the tokens quantized on the way in), and the routed expert layer of a
decode step, router included.

    linear   Y = X W^T with X quantized to int8 rows (one scale per token), W int8 rows (one scale
             per output channel): quantize_rows_i8, then qgemm_i8
    product  the same product from tokens that are int8 already: qgemm_i8
    moe      router logits, softmax, top-k, renormalised weights, gated experts, shared expert:
             moe_layer, for 1 to 8 tokens

With `own` false, run() computes them with elementary torch operations; with `own` true it calls
the package.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
Q8_0, Q4_0, I4_ROW, I2_ROW = 1, 2, 3, 4
GELU_TANH, SILU = 1, 2
TINY_SCALE = 2.0 ** -100  # a row whose scale would be below this is held as zeros


# ---------------------------------------------------------------- cases
def _linear(name, tokens, k, n, dtype, out, bias=False, pad=0):
    return {"name": name, "op": "linear", "tokens": tokens, "k": k, "n": n, "dtype": dtype, "out": out, "bias": bias,
            "pad": pad}


def _product(name, tokens, k, n, out, bias=False):
    return {"name": name, "op": "product", "tokens": tokens, "k": k, "n": n, "out": out, "bias": bias}


def _moe(name, tokens, hidden, experts, top_k, inter, fmt, act, shared=0, shared_fmt=0):
    return {"name": name, "op": "moe", "tokens": tokens, "hidden": hidden, "experts": experts, "top_k": top_k,
            "inter": inter, "fmt": fmt, "act": act, "shared": shared, "shared_fmt": shared_fmt}


def listed():
    return [
        # one decoded token through a small key/value projection: latency is all there is
        _linear("linear_1x2048x256", 1, 2048, 256, "bf16", "bf16"),
        # one decoded token through the widest projection: the weight stream counts
        _linear("linear_1x4096x14336", 1, 4096, 14336, "f16", "f16"),
        # a ragged batch of sequences, channels and width off every tile, with a bias and a row pitch
        _linear("linear_100x2051x1000_bias", 100, 2051, 1000, "bf16", "bf16", True, 5),
        # a prefill chunk of 128 tokens
        _linear("linear_128x4096x14336", 128, 4096, 14336, "f16", "f16"),
        # a long prompt into a narrow projection: the quantization of the tokens weighs most
        _linear("linear_8192x4096x1024", 8192, 4096, 1024, "bf16", "bf16"),
        # a few sequences decoded together, fp32 logits
        _product("product_24x4096x4096", 24, 4096, 4096, "f32"),
        # a long prompt through the widest projection: the integer tensor cores count
        _product("product_8192x4096x14336", 8192, 4096, 14336, "bf16"),
        # a small layer, one token: latency is all there is
        _moe("moe_small_t1", 1, 512, 16, 2, 256, Q8_0, SILU),
        # the 128-expert layer with a shared expert: one token, and a few sequences at once
        _moe("moe_128e_t1", 1, 2816, 128, 8, 704, Q4_0, GELU_TANH, 2112, Q8_0),
        _moe("moe_128e_t5", 5, 2816, 128, 8, 704, Q4_0, GELU_TANH, 2112, Q8_0),
        # the 256-expert int4 layer: one token, and the most tokens of the call
        _moe("moe_256e_t1", 1, 6144, 256, 8, 2048, I4_ROW, SILU),
        _moe("moe_256e_t8", 8, 6144, 256, 8, 2048, I4_ROW, SILU),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "product", "moe"])
    if op != "moe":
        while True:
            tokens, k, n = _log(rng, 1, 8192), _log(rng, 32, 8192), _log(rng, 8, 14336)
            if tokens * k * n <= 8192 * 4096 * 14336:
                break
        out, bias = rng.choice(["f32", "f16", "bf16"]), rng.random() < 0.5
        if op == "product":
            return {"op": op, "tokens": tokens, "k": k, "n": n, "out": out, "bias": bias}
        return {"op": op, "tokens": tokens, "k": k, "n": n, "dtype": rng.choice(["f32", "f16", "bf16"]), "out": out,
                "bias": bias, "pad": rng.choice([0, 0, rng.randint(1, 40)])}
    fmt = rng.choice([Q8_0, Q4_0, I4_ROW, I2_ROW])
    shared_fmt = rng.choice([0, Q8_0, Q4_0, I4_ROW, I2_ROW])
    step = 64 if I2_ROW in (fmt, shared_fmt) else 32
    hidden, inter = (step * _log(rng, 256 // step, 4096 // step) for _ in range(2))
    experts = _log(rng, 4, 256)
    while experts * inter * hidden > 128 * 1024 * 2816:
        experts //= 2
    experts = max(experts, 2)
    return {"op": op, "tokens": rng.randint(1, 8), "hidden": hidden, "experts": experts,
            "top_k": rng.randint(1, min(8, experts)), "inter": inter, "fmt": fmt, "act": rng.choice([GELU_TANH, SILU]),
            "shared": step * _log(rng, 128 // step, 2816 // step) if shared_fmt else 0, "shared_fmt": shared_fmt}


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _uniform(g, shape, lo, hi):
    return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo


def _row_bytes(fmt, cols):
    return {Q8_0: cols // 32 * 34, Q4_0: cols // 32 * 18, I4_ROW: cols // 2, I2_ROW: cols // 4}[fmt]


def _matrix_bytes(fmt, rows, cols):
    n = rows * _row_bytes(fmt, cols)
    return n if fmt in (Q8_0, Q4_0) else (n + 15) // 16 * 16 + 4 * rows


def _matrices(g, fmt, count, rows, cols):
    """`count` matrices in the library's byte layout, one after another at a stride of whole 16 bytes."""
    size = _matrix_bytes(fmt, rows, cols)
    stride = (size + 15) // 16 * 16
    W = torch.randint(0, 256, (count, stride), generator=g, device="cuda", dtype=torch.uint8)
    packed = rows * _row_bytes(fmt, cols)
    if fmt in (Q8_0, Q4_0):
        blocks = W[:, :packed].unflatten(1, (rows * cols // 32, -1))
        d = _uniform(g, (count, rows * cols // 32, 1), 1e-3, 1e-2).half()
        blocks[..., :2] = d.view(torch.uint8)
        if fmt == Q8_0:
            q = blocks[..., 2:]
            q.masked_fill_(q == 128, 0)  # int8 values in [-127, 127]
    else:
        d = _uniform(g, (count, rows), 1e-3, 1e-2)
        at = (packed + 15) // 16 * 16
        W[:, packed:at] = 0
        W[:, at:at + 4 * rows] = d.view(torch.uint8)
    return W.reshape(-1), stride


def _int8_rows(g, rows, k):
    """int8 rows of Gaussian values as a quantizer leaves them, at a pitch of whole 16 bytes."""
    pitch = (k + 15) // 16 * 16
    q = torch.empty(rows, pitch, dtype=torch.int8, device="cuda")
    q[:, :k] = (torch.randn(rows, k, generator=g, device="cuda") * 32).round_().clamp_(-127, 127)
    q[:, k:] = 99  # what lies between the rows belongs to nobody
    return q[:, :k]


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] != "moe":
        tokens, k, n = case["tokens"], case["k"], case["n"]
        s = {"case": case, "W": _int8_rows(g, n, k), "sw": _uniform(g, (n,), 1e-4, 1e-3),
             "bias": torch.randn(n, generator=g, device="cuda") if case["bias"] else None}
        if case["op"] == "linear":
            # activations with a few channels that stand out, as a transformer's do
            gain = 1 + 12 * (torch.rand(k, generator=g, device="cuda") < 0.01)
            X = torch.empty(tokens, k + case["pad"], dtype=DTYPES[case["dtype"]], device="cuda")
            X[:, :k] = torch.randn(tokens, k, generator=g, device="cuda") * gain
            X[:, k:] = 1e4
            s["X"] = X[:, :k]
        else:
            s["X"], s["sx"] = _int8_rows(g, tokens, k), _uniform(g, (tokens,), 0.01, 0.05)
        return s
    T, H, E, I, fmt = case["tokens"], case["hidden"], case["experts"], case["inter"], case["fmt"]
    gate, gs = _matrices(g, fmt, E, I, H)
    up, us = _matrices(g, fmt, E, I, H)
    down, ds = _matrices(g, fmt, E, H, I)
    s = {"case": case, "experts": ((gate, gs), (up, us), (down, ds)), "shared": None,
         "R": torch.randn(E, H, generator=g, device="cuda") * 0.02, "x": torch.randn(T, H, generator=g, device="cuda")}
    if case["shared"]:
        S, f = case["shared"], case["shared_fmt"]
        s["shared"] = tuple(_matrices(g, f, 1, r, c)[0] for r, c in ((S, H), (S, H), (H, S)))
    if own:  # the layer's handle and workspace, which a program makes once, at start-up
        import block_quant_gemv_b200 as bqg
        shared = None if s["shared"] is None else (case["shared_fmt"], case["shared"]) + s["shared"]
        s["layer"] = bqg.MoELayer(E, case["top_k"], H, I, fmt, case["act"], gate, up, down, gs, us, ds, shared)
        s["workspace"] = bqg.moe_layer_workspace(s["layer"], T, "cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if own:
        import block_quant_gemv_b200 as bqg
        if op == "moe":
            y, idx, w = bqg.moe_layer(s["layer"], s["R"], s["x"], workspace=s["workspace"])
            return {"y": y, "idx": idx, "w": w}
        out = DTYPES[s["case"]["out"]]
        if op == "product":
            return {"y": bqg.qgemm_i8(s["X"], s["sx"], s["W"], s["sw"], out_dtype=out, bias=s["bias"])}
        q, sx = bqg.quantize_rows_i8(s["X"])
        return {"y": bqg.qgemm_i8(q, sx, s["W"], s["sw"], out_dtype=out, bias=s["bias"]), "scale": sx}
    if op == "moe":
        return _plain_moe(s)
    if op == "product":
        return {"y": _plain_product(s, s["X"], s["sx"])}
    q, sx = _plain_quantize(s["X"])
    return {"y": _plain_product(s, q, sx), "scale": sx}


def _plain_quantize(X):
    x = X.float()
    most = x.abs().amax(1)
    scale = (most.double() / 127).float()  # rounded once
    scale = torch.where(scale < TINY_SCALE, torch.zeros_like(scale), scale)
    scale = torch.where(torch.isfinite(most), scale, torch.full_like(scale, math.nan))
    # the quotient in 64 bits: values next to a border between two integers
    q = torch.round(x.double() / scale.double()[:, None])
    q = torch.where((scale > 0)[:, None], q, torch.zeros_like(q))
    return q.to(torch.int8), scale


def _plain_product(s, q, sx):
    y = q.float() @ s["W"].float().T
    y = y * sx[:, None] * s["sw"][None, :]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(DTYPES[s["case"]["out"]])


def _decode(W, fmt, rows, cols):
    """fp32 [count, rows, cols] of byte matrices W [count, >= matrix bytes]."""
    packed = rows * _row_bytes(fmt, cols)
    b = W[:, :packed]
    if fmt in (Q8_0, Q4_0):
        b = b.unflatten(1, (rows, cols // 32, -1))
        d = b[..., :2].contiguous().view(torch.float16).float()
        q = b[..., 2:]
        if fmt == Q8_0:
            v = q.contiguous().view(torch.int8).float()
        else:
            v = torch.stack((q & 15, q >> 4), -1).flatten(-2).float() - 8
        return (v * d).flatten(-2)
    at = (packed + 15) // 16 * 16
    scale = W[:, at:at + 4 * rows].contiguous().view(torch.float32)
    b = b.unflatten(1, (rows, -1))
    if fmt == I4_ROW:
        v = torch.stack((b & 15, b >> 4), -1).flatten(-2).to(torch.int8)
        v = v - 16 * (v > 7)
    else:
        v = torch.stack((b & 3, (b >> 2) & 3, (b >> 4) & 3, b >> 6), -1).flatten(-2).to(torch.int8)
        v = v - 4 * (v > 1)
    return v.float() * scale[..., None]


def _act(kind, g):
    if kind == SILU:
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))


def _plain_moe(s):
    c = s["case"]
    T, H, I, k, fmt = c["tokens"], c["hidden"], c["inter"], c["top_k"], c["fmt"]
    x = s["x"]
    # 64 bits up to the choice of experts: logits next to one another
    logits = x.double() @ s["R"].double().T
    best, order = torch.sort(logits, dim=1, descending=True, stable=True)
    idx = order[:, :k]
    p = torch.exp(best - best[:, :1])
    p = p / p.sum(1, keepdim=True)
    w = p[:, :k] / p[:, :k].sum(1, keepdim=True)
    pairs = idx.reshape(-1)
    xs = x.repeat_interleave(k, 0)[:, :, None]
    (gate, gs), (up, us), (down, ds) = s["experts"]
    g = (_decode(gate.view(-1, gs)[pairs], fmt, I, H) @ xs)
    u = (_decode(up.view(-1, us)[pairs], fmt, I, H) @ xs)
    o = _decode(down.view(-1, ds)[pairs], fmt, H, I) @ (_act(c["act"], g) * u)
    y = (o.view(T, k, H) * w.float()[:, :, None]).sum(1)
    if s["shared"] is not None:
        S, f = c["shared"], c["shared_fmt"]
        sg, su, sd = (_decode(m[None], f, r, q)[0] for m, r, q in zip(s["shared"], (S, S, H), (H, H, S)))
        y = y + (_act(c["act"], x @ sg.T) * (x @ su.T)) @ sd.T
    return {"y": y, "idx": idx.to(torch.int32), "w": w.float()}


# ---------------------------------------------------------------- the work of one pass
def work(case):
    if case["op"] != "moe":
        t, k, n = case["tokens"], case["k"], case["n"]
        size = {"f32": 4, "f16": 2, "bf16": 2}
        read = t * k * size[case["dtype"]] if case["op"] == "linear" else t * k + 4 * t
        wrote = t * n * size[case["out"]] + (4 * t if case["op"] == "linear" else 0)
        return {"bytes": read + n * k + 4 * n + (4 * n if case["bias"] else 0) + wrote, "flops": 2 * t * n * k}
    T, H, E, k, I = case["tokens"], case["hidden"], case["experts"], case["top_k"], case["inter"]
    touched = E * (1 - (1 - k / E) ** T)  # different experts that T tokens choose, on average
    expert = 2 * _matrix_bytes(case["fmt"], I, H) + _matrix_bytes(case["fmt"], H, I)
    flops = 2 * T * E * H + 6 * T * k * I * H
    size = touched * expert + 4 * E * H + 8 * T * H + 8 * T * k
    if case["shared"]:
        S, f = case["shared"], case["shared_fmt"]
        size += 2 * _matrix_bytes(f, S, H) + _matrix_bytes(f, H, S)
        flops += 6 * T * S * H
    return {"bytes": int(size), "flops": int(flops)}


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_moe(s) if case["op"] == "moe" else _exact_linear(s)


def _exact_linear(s):
    case = s["case"]
    out = {}
    if case["op"] == "linear":
        x = s["X"].to(torch.float64)
        # the scale is a 32-bit number by definition: the largest magnitude over 127, rounded once
        sx = (x.abs().max(dim=1).values / 127).to(torch.float32)
        out["scale"] = sx.double()
        q = torch.round(x / out["scale"].unsqueeze(1))
        sx = out["scale"]
    else:
        q, sx = s["X"].to(torch.float64), s["sx"].to(torch.float64)
    y = torch.einsum("tk,nk->tn", q, s["W"].to(torch.float64))
    y *= torch.outer(sx, s["sw"].to(torch.float64))
    out["y"] = y if s["bias"] is None else y + s["bias"].to(torch.float64)
    return out


def _row_values(raw, fmt, rows, cols):
    """One matrix in 64 bits, each stored code through a table of the values that it stands for."""
    per = {Q8_0: 1, Q4_0: 2, I4_ROW: 2, I2_ROW: 4}[fmt]
    code = torch.arange(256, device=raw.device)
    if fmt == Q8_0:
        table = ((code + 128) % 256 - 128)[:, None]
    else:
        bits = 8 // per
        part = torch.stack([(code >> (bits * i)) % (1 << bits) for i in range(per)], 1)
        half = 1 << (bits - 1)
        table = part - 8 if fmt == Q4_0 else (part + half) % (2 * half) - half
    table = table.double()
    n = rows * _row_bytes(fmt, cols)
    if fmt in (Q8_0, Q4_0):
        blk = raw[:n].reshape(rows * cols // 32, -1)
        d = blk[:, :2].contiguous().view(torch.float16).double()
        v = table[blk[:, 2:].long()].reshape(-1, 32) * d
        return v.reshape(rows, cols)
    at = -(-n // 16) * 16
    d = raw[at:at + 4 * rows].clone().view(torch.float32).double()
    return table[raw[:n].long()].reshape(rows, cols) * d[:, None]


def _exact_ffn(mats, fmt, act, x, H, I):
    g = _row_values(mats[0], fmt, I, H) @ x
    u = _row_values(mats[1], fmt, I, H) @ x
    if act == SILU:
        h = g * torch.sigmoid(g) * u
    else:
        h = g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) / 2 * u
    return _row_values(mats[2], fmt, H, I) @ h


def _exact_moe(s):
    c = s["case"]
    T, H, I, k = c["tokens"], c["hidden"], c["inter"], c["top_k"]
    X = s["x"].to(torch.float64)
    logits = torch.einsum("th,eh->te", X, s["R"].to(torch.float64))
    prob = torch.softmax(logits, 1)
    y = torch.zeros(T, H, dtype=torch.float64, device=X.device)
    idx = torch.zeros(T, k, dtype=torch.int32, device=X.device)
    w = torch.zeros(T, k, dtype=torch.float64, device=X.device)
    for t in range(T):
        row = logits[t].tolist()
        chosen = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        idx[t] = torch.tensor(chosen, dtype=torch.int32)
        w[t] = prob[t, chosen] / prob[t, chosen].sum()
        for j, e in enumerate(chosen):
            mats = [m[e * stride:(e + 1) * stride] for m, stride in s["experts"]]
            y[t] += w[t, j] * _exact_ffn(mats, c["fmt"], c["act"], X[t], H, I)
        if s["shared"] is not None:
            y[t] += _exact_ffn(s["shared"], c["shared_fmt"], c["act"], X[t], H, c["shared"])
    return {"y": y, "idx": idx, "w": w}
