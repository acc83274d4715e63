"""Cases that measure the 8-bit projection operators: the RMSNorm that adds the residual and writes
E4M3 rows with one power-of-two scale per 128 values, the quantisation of weights in 128 x 128
blocks, and the product of the two with 1 to 4 weight matrices over the same rows.

Layouts: E4M3 rows of k values lie at a pitch of k rounded up to 16 bytes; their scales are E8M0
bytes (value 2^(byte - 127)), one per 128 values, at a pitch of ceil(k / 128) rounded up to 4 bytes;
a weight matrix has one scale row per 128 rows.
"""

import torch

own = False

EPS = 1e-6
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def up(x, a):
    return -(-x // a) * a


def listed():
    return [
        # decode: the norm in front of one token's projections
        {"name": "norm_1x4096_bf16", "op": "norm", "n": 1, "d": 4096, "dtype": "bf16", "residual": True, "gain": True},
        # a decode step of 32 sequences
        {"name": "norm_32x4096_bf16", "op": "norm", "n": 32, "d": 4096, "dtype": "bf16", "residual": True, "gain": True},
        # a prefill chunk
        {"name": "norm_4096x4096_bf16", "op": "norm", "n": 4096, "d": 4096, "dtype": "bf16", "residual": True, "gain": True},
        # a ragged chunk of an fp32 layer, no residual and no gain, the last block of a row 8 wide
        {"name": "norm_437x1544_f32", "op": "norm", "n": 437, "d": 1544, "dtype": "f32", "residual": False, "gain": False},
        # four chunks of a wide layer in one call
        {"name": "norm_16384x7168_bf16", "op": "norm", "n": 16384, "d": 7168, "dtype": "bf16", "residual": True, "gain": True},
        # loading one projection of a ratio-4 layer's attention lane
        {"name": "quant_1024x4096_bf16", "op": "quant", "n": 1024, "k": 4096, "dtype": "bf16"},
        # loading a large fp32 matrix
        {"name": "quant_8192x8192_f32", "op": "quant", "n": 8192, "k": 8192, "dtype": "f32"},
        # one token through the four projections of a ratio-4 layer
        {"name": "proj_1_f32", "op": "mm", "m": 1, "ns": "1024,1024,256,256", "k": 4096, "out": "f32"},
        # a decode step of 32 sequences through them
        {"name": "proj_32_f32", "op": "mm", "m": 32, "ns": "1024,1024,256,256", "k": 4096, "out": "f32"},
        # a prefill chunk through them
        {"name": "proj_4096_f32", "op": "mm", "m": 4096, "ns": "1024,1024,256,256", "k": 4096, "out": "f32"},
        # nothing a multiple of a tile, an odd k
        {"name": "mm_437x1000x1541_bf16", "op": "mm", "m": 437, "ns": "1000", "k": 1541, "out": "bf16"},
        # the largest product
        {"name": "mm_8192x8192x8192_bf16", "op": "mm", "m": 8192, "ns": "8192", "k": 8192, "out": "bf16"},
    ]


def _size(rng, lo, hi, step=1):
    """A size spread over the logarithm of lo .. hi; mostly a multiple of `step`, odd ones among them."""
    v = lo * (hi / lo) ** rng.random()
    v = int(round(v))
    if step > 1 and rng.random() < 0.7:
        v = max(step, v // step * step)
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["norm", "norm", "quant", "mm", "mm", "mm"])
    if op == "norm":
        while True:
            n, d = _size(rng, 1, 16384), _size(rng, 64, 8192, 128)
            if n * d <= 16384 * 7168:
                return {"op": "norm", "n": n, "d": d, "dtype": rng.choice(["bf16", "f32"]) if n * d <= 8192 * 7168 else "bf16",
                        "residual": rng.random() < 0.7, "gain": rng.random() < 0.7}
    if op == "quant":
        return {"op": "quant", "n": _size(rng, 16, 8192, 64), "k": _size(rng, 64, 8192, 64), "dtype": rng.choice(["bf16", "f32"])}
    m, k = _size(rng, 1, 8192), _size(rng, 64, 8192, 128)
    groups = rng.choice([1, 1, 2, 4])
    ns = [_size(rng, 16, 8192 // groups, 64) for _ in range(groups)]
    return {"op": "mm", "m": m, "ns": ",".join(map(str, ns)), "k": k, "out": rng.choice(["f32", "bf16"])}


def _type(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _pow2(e):
    """2^e in 32 bits, exactly, for whole numbers e from -149 to 127."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _blocks(t, rows):
    """t [n][k] cut into blocks of `rows` x 128, padded with zeros: [n/rows][rows][k/128][128]."""
    n, k = t.shape
    t = torch.nn.functional.pad(t, (0, up(k, 128) - k, 0, up(n, rows) - n))
    return t.view(up(n, rows) // rows, rows, up(k, 128) // 128, 128)


def _quantise(y, rows):
    """E4M3 values (in y's type) and exponents of y [n][k] in blocks of `rows` x 128: the smallest e
    with max|y| <= 448 * 2^e, at least -127, and 0 for a block of zeros."""
    n, k = y.shape
    b = _blocks(y, rows)
    amax = b.abs().amax(dim=(1, 3), keepdim=True)
    mant, ex = torch.frexp(amax)                               # amax = mant * 2^ex, 448 = 0.875 * 2^9
    e = torch.where(mant <= 0.875, ex - 9, ex - 8).clamp(min=-127)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    v = b * _pow2(-e)
    return v.reshape(-1, b.shape[2] * 128)[:n, :k], e.view(b.shape[0], b.shape[2])


def _stored(y, rows):
    """(q, scale) of y as they are stored: E4M3 rows and E8M0 bytes at their pitches."""
    n, k = y.shape
    v, e = _quantise(y, rows)
    q = torch.zeros(n, up(k, 16), dtype=F8, device=y.device)[:, :k]
    q.copy_(v.to(F8))
    s = torch.zeros(e.shape[0], up(e.shape[1], 4), dtype=torch.uint8, device=y.device)
    s[:, :e.shape[1]] = (e + 127).to(torch.uint8)
    return q, s


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _hidden(gen, n, k):
    """Rows as a residual stream holds them: normal values, a few channels far larger than the rest."""
    ch = torch.exp(0.5 * _normal(gen, k))
    ch[torch.randint(0, k, (max(1, k // 256),), generator=gen, device="cuda")] *= 30.0
    return _normal(gen, n, k) * ch


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        n, d, t = case["n"], case["d"], _type(case["dtype"])
        s["x"] = _hidden(gen, n, d).to(t)
        if n > 64:
            s["x"][n // 2] = 0.0                               # a padded row of the batch
        s["residual"] = (3.0 * _normal(gen, n, d)).to(t) if case["residual"] else None
        s["gain"] = 1.0 + 0.1 * _normal(gen, d) if case["gain"] else None
        s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["q"] = torch.empty(n, up(d, 16), dtype=F8, device="cuda")[:, :d]
        s["scale"] = torch.zeros(n, up(-(-d // 128), 4), dtype=torch.uint8, device="cuda")
    elif case["op"] == "quant":
        n, k = case["n"], case["k"]
        s["w"] = (0.02 * _normal(gen, n, k) * torch.exp(0.5 * _normal(gen, n, 1))).to(_type(case["dtype"]))
        s["q"] = torch.empty(n, up(k, 16), dtype=F8, device="cuda")[:, :k]
        s["scale"] = torch.zeros(up(n, 128) // 128, up(-(-k // 128), 4), dtype=torch.uint8, device="cuda")
    else:
        m, k = case["m"], case["k"]
        s["q"], s["scale"] = _stored(_hidden(gen, m, k), 1)
        s["w"] = [_stored(0.02 * _normal(gen, int(n), k), 128) for n in case["ns"].split(",")]
        s["out"] = [torch.empty(m, int(n), dtype=_type(case["out"]), device="cuda") for n in case["ns"].split(",")]
        if own:                                                # the weights' handle, which a program keeps
            from compressed_kv_sparse_compressor_gb300 import fp8
            s["linear"] = fp8.Linear([fp8.Fp8Weight(q, sc) for q, sc in s["w"]])
    return s


def _values(q, scale, rows):
    """The values that E4M3 rows and their scale bytes stand for, in 32 bits."""
    n, k = q.shape
    f = _pow2(scale[:, :-(-k // 128)].int() - 127)
    f = f.repeat_interleave(rows, 0)[:n].repeat_interleave(128, 1)[:, :k] if rows > 1 else f.repeat_interleave(128, 1)[:, :k]
    return q.float() * f


def run(state):
    case = state["case"]
    if own:
        from compressed_kv_sparse_compressor_gb300 import fp8
    if case["op"] == "norm":
        x, r, g = state["x"], state["residual"], state["gain"]
        if own:
            fp8.rmsnorm(x, g, residual=r, residual_out=state["h"], eps=EPS, q=state["q"], scale=state["scale"])
            q, scale, h = state["q"], state["scale"], state["h"]
        else:
            h = x if r is None else (x.float() + r.float()).to(x.dtype)
            # the row's statistic in 64 bits: a code next to a rounding border hangs on it
            rstd = torch.rsqrt(h.double().square().mean(dim=1, keepdim=True) + EPS).float()
            y = h.float() * rstd
            q, scale = _stored(y if g is None else y * g, 1)
            h = None if r is None else h
        return {"q": q, "scale": scale.view(E8), "h": h}
    if case["op"] == "quant":
        if own:
            fp8.quantize_weight(state["w"], q=state["q"], scale=state["scale"])
            return {"q": state["q"], "scale": state["scale"].view(E8)}
        q, scale = _stored(state["w"].float(), 128)
        return {"q": q, "scale": scale.view(E8)}
    if own:
        return state["linear"](state["q"], state["scale"], out=state["out"])
    a = _values(state["q"], state["scale"], 1)
    return [(a @ _values(q, s, 128).T).to(o.dtype) for (q, s), o in zip(state["w"], state["out"])]


def work(case):
    if case["op"] == "norm":
        n, d = case["n"], case["d"]
        e = 4 if case["dtype"] == "f32" else 2
        return {"bytes": n * d * (e + 1 + (2 * e if case["residual"] else 0)) + n * -(-d // 128) + (4 * d if case["gain"] else 0),
                "flops": 10 * n * d}
    if case["op"] == "quant":
        n, k = case["n"], case["k"]
        return {"bytes": n * k * ((4 if case["dtype"] == "f32" else 2) + 1) + -(-n // 128) * -(-k // 128), "flops": 3 * n * k}
    m, k, ns = case["m"], case["k"], [int(n) for n in case["ns"].split(",")]
    kb, e = -(-k // 128), 4 if case["out"] == "f32" else 2
    return {"bytes": m * (k + kb) + sum(n * k + -(-n // 128) * kb + m * n * e for n in ns), "flops": 2 * m * k * sum(ns)}


def _exponents(amax):
    """The smallest e with amax <= 448 * 2^e, from the logarithm, put right by comparing."""
    e = torch.ceil(torch.log2(torch.clamp(amax, min=1e-300) / 448.0))
    e = torch.where(amax <= 448.0 * 2.0 ** (e - 1), e - 1, e)
    e = torch.where(amax > 448.0 * 2.0 ** e, e + 1, e)
    return torch.where(amax > 0, torch.clamp(e, min=-127.0), torch.zeros_like(e))


def _exact_stored(y, rows):
    """The scaled values before their rounding to 8 bits, and 2^e at the scales' pitch."""
    n, k = y.shape
    kb, nb = -(-k // 128), -(-n // rows)
    v, f = torch.empty_like(y), torch.ones(nb, up(kb, 4), dtype=torch.float64, device=y.device)
    f[:, kb:] = 2.0 ** -127                                    # the pitch's padding is left as prepare made it: byte 0
    for b in range(kb):
        part = y[:, 128 * b:128 * (b + 1)]
        amax = torch.nn.functional.pad(part.abs().amax(dim=1), (0, nb * rows - n)).view(nb, rows).amax(dim=1)
        f[:, b] = 2.0 ** _exponents(amax)
        v[:, 128 * b:128 * (b + 1)] = part / f[:, b].repeat_interleave(rows)[:n, None]
    return v, f


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        stored = h
        if s["residual"] is not None:
            h = h + s["residual"].double()
            stored = h.to(s["x"].dtype).double()               # the norm is of the stream as it is stored
        y = stored / torch.sqrt((stored * stored).sum(dim=1, keepdim=True) / case["d"] + EPS)
        v, f = _exact_stored(y if s["gain"] is None else y * s["gain"].double(), 1)
        return {"q": v, "scale": f, "h": h if s["residual"] is not None else None}
    if case["op"] == "quant":
        v, f = _exact_stored(s["w"].double(), 128)
        return {"q": v, "scale": f}
    q, sa = s["q"].double(), 2.0 ** (s["scale"].double() - 127.0)
    outs = []
    for w, sw in s["w"]:
        w, fw = w.double(), 2.0 ** (sw.double() - 127.0)
        acc = torch.zeros(q.shape[0], w.shape[0], dtype=torch.float64, device=q.device)
        at = torch.arange(w.shape[0], device=q.device) // 128
        for b in range(-(-case["k"] // 128)):
            cols = slice(128 * b, 128 * (b + 1))
            acc += (q[:, cols] * sa[:, b:b + 1]) @ (w[:, cols] * fw[at, b:b + 1]).T
        outs.append(acc)
    return outs
