"""What is measured of the 4-bit operators, and their plain forms.

Three operators in OCP microscaling FP4 (E2M1 elements, one E8M0 scale byte per
32 elements of a row):

  quantize  x -> codes and scales, along the rows and, where asked, along the
            columns too; to nearest even or stochastically
  product   y = A B^T of two quantized operands, bf16 out
  moe       a mixture-of-experts layer for a few tokens: router, the chosen
            experts' gated two-layer networks with 4-bit weights, the sum

and the three products of one linear layer's training step, with the
quantizations that feed them.

`run` computes them from elementary torch operations in 32 bits; with `own`
set it makes the calls a user makes of fp8_scaled_matmul_amd.
"""
import math

import torch

own = False

BLOCK = 32          # elements that share a scale
FMAX = 6.0          # largest E2M1 value
MASK = 0xFFFFFFFF
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token's hidden state on its way into a 4-bit projection: latency
        {"name": "quantize_token", "op": "quantize", "rows": 1, "cols": 4096, "dtype": "bf16", "both": False, "stochastic": False},
        # activations of a training step, needed along both axes (forward and weight gradient)
        {"name": "quantize_activations", "op": "quantize", "rows": 16384, "cols": 2048, "dtype": "bf16", "both": True, "stochastic": False},
        # output gradients of a ragged batch, rounded stochastically, along both axes
        {"name": "quantize_gradient", "op": "quantize", "rows": 8191, "cols": 5000, "dtype": "bf16", "both": True, "stochastic": True},
        # a large fp32 master tensor after the optimizer step
        {"name": "quantize_master", "op": "quantize", "rows": 8192, "cols": 8192, "dtype": "fp32", "both": False, "stochastic": False},
        # decoding: one row against a whole weight
        {"name": "product_token", "op": "product", "m": 1, "n": 8192, "k": 8192},
        # a ragged batch against odd sizes
        {"name": "product_ragged", "op": "product", "m": 333, "n": 1000, "k": 1568},
        # a prefill chunk
        {"name": "product_chunk", "op": "product", "m": 1024, "n": 4096, "k": 4096},
        # a training batch's forward product
        {"name": "product_large", "op": "product", "m": 16384, "n": 8192, "k": 7168},
        # forward, input gradient and weight gradient of one linear layer
        {"name": "linear_step", "op": "linear", "m": 16384, "n": 2048, "k": 7168},
        # one token through a mixture of experts: latency
        {"name": "moe_token", "op": "moe", "tokens": 1, "experts": 64, "top_k": 8, "hidden": 2048, "inner": 1408, "renormalize": True},
        # a few tokens, sizes that divide nothing
        {"name": "moe_ragged", "op": "moe", "tokens": 7, "experts": 37, "top_k": 3, "hidden": 1000, "inner": 531, "renormalize": False},
        # a decoding batch that reaches nearly every expert
        {"name": "moe_batch", "op": "moe", "tokens": 64, "experts": 128, "top_k": 8, "hidden": 4096, "inner": 1024, "renormalize": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "product", "product", "product", "linear", "moe", "moe"])
    if op == "quantize":
        rows, cols = _log(rng, 1, 16384), _log(rng, 32, 16384)
        rows = max(1, min(rows, (1 << 25) // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "fp32"]),
                "both": rng.random() < 0.5, "stochastic": rng.random() < 0.4}
    if op == "product":
        m, n, k = _log(rng, 1, 16384), _log(rng, 16, 16384), _log(rng, 32, 8192)
        m = max(1, min(m, 16384 * 8192 * 7168 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k}
    if op == "linear":
        return {"op": op, "m": _log(rng, 64, 16384), "n": _log(rng, 64, 2048), "k": _log(rng, 64, 7168)}
    experts = _log(rng, 4, 128)
    return {"op": op, "tokens": _log(rng, 1, 64), "experts": experts, "top_k": rng.randint(1, min(8, experts)),
            "hidden": _log(rng, 256, 4096), "inner": _log(rng, 128, 1024), "renormalize": rng.random() < 0.5}


# ------------------------------------------------------------------ what has to be moved and computed
def _held(rows, cols):
    """Bytes of a quantized [rows, cols]: half a byte an element, one a block."""
    return rows * (cols / 2 + -(-cols // BLOCK))


def work(case):
    c = case
    if c["op"] == "quantize":
        r, n = c["rows"], c["cols"]
        size = 2 if c["dtype"] == "bf16" else 4
        held = _held(r, n) + (_held(n, r) if c["both"] else 0)
        values = r * n * size * (2 if c["both"] else 1)
        # x read, the codes and scales written, and read again for the values returned
        return {"bytes": r * n * size + 2 * held + values, "flops": 4.0 * r * n}
    if c["op"] == "product":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": _held(m, k) + _held(n, k) + 2 * m * n, "flops": 2.0 * m * n * k}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": 2 * m * k + 2 * m * n + _held(n, k) + _held(k, n) + 2 * m * n + 2 * m * k + 2 * n * k,
                "flops": 6.0 * m * n * k}
    t, e, k, h, i = c["tokens"], c["experts"], c["top_k"], c["hidden"], c["inner"]
    reached = e * (1 - (1 - k / e) ** t)      # experts that some token chooses, on average
    return {"bytes": 4 * t * h + 2 * e * h + reached * (_held(2 * i, h) + _held(h, i)),
            "flops": 2.0 * t * e * h + 6.0 * t * k * h * i}


# ------------------------------------------------------------------ the plain form
def _random16(rows, cols, seed, device):
    """The 16 random bits of every element: two multiply-and-shift mixes of the
    row and the column pair; even columns take the low half."""
    def mix(v):
        v = v ^ (v >> 16)
        v = (v * 0x6A09E667) & MASK
        v = v ^ (v >> 15)
        v = (v * 0xBB67AE85) & MASK
        return v ^ (v >> 16)

    s = seed.to(torch.int64)
    row = torch.arange(rows, device=device, dtype=torch.int64)
    col = torch.arange(cols, device=device, dtype=torch.int64)
    per_row = mix((row * 0x9E3779B1 + (s & MASK)) & MASK)
    pair = ((col >> 1) * 0x3C6EF373 + ((s >> 32) & MASK)) & MASK
    v = mix(per_row[:, None] ^ pair[None, :])
    return torch.where((col & 1)[None, :] == 1, v >> 16, v & 0xFFFF)


def _blocks(x, cols):
    """[rows, cols] fp32 -> [rows, blocks, 32], zeros past the end."""
    pad = -cols % BLOCK
    if pad:
        x = torch.nn.functional.pad(x, (0, pad))
    return x.reshape(x.shape[0], -1, BLOCK)


def _grid(a):
    """|v| <= 6 to the nearest E2M1 value, ties to the even code."""
    def f(b):
        return b.to(a.dtype)
    return (0.5 * (f(a > 0.25) + f(a >= 0.75) + f(a > 1.25) + f(a >= 1.75)) + f(a > 2.5) + f(a >= 3.5) + 2 * f(a > 5.0))


def _fake_quantize(x, random=None):
    """[rows, cols] -> (values on the grid, the blocks' scales), both fp32.
    The scale is the smallest power of two s with amax / s <= 6 (1 for an
    all-zero block, at least 2^-126)."""
    rows, cols = x.shape
    b = _blocks(x.float(), cols)
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)                  # amax = m 2^e, m in [0.5, 1)
    e = e - 3 + (m > 0.75).to(e.dtype)
    e = torch.where(amax > 0, e.clamp(-126, 126), torch.zeros_like(e))
    s = torch.ldexp(torch.ones_like(amax), e)
    v = b / s[..., None]
    a = v.abs()
    if random is None:
        g = _grid(a)
    else:
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        low = torch.floor(a / step) * step
        r = _blocks(random.float(), cols)
        g = low + step * (((a - low) / step) * 65536.0 >= 65536.0 - r).float()
    return torch.copysign(g, v), s


def _values(x, random=None):
    """The values that x's codes and scales stand for, [rows, cols] fp32."""
    g, s = _fake_quantize(x, random)
    return (g * s[..., None]).reshape(x.shape[0], -1)[:, : x.shape[1]]


def _encode(x):
    """x [rows, cols] as the library holds it: codes [rows, 128 ceil(cols/256)],
    two to a byte (even element in the low half), and scale bytes
    [ceil(cols/512), rows, 16], the 16 blocks of 512 columns of a row side by
    side; codes past the end are 0, scale bytes 127."""
    rows, cols = x.shape
    g, s = _fake_quantize(x)
    a = g.abs()
    code = (2 * torch.where(a <= 2, a, torch.where(a <= 4, a / 2 + 1, a / 4 + 2))).to(torch.uint8)
    # 0, 0.5, 1, 1.5, 2, 3, 4, 6 are codes 0 .. 7; bit 3 is the sign
    code = code + 8 * torch.signbit(g).to(torch.uint8)
    code = code.reshape(rows, -1)
    code = torch.nn.functional.pad(code, (0, -(-cols // 256) * 256 - code.shape[1]))
    q = code[:, 0::2] + 16 * code[:, 1::2]
    sb = (torch.frexp(s)[1] + 126).to(torch.uint8)
    sb = torch.nn.functional.pad(sb, (0, -(-cols // 512) * 16 - sb.shape[1]), value=127)
    return q, sb.reshape(rows, -1, 16).transpose(0, 1).contiguous()


def _encode_experts(x, experts):
    """The same of `experts` matrices stacked in x: codes [experts, rows, ..],
    scale bytes [experts, ceil(cols/512), rows, 16]."""
    q, sb = _encode(x)
    sb = sb.reshape(sb.shape[0], experts, -1, 16).transpose(0, 1).contiguous()
    return q.reshape(experts, -1, q.shape[1]), sb


def _decode(q, sb, cols):
    """Codes and scale bytes to fp32 values [..., cols]."""
    sb = sb.transpose(-3, -2).flatten(-2)
    code = torch.stack((q & 15, q >> 4), -1).reshape(*q.shape[:-1], -1)[..., : -(-cols // BLOCK) * BLOCK]
    c = (code & 7).float()
    mag = torch.where(c < 4, 0.5 * c, torch.where(c < 6, c - 2, 2 * c - 8))
    v = torch.where(code >= 8, -mag, mag)
    s = torch.ldexp(torch.ones_like(sb[..., : -(-cols // BLOCK)], dtype=torch.float32), sb[..., : -(-cols // BLOCK)].int() - 127)
    return (v * s.repeat_interleave(BLOCK, -1))[..., :cols]


def _moe_plain(s):
    c, x = s["case"], s["x"]
    t, e, k, h, i = c["tokens"], c["experts"], c["top_k"], c["hidden"], c["inner"]
    # the border between chosen and not chosen is looked at in 64 bits
    logits = x.double() @ s["router"].double().t()
    best, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    best, ids = best[:, :k].float(), ids[:, :k]
    if c["renormalize"]:
        p = torch.exp(best - best[:, :1])
        p = p / p.sum(-1, keepdim=True)
    else:
        p = torch.exp(best - best[:, :1]) / torch.exp(logits.float() - best[:, :1]).sum(-1, keepdim=True)
    if t * k < e:             # few pairs: only their experts' weights
        at = ids.flatten()
        pair = x.float().repeat_interleave(k, 0)
        gu = (_decode(s["w1q"][at], s["w1s"][at], h) * pair[:, None, :]).sum(-1).reshape(t, k, 2, i)
    else:                     # every expert for every token, then the chosen ones
        w1 = _decode(s["w1q"], s["w1s"], h).reshape(e * 2 * i, h)
        gu = (x.float() @ w1.t()).reshape(t, e, 2, i)
        gu = torch.gather(gu, 1, ids[:, :, None, None].expand(t, k, 2, i))
    g, u = gu[:, :, 0], gu[:, :, 1]
    a = g / (1 + torch.exp(-g)) * u * p[..., None]
    if t * k < e:
        y = (_decode(s["w2q"][at], s["w2s"][at], i) * a.reshape(t * k, 1, i)).sum(-1).reshape(t, k, h).sum(1)
    else:
        dense = torch.zeros(t, e, i, device=x.device).scatter_(1, ids[:, :, None].expand(t, k, i), a)
        w2 = _decode(s["w2q"], s["w2s"], i)
        y = dense.reshape(t, e * i) @ w2.permute(0, 2, 1).reshape(e * i, h)
    return {"y": y.bfloat16(), "ids": ids.int(), "weights": p}


def _plain(s):
    c = s["case"]
    if c["op"] == "quantize":
        x = s["x"]
        r = _random16(c["rows"], c["cols"], s["seed"], x.device) if c["stochastic"] else None
        out = {"values": _values(x, r).to(x.dtype)}
        if c["both"]:
            out["values_t"] = _values(x.t().contiguous(), None if r is None else r.t()).to(x.dtype)
        return out
    if c["op"] == "product":
        return {"y": (_decode(s["aq"], s["as"], c["k"]) @ _decode(s["bq"], s["bs"], c["k"]).t()).bfloat16()}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        r = _random16(m, n, s["seed"], s["dy"].device)
        y = _values(s["x"]) @ _decode(s["wq"], s["ws"], k).t()
        dx = _values(s["dy"], r) @ _decode(s["wtq"], s["wts"], n).t()
        dw = _values(s["dy"].t().contiguous(), r.t()) @ _values(s["x"].t().contiguous()).t()
        return {"y": y.bfloat16(), "dx": dx.bfloat16(), "dw": dw.bfloat16()}
    return _moe_plain(s)


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import fp8_scaled_matmul_amd as fm
    c = s["case"]
    if c["op"] == "quantize":
        q, qt = fm.mx4_quantize(s["x"], want_t=c["both"], seed=s["seed"] if c["stochastic"] else None)
        out = {"values": fm.mx4_dequantize(q, s["x"].dtype)}
        if c["both"]:
            out["values_t"] = fm.mx4_dequantize(qt, s["x"].dtype)
        return out
    if c["op"] == "product":
        return {"y": fm.mx4_mm(fm.Mx4(s["aq"], s["as"], c["k"]), fm.Mx4(s["bq"], s["bs"], c["k"]))}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        xq, xqt = fm.mx4_quantize(s["x"], want_t=True)
        y = fm.mx4_mm(xq, fm.Mx4(s["wq"], s["ws"], k))
        dq, dqt = fm.mx4_quantize(s["dy"], want_t=True, seed=s["seed"])
        dx = fm.mx4_mm(dq, fm.Mx4(s["wtq"], s["wts"], n))
        dw = fm.mx4_mm(dqt, xqt)
        return {"y": y, "dx": dx, "dw": dw}
    if "layer" not in s:      # set up once, as a program that serves the layer keeps it
        s["layer"] = fm.MoeMx4(s["router"], fm.Mx4(s["w1q"], s["w1s"], c["hidden"]), fm.Mx4(s["w2q"], s["w2s"], c["inner"]),
                               c["top_k"], max_tokens=c["tokens"], renormalize=c["renormalize"])
    y, ids, weights = s["layer"](s["x"])
    return {"y": y, "ids": ids, "weights": weights}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, std, device, channels=0.0):
    """N(0, std) with a share of the columns 100 times as large."""
    x = torch.randn(*shape, generator=gen, device=device) * std
    if channels:
        x[..., torch.rand(shape[-1], generator=gen, device=device) < channels] *= 100.0
    return x


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=device).manual_seed(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] in ("quantize", "linear"):
        s["seed"] = torch.randint(0, 1 << 62, (1,), generator=g, device=device)
    if c["op"] == "quantize":
        std, channels = (1e-3, 0.0) if c["stochastic"] else (1.0, 0.01)
        s["x"] = _normal(g, (c["rows"], c["cols"]), std, device, channels).to(DTYPES[c["dtype"]])
    elif c["op"] == "product":
        s["aq"], s["as"] = _encode(_normal(g, (c["m"], c["k"]), 1.0, device, 0.01).bfloat16())
        s["bq"], s["bs"] = _encode(_normal(g, (c["n"], c["k"]), 0.02, device).bfloat16())
    elif c["op"] == "linear":
        s["x"] = _normal(g, (c["m"], c["k"]), 1.0, device, 0.01).bfloat16()
        s["dy"] = _normal(g, (c["m"], c["n"]), 1e-3, device).bfloat16()
        w = _normal(g, (c["n"], c["k"]), 0.02, device).bfloat16()
        s["wq"], s["ws"] = _encode(w)
        s["wtq"], s["wts"] = _encode(w.t().contiguous())
    else:
        t, e, h, i = c["tokens"], c["experts"], c["hidden"], c["inner"]
        s["x"] = _normal(g, (t, h), 1.0, device).bfloat16()
        s["router"] = _normal(g, (e, h), h ** -0.5, device).bfloat16()
        s["w1q"], s["w1s"] = _encode_experts(_normal(g, (e * 2 * i, h), h ** -0.5, device), e)
        s["w2q"], s["w2s"] = _encode_experts(_normal(g, (e * h, i), i ** -0.5, device), e)
    return s


# ------------------------------------------------------------------ the definitions in 64 bits
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _held_values(q, sb, cols):
    table = torch.tensor(E2M1, dtype=torch.float64, device=q.device)
    pairs = torch.stack((table[(q % 16).long()], table[torch.div(q, 16, rounding_mode="floor").long()]), -1)
    v = pairs.flatten(-2)[..., :cols]
    at = torch.arange(cols, device=q.device) // BLOCK
    rows = torch.arange(q.shape[-2], device=q.device)
    scale = torch.exp2(sb.double() - 127)[..., at[None, :] // 16, rows[:, None], at[None, :] % 16]
    return v * scale


def _bits(rows, cols, seed, device):
    """The element's 16 random bits, with products taken in two halves."""
    def times(v, c):
        return ((v % 65536) * c + (((v // 65536) * c) % 65536) * 65536) % (1 << 32)

    def mix(v):
        v = torch.bitwise_xor(v, v // 65536)
        v = times(v, 1779033703)
        v = torch.bitwise_xor(v, v // 32768)
        v = times(v, 3144134277)
        return torch.bitwise_xor(v, v // 65536)

    lo, hi = int(seed) % (1 << 32), int(seed) >> 32
    r = mix((times(torch.arange(rows, device=device), 2654435761) + lo) % (1 << 32))
    pairs = (cols + 1) // 2
    p = (times(torch.arange(pairs, device=device), 1013904243) + hi) % (1 << 32)
    v = mix(torch.bitwise_xor(r.unsqueeze(1), p.unsqueeze(0)))
    return torch.stack((v % 65536, v // 65536), -1).flatten(1)[:, :cols]


def _quantized64(x, bits=None):
    """Nearest (or random) E2M1 multiple of each block's scale, row by row."""
    rows, cols = x.shape
    x = x.double()
    wide = torch.zeros(rows, -(-cols // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    wide[:, :cols] = x
    big = wide.unflatten(1, (-1, BLOCK)).abs().max(-1).values
    e = torch.ceil(torch.log2(torch.where(big > 0, big, 6.0) / 6.0))
    e = torch.where(big > 6 * torch.exp2(e), e + 1, e)
    e = torch.where(big <= 6 * torch.exp2(e - 1), e - 1, e).clamp(-126, 126)
    e = torch.where(big > 0, e, torch.zeros_like(e))
    s = torch.exp2(e).repeat_interleave(BLOCK, 1)[:, :cols]
    a = (x / s).abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(1.0, 4.0))) - 1)
    n = a / step
    if bits is None:
        n = torch.round(n)                    # halves to even; even multiples are even codes
    else:
        n = torch.floor(n) + (torch.floor((n - torch.floor(n)) * 65536) + bits >= 65536).double()
    return torch.where(x < 0, -n, n) * step * s


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "quantize":
        x = s["x"]
        bits = _bits(c["rows"], c["cols"], s["seed"].item(), x.device) if c["stochastic"] else None
        out = {"values": _quantized64(x, bits)}
        if c["both"]:
            out["values_t"] = _quantized64(x.t().contiguous(), None if bits is None else bits.t())
        return out
    if c["op"] == "product":
        return {"y": _held_values(s["aq"], s["as"], c["k"]) @ _held_values(s["bq"], s["bs"], c["k"]).t()}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        bits = _bits(m, n, s["seed"].item(), s["dy"].device)
        return {"y": _quantized64(s["x"]) @ _held_values(s["wq"], s["ws"], k).t(),
                "dx": _quantized64(s["dy"], bits) @ _held_values(s["wtq"], s["wts"], n).t(),
                "dw": _quantized64(s["dy"].t().contiguous(), bits.t()) @ _quantized64(s["x"].t().contiguous()).t()}
    x, k, i = s["x"].double(), c["top_k"], c["inner"]
    logits = x @ s["router"].double().t()
    rank = torch.argsort(-logits, dim=-1, stable=True)[:, :k]
    p = torch.softmax(logits, -1)
    y = torch.zeros_like(x)
    weights = torch.gather(p, 1, rank)
    if c["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    for e in range(c["experts"]):
        tok, slot = torch.nonzero(rank == e, as_tuple=True)
        if not len(tok):
            continue
        w1 = _held_values(s["w1q"][e], s["w1s"][e], c["hidden"])
        w2 = _held_values(s["w2q"][e], s["w2s"][e], i)
        gate, up = x[tok] @ w1[:i].t(), x[tok] @ w1[i:].t()
        y[tok] += weights[tok, slot].unsqueeze(1) * ((gate * torch.sigmoid(gate) * up) @ w2.t())
    return {"y": y, "ids": rank.int(), "weights": weights}
