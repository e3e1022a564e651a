"""What is measured of the training operators around the linear layers, and
their plain forms.

  loss      softmax cross entropy of a projection onto a vocabulary, from the
            hidden states and the projection's weight: each token's loss,
            without the logits as a result (scoring, evaluation)
  head      the same with its gradients for both operands (a training step)
  route     a mixture of experts' router in training: the chosen experts and
            their weights, the tokens of each expert, the balance loss, and
            the gradient of the router's logits
  dropout   with a counter-based generator, onto a residual or not, forward
            and backward; the mask is never stored

`run` computes them from elementary torch operations in 32 bits; with `own`
set it makes the calls a user makes of fp8_scaled_matmul_amd.
"""
import math

import torch

own = False

MASK = 0xFFFFFFFF
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # scoring one token against a vocabulary: the weight's bytes
        {"name": "loss_token", "op": "loss", "tokens": 1, "vocab": 32768, "hidden": 2048, "softcap": 0.0, "ignored": 0.0},
        # evaluation on a ragged batch, sizes that divide nothing, capped logits
        {"name": "loss_ragged", "op": "loss", "tokens": 2001, "vocab": 50001, "hidden": 1000, "softcap": 30.0, "ignored": 0.1},
        # fine-tuning on a few tokens
        {"name": "head_few", "op": "head", "tokens": 64, "vocab": 50304, "hidden": 768, "softcap": 0.0, "ignored": 0.0},
        # a padded batch of a small model with capped logits
        {"name": "head_ragged", "op": "head", "tokens": 1023, "vocab": 50001, "hidden": 1000, "softcap": 15.0, "ignored": 0.3},
        # a training step's batch
        {"name": "head_step", "op": "head", "tokens": 8192, "vocab": 65536, "hidden": 2048, "softcap": 0.0, "ignored": 0.02},
        # the largest: a wide model with a large vocabulary
        {"name": "head_large", "op": "head", "tokens": 8192, "vocab": 131072, "hidden": 4096, "softcap": 0.0, "ignored": 0.0},
        # one token's router: latency
        {"name": "route_token", "op": "route", "tokens": 1, "experts": 64, "top_k": 8, "dtype": "bf16", "renormalize": True, "masked": 0.0},
        # a padded batch, an odd number of experts
        {"name": "route_ragged", "op": "route", "tokens": 8191, "experts": 37, "top_k": 3, "dtype": "fp32", "renormalize": False, "masked": 0.2},
        # a training step's batch
        {"name": "route_step", "op": "route", "tokens": 65536, "experts": 128, "top_k": 8, "dtype": "bf16", "renormalize": True, "masked": 0.0},
        # one token's hidden state: latency
        {"name": "dropout_token", "op": "dropout", "rows": 1, "cols": 4096, "dtype": "bf16", "rate": 0.1, "residual": False},
        # activations of a training step, onto the residual stream
        {"name": "dropout_residual", "op": "dropout", "rows": 16384, "cols": 2048, "dtype": "bf16", "rate": 0.1, "residual": True},
        # a ragged fp32 tensor
        {"name": "dropout_ragged", "op": "dropout", "rows": 8191, "cols": 5000, "dtype": "fp32", "rate": 0.25, "residual": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["loss", "loss", "head", "head", "head", "route", "route", "dropout", "dropout"])
    if op in ("loss", "head"):
        vocab, hidden = _log(rng, 1000, 131072), _log(rng, 64, 4096)
        if rng.random() < 0.5:          # widths of models are most often multiples of a power of two
            hidden = -(-hidden // 64) * 64
        tokens = min(_log(rng, 1, 16384), (8192 * 131072 * 4096) // (vocab * hidden))
        return {"op": op, "tokens": tokens, "vocab": vocab, "hidden": hidden,
                "softcap": rng.choice([0.0, 0.0, 15.0, 30.0]), "ignored": rng.choice([0.0, 0.0, 0.1, 0.5])}
    if op == "route":
        experts = _log(rng, 2, 256)
        return {"op": op, "tokens": _log(rng, 1, 65536), "experts": experts, "top_k": rng.randint(1, min(8, experts)),
                "dtype": rng.choice(["bf16", "fp32"]), "renormalize": rng.random() < 0.5,
                "masked": rng.choice([0.0, 0.0, 0.25])}
    rows, cols = _log(rng, 1, 16384), _log(rng, 32, 16384)
    rows = max(1, min(rows, (1 << 25) // cols))
    return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "fp32"]),
            "rate": rng.choice([0.05, 0.1, 0.25, 0.5]), "residual": rng.random() < 0.5}


# ------------------------------------------------------------------ what has to be moved and computed
def work(case):
    c = case
    if c["op"] in ("loss", "head"):
        t, v, h = c["tokens"], c["vocab"], c["hidden"]
        operands = 2 * t * h + 2 * v * h
        if c["op"] == "loss":       # operands and targets read, loss and log-sum written
            return {"bytes": operands + 8 * t + 8 * t, "flops": 2.0 * t * v * h}
        # operands read, their gradients written; the logits' gradient in between
        return {"bytes": 2 * operands + 8 * t + 12 * t, "flops": 6.0 * t * v * h}
    if c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        size = 2 if c["dtype"] == "bf16" else 4
        # logits and the weights' gradient read, ids, weights and the logits' gradient written
        return {"bytes": 2 * t * e * size + 12 * t * k + 8 * e, "flops": 10.0 * t * e}
    size = 2 if c["dtype"] == "bf16" else 4
    return {"bytes": c["rows"] * c["cols"] * size * (5 if c["residual"] else 4), "flops": 4.0 * c["rows"] * c["cols"]}


# ------------------------------------------------------------------ the plain form
def _capped(l, cap):
    return cap * torch.tanh(l / cap) if cap else l


def _head_plain(s):
    c = s["case"]
    x, w, t = s["x"].float(), s["w"].float(), s["targets"]
    z = _capped(x @ w.t(), c["softcap"])
    big = z.amax(-1, keepdim=True)
    p = torch.exp(z - big)
    total = p.sum(-1, keepdim=True)
    lse = (torch.log(total) + big)[:, 0]
    valid = t >= 0
    at = t.clamp(min=0)
    loss = torch.where(valid, lse - torch.gather(z, 1, at[:, None])[:, 0], torch.zeros_like(lse))
    if c["op"] == "loss":
        return {"loss": loss, "lse": lse}
    d = p.div_(total)
    d.scatter_add_(1, at[:, None], torch.full_like(lse, -1.0)[:, None])
    d.mul_(torch.where(valid, s["grad"], torch.zeros_like(lse))[:, None])
    if c["softcap"]:
        d.mul_(1 - (z / c["softcap"]) ** 2)
    return {"loss": loss, "lse": lse, "dx": (d @ w).bfloat16(), "dw": (d.t() @ x).bfloat16()}


def _route_plain(s):
    c, l = s["case"], s["logits"].float()
    e, k, mask = c["experts"], c["top_k"], s["mask"]
    p = torch.exp(l - l.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    ids = torch.sort(l, dim=-1, descending=True, stable=True)[1][:, :k]
    weights = torch.gather(p, 1, ids)
    norm = weights.sum(-1, keepdim=True)
    if c["renormalize"]:
        weights = weights / norm
    valid = torch.ones(len(l), dtype=torch.bool, device=l.device) if mask is None else mask
    v = valid[:, None]
    chosen = torch.zeros_like(p).scatter_(1, ids, 1.0) * v
    counts = chosen.double().sum(0)
    n = valid.sum().clamp(min=1).double()
    share = e * counts / (n * n * k)          # the balance loss' gradient for each probability
    balance = (share * (p * v).double().sum(0)).sum().float()
    # gradient: of the balance loss through every probability, of the weights through the chosen ones
    down = s["dbalance"] * share.float()
    dp = down.expand_as(p)
    dl = p * (dp - (p * dp).sum(-1, keepdim=True))
    if c["renormalize"]:
        dw = weights * (s["dweights"] - (weights * s["dweights"]).sum(-1, keepdim=True))
        dl = dl.scatter_add(1, ids, dw)
    else:
        wd = weights * s["dweights"]
        dl = dl.scatter_add(1, ids, wd) - p * wd.sum(-1, keepdim=True)
    zero = torch.zeros((), device=l.device)
    return {"ids": torch.where(v, ids, -1).int(), "weights": torch.where(v, weights, zero), "counts": counts.int(),
            "balance": balance, "dlogits": torch.where(v, dl, zero).to(s["logits"].dtype)}


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
    col = torch.arange((cols + 1) // 2, device=device, dtype=torch.int64)
    per_row = mix((row * 0x9E3779B1 + (s & MASK)) & MASK)
    pair = (col * 0x3C6EF373 + (((s >> 32) & MASK) ^ 0xA54FF53A)) & MASK
    v = mix(per_row[:, None] ^ pair[None, :])
    return torch.stack((v & 0xFFFF, v >> 16), -1).flatten(1)[:, :cols]


def _dropout_plain(s):
    c = s["case"]
    x, dy = s["x"], s["dy"]
    cut = int(round(c["rate"] * 65536))
    keep = _random16(c["rows"], c["cols"], s["seed"], x.device) >= cut
    zero = torch.zeros((), device=x.device)
    scale = 65536.0 / (65536 - cut)
    y = torch.where(keep, x.float() * scale, zero)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(x.dtype), "dx": torch.where(keep, dy.float() * scale, zero).to(x.dtype)}


# ------------------------------------------------------------------ the framework's calls
def _own(s):
    import fp8_scaled_matmul_amd as fm
    c = s["case"]
    if c["op"] == "loss":
        loss, lse = fm.linear_cross_entropy(s["x"], s["w"], s["targets"], softcap=c["softcap"])
        return {"loss": loss, "lse": lse}
    if c["op"] == "head":
        loss, lse = fm.linear_cross_entropy(s["x"], s["w"], s["targets"], softcap=c["softcap"])
        dx, dw = fm.linear_cross_entropy_backward(s["x"], s["w"], s["targets"], lse, s["grad"], softcap=c["softcap"])
        return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}
    if c["op"] == "route":
        r = fm.moe_route(s["logits"], c["top_k"], renormalize=c["renormalize"], mask=s["mask"])
        dl = fm.moe_route_backward(s["logits"], r, s["dweights"], s["dbalance"])
        return {"ids": r.ids, "weights": r.weights, "counts": r.counts, "balance": r.balance, "dlogits": dl}
    y = fm.dropout(s["x"], c["rate"], s["seed"], residual=s["residual"])
    return {"y": y, "dx": fm.dropout(s["dy"], c["rate"], s["seed"])}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _route_plain(state) if op == "route" else _dropout_plain(state) if op == "dropout" else _head_plain(state)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=device)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=device)

    c = dict(case)
    s = {"case": c}
    if c["op"] in ("loss", "head"):
        t, v, h = c["tokens"], c["vocab"], c["hidden"]
        s["w"] = (normal(v, h) * h ** -0.5).bfloat16()
        targets = torch.randint(0, v, (t,), generator=g, device=device)
        # some tokens are foreseen well, most not: part of the target's row in the hidden state
        s["x"] = (normal(t, h) + 12 * uniform(t, 1) ** 2 * s["w"][targets].float()).bfloat16()
        targets[uniform(t) < c["ignored"]] = -100
        s["targets"] = targets
        if c["op"] == "head":           # the mean over the tokens that count
            s["grad"] = torch.full((t,), 1.0, device=device) / (targets >= 0).sum().clamp(min=1)
    elif c["op"] == "route":
        t, e, k = c["tokens"], c["experts"], c["top_k"]
        s["logits"] = (normal(t, e) * 1.5 + normal(1, e)).to(DTYPES[c["dtype"]])
        s["mask"] = uniform(t) >= c["masked"] if c["masked"] else None
        s["dweights"] = normal(t, k) * 1e-2
        s["dbalance"] = torch.full((), 0.01, device=device)
    else:
        shape = (c["rows"], c["cols"])
        s["x"] = normal(*shape).to(DTYPES[c["dtype"]])
        s["dy"] = (normal(*shape) * 1e-3).to(DTYPES[c["dtype"]])
        s["residual"] = (normal(*shape) * 4).to(DTYPES[c["dtype"]]) if c["residual"] else None
        s["seed"] = torch.randint(0, 1 << 62, (1,), generator=g, device=device)
    return s


# ------------------------------------------------------------------ the definitions in 64 bits
def _head_exact(s):
    c, cap = s["case"], s["case"]["softcap"]
    w, t = s["w"].double(), s["targets"]
    out = {"loss": [], "lse": [], "dx": []}
    dw = torch.zeros_like(w) if c["op"] == "head" else None
    for lo in range(0, c["tokens"], 2048):
        x, at = s["x"][lo:lo + 2048].double(), t[lo:lo + 2048]
        z = x @ w.t()
        slope = None
        if cap:
            th = torch.tanh(z / cap)
            z, slope = cap * th, 1 - th * th
        lse = torch.logsumexp(z, -1)
        rows = torch.nonzero(at >= 0)[:, 0]
        loss = torch.zeros_like(lse)
        loss[rows] = lse[rows] - z[rows, at[rows]]
        out["loss"].append(loss)
        out["lse"].append(lse)
        if dw is None:
            continue
        d = torch.exp(z - lse[:, None])
        d[rows, at[rows]] -= 1
        if cap:
            d *= slope
        gain = torch.zeros_like(lse)
        gain[rows] = s["grad"][lo:lo + 2048][rows].double()
        d *= gain[:, None]
        out["dx"].append(d @ w)
        dw += d.t() @ x
    r = {"loss": torch.cat(out["loss"]), "lse": torch.cat(out["lse"])}
    return r if dw is None else {**r, "dx": torch.cat(out["dx"]), "dw": dw}


def _route_exact(s):
    c, l = s["case"], s["logits"].double()
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    on = torch.arange(t, device=l.device) if s["mask"] is None else torch.nonzero(s["mask"])[:, 0]
    ids = torch.full((t, k), -1, dtype=torch.int32, device=l.device)
    weights = torch.zeros(t, k, dtype=torch.float64, device=l.device)
    dl = torch.zeros_like(l)
    a = l[on]
    p = torch.softmax(a, -1)
    best = torch.argsort(-a, dim=-1, stable=True)[:, :k]
    picked = torch.softmax(torch.gather(a, 1, best), -1) if c["renormalize"] else torch.gather(p, 1, best)
    counts = torch.bincount(best.flatten(), minlength=e)
    n = max(len(on), 1)
    fraction = counts.double() / (n * k)
    balance = e * (fraction * (p.sum(0) / n)).sum()
    gain = s["dweights"].double()[on]
    back = s["dbalance"].double() * e / n * p * (fraction - (p @ fraction)[:, None])
    inner = (picked * gain).sum(-1, keepdim=True)
    if c["renormalize"]:
        back = back.scatter_add(1, best, picked * (gain - inner))
    else:
        back = back.scatter_add(1, best, picked * gain) - p * inner
    ids[on], weights[on], dl[on] = best.int(), picked, back
    return {"ids": ids, "weights": weights, "counts": counts.int(), "balance": balance, "dlogits": dl}


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

    lo, hi = int(seed) % (1 << 32), (int(seed) >> 32) % (1 << 32)
    r = mix((times(torch.arange(rows, device=device), 2654435761) + lo) % (1 << 32))
    p = (times(torch.arange((cols + 1) // 2, device=device), 1013904243) + (hi ^ 2773480762)) % (1 << 32)
    v = mix(torch.bitwise_xor(r.unsqueeze(1), p.unsqueeze(0)))
    return torch.stack((v % 65536, v // 65536), -1).flatten(1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] in ("loss", "head"):
        return _head_exact(s)
    if c["op"] == "route":
        return _route_exact(s)
    cut = int(round(c["rate"] * 65536))
    gain = torch.where(_bits(c["rows"], c["cols"], s["seed"].item(), s["x"].device) < cut, 0.0, 65536 / (65536 - cut)).double()
    y = s["x"].double() * gain
    return {"y": y if s["residual"] is None else y + s["residual"].double(), "dx": s["dy"].double() * gain}
