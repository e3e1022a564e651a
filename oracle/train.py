"""float64 oracle of the training operators around the linear layers, in numpy
and from their definitions: the vocabulary loss, the experts' router, dropout.
Shares no code with the HIP path."""
import numpy as np

MASK = 0xFFFFFFFF


def logits(x, w, softcap=0.0):
    """(z, dz/dl) of x [tokens, hidden], w [vocab, hidden]."""
    l = x.astype(np.float64) @ w.astype(np.float64).T
    if softcap == 0:
        return l, np.ones_like(l)
    th = np.tanh(l / softcap)
    return softcap * th, 1.0 - th * th


def cross_entropy(x, w, targets, softcap=0.0):
    """(loss, lse)."""
    z, _ = logits(x, w, softcap)
    big = z.max(1)
    lse = big + np.log(np.exp(z - big[:, None]).sum(1))
    loss = np.zeros_like(lse)
    for t, at in enumerate(targets):
        if at >= w.shape[0]:
            loss[t] = np.nan
        elif at >= 0:
            loss[t] = lse[t] - z[t, at]
    return loss, lse


def logits_grad(x, w, targets, grad, softcap=0.0):
    """(dl, softmax probabilities times |grad| and slope): tokens whose target
    lies outside the vocabulary are zeros."""
    z, slope = logits(x, w, softcap)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    on = (targets >= 0) & (targets < w.shape[0])
    d = p.copy()
    rows = np.nonzero(on)[0]
    d[rows, targets[rows]] -= 1.0
    g = np.where(on, grad, 0.0)[:, None]
    return np.where(on[:, None], d * g * slope, 0.0), np.where(on[:, None], p * np.abs(g) * slope, 0.0)


def cross_entropy_backward(x, w, targets, grad, softcap=0.0):
    """(dx, dw)."""
    d, _ = logits_grad(x, w, targets, grad, softcap)
    on = (targets >= 0) & (targets < w.shape[0])
    return d @ w.astype(np.float64), d.T @ np.where(on[:, None], x, 0).astype(np.float64)


def route(l, top_k, renormalize=True, mask=None):
    """ids, weights, counts, balance."""
    l = l.astype(np.float64)
    tokens, experts = l.shape
    ids = np.full((tokens, top_k), -1, np.int32)
    weights = np.zeros((tokens, top_k))
    mean = np.zeros(experts)
    counts = np.zeros(experts, np.int64)
    n = 0
    for t in range(tokens):
        if (mask is not None and not mask[t]) or np.all(l[t] == -np.inf):
            continue
        n += 1
        order = sorted(range(experts), key=lambda e: (np.isnan(l[t, e]), -l[t, e] if not np.isnan(l[t, e]) else 0, e))
        ids[t] = order[:top_k]
        p = np.exp(l[t] - np.nanmax(l[t]))
        weights[t] = p[ids[t]] / (p[ids[t]].sum() if renormalize else p.sum())
        mean += p / p.sum()
        np.add.at(counts, ids[t], 1)
    balance = experts * (counts / (n * top_k) * (mean / n)).sum() if n else 0.0
    return ids, weights, counts, balance


def route_backward(l, ids, counts, renormalize, grad_weights=None, grad_balance=0.0):
    """dlogits, from the choice as given."""
    l = l.astype(np.float64)
    tokens, experts = l.shape
    top_k = ids.shape[1]
    n = counts.sum() / top_k
    out = np.zeros_like(l)
    for t in range(tokens):
        if ids[t, 0] < 0:
            continue
        p = np.exp(l[t] - l[t].max())
        p /= p.sum()
        dp = grad_balance * experts * counts / (n * n * top_k)
        out[t] = p * (dp - (p * dp).sum())
        if grad_weights is None:
            continue
        g = grad_weights[t].astype(np.float64)
        if renormalize:
            w = p[ids[t]] / p[ids[t]].sum()
            out[t, ids[t]] += w * (g - (w * g).sum())
        else:
            w = p[ids[t]]
            out[t, ids[t]] += w * g
            out[t] -= p * (w * g).sum()
    return out


def dropout_bits(rows, cols, seed):
    """The 16 random bits of every element, in Python integers."""
    def mix(v):
        v ^= v >> 16
        v = v * 0x6A09E667 & MASK
        v ^= v >> 15
        v = v * 0xBB67AE85 & MASK
        return v ^ v >> 16

    lo, hi = seed & MASK, seed >> 32 & MASK ^ 0xA54FF53A
    out = np.empty((rows, cols), np.int64)
    for r in range(rows):
        key = mix(r * 0x9E3779B1 + lo & MASK)
        for c in range(0, cols, 2):
            v = mix(key ^ (c // 2 * 0x3C6EF373 + hi & MASK))
            out[r, c] = v & 0xFFFF
            if c + 1 < cols:
                out[r, c + 1] = v >> 16
    return out


def dropout(x, rate, seed, residual=None, bits=None):
    cut = int(round(rate * 65536))
    bits = dropout_bits(*x.shape, seed) if bits is None else bits
    gain = 65536.0 / (65536 - cut) if cut < 65536 else 0.0
    with np.errstate(invalid="ignore"):
        y = np.where(bits >= cut, x.astype(np.float64) * gain, 0.0)
    return y if residual is None else y + residual.astype(np.float64)
