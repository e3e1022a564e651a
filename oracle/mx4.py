"""CPU oracle of the 4-bit (OCP MXFP4) operators -- TEST INFRASTRUCTURE ONLY,
like the rest of this package.  Plain numpy in float64, from the definitions
in include/fp8mi.h; shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([GRID, -GRID])      # by code


def random_bits(rows: int, cols: int, seed: int, row0: int = 0) -> np.ndarray:
    """The 16 random bits of each element, integers [rows, cols]."""
    def mix(v):
        v = (v ^ (v >> 16)) * 0x6A09E667 % (1 << 32)
        v = (v ^ (v >> 15)) * 0xBB67AE85 % (1 << 32)
        return v ^ (v >> 16)

    r = np.arange(row0, row0 + rows, dtype=np.uint64)
    c = np.arange(cols, dtype=np.uint64)
    seed = int(seed) & 0xFFFFFFFFFFFFFFFF
    lo, hi = np.uint64(seed & 0xFFFFFFFF), np.uint64(seed >> 32)
    row = mix((r * np.uint64(0x9E3779B1) + lo) % np.uint64(1 << 32))
    pair = ((c // 2) * np.uint64(0x3C6EF373) + hi) % np.uint64(1 << 32)
    v = mix(row[:, None] ^ pair[None, :])
    return np.where((c % 2 == 1)[None, :], v >> np.uint64(16), v & np.uint64(0xFFFF)).astype(np.int64)


def block_exponent(amax: float) -> int:
    """Smallest e >= -126 with amax <= 6 * 2^e (0 for amax 0), by search."""
    if amax == 0.0:
        return 0
    e = -126
    while amax > 6.0 * 2.0 ** e:
        e += 1
    return e


def quantize(x: np.ndarray, bits: np.ndarray | None = None):
    """x [rows, cols] (float64 holding the input's values) to (codes uint8
    [rows, cols], scale bytes uint8 [rows, ceil(cols/32)], counters)."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = -(-cols // 32)
    codes = np.zeros((rows, cols), dtype=np.uint8)
    sb = np.full((rows, nb), 127, dtype=np.uint8)
    ctr = {"saturated": int(np.isinf(x).sum()), "underflow": 0, "nan": int(np.isnan(x).sum())}
    for b in range(nb):
        blk = x[:, 32 * b: 32 * b + 32]
        fin = np.where(np.isfinite(blk), np.abs(blk), 0.0)
        amax = fin.max(axis=1)
        e = np.array([block_exponent(a) for a in amax])
        bad = np.isnan(blk).any(axis=1)
        with np.errstate(invalid="ignore"):
            v = np.where(np.isinf(blk), 6.0, np.abs(np.where(np.isnan(blk), 0.0, blk)) / 2.0 ** e[:, None])
        if bits is None:
            d = np.abs(v[..., None] - GRID)
            near = d.min(axis=-1, keepdims=True)
            # of two equally near codes the even one
            c = np.argmax((d == near) & ((d == near).sum(axis=-1, keepdims=True) == 1) |
                          (d == near) & (np.arange(8) % 2 == 0), axis=-1)
        else:
            c = (v[..., None] >= GRID).sum(axis=-1) - 1
            up = np.minimum(c + 1, 7)
            gap = np.where(up > c, GRID[up] - GRID[c], 1.0)
            frac = (v - GRID[c]) / gap
            c = np.where(frac * 65536 + bits[:, 32 * b: 32 * b + 32] >= 65536, up, c)
        c = np.where(bad[:, None], 0, c + 8 * np.signbit(blk))
        codes[:, 32 * b: 32 * b + 32] = c
        sb[:, b] = np.where(bad, 255, e + 127)
        ctr["underflow"] += int(((blk != 0) & (c % 8 == 0) & ~bad[:, None]).sum())
    return codes, sb, ctr


def pack(codes: np.ndarray, sb: np.ndarray):
    """Codes and scale bytes as the library lays them out."""
    rows, cols = codes.shape
    full = np.zeros((rows, 256 * -(-cols // 256)), dtype=np.uint8)
    full[:, :cols] = codes
    panels = -(-cols // 512)
    s = np.full((rows, 16 * panels), 127, dtype=np.uint8)
    s[:, : sb.shape[1]] = sb
    return full[:, 0::2] | (full[:, 1::2] << 4), np.ascontiguousarray(s.reshape(rows, panels, 16).transpose(1, 0, 2))


def values(codes: np.ndarray, sb: np.ndarray) -> np.ndarray:
    """What codes and scales stand for, float64."""
    scale = np.where(sb == 255, np.nan, 2.0 ** (sb.astype(np.float64) - 127))
    return VALUES[codes] * np.repeat(scale, 32, axis=1)[:, : codes.shape[1]]


def unpack(q: np.ndarray, s: np.ndarray, cols: int):
    """The library's layout to (codes, scale bytes)."""
    codes = np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[0], -1)[:, :cols]
    sb = s.transpose(1, 0, 2).reshape(q.shape[0], -1)[:, : -(-cols // 32)]
    return codes, sb


def mm(a: np.ndarray, b: np.ndarray):
    """(A B^T, |A| |B|^T) of float64 values: the product and the size of what
    is summed, for error bounds."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def moe(x, router, w1, w2, top_k: int, renormalize: bool):
    """x [t, h], router [e, h], w1 [e, 2 i, h] (gate rows, then up rows), w2
    [e, h, i], all float64: (y [t, h], ids [t, k], weights [t, k]); equal
    logits go to the lower expert."""
    logits = x @ router.T
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :top_k]
    z = np.exp(logits - logits.max(axis=1, keepdims=True))
    p = np.take_along_axis(z / z.sum(axis=1, keepdims=True), ids, axis=1)
    if renormalize:
        z = np.take_along_axis(z, ids, axis=1)
        p = z / z.sum(axis=1, keepdims=True)
    i = w2.shape[2]
    y = np.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(top_k):
            e = ids[t, j]
            g, u = w1[e, :i] @ x[t], w1[e, i:] @ x[t]
            y[t] += p[t, j] * (w2[e] @ (g / (1 + np.exp(-g)) * u))
    return y, ids, p
