"""Dropout of tensors that are read and written past the caches (more than 256 MiB
moved): each type, with and without a residual, ragged rows, views, in place; every
element against the definition in float64 on the GPU."""
import numpy as np
import pytest
import torch

import fp8_scaled_matmul_amd as fm
from oracle import train

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "fp32": (torch.float32, 2.0 ** -24)}
MASK = 0xFFFFFFFF


def bits(rows, cols, seed, device="cuda"):
    """train.dropout_bits in int64 tensors (products below 2^64: mod 2^32 they wrap
    rightly)."""
    def mix(v):
        v = v ^ v >> 16
        v = v * 0x6A09E667 & MASK
        v = v ^ v >> 15
        v = v * 0xBB67AE85 & MASK
        return v ^ v >> 16

    lo, hi = seed & MASK, seed >> 32 & MASK ^ 0xA54FF53A
    row = mix(torch.arange(rows, device=device) * 0x9E3779B1 + lo & MASK)
    col = torch.arange((cols + 1) // 2, device=device) * 0x3C6EF373 + hi & MASK
    v = mix(row[:, None] ^ col[None, :])
    return torch.stack((v & 0xFFFF, v >> 16), -1).flatten(1)[:, :cols]


def test_bits_are_the_oracles():
    for rows, cols, seed in ((40, 33, 77), (3, 130, -5), (9, 8, 1 << 40 | 3)):
        assert np.array_equal(bits(rows, cols, seed).cpu().numpy(), train.dropout_bits(rows, cols, seed))


def check(x, rate, seed, residual, y, dtype):
    """One product and one sum in fp32 (the scale is off by half a step), one
    rounding to the type."""
    cut = round(rate * 65536)
    drop = torch.where(bits(*x.shape, seed) >= cut, x.double() * (65536.0 / (65536 - cut)), 0.0)
    ref = drop if residual is None else drop + residual.double()
    bound = 2 * 2.0 ** -24 * drop.abs() + DTYPES[dtype][1] * ref.abs() * (1 + 2.0 ** -20) + 2.0 ** -126
    assert ((y.double() - ref).abs() <= bound).all()
    if residual is None:
        assert torch.equal(y == 0, ref == 0)


@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("dtype,rows,cols", [("bf16", 8003, 9001), ("bf16", 70001, 1027), ("fp32", 8003, 5001), ("fp32", 20001, 2050)])
def test_past_the_caches(dtype, rows, cols, with_residual):
    gen = torch.Generator(device="cuda").manual_seed(cols)
    size = 2 if dtype == "bf16" else 4
    assert rows * cols * size * (3 if with_residual else 2) > 256 << 20

    def make(pad):
        """A view that leaves pad columns on either side, and what it lies in."""
        big = torch.full((rows + 2, cols + 2 * pad), 7.0, dtype=DTYPES[dtype][0], device="cuda")
        v = big[1:-1, pad:-pad]
        v.copy_(torch.randn(rows, cols, generator=gen, device="cuda") * 3)
        return big, v

    seed, s = 1 << 50 | 12345, torch.tensor([1 << 50 | 12345], device="cuda")
    (_, x), (_, res), (big, out) = make(1), make(3), make(8)
    if not with_residual:
        res = None
    held = x.clone()
    y = fm.dropout(x, 0.25, s, residual=res)
    assert torch.equal(x, held)
    check(x, 0.25, seed, res, y, dtype)
    assert fm.dropout(x, 0.25, s, residual=res, out=out) is out and torch.equal(out, y)
    out.fill_(7.0)
    assert (big == 7.0).all()
    into = x if res is None else res
    fm.dropout(x, 0.25, s, residual=res, out=into)
    assert torch.equal(into, y) and (res is None or torch.equal(x, held))
