"""Dropout on the GPU against the float64 oracle: the mask exactly, the values
to one rounding."""
import numpy as np
import pytest
import torch

import fp8_scaled_matmul_amd as fm
from oracle import train

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def seed_of(v):
    return torch.tensor([v], dtype=torch.int64, device="cuda")


def check(x, rate, seed, residual, y, dtype, bits=None):
    """One product and one sum in fp32 (the scale is off by half a step), one
    rounding to the type."""
    X, R = x.double().numpy(), None if residual is None else residual.double().numpy()
    ref = train.dropout(X, rate, seed, R, bits)
    drop = train.dropout(X, rate, seed, None, bits)
    bound = 2 * 2.0 ** -24 * np.abs(drop) + HALF[dtype] * np.abs(ref) * (1 + 2.0 ** -20) + 2.0 ** -126
    got = y.double().cpu().numpy()
    assert (np.abs(got - ref) <= bound).all()
    if residual is None:
        assert np.array_equal(got == 0, ref == 0)


@pytest.mark.parametrize("rate", [0.0, 0.1, 0.5, 1.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 9), (3, 64), (5, 33), (70, 7), (9, 520), (2, 1031), (33, 512)])
def test_against_oracle(rows, cols, dtype, rate):
    rng = np.random.default_rng(rows + cols)
    x, res = [torch.from_numpy((rng.normal(size=(rows, cols)) * 3).astype(np.float32)).to(DTYPES[dtype]) for _ in range(2)]
    seed = int(rng.integers(-2 ** 63, 2 ** 63))
    bits = train.dropout_bits(rows, cols, seed)
    for r in (None, res):
        y = fm.dropout(x.cuda(), rate, seed_of(seed), residual=None if r is None else r.cuda())
        assert y.dtype == x.dtype
        check(x, rate, seed, r, y, dtype, bits)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides_alignment_and_in_place(dtype):
    rng = np.random.default_rng(4)
    x, res = [torch.from_numpy(rng.normal(size=(20, 77)).astype(np.float32)).to(DTYPES[dtype]) for _ in range(2)]
    want = fm.dropout(x.cuda(), 0.3, seed_of(7), residual=res.cuda())
    check(x, 0.3, 7, res, want, dtype)
    for pad in (1, 3, 8):
        bufs = [torch.full((22, 77 + 2 * pad), 7.0, dtype=DTYPES[dtype], device="cuda") for _ in range(3)]
        vx, vr, vo = [b[1:-1, pad:-pad] for b in bufs]
        vx.copy_(x)
        vr.copy_(res)
        assert fm.dropout(vx, 0.3, seed_of(7), residual=vr, out=vo) is vo
        assert torch.equal(vo, want)
        vo.fill_(7.0)
        assert (bufs[2] == 7.0).all()
        fm.dropout(vx, 0.3, seed_of(7), residual=vr, out=vr)
        assert torch.equal(vr, want)
        fm.dropout(vx, 0.3, seed_of(7), out=vx)
        assert torch.equal(vx, fm.dropout(x.cuda(), 0.3, seed_of(7)))


def test_backward_draws_the_same_mask_and_the_gradient_is_linear():
    x = torch.randn(100, 300, device="cuda") + 10
    s = seed_of(99)
    y, dx = fm.dropout(x, 0.4, s), fm.dropout(torch.ones_like(x), 0.4, s)
    assert torch.equal(y == 0, dx == 0)
    # y = x dx for one and the same fp32 factor
    assert torch.equal(y, x * dx)


def test_dropped_elements_may_hold_anything():
    x = torch.randn(50, 130)
    drop = torch.from_numpy(train.dropout(np.ones((50, 130)), 0.5, 3) == 0)
    x2 = x.clone()
    x2[drop] = float("nan")
    x2[0][drop[0]] = float("inf")
    assert torch.equal(fm.dropout(x2.cuda(), 0.5, seed_of(3)), fm.dropout(x.cuda(), 0.5, seed_of(3)))


def test_the_rate_holds():
    # 2^22 draws: a standard deviation of 2^-11 sqrt(p (1 - p))
    x = torch.ones(2048, 2048, dtype=torch.bfloat16, device="cuda")
    for rate in (0.1, 0.5, 0.9):
        share = (fm.dropout(x, rate, seed_of(11)) == 0).double().mean().item()
        assert abs(share - round(rate * 65536) / 65536) < 5 * 2.0 ** -11 * (rate * (1 - rate)) ** 0.5


def test_far_offsets_and_no_elements():
    """Elements past 2^32 bytes from the first: the bits go by row and column."""
    rows, cols = 140000, 16384
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    y = fm.dropout(x, 0.25, seed_of(5))
    last = x[-3:, -200:].cpu()
    def mix(v):
        v ^= v >> 16
        v = v * 0x6A09E667 & 0xFFFFFFFF
        v ^= v >> 15
        v = v * 0xBB67AE85 & 0xFFFFFFFF
        return v ^ v >> 16
    got = y[-3:, -200:].cpu()
    for r in range(3):
        key = mix((rows - 3 + r) * 0x9E3779B1 + 5 & 0xFFFFFFFF)
        for c in range(0, 200, 2):
            v = mix(key ^ ((cols - 200 + c) // 2 * 0x3C6EF373 + 0xA54FF53A & 0xFFFFFFFF))
            assert (got[r, c] != 0) == ((v & 0xFFFF) >= 16384) and (got[r, c + 1] != 0) == ((v >> 16) >= 16384)
    assert last.shape == (3, 200)
    for shape in ((0, 5), (5, 0)):
        e = torch.empty(shape, device="cuda")
        assert fm.dropout(e, 0.5, seed_of(1)).shape == shape


def test_captured_graph_reads_the_seed_anew():
    x, s = torch.randn(64, 256, device="cuda").bfloat16(), seed_of(1)
    y = torch.empty_like(x)
    fm.dropout(x, 0.5, s, out=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fm.dropout(x, 0.5, s, out=y)
    seen = []
    for v in (1, 2, -3):
        s.fill_(v)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, fm.dropout(x, 0.5, seed_of(v)))
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        z = fm.dropout(x, 0.5, s)
    side.synchronize()
    assert torch.equal(z, y)
