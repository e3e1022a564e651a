"""Pins of the 4-bit oracle: closed forms and exhaustive properties, CPU."""
import numpy as np
import pytest

from oracle import mx4


def _all_bf16():
    b = np.arange(65536, dtype=np.uint32) << 16
    return b.view(np.float32).astype(np.float64)


def test_block_exponent_is_the_smallest():
    for v in np.unique(np.abs(_all_bf16()[np.isfinite(_all_bf16())]))[::37]:
        e = mx4.block_exponent(v)
        if v == 0:
            assert e == 0
        else:
            assert v <= 6 * 2.0 ** e and (e == -126 or v > 6 * 2.0 ** (e - 1))


@pytest.mark.parametrize("v,code", [(0.25, 0), (0.2500001, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6),
                                    (5.0, 6), (5.01, 7), (6.0, 7), (-0.2, 8), (-5.0, 14)])
def test_ties_go_to_the_even_code(v, code):
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1] = 6.0, v          # the block's scale is 1
    codes, sb, _ = mx4.quantize(x)
    assert sb[0, 0] == 127 and codes[0, 1] == code


def test_grid_values_are_kept_and_zero_blocks_get_scale_one():
    x = np.concatenate([mx4.VALUES, np.zeros(32 - 16), np.zeros(32)])[None, :] * 0.125
    codes, sb, ctr = mx4.quantize(x)
    assert np.array_equal(mx4.values(codes, sb), x) and list(sb[0]) == [124, 127] and ctr["underflow"] == 0


def test_nonfinite_blocks():
    x = np.ones((3, 64))
    x[0, 3] = np.inf
    x[1, 40] = np.nan
    x[2, 0], x[2, 1] = -np.inf, np.nan
    codes, sb, ctr = mx4.quantize(x)
    assert codes[0, 3] == 7 and sb[0, 0] == 125 and sb[1, 1] == 255 and (codes[1, 32:] == 0).all()
    assert ctr["saturated"] == 2 and ctr["nan"] == 2
    assert np.isnan(mx4.values(codes, sb)[2, :32]).all()


def test_stochastic_mean_is_the_value():
    """The mean over the 65536 equally likely draws is floor(v's fraction)."""
    x = np.zeros((1, 32))
    x[0, :4] = 6.0, 0.3, 2.7, 5.5
    r = np.arange(65536)
    for c in (1, 2, 3):
        k, lo = 0.0, mx4.GRID[(mx4.GRID <= x[0, c]).sum() - 1]
        gap = 0.5 if lo < 2 else 1.0 if lo < 4 else 2.0
        k = np.floor((x[0, c] - lo) / gap * 65536)
        bits = np.zeros((65536, 32), dtype=np.int64)
        bits[:, c] = r
        codes, sb, _ = mx4.quantize(np.repeat(x, 65536, 0), bits)
        assert np.isclose(mx4.values(codes, sb)[:, c].mean(), lo + gap * k / 65536, rtol=0, atol=1e-12)


def test_random_bits_are_spread():
    """Each of the 16 bits is set half the time, neighbours are uncorrelated."""
    r = mx4.random_bits(512, 512, 0x1234567890)
    n = r.size
    for b in range(16):
        bit = (r >> b) & 1
        assert abs(bit.mean() - 0.5) < 5 * 0.5 / np.sqrt(n)
        for d in ((0, 1), (1, 0), (0, 2)):
            u, v = bit[: 512 - d[0], : 512 - d[1]], bit[d[0]:, d[1]:]
            assert abs((u == v).mean() - 0.5) < 5 * 0.5 / np.sqrt(u.size)
    assert (mx4.random_bits(8, 8, 1) != mx4.random_bits(8, 8, 2)).any()


def test_layout_round_trip():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (5, 700)).astype(np.uint8)
    sb = rng.integers(0, 255, (5, 22)).astype(np.uint8)
    q, s = mx4.pack(codes, sb)
    assert q.shape == (5, 384) and s.shape == (2, 5, 16)
    assert s[1, 3, 2] == sb[3, 18] and q[2, 10] == codes[2, 20] + 16 * codes[2, 21]
    c2, s2 = mx4.unpack(q, s, 700)
    assert np.array_equal(c2, codes) and np.array_equal(s2, sb)


def test_moe_closed_form():
    """One expert, identity-like weights: y = silu(x) * x."""
    x = np.array([[0.5, -1.0]])
    w1 = np.concatenate([np.eye(2), np.eye(2)])[None]
    y, ids, p = mx4.moe(x, np.zeros((1, 2)), w1, np.eye(2)[None], 1, True)
    assert np.allclose(y, x / (1 + np.exp(-x)) * x) and ids[0, 0] == 0 and p[0, 0] == 1
    # equal logits: the lower experts
    _, ids, p = mx4.moe(x, np.zeros((4, 2)), np.repeat(w1, 4, 0), np.repeat(np.eye(2)[None], 4, 0), 2, False)
    assert list(ids[0]) == [0, 1] and np.allclose(p, 0.25)
