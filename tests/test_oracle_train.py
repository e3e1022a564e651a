"""The float64 oracle of the training operators: gradients against differences,
hand-made cases, the generator's bits."""
import numpy as np
import pytest

from oracle import train


def _numeric(f, a, step=1e-6):
    g = np.zeros_like(a)
    for i in np.ndindex(*a.shape):
        hi, lo = a.copy(), a.copy()
        hi[i] += step
        lo[i] -= step
        g[i] = (f(hi) - f(lo)) / (2 * step)
    return g


# central differences with a step of 1e-6: truncation 1e-12 of third
# derivatives of order 1, rounding 2^-53 of losses of order 10 over 2e-6, 1e-9
@pytest.mark.parametrize("softcap", [0.0, 2.0])
def test_cross_entropy_gradient_matches_differences(softcap):
    rng = np.random.default_rng(1)
    x, w = rng.normal(size=(4, 5)), rng.normal(size=(7, 5))
    t, g = np.array([3, -100, 0, 6]), rng.normal(size=4)
    dx, dw = train.cross_entropy_backward(x, w, t, g, softcap)
    f = lambda a, b: (train.cross_entropy(a, b, t, softcap)[0] * g).sum()
    assert np.abs(dx - _numeric(lambda a: f(a, w), x)).max() < 1e-7
    assert np.abs(dw - _numeric(lambda b: f(x, b), w)).max() < 1e-7


def test_cross_entropy_by_hand():
    x, w = np.array([[1.0, 2.0], [1.0, 2.0]]), np.array([[0.0, 0.0], [0.0, 1.0], [1.0, 0.5]])
    loss, lse = train.cross_entropy(x, w, np.array([0, 3]))       # logits 0, 2, 2
    assert np.allclose(lse, np.log(1 + 2 * np.exp(2.0)))
    assert np.isclose(loss[0], lse[0]) and np.isnan(loss[1])


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_matches_differences(renormalize):
    rng = np.random.default_rng(2)
    l, gw, gb = rng.normal(size=(5, 6)), rng.normal(size=(5, 2)), 0.7
    mask = np.array([1, 1, 0, 1, 1], bool)
    ids, _, counts, _ = train.route(l, 2, renormalize, mask)

    def f(a):       # the choice is held: differences do not cross a border
        i, w, c, b = train.route(a, 2, renormalize, mask)
        assert np.array_equal(i, ids)
        return (w * gw).sum() + gb * b

    d = train.route_backward(l, ids, counts, renormalize, gw, gb)
    assert np.abs(d - _numeric(f, l)).max() < 1e-7


def test_route_order_and_empty_rows():
    l = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [0.0, 0.0, 0.0, 0.0]])
    ids, w, counts, balance = train.route(l, 2, True)
    assert ids.tolist() == [[1, 2], [-1, -1], [0, 1]] and w[0].tolist() == [0.5, 0.5] and w[1].tolist() == [0, 0]
    assert counts.tolist() == [1, 2, 1, 0]
    ids, *_ = train.route(np.array([[np.nan, -1.0, 2.0]]), 3, True)
    assert ids.tolist() == [[2, 1, 0]]


def test_dropout_bits_are_even_and_apart_from_the_rounding_bits():
    b = train.dropout_bits(64, 257, 1234567890123456789)
    # 16448 draws of a uniform 16-bit number: the mean lies within 5 standard
    # deviations (65536 / sqrt(12 * 16448) = 147.5) of its expectation
    assert abs(b.mean() - 32767.5) < 5 * 147.5
    assert not np.array_equal(b, train.dropout_bits(64, 257, 1234567890123456790))
    from oracle import mx4
    # two streams agree on an element with probability 2^-16
    assert (mx4.random_bits(64, 257, 1234567890123456789) == b).mean() < 0.01
    x = np.ones((64, 257))
    y = train.dropout(x, 0.25, 5)
    assert set(np.unique(y)) == {0.0, 65536.0 / (65536 - 16384)}
    # 16448 draws at 0.25: standard deviation 0.0034
    assert abs((y == 0).mean() - 0.25) < 5 * 0.0034
    assert (train.dropout(x, 1.0, 5) == 0).all() and (train.dropout(x, 0.0, 5) == x).all()
