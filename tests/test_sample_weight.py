"""The sampler's exponentials (csrc/sample_weight.h, compiled for the host)
against long double."""
import numpy as np
import pytest

from tests.weight_host import WeightHost

SETTINGS = [(14.32, 0.8), (14.32, 0.9), (0.0, 1.0), (5.5, 0.3), (-20.0, 2.0), (88.0, 1.3), (3.0e4, 700.0)]


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    return WeightHost(str(tmp_path_factory.mktemp("weight")))


def grid(m, T, n, seed, least=0.0):
    """Logits whose y = (m - x) log2(e) / T is anywhere from `least` to 45, half of them where the table's step ends."""
    rng = np.random.default_rng(seed)
    y = np.concatenate([rng.uniform(least, 45, n), (rng.integers(int(64 * least), 64 * 45, n) + 0.5 + rng.uniform(-0.02, 0.02, n)) / 64])
    return (m - y * T * np.log(2)).astype(np.float32)


@pytest.mark.parametrize("m,T", SETTINGS)
def test_whole_numbers_far_from_the_largest(host, m, T):
    """y from 8 on, where the second part of 1 - 2^-r is largest: its whole number is no other than the one nearest.

    Bound: ah al <= 2^-7.5 2^-17.5 of the weight, the other terms together below 2^-35 of it."""
    rel, _ = host.errors(grid(m, T, 200000, 1, least=8.0), m, T)
    assert rel.max() <= 2.0 ** -24.9, np.log2(rel.max())


@pytest.mark.parametrize("m,T", SETTINGS)
def test_weights_are_good_to_their_bound(host, m, T):
    """Within 2^-35 of themselves and half a unit, wherever they are.

    Of the weight: the table's 15 low bits left out times |1 - 2^-r| < 2^-7.5: 2^-36.5; two whole numbers rounded, 2^-38;
    fp32 roundings of v (below 2^-15.5), 2^-39; al^2 / 2, 2^-36.2; what is left of the series, the shift and the table's
    own rounding, below 2^-43 together."""
    rel, exact = host.errors(grid(m, T, 500000, 2), m, T)
    assert rel.max() <= 2.0 ** -35, np.log2(rel.max())
    assert (rel * exact).max() <= 2.0 ** (44 - 36), np.log2((rel * exact).max())  # of the largest weight, where al is small


def test_weights_at_the_ends(host):
    """The largest itself, what is below half a unit, infinite and huge differences."""
    w = host.weights([2.0, 2.0 - 31.5, -1e30, -np.inf, -3.4e38], 2.0, 1.0)
    assert w.tolist() == [1 << 44, 0, 0, 0, 0]
    assert host.weights([3.3e38, -3.3e38], 3.3e38, 1.0).tolist() == [1 << 44, 0]
    assert host.weights([0.0, 1.0], 1.0, 3e38).tolist() == [1 << 44, 1 << 44]
    assert host.weights([1.0, np.nextafter(np.float32(1), np.float32(0))], 1.0, 1e-30).tolist() == [1 << 44, 0]
