"""Pins of the MXFP4 oracle: the format's values, rounding by brute force, the scale rule, and packing."""
import numpy as np
import pytest
import torch

from oracle import mx4


def test_values():
    assert mx4.VALUES.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert mx4.TABLE[8:].tolist() == [-0.0, -0.5, -1, -1.5, -2, -3, -4, -6]


def test_ties_go_to_the_even_code():
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6}
    for v, c in ties.items():
        assert mx4.encode(np.array([v, -v])).tolist() == [c, c + 8]
        assert mx4.encode(np.array([np.nextafter(v, 0), np.nextafter(v, 9)])).tolist() == sorted({c, c + 1, c - 1} & {
            int(np.searchsorted(mx4.VALUES, v)) - 1, int(np.searchsorted(mx4.VALUES, v))})
    assert mx4.encode(np.array([6.0, 7.9, 100.0, -1e30, 0.0, -0.0])).tolist() == [7, 7, 7, 15, 0, 8]


@pytest.mark.parametrize("amax,byte", [(0.0, 0), (6.0, 127), (4.0, 127), (7.99, 127), (8.0, 128), (1.0, 125), (2.0 ** -130, 0),
                                       (2.0 ** 127, 252)])
def test_scale_rule(amax, byte):
    v = np.zeros((1, 32))
    v[0, 5] = -amax
    assert mx4.quantise(v)[1].tolist() == [[byte]]


def test_broken_blocks():
    v = np.ones((2, 64))
    v[0, 3], v[1, 40] = np.nan, -np.inf
    c, s = mx4.quantise(v)
    assert s.tolist() == [[255, 125], [125, 255]] and not c[0, :32].any() and c[0, 32:].all()


def test_packing_and_values():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 256, (5, 128), dtype=np.uint8)
    scales = rng.integers(100, 150, (2, 5, 4), dtype=np.uint8)
    m = mx4.values(codes, scales)
    for n, k in [(0, 0), (4, 255), (2, 131), (3, 64)]:
        code = (codes[n, k // 2] >> (4 * (k % 2))) & 15
        assert m[n, k] == mx4.TABLE[code] * 2.0 ** (int(scales[k // 128, n, k % 128 // 32]) - 127)


def test_representable_values_return():
    rng = np.random.default_rng(1)
    c = rng.integers(0, 16, (7, 96))
    c[:, ::32] = 7      # every block holds the largest value, so its scale comes back
    v = mx4.TABLE[c] * 2.0 ** rng.integers(-20, 20, (7, 3)).repeat(32, axis=1)
    got, s = mx4.quantise(v)
    assert np.array_equal(got, c) and np.array_equal(mx4.TABLE[got] * np.repeat(2.0 ** (s.astype(int) - 127), 32, axis=1), v)


def test_swiglu_is_torchs():
    a, u = np.random.default_rng(2).normal(size=(2, 50)) * 4
    want = torch.nn.functional.silu(torch.tensor(a)) * torch.tensor(u)
    assert np.allclose(mx4.swiglu(a, u), want.numpy(), rtol=1e-14)
