"""Pins of oracle/paged.py (CPU): rotations against complex products and finite differences,
attention against a dense masked softmax, and the cases that leave a row empty."""

import numpy as np
import pytest

from oracle import attention as dense
from oracle import e4m3, paged, rope


def test_rotation_is_roformers_on_the_whole_head():
    x = np.random.default_rng(0).standard_normal((7, 2, 64))
    th, gain = paged.frequencies(64)
    got = paged.rotate(x, np.arange(7), th, gain)
    np.testing.assert_allclose(got, rope.rope(x[None])[0], rtol=0, atol=1e-14)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0)])
def test_transposed_rotation_is_the_gradient(half, scaling, factor):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((2, 5, 3, 64))
    pos = rng.integers(0, 100000, 5)
    th, gain = paged.frequencies(32, 10000.0, scaling, factor, 4096.0)
    dx = paged.rotate(dy, pos, th, gain, half, transpose=True)
    for _ in range(20):
        e = rng.standard_normal(x.shape)
        d = (paged.rotate(x + e, pos, th, gain, half) - paged.rotate(x - e, pos, th, gain, half)) / 2
        np.testing.assert_allclose((d * dy).sum(), (e * dx).sum(), rtol=1e-11, atol=1e-11)


def test_stretched_frequencies():
    th, _ = paged.frequencies(64)
    np.testing.assert_allclose(paged.frequencies(64, scaling="linear", factor=4.0)[0], th / 4)
    ntk = paged.frequencies(64, scaling="ntk", factor=8.0)[0]
    np.testing.assert_allclose([ntk[0], ntk[-1]], [th[0], th[-1] / 8])      # highest kept, lowest divided
    y, gain = paged.frequencies(64, scaling="yarn", factor=16.0, length=4096.0)
    turns = 4096 * th / (2 * np.pi)
    np.testing.assert_allclose(y[turns >= 32], th[turns >= 32])
    np.testing.assert_allclose(y[turns <= 1], th[turns <= 1] / 16)
    assert np.all((y <= th) & (y >= th / 16)) and gain == 0.1 * np.log(16.0) + 1


def test_rows_quantise_to_their_largest_value():
    x = np.random.default_rng(2).standard_normal((9, 64))
    x[3] = 0
    codes, scale, pre = paged.quantise_rows(x)
    val = e4m3.decode(codes) * scale[:, None]
    assert scale[3] == 1 and np.all(codes[3] == 0)
    assert np.all(np.abs(val - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale[:, None]))
    live = np.arange(9) != 3
    np.testing.assert_allclose(np.abs(val).max(-1)[live], np.abs(x).max(-1)[live])


def test_chain_is_causal_attention():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 12, 2, 64))
    o, lse, *_ = paged.tree_attention(q[5:], k, v, 5, None, 0.125)
    O, LSE = dense.attention(q[None], k[None], v[None], causal=True)
    np.testing.assert_allclose(o, O[0, 5:], atol=1e-12)
    np.testing.assert_allclose(lse, LSE[0, :, 5:], atol=1e-12)


def test_tree_sees_ancestors_only_and_empty_rows_are_zero():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 3, 1, 64))
    o, lse, *_ = paged.tree_attention(q, k, v, 0, [0b001, 0b000, 0b101], 0.125)
    np.testing.assert_allclose(o[0, 0], v[0, 0])
    assert np.all(o[1] == 0) and lse[0, 1] == -np.inf
    x = 0.125 * (k[[0, 2], 0] @ q[2, 0])
    np.testing.assert_allclose(lse[0, 2], np.log(np.exp(x).sum()))
