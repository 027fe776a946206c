"""Pins of the oracle of rotary positions, head norms and chunks: closed forms and invariants."""
import math

import numpy as np
import pytest

from oracle import serve


def test_rope_by_hand():
    x = np.array([[[1.0, 0.0, 3.0, 7.0]]])
    y, size = serve.rope(x, [1], [math.pi / 2], "interleaved", 2.0)
    assert np.allclose(y, [[[0.0, 2.0, 3.0, 7.0]]], atol=1e-15) and np.allclose(size, [[[2, 2, 3, 7]]])
    y, _ = serve.rope(x, [1], [math.pi / 2, math.pi], "half", 1.0)
    assert np.allclose(y, [[[-3.0, 0.0, 1.0, -7.0]]], atol=1e-15)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_products_depend_on_distance(layout):
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 16))
    f, _ = serve.freqs(12)
    dot = lambda a, b: float((serve.rope(q, [a], f, layout, 1.0)[0] * serve.rope(k, [b], f, layout, 1.0)[0]).sum())  # noqa: E731
    assert abs(dot(7, 3) - dot(1000007, 1000003)) < 1e-9 and abs(dot(7, 3) - dot(7, 4)) > 1e-3


def test_norm_closed_forms():
    x = np.array([[[3.0, 4.0]]])
    assert np.allclose(serve.norm(x, None, 2 ** -0.5, 0.0), [[[0.6, 0.8]]])
    assert np.allclose(serve.norm(x, [0.0, 1.0], 1.0, 0.0), np.array([[[3.0, 8.0]]]) / math.sqrt(12.5))
    assert np.allclose(serve.norm(x, None, 1.0, 12.5), np.array([[[0.6, 0.8]]]))


def test_freqs():
    f, m = serve.freqs(8, 10000.0)
    assert np.allclose(f, [1, 0.1, 0.01, 0.001]) and m == 1
    assert np.allclose(serve.freqs(8, scaling="linear", factor=4)[0], f / 4)
    g, _ = serve.freqs(8, scaling="base", factor=4)
    assert g[0] == 1 and math.isclose(g[-1], f[-1] / 4)
    for scaling in ("by_pair", "by_turns"):
        g, m = serve.freqs(128, scaling=scaling, factor=8, original=4096, low=1, high=32)
        f, _ = serve.freqs(128)
        turns = f * 4096 / (2 * math.pi)
        assert np.allclose(g[turns > 40], f[turns > 40]) and np.allclose(g[turns < 0.8], f[turns < 0.8] / 8)
        assert (np.diff(g) < 0).all() and (g <= f).all() and (g >= f / 8 * (1 - 1e-15)).all()
        assert math.isclose(m, 1 + 0.1 * math.log(8) if scaling == "by_pair" else 1)


def test_chunk_rows():
    req, sees = serve.chunk_rows([1, 3, 3, 6], [5, 9, 2], 8)
    assert req.tolist() == [-1, 0, 0, 2, 2, 2, -1, -1]
    assert sees.tolist() == [0, 4, 5, 0, 1, 2, 0, 0]


def test_chunk_is_causal_attention():
    rng = np.random.default_rng(1)
    n, d = 7, 4
    q, k, v = rng.standard_normal((3, n, 1, d))
    kc, vc = (np.zeros((2, 1, 4, d)) for _ in range(2))
    table = np.array([[1, 0]], np.int32)
    for t in range(n):
        kc[table[0, t // 4], :, t % 4], vc[table[0, t // 4], :, t % 4] = k[t], v[t]
    o, lse, _ = serve.attend_chunk(q, kc, vc, table, [0, n], [n])
    x = q[:, 0] @ k[:, 0].T / math.sqrt(d)
    x[np.triu_indices(n, 1)] = -np.inf
    p = np.exp(x)
    assert np.allclose(o[:, 0], p @ v[:, 0] / p.sum(1, keepdims=True)) and np.allclose(lse[:, 0], np.log(p.sum(1)))
