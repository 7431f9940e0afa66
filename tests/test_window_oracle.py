"""Pins of the windowed-attention oracle: scalar loops, central differences, the 8-bit
format's own value table."""
import math

import numpy as np
import pytest

from oracle import window as W


@pytest.mark.parametrize("left,right,sinks", [(-1, -1, 0), (2, 0, 1), (0, 0, 0), (3, 2, 2), (-1, 0, 0), (0, 4, 9)])
def test_attend_against_scalar_loops(left, right, sinks):
    rng = np.random.default_rng(1)
    n, d, scale = 9, 3, 0.7
    q, K, V = rng.normal(size=(n, d)), rng.normal(size=(n, d)), rng.normal(size=(n, d))
    o, lse = W.attend(q, K, V, W.visible(np.arange(n), n, left, right, sinks), scale)
    for p in range(n):
        num, den = [0.0] * d, 0.0
        for j in range(n):
            if right >= 0 and j > p + right:
                continue
            if left >= 0 and j < p - left and j >= sinks:
                continue
            w = math.exp(scale * sum(q[p, c] * K[j, c] for c in range(d)))
            den += w
            for c in range(d):
                num[c] += w * V[j, c]
        assert np.allclose(o[p], [x / den for x in num], rtol=1e-12) and abs(lse[p] - math.log(den)) < 1e-12


def test_row_that_sees_nothing():
    o, lse = W.attend(np.ones((2, 4)), np.ones((3, 4)), np.ones((3, 4)), np.array([[0, 0, 0], [1, 0, 1]], bool), 1.0)
    assert np.all(o[0] == 0) and lse[0] == -np.inf and np.allclose(o[1], 1)


def test_gradients_against_central_differences():
    rng = np.random.default_rng(2)
    B, Hq, Hkv, N, d = 1, 4, 2, 6, 3
    args = dict(left=2, right=1, sinks=1, scale=0.9)
    Q, K, V = (rng.normal(size=(B, h, N, d)) for h in (Hq, Hkv, Hkv))
    dO = rng.normal(size=Q.shape)
    grads = W.window_attention_backward(dO, Q, K, V, **args)
    loss = lambda: float((W.window_attention(Q, K, V, **args)[0] * dO).sum())  # noqa: E731
    for x, g in zip((Q, K, V), grads):
        for at in rng.choice(x.size, 12, replace=False):
            i, eps = np.unravel_index(at, x.shape), 1e-5
            x[i] += eps
            up = loss()
            x[i] -= 2 * eps
            down = loss()
            x[i] += eps
            assert abs((up - down) / (2 * eps) - g[i]) < 1e-8


def test_e4m3_round_against_the_value_table():
    torch = pytest.importorskip("torch")
    table = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    values = np.unique(table[np.isfinite(table)])
    assert values.max() == 448
    y = np.concatenate([values, (values[1:] + values[:-1]) / 2, np.random.default_rng(3).uniform(-448, 448, 2000),
                        np.random.default_rng(4).normal(size=500) * 0.02])
    got = W.e4m3_round(y)
    best = np.abs(values[None, :] - y[:, None]).min(axis=1)
    assert np.isin(got, values).all() and np.array_equal(np.abs(got - y), best)
    # on a tie, the code with the even mantissa: the neighbours' codes differ by one
    code = {v: i for i, v in enumerate(values[values >= 0])}
    for v, m in zip(values[:-1], (values[1:] + values[:-1]) / 2):
        if v >= 0:
            assert code[float(W.e4m3_round(m))] % 2 == 0


def test_quantised_rows_hold_the_value_to_half_a_step():
    x = np.random.default_rng(5).normal(size=(50, 64)).astype(np.float32)
    x[7] = 0
    code, scale = W.quantise_rows(x)
    err = np.abs(code * scale[:, None].astype(np.float64) - x)
    top = np.abs(x).max(axis=1, keepdims=True)
    assert np.all(err <= np.maximum(np.abs(x) * 2.0 ** -4, top / 448 * 2.0 ** -10) * (1 + 1e-6))
    assert np.all(code[7] == 0)
