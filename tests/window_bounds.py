"""How far the kernels' results may be from the fp64 oracle's, element by element, from the
roundings that the kernels make (u = 2^-8 is half a bf16 step, relative):

  s       fp32 sum of d exact products: |s - s*| <= eps_s = (d + 8) 2^-24 scale max sum|q k|,
          and the base-2 exponential and logarithm add at most 2^-20 (relative / absolute);
  p       relative error at most e = 2 eps_s + 2^-19 (its own score and the row's sum);
  O       p rounded to bf16, O rounded to bf16, sums of n fp32 terms (any split of the keys):
          (u + e + n 2^-24) sum p|v| + u |O|;
  lse     2 eps_s + 2^-19 + 2^-22 |lse|;
  dV      p and dV rounded: (u + e + n 2^-24) sum p|do| + u |dV|;
  delta   from the O that the forward call rounded: sum |do| tol(O);
  ds      p (tol(delta) + e (|dp| + |delta|) + d 2^-24 (sum |do v|)) + u |ds|;
  dQ, dK  sums of tol(ds) |k| (|q|), plus n 2^-24 sum |ds k|, plus u |dQ| (|dK|).

Weights and gradients below 2^-126 are lost in fp32 (underflow); times a factor of at most 2^10
and summed over at most 2^14 rows that is under 2^-102, so every bound has 2^-100 added.

Every bound gets 10% on top for products of two errors. With independent roundings the norms
are closer: each of the two (O, dV) or three (dQ, dK, through delta) roundings has an RMS of
at most u / sqrt(3), so a relative L2 error of u covers them."""
from __future__ import annotations

import numpy as np

from oracle import window as W

U = 2.0 ** -8
SLACK = 1.1
LOST = 2.0 ** -100


def _score_error(q, K, scale):
    top = scale * float((np.abs(q) @ np.abs(K).T).max(initial=0.0))
    return (q.shape[-1] + 8) * 2.0 ** -24 * top


def forward(q, K, V, see, scale):
    """(o, lse, tol_o, tol_lse) of one head."""
    o, lse = W.attend(q, K, V, see, scale)
    eps = _score_error(q, K, scale)
    p = W.weights(q, K, see, scale)
    e = 2 * eps + 2.0 ** -19
    tol = (U + e + K.shape[0] * 2.0 ** -24) * (p @ np.abs(V)) + U * np.abs(o)
    with np.errstate(invalid="ignore"):
        tol_lse = np.where(np.isfinite(lse), 2 * eps + 2.0 ** -19 + 2.0 ** -22 * np.abs(lse), 0.0)
    return o, lse, SLACK * tol, SLACK * tol_lse


def backward(do, q, K, V, see, scale):
    """(dq, dk, dv, tol_dq, tol_dk, tol_dv) of one head; dk, dv tolerances without the final rounding."""
    o, _, tol_o, _ = forward(q, K, V, see, scale)
    dq, dk, dv = W.attend_backward(do, q, K, V, see, scale)
    p = W.weights(q, K, see, scale)
    e = 2 * _score_error(q, K, scale) + 2.0 ** -19
    n, d = K.shape[0], q.shape[1]
    dp = do @ V.T
    delta = (p * dp).sum(axis=1, keepdims=True)
    ds = p * (dp - delta)
    t_delta = (np.abs(do) * tol_o).sum(axis=1, keepdims=True)
    t_ds = p * (t_delta + e * (np.abs(dp) + np.abs(delta)) + d * 2.0 ** -24 * (np.abs(do) @ np.abs(V).T)) + U * np.abs(ds)
    f = 2.0 ** -24
    tq = scale * (t_ds + n * f * np.abs(ds)) @ np.abs(K) + U * np.abs(dq)
    tk = scale * (t_ds + n * f * np.abs(ds)).T @ np.abs(q)
    tv = ((U + e + n * f) * p).T @ np.abs(do)
    return dq, dk, dv, SLACK * tq, SLACK * tk, SLACK * tv


def check(got, want, tol, what):
    """Element by element; infinities have to be equal."""
    got = np.asarray(got, np.float64)
    fin = np.isfinite(want)
    assert np.array_equal(fin, np.isfinite(got)), f"{what}: not finite in other places"
    assert np.array_equal(got[~fin], want[~fin]), f"{what}: infinities differ"
    over = np.abs(got[fin] - want[fin]) - tol[fin] - LOST
    assert not over.size or over.max() <= 0, f"{what}: {over.max():.3e} over its bound, {(over > 0).sum()} of {over.size}"


def check_norm(got, want, what, most=U):
    off = float(np.linalg.norm(np.asarray(got, np.float64) - want)) / max(float(np.linalg.norm(want)), 1e-300)
    assert off <= most, f"{what}: relative L2 error {off:.3e} over {most:.3e}"
