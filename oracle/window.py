"""fp64 oracle of the windowed attention, its gradient, the quantised cache rows and the
attention over a paged cache. Plain NumPy, one head and one sequence at a time, from the
definitions; it shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def visible(pos, n: int, left: int, right: int, sinks: int) -> np.ndarray:
    """[rows, n] truth values: the query at pos[r] sees key j."""
    p, j = np.asarray(pos)[:, None], np.arange(n)[None, :]
    see = np.ones((len(pos), n), bool)
    if left >= 0:
        see &= (j >= p - left) | (j < sinks)
    if right >= 0:
        see &= j <= p + right
    return see


def attend(q, K, V, see, scale):
    """One head: (o [rows, d], lse [rows]); rows that see nothing give 0 and -inf."""
    s = np.where(see, scale * (q @ K.T), -np.inf)
    m = s.max(axis=1, initial=-np.inf)
    m0 = np.where(np.isfinite(m), m, 0.0)
    e = np.where(see, np.exp(s - m0[:, None]), 0.0)
    l = e.sum(axis=1)
    o = (e / np.where(l > 0, l, 1.0)[:, None]) @ V
    with np.errstate(divide="ignore"):
        return o, m0 + np.log(l)


def weights(q, K, see, scale):
    """The softmax weights p [rows, n]."""
    s = np.where(see, scale * (q @ K.T), -np.inf)
    m = s.max(axis=1, initial=-np.inf)
    e = np.where(see, np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, None]), 0.0)
    l = e.sum(axis=1, keepdims=True)
    return e / np.where(l > 0, l, 1.0)


def attend_backward(do, q, K, V, see, scale):
    """One head: (dq, dk, dv) of o = attend(...)."""
    p = weights(q, K, see, scale)
    dp = do @ V.T
    ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
    return scale * ds @ K, scale * ds.T @ q, p.T @ do


def window_attention(Q, K, V, left, right, sinks, scale):
    """Q [B, Hq, N, d], K, V [B, Hkv, N, d] -> (O, lse)."""
    B, Hq, N, d = Q.shape
    G = Hq // K.shape[1]
    see = visible(np.arange(N), N, left, right, sinks)
    O, lse = np.zeros(Q.shape), np.zeros((B, Hq, N))
    for b in range(B):
        for h in range(Hq):
            O[b, h], lse[b, h] = attend(Q[b, h], K[b, h // G], V[b, h // G], see, scale)
    return O, lse


def window_attention_backward(dO, Q, K, V, left, right, sinks, scale):
    """(dQ, dK, dV); the gradients of a shared key head are summed over its query heads."""
    B, Hq, N, d = Q.shape
    G = Hq // K.shape[1]
    see = visible(np.arange(N), N, left, right, sinks)
    dQ, dK, dV = np.zeros(Q.shape), np.zeros(K.shape), np.zeros(V.shape)
    for b in range(B):
        for h in range(Hq):
            dQ[b, h], dk, dv = attend_backward(dO[b, h], Q[b, h], K[b, h // G], V[b, h // G], see, scale)
            dK[b, h // G] += dk
            dV[b, h // G] += dv
    return dQ, dK, dV


def e4m3_round(y):
    """Nearest e4m3 value (ties to the even code), |y| <= 448: 3 mantissa bits, least step 2^-9."""
    y = np.asarray(y, np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    step = np.exp2(e - 3)
    return np.clip(np.round(y / step) * step, -448.0, 448.0)


def quantise_rows(x):
    """(code values, scale) of rows x [..., d]: the definition's fp32 scale and quotient."""
    x = np.asarray(x, np.float32)
    scale = np.maximum(np.abs(x).max(axis=-1) / np.float32(448), np.float32(2.0 ** -126)).astype(np.float32)
    return e4m3_round((x / scale[..., None]).astype(np.float32)), scale


def gather(pages, table_row, n: int):
    """Rows [0, n) [Hkv, n, d] of one sequence from pages [num_pages, Hkv, page, d]."""
    page = pages.shape[2]
    at = [int(table_row[i]) for i in range(-(-n // page))]
    if not at:
        return np.zeros((pages.shape[1], 0, pages.shape[3]))
    return np.concatenate([pages[i] for i in at], axis=1)[:, :n]


def paged_attention(Q, Kp, Vp, table, kv_lens, q_lens, left, right, sinks, scale):
    """Q [B, Hq, N, d] over pages of VALUES (codes times scales) -> (O, lse); rows
    t >= q_len are NaN."""
    B, Hq, N, d = Q.shape
    G = Hq // Kp.shape[1]
    O, lse = np.full(Q.shape, np.nan), np.full((B, Hq, N), np.nan)
    for b in range(B):
        n, m = int(kv_lens[b]), int(q_lens[b])
        K, V = gather(Kp, table[b], n), gather(Vp, table[b], n)
        see = visible(n - m + np.arange(m), n, left, right, sinks)
        for h in range(Hq):
            O[b, h, :m], lse[b, h, :m] = attend(Q[b, h, :m], K[h // G], V[h // G], see, scale)
    return O, lse
