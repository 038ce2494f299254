"""CPU fp64 oracle of the 4-bit cache, the accumulated attention weights and the eviction.

TEST INFRASTRUCTURE ONLY, like ``mla_oracle``: it shares no code with the CUDA
library.  Rows are given as the numbers they stand for ([T, d_c + d_r] fp64);
packed rows are bytes, read and written here from the layout's definition:

    bytes [0, d_c/2)               codes q + 8: element 8w + 2j of 32-bit word w in bits 4j..4j+3,
                                   element 8w + 2j + 1 in bits 16 + 4j..19 + 4j
    bytes [d_c/2, d_c/2 + d_c/16)  scales, e * 8 + m standing for 2^(e-21) (1 + m/8)
    from there, rounded up to 16   the RoPE key in the cache's type

``tests/test_cache_oracle.py`` pins each function against hand examples and invariants.
"""
from __future__ import annotations

import numpy as np

GROUP = 16
SCALES = np.array([2.0 ** (c // 8 - 21) * (1 + (c % 8) / 8) for c in range(256)])
LARGEST = 7 * SCALES[255]


def quantise(c: np.ndarray):
    """Codes q (-7..7) and scale bytes of latents c [..., d_c]; NaN is 0, what is too large is clipped."""
    x = np.clip(np.nan_to_num(np.asarray(c, np.float64), nan=0.0, posinf=np.inf, neginf=-np.inf), -LARGEST, LARGEST)
    x = x.reshape(x.shape[:-1] + (-1, GROUP))
    code = np.searchsorted(7 * SCALES, np.abs(x).max(-1))  # the first scale that is not below max / 7
    q = np.rint(x / SCALES[code][..., None])               # numpy rounds halves to even
    return q.reshape(c.shape).astype(np.int64), code.astype(np.uint8)


def quantised(c: np.ndarray) -> np.ndarray:
    """The latents a packed row of c stands for."""
    q, code = quantise(c)
    return q * np.repeat(SCALES[code], GROUP, axis=-1)


def unpack_latents(row: np.ndarray, d_c: int) -> np.ndarray:
    """Latents [..., d_c] of packed bytes [..., >= row bytes]."""
    row = np.asarray(row, np.uint8)
    out = np.empty(row.shape[:-1] + (d_c,))
    for c in range(d_c):
        bit = 32 * (c // 8) + 4 * ((c % 8) // 2) + 16 * (c % 2)
        n = (row[..., bit // 8] >> (bit % 8)) & 15
        out[..., c] = (n.astype(np.float64) - 8) * SCALES[row[..., d_c // 2 + c // GROUP]]
    return out


def attend(q_hat: np.ndarray, rows: np.ndarray, n_keys: int, d_c: int, scale: float):
    """o [H, d_c] and lse [H] of folded queries q_hat [H, d_c + d_r] over rows 0..n_keys-1."""
    s = scale * q_hat @ rows[:n_keys].T
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(-1, keepdims=True)
    return (p / total) @ rows[:n_keys, :d_c], (m + np.log(total))[:, 0]


def row_weights(q_hat: np.ndarray, lse: np.ndarray, rows: np.ndarray, seqlen: int, scale: float) -> np.ndarray:
    """Weight each of the rows 0..seqlen-1 receives from queries q_hat [q_len, H, d] with lse [q_len, H]."""
    q_len = q_hat.shape[0]
    w = np.zeros(seqlen)
    for i in range(q_len):
        n = seqlen - q_len + 1 + i
        for h in range(q_hat.shape[1]):
            if lse[i, h] > -np.inf:
                w[:n] += np.exp(scale * rows[:n] @ q_hat[i, h] - lse[i, h])
    return w


def kept_rows(weights: np.ndarray, seqlen: int, budget: int, n_sink: int, n_recent: int) -> np.ndarray:
    """Indexes of the rows that stay, ascending."""
    if seqlen <= budget:
        return np.arange(seqlen)
    middle = sorted(range(n_sink, seqlen - n_recent),
                    key=lambda t: (np.isnan(weights[t]), -weights[t] if not np.isnan(weights[t]) else 0.0, t))
    best = middle[:budget - n_sink - n_recent]
    return np.array(sorted(list(range(n_sink)) + best + list(range(seqlen - n_recent, seqlen))))
