"""Pins for the fp64 oracle of the 4-bit cache, the row weights and the eviction: hand examples and invariants."""
import numpy as np
import pytest

from oracle import cache_oracle as co
from oracle import decode_absorbed


def test_scale_bytes():
    assert co.SCALES[0] == 2.0 ** -21 and co.SCALES[168] == 1.0 and co.SCALES[255] == 1920.0 and co.LARGEST == 13440.0
    assert np.all(np.diff(co.SCALES) > 0)


def test_quantise_by_hand():
    x = np.zeros(16)
    x[:6] = [7.0, -7.0, 0.5, 1.5, -2.5, 3.49]  # scale 1: halves go to the even neighbour
    q, code = co.quantise(x)
    assert code.tolist() == [168] and q[:6].tolist() == [7, -7, 0, 2, -2, 3]
    x[0] = 7.01  # one past 7 * 1: the next scale, 9/8
    q, code = co.quantise(x)
    assert code.tolist() == [169] and q[0] == 6
    q, code = co.quantise(np.full(16, np.nan))
    assert code.tolist() == [0] and not q.any()
    q, code = co.quantise(np.r_[np.inf, -1e9, np.zeros(14)])
    assert code.tolist() == [255] and q[:2].tolist() == [7, -7]


def test_quantised_error_is_at_most_half_a_step():
    x = np.random.default_rng(0).standard_normal((50, 64)) * 10.0 ** np.random.default_rng(1).integers(-3, 3, (50, 1))
    q, code = co.quantise(x)
    step = np.repeat(co.SCALES[code], 16, axis=-1)
    assert np.all(np.abs(q) <= 7) and np.all(np.abs(x - q * step) <= step / 2 * (1 + 1e-12))
    assert np.array_equal(co.quantised(x), q * step)


def test_unpack_by_hand():
    row = np.zeros(32, np.uint8)
    row[:4] = [0x21, 0x43, 0x65, 0x87]   # elements 0, 2, 4, 6 in the low half word, 1, 3, 5, 7 in the high one
    row[8], row[9] = 168, 0
    assert co.unpack_latents(row, 16)[:8].tolist() == [1 - 8, 5 - 8, 2 - 8, 6 - 8, 3 - 8, 7 - 8, 4 - 8, 8 - 8]


def test_attend_agrees_with_the_decode_oracle_and_weights_sum_to_heads():
    rng = np.random.default_rng(2)
    H, d_c, d_r, T, q_len = 3, 16, 4, 9, 2
    qn, qr = rng.standard_normal((1, q_len, H, 6)), rng.standard_normal((1, q_len, H, d_r))
    W_UK, W_UV = rng.standard_normal((H, 6, d_c)), rng.standard_normal((H, 5, d_c))
    c, k = rng.standard_normal((T, d_c)), rng.standard_normal((T, d_r))
    from oracle import cache_rows, rope
    rows = cache_rows(c, k, np.arange(T))
    ref = decode_absorbed(qn, qr, W_UK, W_UV, [(c, k)], q_len, 10000.0)
    scale = 1 / np.sqrt(6 + d_r)
    q_hat = np.concatenate([np.einsum("hdc,ihd->ihc", W_UK, qn[0]),
                            rope(qr[0], (T - q_len + np.arange(q_len))[:, None])], -1)
    lse = np.zeros((q_len, H))
    for i in range(q_len):
        o, lse[i] = co.attend(q_hat[i], rows, T - q_len + 1 + i, d_c, scale)
        np.testing.assert_allclose(np.einsum("hvc,hc->hv", W_UV, o), ref[0, i], rtol=1e-12, atol=1e-12)
    w = co.row_weights(q_hat, lse, rows, T, scale)
    assert w.sum() == pytest.approx(q_len * H, rel=1e-12)
    one = co.row_weights(q_hat[1:], lse[1:], rows, T, scale)
    assert w[T - 1] == pytest.approx(one[T - 1], rel=1e-12)  # only the last query sees the last row


def test_kept_rows_by_hand():
    w = np.array([0.0, 5.0, 1.0, 3.0, 3.0, np.nan, 2.0, 9.0])
    assert co.kept_rows(w, 8, 8, 0, 0).tolist() == list(range(8))
    assert co.kept_rows(w, 8, 4, 1, 1).tolist() == [0, 1, 3, 7]     # 5 and the lower of the two 3s between the safe rows
    assert co.kept_rows(w, 8, 7, 0, 0).tolist() == [0, 1, 2, 3, 4, 6, 7]  # the NaN goes first
    assert co.kept_rows(w, 8, 3, 2, 1).tolist() == [0, 1, 7]
    assert co.kept_rows(w, 0, 3, 2, 1).tolist() == []
