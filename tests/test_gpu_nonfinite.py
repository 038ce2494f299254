"""NaN and infinities in what an attention sees: a NaN score makes its query's output and log-sum-exp NaN, however the sequence was
cut and whichever piece holds it, and nothing else changes by a bit.  (A score's NaN does not show in the running maximum, and a cut
sequence is merged from pieces by their log-sum-exps, so it could be taken for a piece that holds nothing.)"""
import numpy as np
import pytest
import torch

from mla_testutil import as_f64
from oracle import cache_oracle as co
from test_gpu_packed import TINY, V3, check_attention, decode_inputs, dims_of, i32, make_cache, rand, stored_rows

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def poison(cache, g, row, value, element=0):
    """One element of row `row`'s RoPE key of sequence 0, in a copy of the cache."""
    H, d_c, d_r, _, _, dt = g
    out = cache.clone()
    if cache.dtype == torch.uint8:
        at = (d_c // 2 + d_c // 16 + 15) // 16 * 16
        out[0, row, at:at + d_r * dt.itemsize].view(dt)[element] = value
    else:
        out[0, row, d_c + element] = value
    return out


def case(lib, g, T, q_len, packed):
    H, d_c, d_r, _, _, dt = g
    dims = dims_of(lib, g)
    cache = make_cache(lib, dims, g, T)[0] if packed else rand(9, len(T), max(T), d_c + d_r, dtype=dt)
    q = rand(3, len(T), q_len, H, d_c + d_r, dtype=dt, std=0.25)
    call = lib.attend_packed if packed else lib.attend_latent_lse

    def attend(q, cache, **opts):
        lse = torch.zeros(len(T), q_len, H, device="cuda")
        return call(dims, q, cache, i32(*T), lse=lse, opts=lib.opts(**opts)), lse
    return cache, q, attend


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


# whole sequences, cut ones (pieces merged by one warp each and by two), several queries
CUTS = [((2000,), 1, 1), ((2000,), 1, 16), ((4096, 700), 1, 0), ((900, 77), 2, 16), ((640,) * 7, 1, 8)]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,q_len,pairs", CUTS)
def test_nan_in_a_query_head(lib, T, q_len, pairs, packed):
    cache, q, attend = case(lib, V3, T, q_len, packed)
    clean = attend(q, cache, num_pairs=pairs)
    for value in (NAN, INF):
        bad = q.clone()
        bad[0, -1, 7, 3] = value            # (an infinity times latents of both signs: scores of both infinities)
        o, lse = attend(bad, cache, num_pairs=pairs)
        assert lib.device_status() == 0 and lib.last_path() == "sm100"
        assert o[0, -1, 7].isnan().all() and lse[0, -1, 7].isnan()
        o[0, -1, 7], lse[0, -1, 7] = clean[0][0, -1, 7], clean[1][0, -1, 7]
        assert same((o, lse), clean)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,q_len,pairs", CUTS)
def test_nan_in_a_key(lib, T, q_len, pairs, packed):
    cache, q, attend = case(lib, V3, T, q_len, packed)
    clean = attend(q, cache, num_pairs=pairs)
    for row in (0, 300, T[0] // 2, T[0] - q_len):   # in the first, the middle and the last piece, seen by every query
        o, lse = attend(q, poison(cache, V3, row, NAN), num_pairs=pairs)
        assert lib.device_status() == 0
        assert o[0].isnan().all() and lse[0].isnan().all(), f"row {row}"
        assert same((o[1:], lse[1:]), (clean[0][1:], clean[1][1:]))


@pytest.mark.parametrize("T", [(2000,), (2000, 300), (700,) * 12])   # merged by the projection of few rows, by the combine
def test_nan_in_a_key_through_the_decode(lib, T):
    dims = dims_of(lib, V3)
    cache = rand(9, len(T), max(T), 576, dtype=torch.bfloat16)
    ins = decode_inputs(V3, len(T), 1)
    clean = lib.decode(dims, *ins, cache, i32(*T))
    assert clean.isfinite().all()
    for row in (0, 300, T[0] - 1):
        out = lib.decode(dims, *ins, poison(cache, V3, row, NAN), i32(*T))
        assert out[0].isnan().all() and torch.equal(out[1:], clean[1:])
    packed = make_cache(lib, dims, V3, T)[0]
    clean = lib.decode_packed(dims, *ins, packed, i32(*T))
    for row in (0, 300, T[0] - 1):
        out = lib.decode_packed(dims, *ins, poison(packed, V3, row, NAN), i32(*T))
        assert out[0].isnan().all() and torch.equal(out[1:], clean[1:])
    assert lib.device_status() == 0


# ------------------------------------------------------------------ the CUDA-core form, and scores of -infinity in both

GENERIC = [(TINY, (40, 9), 2), (TINY, (3,), 1), (V3, (300, 7), 2)]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("g,T,q_len", GENERIC)
def test_nan_on_cuda_cores(lib, g, T, q_len, packed):
    cache, q, attend = case(lib, g, T, q_len, packed)
    clean = attend(q, cache, path=2)
    for row in (0, 1, T[0] - q_len):                 # (a warp takes every eighth row: alone in it, first, last)
        o, lse = attend(q, poison(cache, g, row, NAN), path=2)
        assert lib.last_path() == "generic" and lib.device_status() == 0
        assert o[0].isnan().all() and lse[0].isnan().all(), f"row {row}"
        assert same((o[1:], lse[1:]), (clean[0][1:], clean[1][1:]))
        if not packed:                               # the attention without log-sum-exps has a kernel of its own
            dims, opts = dims_of(lib, g), lib.opts(path=2)
            o = lib.attend_latent(dims, q, poison(cache, g, row, NAN), i32(*T), opts=opts)
            assert o[0].isnan().all() and torch.equal(o[1:], lib.attend_latent(dims, q, cache, i32(*T), opts=opts)[1:])
            o = lib.attend_latent(dims, q, poison(cache, g, row, -INF), i32(*T), opts=opts)
            assert torch.equal(o[1:], lib.attend_latent(dims, q, cache, i32(*T), opts=opts)[1:])
    bad = q.clone()
    bad[0, -1, 2, 1] = NAN
    o, lse = attend(bad, cache, path=2)
    assert o[0, -1, 2].isnan().all() and lse[0, -1, 2].isnan()
    o[0, -1, 2], lse[0, -1, 2] = clean[0][0, -1, 2], clean[1][0, -1, 2]
    assert same((o, lse), clean)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("g,T,path", [(V3, (900, 70), 0), (V3, (300, 70), 2), (TINY, (40, 9), 2)])
def test_scores_of_minus_infinity(lib, g, T, path, packed):
    # such rows have no weight, whether they come first, alone or last; only such rows: zeros and a log-sum-exp of -infinity
    H, d_c, d_r, d_n, _, dt = g
    cache, q, attend = case(lib, g, T, 1, packed)
    q[..., d_c] = q[..., d_c].abs() + 0.01
    dead = [0, 1, 8, 16, T[0] - 1]
    low = cache
    for row in dead:
        low = poison(low, g, row, -INF)
    o, lse = attend(q, low, path=path)
    dims = dims_of(lib, g)
    rows = stored_rows(lib, dims, cache, T) if packed else [as_f64(cache[b, :t]) for b, t in enumerate(T)]
    rows[0] = np.delete(rows[0], dead, 0)
    left = tuple(len(r) for r in rows)
    if packed or dt == torch.float32:
        check_attention(o, lse, q, rows, left, 1, g, (d_n + d_r) ** -0.5)
    else:                                            # (the full-width form holds the weights in bf16)
        want = [co.attend(as_f64(q)[b, 0], rows[b], t, d_c, (d_n + d_r) ** -0.5) for b, t in enumerate(left)]
        for b, (wo, wl) in enumerate(want):
            assert np.linalg.norm(as_f64(o)[b, 0] - wo) <= 5e-3 * np.linalg.norm(wo)
            assert np.all(np.abs(as_f64(lse)[b, 0] - wl) <= 1e-4 * (1 + np.abs(wl)))
    all_low = cache
    for row in range(9):
        all_low = poison(all_low, g, row, -INF)
    few = i32(*([9] + list(T[1:])))
    call = lib.attend_packed if packed else lib.attend_latent_lse
    z = torch.zeros_like(lse)
    o = call(dims, q, all_low, few, lse=z, opts=lib.opts(path=path))
    if not packed:
        for c, n in ((low, i32(*T)), (all_low, few)):
            plain = lib.attend_latent(dims, q, c, n, opts=lib.opts(path=path))
            assert plain.isfinite().all() and (n is not few or not plain[0].any())
    assert not o[0].any() and torch.all(z[0] == -INF) and o[1:].isfinite().all() and z[1:].isfinite().all()
    assert lib.device_status() == 0


# ------------------------------------------------------------------ new tokens past a query

@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,q_len", [((700, 77), 2), ((64, 65, 63, 130), 3), ((16, 300), 16)])
def test_nan_in_a_token_past_the_query(lib, T, q_len, packed):
    # only the last query sees the last token: the others' outputs keep their bits
    cache, q, attend = case(lib, V3, T, q_len, packed)
    for path in (0, 2):
        clean = attend(q, cache, path=path)
        for value in (NAN, INF):
            bad = poison(cache, V3, T[0] - 1, value)
            if not packed:
                bad[0, T[0] - 1, 100:300] = value       # its latents too, as long as they can be NaN
            o, lse = attend(q, bad, path=path)
            assert o[0, -1].isnan().any() and lib.device_status() == 0
            assert same((o[0, :-1], lse[0, :-1], o[1:], lse[1:]), (clean[0][0, :-1], clean[1][0, :-1], clean[0][1:], clean[1][1:]))


# ------------------------------------------------------------------ accumulated weights

@pytest.mark.parametrize("path", [0, 2])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,q_len", [((300, 40), 1), ((600,), 5), ((2500, 2500), 2)])
def test_weights_of_queries_that_count_nothing(lib, T, q_len, packed, path):
    # a log-sum-exp of -infinity: the query's scores do not matter, not even NaN or infinite ones
    dims = dims_of(lib, V3)
    cache, q, _ = case(lib, V3, T, q_len, packed)
    lse = rand(8, len(T), q_len, 128) + 5
    lse[0, 0, ::3] = -INF
    lse[-1, -1, 64:] = -INF
    want = lib.accumulate_weights(dims, q, lse, cache, i32(*T), torch.zeros(len(T), max(T), device="cuda"), opts=lib.opts(path=path))
    bad = torch.where((lse == -INF)[..., None], torch.tensor(NAN, device="cuda", dtype=q.dtype), q)
    bad[0, 0, 3, 9], bad[0, 0, 6] = INF, -INF        # (heads 3 and 6 count nothing)
    got = lib.accumulate_weights(dims, bad, lse, cache, i32(*T), torch.zeros(len(T), max(T), device="cuda"), opts=lib.opts(path=path))
    assert lib.device_status() == 0
    assert want.isfinite().all() and torch.equal(got, want)
    # a NaN among the scores of a query that counts stays in the sums of the rows it sees
    bad = q.clone()
    bad[0, 0, 1, 9] = NAN
    got = lib.accumulate_weights(dims, bad, lse, cache, i32(*T), torch.zeros(len(T), max(T), device="cuda"), opts=lib.opts(path=path))
    n = T[0] - q_len + 1
    assert got[0, :n].isnan().all() and torch.equal(got[0, n:], want[0, n:]) and torch.equal(got[1:], want[1:])
