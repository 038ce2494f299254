"""Calls that the documentation allows at the edges of what the checks see (CPU), and refusals of what they must not let through."""
import ctypes
import itertools

import pytest
import torch

from latent_compressed_attention_absorbed_b200 import binding as bd

ARG, SHAPE, CUDA, WORKSPACE = -1, -2, -4, -7
TINY = bd.Dims(4, 32, 8, 16, 16, bd.MLA_DTYPE_F32, 10000.0, 0.0)   # rows of 160 bytes, packed 64


@pytest.fixture(scope="module")
def L():
    from latent_compressed_attention_absorbed_b200 import build
    return bd.Library(build.build()).lib


@pytest.fixture(scope="module")
def a():
    buf = ctypes.create_string_buffer(1 << 16)
    yield (ctypes.addressof(buf) + 255) & ~255


def P(x):
    return None if x is None else ctypes.c_void_p(x)


# ------------------------------------------------------------------ views that lie between each other

def evict(L, a, src, dst, w=(40000, 32), wo=(50000, 32), B=2, fmt=0, budget=4):
    """The return code of an eviction without workspace, which is asked for last: WORKSPACE says that every view was taken.
    src, dst: (offset, T_max, stride_b, stride_t); w, wo: (offset in bytes, stride)."""
    def cache(v):
        return bd.Cache(a + v[0], B, v[1], v[2], v[3])
    return L.mla_evict(ctypes.byref(TINY), ctypes.byref(cache(src)), fmt, P(a + w[0]), w[1], P(a), B, budget, 1, 1,
                       ctypes.byref(cache(dst)), P(a + wo[0]), wo[1], P(a), None, None, 0, None)


def touched(offset, B, stride_b, rows, stride_t, row):
    return {offset + b * stride_b + t * stride_t + i for b in range(B) for t in range(rows) for i in range(row)}


def test_views_between_each_other_are_taken(L, a):
    # halves of every sequence of one array; rows beside each other; both, one sequence only
    assert evict(L, a, (0, 8, 16 * 40, 40), (8 * 160, 8, 16 * 40, 40)) == WORKSPACE
    assert evict(L, a, (8 * 160, 8, 16 * 40, 40), (0, 8, 16 * 40, 40)) == WORKSPACE
    assert evict(L, a, (0, 8, 8 * 80, 80), (160, 8, 8 * 80, 80)) == WORKSPACE
    assert evict(L, a, (160, 8, 8 * 80, 80), (0, 8, 8 * 80, 80), B=1) == WORKSPACE
    # sharing a byte of one row, in the same places and a period on
    assert evict(L, a, (0, 8, 16 * 40, 40), (7 * 160, 8, 16 * 40, 40)) == ARG
    assert evict(L, a, (0, 8, 8 * 80, 80), (144, 8, 8 * 80, 80)) == ARG
    assert evict(L, a, (0, 8, 16 * 40, 40), (16 * 160 + 160, 8, 16 * 40, 40)) == ARG
    assert evict(L, a, (0, 8, 8 * 80, 80), (3 * 320, 8, 8 * 80, 80)) == ARG
    # running weights: rows of one array in turn
    src, dst = (0, 8, 8 * 40, 40), (4096, 8, 8 * 40, 40)
    assert evict(L, a, src, dst, w=(40000, 16), wo=(40032, 16)) == WORKSPACE
    assert evict(L, a, src, dst, w=(40000, 16), wo=(40028, 16)) == ARG
    assert evict(L, a, src, dst, w=(40000, 16), wo=(40032, 17)) == ARG   # not in step

    def weights(prev, w, stride):
        full = bd.Cache(a, 2, 4, 160, 40)
        return L.mla_accumulate_weights(ctypes.byref(TINY), P(a), P(a), ctypes.byref(full), 0, P(a), 2, 1, 1.0, P(a + prev), P(a + w),
                                        stride, None, None)
    taken = CUDA if not torch.cuda.is_available() else 0
    if taken == CUDA:                        # (with a device the calls would run on these host addresses)
        assert weights(40000, 40016, 8) == taken and weights(40016, 40000, 8) == taken
    assert weights(40000, 40012, 8) == ARG and weights(40000, 40004, 8) == ARG and weights(40000, 40048 - 4, 8) == ARG


def test_no_view_that_shares_a_byte_is_taken(L, a):
    # every pair of small views of one array, against the bytes they touch; a pair that is refused shares one, where the strides agree
    for B, (sb, st), T in itertools.product((1, 2, 3), ((4, 40), (8, 40), (8, 80), (9, 80)), (2, 4)):
        stride_b, stride_t = sb * 2 * st, st
        if stride_b % 4 or B > 1 and stride_b < T * stride_t:
            continue
        x = (6400, T, stride_b, stride_t)
        mine = touched(6400, B, 4 * stride_b, T, 4 * stride_t, 160)
        for off in range(0, 12800, 80):
            y = (off, T, stride_b, stride_t)
            rc = evict(L, a, x, y, B=B, budget=T)
            if off == 6400:
                assert rc == WORKSPACE
                continue
            shares = bool(mine & touched(off, B, 4 * stride_b, T, 4 * stride_t, 160))
            assert rc in (ARG, WORKSPACE)
            assert not (shares and rc == WORKSPACE), (B, x, y)
            if stride_b % stride_t == 0 and off % 160 == 0 and rc == ARG and B == 1:
                assert shares, (B, x, y)


# ------------------------------------------------------------------ options that would not fit the planners' 32 bits

def test_charges_past_the_planners_range_are_refused(L, a):
    d, B, T = ctypes.byref(TINY), 2, 4
    full, packed = bd.Cache(a, B, T, 4 * 40, 40), bd.Cache(a, B, T, 4 * 64, 64)
    p, big = P(a), 1 << 24

    def calls(**o):
        opts = ctypes.byref(bd.Library.opts(path=2, **o))   # (the CUDA-core form, which runs anywhere else)
        return [L.mla_decode_ex(d, p, p, p, p, ctypes.byref(full), p, B, 1, p, None, 0, opts, None),
                L.mla_attend_latent(d, p, ctypes.byref(full), p, B, 1, p, None, 0, opts, None),
                L.mla_attend_latent_lse(d, p, ctypes.byref(full), p, B, 1, p, p, None, 0, opts, None),
                L.mla_attend_packed(d, p, ctypes.byref(packed), p, B, 1, p, None, None, 0, opts, None),
                L.mla_decode_packed(d, p, p, p, p, ctypes.byref(packed), p, None, B, 1, p, None, None, None, 0, opts, None)]
    for charge in (2 ** 31 - 1, 2 ** 30, big, big // 2):
        assert calls(overhead_tiles=charge) == [ARG] * 5
        assert b"overhead_tiles" in L.mla_last_error()
    if not torch.cuda.is_available():        # (with a device the other three would run on these host addresses)
        for o in (dict(overhead_tiles=big // 2 - 1), dict(overhead_tiles=-5), dict(min_tiles=2 ** 31 - 1)):
            assert calls(**o) == [WORKSPACE, CUDA, CUDA, CUDA, WORKSPACE]
