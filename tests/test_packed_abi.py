"""Refusals of the 4-bit cache, row-weight and eviction entry points: bad arguments are turned down before any launch, on the CPU."""
import ctypes

import pytest
import torch

from latent_compressed_attention_absorbed_b200 import binding as bd

ARG, SHAPE, ALIGN, WORKSPACE = -1, -2, -3, -7


@pytest.fixture(scope="module")
def L():
    from latent_compressed_attention_absorbed_b200 import build
    return bd.Library(build.build()).lib


@pytest.fixture(scope="module")
def mem():
    buf = ctypes.create_string_buffer(1 << 16)
    a = (ctypes.addressof(buf) + 255) & ~255
    return buf, a


V3 = bd.Dims(128, 512, 64, 128, 128, bd.MLA_DTYPE_BF16, 10000.0, 0.0)
TINY = bd.Dims(4, 32, 8, 16, 16, bd.MLA_DTYPE_F32, 10000.0, 0.0)
ODD = bd.Dims(4, 40, 8, 16, 16, bd.MLA_DTYPE_F32, 10000.0, 0.0)


def test_row_bytes(L):
    assert L.mla_packed_row_bytes(ctypes.byref(V3)) == 416
    assert L.mla_packed_row_bytes(ctypes.byref(TINY)) == 64  # 16 + 2, rounded up to 32, and 8 fp32
    assert L.mla_packed_row_bytes(ctypes.byref(ODD)) == 0    # d_c is no multiple of 16
    assert L.mla_packed_row_bytes(None) == 0
    assert L.mla_packed_workspace_bytes(ctypes.byref(ODD), 1, 1) == 0
    assert L.mla_packed_workspace_bytes(ctypes.byref(TINY), 1, 0) == 0
    assert L.mla_packed_workspace_bytes(ctypes.byref(TINY), 2, 3) > 2 * 3 * 4 * (40 + 32) * 4
    assert L.mla_evict_workspace_bytes(ctypes.byref(TINY), 0, 2, 0) == 0
    assert L.mla_evict_workspace_bytes(ctypes.byref(TINY), 7, 2, 5) == 0
    assert L.mla_evict_workspace_bytes(ctypes.byref(ODD), 1, 2, 5) == 0
    assert L.mla_evict_workspace_bytes(ctypes.byref(TINY), 1, 2, 5) >= 2 * 5 * 4


def test_append_and_load_refusals(L, mem):
    _, a = mem
    p, bad = ctypes.c_void_p(a), ctypes.c_void_p(a + 2)
    d = ctypes.byref(TINY)
    ok = bd.Cache(a, 2, 4, 4 * 64, 64)

    def append(dims=d, c=p, k=p, pos=p, rows=None, B=2, n=1, cache=ok):
        return L.mla_append_packed(dims, c, k, pos, rows, B, n, ctypes.byref(cache) if cache else None, None)

    assert append(dims=None) == ARG
    assert append(dims=ctypes.byref(ODD)) == SHAPE
    assert append(B=-1) == ARG and append(n=-1) == ARG
    assert append(B=0, c=None) == 0 and append(n=0, c=None) == 0
    assert append(c=None) == ARG and append(k=None) == ARG and append(pos=None) == ARG and append(cache=None) == ARG
    assert append(c=bad) == ALIGN and append(rows=bad) == ALIGN and append(pos=bad) == ALIGN
    assert append(cache=bd.Cache(a, 1, 4, 256, 64)) == SHAPE           # too few sequences
    assert append(cache=bd.Cache(a, 2, 4, 256, 48)) == SHAPE           # rows narrower than a packed row
    assert append(cache=bd.Cache(a, 2, 4, 128, 64)) == SHAPE           # sequences overlap
    assert append(cache=bd.Cache(a, 2, 4, 4 * 72, 72)) == ALIGN
    assert append(cache=bd.Cache(a + 8, 2, 4, 256, 64)) == ALIGN
    assert append(cache=bd.Cache(a, 2, 0, 256, 64)) == SHAPE
    full = bd.Cache(a, 2, 4, 160, 40)
    assert L.mla_append_rows(d, p, p, None, p, 2, 1, ctypes.byref(full), None) == ARG
    assert L.mla_append_rows(d, p, p, p, bad, 2, 1, ctypes.byref(full), None) == ALIGN
    assert L.mla_load_packed(d, ctypes.byref(ok), None, 2, 1, p, None) == ARG
    assert L.mla_load_packed(d, ctypes.byref(ok), p, 2, 1, bad, None) == ALIGN
    assert L.mla_load_packed(ctypes.byref(ODD), ctypes.byref(ok), p, 2, 1, p, None) == SHAPE
    assert L.mla_load_packed(d, ctypes.byref(ok), p, 2, 0, None, None) == 0


def test_attend_and_decode_refusals(L, mem):
    _, a = mem
    p, bad = ctypes.c_void_p(a), ctypes.c_void_p(a + 2)
    d = ctypes.byref(TINY)
    ok = bd.Cache(a, 2, 4, 4 * 64, 64)

    def attend(dims=d, q=p, cache=ok, s=p, B=2, q_len=1, o=p, lse=None, opts=None):
        return L.mla_attend_packed(dims, q, ctypes.byref(cache), s, B, q_len, o, lse, p, 1 << 15, opts, None)

    assert attend(dims=None) == ARG and attend(dims=ctypes.byref(ODD)) == SHAPE
    assert attend(q_len=0) == ARG and attend(q_len=17) == ARG and attend(B=-1) == ARG and attend(B=0, q=None) == 0
    assert attend(q=None) == ARG and attend(s=None) == ARG and attend(o=None) == ARG
    assert attend(lse=bad) == ALIGN and attend(q=bad) == ALIGN
    assert attend(cache=bd.Cache(a, 2, 4, 256, 48)) == SHAPE
    o = bd.Library.opts(path=3)
    assert attend(opts=ctypes.byref(o)) == ARG

    def decode(n_seen=None, ws=p, nbytes=1 << 15, q_hat=None, lse=None, out=p):
        return L.mla_decode_packed(d, p, p, p, p, ctypes.byref(ok), p, n_seen, 2, 1, out, q_hat, lse, ws, nbytes, None, None)

    assert decode(ws=None) == WORKSPACE and decode(nbytes=64) == WORKSPACE
    assert decode(n_seen=bad) == ALIGN and decode(q_hat=bad) == ALIGN and decode(lse=bad) == ALIGN and decode(out=None) == ARG
    full = bd.Cache(a, 2, 4, 160, 40)
    assert L.mla_attend_latent_lse(d, p, ctypes.byref(full), p, 2, 1, p, None, p, 1 << 15, None, None) == ARG
    assert L.mla_attend_latent_lse(d, p, ctypes.byref(full), p, 2, 1, p, bad, p, 1 << 15, None, None) == ALIGN


def test_weights_refusals(L, mem):
    _, a = mem
    p, bad = ctypes.c_void_p(a), ctypes.c_void_p(a + 2)
    d = ctypes.byref(TINY)
    full = bd.Cache(a, 2, 4, 160, 40)

    def weights(q=p, lse=p, cache=full, fmt=0, s=p, B=2, q_len=1, decay=1.0, prev=None, w=p, stride=4):
        return L.mla_accumulate_weights(d, q, lse, ctypes.byref(cache), fmt, s, B, q_len, decay, prev, w, stride, None, None)

    assert weights(fmt=2) == ARG and weights(fmt=-1) == ARG
    assert weights(fmt=1) == SHAPE                                   # full-width strides are too narrow in bytes
    assert weights(stride=3) == SHAPE
    assert weights(decay=float("nan")) == ARG and weights(decay=float("inf")) == ARG
    assert weights(q=None) == ARG and weights(lse=None) == ARG and weights(w=None) == ARG and weights(s=None) == ARG
    assert weights(w=bad) == ALIGN and weights(prev=bad) == ALIGN and weights(lse=bad) == ALIGN
    assert weights(B=0, q=None) == 0
    assert weights(prev=ctypes.c_void_p(a + 4)) == ARG               # overlaps weights, one entry on


def test_evict_refusals(L, mem):
    _, a = mem
    p, bad = ctypes.c_void_p(a), ctypes.c_void_p(a + 2)
    d = ctypes.byref(TINY)
    src = bd.Cache(a, 2, 8, 8 * 40, 40)                              # 2 x 8 rows of 160 bytes
    dst = bd.Cache(a + 4096, 2, 4, 4 * 40, 40)
    w, wo = ctypes.c_void_p(a + 8192), ctypes.c_void_p(a + 12288)

    def evict(cache=src, fmt=0, w=w, sw=8, s=p, B=2, budget=4, sink=1, recent=1, to=dst, wo=wo, so=4, n=p, kept=None, ws=p,
              nbytes=1 << 15):
        return L.mla_evict(d, ctypes.byref(cache), fmt, w, sw, s, B, budget, sink, recent, ctypes.byref(to), wo, so, n, kept,
                           ws, nbytes, None)

    assert evict(budget=0) == ARG and evict(sink=-1) == ARG and evict(recent=-1) == ARG and evict(B=-1) == ARG
    assert evict(sink=3, recent=2) == ARG and evict(sink=2**31 - 1, recent=2**31 - 1) == ARG
    assert evict(B=0, w=None) == 0
    assert evict(w=None) == ARG and evict(s=None) == ARG and evict(wo=None) == ARG and evict(n=None) == ARG
    assert evict(w=bad) == ALIGN and evict(kept=bad) == ALIGN
    assert evict(fmt=5) == ARG
    assert evict(sw=7) == SHAPE and evict(so=3) == SHAPE
    assert evict(to=bd.Cache(a + 4096, 2, 3, 3 * 40, 40)) == SHAPE   # cannot hold the budget
    assert evict(to=bd.Cache(a + 160, 2, 4, 4 * 40, 40)) == ARG      # overlaps the cache, shifted by a row
    assert evict(to=bd.Cache(a, 2, 4, 4 * 40, 40)) == ARG            # the same start with other strides
    assert evict(wo=ctypes.c_void_p(a + 8192 + 16)) == ARG
    assert evict(wo=w, so=9) == ARG
    assert evict(ws=None) == WORKSPACE and evict(nbytes=16) == WORKSPACE


def test_eviction_of_seqlens_shifted_and_of_budgets_past_32_bits(L, mem):
    _, a = mem
    d, p = ctypes.byref(TINY), ctypes.c_void_p(a)
    src, dst = bd.Cache(a, 2, 8, 8 * 40, 40), bd.Cache(a + 4096, 2, 8, 8 * 40, 40)
    w, wo = ctypes.c_void_p(a + 8192), ctypes.c_void_p(a + 12288)

    def evict(s, n, budget=4):
        return L.mla_evict(d, ctypes.byref(src), 0, w, 8, s, 2, budget, 1, 1, ctypes.byref(dst), wo, 8, n, None, p, 16, None)

    assert evict(p, ctypes.c_void_p(a + 4)) == ARG and evict(ctypes.c_void_p(a + 4), p) == ARG  # a sequence's length under another's
    assert evict(p, p) == WORKSPACE and evict(p, ctypes.c_void_p(a + 8)) == WORKSPACE           # (16 bytes are too few)
    for budget in (2**30 + 1, 2**31 - 1):  # counting the chunks of such a budget would wrap
        assert evict(p, p, budget=budget) == ARG
        assert L.mla_evict_workspace_bytes(d, 0, 2, budget) == 0
    assert evict(p, p, budget=2**30) == WORKSPACE
    assert L.mla_evict_workspace_bytes(d, 0, 2, 2**30) >= 2 * 2**30 * 4


def test_binding_refuses_wrong_tensors():
    # every check comes before the library is called, on the CPU
    lib = bd.Library()
    dims = lib.dims(4, 32, 8, 16, 16, torch.float32)
    assert lib.packed_row_bytes(dims) == 64
    with pytest.raises(ValueError):
        lib.packed_row_bytes(lib.dims(4, 40, 8, 16, 16, torch.float32))
    cpu = torch.zeros(2, 4, 64, dtype=torch.uint8)
    c, k, pos = torch.zeros(2, 1, 32), torch.zeros(2, 1, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        lib.append_packed(dims, cpu, c, k, pos)
    with pytest.raises(TypeError):
        lib.append_packed(dims, torch.zeros(2, 4, 40, dtype=torch.float16), c, k, pos)
    with pytest.raises(ValueError):
        lib.evict(dims, torch.zeros(2, 4, 40), torch.zeros(2, 4), pos, 2)
