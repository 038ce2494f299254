"""The 4-bit cache on the GPU: append, load, attention and decode against the fp64 oracle.

Tolerances.  Codes are exact: the packed rows' values must equal the oracle's.
A rotated key is rounded once to the cache's type from an fp32 rotation whose
angle is good to 2^-23: half a step plus a few fp32 units.

Attention, per element, with A = sum_j p_j |c_j| and dS = 40 * 2^-23 * scale * max_j sum_e |q_e row_e|, the rounding of
at most 40 fp32 accumulations of a score:
  the output's rounding, half a step of its type          eps/2 * |o|
  the weights held in fp16 by the tensor-core kernel      2^-11 * A   (bf16 calls)
  the scores, in numerator and denominator                2 dS * A
  fp32 sums and exponentials of the weights               2^-16 * A
  weights too small for their type: fp32 arithmetic drops what is below 2^-126 of the row's largest weight, and fp16 rounds
  to multiples of 2^-24, half a step of which is 2^-25 where the largest weight is held as 2^7 or more (and the sum of
  weights is no smaller): at most 2^-126 and 2^-32 of the row's sum for every key, times sum_j |c_j|
  (an output whose large weights all meet latents that are exactly 0 consists of such weights alone)
  lse: dS, its own fp32 rounding 2^-23 |lse|, and 2^-16 for the sum and the two logarithms
"""
import numpy as np
import pytest
import torch

from latent_compressed_attention_absorbed_b200 import workload as wl
from mla_testutil import as_f64, check_close
from oracle import cache_oracle as co
from oracle import rope

pytestmark = pytest.mark.gpu

V3 = (128, 512, 64, 128, 128, torch.bfloat16)
TINY = (4, 32, 8, 16, 16, torch.float32)
# (H, d_c, d_r, d_n, d_v, dtype): the tensor-core geometry, the fp32 one, one head, widths that leave padding in a row,
# and an RoPE-free one
GEOMETRIES = {"v3": V3, "tiny": TINY, "one_head": (1, 16, 2, 4, 4, torch.bfloat16),
              "padded": (5, 80, 6, 8, 8, torch.bfloat16), "wide": (3, 1024, 128, 16, 16, torch.float32),
              "norope": (2, 48, 0, 8, 8, torch.float32)}


def dims_of(lib, g):
    return lib.dims(*g)


def rand(seed, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make_cache(lib, dims, g, T, T_max=None, seed=1, stride=None, fill=0):
    """A packed cache of sequences of T[b] tokens, the fp64 rows it stands for, and its raw tokens."""
    H, d_c, d_r, _, _, dt = g
    T_max = T_max or max(T)
    cache = torch.full((len(T), T_max, stride or lib.packed_row_bytes(dims)), fill, dtype=torch.uint8, device="cuda")
    rows = []
    for b, t in enumerate(T):
        c, k = rand(seed + b, 1, t, d_c, dtype=dt), rand(seed + 1000 + b, 1, t, d_r, dtype=dt)
        lib.append_packed(dims, cache[b:b + 1], c, k, i32(0))
        key = rope(as_f64(k)[0], np.arange(t)) if d_r else np.zeros((t, 0))
        key = as_f64(torch.from_numpy(key).to(torch.float32).to(dt))
        rows.append(np.concatenate([co.quantised(as_f64(c)[0]), key], -1))
    assert lib.device_status() == 0
    return cache, rows


def stored_rows(lib, dims, cache, T):
    """The rows the cache stands for, read back (their keys carry the append's own rounding)."""
    return [as_f64(lib.load_packed(dims, cache[b:b + 1], i32(0), t))[0] for b, t in enumerate(T)]


# ------------------------------------------------------------------ append and load

@pytest.mark.parametrize("name", list(GEOMETRIES))
@pytest.mark.parametrize("n_tok", [1, 3, 37])
def test_append_and_load(lib, name, n_tok):
    g = GEOMETRIES[name]
    H, d_c, d_r, _, _, dt = g
    dims, B, T_max = dims_of(lib, g), 3, 50
    c = rand(5, B, n_tok, d_c, dtype=dt) * torch.tensor([1e-5, 1.0, 900.0], device="cuda")[:, None, None].to(dt)
    c[1, 0, :16] = 0                                                      # a group of zeros
    c[0, 0, :3] = torch.tensor([3.5, -0.5, 7.0]).to(dt)                   # halves: scale 1
    k = rand(6, B, n_tok, d_r, dtype=dt)
    pos, row = [0, 100003, 17], [T_max - n_tok, 0, 5]
    cache = torch.full((B, T_max, lib.packed_row_bytes(dims)), 0xA5, dtype=torch.uint8, device="cuda")
    lib.append_packed(dims, cache, c, k, i32(*pos), rows=i32(*row))
    got = as_f64(lib.load_packed(dims, cache, i32(*row), n_tok))
    assert lib.device_status() == 0
    raw = cache.cpu().numpy()
    for b in range(B):
        want = co.quantised(as_f64(c)[b])
        np.testing.assert_array_equal(got[b, :, :d_c], want)
        np.testing.assert_array_equal(co.unpack_latents(raw[b, row[b]:row[b] + n_tok], d_c), want)
        key = rope(as_f64(k)[b], pos[b] + np.arange(n_tok)) if d_r else np.zeros((n_tok, 0))
        size = np.repeat(np.hypot(key[..., ::2], key[..., 1::2]), 2, axis=-1)
        assert np.all(np.abs(got[b, :, d_c:] - key) <= torch.finfo(dt).eps / 2 * np.abs(key) + 2.0 ** -21 * size)
        others = np.ones(T_max, bool)
        others[row[b]:row[b] + n_tok] = False
        assert np.all(raw[b, others] == 0xA5)


def test_append_defaults_to_the_position(lib):
    dims = dims_of(lib, TINY)
    c, k = rand(1, 2, 2, 32), rand(2, 2, 2, 8)
    a, b = (torch.zeros(2, 9, 64, dtype=torch.uint8, device="cuda") for _ in range(2))
    lib.append_packed(dims, a, c, k, i32(3, 7))
    lib.append_packed(dims, b, c, k, i32(3, 7), rows=i32(3, 7))
    assert torch.equal(a, b) and a.any()


def test_quantisation_next_to_a_half_and_to_a_scale(lib):
    # every scale's border, 7 s, and the numbers beside it; halves of a step and the numbers beside them (fp32)
    dims = dims_of(lib, (1, 16, 2, 4, 4, torch.float32))
    s = co.SCALES.astype(np.float32)
    x = np.zeros((256, 6, 16), np.float32)
    for j, top in enumerate((7 * s, np.nextafter(7 * s, np.float32(0)), np.nextafter(7 * s, np.float32(np.inf)))):
        x[:, j, 0] = np.minimum(top, 13440)
    half = (np.arange(14) - 6.5).astype(np.float32)[None, :] * s[:, None]
    for j, v in enumerate((half, np.nextafter(half, np.float32(0)), np.nextafter(half, np.float32(np.inf) * np.sign(half)))):
        x[:, 3 + j, 0], x[:, 3 + j, 2:] = 7 * s, v
    x = x.reshape(1, -1, 16)
    cache = torch.zeros(1, x.shape[1], lib.packed_row_bytes(dims), dtype=torch.uint8, device="cuda")
    lib.append_packed(dims, cache, torch.from_numpy(x).cuda(), torch.zeros(1, x.shape[1], 2, device="cuda"), i32(0))
    assert lib.device_status() == 0
    np.testing.assert_array_equal(as_f64(lib.load_packed(dims, cache, i32(0), x.shape[1]))[0, :, :16], co.quantised(x[0].astype(np.float64)))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_latents_that_do_not_fit(lib, dt):
    dims = dims_of(lib, (1, 48, 2, 4, 4, dt))
    c = torch.ones(1, 2, 48, device="cuda", dtype=dt)
    c[0, 0, 3], c[0, 0, 17], c[0, 1, 40], c[0, 1, 41] = float("nan"), float("inf"), -float("inf"), 20000.0
    cache = torch.zeros(1, 2, lib.packed_row_bytes(dims), dtype=torch.uint8, device="cuda")
    lib.append_packed(dims, cache, c, torch.zeros(1, 2, 2, device="cuda", dtype=dt), i32(0))
    assert lib.device_status() == 8
    got = as_f64(lib.load_packed(dims, cache, i32(0), 2))[0, :, :48]
    np.testing.assert_array_equal(got, co.quantised(as_f64(c)[0]))
    assert got[0, 3] == 0 and got[0, 17] == 13440 and got[1, 40] == -13440 and got[1, 41] == 13440


def test_rows_out_of_range(lib):
    dims = dims_of(lib, TINY)
    c, k = rand(1, 5, 2, 32), rand(2, 5, 2, 8)
    cache = torch.full((5, 8, 64), 7, dtype=torch.uint8, device="cuda")
    lib.append_packed(dims, cache, c, k, i32(0, 0, -1, 2**31 - 1, 6), rows=i32(7, -1, 0, 0, 6))
    assert lib.device_status() == 1
    assert torch.all(cache[:4] == 7) and torch.any(cache[4, 6] != 7)  # only the last sequence's rows fit
    lib.append_packed(dims, cache[:, :1], c, k, i32(0, 0, 0, 0, 0))   # two tokens into one row
    assert lib.device_status() == 1
    out = lib.load_packed(dims, cache, i32(7, -1, 0, 2**31 - 1, 6), 2)
    assert lib.device_status() == 1
    assert not out[0].any() and not out[1].any() and not out[3].any() and out[2].any() and out[4].any()


def test_append_rows_is_append_cache_at_another_row(lib):
    for g in (V3, TINY, GEOMETRIES["padded"]):
        H, d_c, d_r, _, _, dt = g
        dims = dims_of(lib, g)
        w = (d_c + d_r + 7) // 8 * 8
        c, k = rand(1, 2, 3, d_c, dtype=dt), rand(2, 2, 3, d_r, dtype=dt)
        a, b = (torch.zeros(2, 40, w, dtype=dt, device="cuda") for _ in range(2))
        lib.append_cache(dims, a, c, k, i32(20, 31))
        lib.append_rows(dims, b, c, k, i32(20, 31), i32(4, 37))
        assert lib.device_status() == 0
        assert torch.equal(a[0, 20:23], b[0, 4:7]) and torch.equal(a[1, 31:34], b[1, 37:40])
        b[0, 4:7] = 0
        b[1, 37:40] = 0
        assert not b.any()
        lib.append_rows(dims, b, c, k, i32(0, 0), i32(38, -1))
        assert lib.device_status() == 1 and not b.any()


# ------------------------------------------------------------------ attention

def check_attention(o, lse, q_hat, rows, T, q_len, g, scale, what=""):
    H, d_c, _, _, _, dt = g
    o, lse, q = as_f64(o), lse.double().cpu().numpy(), as_f64(q_hat)
    half = torch.finfo(dt).eps / 2
    held, least = (2.0 ** -11, 2.0 ** -32) if dt == torch.bfloat16 else (0.0, 2.0 ** -126)
    for b, t in enumerate(T):
        for i in range(q_len):
            n = t - q_len + 1 + i
            ref, ref_lse = co.attend(q[b, i], rows[b], n, d_c, scale)
            s = scale * q[b, i] @ rows[b][:n].T
            p = np.exp(s - ref_lse[:, None])
            size = p @ np.abs(rows[b][:n, :d_c])
            dS = 40 * 2.0 ** -23 * scale * (np.abs(q[b, i]) @ np.abs(rows[b][:n]).T).max(-1)
            tol = half * np.abs(ref) + (held + 2.0 ** -16 + 2 * dS[:, None]) * size + least * np.abs(rows[b][:n, :d_c]).sum(0)
            err = np.abs(o[b, i] - ref)
            assert np.all(err <= tol), f"{what} sequence {b} query {i}: {np.max(err / tol):.3g} of the tolerance"
            lerr = np.abs(lse[b, i] - ref_lse)
            ltol = dS + 2.0 ** -23 * np.abs(ref_lse) + 2.0 ** -16
            assert np.all(lerr <= ltol), f"{what} lse {b} {i}: {np.max(lerr / ltol):.3g} of the tolerance"


def attend_case(lib, g, T, q_len, opts=None, T_max=None, stride=None, std=None, seed=3, fill=0):
    H, d_c, d_r, _, _, dt = g
    dims = dims_of(lib, g)
    cache, _ = make_cache(lib, dims, g, T, T_max=T_max, stride=stride, fill=fill)
    rows = stored_rows(lib, dims, cache, T)
    q = rand(seed, len(T), q_len, H, d_c + d_r, dtype=dt, std=std or 0.25)
    lse = torch.full((len(T), q_len, H), 99.0, device="cuda")
    o = lib.attend_packed(dims, q, cache, i32(*T), lse=lse, opts=opts)
    return dims, cache, rows, q, o, lse


ATTEND = [
    ((1,), 1, 0), ((2,), 2, 0), ((16,), 16, 0), ((63, 64, 65), 1, 0), ((127, 128, 129, 1), 1, 0), ((257, 700), 2, 3),
    ((255, 256, 1, 130), 1, 1),          # one cluster does everything
    ((1000, 999), 2, 16), ((513, 2000, 5), 3, 7), ((257, 1024), 4, 5), ((4096,), 1, 64), ((4096,), 1, 0),
    ((4000,) + (5,) * 24, 1, 0), ((1500, 9, 260), 8, 0), ((16, 700), 16, 5), ((640,) * 7, 1, 8), ((384,) * 7, 2, 8),
    ((200,) * 80, 1, 0),                 # more sequences than clusters
]


@pytest.mark.parametrize("T,q_len,pairs", ATTEND)
def test_attend_v3(lib, T, q_len, pairs):
    dims, cache, rows, q, o, lse = attend_case(lib, V3, T, q_len, lib.opts(num_pairs=pairs))
    assert lib.device_status() == 0 and lib.last_path() == "sm100"
    check_attention(o, lse, q, rows, T, q_len, V3, 192 ** -0.5, f"{T} {q_len} {pairs}")


@pytest.mark.parametrize("name", [n for n in GEOMETRIES if n != "v3"])
@pytest.mark.parametrize("T,q_len", [((1,), 1), ((40, 3, 129), 2), ((300,), 5)])
def test_attend_other_geometries(lib, name, T, q_len):
    g = GEOMETRIES[name]
    T = tuple(max(t, q_len) for t in T)
    dims, cache, rows, q, o, lse = attend_case(lib, g, T, q_len)
    assert lib.device_status() == 0 and lib.last_path() == "generic"
    check_attention(o, lse, q, rows, T, q_len, g, (g[3] + g[2]) ** -0.5, name)


def test_generic_path_v3(lib):
    T = (130, 7)
    dims, cache, rows, q, o, lse = attend_case(lib, V3, T, 2, lib.opts(path=2))
    assert lib.last_path() == "generic"
    check_attention(o, lse, q, rows, T, 2, V3, 192 ** -0.5)


@pytest.mark.parametrize("std", [2.0, 30.0])
def test_sharp_and_one_sided_rows(lib, std):
    # scores over hundreds of log2 units: most weights vanish, and the running maximum moves often
    T = (900, 70, 131)
    dims, cache, rows, q, o, lse = attend_case(lib, V3, T, 2, std=std)
    assert lib.device_status() == 0
    check_attention(o, lse, q, rows, T, 2, V3, 192 ** -0.5)


def test_rows_past_the_length_may_hold_anything(lib):
    T = (70, 5, 129, 128)
    dims, cache, rows, q, o, lse = attend_case(lib, V3, T, 1, T_max=300)
    for b, t in enumerate(T):
        cache[b, t:] = 0xFF   # every code and scale at its largest, and NaN keys
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    lib.attend_packed(dims, q, cache, i32(*T), out=o2, lse=lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_attention(o2, lse2, q, rows, T, 1, V3, 192 ** -0.5)


def test_strided_cache(lib):
    T = (300, 17, 129)
    dims, cache, rows, q, o, lse = attend_case(lib, V3, T, 2, stride=448)
    check_attention(o, lse, q, rows, T, 2, V3, 192 ** -0.5)
    wide = torch.full((6, 301, 432), 0xFF, dtype=torch.uint8, device="cuda")
    view = wide[::2, :300, :416]
    view.copy_(cache[:, :, :416])
    o2 = lib.attend_packed(dims, q, view, i32(*T))
    assert torch.equal(o, o2) and lib.device_status() == 0


def test_bad_lengths(lib):
    T = (100, 60, 50, 33)
    dims, cache, rows, q, o, lse = attend_case(lib, V3, T, 2)
    for path in (0, 2):
        o2, lse2 = torch.full_like(o, 5.0), torch.full_like(lse, 5.0)
        lib.attend_packed(dims, q, cache, i32(100, 101, 1, -3), out=o2, lse=lse2, opts=lib.opts(path=path))
        assert lib.device_status() == 2
        assert not o2[1:].float().any() and torch.all(lse2[1:] == -float("inf"))
        check_attention(o2[:1], lse2[:1], q[:1], rows[:1], T[:1], 2, V3, 192 ** -0.5)


def test_without_lse_and_repeated(lib):
    T = (900, 77)
    dims, cache, rows, q, o, lse = attend_case(lib, V3, T, 2, lib.opts(num_pairs=5))
    for _ in range(3):
        assert torch.equal(lib.attend_packed(dims, q, cache, i32(*T), opts=lib.opts(num_pairs=5)), o)


def test_attend_latent_lse(lib):
    # the full-width attention: the same output as without the log-sum-exps, and their values
    for g, T, q_len, pairs in ((V3, (700, 333, 64), 1, 3), (V3, (1000, 999), 2, 16), (V3, (640,) * 7, 1, 8), (TINY, (64, 3), 2, 0)):
        H, d_c, d_r, _, _, dt = g
        dims = dims_of(lib, g)
        cache = rand(9, len(T), max(T), d_c + d_r, dtype=dt)
        q = rand(3, len(T), q_len, H, d_c + d_r, dtype=dt, std=0.25)
        lse = torch.full((len(T), q_len, H), 99.0, device="cuda")
        opts = lib.opts(num_pairs=pairs)
        o = lib.attend_latent_lse(dims, q, cache, i32(*T), lse, opts=opts)
        assert lib.device_status() == 0
        ref = lib.attend_latent(dims, q, cache, i32(*T), opts=opts)
        if dt == torch.bfloat16:
            assert torch.equal(o, ref)
        rows = as_f64(cache)
        scale = (g[3] + d_r) ** -0.5
        for b, t in enumerate(T):
            for i in range(q_len):
                want_o, want = co.attend(as_f64(q)[b, i], rows[b], t - q_len + 1 + i, d_c, scale)
                dS = 40 * 2.0 ** -23 * scale * (np.abs(as_f64(q)[b, i]) @ np.abs(rows[b][:t]).T).max(-1)
                got = lse[b, i].double().cpu().numpy()
                assert np.all(np.abs(got - want) <= dS + 2.0 ** -23 * np.abs(want) + 2.0 ** -16)
        lse.fill_(5.0)
        lib.attend_latent_lse(dims, q, cache, i32(*([max(T) + 1] + list(T[1:]))), lse, opts=opts)
        assert lib.device_status() == 2 and torch.all(lse[0] == -float("inf")) and torch.all(torch.isfinite(lse[1:]))


# ------------------------------------------------------------------ decode

def decode_inputs(g, B, q_len, seed=31):
    H, d_c, d_r, d_n, d_v, dt = g
    std = 0.02 if d_c == 512 else d_c ** -0.5
    return (rand(seed, B, q_len, H, d_n, dtype=dt), rand(seed + 1, B, q_len, H, d_r, dtype=dt),
            rand(seed + 2, H, d_n, d_c, dtype=dt, std=std), rand(seed + 3, H, d_v, d_c, dtype=dt, std=std))


def decode_reference(g, qn, qr, uk, uv, rows, T, seen, q_len):
    H, d_c, d_r, d_n, d_v, dt = g
    out = []
    for b, t in enumerate(T):
        pos = seen[b] - q_len + np.arange(q_len)
        q = np.concatenate([np.einsum("hdc,ihd->ihc", as_f64(uk), as_f64(qn)[b]), rope(as_f64(qr)[b], pos[:, None])], -1)
        o = [co.attend(q[i], rows[b], t - q_len + 1 + i, d_c, (d_n + d_r) ** -0.5)[0] for i in range(q_len)]
        out.append(np.einsum("hvc,ihc->ihv", as_f64(uv), np.array(o)))
    return np.array(out)


@pytest.mark.parametrize("g,T,q_len", [(V3, (1,), 1), (V3, (700, 65), 1), (V3, (333, 130, 64, 7, 9), 2), (V3, (150,) * 20, 1),
                                       (TINY, (64, 9), 1), (TINY, (40, 5), 3)])
def test_decode(lib, g, T, q_len):
    H, d_c, d_r, _, _, dt = g
    dims = dims_of(lib, g)
    cache, _ = make_cache(lib, dims, g, T, T_max=max(T) + 3)
    rows = stored_rows(lib, dims, cache, T)
    ins = decode_inputs(g, len(T), q_len)
    out = lib.decode_packed(dims, *ins, cache, i32(*T))
    assert lib.device_status() == 0
    kind = "bf16" if dt == torch.bfloat16 else "f32"
    check_close(as_f64(out), decode_reference(g, *ins, rows, T, T, q_len), kind, "decode")
    # tokens counted apart from rows, and the folded queries and log-sum-exps handed out
    seen = tuple(t + 1000 * (b + 1) for b, t in enumerate(T))
    q_hat = torch.zeros(len(T), q_len, H, d_c + d_r, dtype=dt, device="cuda")
    lse = torch.zeros(len(T), q_len, H, device="cuda")
    out = lib.decode_packed(dims, *ins, cache, i32(*T), n_seen=i32(*seen), q_hat=q_hat, lse=lse)
    assert lib.device_status() == 0
    check_close(as_f64(out), decode_reference(g, *ins, rows, T, seen, q_len), kind, "decode with n_seen")
    assert torch.equal(q_hat, lib.absorb_query(dims, ins[0], ins[1], ins[2], i32(*seen)))
    lse2 = torch.zeros_like(lse)
    lib.attend_packed(dims, q_hat, cache, i32(*T), lse=lse2)
    assert torch.equal(lse, lse2)


def test_decode_in_a_graph_and_on_another_stream(lib):
    T, q_len = (700, 333), 2
    dims = dims_of(lib, V3)
    cache, _ = make_cache(lib, dims, V3, T)
    ins = decode_inputs(V3, 2, q_len)
    ref = lib.decode_packed(dims, *ins, cache, i32(*T))
    seq = i32(*T)
    out = torch.zeros_like(ref)
    ws = torch.empty(lib.packed_workspace_bytes(dims, 2, q_len), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.decode_packed(dims, *ins, cache, seq, out=out, workspace=ws)
    s.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.decode_packed(dims, *ins, cache, seq, out=out, workspace=ws)
    for t in ((700, 333), (650, 300)):  # lengths are read when the graph runs
        seq.copy_(i32(*t))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, lib.decode_packed(dims, *ins, cache, i32(*t)))
    assert lib.device_status() == 0


def test_two_calls_at_once(lib):
    T = (2000, 1000, 300)
    dims = dims_of(lib, V3)
    cache, _ = make_cache(lib, dims, V3, T)
    q = [rand(s, 3, 1, 128, 576, dtype=torch.bfloat16, std=0.25) for s in (1, 2)]
    ref = [lib.attend_packed(dims, x, cache, i32(*T)) for x in q]
    streams = [torch.cuda.Stream() for _ in q]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for x, s in zip(q, streams):
            with torch.cuda.stream(s):
                got.append(lib.attend_packed(dims, x, cache, i32(*T)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref[n % 2]) for n, o in enumerate(got))
    assert lib.device_status() == 0


def test_cache_of_more_than_two_to_the_31_bytes(lib):
    # the last of the sequences starts beyond 2^31 bytes
    dims = dims_of(lib, V3)
    T_max = 700000
    cache = torch.empty(9, T_max, 416, dtype=torch.uint8, device="cuda")
    small, _ = make_cache(lib, dims, V3, (300,))
    c, k = rand(1, 1, 300, 512, dtype=torch.bfloat16), rand(1001, 1, 300, 64, dtype=torch.bfloat16)
    lib.append_packed(dims, cache[8:], c, k, i32(0))
    lib.append_packed(dims, cache[8:], c, k, i32(0), rows=i32(T_max - 300))
    assert torch.equal(cache[8, :300], small[0]) and torch.equal(cache[8, T_max - 300:], small[0])
    q = rand(2, 9, 1, 128, 576, dtype=torch.bfloat16, std=0.25)
    lse = torch.zeros(9, 1, 128, device="cuda")
    seq = i32(*([1] * 8 + [300]))
    cache[:8, 0] = small[0, 0]
    one = lib.opts(num_pairs=1)  # no sequence is cut, so that the bits do not depend on the rest of the batch
    o = lib.attend_packed(dims, q, cache, seq, lse=lse, opts=one)
    assert lib.device_status() == 0
    assert torch.equal(o[8:], lib.attend_packed(dims, q[8:], small, i32(300), opts=one))
    assert torch.equal(lib.load_packed(dims, cache, i32(*([0] * 8 + [T_max - 1])), 1)[8:], lib.load_packed(dims, small, i32(299), 1))


# ------------------------------------------------------------------ edges of the calls

def test_many_short_sequences(lib):
    # more sequences than threads of a block plan for, some of them invalid, against the CUDA-core path
    B, T_max, q_len = 1500, 300, 2
    dims = dims_of(lib, V3)
    g = torch.Generator().manual_seed(3)
    T = torch.randint(2, T_max + 1, (B,), generator=g)
    T[::97] = 1                                   # shorter than the queries
    T[5] = T_max + 1
    cache = torch.randint(0, 256, (B, T_max, 416), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.uint8)
    cache[:, :, 256:288] = 160                    # every scale 1/2, so that the values are of one size
    cache[:, :, 288:] = torch.randn(B, T_max, 64, device="cuda").bfloat16().view(torch.uint8)
    q = rand(2, B, q_len, 128, 576, dtype=torch.bfloat16, std=0.05)
    seq = T.to(torch.int32).cuda()
    out = {}
    for path in (0, 2):
        lse = torch.zeros(B, q_len, 128, device="cuda")
        o = lib.attend_packed(dims, q, cache, seq, lse=lse, opts=lib.opts(path=path))
        assert lib.device_status() == 2
        out[path] = (o.float(), lse)
    bad = (T < q_len) | (T > T_max)
    assert not out[0][0][bad].any() and torch.all(out[0][1][bad] == -float("inf"))
    good = (~bad).cuda()
    # both paths round the output once (2^-8 each) and hold the weights to 2^-11
    a, b = out[0][0][good], out[2][0][good]
    assert torch.all((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -9 * 4)   # |latents| <= 4
    assert torch.all((out[0][1][good] - out[2][1][good]).abs() <= 1e-4)


def test_sixteen_byte_alignment_is_enough(lib):
    T = (300, 77)
    dims, cache, rows, q, o, lse = attend_case(lib, V3, T, 2)

    def off(t):  # the same tensor 16 bytes into a buffer
        n = t.numel() * t.element_size()
        buf = torch.zeros(n + 32, dtype=torch.uint8, device="cuda")
        at = 16 if buf.data_ptr() % 32 == 0 else 0
        v = buf[at:at + n].view(t.dtype).view(t.shape)
        v.copy_(t)
        return v
    o2 = off(torch.zeros_like(o))
    ws = torch.empty(lib.packed_workspace_bytes(dims, 2, 2) + 16, dtype=torch.uint8, device="cuda")[16:]
    lib.attend_packed(dims, off(q), off(cache), off(i32(*T)), out=o2, workspace=ws)
    assert lib.device_status() == 0 and torch.equal(o, o2)


def test_empty_calls(lib):
    dims = dims_of(lib, V3)
    e = torch.empty
    u8, bf = dict(dtype=torch.uint8, device="cuda"), dict(dtype=torch.bfloat16, device="cuda")
    none = i32()
    cache = torch.zeros(2, 8, 416, **u8)
    lib.append_packed(dims, cache, e(0, 1, 512, **bf), e(0, 1, 64, **bf), none)
    lib.append_packed(dims, cache, e(2, 0, 512, **bf), e(2, 0, 64, **bf), i32(0, 0))
    assert lib.load_packed(dims, cache, none, 3).shape == (0, 3, 576)
    assert lib.attend_packed(dims, e(0, 1, 128, 576, **bf), cache, none).shape == (0, 1, 128, 512)
    lib.accumulate_weights(dims, e(0, 1, 128, 576, **bf), e(0, 1, 128, device="cuda"), cache, none, e(0, 8, device="cuda"))
    lib.evict(dims, cache, e(0, 8, device="cuda"), none, 4)
    assert lib.device_status() == 0 and not cache.any()


@pytest.mark.parametrize("T,q_len,pairs", [((700, 333, 64), 1, 2), ((900, 77), 2, 4), ((5000,), 1, 1)])
def test_expired_wait(lib, T, q_len, pairs):
    # the loaders stop before the third 64-key tile, so that a bounded wait runs out (50 ms); the kernel reports it, ends in
    # order, and the next call is right
    from latent_compressed_attention_absorbed_b200 import binding
    dims, cache, rows, q, o, lse = attend_case(lib, V3, T, q_len, lib.opts(num_pairs=pairs))
    lib.attend_packed(dims, q, cache, i32(*T), opts=lib.opts(num_pairs=pairs, wait_limit_ns=50_000_000, withhold_tile=3))
    assert lib.device_status() & binding.STATUS_TIMEOUT
    assert torch.equal(lib.attend_packed(dims, q, cache, i32(*T), opts=lib.opts(num_pairs=pairs)), o)
    assert lib.device_status() == 0


def test_new_memory_belongs_to_the_calls_stream(lib, monkeypatch):
    # memory of the current stream may still be in use there, and would be handed out again there too early
    T = (300, 40)
    dims = dims_of(lib, V3)
    cache, _ = make_cache(lib, dims, V3, T)
    full = rand(3, 2, 300, 576, dtype=torch.bfloat16)
    ins = decode_inputs(V3, 2, 1)
    q = rand(2, 2, 1, 128, 576, dtype=torch.bfloat16, std=0.25)
    seq, first, lse, w = i32(*T), i32(0, 0), torch.zeros(2, 1, 128, device="cuda"), rand(4, 2, 300)
    calls = (lambda s: lib.attend_packed(dims, q, cache, seq, stream=s),
             lambda s: lib.decode_packed(dims, *ins, cache, seq, stream=s),
             lambda s: lib.load_packed(dims, cache, first, 40, stream=s),
             lambda s: lib.attend_latent_lse(dims, q, full, seq, lse, stream=s))
    ref = [call(None) for call in calls]
    used, empty = [], torch.empty

    def recorded(*a, **k):
        used.append(torch.cuda.current_stream())
        return empty(*a, **k)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", recorded)
    got = [call(s) for call in calls]
    lib.evict(dims, cache, w, seq, 100, stream=s)
    s.synchronize()
    assert used and all(u == s for u in used)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert seq.tolist() == [100, 40] and lib.device_status() == 0
