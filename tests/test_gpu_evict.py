"""Accumulated attention weights and eviction on the GPU against the fp64 oracle.

Tolerance of a row's weight w, with dS the rounding of a score (at most 40 fp32 accumulations, as for the attention) and
x the largest exponent argument: each term exp(s - lse) is off by dS, by the fp32 rounding of its argument
(2^-23 (|s| + |lse|)) and by 2^-21 for the exponential; the fp32 sum of at most 16 * 128 terms, in at most 512 steps, by
2^-15; everything relative to w.  Eviction moves bytes and must be exact.
"""
import numpy as np
import pytest
import torch

from mla_testutil import as_f64
from oracle import cache_oracle as co
from test_gpu_packed import GEOMETRIES, TINY, V3, decode_inputs, decode_reference, dims_of, i32, make_cache, rand, stored_rows

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ weights

def weights_case(lib, g, T, q_len, packed, T_max=None, opts=None, prev=None, decay=1.0, std=0.25):
    H, d_c, d_r, d_n, _, dt = g
    dims = dims_of(lib, g)
    T_max = T_max or max(T)
    if packed:
        cache, _ = make_cache(lib, dims, g, T, T_max=T_max, fill=0xFF)
        rows = stored_rows(lib, dims, cache, T)
    else:
        cache = torch.full((len(T), T_max, (d_c + d_r + 7) // 8 * 8), float("nan"), dtype=dt, device="cuda")
        for b, t in enumerate(T):
            cache[b, :t] = rand(50 + b, t, cache.shape[2], dtype=dt)
        rows = [as_f64(cache[b, :t, :d_c + d_r]) for b, t in enumerate(T)]
    q = rand(3, len(T), q_len, H, d_c + d_r, dtype=dt, std=std)
    scale = (d_n + d_r) ** -0.5
    lse = np.array([[co.attend(as_f64(q)[b, i], rows[b], t - q_len + 1 + i, d_c, scale)[1] for i in range(q_len)]
                    for b, t in enumerate(T)])
    lse = torch.from_numpy(lse).float().cuda()
    w = torch.full((len(T), T_max), -1.0, device="cuda")
    prev = prev(w) if callable(prev) else prev
    before = (prev if prev is not None else torch.zeros_like(w)).double().cpu().numpy()
    lib.accumulate_weights(dims, q, lse, cache, i32(*T), w, prev=prev, decay=decay, opts=opts)
    return dims, cache, rows, q, lse, w, before, scale


def check_weights(w, before, decay, q, lse, rows, T, q_len, scale, untouched=-1.0):
    w, q, z = w.double().cpu().numpy(), as_f64(q), lse.double().cpu().numpy()
    for b, t in enumerate(T):
        new = co.row_weights(q[b], z[b], rows[b], t, scale)
        want = decay * before[b, :t] + new
        size = np.abs(q[b]).reshape(-1, q.shape[-1]).astype(np.float64)
        reach = scale * (size @ np.abs(rows[b]).T).max()
        rel = 40 * 2.0 ** -23 * reach + 2.0 ** -23 * (reach + np.abs(z[b]).max()) + 2.0 ** -21 + 2.0 ** -15
        tol = rel * new + 2.0 ** -23 * (np.abs(decay * before[b, :t]) + np.abs(want))
        err = np.abs(w[b, :t] - want)
        assert np.all(err <= tol), f"sequence {b}: {np.max(err / tol):.3g} of the tolerance"
        if untouched is not None:
            assert np.all(w[b, t:] == untouched)


WEIGHTS = [((1,), 1), ((127, 128, 129, 1), 1), ((16,), 16), ((300, 17), 2), ((1000, 513, 2), 2), ((2000,), 3), ((140,) * 160, 1),
           ((700, 260, 33), 8)]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,q_len", WEIGHTS)
def test_weights_v3(lib, T, q_len, packed):
    dims, cache, rows, q, lse, w, before, scale = weights_case(lib, V3, T, q_len, packed, T_max=max(T) + 5)
    assert lib.device_status() == 0 and lib.last_path() == "sm100"
    check_weights(w, before, 1.0, q, lse, rows, T, q_len, scale)
    assert w[w >= 0].sum().item() == pytest.approx(len(T) * q_len * 128, rel=1e-3)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("name", [n for n in GEOMETRIES if n != "v3"])
def test_weights_other_geometries(lib, name, packed):
    T = (130, 5, 9)
    dims, cache, rows, q, lse, w, before, scale = weights_case(lib, GEOMETRIES[name], T, 3, packed)
    assert lib.device_status() == 0 and lib.last_path() == "generic"
    check_weights(w, before, 1.0, q, lse, rows, T, 3, scale)


@pytest.mark.parametrize("path", [0, 2])
@pytest.mark.parametrize("packed", [False, True])
def test_weights_added_to_earlier_ones(lib, packed, path):
    T = (260, 40)
    for how in ("apart", "itself"):
        prev = rand(8, 2, 260).abs() if how == "apart" else (lambda w: w)
        dims, cache, rows, q, lse, w, before, scale = weights_case(lib, V3, T, 2, packed, prev=prev, decay=0.75, opts=lib.opts(path=path))
        check_weights(w, before, 0.75, q, lse, rows, T, 2, scale)


def test_weights_rows_without_queries_and_bad_lengths(lib):
    T = (140, 60, 50)
    for path in (0, 2):
        dims, cache, rows, q, lse, w, before, scale = weights_case(lib, V3, T, 2, True, opts=lib.opts(path=path))
        lse[0, 0] = -float("inf")          # a query that counts nothing
        w2 = torch.full_like(w, -1.0)
        lib.accumulate_weights(dims, q, lse, cache, i32(140, 141, 1), w2, opts=lib.opts(path=path))
        assert lib.device_status() == 2
        assert torch.all(w2[1:] == -1)
        check_weights(w2[:1], before[:1], 1.0, q[:1], lse[:1], rows[:1], T[:1], 2, scale)


def test_weights_strides_and_repeats(lib):
    T = (300, 129)
    dims, cache, rows, q, lse, w, before, scale = weights_case(lib, V3, T, 2, False)
    big = torch.full((2, 1000), 4.0, device="cuda")
    lib.accumulate_weights(dims, q, lse, cache, i32(*T), big[:, 10:310])
    assert torch.equal(big[0, 10:310], w[0]) and torch.equal(big[1, 10:139], w[1, :129])
    assert torch.all(big[:, :10] == 4) and torch.all(big[:, 310:] == 4) and torch.all(big[1, 139:] == 4)
    for _ in range(3):
        again = torch.zeros_like(w)
        lib.accumulate_weights(dims, q, lse, cache, i32(*T), again)
        assert torch.equal(again[0], w[0])
    # the sums do not depend on what else is in the batch
    alone = torch.zeros(1, 300, device="cuda")
    lib.accumulate_weights(dims, q[:1], lse[:1], cache[:1], i32(300), alone)
    assert torch.equal(alone[0], w[0])


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,q_len", [((2000, 700), 1), ((1500,), 3)])
def test_weights_expired_wait(lib, packed, T, q_len):
    dims, cache, rows, q, lse, w, before, scale = weights_case(lib, V3, T, q_len, packed)
    lib.accumulate_weights(dims, q, lse, cache, i32(*T), torch.zeros_like(w),
                           opts=lib.opts(wait_limit_ns=50_000_000, withhold_tile=1))
    assert lib.device_status() & 4
    again = torch.full_like(w, -1.0)
    lib.accumulate_weights(dims, q, lse, cache, i32(*T), again)
    assert lib.device_status() == 0 and torch.equal(again, w)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,q_len", [((5,), 2), ((300,), 3), ((128, 900, 257), 4), ((600,), 5), ((1000, 16, 31), 16), ((2500, 2500), 8),
                                     ((4096,), 16)])
def test_weights_queries_shared_by_a_cluster(lib, T, q_len, packed):
    """Few tiles and several queries: a cluster's CTAs take the queries of a tile between them.  The same sequences in a cache so
    large that one CTA takes them all give the same sums (added up in another order)."""
    dims, cache, rows, q, lse, w, before, scale = weights_case(lib, V3, T, q_len, packed, T_max=max(T) + 3)
    assert lib.device_status() == 0 and lib.last_path() == "sm100"
    check_weights(w, before, 1.0, q, lse, rows, T, q_len, scale)
    again = torch.full_like(w, -1.0)
    lib.accumulate_weights(dims, q, lse, cache, i32(*T), again, prev=None)
    twice = torch.full_like(w, -1.0)
    lib.accumulate_weights(dims, q, lse, cache, i32(*T), twice, prev=None)
    assert torch.equal(again, twice)
    wide = torch.zeros(len(T), 60000, cache.shape[2], dtype=cache.dtype, device="cuda")
    wide[:, :cache.shape[1]] = cache
    one = torch.full((len(T), 60000), -1.0, device="cuda")
    lib.accumulate_weights(dims, q, lse, wide, i32(*T), one)
    assert lib.device_status() == 0
    n = cache.shape[1]
    # the terms are the same; up to q_len partial sums are added in another order, each step off by 2^-24 of at most the sum
    assert torch.all((again - one[:, :n]).abs() <= 2 * q_len * 2.0 ** -24 * one[:, :n].abs())
    assert torch.all(one[:, n:] == -1)
    # a wait that runs out in some CTA of a cluster ends all of them in order
    lib.accumulate_weights(dims, q, lse, cache, i32(*T), torch.zeros_like(w), opts=lib.opts(wait_limit_ns=50_000_000, withhold_tile=1))
    assert lib.device_status() & 4 or max(T) <= 64
    lib.accumulate_weights(dims, q, lse, cache, i32(*T), twice)
    assert lib.device_status() == 0 and torch.equal(again, twice)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("B,T_max,q_len", [(300, 700, 3), (1500, 200, 2)])
def test_weights_again_and_again(lib, packed, B, T_max, q_len):
    # a row that is overwritten while it is still being read shows once in hundreds of calls
    dims = dims_of(lib, V3)
    T = torch.randint(q_len, T_max + 1, (B,), generator=torch.Generator().manual_seed(5)).to(torch.int32).cuda()
    q = rand(2, B, q_len, 128, 576, dtype=torch.bfloat16, std=0.25)
    lse = torch.full((B, q_len, 128), 5.0, device="cuda")
    if packed:
        cache = torch.randint(0, 256, (B, T_max, 416), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.uint8)
        cache[:, :, 256:288] = 160
        cache[:, :, 288:] = rand(4, B, T_max, 64, dtype=torch.bfloat16).view(torch.uint8)
    else:
        cache = rand(3, B, T_max, 576, dtype=torch.bfloat16)
    first = lib.accumulate_weights(dims, q, lse, cache, T, torch.zeros(B, T_max, device="cuda"))
    w, differ = torch.empty_like(first), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(1000):
        w.zero_()
        lib.accumulate_weights(dims, q, lse, cache, T, w)
        differ += (w != first).any()
    assert torch.isfinite(first).all() and differ.item() == 0 and lib.device_status() == 0


@pytest.mark.parametrize("T,q_len", [((4096,), 1), ((700, 333, 5, 1200), 2)])
def test_packed_attention_again_and_again(lib, T, q_len):
    dims = dims_of(lib, V3)
    cache, _ = make_cache(lib, dims, V3, T)
    q = rand(2, len(T), q_len, 128, 576, dtype=torch.bfloat16, std=0.25)
    first = lib.attend_packed(dims, q, cache, i32(*T))
    out, seq, differ = torch.empty_like(first), i32(*T), torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(1000):
        out.zero_()
        lib.attend_packed(dims, q, cache, seq, out=out)
        differ += (out != first).any()
    assert differ.item() == 0 and lib.device_status() == 0


@pytest.mark.parametrize("q_len", [2, 3])
def test_weights_of_ranges_of_several_blocks(lib, q_len):
    # more than eight tiles a CTA: blocks of two, which end inside sequences and ranges; against the CUDA-core path
    T = torch.randint(3000, 4701, (48,), generator=torch.Generator().manual_seed(6))
    dims, seq, T_max = dims_of(lib, V3), T.to(torch.int32).cuda(), 4700
    cache = rand(3, 48, T_max, 576, dtype=torch.bfloat16)
    q = rand(2, 48, q_len, 128, 576, dtype=torch.bfloat16, std=0.05)
    lse = torch.zeros(48, q_len, 128, device="cuda")
    lib.attend_latent_lse(dims, q, cache, seq, lse)
    w, v = torch.full((48, T_max), -1.0, device="cuda"), torch.full((48, T_max), -1.0, device="cuda")
    lib.accumulate_weights(dims, q, lse, cache, seq, w)
    assert lib.last_path() == "sm100"
    lib.accumulate_weights(dims, q, lse, cache, seq, v, opts=lib.opts(path=2))
    assert lib.device_status() == 0
    past = torch.arange(T_max, device="cuda") >= seq[:, None]
    assert torch.all(w[past] == -1) and torch.all((w - v).abs() <= 2e-4 * v.abs() + 1e-6)


@pytest.mark.parametrize("packed", [False, True])
def test_weights_of_many_short_sequences(lib, packed):
    # more sequences than a block has threads, some invalid: every valid sequence's weights add up to its queries and heads
    B, T_max, q_len = 1500, 200, 2
    dims = dims_of(lib, V3)
    T = torch.randint(2, T_max + 1, (B,), generator=torch.Generator().manual_seed(4))
    T[::89] = 1
    seq = T.to(torch.int32).cuda()
    q = rand(2, B, q_len, 128, 576, dtype=torch.bfloat16, std=0.05)
    lse = torch.zeros(B, q_len, 128, device="cuda")
    if packed:
        cache = torch.randint(0, 256, (B, T_max, 416), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.uint8)
        cache[:, :, 256:288] = 160
        cache[:, :, 288:] = torch.randn(B, T_max, 64, device="cuda").bfloat16().view(torch.uint8)
        lib.attend_packed(dims, q, cache, seq, lse=lse)
    else:
        cache = rand(3, B, T_max, 576, dtype=torch.bfloat16)
        lib.attend_latent_lse(dims, q, cache, seq, lse)
    w = torch.zeros(B, T_max, device="cuda")
    lib.accumulate_weights(dims, q, lse, cache, seq, w)
    assert lib.device_status() == 2
    # each of 256 terms of a sequence's total carries the score's and the exponential's rounding, below 1e-4
    want = torch.where(T.cuda() < q_len, 0.0, 256.0)
    assert torch.all((w.sum(1) - want).abs() <= 256 * 1e-4)
    v = torch.zeros(B, T_max, device="cuda")
    lib.accumulate_weights(dims, q, lse, cache, seq, v, opts=lib.opts(path=2))
    assert lib.device_status() == 2
    assert torch.all((w - v).abs() <= 2e-4 * v + 1e-6)


# ------------------------------------------------------------------ evict

def evict_case(lib, g, T, budget, sink, recent, packed=False, T_max=None, in_place=False, w=None, seed=4, strided=False):
    H, d_c, d_r, _, _, dt = g
    dims = dims_of(lib, g)
    B, T_max = len(T), T_max or max(max(T), 1)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    width = lib.packed_row_bytes(dims) if packed else (d_c + d_r + 7) // 8 * 8
    row = width if packed else d_c + d_r
    raw = torch.randint(0, 256, (B, T_max, width * (1 if packed else dt.itemsize)), generator=gen, device="cuda", dtype=torch.uint8)
    cache = raw if packed else raw.view(dt)
    if strided:
        big = torch.zeros(2 * B, T_max, width + 16, dtype=cache.dtype, device="cuda")
        big[::2, :, :width] = cache
        cache = big[::2, :, :width]
    if w is None:
        w = torch.randint(0, max(2, T_max // 3), (B, T_max), generator=gen, device="cuda").float()  # many equal ones
    seq = i32(*T)
    bits = lambda t: t.contiguous().view(torch.uint8).cpu().numpy()
    src, w0 = bits(cache[:, :, :row]).copy(), w.cpu().numpy().copy()
    kept = torch.full((B, budget), -7, dtype=torch.int32, device="cuda")
    if in_place:
        lib.evict(dims, cache, w, seq, budget, n_sink=sink, n_recent=recent, kept=kept)
        out, ow, n = cache, w, seq
        old_rows, old_w = src, w0
    else:
        T_out = budget + 2
        out = torch.full((B, T_out, width), 3, dtype=cache.dtype, device="cuda")
        ow, n = torch.full((B, T_out), 5.0, device="cuda"), i32(*[-9] * B)
        old_rows, old_w = bits(out[:, :, :row]).copy(), ow.cpu().numpy().copy()
        lib.evict(dims, cache, w, seq, budget, n_sink=sink, n_recent=recent, out=out, out_weights=ow, out_seqlens=n, kept=kept)
        assert np.array_equal(bits(cache[:, :, :row]), src)
        np.testing.assert_array_equal(w.cpu().numpy(), w0)
    bad = any(t < 0 or t > T_max for t in T)
    assert lib.device_status() == (2 if bad else 0)
    got, gw, gk = bits(out[:, :, :row]), ow.cpu().numpy(), kept.cpu().numpy()
    for b, t in enumerate(T):
        want = co.kept_rows(w0[b], t, budget, sink, recent) if 0 <= t <= T_max else np.zeros(0, int)
        k = len(want)
        assert n[b].item() == k
        np.testing.assert_array_equal(gk[b], np.r_[want, np.full(budget - k, -1)])
        np.testing.assert_array_equal(got[b, :k], src[b, want])
        np.testing.assert_array_equal(gw[b, :k], w0[b, want])
        np.testing.assert_array_equal(got[b, k:], old_rows[b, k:])
        np.testing.assert_array_equal(gw[b, k:], old_w[b, k:])


EVICT = [
    ((5,), 1, 0, 0), ((5,), 1, 1, 0), ((5,), 1, 0, 1), ((5, 4, 3, 0), 4, 1, 1), ((100, 33, 32, 31), 32, 4, 8),
    ((700, 2, 699), 350, 0, 350), ((700, 2, 699), 350, 350, 0), ((300,), 299, 3, 5), ((2000, 1999, 77), 60, 4, 16),
    ((9000, 8193, 20), 4500, 4, 512), ((8192, 8191), 1000, 0, 0), ((20000,), 19000, 16, 1000), ((20000, 100), 25000, 4, 4),
    ((50,) * 200, 20, 2, 2), ((-1, 40, 41, 2**31 - 1), 20, 1, 1),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,budget,sink,recent", EVICT)
def test_evict(lib, T, budget, sink, recent, in_place):
    T_max = 40 if -1 in T else None
    evict_case(lib, V3, T, budget, sink, recent, T_max=T_max, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("name", list(GEOMETRIES))
def test_evict_row_widths(lib, name, packed, in_place):
    evict_case(lib, GEOMETRIES[name], (400, 90, 10), 77, 3, 20, packed=packed, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_strided(lib, in_place):
    evict_case(lib, V3, (400, 90, 10), 77, 3, 20, in_place=in_place, strided=True)
    evict_case(lib, V3, (400, 90, 10), 77, 3, 20, packed=True, in_place=in_place, strided=True)


@pytest.mark.parametrize("T", [3000, 9001])
def test_evict_weights_of_every_kind(lib, T):
    # zeros of both signs, negative ones, subnormal ones, infinities, NaN, and all equal
    gen = torch.Generator(device="cuda").manual_seed(1)
    odd = torch.tensor([0.0, -0.0, 1e-42, -1e-42, 2e-42, float("inf"), -float("inf"), float("nan"), 1.0, -1.0, 3e38], device="cuda")
    w = odd[torch.randint(0, len(odd), (1, T), generator=gen, device="cuda")]
    for budget in (100, T // 4, T // 2, T - 1):
        evict_case(lib, TINY, (T,), budget, 2, 30, w=w.clone())
        evict_case(lib, TINY, (T,), budget, 2, 30, w=w.clone(), in_place=True)
    for value in (0.0, float("nan"), 7.0):
        evict_case(lib, TINY, (T,), T // 2, 2, 30, w=torch.full((1, T), value, device="cuda"), in_place=True)


def test_evict_beyond_one_slab(lib):
    # more rows than the selection's registers hold (131072), in and out of place, next to a short sequence
    for in_place in (False, True):
        evict_case(lib, TINY, (300000, 140001, 500), 100000, 16, 1000, in_place=in_place)


def test_evict_many_sequences(lib):
    T = torch.randint(0, 300, (1500,), generator=torch.Generator().manual_seed(5)).tolist()
    evict_case(lib, TINY, tuple(T), 100, 4, 20, T_max=299, in_place=True)


def test_evict_long_in_place(lib):
    # many chunks that wait on one another; the largest and the smallest part of the history kept
    for budget in (3000, 60000, 99000):
        evict_case(lib, V3, (100000, 70000), budget, 16, 1000, in_place=True)


def test_evict_in_a_graph_twice(lib):
    # two captured evictions that share a workspace, replayed, against eager calls
    dims = dims_of(lib, V3)
    B, T_max, budget = 3, 500, 200
    c0 = rand(1, B, T_max, 576, dtype=torch.bfloat16)
    w0 = rand(2, B, T_max).abs()
    ref_c, ref_w, ref_n = c0.clone(), w0.clone(), i32(500, 300, 100)
    lib.evict(dims, ref_c, ref_w, ref_n, budget, 4, 50)
    cs, ws, ns = [torch.empty_like(c0) for _ in range(2)], [torch.empty_like(w0) for _ in range(2)], [i32(0, 0, 0) for _ in range(2)]
    work = torch.empty(lib.evict_workspace_bytes(dims, B, budget), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graphs = []
    for c, w, n in zip(cs, ws, ns):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.evict(dims, c, w, n, budget, 4, 50, workspace=work)
        graphs.append(graph)
    for _ in range(3):
        for c, w, n, graph in zip(cs, ws, ns, graphs):
            c.copy_(c0)
            w.copy_(w0)
            n.copy_(i32(500, 300, 100))
            graph.replay()
    torch.cuda.synchronize()
    for c, w, n in zip(cs, ws, ns):
        assert torch.equal(c, ref_c) and torch.equal(w, ref_w) and torch.equal(n, ref_n)
    assert lib.device_status() == 0


# ------------------------------------------------------------------ together, as they are used

@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("g", [V3, TINY], ids=["v3", "tiny"])
def test_decoding_within_a_budget(lib, g, packed):
    """Prompt, then steps of append, decode, accumulate, evict: every step's output against the fp64 oracle on the rows the
    oracle says are left, at the positions the tokens had."""
    H, d_c, d_r, d_n, d_v, dt = g
    dims = dims_of(lib, g)
    B, prompt, budget, sink, recent, q_len = 2, (150, 90), 128, 4, 32, 2
    T_max = 160
    width = lib.packed_row_bytes(dims) if packed else d_c + d_r
    cache = torch.zeros(B, T_max, width, dtype=torch.uint8 if packed else dt, device="cuda")
    append = lib.append_packed if packed else lib.append_rows
    for b, t in enumerate(prompt):
        append(dims, cache[b:b + 1], rand(70 + b, 1, t, d_c, dtype=dt), rand(80 + b, 1, t, d_r, dtype=dt), i32(0), rows=i32(0))
    rows_n, seen = i32(*prompt), i32(*prompt)
    w = torch.zeros(B, T_max, device="cuda")
    kind = "bf16" if dt == torch.bfloat16 else "f32"
    for step in range(4):
        append(dims, cache, rand(100 + step, B, q_len, d_c, dtype=dt), rand(200 + step, B, q_len, d_r, dtype=dt), seen, rows=rows_n)
        rows_n += q_len
        seen += q_len
        T, S = rows_n.tolist(), seen.tolist()
        stored = stored_rows(lib, dims, cache, T) if packed else [as_f64(cache[b, :t]) for b, t in enumerate(T)]
        ins = decode_inputs(g, B, q_len, seed=300 + 10 * step)
        q_hat = torch.zeros(B, q_len, H, d_c + d_r, dtype=dt, device="cuda")
        lse = torch.zeros(B, q_len, H, device="cuda")
        if packed:
            out = lib.decode_packed(dims, *ins, cache, rows_n, n_seen=seen, q_hat=q_hat, lse=lse)
        else:
            lib.absorb_query(dims, ins[0], ins[1], ins[2], seen, out=q_hat)
            o_lat = lib.attend_latent_lse(dims, q_hat, cache, rows_n, lse)
            out = lib.project_out(dims, o_lat, ins[3])
        from mla_testutil import check_close
        check_close(as_f64(out), decode_reference(g, *ins, stored, T, S, q_len), kind, f"step {step}")
        for b in range(B):
            w[b, T[b] - q_len:T[b]] = 0
        lib.accumulate_weights(dims, q_hat, lse, cache, rows_n, w, prev=w, decay=0.9)
        host_w = w.cpu().numpy().copy()
        lib.evict(dims, cache, w, rows_n, budget, n_sink=sink, n_recent=recent)
        assert lib.device_status() == 0
        for b in range(B):
            keep = co.kept_rows(host_w[b], T[b], budget, sink, recent)
            assert rows_n[b].item() == len(keep)
            now = stored_rows(lib, dims, cache[b:b + 1], [len(keep)])[0] if packed else as_f64(cache[b, :len(keep)])
            np.testing.assert_array_equal(now, stored[b][keep])
            np.testing.assert_array_equal(w[b, :len(keep)].cpu().numpy(), host_w[b, keep])
    assert rows_n[0].item() == budget and lib.device_status() == 0
