"""Calls that the documentation allows at the edges: views of one array, calls from several threads, expired waits of the eviction,
token counts that cannot be, the quantiser at every border."""
import numpy as np
import pytest
import torch

from mla_testutil import as_f64
from oracle import cache_oracle as co
from test_gpu_packed import TINY, V3, attend_case, check_attention, decode_inputs, dims_of, i32, make_cache, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("g", [V3, TINY], ids=["v3", "tiny"])
def test_views_between_each_other(lib, g):
    # earlier and later weights, the cache and where it is cut down to: halves of one array, and columns of one array
    H, d_c, d_r, _, _, dt = g
    dims, T, B, rows, width = dims_of(lib, g), (300, 129), 2, 300, d_c + d_r
    cache, q = rand(1, B, rows, width, dtype=dt), rand(2, B, 1, H, width, dtype=dt, std=0.25)
    lse, prev = rand(3, B, 1, H) + 5, rand(4, B, rows).abs()
    want = lib.accumulate_weights(dims, q, lse, cache, i32(*T), torch.zeros(B, rows, device="cuda"), prev=prev)
    both = torch.zeros(B, 2, rows, device="cuda")
    both[:, 0] = prev
    lib.accumulate_weights(dims, q, lse, cache, i32(*T), both[:, 1], prev=both[:, 0])
    assert torch.equal(both[:, 1], want) and torch.equal(both[:, 0], prev)

    budget = 100
    out, ow, n = torch.zeros(B, budget, width, dtype=dt, device="cuda"), torch.zeros(B, budget, device="cuda"), i32(0, 0)
    lib.evict(dims, cache, want, i32(*T), budget, 3, 20, out=out, out_weights=ow, out_seqlens=n)
    half = torch.zeros(B, 2, rows, width, dtype=dt, device="cuda")
    beside = torch.zeros(B, rows, 2, width, dtype=dt, device="cuda")
    for one in (half, beside):
        a, b = (one[:, 0], one[:, 1]) if one is half else (one[:, :, 0], one[:, :, 1])
        a.copy_(cache)
        both[:, 0], m = want, i32(0, 0)
        both[:, 1] = 0
        lib.evict(dims, a, both[:, 0], i32(*T), budget, 3, 20, out=b, out_weights=both[:, 1], out_seqlens=m)
        assert torch.equal(a, cache) and torch.equal(b[:, :budget], out) and not b[:, budget:].any()
        assert torch.equal(both[:, 0], want) and torch.equal(both[:, 1, :budget], ow) and torch.equal(m, n)
    assert lib.device_status() == 0


def test_largest_options_of_the_split(lib):
    # a share that no batch fills is one cluster's; a charge far above the tiles only moves the cuts
    T, q_len = (900, 77, 333), 2
    dims = dims_of(lib, V3)
    full = rand(9, 3, 900, 576, dtype=torch.bfloat16)
    _, cache, rows, q, one, _ = attend_case(lib, V3, T, q_len, lib.opts(num_pairs=q_len))
    for tiles in (2 ** 31 - 1, 2 ** 25):
        opts = lib.opts(min_tiles=tiles)
        assert torch.equal(lib.attend_packed(dims, q, cache, i32(*T), opts=opts), one)
        assert torch.equal(lib.attend_latent(dims, q, full, i32(*T), opts=opts),
                           lib.attend_latent(dims, q, full, i32(*T), opts=lib.opts(num_pairs=q_len)))
    lse = torch.zeros(3, q_len, 128, device="cuda")
    for charge in (1000, 2 ** 22):
        o = lib.attend_packed(dims, q, cache, i32(*T), lse=lse, opts=lib.opts(overhead_tiles=charge))
        check_attention(o, lse, q, rows, T, q_len, V3, 192 ** -0.5, f"charge {charge}")
    assert lib.device_status() == 0


# ------------------------------------------------------------------ the eviction's waits

@pytest.mark.parametrize("packed", [False, True])
def test_evict_expired_wait(lib, packed):
    # the second part of every sequence does not say that its rows are loaded: the third, which moves over them, gives up after
    # 20 ms; the call reports it and ends, and the next one with the same workspace is right
    dims, B, rows, budget = dims_of(lib, V3), 3, 5000, 4000
    width = 416 if packed else 576
    gen = torch.Generator(device="cuda").manual_seed(1)
    raw = torch.randint(0, 256, (B, rows, width * (1 if packed else 2)), generator=gen, device="cuda", dtype=torch.uint8)
    cache = raw if packed else raw.view(torch.bfloat16)
    weights, T = rand(2, B, rows).abs(), (5000, 4500, 4000)
    bits = lambda t: t.view(torch.uint8)
    work = torch.empty(lib.evict_workspace_bytes(dims, B, budget, packed), dtype=torch.uint8, device="cuda")

    def run(**o):
        c, w, n = cache.clone(), weights.clone(), i32(*T)
        lib.evict(dims, c, w, n, budget, 4, 500, workspace=work, opts=lib.opts(**o) if o else None)
        return c, w, n, lib.device_status()
    c, w, n, status = run()
    assert status == 0 and n.tolist() == [4000] * 3
    *_, status = run(wait_limit_ns=20_000_000, withhold_tile=2)
    assert status == 4
    for o in ({}, dict(wait_limit_ns=20_000_000)):
        c2, w2, n2, status = run(**o)
        assert status == 0 and torch.equal(bits(c2), bits(c)) and torch.equal(w2, w) and torch.equal(n2, n)
    # apart from the cache nothing waits
    out, ow, on = torch.zeros_like(cache), torch.zeros_like(weights), i32(0, 0, 0)
    lib.evict(dims, cache, weights, i32(*T), budget, 4, 500, out=out, out_weights=ow, out_seqlens=on, workspace=work,
              opts=lib.opts(wait_limit_ns=1, withhold_tile=2))
    assert lib.device_status() == 0 and torch.equal(on, n)
    assert torch.equal(bits(out[:, :budget].contiguous()), bits(c[:, :budget].contiguous()))


# ------------------------------------------------------------------ several threads

def test_first_calls_of_several_threads_at_once(lib, tmp_path):
    # a library of its own (a copy of the file), so that what is found out at the first call is found out by all threads at once
    import shutil
    import threading
    from latent_compressed_attention_absorbed_b200 import binding
    T, q_len = (700, 333), 2
    dims = dims_of(lib, V3)
    packed, _ = make_cache(lib, dims, V3, T)
    full, q = rand(9, 2, 700, 576, dtype=torch.bfloat16), rand(3, 2, q_len, 128, 576, dtype=torch.bfloat16, std=0.25)
    lse, seq = rand(8, 2, q_len, 128) + 5, i32(*T)

    def calls(one, stream):
        zeros = lambda: torch.zeros(2, 700, device="cuda")
        with torch.cuda.stream(stream):
            w = [one.accumulate_weights(dims, q, lse, c, seq, zeros()) for c in (full, packed)]
            z = torch.zeros_like(lse)
            o = [one.attend_packed(dims, q, packed, seq), one.attend_latent_lse(dims, q, full, seq, z), z]
            c, n = full.clone(), seq.clone()
            one.evict(dims, c, w[0], n, 100, 4, 20)
        return w + o + [c[0, :100], n]
    ref = calls(lib, torch.cuda.current_stream())
    torch.cuda.synchronize()
    for attempt in range(3):
        copy = tmp_path / f"copy{attempt}.so"
        shutil.copy(lib.path, copy)
        fresh = binding.Library(str(copy))
        gate, got, streams = threading.Barrier(8), [None] * 8, [torch.cuda.Stream() for _ in range(8)]

        def work(i):
            gate.wait()
            got[i] = calls(fresh, streams[i])
        threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        for one in got:
            assert one is not None and all(torch.equal(a, b) for a, b in zip(one, ref))
        assert fresh.device_status() == 0


# ------------------------------------------------------------------ token counts

@pytest.mark.parametrize("path", [0, 2])
def test_token_counts_below_the_queries_are_flagged(lib, path):
    T, q_len = (300, 40, 64), 2
    dims, opts = dims_of(lib, V3), lib.opts(path=path)
    cache, _ = make_cache(lib, dims, V3, T)
    ins = decode_inputs(V3, 3, q_len)
    seen = (300, 1000, 2)                    # (the smallest that can be)
    ref = lib.decode_packed(dims, *ins, cache, i32(*T), n_seen=i32(*seen), opts=opts)
    assert lib.device_status() == 0
    for bad in (1, 0, -5, -2 ** 31):
        out = lib.decode_packed(dims, *ins, cache, i32(*T), n_seen=i32(300, bad, 2), opts=opts)
        assert lib.device_status() == 2
        assert torch.equal(out[0], ref[0]) and torch.equal(out[2], ref[2])


# ------------------------------------------------------------------ the bf16 quantiser at every border

def test_quantisation_of_every_bf16_latent_at_every_scale(lib):
    # bf16 latents are quantised by arithmetic of their own.  For each of the 256 scales s: every bf16 value from s / 5 to 7 s, of both
    # signs (all halves of a step that there are, and the numbers on both sides), in groups whose largest is 7 s
    dims = dims_of(lib, (1, 512, 2, 4, 4, torch.bfloat16))
    every = (np.arange(0x4653, dtype=np.uint32) << 16).view(np.float32)     # 0 .. 13440
    groups = []
    for s in co.SCALES:
        v = every[(every >= s / 5) & (every <= 7 * s)]
        v = np.r_[0.0, every[1], v, -v, -every[1]]
        v = np.r_[v, np.zeros(-len(v) % 15)].reshape(-1, 15)
        groups.append(np.c_[np.full(len(v), 7 * s), v])
    x = np.concatenate(groups)
    # and every bf16 magnitude as the largest of its group, with values below it
    x = np.concatenate([x, every[:, None] * np.r_[1.0, -0.5, np.zeros(14)]])
    x = np.r_[x, np.zeros((-len(x) % 32, 16))].reshape(1, -1, 512)
    c = torch.from_numpy(x).to(torch.bfloat16).cuda()
    n = c.shape[1]
    cache = torch.zeros(1, n, lib.packed_row_bytes(dims), dtype=torch.uint8, device="cuda")
    lib.append_packed(dims, cache, c, torch.zeros(1, n, 2, dtype=torch.bfloat16, device="cuda"), i32(0))
    assert lib.device_status() == 0
    q, code = co.quantise(as_f64(c)[0])
    raw = cache[0].cpu().numpy()
    np.testing.assert_array_equal(raw[:, 256:288], code)
    np.testing.assert_array_equal(co.unpack_latents(raw, 512), co.quantised(as_f64(c)[0]))
    np.testing.assert_array_equal(as_f64(lib.load_packed(dims, cache, i32(0), n))[0, :, :512], co.quantised(as_f64(c)[0]))
    word = raw[:, :256].copy().view(np.uint32)
    for e in range(8):                       # codes, too: 0 has one code at any scale
        np.testing.assert_array_equal((word >> (4 * (e // 2) + 16 * (e % 2)) & 15).astype(int) - 8, q[:, e::8])


# ------------------------------------------------------------------ a bound on the lengths as T_max

@pytest.mark.parametrize("packed", [False, True])
def test_a_view_of_the_first_rows(lib, packed):
    # the calls choose their split by T_max: a long cache seen through a view gives the bits of a cache of that length
    T, q_len, bound, cap = (600, 77), 16, 640, 20000
    dims = dims_of(lib, V3)
    width, dt = (416, torch.uint8) if packed else (576, torch.bfloat16)
    long = torch.full((2, cap, width), 0xFF if packed else float("nan"), dtype=dt, device="cuda")
    long[:, :bound] = make_cache(lib, dims, V3, T, T_max=bound)[0] if packed else rand(9, 2, bound, 576, dtype=dt)
    tight, view = long[:, :bound].contiguous(), long[:, :bound]
    q, lse = rand(3, 2, q_len, 128, 576, dtype=torch.bfloat16, std=0.25), rand(8, 2, q_len, 128) + 5
    want = lib.accumulate_weights(dims, q, lse, tight, i32(*T), torch.zeros(2, bound, device="cuda"))
    w = torch.full((2, cap), -1.0, device="cuda")
    lib.accumulate_weights(dims, q, lse, view, i32(*T), w)
    assert all(torch.equal(w[b, :t], want[b, :t]) and torch.all(w[b, t:] == -1) for b, t in enumerate(T))
    n, m = i32(*T), i32(*T)
    lib.evict(dims, tight, want, n, 200, 4, 50)
    behind = long[:, bound:].view(torch.uint8).clone()
    lib.evict(dims, view, w, m, 200, 4, 50)
    assert torch.equal(n, m) and torch.equal(tight.view(torch.uint8), view.contiguous().view(torch.uint8))
    assert all(torch.equal(w[b, :t], want[b, :t]) for b, t in enumerate(T)) and torch.equal(long[:, bound:].view(torch.uint8), behind)
    assert lib.device_status() == 0
    lib.evict(dims, view, w, i32(bound + 1, 100), 200)   # a length past the bound
    assert lib.device_status() == 2
