"""Operators on the compressed cache that are measured one by one: their cases, their plain forms and the calls a user makes.

  append   new tokens quantised into the 4-bit cache and read back as the rows it holds
  attend   one step of latent attention over the 4-bit cache, with the log-sum-exp of every score row
  weights  the attention weight every cached row received in a step, added to its running sum
  evict    a cache cut down to a budget of rows: the first ones, the latest ones, and those with the most weight between

A row of the 4-bit cache stands for 512 latent values and a 64-wide rotated RoPE key in 416 bytes:
  bytes   0..255  latent codes, 4 bits each, n = q + 8 with q in -7..7: in 32-bit word w, element 8w + 2j sits at bit 4j
                  and element 8w + 2j + 1 at bit 16 + 4j (j = 0..3)
  bytes 256..287  one scale for each 16 latents, e * 8 + m, which stands for 2^(e - 21) * (1 + m / 8)
  bytes 288..415  the RoPE key in bf16
The value of a latent is q * scale.  The scale of a group is the smallest one that is not below max|x| / 7.

Where `own` is false, run() uses elementary torch operations in 32 bits (64 for angles and next to a rounding border).
"""
import math
import random

import torch

own = False

H, D_C, D_R = 128, 512, 64
ROW = D_C + D_R
PACKED = 416
GROUP = 16
SCALE = 1.0 / math.sqrt(128 + 64)
ROPE_BASE = 10000.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a batch: one new token for each of 64 sequences
        dict(name="append step b64", op="append", B=64, n_tok=1, first=4095),
        # prompts of four sequences written at once
        dict(name="append prompt 4x4093", op="append", B=4, n_tok=4093, first=0),
        # one sequence, one query: latency
        dict(name="attend b1", op="attend", B=1, q_len=1, T_lo=4096, T_hi=4096, lengths=0),
        # a batch of equal lengths
        dict(name="attend b64", op="attend", B=64, q_len=1, T_lo=4096, T_hi=4096, lengths=0),
        # few long histories
        dict(name="attend long", op="attend", B=8, q_len=1, T_lo=131072, T_hi=131072, lengths=0),
        # ragged lengths, main token and draft token
        dict(name="attend ragged verify", op="attend", B=128, q_len=2, T_lo=2048, T_hi=16384, lengths=0),
        # running weights next to a decode of one sequence
        dict(name="weights b1", op="weights", packed=False, B=1, q_len=1, T_lo=4001, T_hi=4001, lengths=0),
        # few long histories in the full-width cache
        dict(name="weights long", op="weights", packed=False, B=8, q_len=1, T_lo=65536, T_hi=131072, lengths=1),
        # ragged lengths and two queries over the 4-bit cache
        dict(name="weights packed verify", op="weights", packed=True, B=64, q_len=2, T_lo=2048, T_hi=16384, lengths=2),
        # one sequence that has just passed its budget
        dict(name="evict b1", op="evict", B=1, budget=4000, sink=4, recent=256, T_lo=4096, T_hi=4096, lengths=0),
        # a batch halved; a few of its sequences are still below the budget
        dict(name="evict b64", op="evict", B=64, budget=2048, sink=4, recent=512, T_lo=1500, T_hi=8192, lengths=3),
        # long histories cut to a quarter
        dict(name="evict long", op="evict", B=8, budget=32768, sink=16, recent=4096, T_lo=131072, T_hi=131072, lengths=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "weights", "weights", "evict"))
    if op == "append":
        B = _log(rng, 1, 128)
        return dict(op=op, B=B, n_tok=_log(rng, 1, max(1, 16384 // B)), first=rng.randrange(0, 100000))
    B = _log(rng, 1, 192)
    # at most a million rows in all, and 131072 in one sequence
    T_hi = _log(rng, 17, min(131072, 1048576 // B))
    T_lo = rng.choice((T_hi, max(17, T_hi // 8)))
    if op == "evict":
        budget = max(1, int(T_hi * rng.uniform(0.1, 0.95)))
        sink = min(budget, rng.choice((0, 1, 4, 16)))
        recent = int((budget - sink) * rng.choice((0.0, 0.1, 0.5, 1.0)))
        return dict(op=op, B=B, budget=budget, sink=sink, recent=recent, T_lo=T_lo, T_hi=T_hi, lengths=rng.randrange(1000))
    q_len = rng.choice((1, 1, 1, 2, 2, 3, 4, 8, 16)) if B * T_hi <= 65536 else rng.choice((1, 1, 2))
    c = dict(op=op, B=B, q_len=q_len, T_lo=T_lo, T_hi=T_hi, lengths=rng.randrange(1000))
    if op == "weights":
        c["packed"] = rng.random() < 0.5
    return c


def _lengths(case):
    r = random.Random(case["lengths"])
    return [r.randint(case["T_lo"], case["T_hi"]) for _ in range(case["B"])]


def work(case):
    if case["op"] == "append":
        n = case["B"] * case["n_tok"]
        return {"bytes": n * 2 * (2 * ROW + PACKED) + 4 * case["B"], "flops": 0}
    T = _lengths(case)
    if case["op"] == "evict":
        kept = sum(min(t, case["budget"]) for t in T)
        return {"bytes": sum(T) * 4 + kept * (2 * 2 * ROW + 4) + case["B"] * (case["budget"] * 4 + 8), "flops": 0}
    q_len, tokens = case["q_len"], case["B"] * case["q_len"]
    pairs = sum(t - q_len + 1 + i for t in T for i in range(q_len))
    row = PACKED if case["op"] == "attend" or case["packed"] else 2 * ROW
    read = sum(T) * row + tokens * H * ROW * 2 + case["B"] * 4
    if case["op"] == "attend":
        return {"bytes": read + tokens * H * (D_C * 2 + 4), "flops": 2 * H * pairs * (ROW + D_C)}
    return {"bytes": read + tokens * H * 4 + sum(T) * 8, "flops": 2 * H * pairs * ROW}


# ------------------------------------------------------------------ inputs

def _normal(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda") * std


def _pack_rows(c, k):
    """Packed rows of latents c [n, 512] and rotated keys k [n, 64]: inputs only, near enough to the nearest codes."""
    x = c.view(-1, D_C // GROUP, GROUP)
    code = (torch.log2((x.abs().amax(-1) / 7).clamp_min(2.0 ** -21)) + 21).mul(8).ceil().clamp(0, 255)
    code = code.to(torch.int32)
    s = torch.exp2((code // 8 - 21).float()) * (1 + (code % 8).float() / 8)
    n = ((x / s[..., None]).round().clamp(-7, 7) + 8).to(torch.int32).view(-1, D_C // 8, 4, 2)
    return _bytes_of(n, code, k)


def _bytes_of(n, code, k):
    """n [..., 64, 4, 2] codes, code [..., 32] scales, k [..., 64] keys -> [..., 416] bytes."""
    e, o = n[..., 0], n[..., 1]
    b = torch.stack((e[..., 0] | e[..., 1] << 4, e[..., 2] | e[..., 3] << 4, o[..., 0] | o[..., 1] << 4, o[..., 2] | o[..., 3] << 4), -1)
    return torch.cat((b.flatten(-2).to(torch.uint8), code.to(torch.uint8), k.to(torch.bfloat16).contiguous().view(torch.uint8)), -1)


def _lse_of(q, rows, n_keys):
    """Log-sum-exp of the scores of q [q_len, 128, 576] against rows [T, 576], for inputs."""
    s = (q.float().flatten(0, 1) @ rows.float().t()).mul_(SCALE).view(q.shape[0], H, -1)
    t = torch.arange(rows.shape[0], device="cuda")
    for i, n in enumerate(n_keys):
        s[i].masked_fill_(t >= n, -math.inf)
    return torch.logsumexp(s, -1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    B = case["B"]
    if case["op"] == "append":
        n = case["n_tok"]
        st = dict(op="append", n_tok=n)
        st["c_kv"] = _normal(gen, B, n, D_C).bfloat16()
        st["k_rope"] = _normal(gen, B, n, D_R).bfloat16()
        # positions differ from sequence to sequence; the cache holds the new rows and a few before them
        st["pos"] = (case["first"] + torch.randint(0, 64, (B,), generator=gen, device="cuda")).to(torch.int32)
        st["row"] = torch.randint(0, 8, (B,), generator=gen, device="cuda").to(torch.int32)
        st["cache"] = torch.zeros(B, n + 8, PACKED, dtype=torch.uint8, device="cuda")
        return st
    lengths = _lengths(case)
    T_max = max(lengths)
    st = dict(op=case["op"], seqlens=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    packed = case["op"] == "attend" or bool(case.get("packed"))
    if packed:
        cache = torch.zeros(B, T_max, PACKED, dtype=torch.uint8, device="cuda")
    else:
        cache = torch.zeros(B, T_max, ROW, dtype=torch.bfloat16, device="cuda")
    for b, T in enumerate(lengths):
        if packed:
            cache[b, :T] = _pack_rows(_normal(gen, T, D_C), _normal(gen, T, D_R))
        else:
            cache[b, :T] = _normal(gen, T, ROW).bfloat16()
    st["cache"] = cache
    if case["op"] == "evict":
        # accumulated weights: a heavy tail, rounded so that equal ones occur, and rows that never got any
        w = torch.exp(1.5 * _normal(gen, B, T_max)).bfloat16().float()
        st["weights"] = torch.where(torch.rand(B, T_max, generator=gen, device="cuda") < 0.05, 0.0, w)
        st["budget"], st["sink"], st["recent"] = case["budget"], case["sink"], case["recent"]
        st["to_cache"] = torch.zeros(B, case["budget"], ROW, dtype=torch.bfloat16, device="cuda")
        st["to_weights"] = torch.zeros(B, case["budget"], device="cuda")
        st["to_seqlens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        st["kept"] = torch.zeros(B, case["budget"], dtype=torch.int32, device="cuda")
        return st
    q_len = case["q_len"]
    # folded queries: 128 products with weights of std 0.02, then the rotated RoPE part
    st["q_hat"] = torch.cat((_normal(gen, B, q_len, H, D_C, std=0.02 * math.sqrt(128)), _normal(gen, B, q_len, H, D_R)), -1).bfloat16()
    st["lse"] = torch.zeros(B, q_len, H, device="cuda")
    if case["op"] == "weights":
        for b, T in enumerate(lengths):
            rows = _values(cache[b, :T]) if packed else cache[b, :T]
            st["lse"][b] = _lse_of(st["q_hat"][b], rows, [T - q_len + 1 + i for i in range(q_len)])
        st["sums"] = torch.rand(B, T_max, generator=gen, device="cuda")
        st["to_sums"] = torch.zeros(B, T_max, device="cuda")
    else:
        st["o_lat"] = torch.zeros(B, q_len, H, D_C, dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms

def _values(cache):
    """[..., 576] values in fp32 of packed rows [..., 416]."""
    b = cache[..., :D_C // 2].unflatten(-1, (D_C // 8, 2, 2))  # word, parity of the element, byte within the half word
    n = torch.stack((b & 15, b >> 4), -1).flatten(-2).transpose(-1, -2)  # word, j, parity
    code = cache[..., D_C // 2:D_C // 2 + D_C // GROUP].to(torch.int32)
    s = torch.exp2((code // 8 - 21).float()) * (1 + (code % 8).float() / 8)
    c = (n.flatten(-3).to(torch.float32) - 8).unflatten(-1, (D_C // GROUP, GROUP)) * s[..., None]
    k = cache[..., D_C // 2 + D_C // GROUP:].contiguous().view(torch.bfloat16)
    return torch.cat((c.flatten(-2), k.float()), -1)


def _plain_append(st):
    c = st["c_kv"].double().unflatten(-1, (D_C // GROUP, GROUP))
    code = torch.arange(256, device=c.device)
    table = torch.exp2((code // 8 - 21).double()) * (1 + (code % 8).double() / 8)
    code = torch.searchsorted(7 * table, c.abs().amax(-1)).clamp_max(255)
    n = (c / table[code][..., None]).round().clamp(-7, 7).to(torch.int32) + 8
    tok = torch.arange(st["n_tok"], device=c.device)
    freq = ROPE_BASE ** (-torch.arange(0, D_R, 2, device=c.device).double() / D_R)
    a = (st["pos"].double()[:, None] + tok)[..., None] * freq
    k = st["k_rope"].float().unflatten(-1, (D_R // 2, 2))
    cos, sin = a.cos().float(), a.sin().float()
    k = torch.stack((k[..., 0] * cos - k[..., 1] * sin, k[..., 0] * sin + k[..., 1] * cos), -1).flatten(-2)
    rows = _bytes_of(n.flatten(-2).unflatten(-1, (D_C // 8, 4, 2)), code, k)
    at = (st["row"].long()[:, None] + tok)[..., None].expand(-1, -1, PACKED)
    st["cache"].scatter_(1, at, rows)
    return {"rows": _values(st["cache"].gather(1, at)).bfloat16()}


def _visible(st, q_len):
    """[B, q_len, 1, T]: whether query i sees row t."""
    t = torch.arange(st["cache"].shape[1], device="cuda")
    i = torch.arange(q_len, device="cuda")
    return t < (st["seqlens"][:, None] - q_len + 1 + i)[:, :, None, None]


def _scores(st, rows):
    q = st["q_hat"]
    s = torch.matmul(q.float().flatten(1, 2), rows.transpose(1, 2)).mul_(SCALE)
    return s.unflatten(1, (q.shape[1], H))


def _plain_attend(st):
    rows = _values(st["cache"])
    s = _scores(st, rows).masked_fill_(~_visible(st, st["q_hat"].shape[1]), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(1, 2), rows[..., :D_C]).unflatten(1, p.shape[1:3]) / total
    return {"o_lat": o.bfloat16(), "lse": (m + total.log())[..., 0]}


def _plain_weights(st):
    rows = _values(st["cache"]) if st["cache"].dtype == torch.uint8 else st["cache"].float()
    p = _scores(st, rows).sub_(st["lse"][..., None]).exp_()
    w = p.masked_fill_(~_visible(st, st["q_hat"].shape[1]), 0.0).sum((1, 2))
    t = torch.arange(w.shape[1], device=w.device)
    return {"sums": torch.where(t < st["seqlens"][:, None], st["sums"] + w, st["to_sums"])}


def _plain_evict(st):
    T, w, budget = st["seqlens"].long()[:, None], st["weights"], st["budget"]
    t = torch.arange(w.shape[1], device=w.device)
    safe = (t < st["sink"]) | (t >= T - st["recent"])
    rank = torch.where(t >= T, -math.inf, torch.where(safe, math.inf, w))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :budget]
    order = torch.where(order < T, order, w.shape[1]).sort(dim=1).values
    order = torch.nn.functional.pad(order, (0, budget - order.shape[1]), value=w.shape[1])
    there = order < w.shape[1]
    at = torch.where(there, order, 0)
    rows = st["cache"].gather(1, at[..., None].expand(-1, -1, ROW))
    return {"rows": torch.where(there[..., None], rows, st["to_cache"]), "weights": torch.where(there, w.gather(1, at), st["to_weights"]),
            "kept": torch.where(there, order, -1).to(torch.int32), "seqlens": there.sum(1).to(torch.int32)}


# ------------------------------------------------------------------ the framework's calls

_held = []


def _library():
    if not _held:
        from latent_compressed_attention_absorbed_b200 import binding
        lib = binding.load()
        _held.extend((lib, lib.dims(H, D_C, D_R, 128, 128, torch.bfloat16, ROPE_BASE)))
    return _held


def _own(st):
    lib, dims = _library()
    if st["op"] == "append":
        lib.append_packed(dims, st["cache"], st["c_kv"], st["k_rope"], st["pos"], rows=st["row"])
        return {"rows": lib.load_packed(dims, st["cache"], st["row"], st["n_tok"])}
    if st["op"] == "attend":
        if "workspace" not in st:
            n = lib.packed_workspace_bytes(dims, st["q_hat"].shape[0], st["q_hat"].shape[1])
            st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        lib.attend_packed(dims, st["q_hat"], st["cache"], st["seqlens"], out=st["o_lat"], lse=st["lse"], workspace=st["workspace"])
        return {"o_lat": st["o_lat"], "lse": st["lse"]}
    if st["op"] == "weights":
        lib.accumulate_weights(dims, st["q_hat"], st["lse"], st["cache"], st["seqlens"], st["to_sums"], prev=st["sums"])
        return {"sums": st["to_sums"]}
    if "workspace" not in st:
        n = lib.evict_workspace_bytes(dims, st["cache"].shape[0], st["budget"])
        st["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    lib.evict(dims, st["cache"], st["weights"], st["seqlens"], st["budget"], n_sink=st["sink"], n_recent=st["recent"], out=st["to_cache"],
              out_weights=st["to_weights"], out_seqlens=st["to_seqlens"], kept=st["kept"], workspace=st["workspace"])
    return {"rows": st["to_cache"], "weights": st["to_weights"], "kept": st["kept"], "seqlens": st["to_seqlens"]}


def run(state):
    if own:
        return _own(state)
    plain = {"append": _plain_append, "attend": _plain_attend, "weights": _plain_weights, "evict": _plain_evict}
    return plain[state["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rows(cache):
    """Values [T, 576] in fp64 of the packed rows of one sequence, from the layout of a row."""
    word = cache[:, :256].contiguous().view(torch.int32).long() & 0xFFFFFFFF
    out = torch.empty(cache.shape[0], ROW, dtype=torch.float64, device=cache.device)
    scale = cache[:, 256:288].double()
    scale = 2.0 ** (torch.floor(scale / 8) - 21) * (8 + scale % 8) / 8
    for e in range(8):
        out[:, e:D_C:8] = ((word >> (4 * (e // 2) + 16 * (e % 2))) & 15).double() - 8
    out[:, :D_C] *= scale.repeat_interleave(GROUP, dim=1)
    out[:, D_C:] = cache[:, 288:].contiguous().view(torch.bfloat16).double()
    return out


def exact(case, seed):
    st = prepare(case, seed)
    B = case["B"]
    if case["op"] == "append":
        x = st["c_kv"].double().view(-1, GROUP)
        top = x.abs().amax(1) / 7
        e = torch.floor(torch.log2(top)).clamp(-21, 10)
        e = e - (2.0 ** e > top).double()  # the power of two at or below the quotient
        e = e.clamp(-21, 10)
        s = (2.0 ** e * torch.ceil((top / 2.0 ** e * 8)).clamp(8, 16) / 8)[:, None]
        low = torch.floor(x / s)
        rest = x - low * s
        up = (rest * 2 > s) | ((rest * 2 == s) & (low % 2 != 0))
        lat = ((low + up.double()) * s).view(B, -1, D_C)
        z = torch.view_as_complex(st["k_rope"].double().view(B, -1, D_R // 2, 2).contiguous())
        p = st["pos"].double().view(B, 1, 1) + torch.arange(case["n_tok"], device="cuda").double().view(1, -1, 1)
        turn = p * torch.exp(-math.log(ROPE_BASE) * torch.arange(D_R // 2, device="cuda").double() / (D_R // 2))
        key = torch.view_as_real(z * torch.polar(torch.ones_like(turn), turn)).flatten(-2)
        return {"rows": torch.cat((lat, key), -1)}
    T = _lengths(case)
    if case["op"] == "evict":
        rows, sums = st["to_cache"].double(), st["to_weights"].double()
        for b in range(B):
            w = st["weights"][b].tolist()
            middle = range(min(case["sink"], T[b]), max(case["sink"], T[b] - case["recent"]))
            room = case["budget"] - case["sink"] - case["recent"]
            if T[b] <= case["budget"]:
                keep = list(range(T[b]))
            else:
                best = sorted(middle, key=lambda t: (-w[t], t))[:room]
                keep = list(range(case["sink"])) + sorted(best) + list(range(T[b] - case["recent"], T[b]))
            at = torch.tensor(keep, device="cuda")
            rows[b, :len(keep)] = st["cache"][b, at].double()
            sums[b, :len(keep)] = st["weights"][b, at].double()
        return {"rows": rows, "weights": sums, "kept": None, "seqlens": None}
    q_len = case["q_len"]
    o, lse = [], []
    sums = st["to_sums"].double() if case["op"] == "weights" else None
    for b in range(B):
        rows = st["cache"][b, :T[b]]
        rows = _exact_rows(rows) if rows.dtype == torch.uint8 else rows.double()
        total = 0
        for i in range(q_len):
            seen = rows[:T[b] - q_len + 1 + i]
            s = (st["q_hat"][b, i].double() @ seen.T) / math.sqrt(192.0)
            if sums is None:
                z = torch.logsumexp(s, 1)
                o.append(torch.softmax(s, 1) @ seen[:, :D_C])
                lse.append(z)
            else:
                w = torch.exp(s - st["lse"][b, i].double()[:, None]).sum(0)
                total = total + torch.nn.functional.pad(w, (0, T[b] - w.shape[0]))
        if sums is not None:
            sums[b, :T[b]] = st["sums"][b, :T[b]].double() + total
    if sums is not None:
        return {"sums": sums}
    return {"o_lat": torch.stack(o).view(B, q_len, H, D_C), "lse": torch.stack(lse).view(B, q_len, H)}
