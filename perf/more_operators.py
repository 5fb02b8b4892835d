"""Measured cases of the operators around a long cache: rotary positions (with
their gradients, and as queries are rotated and keys and values go into a paged
16-bit cache), attention of a chunk of new tokens over such a cache, the
attention weight that every cached key has received, and eviction of the keys
that received least.

Each case is a dict of plain values. ``prepare`` draws what a program holds
before the call, ``run`` makes one pass (the library's entry points where
``own`` is true, elementary torch operations otherwise, in 32 bits, angles in
64), ``exact`` gives the same outputs from the definitions in 64 bits.

Rotary positions: pair i of the first ``rot`` columns of a row is turned by the
angle position * inv_freq[i] and multiplied by ``mscale``; a pair is columns i
and i + rot / 2 (half layout) or 2 i and 2 i + 1 (interleaved). Columns from
``rot`` on stay.

Chunk attention: the last query of a sequence is at its last key, query t sees
key j if j <= t's position and (that is less than ``window`` away, or window is
0, or j < sinks). Weight of a key: the sum of its softmax weights over the
chunk's queries and the query heads that read its key head. Eviction keeps the
first ``sinks`` and the last ``recent`` keys of a sequence and those of greatest
weight between them, ``keep`` in all, ties to the earlier key, in their order.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # a training step's queries and keys, 16 packed sequences of 64 to 2048 tokens: rotated, and their gradients
        {"name": "rope_train_packed", "op": "rope", "B": 16, "lo": 64, "hi": 2048, "lens_seed": 5, "H": 32, "Hkv": 8,
         "D": 128, "dtype": "bf16", "rot": 128, "interleaved": False, "scaling": "none"},
        # the same of a small model: dense, an odd length, half of each head rotated, neighbouring columns paired
        {"name": "rope_dense_odd", "op": "rope", "B": 2, "S": 777, "H": 6, "Hkv": 2, "D": 64, "dtype": "fp16",
         "rot": 32, "interleaved": True, "scaling": "linear"},
        # one new token of each of 64 sequences: queries rotated, keys and values into the cache
        {"name": "write_step", "op": "write", "B": 64, "lo": 1, "hi": 1, "lens_seed": 8, "start_hi": 4000, "shift": 0,
         "H": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "block": 16, "rot": 128, "interleaved": False,
         "scaling": "none"},
        # chunks of 16 prompts, 64 to 2048 tokens, far into a long context: frequencies scaled by parts, positions
        # ahead of the cache's (it has been evicted from)
        {"name": "write_prompts", "op": "write", "B": 16, "lo": 64, "hi": 2048, "lens_seed": 5, "start_hi": 2000,
         "shift": 100000, "H": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "block": 16, "rot": 128,
         "interleaved": False, "scaling": "parts"},
        # a 2048-token chunk of one long prompt behind 30000 cached keys
        {"name": "chunk_prefill", "op": "chunk", "B": 1, "lo": 2048, "hi": 2048, "pre_lo": 30000, "pre_hi": 30000,
         "lens_seed": 11, "H": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "block": 16, "window": 0, "sinks": 0},
        # a serving batch: chunks of 1 to 512 tokens of 16 conversations of up to 8192 keys
        {"name": "chunk_batch", "op": "chunk", "B": 16, "lo": 1, "hi": 512, "pre_lo": 0, "pre_hi": 7680,
         "lens_seed": 12, "H": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "block": 16, "window": 0, "sinks": 0},
        # five drafted tokens of each of 16 conversations are checked
        {"name": "chunk_draft", "op": "chunk", "B": 16, "lo": 5, "hi": 5, "pre_lo": 4100, "pre_hi": 8192,
         "lens_seed": 13, "H": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "block": 16, "window": 0, "sinks": 0},
        # two short chunks, seven query heads to a key head, a window and sinks: latency
        {"name": "chunk_short", "op": "chunk", "B": 2, "lo": 33, "hi": 100, "pre_lo": 200, "pre_hi": 700,
         "lens_seed": 14, "H": 14, "Hkv": 2, "D": 64, "dtype": "fp16", "block": 32, "window": 256, "sinks": 4},
        # what the last 512 tokens of four long prompts gave to every key
        {"name": "weights_chunk", "op": "weights", "B": 4, "lo": 512, "hi": 512, "pre_lo": 8192, "pre_hi": 16384,
         "lens_seed": 15, "H": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "block": 16, "window": 0, "sinks": 0},
        # what one generated token of each of 16 conversations gave
        {"name": "weights_step", "op": "weights", "B": 16, "lo": 1, "hi": 1, "pre_lo": 4100, "pre_hi": 8192,
         "lens_seed": 16, "H": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "block": 16, "window": 0, "sinks": 0},
        # four long caches down to 4096 keys each
        {"name": "evict_long", "op": "evict", "B": 4, "lo": 16384, "hi": 32768, "lens_seed": 17, "Hkv": 8, "D": 128,
         "dtype": "bf16", "block": 16, "keep": 4096, "sinks": 4, "recent": 512},
        # two short ones: latency
        {"name": "evict_short", "op": "evict", "B": 2, "lo": 200, "hi": 777, "lens_seed": 18, "Hkv": 2, "D": 64,
         "dtype": "fp16", "block": 32, "keep": 130, "sinks": 1, "recent": 33},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "chunk", "chunk", "chunk", "weights", "weights", "evict"])
    D = rng.choice([64, 128])
    Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8])
    c = {"op": op, "D": D, "dtype": rng.choice(["bf16", "fp16"]), "Hkv": Hkv, "lens_seed": rng.randrange(1 << 30)}
    if op in ("rope", "write"):
        c.update(H=min(Hkv * G, 32) // Hkv * Hkv, rot=rng.choice([16, 32, 64, D]), interleaved=rng.random() < 0.5,
                 scaling=rng.choice(["none", "linear", "parts"]))
        n = _log_int(rng, 1, 2000)
        if op == "rope":
            if rng.random() < 0.5:
                c.update(B=rng.randint(1, 12), lo=max(1, n // 16), hi=n)
            else:
                c.update(B=rng.randint(1, 4), S=n)
            return c
        c.update(B=rng.randint(1, 16), lo=rng.randint(1, n), hi=n, start_hi=rng.choice([0, 1000]),
                 shift=rng.choice([0, 0, 500, 1 << 20]), block=rng.choice([16, 32, 64, 128]))
        return c
    c.update(block=rng.choice([16, 32, 64, 128]))
    if op == "evict":
        hi = _log_int(rng, 1, 30000)
        lo = rng.randint(1, hi)
        keep = _log_int(rng, 1, hi)
        sinks = min(rng.choice([0, 1, 4, 20]), keep)
        c.update(B=rng.randint(1, 4), lo=lo, hi=hi, keep=keep, sinks=sinks, recent=rng.randint(0, keep - sinks))
        return c
    hi, pre = _log_int(rng, 1, 1500), rng.choice([0, _log_int(rng, 1, 16000), _log_int(rng, 1, 16000)])
    c.update(B=rng.randint(1, 8), H=Hkv * G, lo=rng.randint(1, hi), hi=hi, pre_lo=rng.randint(0, pre), pre_hi=pre,
             window=rng.choice([0, 0, _log_int(rng, 1, 4000)]), sinks=rng.choice([0, 1, 4, 20]))
    return c


def _lengths(c):
    """New tokens (or, of an eviction, keys) of each sequence."""
    if "S" in c:
        return [c["S"]] * c["B"]
    r = random.Random(c["lens_seed"])
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]


def _before(c):
    """Keys of each sequence ahead of its new tokens."""
    r = random.Random(c["lens_seed"] + 1)
    lo, hi = (0, c["start_hi"]) if "start_hi" in c else (c["pre_lo"], c["pre_hi"])
    return [r.randint(lo, hi) for _ in range(c["B"])]


def _seen(pre, n, window, sinks):
    """(query, key) pairs of a chunk of n queries behind pre keys, and the number of keys that any of them sees."""
    if window == 0 or window >= pre + n:
        return n * pre + n * (n + 1) // 2, pre + n
    pairs = 0
    for i in range(n):
        k = pre + i + 1
        w = min(window, k)
        pairs += w + min(sinks, k - w)
    first = max(pre - window + 1, 0)  # of the first query's window
    return pairs, pre + n - first + min(sinks, first)


def work(c):
    D, Hkv, lens = c["D"], c["Hkv"], _lengths(c)
    T = sum(lens)
    if c["op"] == "rope":  # each of q, k and their gradients read and written
        rows = T * (c["H"] + Hkv)
        return {"bytes": 2 * rows * 4 * D + 4 * T, "flops": 2 * rows * 3 * c["rot"]}
    if c["op"] == "write":
        return {"bytes": T * (c["H"] + 2 * Hkv) * 4 * D + 4 * T, "flops": T * (c["H"] + Hkv) * 3 * c["rot"]}
    if c["op"] == "evict":
        kept = sum(min(n, c["keep"]) for n in lens) * Hkv
        return {"bytes": 4 * T * Hkv + kept * (2 * 4 * D + 8), "flops": T * Hkv}
    both = [_seen(p, n, c["window"], c["sinks"]) for p, n in zip(_before(c), lens)]
    pairs, keys = sum(x for x, _ in both) * c["H"], sum(x for _, x in both) * Hkv
    if c["op"] == "chunk":
        return {"bytes": 2 * keys * 2 * D + T * c["H"] * (4 * D + 4), "flops": 4 * D * pairs}
    return {"bytes": keys * (2 * D + 4) + T * c["H"] * (2 * D + 4), "flops": 2 * D * pairs}


# ------------------------------------------------------------------ inputs --

def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _int32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _tables(g, block, *ends):
    """Permuted block tables for sequences of the given lengths, one table for each list of them, with no page in
    common (three spare pages; entries behind a sequence's blocks name no page), and the number of pages."""
    per = [[-(-n // block) for n in e] for e in ends]
    count = sum(map(sum, per)) + 3
    perm = torch.randperm(count, generator=g, device="cuda").to(torch.int32)
    tables, at = [], 0
    for p in per:
        t = torch.full((len(p), max(max(p), 1)), -1, dtype=torch.int32, device="cuda")
        for b, n in enumerate(p):
            t[b, :n] = perm[at:at + n]
            at += n
        tables.append(t)
    return tables, count


def _frequencies(c):
    """inv_freq (32 bits) and mscale: base 10000, plain, all divided by 8, or by parts: frequencies that turn less
    than once in 4096 positions divided by 8, those that turn over 32 times kept, and in between a blend."""
    f = 10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
    if c["scaling"] == "linear":
        return (f / 8).float().cuda(), 1.0
    if c["scaling"] == "parts":
        keep = ((4096 * f / (2 * math.pi) - 1) / 31).clamp(0, 1)
        return (f * keep + f / 8 * (1 - keep)).float().cuda(), 0.1 * math.log(8) + 1.0
    return f.float().cuda(), 1.0


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator("cuda").manual_seed(int(seed))
    dt, D, Hkv, lens = DTYPES[c["dtype"]], c["D"], c["Hkv"], _lengths(c)
    T = sum(lens)
    st = {"c": c, "lens": lens, "cu": _int32(_cu(lens)), "max": max(lens), "scale": 1.0 / math.sqrt(D)}
    if c["op"] in ("rope", "write"):
        st["inv_freq"], st["mscale"] = _frequencies(c)
    if c["op"] == "rope":
        shape = (lambda h: (c["B"], h, c["S"], D)) if "S" in c else (lambda h: (T, h, D))
        for name, h in (("q", c["H"]), ("k", Hkv), ("dq", c["H"]), ("dk", Hkv)):
            st[name] = _randn(g, shape(h), dt)
        # packed tokens count from their sequence's start; dense ones are at 0 .. S - 1
        st["positions"] = None if "S" in c else _int32([i for n in lens for i in range(n)])
        return st
    if c["op"] == "evict":
        (st["table"], st["new_table"]), count = _tables(g, c["block"], lens, [min(n, c["keep"]) for n in lens])
        rows = (count, Hkv, c["block"], D)
        st["k_cache"], st["v_cache"] = _randn(g, rows, dt), _randn(g, rows, dt)
        st["seq_lens"] = _int32(lens)
        # sums of softmax weights: a few keys have most, many have next to none, some the same
        w = torch.randn((c["B"], Hkv, st["table"].shape[1] * c["block"]), generator=g, device="cuda")
        w = torch.floor(torch.exp(2 * w) * 256) / 256
        here = torch.arange(w.shape[2], device="cuda") < st["seq_lens"][:, None, None]
        st["weights"] = torch.where(here, w, torch.zeros_like(w))
        return st
    pre = _before(c)
    (st["table"],), count = _tables(g, c["block"], [p + n for p, n in zip(pre, lens)])
    rows = (count, Hkv, c["block"], D)
    st["pre"], st["seq_lens"] = pre, _int32([p + n for p, n in zip(pre, lens)])
    st["q"] = _randn(g, (T, c["H"], D), dt)
    if c["op"] == "write":
        st["k"], st["v"] = _randn(g, (T, Hkv, D), dt), _randn(g, (T, Hkv, D), dt)
        st["k_cache"], st["v_cache"] = torch.zeros(rows, dtype=dt, device="cuda"), torch.zeros(rows, dtype=dt, device="cuda")
        st["starts"] = _int32(pre)
        shift = c["shift"]
        st["positions"] = _int32([p + shift + i for p, n in zip(pre, lens) for i in range(n)]) if shift else None
        return st
    st["k_cache"], st["v_cache"] = _randn(g, rows, dt), _randn(g, rows, dt)
    if c["op"] == "weights":
        # the attention that ran before gave each query's log-sum-exp
        st["lse"] = _chunk_plain(st, c, "lse")
        del st["v_cache"]
    return st


# --------------------------------------------------------------------- run --

def run(st):
    c = st["c"]
    if own:
        return _run_own(st, c)
    if c["op"] == "rope":
        pos = torch.arange(c["S"], device="cuda") if st["positions"] is None else st["positions"][:, None]
        turn = _turns(pos, st["inv_freq"])
        out = {n: _rope_plain(st[n], turn, c, st["mscale"], 1) for n in ("q", "k")}
        out.update({n: _rope_plain(st[n], turn, c, st["mscale"], -1) for n in ("dq", "dk")})
        return out
    if c["op"] == "write":
        return _write_plain(st, c)
    if c["op"] == "chunk":
        return _chunk_plain(st, c, "o")
    if c["op"] == "weights":
        return {"weights": _chunk_plain(st, c, "weights")}
    return _evict_plain(st, c)


def _run_own(st, c):
    import exact_attention_54_gb300 as fa

    if c["op"] == "rope":
        more = {"positions": st["positions"], "interleaved": c["interleaved"], "mscale": st["mscale"]}
        out = {n: fa.flash_rope(st[n], st["inv_freq"], **more) for n in ("q", "k")}
        out.update({n: fa.flash_rope_bwd(st[n], st["inv_freq"], **more) for n in ("dq", "dk")})
        return out
    if c["op"] == "write":
        q = fa.flash_rope_kv_write(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["cu"],
                                   st["max"], st["inv_freq"], starts=st["starts"], positions=st["positions"],
                                   interleaved=c["interleaved"], mscale=st["mscale"])
        return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if c["op"] == "chunk":
        o, lse = fa.flash_attention_paged(st["q"], st["k_cache"], st["v_cache"], st["table"], st["cu"], st["seq_lens"],
                                          st["max"], c["window"], c["sinks"])
        return {"o": o, "lse": lse}
    if c["op"] == "weights":
        return {"weights": fa.flash_kv_weights(st["q"], st["lse"], st["k_cache"], st["table"], st["cu"],
                                               st["seq_lens"], st["max"], c["window"], c["sinks"])}
    kept, new_lens, weights = fa.flash_kv_evict(st["k_cache"], st["v_cache"], st["weights"], st["table"],
                                                st["seq_lens"], st["new_table"], c["keep"], c["sinks"], c["recent"])
    return {"kept": kept, "new_lens": new_lens, "weights": weights, "k_cache": st["k_cache"],
            "v_cache": st["v_cache"]}


def _turns(pos, inv_freq):
    """cos and sin (32 bits) of the angles, which are formed in 64."""
    a = pos.double()[..., None] * inv_freq.double()
    return torch.cos(a).float(), torch.sin(a).float()


def _rope_plain(x, turn, c, mscale, sign):
    r, (cos, sin) = c["rot"], turn
    y = x.float()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if c["interleaved"] else (y[..., :r // 2], y[..., r // 2:r])
    sin = sin * sign
    a, b = (a * cos - b * sin) * mscale, (b * cos + a * sin) * mscale
    both = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((both, y[..., r:]), -1).to(x.dtype)


def _places(st, c):
    """Page, row within the page and place in its sequence of every packed token."""
    cu = st["cu"].long()
    t = torch.arange(st["q"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = st["starts"].long()[b] + t - cu[b]
    return st["table"].long()[b, pos // c["block"]], pos % c["block"], pos


def _write_plain(st, c):
    page, row, pos = _places(st, c)
    if st["positions"] is not None:
        pos = st["positions"]
    turn = _turns(pos[:, None], st["inv_freq"])
    st["k_cache"][page, :, row] = _rope_plain(st["k"], turn, c, st["mscale"], 1)
    st["v_cache"][page, :, row] = st["v"]
    return {"q": _rope_plain(st["q"], turn, c, st["mscale"], 1), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _keys(cache, table_row, block, n):
    """A sequence's rows [Hkv, n, D], in 32 bits."""
    x = cache[table_row[:-(-n // block)].long()]
    return x.transpose(0, 1).flatten(1, 2)[:, :n].float()


def _chunk_plain(st, c, what):
    """Sequence by sequence: o and lse ("o"), lse alone, or the weights that the keys receive, given lse."""
    H, Hkv, D, T = c["H"], c["Hkv"], c["D"], st["q"].shape[0]
    G = H // Hkv
    o, lse = torch.empty_like(st["q"]), torch.empty((H, T), device="cuda")
    weights = torch.zeros((c["B"], Hkv, st["table"].shape[1] * c["block"]), device="cuda") if what == "weights" else None
    at = 0
    for b, (p, n) in enumerate(zip(st["pre"], st["lens"])):
        L = p + n
        q = st["q"][at:at + n].float().view(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * n, D)
        s = (q @ _keys(st["k_cache"], st["table"][b], c["block"], L).transpose(1, 2)) * st["scale"]
        i, j = torch.arange(p, L, device="cuda")[:, None], torch.arange(L, device="cuda")
        seen = (j <= i) & ((i - j < (c["window"] or L)) | (j < c["sinks"]))
        s = s.view(Hkv, G, n, L).masked_fill_(~seen, float("-inf"))
        if what == "weights":
            z = st["lse"][:, at:at + n].view(Hkv, G, n, 1)
            weights[b, :, :L] = torch.exp(s - z).sum((1, 2))
        else:
            m = s.amax(-1, keepdim=True)
            s = s.sub_(m).exp_()
            z = s.sum(-1, keepdim=True)
            lse[:, at:at + n] = (m + torch.log(z)).view(H, n)
            if what == "o":
                v = _keys(st["v_cache"], st["table"][b], c["block"], L)
                r = (s.div_(z).view(Hkv, G * n, L) @ v).view(Hkv, G, n, D)
                o[at:at + n] = r.permute(2, 0, 1, 3).reshape(n, H, D).to(o.dtype)
        at += n
    return weights if what == "weights" else {"o": o, "lse": lse} if what == "o" else lse


def _evict_plain(st, c):
    B, Hkv, keep, block = c["B"], c["Hkv"], c["keep"], c["block"]
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    weights = torch.zeros((B, Hkv, st["new_table"].shape[1] * block), device="cuda")
    new_lens = st["seq_lens"].clamp(max=keep)
    heads = torch.arange(Hkv, device="cuda")[:, None]
    for b, n in enumerate(st["lens"]):
        m = min(n, keep)
        rank = st["weights"][b, :, :n].clone()
        if n > keep:
            rank[:, :c["sinks"]] = float("inf")
            rank[:, n - c["recent"]:] = float("inf")
        idx = torch.sort(rank, dim=-1, descending=True, stable=True).indices[:, :m].sort(-1).values
        kept[b, :, :m] = idx.int()
        weights[b, :, :m] = st["weights"][b].gather(1, idx)
        src, dst = st["table"][b].long()[idx // block], st["new_table"][b].long()[torch.arange(m, device="cuda") // block]
        for x in (st["k_cache"], st["v_cache"]):
            x[dst, heads, torch.arange(m, device="cuda") % block] = x[src, heads, idx % block]
    return {"kept": kept, "new_lens": new_lens, "weights": weights, "k_cache": st["k_cache"],
            "v_cache": st["v_cache"]}


# ------------------------------------------------------------------- exact --

def exact(case, seed):
    c = dict(case)
    st = prepare(c, seed)
    if c["op"] == "rope":
        pos = torch.arange(c["S"], device="cuda") if st["positions"] is None else st["positions"][:, None]
        out = {n: _exact_rope(st[n], pos, st, c, False) for n in ("q", "k")}
        out.update({n: _exact_rope(st[n], pos, st, c, True) for n in ("dq", "dk")})
        return out
    if c["op"] == "write":
        at, kc, vc = 0, st["k_cache"].double(), st["v_cache"].double()
        pos = [p + c["shift"] + i for p, n in zip(st["pre"], st["lens"]) for i in range(n)]
        pos = torch.tensor(pos, device="cuda")[:, None]
        k = _exact_rope(st["k"], pos, st, c, False)
        for b, (p, n) in enumerate(zip(st["pre"], st["lens"])):
            j = torch.arange(p, p + n, device="cuda")
            page = st["table"][b][torch.div(j, c["block"], rounding_mode="floor")].long()
            kc[page, :, j % c["block"]] = k[at:at + n]
            vc[page, :, j % c["block"]] = st["v"][at:at + n].double()
            at += n
        return {"q": _exact_rope(st["q"], pos, st, c, False), "k_cache": kc, "v_cache": vc}
    if c["op"] == "evict":
        return _exact_evict(st, c)
    return _exact_chunk(st, c)


def _exact_rope(x, pos, st, c, inverse):
    """A product of complex numbers; the gradient's is with the conjugate."""
    r = c["rot"]
    z = x.double().clone()
    first = torch.arange(0, r, 2, device="cuda") if c["interleaved"] else torch.arange(r // 2, device="cuda")
    second = first + (1 if c["interleaved"] else r // 2)
    a = pos.double()[..., None] * st["inv_freq"].double()
    turn = torch.polar(torch.full_like(a, st["mscale"]), -a if inverse else a)
    y = torch.complex(z[..., first], z[..., second]) * turn
    z[..., first], z[..., second] = y.real, y.imag
    return z


def _exact_chunk(st, c):
    """Head by head, from the definition."""
    G, T, block = c["H"] // c["Hkv"], st["q"].shape[0], c["block"]
    if c["op"] == "chunk":
        res = {"o": torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"),
               "lse": torch.zeros((c["H"], T), dtype=torch.float64, device="cuda")}
    else:
        res = {"weights": torch.zeros((c["B"], c["Hkv"], st["table"].shape[1] * block), dtype=torch.float64,
                                      device="cuda")}
    cu = st["cu"].tolist()
    for b, L in enumerate(st["seq_lens"].tolist()):
        j = torch.arange(L, device="cuda")
        page = st["table"][b][torch.div(j, block, rounding_mode="floor")].long()
        at = torch.arange(L - (cu[b + 1] - cu[b]), L, device="cuda").unsqueeze(1)
        hidden = j > at
        if c["window"]:
            hidden |= (j <= at - c["window"]) & (j >= c["sinks"])
        for h in range(c["H"]):
            k = st["k_cache"][page, h // G, j % block].double()
            z = torch.einsum("id,jd->ij", st["q"][cu[b]:cu[b + 1], h].double(), k).mul_(st["scale"])
            z.masked_fill_(hidden, -math.inf)
            if c["op"] == "weights":
                res["weights"][b, h // G, :L] += z.sub_(st["lse"][h, cu[b]:cu[b + 1], None].double()).exp_().sum(0)
                continue
            lse = torch.logsumexp(z, -1)
            v = st["v_cache"][page, h // G, j % block].double()
            res["lse"][h, cu[b]:cu[b + 1]] = lse
            res["o"][cu[b]:cu[b + 1], h] = torch.einsum("ij,jd->id", z.sub_(lse.unsqueeze(-1)).exp_(), v)
    return res


def _exact_evict(st, c):
    block, keep = c["block"], c["keep"]
    kept = torch.full((c["B"], c["Hkv"], keep), -1, dtype=torch.int32)
    weights = torch.zeros((c["B"], c["Hkv"], st["new_table"].shape[1] * block), dtype=torch.float64)
    caches = st["k_cache"].double(), st["v_cache"].double()
    w, old, new = st["weights"].cpu(), st["table"].cpu(), st["new_table"].cpu()
    for b, n in enumerate(st["lens"]):
        for h in range(c["Hkv"]):
            order = w[b, h, :n].tolist()
            if n <= keep:
                chosen = list(range(n))
            else:
                middle = sorted(range(c["sinks"], n - c["recent"]), key=lambda j: (-order[j], j))
                chosen = sorted(list(range(c["sinks"])) + middle[:keep - c["sinks"] - c["recent"]] +
                                list(range(n - c["recent"], n)))
            x, at = torch.tensor(chosen), torch.arange(len(chosen))
            kept[b, h, :len(chosen)] = x.int()
            weights[b, h, :len(chosen)] = w[b, h][x].double()
            src = (old[b][x // block].long().cuda(), h, (x % block).cuda())
            dst = (new[b][at // block].long().cuda(), h, (at % block).cuda())
            for cache in caches:
                cache[dst] = cache[src]
    return {"kept": kept.cuda(), "new_lens": torch.tensor([min(n, keep) for n in st["lens"]], dtype=torch.int32).cuda(),
            "weights": weights.cuda(), "k_cache": caches[0], "v_cache": caches[1]}
