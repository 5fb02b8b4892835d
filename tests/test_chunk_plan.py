"""How fa_fwd_paged cuts its work, as a model on the CPU: key tiles of a unit,
steps of a part, the runs of the CTAs and the parts that are joined. The model
states the rules of csrc/fa_chunk.cuh; every (query, visible key) pair has to be
computed once, every step to be used by a query tile, and every unit's parts to
be found by the launch that joins them."""
import random

import pytest

START = 3  # a unit's start, in key tiles


def tiles(pos0, Lq, tokens, window, sinks, pair):
    sink_tiles = -(-sinks // 128) if window > 0 else 0
    k = {"tok": [], "ntok": [], "hi": [], "wlo": [], "sink": []}
    ns, lo, end = 0, 1 << 31, 0
    for t in range(2):
        tok = (2 * pair + t) * tokens
        ntok = min(max(Lq - tok, 0), tokens)
        first, last = pos0 + tok, pos0 + tok + ntok - 1
        hi = last // 128 + 1 if ntok > 0 and last >= 0 else 0
        wlo = max(first - window + 1, 0) // 128 if window > 0 else 0
        sink = min(sink_tiles, hi)
        for n, v in (("tok", tok), ("ntok", ntok), ("hi", hi), ("wlo", wlo), ("sink", sink)):
            k[n].append(v)
        if hi > 0:
            ns, lo, end = max(ns, sink), min(lo, wlo), max(end, hi)
    lo = max(min(lo, end), ns)
    return {**k, "ns": ns, "lo": lo, "steps": ns + max(end - lo, 0)}


def tile_at(k, j):
    return j if j < k["ns"] else j - k["ns"] + k["lo"]


def visits(k, t, j):
    x = tile_at(k, j)
    return x < k["hi"][t] and (x < k["sink"][t] or x >= k["wlo"][t])


def visited(k, t, s0, s1):
    both = lambda a, b: max(min(b, s1) - max(a, s0), 0)  # noqa: E731
    start = max(k["wlo"][t], k["sink"][t])
    return both(0, k["sink"][t]) + both(start, min(k["hi"][t], k["ns"])) + \
        both(max(start, k["lo"]) - k["lo"] + k["ns"], k["hi"][t] - k["lo"] + k["ns"])


@pytest.mark.parametrize("seed", range(40))
def test_tiles_of_a_unit(seed):
    r = random.Random(seed)
    tokens = r.choice([1, 4, 18, 32, 128])
    Lq, L = r.randint(1, 6 * tokens), r.randint(0, 2500)
    window, sinks = r.choice([0, 1, 100, 128, 300, 900]), r.choice([0, 1, 4, 128, 200, 600])
    pos0 = L - Lq
    for pair in range(-(-Lq // (2 * tokens))):
        k = tiles(pos0, Lq, tokens, window, sinks, pair)
        for t in range(2):
            seen = set()
            for i in range(k["ntok"][t]):
                p = pos0 + k["tok"][t] + i
                seen |= {j // 128 for j in range(0, p + 1) if window == 0 or p - j < window or j < sinks}
            mine = [tile_at(k, j) for j in range(k["steps"]) if visits(k, t, j)]
            assert len(mine) == len(set(mine)) and seen <= set(mine)
            if mine:
                assert max(mine) * 128 < L
            s0 = r.randint(0, k["steps"])
            s1 = r.randint(s0, k["steps"])
            assert visited(k, t, s0, s1) == sum(visits(k, t, j) for j in range(s0, s1))
        assert all(visits(k, 0, j) or visits(k, 1, j) for j in range(k["steps"]))


@pytest.mark.parametrize("seed", range(60))
def test_runs_and_parts(seed):
    r = random.Random(seed)
    grid, min_run = r.choice([3, 8, 152]), r.choice([1, 6])
    tokens, Hkv = r.choice([4, 32, 128]), r.randint(1, 4)
    window, sinks = r.choice([0, 0, 200]), r.choice([0, 4, 300])
    seqs = []
    for _ in range(r.randint(1, 6)):
        Lq = r.choice([0, 1, 3, 70, 500])
        seqs.append((Lq, r.choice([0, Lq, Lq + r.randint(0, 6000)])))
    units = []
    for b, (Lq, L) in enumerate(seqs):
        for hk in range(Hkv):
            for pair in range(-(-Lq // (2 * tokens))):
                units.append((b, hk, pair, tiles(L - Lq, Lq, tokens, window, sinks, pair)["steps"]))
    total = sum(u[3] + START for u in units)
    per = max(-(-total // grid), min_run)
    done, slots, records = {}, {}, {}
    for cta in range(grid):
        at = min(cta * per, total)
        rem = min(per, total - at)
        i, off = 0, at
        while rem > 0 and off >= units[i][3] + START:
            off -= units[i][3] + START
            i += 1
        first, joins = True, 0
        while rem > 0:
            b, hk, pair, steps = units[i]
            n = steps + START
            take = min(rem, n - off)
            s0, s1 = max(off - START, 0), max(off + take - START, 0)
            rest = n - off - take
            whole, slot = s0 == 0 and s1 == steps, 0 if first else 1
            if s1 > s0 or (steps == 0 and off == 0):
                done.setdefault((b, hk, pair), []).append((s0, s1))
                if not whole:
                    assert (cta, slot) not in slots
                    slots[cta, slot] = (b, hk, pair, s0, s1)
                else:
                    done[b, hk, pair].append("whole")
                if s0 == 0 and s1 > 0 and rest > 0:
                    records[cta] = (b, hk, pair, 1 + -(-rest // per), slot)
                    joins += 1
            rem, first, off, i = rem - take, False, 0, i + 1
        assert joins <= 1
    for b, hk, pair, steps in units:
        parts = done[b, hk, pair]
        if "whole" in parts:
            assert len(parts) == 2
            continue
        parts.sort()
        assert parts[0][0] == 0 and parts[-1][1] == steps and all(a[1] == c[0] for a, c in zip(parts, parts[1:]))
        mine = [(c, v) for c, v in records.items() if v[:3] == (b, hk, pair)]
        assert len(mine) == 1
        cta, (_, _, _, n, slot) = mine[0]
        found = [slots[cta + x, slot if x == 0 else 0] for x in range(n)]
        assert [f[3:] for f in found] == parts and all(f[:3] == (b, hk, pair) for f in found)
