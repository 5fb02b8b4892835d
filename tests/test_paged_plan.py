"""How a CTA of fa_fwd_paged and fa_kv_weights finds its place in the work, as a
model on the CPU of the look-up in csrc/fa_paged.cuh: sums over sequences (or, of
more than the table holds, over several each), the entry, the sequence, the key
head and the unit, of which a range costs the same. It has to be the place that
walking all units one by one gives, and every unit of the weights has to be taken
by the one CTA in whose run it starts. On the GPU: numbers of sequences on both
sides of what the table and the list of loaded sequences hold."""
import random

import pytest
import torch

import exact_attention_54_gb300 as fa
from test_chunk import check, make, reference
from test_chunk_plan import START, tiles
from test_kv_weights import check_weights, reference_weights, true_lse

KEYS = 256  # of a unit of the weights


class ChunkUnits:
    def __init__(self, tokens, window, sinks):
        self.tokens, self.window, self.sinks = tokens, window, sinks

    def count(self, s):
        return -(-s[0] // (2 * self.tokens))

    def cost(self, s, i):
        return tiles(s[1] - s[0], s[0], self.tokens, self.window, self.sinks, i)["steps"] + START

    def flat(self, s, n):
        return 0, 0


class WeightUnits(ChunkUnits):
    def count(self, s):
        return -(-s[1] // KEYS) if s[0] > 0 else 0

    def seen(self, s, i):
        """Tokens [t0, t1) of the chunk that see a key of unit i."""
        k0, pos0 = i * KEYS, s[1] - s[0]
        t0, t1 = max(k0 - pos0, 0), s[0]
        if self.window > 0 and k0 >= self.sinks:
            t1 = min(t1, max(k0 + KEYS - 1 + self.window - pos0, 0))
        return t0, t1

    def cost(self, s, i):
        t0, t1 = self.seen(s, i)
        return -(-(t1 - t0) // self.tokens) + 1 if t1 > t0 else 0

    def flat(self, s, n):
        pos0 = s[1] - s[0]
        to = min(n, pos0 // KEYS + 1) if pos0 >= 0 else 0
        return 0, min(to, -(-self.sinks // KEYS)) if self.window > 0 else to


def seq_cost(u, s):
    n = u.count(s)
    a, b = u.flat(s, n)
    return sum(u.cost(s, i) for i in [*range(a), *range(b, n)]) + ((b - a) * u.cost(s, a) if b > a else 0)


def place(u, seqs, Hkv, grid, cta, table):
    """(length of the run, b, hk, unit, off) by the look-up."""
    each = -(-len(seqs) // table)
    entries = -(-len(seqs) // each)
    prefix = [0] * (entries + 1)
    for b, s in enumerate(seqs):
        prefix[b // each + 1] += seq_cost(u, s)
    for e in range(entries):
        prefix[e + 1] += prefix[e]
    total = prefix[entries] * Hkv
    per = max(-(-total // grid), 1)
    at = min(cta * per, total)
    if min(per, total - at) <= 0:
        return per, None
    lo, hi = 0, entries
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if prefix[mid] * Hkv <= at else (lo, mid)
    x, b = at - prefix[lo] * Hkv, lo * each
    while True:
        c = prefix[b + 1] - prefix[b] if each == 1 else seq_cost(u, seqs[b])
        if x < c * Hkv or b + 1 >= len(seqs):
            break
        x -= c * Hkv
        b += 1
    hk, x, s = x // c, x % c, seqs[b]
    n = u.count(s)
    f0, f1 = u.flat(s, n)

    def among(i0, i1, x):
        for i in range(i0, i1):
            if x < u.cost(s, i):
                return i, x
            x -= u.cost(s, i)
        return None, x

    unit, x = among(0, f0, x)
    if unit is None:
        one = u.cost(s, f0) if f1 > f0 else 0
        if x < (f1 - f0) * one:
            unit, x = f0 + x // one, x % one
        else:
            unit, x = among(f1, n, x - (f1 - f0) * one)
    return per, (min(per, total - at), b, hk, unit, x)


def batch(r, count, small):
    seqs = []
    for _ in range(count):
        Lq = r.choice([0, 0, 1, 2, 40] if small else [0, 1, 3, 70, 500])
        seqs.append((Lq, r.choice([0, Lq, Lq // 2, Lq + r.randint(0, 300 if small else 6000)])))
    return seqs


@pytest.mark.parametrize("seed", range(60))
@pytest.mark.parametrize("kind", [ChunkUnits, WeightUnits])
def test_place_of_a_run(kind, seed):
    r = random.Random(seed)
    # (a table of 8 entries stands for the kernels' 4096)
    count, table, small = r.choice([(1, 8, False), (6, 8, False), (8, 8, True), (9, 8, True), (37, 8, True), (700, 64, True)])
    u = kind(r.choice([1, 4, 32, 128]), r.choice([0, 0, 1, 200, 3000]), r.choice([0, 4, 256, 300]))
    seqs, Hkv, grid = batch(r, count, small), r.randint(1, 4), r.choice([3, 8, 152])
    units = [(b, hk, i, u.cost(s, i)) for b, s in enumerate(seqs) for hk in range(Hkv) for i in range(u.count(s))]
    for s in seqs:  # the range that is said to cost the same does
        f0, f1 = u.flat(s, u.count(s))
        assert 0 <= f0 <= max(f1, f0) <= u.count(s) and len({u.cost(s, i) for i in range(f0, f1)}) <= 1
    ends, at = [], 0
    for x in units:
        at += x[3]
        ends.append(at)
    taken, covered = {}, 0
    for cta in range(grid):
        per, got = place(u, seqs, Hkv, grid, cta, table)
        assert per == max(-(-at // grid), 1)
        if got is None:
            assert cta * per >= at
            continue
        length, b, hk, unit, off = got
        begin = cta * per
        i = next(i for i, e in enumerate(ends) if e > begin)
        assert (b, hk, unit) == units[i][:3] and off == begin - (ends[i] - units[i][3])
        assert length == min(per, at - begin)
        covered += length
        # the weights: a CTA takes the units that start in its run, whole
        while i < len(units) and ends[i] - units[i][3] < begin + length:
            if ends[i] - units[i][3] >= begin and units[i][3] > 0:
                assert taken.setdefault(units[i][:3], cta) == cta
            i += 1
    assert covered == at and set(taken) == {x[:3] for x in units if x[3] > 0}


@pytest.mark.parametrize("seed", range(40))
def test_units_of_the_weights_reach_every_pair(seed):
    r = random.Random(1000 + seed)
    u = WeightUnits(r.choice([1, 18, 128]), r.choice([0, 1, 100, 700]), r.choice([0, 1, 5, 256, 400]))
    for s in batch(r, 20, seed % 2 == 0):
        Lq, L = s
        for i in range(u.count(s)):
            t0, t1 = u.seen(s, i)
            for t in range(Lq):
                p = L - Lq + t
                sees = any(j <= p and (u.window == 0 or p - j < u.window or j < u.sinks)
                           for j in range(i * KEYS, min(L, (i + 1) * KEYS)))
                assert not sees or t0 <= t < t1


@pytest.mark.gpu
@pytest.mark.parametrize("B", [511, 513, 1100, 4096, 4097])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 3)])
def test_numbers_of_sequences(B, window, sinks):
    """With sequences that have no queries, no keys, fewer keys than queries, and units that nobody sees."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 60, (B,), generator=g)
    lens[torch.randint(0, B, (3,), generator=g)] = 900
    chunks = torch.randint(0, 5, (B,), generator=g) * (torch.rand(B, generator=g) < 0.7)
    lens, chunks = lens.tolist(), chunks.tolist()
    q, kc, vc, table, sl, cu = make(chunks, lens, 2, 1, 64, 8, torch.bfloat16, B)
    ref = reference(q, kc, vc, table, lens, cu, window, sinks, 0.125)
    d = [t.cuda() for t in (q, kc, vc, table, cu, sl)]
    o, lse = fa.flash_attention_paged(*d, 4, window, sinks)
    rl = true_lse(q, kc, table, lens, cu, window, sinks, 0.125)
    w = fa.flash_kv_weights(d[0], rl.cuda(), d[1], *d[3:], 4, window, sinks)
    fa.fa_check_device_error()
    check(o, lse, ref)
    check_weights(w, reference_weights(q, rl, kc, table, lens, cu, window, sinks, 0.125))
