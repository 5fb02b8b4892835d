"""What each cached key receives (fa_kv_weights) against its definition in 64
bits, the calls it refuses, and a whole step: tokens rotated into a cache,
attended, their weights summed, the cache evicted, and attended again."""
import math

import pytest
import torch

import exact_attention_54_gb300 as fa
from exact_attention_54_gb300 import build as fabuild
from exact_attention_54_gb300 import inputs
from test_chunk import check, make, reference, rows_of, visible_behind

OK, NULL, SHAPE, HEADDIM, DTYPE, ALIGN, SCALE = 0, -1, -2, -3, -4, -5, -7
TIMEOUT, DEV_INDEX, DEV_SEQLENS = -9, -11, -13
A, MIS = 0x10000, 0x10008
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


def reference_weights(q, lse, kc, table, lens, cu, window, sinks, scale):
    """[B, Hkv, width] in double; lse [H, T]."""
    G, block = q.shape[1] // kc.shape[1], kc.shape[2]
    w = torch.zeros(len(lens), kc.shape[1], table.shape[1] * block, dtype=torch.float64)
    for b, L in enumerate(int(x) for x in lens):
        sl = slice(int(cu[b]), int(cu[b + 1]))
        n = sl.stop - sl.start
        if n == 0 or L == 0:
            continue
        seen = visible_behind(n, L, window, sinks)
        for h in range(q.shape[1]):
            s = q[sl, h].double() @ rows_of(kc, table[b], h // G, L).t() * scale
            p = torch.exp(s - lse[h, sl, None].double())
            w[b, h // G, :L] += torch.where(seen, p, torch.zeros_like(p)).sum(0)
    return w


def check_weights(w, ref, before=None, what=""):
    """Each term's exponent is off by 2^-13 at most (scores in fp32, as in plain_ops; |lse| under 64 rounded twice to
    2^-24 of it), the sum of at most 2^12 terms by 2^-12 of itself, the addition to what was there by 2^-24."""
    w = w.double().cpu()
    before = torch.zeros_like(ref) if before is None else before.double()
    bad = ~((w - before - ref).abs() <= 2.0 ** -12 * ref + 2.0 ** -23 * before.abs() + 1e-37)
    assert not bad.any(), (what, torch.nonzero(bad)[0].tolist(), int(bad.sum()),
                           float(((w - before - ref).abs() / (ref + 1e-30)).max()))


def true_lse(q, kc, table, lens, cu, window, sinks, scale):
    return reference(q, kc, kc, table, lens, cu, window, sinks, scale)[1].float()


# -------------------------------------------------------------- on the CPU --

def test_validation(lib):
    def call(q=A, lse=A, kc=A, bt=A, cu=A, sl=A, w=A, lh=100, lt=1, n=2, total=100, mx=64, H=8, Hkv=2, D=128, nb=8, bs=16,
             mb=4, window=0, sinks=0, add=1, scale=0.1, dtype=1):
        return lib.fa_kv_weights(q, lse, kc, bt, cu, sl, w, lh, lt, n, total, mx, H, Hkv, D, nb, bs, mb, window, sinks,
                                 add, scale, dtype, None)

    for kw in ("q", "lse", "kc", "bt", "cu", "sl", "w"):
        assert call(**{kw: None}) == NULL, kw
    assert call(dtype=2) == DTYPE
    for d in (32, 96, 256):
        assert call(D=d) == HEADDIM
    for kw in ({"n": 0}, {"total": 0}, {"mx": 0}, {"H": 0}, {"Hkv": 3}, {"nb": 0}, {"bs": 24}, {"mb": 0}, {"window": -1},
               {"sinks": -1}, {"H": 258}, {"lh": -1}, {"lt": -1}, {"lh": 1 << 41}):
        assert call(**kw) == SHAPE, kw
    assert call(scale=-1.0) == SCALE
    for kw in ("q", "kc"):
        assert call(**{kw: MIS}) == ALIGN, kw
    for kw in ("lse", "bt", "cu", "sl", "w"):
        assert call(**{kw: A + 2}) == ALIGN, kw


def test_binding_refuses():
    q, c = torch.zeros(5, 4, 64, dtype=BF), torch.zeros(8, 2, 16, 64, dtype=BF)
    bt, cu = torch.zeros(1, 4, dtype=torch.int32), torch.tensor([0, 5], dtype=torch.int32)
    sl, lse = torch.tensor([5], dtype=torch.int32), torch.zeros(4, 5)
    call = lambda q=q, lse=lse, c=c, w=torch.zeros(1, 2, 64): fa.flash_kv_weights(q, lse, c, bt, cu, sl, 5, weights=w)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(TypeError, match="lse"):
        call(lse=lse.double())
    with pytest.raises(ValueError, match="lse"):
        call(lse=lse.t())
    with pytest.raises(ValueError, match="weights"):
        call(w=torch.zeros(1, 2, 63))
    with pytest.raises(TypeError, match="k_cache"):
        call(c=c.half())


def test_binding_refuses_other_dimensions():
    q, c, cu = torch.zeros(5, 4, 64, dtype=BF), torch.zeros(8, 2, 16, 64, dtype=BF), torch.tensor([0, 5], dtype=torch.int32)
    bt = torch.zeros(1, 4, dtype=torch.int32)
    for kc, table in ((c[0, 0], bt), (c, bt[0]), (c, bt[0, 0])):
        with pytest.raises(ValueError, match="block_table"):
            fa.flash_kv_weights(q, torch.zeros(4, 5), kc, table, cu, torch.tensor([5], dtype=torch.int32), 5)


# -------------------------------------------------------------- on the GPU --

@pytest.mark.gpu
@pytest.mark.parametrize("chunks,lens,H,Hkv,D,block,window,sinks,dtype", [
    ([1], [1], 1, 1, 64, 16, 0, 0, BF),
    ([128], [128], 2, 2, 128, 16, 0, 0, BF),
    ([5, 1, 33], [300, 129, 33], 8, 2, 128, 16, 0, 0, BF),
    ([70, 0, 2], [70, 40, 513], 6, 2, 64, 32, 0, 0, FP),
    ([300], [777], 4, 1, 128, 64, 0, 0, FP),
    ([19, 37], [500, 37], 14, 2, 64, 8, 0, 0, BF),        # seven heads to a key head: 126 rows a tile
    ([9], [260], 128, 1, 64, 256, 0, 0, FP),              # one token a tile
    ([2, 3], [1500, 900], 16, 1, 64, 1024, 0, 0, BF),
    ([50], [400], 4, 4, 128, 1, 0, 0, BF),                # pages of 1 and 2 keys
    ([50, 3], [131, 90], 4, 2, 64, 2, 0, 0, FP),
    ([200], [900], 4, 2, 128, 16, 1, 0, BF),              # windows
    ([200, 31], [900, 400], 4, 2, 64, 16, 128, 4, FP),
    ([257], [1300], 2, 1, 128, 32, 300, 200, BF),
    ([64], [700], 4, 1, 64, 64, 129, 129, BF),
    ([33], [600], 7, 1, 128, 16, 5000, 4, FP),
    ([100], [60], 4, 2, 64, 16, 0, 0, BF),                # more queries than keys
    ([100], [60], 4, 2, 128, 16, 20, 2, FP),
    ([3, 4], [0, 10], 4, 2, 64, 16, 0, 0, BF),
    ([700], [1000], 8, 1, 128, 16, 0, 0, BF),             # many query tiles
])
def test_weights(chunks, lens, H, Hkv, D, block, window, sinks, dtype):
    q, kc, _, table, sl, cu = make(chunks, lens, H, Hkv, D, block, dtype, sum(chunks) + sum(lens))
    lse = true_lse(q, kc, table, lens, cu, window, sinks, D ** -0.5)
    ref = reference_weights(q, lse, kc, table, lens, cu, window, sinks, D ** -0.5)
    args = [t.cuda() for t in (q, lse, kc, table, cu, sl)]
    w = fa.flash_kv_weights(*args, max(chunks), window, sinks)
    fa.fa_check_device_error()
    check_weights(w, ref)
    # put where anything was, keys that nobody sees included
    old = torch.full(w.shape, math.nan, device="cuda")
    fa.fa_kv_weights(*args, old, max(chunks), window, sinks, add=False)
    assert torch.equal(old, w)
    # every query that sees a key gives 1 for each head, in all
    give = sum(int(visible_behind(n, L, window, sinks).any(1).sum()) for n, L in zip(chunks, lens) if n and L)
    assert abs(float(w.double().sum()) - give * H) <= 2.0 ** -12 * give * H + 1e-9
    # added to what is there; a token-major lse gives the same bits
    before = torch.rand(w.shape, generator=torch.Generator().manual_seed(1))
    again = fa.flash_kv_weights(args[0], args[1].t().contiguous().t(), *args[2:], max(chunks), window, sinks,
                                weights=before.cuda())
    check_weights(again, ref, before)
    nothing = ref == 0
    assert torch.equal(again.cpu()[nothing], before[nothing])
    assert torch.equal(w, fa.flash_kv_weights(args[0], args[1].t().contiguous().t(), *args[2:], max(chunks), window, sinks))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [300, 5000])
def test_many_sequences(B):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 40, (B,), generator=g)
    chunks = torch.minimum(torch.randint(0, 4, (B,), generator=g), lens)
    q, kc, _, table, sl, cu = make(chunks.tolist(), lens.tolist(), 2, 1, 64, 8, BF, B)
    lse = true_lse(q, kc, table, lens.tolist(), cu, 0, 0, 0.125)
    w = fa.flash_kv_weights(*(t.cuda() for t in (q, lse, kc, table, cu, sl)), 3)
    fa.fa_check_device_error()
    check_weights(w, reference_weights(q, lse, kc, table, lens.tolist(), cu, 0, 0, 0.125))


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks,block", [(0, 0, 16), (60, 5, 16), (60, 0, 128), (200, 140, 64), (33, 4, 4)])
def test_what_nobody_sees_may_hold_anything(window, sinks, block):
    chunks, lens, D = [20, 3, 140], [333, 1000, 500], 64
    q, kc, _, table, sl, cu = make(chunks, lens, 4, 2, D, block, BF, 8, pad=9)
    lse = torch.full((4, q.shape[0]), math.nan)
    q[163:] = math.nan
    lse[:, :163] = true_lse(q[:163], kc, table, lens, cu, window, sinks, D ** -0.5)
    ref = reference_weights(q, lse, kc, table, lens, cu, window, sinks, D ** -0.5)
    seen_rows = torch.zeros(kc.shape[0], block, dtype=torch.bool)
    for b, (n, L) in enumerate(zip(chunks, lens)):
        seen = visible_behind(n, L, window, sinks).any(0)
        at = torch.nonzero(seen).flatten()
        seen_rows[table[b][at // block].long(), at % block] = True
        for x in range(-(-L // block)):
            if not seen[x * block:(x + 1) * block].any():
                table[b, x] = -7
    kc.masked_fill_(~seen_rows[:, None, :, None], math.nan)
    w = fa.flash_kv_weights(*(t.cuda() for t in (q, lse, kc, table, cu, sl)), 150, window, sinks)
    fa.fa_check_device_error()
    check_weights(w, ref)


@pytest.mark.gpu
def test_checks_on_the_device_and_withheld_load():
    chunks, lens = [20, 7], [150, 90]
    q, kc, _, table, sl, cu = make(chunks, lens, 4, 2, 64, 16, BF, 3)
    lse = true_lse(q, kc, table, lens, cu, 0, 0, 0.125).cuda()
    q, kc, table, sl, cu = (t.cuda() for t in (q, kc, table, sl, cu))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def status(cu=cu, table=table, sl=sl, mx=20):
        w = fa.flash_kv_weights(q, lse, kc, table, cu, sl, mx, weights=torch.full((2, 2, table.shape[1] * 16), 3.0, device="cuda"))
        try:
            fa.fa_check_device_error()
        except fa.FAError as e:
            return e.status, w
        return OK, w

    ok, good = status()
    assert ok == OK
    for bad in (i32(0, 28, 27), i32(0, 20, 28), i32(-1, 20, 27), i32(20, 7, 27)):
        st, w = status(cu=bad)
        assert st == DEV_SEQLENS and (w == 3).all()
    assert status(mx=19)[0] == DEV_SEQLENS
    t = table.clone()
    t[0, 2] = kc.shape[0]
    st, w = status(table=t)
    assert st == DEV_INDEX and torch.equal(w[1], good[1]) and torch.isfinite(w).all()
    fa.fa_test_withhold_load(1, 20_000_000)
    try:
        assert status()[0] == TIMEOUT
    finally:
        fa.fa_test_withhold_load(0, 0)
    assert status()[0] == OK and torch.equal(status()[1], good)
    # a query that sees nothing (lse -inf) gives nothing
    none = lse.clone()
    none[:, :20] = -math.inf
    w = fa.flash_kv_weights(q, none, kc, table, cu, sl, 20)
    assert (w[0] == 0).all() and (w[1] > 0).any()


@pytest.mark.gpu
def test_weights_of_a_decode():
    """lse [B,H] of the one-token calls, transposed."""
    lens, H, Hkv, D = [700, 33, 1500], 8, 2, 128
    q, kc, vc, table, sl, cu = make([1, 1, 1], lens, H, Hkv, D, 16, BF, 6)
    args = [t.cuda() for t in (q, kc, vc, table, sl, cu)]
    _, lse = fa.flash_decode_paged_window(args[0][:, :, None], args[1], args[2], args[3], args[4], 64, 4)
    w = fa.flash_kv_weights(args[0], lse.t(), args[1], args[3], args[5], args[4], 1, 64, 4)
    check_weights(w, reference_weights(q, lse.t().cpu(), kc, table, lens, cu, 64, 4, D ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_a_step_from_rotation_to_eviction(captured):
    """Two sequences, a prompt in two chunks each: rotated into the cache, attended over it, the weights summed over both
    chunks; evicted; then three more tokens over what is left, at the positions that they have without eviction."""
    H, Hkv, D, block, keep, sinks, recent = 4, 2, 64, 16, 96, 4, 20
    first, second, more = [150, 90], [60, 31], [3, 3]
    g = torch.Generator().manual_seed(17)
    f, m = fa.rope_frequencies(D, scaling="parts", factor=4)
    lens = [a + b for a, b in zip(first, second)]
    per = [-(-(n + 3) // block) for n in lens]
    nb = 40
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    table = torch.full((2, max(per)), -1, dtype=torch.int32)
    table[0, :per[0]], table[1, :per[1]] = perm[:per[0]], perm[per[0]:sum(per)]
    new = perm[sum(per):sum(per) + 14].view(2, 7)  # 112 rows each
    table, new = table.cuda(), new.contiguous().cuda()
    kc, vc = (torch.zeros(nb, Hkv, block, D, dtype=BF, device="cuda") for _ in range(2))
    weights = torch.zeros(2, Hkv, table.shape[1] * block, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    draw = lambda n: [inputs.randn((n, h, D), BF, g).cuda() for h in (H, Hkv, Hkv)]  # noqa: E731
    qkv = [draw(sum(c)) for c in (first, second, more)]
    cus = [inputs.cu_from_lengths(c).cuda() for c in (first, second, more)]
    starts = [i32([0, 0]), i32(first), i32([keep, keep])]
    ends = [i32(first), i32(lens), i32([keep + 3] * 2)]
    late = i32([n + i for n in lens for i in range(3)])

    def steps():
        out = []
        for x in range(2):
            q, k, v = qkv[x]
            q = fa.flash_rope_kv_write(q, k, v, kc, vc, table, cus[x], max(first), f, starts=starts[x], mscale=m)
            o, lse = fa.flash_attention_paged(q, kc, vc, table, cus[x], ends[x], max(first))
            fa.flash_kv_weights(q, lse, kc, table, cus[x], ends[x], max(first), weights=weights)
            out.append((q, o, lse))
        kept, left, w = fa.flash_kv_evict(kc, vc, weights, table, ends[1], new, keep, sinks, recent)
        q, k, v = qkv[2]
        q = fa.flash_rope_kv_write(q, k, v, kc, vc, new, cus[2], 3, f, starts=left, positions=late, mscale=m)
        o, lse = fa.flash_attention_paged(q, kc, vc, new, cus[2], ends[2], 3)
        return out, kept, w, (q, o, lse)

    if captured:
        steps()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            result = steps()
        weights.zero_()
        graph.replay()
    else:
        result = steps()
    fa.fa_check_device_error()
    out, kept, w, last = result
    # the definition, from the rotated rows that the cache was given
    hk, hv = kc.cpu(), vc.cpu()
    total = torch.zeros_like(weights, dtype=torch.float64, device="cpu")
    for x, (q, o, lse) in enumerate(out):
        q, cu, n = q.cpu(), cus[x].cpu(), ends[x].tolist()
        check(o, lse, reference(q, hk, hv, table.cpu(), n, cu, 0, 0, D ** -0.5), x)
        total += reference_weights(q, lse.cpu(), hk, table.cpu(), n, cu, 0, 0, D ** -0.5)
    check_weights(weights, total)
    from test_evict import chosen
    for b, n in enumerate(lens):
        for h in range(Hkv):
            want = chosen(weights[b, h, :n].tolist(), keep, sinks, recent)
            assert kept[b, h].tolist() == want
            at = torch.tensor(want)
            for c in (hk, hv):
                assert torch.equal(rows_of(c, new[b].cpu(), h, keep), rows_of(c, table[b].cpu(), h, n)[at])
            assert torch.equal(w[b, h, :keep], weights[b, h, at.cuda()]) and (w[b, h, keep:] == 0).all()
    q, o, lse = last
    check(o, lse, reference(q.cpu(), hk, hv, new.cpu(), [keep + 3] * 2, cus[2].cpu(), 0, 0, D ** -0.5))
    # at positions of its own, the third chunk's keys are those of tokens n, n + 1, n + 2
    plain = fa.flash_rope(qkv[2][1], f, late, mscale=m).cpu()
    for b in range(2):
        got = torch.stack([rows_of(hk, new[b].cpu(), h, keep + 3)[keep:] for h in range(Hkv)], 1)
        assert torch.equal(got.to(BF), plain[3 * b:3 * b + 3])


def pairs_that_see(give, n, L, window, sinks):
    """How much each of L keys receives where query t of n gives give[t] (double) to every key that it sees."""
    t, j = torch.arange(n), torch.arange(L)
    pos0 = L - n
    upto = torch.cat((torch.zeros(1, dtype=torch.float64), give.cumsum(0)))
    first = (j - pos0).clamp(0, n)  # the first query at or behind key j
    w = upto[n] - upto[first]
    if window > 0:
        last = torch.maximum((j + window - pos0).clamp(0, n), first)
        w = torch.where(j < sinks, w, upto[last] - upto[first])
    return w


@pytest.mark.gpu
@pytest.mark.parametrize("chunks,lens,H,Hkv,D,block,window,sinks", [
    ([4096], [5000], 16, 1, 64, 64, 0, 0),                # 65536 terms a key
    ([3001, 1, 700], [3001, 900, 4100], 8, 2, 128, 16, 0, 0),
    ([2048, 777], [2048, 5000], 14, 2, 64, 32, 600, 5),
    ([1500], [1400], 5, 1, 128, 128, 0, 0),               # more queries than keys
    ([2000, 300], [6000, 300], 3, 1, 128, 4, 257, 300),
])
def test_every_pair_counts_once(chunks, lens, H, Hkv, D, block, window, sinks):
    """Queries of zeros with lse 0 give exactly 1 to every key that they see, those with lse -inf nothing, so a weight is a
    count, and sums of ones are exact in fp32 up to 2^24: one pair lost or doubled among tens of thousands shows."""
    g = torch.Generator().manual_seed(sum(lens))
    q, kc, _, table, sl, cu = make(chunks, lens, H, Hkv, D, block, BF, 9)
    q.zero_()
    G, T = H // Hkv, q.shape[0]
    for gives in (torch.ones(H, T), (torch.rand(H, T, generator=g) < 0.7).float()):
        lse = torch.where(gives > 0, torch.zeros(H, T), torch.full((H, T), -math.inf))
        ref = torch.zeros(len(lens), Hkv, table.shape[1] * block, dtype=torch.float64)
        for b, (n, L) in enumerate(zip(chunks, lens)):
            for h in range(Hkv):
                give = gives[h * G:h * G + G, int(cu[b]):int(cu[b + 1])].double().sum(0)
                ref[b, h, :L] = pairs_that_see(give, n, L, window, sinks)
        args = [t.cuda() for t in (q, lse, kc, table, cu, sl)]
        w = fa.flash_kv_weights(*args, max(chunks), window, sinks)
        fa.fa_check_device_error()
        assert torch.equal(w.cpu().double(), ref)
        fa.flash_kv_weights(*args, max(chunks), window, sinks, weights=w)
        assert torch.equal(w.cpu().double(), 2 * ref)


def test_pairs_that_see():
    for n, L, window, sinks in ((5, 9, 0, 0), (9, 5, 0, 0), (7, 20, 3, 2), (1, 1, 1, 0), (9, 5, 2, 1)):
        give = torch.arange(1, n + 1, dtype=torch.float64)
        seen = visible_behind(n, L, window, sinks).double()
        assert torch.equal(pairs_that_see(give, n, L, window, sinks), give @ seen)


@pytest.mark.gpu
@pytest.mark.parametrize("chunks,lens,group", [([32], [200], 4), ([1, 1], [900, 50], 8), ([500, 33], [900, 33], 7), ([2000], [2100], 4)])
def test_error_of_exact_scores(chunks, lens, group):
    """q and k of few bits, so that products and their sums are exact however they are added, and scale 1/8. What is left of
    a term's error: the exponent x = s log2(e) / 8 - lse log2(e), whose two products and their constants are rounded to
    2^-24 each and whose sum to 2^-24 of itself, times ln 2; and 2^x, 2^-22 of itself. A weight is joined from 8 running
    sums of 32 terms every second step, 2^-24 each and for the joins."""
    D, H = 64, 2 * group
    g = torch.Generator().manual_seed(group)
    _, kc, _, table, sl, cu = make(chunks, lens, H, 2, D, 16, BF, 5)
    q = (torch.randint(-4, 5, (sum(chunks), H, D), generator=g) / 4).to(BF)
    kc = (torch.randint(-4, 5, kc.shape, generator=g) / 4).to(BF)
    lse = true_lse(q, kc, table, lens, cu, 0, 0, 0.125)
    w = fa.flash_kv_weights(*(t.cuda() for t in (q, lse, kc, table, cu, sl)), max(chunks), scale=0.125)
    fa.fa_check_device_error()
    ref = reference_weights(q, lse, kc, table, lens, cu, 0, 0, 0.125)
    s = D / 8 * 1.4426951  # the largest score there can be, in powers of two
    z = float(lse.abs().max()) * 1.4426951
    tile = min(max(chunks), 128 // group)
    steps = max(-(-n // tile) for n in chunks) + 1
    bound = math.log(2) * (2 * s + 2 * z + s + z) * 2.0 ** -24 + 2.0 ** -22 + (32 * -(-steps // 2) + 4) * 2.0 ** -24
    off = (w.double().cpu() - ref).abs()
    assert (off <= bound * ref + 1e-37).all(), (float((off / (ref + 1e-30)).max()), bound)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks,block", [(0, 0, 16), (60, 5, 16), (60, 0, 128), (200, 140, 64), (33, 4, 4)])
def test_rows_of_128_columns_that_nobody_sees(window, sinks, block):
    """NaNs in them, in pages that do not exist, and in queries and lse of no chunk change no bit of the result."""
    chunks, lens, D = [20, 3, 140], [333, 1000, 500], 128
    q, kc, _, table, sl, cu = make(chunks, lens, 6, 2, D, block, BF, 8, pad=9)
    lse = torch.zeros(6, q.shape[0])
    lse[:, :163] = true_lse(q[:163], kc, table, lens, cu, window, sinks, D ** -0.5)
    ref = reference_weights(q, lse, kc, table, lens, cu, window, sinks, D ** -0.5)
    call = lambda *a: fa.flash_kv_weights(*(t.cuda() for t in a), 150, window, sinks)  # noqa: E731
    clean = call(q, lse, kc, table, cu, sl)
    check_weights(clean, ref)
    q[163:], lse[:, 163:] = math.nan, math.nan
    seen_rows = torch.zeros(kc.shape[0], block, dtype=torch.bool)
    for b, (n, L) in enumerate(zip(chunks, lens)):
        seen = visible_behind(n, L, window, sinks).any(0)
        at = torch.nonzero(seen).flatten()
        seen_rows[table[b][at // block].long(), at % block] = True
        for x in range(-(-L // block)):
            if not seen[x * block:(x + 1) * block].any():
                table[b, x] = 1 << 30
    kc.masked_fill_(~seen_rows[:, None, :, None], math.nan)
    assert torch.equal(call(q, lse, kc, table, cu, sl), clean)
    fa.fa_check_device_error()


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 40])
def test_a_table_much_wider_than_the_sequences(window):
    """Weights that are put (add = 0): zeros in all of the table's other places, an odd number of them."""
    lens, H, Hkv, D, block, wide = [700, 0, 33], 4, 2, 64, 1, 70001
    chunks = [5, 0, 33]
    q, kc, _, table, sl, cu = make(chunks, lens, H, Hkv, D, block, BF, 12)
    lse = true_lse(q, kc, table, lens, cu, window, 0, D ** -0.5)
    ref = reference_weights(q, lse, kc, table, lens, cu, window, 0, D ** -0.5)
    far = torch.full((3, wide), -1, dtype=torch.int32)
    far[:, :table.shape[1]] = table
    old = torch.full((3 * Hkv * wide + 2,), math.nan, device="cuda")
    w = old[1:-1].view(3, Hkv, wide)
    fa.fa_kv_weights(*(t.cuda() for t in (q, lse, kc, far, cu, sl)), w, 33, window, add=False)
    fa.fa_check_device_error()
    check_weights(w[:, :, :table.shape[1]], ref)
    assert (w[:, :, 700:] == 0).all() and torch.isnan(old[0]) and torch.isnan(old[-1])


@pytest.mark.gpu
def test_streams():
    """stream= of the weights (both forms) and of the write ahead of them: behind what is queued on the current stream."""
    lens, chunks, H, Hkv, D, block = [900, 400], [20, 7], 4, 2, 64, 16
    q, kc, vc, table, sl, cu = (t.cuda() for t in make(chunks, lens, H, Hkv, D, block, BF, 14))
    f, _ = fa.rope_frequencies(D)
    g = torch.Generator().manual_seed(3)
    k, v = (inputs.randn((27, Hkv, D), BF, g).cuda() for _ in range(2))
    starts = sl - torch.tensor(chunks, dtype=torch.int32, device="cuda")

    ref_k, ref_v = kc.clone(), vc.clone()
    qr = fa.flash_rope_kv_write(q, k, v, ref_k, ref_v, table, cu, 20, f, starts)
    o, lse = fa.flash_attention_paged(qr, ref_k, ref_v, table, cu, sl, 20)
    w = fa.flash_kv_weights(qr, lse, ref_k, table, cu, sl, 20)
    ref = qr, o, lse, w, fa.flash_kv_weights(qr, lse, ref_k, table, cu, sl, 20, weights=w.clone())
    torch.cuda.synchronize()
    for raw in (False, True):
        side = torch.cuda.Stream()
        a, b, x = kc.clone(), vc.clone(), torch.empty_like(q)
        torch.cuda._sleep(2_000_000)
        x.copy_(q)  # still to come when the calls on the other stream are made
        kw = {"stream": side.cuda_stream if raw else side}
        qr = fa.flash_rope_kv_write(x, k, v, a, b, table, cu, 20, f, starts, **kw)
        o, lse = fa.flash_attention_paged(qr, a, b, table, cu, sl, 20, **kw)
        w = fa.flash_kv_weights(qr, lse, a, table, cu, sl, 20, **kw)
        with torch.cuda.stream(side):
            twice = w.clone()
        got = fa.flash_kv_weights(qr, lse, a, table, cu, sl, 20, weights=twice, **kw)
        assert got is twice
        side.synchronize()
        for n, (y, z) in enumerate(zip((qr, o, lse, w, twice, a, b), (*ref, ref_k, ref_v))):
            assert torch.equal(y, z), (raw, n)
        # the entry points themselves take the stream too
        again = torch.empty_like(w)
        side.wait_stream(torch.cuda.current_stream())
        fa.fa_kv_weights(qr, lse, a, table, cu, sl, again, 20, add=False, **kw)
        fa.fa_rope_kv_write(x, k, v, qr, a, b, table, cu, 20, f, starts, **kw)
        side.synchronize()
        assert torch.equal(again, w) and torch.equal(qr, ref[0]) and torch.equal(a, ref_k)
    fa.fa_check_device_error()
