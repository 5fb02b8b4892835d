"""Attention of chunks of new tokens over a paged cache (fa_fwd_paged) against
its definition in 64 bits, and the calls it refuses."""
import math

import pytest
import torch

import exact_attention_54_gb300 as fa
from exact_attention_54_gb300 import build as fabuild
from exact_attention_54_gb300 import inputs
from plain_ops import half_step, softmax_attention

OK, NULL, SHAPE, HEADDIM, DTYPE, ALIGN, SCALE, WORKSPACE = 0, -1, -2, -3, -4, -5, -7, -12
TIMEOUT, DEV_INDEX, DEV_SEQLENS = -9, -11, -13
A, MIS = 0x10000, 0x10008


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


def visible_behind(nq, nk, window, sinks):
    """[nq, nk]: query i is at position nk - nq + i."""
    i, j = torch.arange(nk - nq, nk)[:, None], torch.arange(nk)[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks) | (window == 0))


def rows_of(cache, pages, h, n):
    """First n rows (double) of one head of a sequence with these pages."""
    block = cache.shape[2]
    return cache[pages[:-(-n // block)].long(), h].reshape(-1, cache.shape[3])[:n].double()


def reference(q, kc, vc, table, lens, cu, window, sinks, scale):
    """o, lse and the bound of o's error. Roundings: o once (h, half a step); P before P V (h; below fp16's normal
    numbers 2^-25 each, of a sum l of at least 1); scores, 2^x and sums in fp32: 2^-13 of what meets in o, as in
    plain_ops.window_attention; joining parts adds a few 2^-22."""
    T, H, D = q.shape
    G, h = H // kc.shape[1], half_step(q.dtype)
    tiny = torch.finfo(q.dtype).smallest_normal * h
    o, bound = torch.zeros(T, H, D, dtype=torch.float64), torch.zeros(T, H, D, dtype=torch.float64)
    lse = torch.full((H, T), -math.inf, dtype=torch.float64)
    for b in range(len(lens)):
        n, L = int(cu[b + 1] - cu[b]), int(lens[b])
        if n == 0 or L == 0:
            continue
        seen = visible_behind(n, L, window, sinks)
        sl = slice(int(cu[b]), int(cu[b + 1]))
        for hk in range(kc.shape[1]):
            k, v = rows_of(kc, table[b], hk, L), rows_of(vc, table[b], hk, L)
            dead = ~seen.any(0)
            k[dead], v[dead] = 0.0, 0.0
            for g in range(hk * G, hk * G + G):
                r, l, p, size = softmax_attention(q[sl, g].double(), k, v, seen, scale)
                o[sl, g], lse[g, sl] = r, l
                bound[sl, g] = h * r.abs() * (1 + 2 * h) + (h * (1 + h) + 2.0 ** -13) * size + \
                    tiny * (seen.double() @ v.abs()) + 2 * tiny
    return o, lse, bound


def check(o, lse, ref, what=""):
    ro, rl, bound = ref
    o, lse = o.double().cpu(), lse.double().cpu()
    bad = ~((o - ro).abs() <= bound)
    assert not bad.any(), (what, torch.nonzero(bad)[0].tolist(), int(bad.sum()),
                           float(((o - ro).abs() / bound).nan_to_num(1e9).max()))
    empty = torch.isinf(rl)
    assert torch.equal(empty, torch.isinf(lse)) and (lse[empty] == -math.inf).all(), what
    off, room = (lse - rl).abs()[~empty], (4e-5 + 2.0 ** -21 * rl.abs())[~empty]
    assert (off <= room).all(), (what, float(off.max()))


def make(chunks, lens, H, Hkv, D, block, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    _, kc, vc, table, sl = inputs.make_paged(len(lens), Hkv, D, block, lens, dtype, seed)
    q = inputs.randn((sum(chunks) + pad, H, D), dtype, g)
    return q, kc, vc, table, sl, inputs.cu_from_lengths(chunks)


def run(q, kc, vc, table, sl, cu, mx, window=0, sinks=0, **kw):
    o, lse = fa.flash_attention_paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), cu.cuda(), sl.cuda(), mx, window,
                                      sinks, **kw)
    fa.fa_check_device_error()
    return o, lse


# -------------------------------------------------------------- on the CPU --

def test_validation(lib):
    need = lib.fa_fwd_paged_workspace_bytes(64, 8, 2, 128)
    assert need >= 4 * 2 * 256 * (128 + 2)

    def call(q=A, kc=A, vc=A, bt=A, cu=A, sl=A, o=A, lse=A, ws=A, wsb=need, n=2, total=100, mx=64, H=8, Hkv=2, D=128, nb=8,
             bs=16, mb=4, window=0, sinks=0, scale=0.1, dtype=1):
        return lib.fa_fwd_paged(q, kc, vc, bt, cu, sl, o, lse, ws, wsb, n, total, mx, H, Hkv, D, nb, bs, mb, window, sinks,
                                scale, dtype, None)

    for kw in ("q", "kc", "vc", "bt", "cu", "sl", "o", "lse", "ws"):
        assert call(**{kw: None}) == NULL, kw
    assert call(dtype=2) == DTYPE
    for d in (32, 96, 256):
        assert call(D=d) == HEADDIM
    for kw in ({"n": 0}, {"total": 0}, {"mx": 0}, {"mx": (1 << 29) + 1}, {"H": 0}, {"Hkv": 0}, {"Hkv": 3}, {"nb": 0},
               {"bs": 24}, {"bs": 2048}, {"mb": 0}, {"mb": 1 << 28}, {"window": -1}, {"sinks": -1}, {"H": 258, "Hkv": 2},
               {"total": 1 << 29, "H": 16}, {"nb": 1 << 30, "Hkv": 4}):
        assert call(**kw) == SHAPE, kw
    for s in (0.0, float("nan"), float("inf"), -1.0):
        assert call(scale=s) == SCALE
    for kw in ("q", "kc", "vc", "o", "ws"):
        assert call(**{kw: MIS}) == ALIGN, kw
    for kw in ("bt", "cu", "sl", "lse"):
        assert call(**{kw: A + 2}) == ALIGN, kw
    assert call(wsb=need - 4) == WORKSPACE
    small = lib.fa_fwd_paged_workspace_bytes(4, 8, 2, 128)
    assert 0 < small < need
    for bad in ((0, 8, 2, 128), (4, 8, 3, 128), (4, 8, 2, 96), (4, 0, 1, 64), (4, 512, 2, 64)):
        assert lib.fa_fwd_paged_workspace_bytes(*bad) == 0, bad


def test_binding_refuses():
    q, c = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    bt, cu = torch.zeros(1, 4, dtype=torch.int32), torch.tensor([0, 5], dtype=torch.int32)
    sl = torch.tensor([5], dtype=torch.int32)
    call = lambda q=q, kc=c, vc=c, bt=bt, cu=cu, sl=sl: fa.flash_attention_paged(q, kc, vc, bt, cu, sl, 5)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(TypeError, match="unsupported dtype"):
        call(q=q.float())
    with pytest.raises(TypeError, match="k_cache"):
        call(kc=c.half())
    with pytest.raises(ValueError, match="v_cache"):
        call(vc=c[:, :1])
    with pytest.raises(ValueError, match="total_q,H,D"):
        call(q=q[0])
    with pytest.raises(TypeError, match="cu_seqlens_q"):
        call(cu=cu.long())
    with pytest.raises(ValueError, match="seq_lens"):
        call(sl=sl.repeat(2))
    with pytest.raises(ValueError, match="block_table"):
        call(bt=bt.repeat(2, 1))
    with pytest.raises(ValueError, match="contiguous"):
        call(q=q.transpose(0, 1).contiguous().transpose(0, 1))


# -------------------------------------------------------------- on the GPU --

BF, FP = torch.bfloat16, torch.float16


@pytest.mark.gpu
@pytest.mark.parametrize("chunks,lens,H,Hkv,D,block,window,sinks,dtype", [
    ([1], [1], 1, 1, 64, 16, 0, 0, BF),
    ([128], [128], 2, 2, 128, 16, 0, 0, BF),
    ([5, 1, 33], [300, 129, 33], 8, 2, 128, 16, 0, 0, BF),
    ([70, 0, 2], [70, 40, 513], 6, 2, 64, 32, 0, 0, FP),
    ([300], [777], 4, 1, 128, 64, 0, 0, FP),
    ([19, 37], [500, 37], 14, 2, 64, 8, 0, 0, BF),        # seven heads to a key head: 126 rows a tile
    ([40], [200], 3, 1, 128, 128, 0, 0, BF),
    ([9], [260], 128, 1, 64, 256, 0, 0, FP),              # one token a tile
    ([2, 3], [1500, 900], 16, 1, 64, 1024, 0, 0, BF),
    ([50], [400], 4, 4, 128, 1, 0, 0, BF),                # pages of 1, 2 and 4 keys
    ([50, 3], [131, 90], 4, 2, 64, 2, 0, 0, FP),
    ([7], [300], 8, 2, 128, 4, 100, 3, BF),
    ([200], [900], 4, 2, 128, 16, 1, 0, BF),              # windows
    ([200, 31], [900, 400], 4, 2, 64, 16, 128, 4, FP),
    ([257], [1300], 2, 1, 128, 32, 300, 200, BF),
    ([64], [700], 4, 1, 64, 64, 129, 129, BF),
    ([33], [600], 7, 1, 128, 16, 5000, 4, FP),            # a window past everything
    ([100], [60], 4, 2, 64, 16, 0, 0, BF),                # more queries than keys
    ([100], [60], 4, 2, 128, 16, 20, 2, FP),
    ([3, 4], [0, 10], 4, 2, 64, 16, 0, 0, BF),            # no keys
])
def test_chunk(chunks, lens, H, Hkv, D, block, window, sinks, dtype):
    q, kc, vc, table, sl, cu = make(chunks, lens, H, Hkv, D, block, dtype, sum(chunks) + sum(lens))
    o, lse = run(q, kc, vc, table, sl, cu, max(chunks), window, sinks)
    check(o, lse, reference(q, kc, vc, table, lens, cu, window, sinks, D ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("n,L,Hkv", [(3, 20001, 1), (40, 9000, 2), (1, 6000, 3)])
def test_one_long_sequence_falls_into_many_parts(n, L, Hkv):
    q, kc, vc, table, sl, cu = make([n], [L], 2 * Hkv, Hkv, 64, 64, BF, n)
    q[:, 0] *= 4  # scores whose maximum moves between parts
    kc[table[0, :3].long()] *= 0.1
    o, lse = run(q, kc, vc, table, sl, cu, n, scale=0.2)
    check(o, lse, reference(q, kc, vc, table, [L], cu, 0, 0, 0.2))
    again = run(q, kc, vc, table, sl, cu, n, scale=0.2)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("n,group,D", [(1, 1, 64), (1, 3, 128), (2, 1, 128), (1, 7, 64), (3, 5, 128), (1, 16, 64), (11, 3, 128)])
def test_parts_of_few_rows(n, group, D):
    """Rows that do not fill a warp's lanes, in up to as many parts as there are CTAs."""
    chunks, lens = [n, n], [17001, 700]
    q, kc, vc, table, sl, cu = make(chunks, lens, group, 1, D, 32, BF, n + group)
    o, lse = run(q, kc, vc, table, sl, cu, n)
    check(o, lse, reference(q, kc, vc, table, lens, cu, 0, 0, D ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [300, 5000])
def test_many_sequences(B):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 40, (B,), generator=g)
    chunks = torch.minimum(torch.randint(0, 4, (B,), generator=g), lens)
    q, kc, vc, table, sl, cu = make(chunks.tolist(), lens.tolist(), 2, 1, 64, 8, BF, B)
    o, lse = run(q, kc, vc, table, sl, cu, 3)
    check(o, lse, reference(q, kc, vc, table, lens.tolist(), cu, 0, 0, 0.125))


@pytest.mark.gpu
def test_rows_of_no_chunk_and_larger_limits():
    chunks, lens = [20, 7], [150, 90]
    q, kc, vc, table, sl, cu = make(chunks, lens, 4, 2, 64, 16, BF, 3, pad=11)
    q[27:] = math.nan
    qd, kd, vd, td, sd, cd = (t.cuda() for t in (q, kc, vc, table, sl, cu))
    o, lse = torch.full_like(qd, 3.0), torch.full((4, 38), 5.0, device="cuda")
    ws = torch.full((fa.fa_fwd_paged_workspace_bytes(64, 4, 2, 64) // 4,), math.nan, device="cuda")
    fa.fa_fwd_paged(qd, kd, vd, td, cd, sd, o, lse, ws, 64)
    fa.fa_check_device_error()
    assert (o[27:] == 3).all() and (lse[:, 27:] == 5).all()
    check(o[:27], lse[:, :27], reference(q[:27], kc, vc, table, lens, cu, 0, 0, 0.125))


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks,block", [(0, 0, 16), (60, 5, 16), (60, 0, 128), (200, 140, 64), (33, 4, 4), (40, 3, 256)])
@pytest.mark.parametrize("D", [64, 128])
def test_what_nobody_sees_may_hold_anything(window, sinks, block, D):
    chunks, lens = [20, 3, 140], [333, 1000, 500]
    q, kc, vc, table, sl, cu = make(chunks, lens, 4, 2, D, block, BF, 8)
    ref = reference(q, kc, vc, table, lens, cu, window, sinks, D ** -0.5)
    seen_rows = torch.zeros(kc.shape[0], block, dtype=torch.bool)
    for b, (n, L) in enumerate(zip(chunks, lens)):
        seen = visible_behind(n, L, window, sinks).any(0)
        at = torch.nonzero(seen).flatten()
        seen_rows[table[b][at // block].long(), at % block] = True
        for x in range(-(-L // block)):  # pages that nobody sees are not looked up
            if not seen[x * block:(x + 1) * block].any():
                table[b, x] = -7 if x % 2 else 1 << 30
    for c, bad in ((kc, math.nan), (vc, math.inf)):
        c.masked_fill_(~seen_rows[:, None, :, None], bad)
    vc[:, 0].masked_fill_(~seen_rows[:, :, None], math.nan)
    o, lse = run(q, kc, vc, table, sl, cu, 140, window, sinks)
    check(o, lse, ref)


@pytest.mark.gpu
def test_checks_on_the_device():
    chunks, lens = [20, 7], [150, 90]
    q, kc, vc, table, sl, cu = (t.cuda() for t in make(chunks, lens, 4, 2, 64, 16, BF, 3))
    ws = torch.empty(fa.fa_fwd_paged_workspace_bytes(20, 4, 2, 64) // 4, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def status(cu=cu, table=table, sl=sl, mx=20):
        o, lse = torch.full_like(q, 3.0), torch.full((4, 27), 5.0, device="cuda")
        fa.fa_fwd_paged(q, kc, vc, table, cu, sl, o, lse, ws, mx)
        try:
            fa.fa_check_device_error()
        except fa.FAError as e:
            return e.status, o, lse
        return OK, o, lse

    ok, good, good_lse = status()
    assert ok == OK
    for bad in (i32(0, 28, 27), i32(0, 20, 28), i32(-1, 20, 27), i32(20, 7, 27)):
        st, o, lse = status(cu=bad)
        assert st == DEV_SEQLENS and (o == 3).all() and (lse == 5).all()
    st, o, _ = status(mx=19)
    assert st == DEV_SEQLENS and (o == 3).all()
    for page in (-1, kc.shape[0], 1 << 30):
        t = table.clone()
        t[0, 2] = page
        st, o, _ = status(table=t)
        assert st == DEV_INDEX and torch.equal(o[20:], good[20:]) and torch.isfinite(o).all()
    # lengths are limited to the table's
    full = table.shape[1] * 16
    assert torch.equal(status(sl=i32(1 << 30, 90))[1], status(sl=i32(full, 90))[1])
    st, o, lse = status(sl=i32(-5, 90))
    assert st == OK and (o[:20] == 0).all() and (lse[:, :20] == -math.inf).all() and torch.equal(o[20:], good[20:])
    assert status()[0] == OK and torch.equal(status()[1], good)


@pytest.mark.gpu
def test_like_prefill_and_like_decode():
    """A chunk that is the whole sequence is the window prefill; one of one token is the paged decode."""
    n, H, Hkv, D = 300, 8, 2, 128
    q, kc, vc, table, sl, cu = make([n], [n], H, Hkv, D, 16, BF, 21)
    k, v = (torch.stack([rows_of(c, table[0], h, n) for h in range(Hkv)]).to(BF) for c in (kc, vc))
    for window, sinks in ((0, 0), (100, 4)):
        ref = reference(q, kc, vc, table, [n], cu, window, sinks, D ** -0.5)
        check(*run(q, kc, vc, table, sl, cu, n, window, sinks), ref)
        o, lse = fa.flash_attention_window(q.transpose(0, 1)[None].contiguous().cuda(), k[None].cuda(), v[None].cuda(),
                                           window or n, sinks)
        check(o[0].transpose(0, 1), lse[0], ref)
        one = torch.tensor([0, 1], dtype=torch.int32)
        o1, l1 = run(q[-1:], kc, vc, table, sl, one, 1, window, sinks)
        od, ld = fa.flash_decode_paged_window(q[-1:, :, None].cuda(), kc.cuda(), vc.cuda(), table.cuda(), sl.cuda(), window,
                                              sinks)
        last = tuple(t[-1:] if t.dim() == 3 else t[:, -1:] for t in ref)
        check(o1, l1, last)
        check(od[:, :, 0], ld.t(), last)


@pytest.mark.gpu
@pytest.mark.parametrize("load", [1, 3])
def test_withheld_load_ends_with_an_error(load):
    q, kc, vc, table, sl, cu = make([40], [20000], 16, 8, 64, 16, BF, 5)  # several steps in every CTA
    good = run(q, kc, vc, table, sl, cu, 40)
    fa.fa_test_withhold_load(load, 20_000_000)
    try:
        fa.flash_attention_paged(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), cu.cuda(), sl.cuda(), 40)
        with pytest.raises(fa.FAError) as e:
            fa.fa_check_device_error()
        assert e.value.status == TIMEOUT
    finally:
        fa.fa_test_withhold_load(0, 0)
    again = run(q, kc, vc, table, sl, cu, 40)
    assert torch.equal(good[0], again[0]) and torch.equal(good[1], again[1])


@pytest.mark.gpu
def test_streams_graphs_and_workspaces():
    a = [t.cuda() for t in make([20, 7], [1500, 900], 4, 2, 64, 16, BF, 3)]
    b = [t.cuda() for t in make([64], [3000], 4, 2, 64, 16, BF, 4)]
    call = lambda x, mx, **kw: fa.flash_attention_paged(*x[:4], x[5], x[4], mx, **kw)  # noqa: E731
    ra, rb = call(a, 20), call(b, 64)
    side = torch.cuda.Stream()
    got = call(a, 20, stream=side)
    also = call(b, 64)  # at the same time, with workspaces of their own
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip((*ra, *rb), (*got, *also)))
    # two graphs with one workspace, replayed in turn
    ws = torch.empty(fa.fa_fwd_paged_workspace_bytes(64, 4, 2, 64) // 4, device="cuda")
    graphs = []
    for x, mx in ((a, 20), (b, 64)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(x, mx, workspace=ws)
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((*ra, *rb), (*graphs[0][1], *graphs[1][1])))
    # longer sequences than at capture: lengths are read on the device
    a[4].copy_(torch.tensor([1400, 800], dtype=torch.int32))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(call(a, 20), graphs[0][1]))
    fa.fa_check_device_error()


@pytest.mark.gpu
def test_many_long_chunks_among_many():
    """More sequences with many query tiles than the plan's list holds: the same as in two calls of half as many."""
    B, n, H = 4200, 36, 128  # one token a tile, 18 pairs a sequence
    g = torch.Generator("cuda").manual_seed(3)
    q = torch.randn(B * n, H, 64, generator=g, device="cuda").to(BF)
    kc, vc = (torch.randn(B, 1, 64, 64, generator=g, device="cuda").to(BF) for _ in range(2))
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    sl = (torch.arange(B, device="cuda") % 29 + n).int()
    cu = (torch.arange(B + 1, device="cuda") * n).int()
    o, lse = fa.flash_attention_paged(q, kc, vc, table, cu, sl, n)
    w = fa.flash_kv_weights(q, lse, kc, table, cu, sl, n)
    half = B // 2
    for sel, rows in ((slice(0, half), slice(0, half * n)), (slice(half, B), slice(half * n, B * n))):
        part = (table[sel].contiguous(), cu[:half + 1].contiguous(), sl[sel].contiguous())
        qp = q[rows].contiguous()
        po, pl = fa.flash_attention_paged(qp, kc, vc, *part, n)
        # (units may be cut at other places: the same but for the joins' rounding)
        assert (po.float() - o[rows].float()).abs().max() <= 2.0 ** -6 and (pl - lse[:, rows]).abs().max() <= 1e-5
        assert torch.equal(fa.flash_kv_weights(qp, lse[:, rows], kc, *part, n), w[sel])
    fa.fa_check_device_error()
    want = reference(q[:n].cpu(), kc.cpu(), vc.cpu(), table.cpu(), sl[:1].cpu(), cu[:2].cpu(), 0, 0, 0.125)
    check(o[:n], lse[:, :n], want)


@pytest.mark.gpu
def test_caches_past_32_bits():
    """Pages behind 2^32 bytes and 2^31 elements of a cache: written, attended, weighed and evicted from, as in a small
    cache with the same rows."""
    Hkv, block, D, H = 8, 16, 128, 16
    count = (1 << 32) // (Hkv * block * D) + 40  # 2^32 elements and some more
    g = torch.Generator().manual_seed(6)
    big = [torch.empty(count, Hkv, block, D, dtype=BF, device="cuda") for _ in range(2)]
    small = [torch.empty(24, Hkv, block, D, dtype=BF, device="cuda") for _ in range(2)]
    far = torch.tensor([count - 1 - 3 * i for i in range(12)] + [5, (1 << 31) // (Hkv * block * D) + 1] +
                       [count - 2 - 3 * i for i in range(10)], dtype=torch.int32)
    near = torch.arange(24, dtype=torch.int32)
    n = 14 * block - 5  # keys
    q, k, v = (inputs.randn((n, h, D), BF, g).cuda() for h in (H, Hkv, Hkv))
    f, _ = fa.rope_frequencies(D)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    results = []
    for (kc, vc), pages in ((big, far), (small, near)):
        table, new = pages[None, :14].contiguous().cuda(), pages[None, 14:18].contiguous().cuda()
        qr = fa.flash_rope_kv_write(q, k, v, kc, vc, table, cu, n, f)
        o, lse = fa.flash_attention_paged(qr, kc, vc, table, cu, sl, n)
        w = fa.flash_kv_weights(qr, lse, kc, table, cu, sl, n)
        kept, left, nw = fa.flash_kv_evict(kc, vc, w, table, sl, new, 60, 2, 10)
        last = fa.flash_attention_paged(qr[-3:].contiguous(), kc, vc, new, torch.tensor([0, 3], dtype=torch.int32).cuda(),
                                        left, 3)
        fa.fa_check_device_error()
        results.append((qr, o, lse, w, kept, nw, *last))
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.gpu
def test_rows_ahead_of_the_first_chunk_and_limits_far_above():
    """cu_seqlens that begin behind row 0, and a max_seqlen_q of millions: only the chunks' rows are written."""
    chunks, lens, ahead = [20, 7], [150, 90], 9
    q, kc, vc, table, sl, cu = make(chunks, lens, 4, 2, 64, 16, BF, 3, pad=ahead + 4)
    ref = reference(q[ahead:ahead + 27], kc, vc, table, lens, cu, 0, 0, 0.125)
    q[:ahead], q[ahead + 27:] = math.nan, math.inf
    qd, kd, vd, td, sd, cd = (t.cuda() for t in (q, kc, vc, table, sl, cu + ahead))
    for mx in (20, 5_000_000):
        o, lse = torch.full_like(qd, 3.0), torch.full((4, q.shape[0]), 5.0, device="cuda")
        ws = torch.full((fa.fa_fwd_paged_workspace_bytes(mx, 4, 2, 64) // 4,), math.nan, device="cuda")
        fa.fa_fwd_paged(qd, kd, vd, td, cd, sd, o, lse, ws, mx)
        w = fa.flash_kv_weights(qd, lse, kd, td, cd, sd, mx)
        fa.fa_check_device_error()
        mine = slice(ahead, ahead + 27)
        check(o[mine], lse[:, mine], ref)
        for r in (slice(0, ahead), slice(ahead + 27, None)):
            assert (o[r] == 3).all() and (lse[:, r] == 5).all()
        assert abs(float(w.double().sum()) - 27 * 4) <= 27 * 4 * 2.0 ** -12
    # the write: rows ahead of the first sequence go nowhere
    f, _ = fa.rope_frequencies(64)
    g = torch.Generator().manual_seed(4)
    k = inputs.randn((q.shape[0], 2, 64), BF, g).cuda()
    a, b = kd.clone(), vd.clone()
    starts = sd - torch.tensor(chunks, dtype=torch.int32, device="cuda")
    qo = torch.full_like(qd, 7.0)
    fa.fa_rope_kv_write(qd, k, k, qo, a, b, td, cd, 20, f, starts)
    c, d = kd.clone(), vd.clone()
    want = fa.flash_rope_kv_write(qd[mine].contiguous(), k[mine].contiguous(), k[mine].contiguous(), c, d, td, cu.cuda(), 20, f,
                                  starts)
    fa.fa_check_device_error()
    assert torch.equal(qo[mine], want) and (qo[:ahead] == 7).all() and (qo[ahead + 27:] == 7).all()
    assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.gpu
def test_no_chunk_has_tokens():
    q, kc, vc, table, sl, _ = (t.cuda() for t in make([5], [300], 4, 2, 64, 16, BF, 3))
    for at in (0, 5):
        cu = torch.tensor([at, at], dtype=torch.int32, device="cuda")
        o, lse = torch.full_like(q, 3.0), torch.full((4, 5), 5.0, device="cuda")
        ws = torch.full((fa.fa_fwd_paged_workspace_bytes(5, 4, 2, 64) // 4,), math.nan, device="cuda")
        fa.fa_fwd_paged(q, kc, vc, table, cu, sl, o, lse, ws, 5)
        old = torch.full((1, 2, table.shape[1] * 16), math.nan, device="cuda")
        fa.fa_kv_weights(q, lse, kc, table, cu, sl, old, 5, add=False)
        more = fa.flash_kv_weights(q, lse, kc, table, cu, sl, 5, weights=torch.ones_like(old))
        fa.fa_check_device_error()
        assert (o == 3).all() and (lse == 5).all() and (old == 0).all() and (more == 1).all()


@pytest.mark.gpu
def test_queries_that_are_not_finite_stay_in_their_rows():
    chunks, lens = [40, 3], [900, 200]
    q, kc, vc, table, sl, cu = make(chunks, lens, 4, 2, 64, 16, BF, 8)
    o, lse = run(q, kc, vc, table, sl, cu, 40)
    bad = q.clone()
    bad[17, 1], bad[41, 2, 5] = math.nan, math.inf
    p, l2 = run(bad, kc, vc, table, sl, cu, 40)
    rest = torch.ones(43, 4, dtype=torch.bool)
    rest[17, 1] = rest[41, 2] = False
    assert torch.equal(p.cpu()[rest], o.cpu()[rest]) and torch.equal(l2.t().cpu()[rest], lse.t().cpu()[rest])
    assert not torch.isfinite(p.cpu()[17, 1]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("chunks,lens,H,Hkv,D,block,window,sinks,dtype", [
    ([3], [20001], 2, 1, 64, 64, 0, 0, BF),
    ([300, 1, 40], [5000, 17000, 40], 8, 2, 128, 16, 0, 0, BF),
    ([257, 64], [3000, 9000], 14, 2, 64, 32, 700, 5, FP),
    ([500], [400], 3, 1, 128, 128, 0, 0, FP),
    ([90, 200], [4000, 6000], 4, 1, 128, 4, 1025, 300, BF),
])
def test_every_key_counts_once(chunks, lens, H, Hkv, D, block, window, sinks, dtype):
    """Queries of zeros give every key that they see a weight of exactly 1, so lse is ln of their number and, with a 1 in
    column j % D of key j's value, o the share of those in each column: sums of whole numbers, exact up to 2^24. o is off by
    one reciprocal, one product (2^-23 each) and its rounding, lse by the logarithm (2^-21 of it and 2^-21)."""
    q, kc, vc, table, sl, cu = make(chunks, lens, H, Hkv, D, block, dtype, 31)
    q.zero_()
    vc.zero_()
    for b, L in enumerate(lens):
        j = torch.arange(L)
        vc[table[b][j // block].long(), :, j % block, j % D] = 1
    o, lse = run(q, kc, vc, table, sl, cu, max(chunks), window, sinks)
    o, lse = o.double().cpu(), lse.double().cpu()
    for b, (n, L) in enumerate(zip(chunks, lens)):
        seen = visible_behind(n, L, window, sinks).double()
        share = seen @ torch.nn.functional.one_hot(torch.arange(L) % D, D).double()
        count, rows = seen.sum(1), slice(int(cu[b]), int(cu[b + 1]))
        want = (share / count.clamp(min=1)[:, None])[:, None].expand(-1, H, -1)
        assert ((o[rows] - want).abs() <= want * (half_step(dtype) * (1 + 2.0 ** -20) + 2.0 ** -21)).all()
        ln = torch.log(count)[None].expand(H, -1)
        none = (count == 0)[None].expand(H, -1)
        got = lse[:, rows]
        assert (got[none] == -math.inf).all()
        assert ((got - ln).abs()[~none] <= (2.0 ** -21 * (1 + ln))[~none]).all()
