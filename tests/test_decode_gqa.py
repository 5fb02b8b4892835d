"""One-token attention with shared key heads, a sliding window and sinks over
the paged 16-bit cache (fa_decode_paged_window) and the 4-bit cache
(fa_decode_paged_q4), against their definition in 64 bits."""
import math

import pytest
import torch

import exact_attention_54_gb300 as fa
import plain_ops
from exact_attention_54_gb300 import build as fabuild
from exact_attention_54_gb300 import inputs
from plain_ops import assert_attention_close

NULL, SHAPE, HEADDIM, DTYPE, ALIGN, SPLITS, SCALE = -1, -2, -3, -4, -5, -6, -7
A, MIS = 0x10000, 0x10008


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


# -------------------------------------------------------------- on the CPU --

@pytest.mark.parametrize("q4", [False, True])
def test_validation(lib, q4):
    cache = ("kc", "ks", "vc", "vs") if q4 else ("kc", "vc")

    def call(B=2, H=8, Hkv=2, D=128, nb=64, bs=16, mb=8, S=4, window=100, sinks=4, scale=0.1, dtype=1, **kw):
        ptr = {n: kw.get(n, A) for n in ("q", *cache, "bt", "sl", "o", "lse", "op", "mp", "lp", "cnt")}
        f = lib.fa_decode_paged_q4 if q4 else lib.fa_decode_paged_window
        return f(*ptr.values(), B, H, Hkv, D, nb, bs, mb, S, window, sinks, scale, dtype, None)

    for n in ("q", *cache, "bt", "sl", "o", "lse", "op", "mp", "lp", "cnt"):
        assert call(**{n: None}) == NULL, n
    assert call(dtype=2) == DTYPE
    for d in (32, 96, 256):
        assert call(D=d) == HEADDIM
    for kw in ({"B": 0}, {"H": 0}, {"Hkv": 0}, {"Hkv": 3}, {"H": 2, "Hkv": 4}, {"nb": 0}, {"bs": 0}, {"bs": 24},
               {"bs": 2048}, {"mb": 0}, {"mb": 1 << 27}, {"window": -1}, {"sinks": -1}, {"B": 1 << 20, "H": 1 << 10}):
        assert call(**kw) == SHAPE, kw
    if q4:  # rows in sixteens past 32 bits
        assert call(nb=1 << 26, Hkv=1, bs=1024) == SHAPE
    for s in (0, -1, 1025):
        assert call(S=s) == SPLITS
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == SCALE
    for n in ("q", *cache, "o", "op"):
        assert call(**{n: MIS}) == ALIGN, n
    for n in ("bt", "sl", "lse", "mp", "lp", "cnt"):
        assert call(**{n: A + 2}) == ALIGN, n


def test_splits(lib):
    for bad in ((0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (-1, -1, -1, -1)):
        assert fa.fa_decode_splits(*bad) == 1
    for args in ((1, 1, 1, 1), (1, 8, 8, 1 << 30), (64, 32, 8, 8192), (1 << 15, 1 << 10, 1 << 10, 5)):
        assert 1 <= fa.fa_decode_splits(*args) <= fa.FA_MAX_SPLITS


def test_binding_refuses():
    q = torch.zeros(2, 6, 1, 64, dtype=torch.float16)
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    bt, sl = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    call = lambda q=q, k=kc, v=kc, bt=bt, sl=sl, **kw: fa.flash_decode_paged_window(q, k, v, bt, sl, 10, 1, **kw)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(TypeError, match="v_cache"):
        call(v=kc.bfloat16())
    with pytest.raises(ValueError, match="k_cache"):
        call(k=kc[..., :32].contiguous())
    with pytest.raises(ValueError, match="block_table"):
        call(bt=bt[:1])
    with pytest.raises(TypeError, match="seq_lens"):
        call(sl=sl.long())
    with pytest.raises(ValueError, match="q must"):
        call(q=q[:, :, 0])
    with pytest.raises(ValueError, match="o_part"):
        call(num_splits=4, workspace=(torch.zeros(10), torch.zeros(48), torch.zeros(48), torch.zeros(12, dtype=torch.int32)))
    with pytest.raises(ValueError, match="counters"):
        call(num_splits=1, workspace=(torch.zeros(2 * 6 * 64), torch.zeros(12), torch.zeros(12), torch.zeros(4, dtype=torch.int32)))
    c = fa.kv_cache_q4(4, 2, 16, 64, torch.bfloat16, device="cpu")
    with pytest.raises(TypeError, match="k_scales"):
        fa.flash_decode_paged_q4(q, c, bt, sl)


# -------------------------------------------------------------- on the GPU --

def make(B, H, Hkv, D, block, lens, dtype, q4, seed):
    """q, the cache (every row no sequence reaches holds NaNs), table and lengths (CPU)."""
    q, kc, vc, table, sl = inputs.make_paged(B, Hkv, D, block, lens, dtype, seed)
    q = inputs.randn((B, H, 1, D), dtype, torch.Generator().manual_seed(seed + 1))
    used = torch.zeros(kc.shape[0], block, dtype=torch.bool)
    for b, n in enumerate(lens):
        for x in range(-(-n // block)):
            used[int(table[b, x]), :min(block, n - x * block)] = True
    hole = ~used[:, None, :, None]
    if not q4:
        return q, (kc.masked_fill(hole, math.nan), vc.masked_fill(hole, math.nan)), table, sl
    cache = []
    for x in (kc, vc):
        n, s = plain_ops.q4_quantise(x)
        cache += [plain_ops.q4_pack(n).masked_fill(hole, 255), s.masked_fill(hole, math.nan)]
    return q, tuple(cache), table, sl


def values(cache, q4, G):
    def f(page, h):
        if q4:
            return (plain_ops.q4_values(cache[0][page, h // G], cache[1][page, h // G]),
                    plain_ops.q4_values(cache[2][page, h // G], cache[3][page, h // G]),
                    cache[3][page, h // G].double().repeat_interleave(32, -1))
        v = cache[1][page, h // G].double()
        return cache[0][page, h // G].double(), v, torch.zeros_like(v)
    return f


def run(q, cache, table, sl, window, sinks, q4, **kw):
    dev = tuple(t.cuda() for t in cache)
    if q4:
        return fa.flash_decode_paged_q4(q.cuda(), fa.KVCacheQ4(*dev), table.cuda(), sl.cuda(), window, sinks, **kw)
    return fa.flash_decode_paged_window(q.cuda(), *dev, table.cuda(), sl.cuda(), window, sinks, **kw)


CASES = [
    # H, Hkv, D, block, lens, dtype, window, sinks, splits
    (1, 1, 64, 16, [1], torch.float16, 0, 0, 1),
    (8, 8, 128, 16, [1000, 1, 0, 257], torch.bfloat16, 0, 0, 8),
    (8, 2, 128, 16, [1000, 33, 0, 500], torch.bfloat16, 256, 4, None),
    (6, 2, 64, 64, [64, 65, 777], torch.float16, 100, 1, 3),
    (14, 2, 64, 32, [200, 777], torch.float16, 256, 4, None),
    (16, 1, 128, 16, [300, 15, 16, 17], torch.float16, 1, 0, 2),       # the newest key only
    (12, 1, 128, 16, [300, 150], torch.bfloat16, 1, 20, 5),             # and sinks over two tiles
    (40, 2, 64, 16, [100, 90], torch.bfloat16, 37, 3, 4),               # 20 heads to a key head
    (4, 4, 128, 1, [37, 5], torch.float16, 9, 2, 37),                   # pages of one key
    (4, 2, 128, 4, [130, 61], torch.bfloat16, 50, 6, 3),                # pages shorter than 16 keys
    (4, 1, 64, 1024, [1500, 1024, 1025], torch.float16, 700, 130, 4),
    (2, 2, 128, 16, [40, 41], torch.bfloat16, 30, 1000, 6),             # sinks past the window: every key
    (2, 1, 64, 16, [100, 99], torch.float16, 10 ** 9, 10 ** 9, 1024),   # more partitions than keys
    (5, 5, 128, 256, [2000], torch.bfloat16, 2 ** 31 - 1, 0, None),
    (24, 3, 128, 128, [3000, 129], torch.float16, 0, 0, None),
]


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
@pytest.mark.parametrize("H,Hkv,D,block,lens,dtype,window,sinks,splits", CASES)
def test_matches_definition(q4, H, Hkv, D, block, lens, dtype, window, sinks, splits):
    q, cache, table, sl = make(len(lens), H, Hkv, D, block, lens, dtype, q4, seed=sum(lens) + H)
    o, lse = run(q, cache, table, sl, window, sinks, q4, num_splits=splits)
    fa.fa_check_device_error()
    ref = plain_ops.decode(q, values(cache, q4, H // Hkv), table, lens, block, window, sinks, D ** -0.5)
    assert_attention_close(o, lse, *ref, dtype)


DEALT = [
    # H, Hkv, D, lens, dtype, window, sinks, splits: tables with room for 46080 keys a sequence and at least 10 units,
    # 28000 tiles of 16 keys: over 32 for each of the 608 CTAs that 152 SMs hold, so runs of tiles are dealt out
    (16, 2, 128, [0, 5, 3000, 700, 1], torch.bfloat16, 0, 0, None),
    (4, 2, 64, [3000, 2800, 3000, 3000, 2999], torch.float16, 0, 0, 2),        # runs as long as a unit
    (2, 2, 128, [0, 0, 0, 0, 0], torch.float16, 0, 0, 5),
    (20, 1, 64, [2500, 0, 60, 1024, 1025, 2047, 31, 33, 3], torch.bfloat16, 45000, 700, 7),  # 20 heads to a key head
    (10, 10, 128, [4000], torch.bfloat16, 45000, 9, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
@pytest.mark.parametrize("H,Hkv,D,lens,dtype,window,sinks,splits", DEALT)
def test_tiles_dealt_out_over_one_wave(q4, H, Hkv, D, lens, dtype, window, sinks, splits):
    block = 1024
    q, cache, table, sl = make(len(lens), H, Hkv, D, block, lens, dtype, q4, seed=sum(lens) + H)
    table = torch.nn.functional.pad(table, (0, 45 - table.shape[1]), value=-1)
    o, lse = run(q, cache, table, sl, window, sinks, q4, num_splits=splits)
    fa.fa_check_device_error()
    ref = plain_ops.decode(q, values(cache, q4, H // Hkv), table, lens, block, window, sinks, D ** -0.5)
    assert_attention_close(o, lse, *ref, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
@pytest.mark.parametrize("B", [512, 513])
def test_many_sequences(q4, B):
    """As many sequences as the dealing out holds, and one more."""
    H, Hkv, D, block = 2, 1, 64, 64
    lens = [(37 * b) % 150 for b in range(B)]
    q, cache, table, sl = make(B, H, Hkv, D, block, lens, torch.float16, q4, seed=B)
    table = torch.nn.functional.pad(table, (0, 12 - table.shape[1]), value=-1)
    o, lse = run(q, cache, table, sl, 0, 0, q4, num_splits=3)
    fa.fa_check_device_error()
    ref = plain_ops.decode(q, values(cache, q4, H // Hkv), table, lens, block, 0, 0, D ** -0.5)
    assert_attention_close(o, lse, *ref, torch.float16)


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_two_calls_at_once_and_pages_shared(q4):
    """Two streams, each with its own workspace; sequences that share a prefix's pages; the same call twice gives
    the same bits."""
    H, Hkv, D, block, lens = 8, 2, 128, 16, [900, 900, 640]
    q, cache, table, sl = make(3, H, Hkv, D, block, lens, torch.bfloat16, q4, seed=17)
    table[1, :30] = table[0, :30]
    ref = plain_ops.decode(q, values(cache, q4, H // Hkv), table, lens, block, 0, 0, D ** -0.5)
    dev = tuple(t.cuda() for t in cache)
    qd, td, sd = q.cuda(), table.cuda(), sl.cuda()
    f = (lambda: fa.flash_decode_paged_q4(qd, fa.KVCacheQ4(*dev), td, sd)) if q4 else \
        (lambda: fa.flash_decode_paged_window(qd, *dev, td, sd, 0))
    torch.cuda.synchronize()
    streams, out = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            out.append(f())
    torch.cuda.synchronize()
    fa.fa_check_device_error()
    assert_attention_close(*out[0], *ref, torch.bfloat16)
    assert all(torch.equal(a, b) for x in out[1:] for a, b in zip(x, out[0]))


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_sizes_of_values(q4, dtype):
    """Value rows (and whole heads) whose sizes differ by many powers of two, large scores, and scales far from 1."""
    H, Hkv, D, block, lens = 8, 2, 128, 16, [400, 130]
    q, kc, vc, table, sl = inputs.make_paged(2, Hkv, D, block, lens, dtype, 3)
    g = torch.Generator().manual_seed(4)
    q = inputs.randn((2, H, 1, D), torch.float32, g) * torch.tensor([1, 1e-3, 8, 1, 0.1, 3, 1, 1])[None, :, None, None]
    q = q.to(dtype)
    lo = -6 if dtype == torch.float16 else -30  # fp16: small values are still normal numbers
    vc = (vc.float() * torch.exp2(torch.randint(lo, 8, vc.shape[:3] + (1,), generator=g).float())).to(dtype)
    cache = (kc, vc)
    if q4:
        (nk, sk), (nv, sv) = plain_ops.q4_quantise(kc), plain_ops.q4_quantise(vc)
        cache = (plain_ops.q4_pack(nk), sk, plain_ops.q4_pack(nv), sv)
    for scale in (D ** -0.5, 0.5):
        o, lse = run(q, cache, table, sl, 200, 4, q4, scale=scale)
        ref = plain_ops.decode(q, values(cache, q4, H // Hkv), table, lens, block, 200, 4, scale)
        # scores up to 0.5 * 8 * 128 * 4: their fp32 error is that of sum |q k| scale, at most 2^-24 * 16 * 2000
        # relative in a weight and absolute in LSE, so both bounds are widened by it
        wide = 2.0 ** -24 * 16 * 2000 if scale == 0.5 else 2.0 ** -24 * 16 * 400
        ro, rl, size, low = ref
        h = plain_ops.half_step(dtype)
        tiny = torch.finfo(dtype).smallest_normal * 2 * h
        err = (o.double().cpu().view(ro.shape) - ro).abs()
        assert (err <= h * ro.abs() * 1.01 + (2.0 ** -13 + 2 * wide) * size + low * 1.01 + tiny).all()
        assert ((lse.double().cpu() - rl).abs() <= 4e-5 + wide + 2.0 ** -21 * rl.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_hidden_keys_may_be_nan_and_their_pages_invalid(q4):
    H, Hkv, D, block, lens = 4, 2, 128, 16, [200, 100]
    q, cache, table, sl = make(2, H, Hkv, D, block, lens, torch.bfloat16, q4, seed=9)
    base = run(q, cache, table, sl, 37, 3, q4)
    cache = [t.clone() for t in cache]
    for b, n in enumerate(lens):
        for key in range(3, n - 37):
            for t in cache:
                t[int(table[b, key // block]), :, key % block] = 255 if t.dtype == torch.uint8 else math.nan
        for x in range(1, (n - 37) // block):
            table[b, x] = -5
    got = run(q, tuple(cache), table, sl, 37, 3, q4)
    fa.fa_check_device_error()
    assert torch.equal(got[0], base[0]) and torch.equal(got[1], base[1])


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_nan_stays_in_its_head(q4):
    """A NaN in a visible value, key or query makes its own head's output NaN and no other's."""
    H, Hkv, D, block, lens = 4, 2, 64, 16, [90]
    q, cache, table, sl = make(1, H, Hkv, D, block, lens, torch.float16, q4, seed=10)
    base = run(q, cache, table, sl, 0, 0, q4)[0].cpu()
    bad = [t.clone() for t in cache]
    bad[1 if q4 else 0][int(table[0, 2]), 1, 5] = math.nan  # a key of key head 1
    o, lse = (t.cpu() for t in run(q, tuple(bad), table, sl, 0, 0, q4))
    assert torch.equal(o[:, :2], base[:, :2]) and torch.isnan(o[:, 2:]).all() and torch.isnan(lse[:, 2:]).all()
    q2 = q.clone()
    q2[0, 1, 0, 3] = math.nan
    o = run(q2, cache, table, sl, 0, 0, q4)[0].cpu()
    assert torch.isnan(o[:, 1]).all() and torch.equal(o[:, [0, 2, 3]], base[:, [0, 2, 3]])


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_bad_visible_page_is_skipped_and_reported(q4):
    H, Hkv, D, block, lens = 4, 2, 128, 16, [64, 64]
    q, cache, table, sl = make(2, H, Hkv, D, block, lens, torch.bfloat16, q4, seed=11)
    good = table.clone()
    table[1, 3] = 10 ** 6
    o, lse = run(q, cache, table, sl, 0, 0, q4)
    with pytest.raises(fa.FAError) as e:
        fa.fa_check_device_error()
    assert e.value.status == -11
    want = plain_ops.decode(q[1:], values(cache, q4, 2), good[1:], [48], block, 0, 0, D ** -0.5)
    assert_attention_close(o[1:], lse[1:], *want, torch.bfloat16)
    want = plain_ops.decode(q[:1], values(cache, q4, 2), good[:1], [64], block, 0, 0, D ** -0.5)
    assert_attention_close(o[:1], lse[:1], *want, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_lengths_are_clamped_to_the_table(q4):
    q, cache, table, sl = make(2, 4, 2, 64, 16, [48, 48], torch.float16, q4, seed=12)
    base = run(q, cache, table, sl, 20, 2, q4)
    got = run(q, cache, table, torch.tensor([10 ** 9, 2 ** 31 - 1], dtype=torch.int32), 20, 2, q4)
    assert torch.equal(got[0], base[0]) and torch.equal(got[1], base[1])
    o, lse = run(q, cache, table, torch.tensor([-3, 0], dtype=torch.int32), 20, 2, q4)
    fa.fa_check_device_error()
    assert torch.equal(o.cpu(), torch.zeros_like(q)) and (lse == -math.inf).all()


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_captured_and_replayed_with_one_workspace(q4):
    """Two graphs share a workspace; replayed in turn with new contents, each gives the eager result, and the
    counters are zero again."""
    H, Hkv, D, block, lens = 8, 2, 128, 16, [700, 300]
    q, cache, table, sl = make(2, H, Hkv, D, block, lens, torch.bfloat16, q4, seed=13)
    S = 16
    ws = (torch.full((2, H, S, D), math.nan, device="cuda"), torch.full((2, H, S), math.nan, device="cuda"),
          torch.full((2, H, S), math.nan, device="cuda"), torch.zeros(2 * H, dtype=torch.int32, device="cuda"))
    dev = tuple(t.cuda() for t in cache)
    qd, td, sd = q.cuda(), table.cuda(), sl.cuda()
    f = (lambda w: fa.flash_decode_paged_q4(qd, fa.KVCacheQ4(*dev), td, sd, w, 4, workspace=ws)) if q4 else \
        (lambda w: fa.flash_decode_paged_window(qd, *dev, td, sd, w, 4, workspace=ws))
    f(100)
    torch.cuda.synchronize()
    graphs = []
    for w in (100, 0):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f(w)
        graphs.append((g, w, out))
    for n in ([700, 300], [1, 0], [33, 299]):
        sd.copy_(torch.tensor(n, dtype=torch.int32))
        qd.copy_(inputs.randn((2, H, 1, D), torch.bfloat16, torch.Generator().manual_seed(n[0])))
        for g, w, out in graphs:
            g.replay()
            got = [t.clone() for t in out]
            want = f(w)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    fa.fa_check_device_error()
    assert int(ws[3].abs().sum()) == 0


@pytest.mark.gpu
def test_written_cache_decodes_like_what_is_read_back():
    """Write, read back and decode together: the 4-bit decode sees what the cache stands for; decoding the
    rows read back (rounded to 16 bits) over a 16-bit cache differs by that rounding only."""
    B, H, Hkv, D, block, dtype = 3, 8, 2, 128, 16, torch.float16
    lens = [150, 16, 77]
    g = torch.Generator().manual_seed(20)
    cu = inputs.cu_from_lengths(lens)
    T = int(cu[-1])
    k, v = inputs.randn((T, Hkv, D), dtype, g).cuda(), inputs.randn((T, Hkv, D), dtype, g).cuda()
    q = inputs.randn((B, H, 1, D), dtype, g)
    _, _, _, table, sl = inputs.make_paged(B, 1, 1, block, lens, dtype, 21)
    nb = sum(-(-n // block) for n in lens) + 3
    cache = fa.kv_cache_q4(nb, Hkv, block, D, dtype)
    td, cud = table.cuda(), cu.cuda()
    # prompts but for the last token, then the last token by itself
    first = [n - 1 for n in lens]
    keep = torch.cat([torch.arange(int(cu[b]), int(cu[b + 1]) - 1) for b in range(B)]).cuda()
    last = (cu[1:] - 1).long().cuda()
    fa.flash_kv_write_q4(k[keep], v[keep], cache, td, inputs.cu_from_lengths(first).cuda(), max(first))
    fa.flash_kv_write_q4(k[last], v[last], cache, td, torch.arange(B + 1, dtype=torch.int32, device="cuda"), 1,
                         starts=torch.tensor(first, dtype=torch.int32, device="cuda"))
    kr, vr = fa.flash_kv_read_q4(cache, td, cud, T, max(lens))
    o, lse = fa.flash_decode_paged_q4(q.cuda(), cache, td, sl.cuda(), 60, 4)
    fa.fa_check_device_error()
    cpu = tuple(t.cpu() for t in cache)
    ref = plain_ops.decode(q, values(cpu, True, H // Hkv), table, lens, block, 60, 4, D ** -0.5)
    assert_attention_close(o, lse, *ref, dtype)
    n, s = plain_ops.q4_quantise(k.cpu())
    assert torch.equal(kr.cpu(), plain_ops.q4_values(plain_ops.q4_pack(n), s).float().to(dtype))
    n, s = plain_ops.q4_quantise(v.cpu())
    assert torch.equal(vr.cpu(), plain_ops.q4_values(plain_ops.q4_pack(n), s).float().to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
def test_pages_past_4_gb(q4):
    """The same pages at the start of a small cache and at the end of one whose arrays pass 2^32 bytes."""
    H, Hkv, D, block, lens = 8, 8, 128, 16, [100, 65]
    q, cache, table, sl = make(2, H, Hkv, D, block, lens, torch.bfloat16, q4, seed=23)
    base = run(q, cache, table, sl, 0, 0, q4)
    n = cache[0].shape[0]
    page_bytes = cache[0][0].numel() * cache[0].element_size()
    blocks = (1 << 32) // page_bytes + 1000
    big = []
    for t in cache:
        x = torch.empty((blocks,) + t.shape[1:], dtype=t.dtype, device="cuda")
        x[-n:] = t.cuda()
        big.append(x)
    far = torch.where(table >= 0, table + (blocks - n), table).to(torch.int32).cuda()
    if q4:
        c = fa.KVCacheQ4(*big)
        got = fa.flash_decode_paged_q4(q.cuda(), c, far, sl.cuda())
        # and rows written and read there
        k, v = (inputs.randn((165, Hkv, D), torch.bfloat16, torch.Generator().manual_seed(i)).cuda() for i in (24, 25))
        cu = inputs.cu_from_lengths(lens).cuda()
        fa.flash_kv_write_q4(k, v, c, far, cu, 100)
        small = fa.KVCacheQ4(*(t.cuda() for t in cache))
        fa.flash_kv_write_q4(k, v, small, table.cuda(), cu, 100)
        for a, b in zip(c, small):
            assert torch.equal(a[-n:].view(torch.uint8), b.view(torch.uint8))
        for a, b in zip(fa.flash_kv_read_q4(c, far, cu, 165, 100), fa.flash_kv_read_q4(small, table.cuda(), cu, 165, 100)):
            assert torch.equal(a, b)
    else:
        got = fa.flash_decode_paged_window(q.cuda(), *big, far, sl.cuda(), 0)
    fa.fa_check_device_error()
    assert torch.equal(got[0], base[0]) and torch.equal(got[1], base[1])
