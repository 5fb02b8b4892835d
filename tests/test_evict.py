"""fa_kv_evict against its definition, exactly, and the calls it refuses."""
import math

import pytest
import torch

import exact_attention_54_gb300 as fa
from exact_attention_54_gb300 import build as fabuild
from exact_attention_54_gb300 import inputs

OK, NULL, SHAPE, HEADDIM, DTYPE, ALIGN, CUDA = 0, -1, -2, -3, -4, -5, -8
DEV_INDEX = -11
A, MIS = 0x10000, 0x10008


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


def chosen(w, keep, sinks, recent):
    """Indices that stay, of one head's weights (a list)."""
    n = len(w)
    if n <= keep:
        return list(range(n))
    rank = lambda j: -math.inf if math.isnan(w[j]) else w[j]  # noqa: E731
    # (a NaN is below -inf)
    middle = sorted(range(sinks, n - recent), key=lambda j: (math.isnan(w[j]), -rank(j), j))
    return sorted([*range(sinks), *middle[:keep - sinks - recent], *range(n - recent, n)])


# -------------------------------------------------------------- on the CPU --

def test_validation(lib):
    def call(kc=A, vc=A, w=A, bt=A, sl=A, nt=A, kept=A, nl=A, nw=A, B=2, Hkv=2, D=64, nb=8, bs=16, mb=4, nmb=2, keep=20,
             sinks=4, recent=8, dtype=1):
        return lib.fa_kv_evict(kc, vc, w, bt, sl, nt, kept, nl, nw, B, Hkv, D, nb, bs, mb, nmb, keep, sinks, recent,
                               dtype, None)

    for kw in ("kc", "vc", "w", "bt", "sl", "nt", "kept", "nl", "nw"):
        assert call(**{kw: None}) == NULL, kw
    assert call(dtype=2) == DTYPE
    for d in (32, 256):
        assert call(D=d) == HEADDIM
    for kw in ({"B": 0}, {"Hkv": 0}, {"B": 1 << 20, "Hkv": 1 << 12}, {"nb": 0}, {"bs": 12}, {"mb": 0}, {"nmb": 0},
               {"keep": 0}, {"sinks": -1}, {"recent": -1}, {"sinks": 13}, {"sinks": (1 << 31) - 1}, {"mb": 1 << 28}):
        assert call(**kw) == SHAPE, kw
    for kw in ("kc", "vc"):
        assert call(**{kw: MIS}) == ALIGN, kw
    for kw in ("w", "bt", "sl", "nt", "kept", "nl", "nw"):
        assert call(**{kw: A + 2}) == ALIGN, kw


def test_outputs_on_inputs_are_refused(lib):
    """Each of these would be written while other CTAs read it, or written twice. None gets as far as a launch: the
    sizes are good ones, so without a GPU a call with arrays apart ends at its launch."""
    B, Hkv, block, mb, nmb, keep = 2, 2, 16, 4, 2, 20
    size = {"w": B * Hkv * mb * block * 4, "bt": B * mb * 4, "sl": B * 4, "nt": B * nmb * 4, "kept": B * Hkv * keep * 4,
            "nl": B * 4, "nw": B * Hkv * nmb * block * 4}
    apart = {n: 0x100000 * (i + 1) for i, n in enumerate(size)}

    def call(**kw):
        a = {**apart, **kw}
        return lib.fa_kv_evict(A, A, a["w"], a["bt"], a["sl"], a["nt"], a["kept"], a["nl"], a["nw"], B, Hkv, 64, 8, block,
                               mb, nmb, keep, 4, 8, 1, None)

    for out in ("kept", "nl", "nw"):
        for other in size:
            if other != out:
                for at in (0, size[other] - 4, 4 - size[out]):  # the same, its last element, all but its first
                    assert call(**{out: apart[other] + at}) == SHAPE, (out, other, at)
    assert call(nt=apart["bt"]) == SHAPE
    if not torch.cuda.is_available():
        assert call() == CUDA
        for out in ("kept", "nl", "nw"):
            for at in (size["w"], -size[out]):  # side by side
                assert call(**{out: apart["w"] + at}) == CUDA, (out, at)


def test_binding_refuses():
    c = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    w, bt, nt = torch.zeros(1, 2, 64), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    sl = torch.zeros(1, dtype=torch.int32)
    call = lambda kc=c, vc=c, w=w, bt=bt, sl=sl, nt=nt, keep=20: fa.flash_kv_evict(kc, vc, w, bt, sl, nt, keep, 4, 8)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(TypeError, match="unsupported dtype"):
        call(kc=c.float(), vc=c.float())
    with pytest.raises(TypeError, match="v_cache"):
        call(vc=c.half())
    with pytest.raises(ValueError, match="weights"):
        call(w=w[:, :, :32])
    with pytest.raises(TypeError, match="weights"):
        call(w=w.double())
    with pytest.raises(ValueError, match="new_table"):
        call(nt=torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(TypeError, match="seq_lens"):
        call(sl=sl.long())
    for keep in (0, -1):
        with pytest.raises(ValueError, match="keep"):
            call(keep=keep)


def test_binding_refuses_other_dimensions():
    c = torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for kc, old, new in ((c[0, 0], bt, bt), (c, bt[0], bt), (c, bt, bt[0])):
        with pytest.raises(ValueError, match="tables"):
            fa.flash_kv_evict(kc, kc, torch.zeros(1, 2, 64), old, sl, new, 20)


def test_definition():
    w = [3.0, 1.0, 5.0, 5.0, math.nan, 5.0, 0.0, 2.0]
    assert chosen(w, 8, 1, 1) == list(range(8))
    assert chosen(w, 4, 1, 1) == [0, 2, 3, 7]
    assert chosen(w, 7, 0, 0) == [0, 1, 2, 3, 5, 6, 7]
    assert chosen(w, 3, 2, 1) == [0, 1, 7]


# -------------------------------------------------------------- on the GPU --

def setup(lens, Hkv, D, block, keep, dtype, seed, new_width=None):
    g = torch.Generator().manual_seed(seed)
    B, both = len(lens), list(lens) + [min(n, keep) for n in lens]
    table = inputs.make_paged(2 * B, 1, 1, block, both, dtype, seed)[3]
    nb = sum(-(-n // block) for n in both) + 3
    old, new = table[:B], table[B:]
    new = new[:, :new_width or max(1, max(-(-min(n, keep) // block) for n in lens))].contiguous()
    kc, vc = inputs.randn((nb, Hkv, block, D), dtype, g), inputs.randn((nb, Hkv, block, D), dtype, g)
    w = torch.exp(2 * torch.randn(B, Hkv, old.shape[1] * block, generator=g))
    return kc, vc, w, old, new


def expect(kc, vc, w, old, new, lens, keep, sinks, recent):
    B, Hkv, block = old.shape[0], kc.shape[1], kc.shape[2]
    kc, vc = kc.clone(), vc.clone()
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32)
    nw = torch.zeros(B, Hkv, new.shape[1] * block)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            idx = torch.tensor(chosen(w[b, h, :n].tolist(), keep, sinks, recent), dtype=torch.int64)
            at = torch.arange(len(idx))
            kept[b, h, :len(idx)] = idx.int()
            nw[b, h, :len(idx)] = w[b, h][idx]
            for c in (kc, vc):
                c[new[b][at // block].long(), h, at % block] = c[old[b][idx // block].long(), h, idx % block]
    return kept, nw, kc, vc


def run_and_check(kc, vc, w, old, new, lens, keep, sinks, recent):
    rk, rw, rkc, rvc = expect(kc, vc, w, old, new, lens, keep, sinks, recent)
    kcd, vcd, wd = kc.cuda(), vc.cuda(), w.cuda()
    kept, nl, nw = fa.flash_kv_evict(kcd, vcd, wd, old.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), new.cuda(),
                                     keep, sinks, recent)
    fa.fa_check_device_error()
    assert nl.tolist() == [min(n, keep) for n in lens]
    assert torch.equal(kept.cpu(), rk)
    same = lambda a, b: torch.equal(a.cpu().view(torch.int16), b.view(torch.int16))  # noqa: E731
    assert torch.equal(nw.cpu().view(torch.int32), rw.view(torch.int32))
    assert same(kcd, rkc) and same(vcd, rvc) and torch.equal(wd.cpu().view(torch.int32), w.view(torch.int32))


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hkv,D,block,keep,sinks,recent,dtype", [
    ([777, 200], 2, 64, 32, 130, 1, 33, torch.float16),
    ([100], 1, 128, 16, 99, 0, 0, torch.bfloat16),
    ([100, 0, 1, 64, 65], 3, 128, 16, 64, 4, 60, torch.bfloat16),   # only sinks and recent ones stay
    ([1000, 999], 2, 64, 1, 1, 0, 0, torch.bfloat16),               # the heaviest key
    ([1000], 2, 64, 1024, 500, 0, 499, torch.float16),              # one candidate's place
    ([5000, 4096, 4095], 4, 128, 128, 4095, 20, 1000, torch.bfloat16),
    ([300, 20], 9, 64, 2, 50, 50, 0, torch.float16),                # only sinks
    ([30, 20], 2, 64, 16, 1000, 50, 0, torch.float16),              # nothing leaves
])
def test_evict(lens, Hkv, D, block, keep, sinks, recent, dtype):
    kc, vc, w, old, new = setup(lens, Hkv, D, block, keep, dtype, sum(lens) + keep)
    run_and_check(kc, vc, w, old, new, lens, keep, sinks, recent)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["equal", "few", "zeros", "signs", "neighbours"])
def test_ties_and_special_weights(kind):
    lens, keep = [3000, 1025], 700
    kc, vc, w, old, new = setup(lens, 2, 64, 16, keep, torch.bfloat16, 4)
    g = torch.Generator().manual_seed(9)
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "few":
        w = torch.floor(w).clamp(max=3.0)
    elif kind == "zeros":  # zeros of both signs are equal; fewer positive weights than places
        w = torch.where(torch.rand(w.shape, generator=g) < 0.05, w, torch.zeros_like(w))
        w = torch.where(torch.rand(w.shape, generator=g) < 0.5, -w, w).abs() * torch.sign(torch.randn(w.shape, generator=g))
        w = torch.where(w < 0, torch.full_like(w, -0.0), w)
    elif kind == "signs":
        w = torch.randn(w.shape, generator=g)
        w[..., ::7] = math.nan
        w[..., ::11] = math.inf
        w[..., ::13] = -math.inf
        w[..., ::17] = -w[..., ::17].abs() * 1e-42  # subnormal
    else:  # weights that differ in their last bits
        w = torch.ones_like(w).view(torch.int32).add_(torch.randint(0, 40, w.shape, generator=g, dtype=torch.int32)).view(torch.float32)
    run_and_check(kc, vc, w, old, new, lens, keep, 3, 10)


@pytest.mark.gpu
def test_more_keys_than_shared_memory_holds():
    lens, keep = [70001, 52000], 9000
    kc, vc, w, old, new = setup(lens, 1, 64, 256, keep, torch.float16, 8)
    run_and_check(kc, vc, torch.floor(w * 8) / 8, old, new, lens, keep, 4, 1000)


@pytest.mark.gpu
def test_shared_pages_bad_pages_and_long_lengths():
    lens, keep = [200, 200], 60
    kc, vc, w, old, new = setup(lens, 2, 64, 16, keep, torch.bfloat16, 11)
    old[1] = old[0]  # the same prompt twice; each is evicted into pages of its own
    run_and_check(kc, vc, w, old, new, lens, keep, 2, 5)
    # lengths past the table are the table's
    cut = torch.tensor([1 << 20, -4], dtype=torch.int32).cuda()
    k2, nl, _ = fa.flash_kv_evict(kc.cuda(), vc.cuda(), w.cuda(), old.cuda(), cut, new.cuda(), keep, 2, 5)
    assert nl.tolist() == [60, 0] and (k2[1] == -1).all()
    assert k2[0, :, -5:].tolist() == [list(range(old.shape[1] * 16 - 5, old.shape[1] * 16))] * 2
    fa.fa_check_device_error()
    for t, value in ((0, kc.shape[0]), (0, -1), (1, kc.shape[0]), (1, -1)):
        tabs = [old.clone(), new.clone()]
        tabs[t][0, 0] = value
        kcd = kc.cuda()
        _, nl, _ = fa.flash_kv_evict(kcd, vc.cuda(), w.cuda(), tabs[0].cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                     tabs[1].cuda(), keep, 2, 5)
        with pytest.raises(fa.FAError) as e:
            fa.fa_check_device_error()
        assert e.value.status == DEV_INDEX and nl.tolist() == [60, 60]
        fa.fa_check_device_error()
    # a table with too few pages for what is kept
    kept, nl, nw = fa.flash_kv_evict(kc.cuda(), vc.cuda(), w.cuda(), old.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                     new[:, :2].contiguous().cuda(), keep, 2, 5)
    with pytest.raises(fa.FAError):
        fa.fa_check_device_error()
    assert nw.shape[2] == 32 and (kept >= 0).all()


@pytest.mark.gpu
def test_neighbouring_arrays_are_accepted():
    """Inputs and outputs side by side in one allocation, and tables that are halves of one."""
    lens, keep = [300, 77], 64
    kc, vc, w, old, new = setup(lens, 2, 64, 16, keep, torch.bfloat16, 13, new_width=4)
    ref = fa.flash_kv_evict(kc.cuda(), vc.cuda(), w.cuda(), old.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                            new.cuda(), keep, 2, 9)
    ints = torch.empty(old.numel() + new.numel() + 4 + 4 * keep, dtype=torch.int32, device="cuda")
    parts = ints.split([old.numel(), new.numel(), 2, 2, 4 * keep])
    table, to, lens_in, lens_out, kept = (p.view(s) for p, s in zip(parts, (old.shape, new.shape, (2,), (2,), (2, 2, keep))))
    table.copy_(old), to.copy_(new), lens_in.copy_(torch.tensor(lens))
    floats = torch.empty(w.numel() + ref[2].numel(), device="cuda")
    wi, wo = floats[:w.numel()].view(w.shape), floats[w.numel():].view(ref[2].shape)
    wi.copy_(w)
    fa.fa_kv_evict(kc.cuda(), vc.cuda(), wi, table, lens_in, to, kept, lens_out, wo, 2, 9)
    fa.fa_check_device_error()
    assert torch.equal(kept, ref[0]) and torch.equal(lens_out, ref[1]) and torch.equal(wo, ref[2])
    assert lens_in.tolist() == lens and torch.equal(wi.cpu(), w)


@pytest.mark.gpu
def test_streams_and_graphs():
    lens, keep = [900, 400], 128
    kc, vc, w, old, new = (t.cuda() for t in setup(lens, 2, 64, 16, keep, torch.bfloat16, 12))
    sl = torch.tensor(lens, dtype=torch.int32).cuda()
    ref_k = kc.clone()
    ref = fa.flash_kv_evict(ref_k, vc.clone(), w, old, sl, new, keep, 1, 9)
    side, mine = torch.cuda.Stream(), kc.clone()
    got = fa.flash_kv_evict(mine, vc.clone(), w, old, sl, new, keep, 1, 9, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, got)) and torch.equal(mine, ref_k)
    graph, buf, cache = torch.cuda.CUDAGraph(), torch.zeros_like(w), kc.clone()
    with torch.cuda.graph(graph):
        got = fa.flash_kv_evict(cache, vc.clone(), buf, old, sl, new, keep, 1, 9)
    buf.copy_(w)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got)) and torch.equal(cache, ref_k)


@pytest.mark.gpu
@pytest.mark.parametrize("digits", [1, 2, 3])
def test_threshold_found_early(digits):
    """Weights that differ in their first 11 bits, their first 22, or only behind those: the keys that stay are known after
    so many digits; and a threshold that all keys of a digit pass, zeros and negative weights at the bottom of it."""
    L, Hkv, D, block = 3000, 2, 64, 16
    g = torch.Generator().manual_seed(digits)
    order = torch.stack([torch.randperm(L, generator=g) for _ in range(Hkv)])
    bits = {1: 1 << 21, 2: 1 << 10, 3: 1}[digits]
    if digits == 1:  # (there are fewer than 3000 such)
        order = order // 2
    w = (0x38000000 - (L // 2 if digits > 1 else 0) * bits + order * bits if digits > 1 else 0x00800000 + (order % 900) * bits)
    w = w.to(torch.int32).view(torch.float32)
    for keep in (1, 2, 900, 1500, 2999):
        for weights in (w, torch.where(w > w.median(), w, torch.zeros_like(w)), -w):
            kc = torch.randn(400, Hkv, block, D, generator=g).to(torch.bfloat16)
            vc = torch.randn(400, Hkv, block, D, generator=g).to(torch.bfloat16)
            pages = (L + block - 1) // block
            table = torch.arange(pages, dtype=torch.int32)[None]
            to = torch.arange(pages, 2 * pages, dtype=torch.int32)[None]
            full = torch.zeros(1, Hkv, pages * block)
            full[0, :, :L] = weights
            kd, vd = kc.cuda(), vc.cuda()
            kept, lens, new = fa.flash_kv_evict(kd, vd, full.cuda(), table.cuda(), torch.tensor([L], dtype=torch.int32).cuda(),
                                                to.cuda(), keep)
            for h in range(Hkv):
                ids = sorted(sorted(range(L), key=lambda j: (-float(weights[h, j]), j))[:keep])
                assert kept[0, h].tolist() == ids
                assert torch.equal(new[0, h, :keep].cpu(), weights[h, ids])
    fa.fa_check_device_error()
