"""The paged 4-bit cache: fa_kv_write_q4 and fa_kv_read_q4 against their
definition, bit for bit, and the calls they refuse."""
import math

import pytest
import torch

import exact_attention_54_gb300 as fa
import plain_ops
from exact_attention_54_gb300 import build as fabuild
from exact_attention_54_gb300 import inputs

OK, NULL, SHAPE, HEADDIM, DTYPE, ALIGN = 0, -1, -2, -3, -4, -5
A, MIS = 0x10000, 0x10008


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


# -------------------------------------------------------------- on the CPU --

@pytest.mark.parametrize("name", ["fa_kv_write_q4", "fa_kv_read_q4"])
def test_validation(lib, name):
    def call(k=A, v=A, kc=A, ks=A, vc=A, vs=A, bt=A, cu=A, st=A, n=2, total=10, mx=8, Hkv=2, D=128, nb=8, bs=16, mb=4,
             dtype=1):
        return getattr(lib, name)(k, v, kc, ks, vc, vs, bt, cu, st, n, total, mx, Hkv, D, nb, bs, mb, dtype, None)

    for kw in ("k", "v", "kc", "ks", "vc", "vs", "bt", "cu"):
        assert call(**{kw: None}) == NULL, kw
    assert call(dtype=2) == DTYPE
    for d in (32, 96, 256):
        assert call(D=d) == HEADDIM
    for kw in ({"n": 0}, {"total": -1}, {"total": (1 << 30) + 1}, {"mx": 0}, {"mx": (1 << 30) + 1}, {"Hkv": 0},
               {"nb": 0}, {"bs": 0}, {"bs": 24}, {"bs": 2048}, {"mb": 0}, {"mb": 1 << 27}, {"nb": 1 << 30, "Hkv": 4},
               {"n": 1 << 20, "mx": 1 << 30}):
        assert call(**kw) == SHAPE, kw
    for kw in ("k", "v", "kc", "ks", "vc", "vs"):
        assert call(**{kw: MIS}) == ALIGN, kw
    for kw in ("bt", "cu", "st"):
        assert call(**{kw: A + 2}) == ALIGN, kw
    assert call(total=0, k=None, v=None) == OK  # nothing to do


def test_binding_refuses():
    c = fa.kv_cache_q4(4, 2, 16, 64, torch.bfloat16, device="cpu")
    assert [tuple(t.shape) for t in c] == [(4, 2, 16, 32), (4, 2, 16, 2)] * 2
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    cu, bt = torch.tensor([0, 5], dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    call = lambda k=k, v=k, c=c, bt=bt, cu=cu, **kw: fa.flash_kv_write_q4(k, v, c, bt, cu, 5, **kw)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(TypeError, match="v must be"):
        call(v=k.half())
    with pytest.raises(TypeError, match="unsupported dtype"):
        call(k=k.float(), v=k.float())
    with pytest.raises(TypeError, match="k_scales"):
        call(c=c._replace(k_scales=c.k_scales.half()))
    with pytest.raises(ValueError, match="v_codes"):
        call(c=c._replace(v_codes=c.v_codes[:, :1]))
    with pytest.raises(ValueError, match="block_table"):
        call(bt=bt[:0])
    with pytest.raises(TypeError, match="cu_seqlens"):
        call(cu=cu.long())
    with pytest.raises(ValueError, match="starts"):
        call(starts=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="contiguous"):
        call(k=k.transpose(0, 1).contiguous().transpose(0, 1))


def test_plain_format_round_trip():
    n = torch.randint(-7, 8, (3, 128), generator=torch.Generator().manual_seed(1))
    assert torch.equal(plain_ops.q4_unpack(plain_ops.q4_pack(n)), n)
    x = torch.randn(50, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    n, s = plain_ops.q4_quantise(x)
    err = (plain_ops.q4_values(plain_ops.q4_pack(n), s) - x.double()).abs().unflatten(-1, (-1, 32))
    # half a step of the grid, and what the rounding of s leaves above 7 s (7 s off by half a step of bf16)
    assert (err <= s.double().unsqueeze(-1) * (0.5 + 7 * 2.0 ** -8)).all()


# -------------------------------------------------------------- on the GPU --

def special_rows(D, dtype):
    """Rows whose groups hold the values where the rounding can go wrong."""
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps  # smallest subnormal
    big = torch.finfo(dtype).max
    rows = torch.zeros(12, D, dtype=torch.float64)
    rows[1] = torch.linspace(-1, 1, D)
    ties = torch.tensor([7, -6.5, -5.5, -4.5, -3.5, -2.5, -1.5, -0.5, 0.5, 1.5, 2.5, 3.5, 4.5, 5.5, 6.5, 0.0],
                        dtype=torch.float64)
    rows[2] = ties.repeat(D // 16) * 0.25      # s = 1/4 exactly: every second value is a tie
    rows[3] = ties.repeat(D // 16) * tiny * 8  # the same among the subnormals
    rows[4] = tiny                             # s rounds to zero
    rows[5] = 3 * tiny
    rows[6] = tiny * torch.arange(1, D + 1) % 23
    rows[7] = big * torch.linspace(-1, 1, D)
    rows[8] = 1.0
    rows[8, ::5] = -1.0
    rows[9] = torch.linspace(-1, 1, D)
    rows[9, 3] = math.inf
    rows[9, D - 1] = -math.inf
    rows[10] = torch.linspace(-1, 1, D)
    rows[10, 40] = math.nan
    rows[11, 31] = -0.0
    rows[11, 32] = -2.0
    return rows.to(dtype)


def same_bits(a, b):
    """Equal bit for bit (NaNs of any pattern are alike)."""
    if a.dtype == torch.uint8:
        return torch.equal(a, b)
    na, nb = torch.isnan(a), torch.isnan(b)
    return torch.equal(na, nb) and torch.equal(a.masked_fill(na, 0).view(torch.int16), b.masked_fill(nb, 0).view(torch.int16))


def make(lens, starts, Hkv, D, block, dtype, seed):
    """New tokens (special rows first, then normal draws of several sizes), an empty cache whose rows hold 0x55
    bytes, and the table."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    def draw():
        x = torch.randn(T, Hkv, D, generator=g) * torch.exp2(torch.randint(-6, 7, (T, Hkv, 1), generator=g).float())
        x = x.to(dtype)
        sp = special_rows(D, dtype)
        flat = x.view(-1, D)
        n = min(len(sp), len(flat))
        flat[torch.randperm(len(flat), generator=g)[:n]] = sp[:n]
        return x
    k, v = draw(), draw()
    ends = [s + n for s, n in zip(starts, lens)]
    _, _, _, table, _ = inputs.make_paged(len(lens), 1, 1, block, ends, torch.float16, seed)
    nb = sum(-(-e // block) for e in ends) + 3
    fill = lambda w: torch.full((nb, Hkv, block, w), 0x55, dtype=torch.uint8)  # noqa: E731
    cache = [fill(D // 2), fill(D // 16).view(dtype), fill(D // 2), fill(D // 16).view(dtype)]
    return k, v, cache, table, inputs.cu_from_lengths(lens), torch.tensor(starts, dtype=torch.int32)


def write_plain(k, v, cache, table, cu, starts, block):
    out = [t.clone() for t in cache]
    nk, sk = plain_ops.q4_quantise(k)
    nv, sv = plain_ops.q4_quantise(v)
    rows = [plain_ops.q4_pack(nk), sk, plain_ops.q4_pack(nv), sv]
    for b in range(len(starts)):
        for t in range(int(cu[b]), int(cu[b + 1])):
            pos = int(starts[b]) + t - int(cu[b])
            for o, r in zip(out, rows):
                o[int(table[b, pos // block]), :, pos % block] = r[t]
    return out


CASES = [
    # lens, starts, Hkv, D, block, dtype
    ([1], [0], 1, 64, 1, torch.float16),
    ([1, 1, 1, 1, 1], [0, 15, 16, 31, 700], 8, 128, 16, torch.bfloat16),
    ([37, 0, 5], [3, 9, 0], 3, 128, 32, torch.float16),
    ([130, 64, 1], [0, 1, 77], 2, 64, 16, torch.bfloat16),
    ([9, 40], [5, 0], 5, 128, 4, torch.bfloat16),
    ([300], [1000], 1, 64, 1024, torch.float16),
    ([3, 2], [0, 6], 40, 128, 16, torch.float16),  # more key heads than rows of a CTA's pass
    ([61, 3], [2, 30], 7, 128, 8, torch.bfloat16),
    ([11, 4], [0, 5], 31, 64, 64, torch.float16),
    ([5], [1], 32, 128, 16, torch.bfloat16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,starts,Hkv,D,block,dtype", CASES)
def test_write_and_read(lens, starts, Hkv, D, block, dtype):
    k, v, cache, table, cu, st = make(lens, starts, Hkv, D, block, dtype, seed=sum(lens) + D)
    want = write_plain(k, v, cache, table, cu, st, block)
    dev = [t.cuda() for t in cache]
    tb, cud, std, n = table.cuda(), cu.cuda(), st.cuda(), max(lens)
    fa.flash_kv_write_q4(k.cuda(), v.cuda(), fa.KVCacheQ4(*dev), tb, cud, n, starts=std)
    fa.fa_check_device_error()
    for name, a, b in zip(("k_codes", "k_scales", "v_codes", "v_scales"), dev, want):
        assert same_bits(a.cpu(), b), name
    # back again; the rows in front of and behind the sequences keep what they held
    T = sum(lens)
    pad = lambda: torch.full((T + 3, Hkv, D), 7.0, dtype=dtype, device="cuda")  # noqa: E731
    ko, vo = pad(), pad()
    fa.fa_kv_read_q4(ko, vo, *dev, tb, (cud + 1), n, starts=std)
    fa.fa_check_device_error()
    for name, got, c, s in (("k", ko, want[0], want[1]), ("v", vo, want[2], want[3])):
        x = plain_ops.q4_values(c, s).float().to(dtype)  # s n is exact in fp32: one rounding
        got = got.cpu()
        for b in range(len(lens)):
            for t in range(int(cu[b]), int(cu[b + 1])):
                pos = int(st[b]) + t - int(cu[b])
                assert same_bits(got[t + 1], x[int(table[b, pos // block]), :, pos % block]), (name, b, t)
        assert torch.equal(got[0], torch.full_like(got[0], 7.0)) and torch.equal(got[T + 1:], torch.full_like(got[T + 1:], 7.0))


@pytest.mark.gpu
def test_starts_default_to_zero_and_other_stream():
    k, v, cache, table, cu, st = make([20, 33], [0, 0], 2, 128, 16, torch.bfloat16, seed=5)
    want = write_plain(k, v, cache, table, cu, st, 16)
    dev, kd, vd, td, cd = [t.cuda() for t in cache], k.cuda(), v.cuda(), table.cuda(), cu.cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        fa.flash_kv_write_q4(kd, vd, fa.KVCacheQ4(*dev), td, cd, 33)
    fa.fa_check_device_error(s)
    assert all(same_bits(a.cpu(), b) for a, b in zip(dev, want))


@pytest.mark.gpu
@pytest.mark.parametrize("fault,status", [("page", -11), ("position", -11), ("offsets", -13), ("length", -13),
                                          ("start", -13), ("behind", -13)])
def test_bad_device_arrays_are_reported_and_skipped(fault, status):
    """One of two sequences is wrong: the other's rows are written, nothing else is."""
    lens, block = [20, 33], 16
    k, v, cache, table, cu, st = make(lens, [0, 0], 2, 64, block, torch.float16, seed=6)
    good = torch.tensor([0, 20], dtype=torch.int32)
    want = write_plain(k[:20], v[:20], cache, table[:1], good, st[:1], block)
    n = 33
    if fault == "page":
        table[1] = torch.tensor([-1, 10 ** 6, -(2 ** 31)], dtype=torch.int32)
    elif fault == "position":
        st[1] = 3 * block
    elif fault == "offsets":
        cu[2] = 10
    elif fault == "length":
        n = 32
    elif fault == "start":
        st[1] = -1
    else:
        cu[2] = 54
    dev = [t.cuda() for t in cache]
    fa.flash_kv_write_q4(k.cuda(), v.cuda(), fa.KVCacheQ4(*dev), table.cuda(), cu.cuda(), n, starts=st.cuda())
    with pytest.raises(fa.FAError) as e:
        fa.fa_check_device_error()
    assert e.value.status == status
    fa.fa_check_device_error()
    assert all(same_bits(a.cpu(), b) for a, b in zip(dev, want))


@pytest.mark.gpu
def test_rows_that_are_16_byte_aligned_only():
    k, v, cache, table, cu, st = make([20, 33], [0, 0], 2, 128, 16, torch.bfloat16, seed=7)
    want = write_plain(k, v, cache, table, cu, st, 16)
    shifted = lambda t: torch.cat([torch.zeros(8, dtype=t.dtype), t.flatten()]).cuda()[8:].view(t.shape)  # noqa: E731
    dev, td, cd = [shifted(t) if t.dtype != torch.uint8 else t.cuda() for t in cache], table.cuda(), cu.cuda()
    fa.flash_kv_write_q4(shifted(k), shifted(v), fa.KVCacheQ4(*dev), td, cd, 33)
    assert all(same_bits(a.cpu(), b) for a, b in zip(dev, want))
    kr, vr = fa.flash_kv_read_q4(fa.KVCacheQ4(*dev), td, cd, 53, 33)
    ko, vo = shifted(torch.zeros_like(k)), shifted(torch.zeros_like(v))
    assert ko.data_ptr() % 32 == 16
    fa.fa_kv_read_q4(ko, vo, *dev, td, cd, 33)
    fa.fa_check_device_error()
    assert same_bits(ko.cpu(), kr.cpu()) and same_bits(vo.cpu(), vr.cpu())


@pytest.mark.gpu
def test_more_sequences_than_a_grid_dimension():
    """70000 sequences, most of them without tokens."""
    n, D = 70000, 64
    lens = torch.zeros(n, dtype=torch.int64)
    lens[[0, 1, 65534, 65535, 65536, n - 1]] = torch.tensor([2, 1, 1, 2, 1, 2])
    cu = torch.zeros(n + 1, dtype=torch.int32)
    cu[1:] = lens.cumsum(0)
    T = int(cu[-1])
    k = inputs.randn((T, 1, D), torch.float16, torch.Generator().manual_seed(8))
    table = torch.full((n, 1), -1, dtype=torch.int32)
    used = torch.nonzero(lens).flatten()
    table[used, 0] = torch.arange(len(used), dtype=torch.int32)
    c = fa.kv_cache_q4(len(used), 1, 2, D, torch.float16)
    fa.flash_kv_write_q4(k.cuda(), (-k).cuda(), c, table.cuda(), cu.cuda(), 2)
    kr, vr = fa.flash_kv_read_q4(c, table.cuda(), cu.cuda(), T, 2)
    fa.fa_check_device_error()
    codes, scales = plain_ops.q4_quantise(k)
    want = plain_ops.q4_values(plain_ops.q4_pack(codes), scales).to(torch.float16)
    assert torch.equal(kr.cpu(), want) and torch.equal(vr.cpu(), -want)


@pytest.mark.gpu
def test_no_tokens():
    c = fa.kv_cache_q4(2, 2, 16, 64, torch.float16)
    cu, bt = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    k = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    fa.flash_kv_write_q4(k, k, c, bt, cu, 1)
    fa.fa_check_device_error()
    assert int(c.k_codes.sum()) == 0


@pytest.mark.parametrize("name", ["fa_kv_write_q4", "fa_kv_read_q4"])
def test_a_longest_sequence_of_no_tokens(name, lib):
    """max_seqlen is at least every number of new tokens: 0 is, where there are none (and only there)."""
    def call(total, mx, k=A, v=A):
        return getattr(lib, name)(k, v, A, A, A, A, A, A, None, 2, total, mx, 2, 64, 4, 16, 3, 1, None)
    assert call(0, 0) == 0 and call(0, 0, None, None) == 0
    assert call(0, -1) == SHAPE and call(1, 0) == SHAPE and call(-1, 0) == SHAPE


@pytest.mark.gpu
def test_a_step_without_new_tokens():
    """What a serving loop passes where no sequence has any: nothing is written, nothing comes back."""
    c = fa.kv_cache_q4(2, 2, 16, 64, torch.float16)
    cu, bt = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    k = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    fa.flash_kv_write_q4(k, k, c, bt, cu, 0)
    kr, vr = fa.flash_kv_read_q4(c, bt, cu, 0, 0)
    fa.fa_check_device_error()
    assert kr.shape == vr.shape == (0, 2, 64) and not any(int((t != 0).sum()) for t in c)
