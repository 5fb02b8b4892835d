"""Rotary positions (fa_rope, its gradient) and new tokens into a paged 16-bit
cache (fa_rope_kv_write): against the definition in 64 bits with angles from
whole-number arithmetic, and the calls they refuse."""
import math
from fractions import Fraction

import pytest
import torch

import exact_attention_54_gb300 as fa
from exact_attention_54_gb300 import build as fabuild
from exact_attention_54_gb300 import inputs
from plain_ops import half_step

OK, NULL, SHAPE, HEADDIM, DTYPE, ALIGN, SCALE, CUDA = 0, -1, -2, -3, -4, -5, -7, -8
DEV_INDEX, DEV_SEQLENS = -11, -13
A, MIS = 0x10000, 0x10008

# pi to 70 digits: 1 / 2 pi as a fraction of 2^200
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164, 10 ** 70)
INV_2PI = int((1 << 200) / (2 * PI))


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


def angles(positions, inv_freq):
    """p * inv_freq modulo a turn, in radians (double): [tokens, pairs]."""
    rows = []
    for p in positions:
        row = []
        for f in inv_freq.tolist():
            n, d = float(f).as_integer_ratio()
            turns = p * n * INV_2PI  # over d 2^200
            row.append(2 * math.pi * float(Fraction(turns % (d << 200), d << 200)))
        rows.append(row)
    return torch.tensor(rows, dtype=torch.float64)


def rotated(x, ang, rot, interleaved, mscale, inverse=False):
    """x [tokens, heads, D] -> (y, bound) in double. The bound: half a step of the output; the cosine and the sine are
    off by 2^-24.35 of a radian times 2 for the rounding of the turn to 24 bits, 2^-22 for sincospi (2 ulp), and with
    mscale, two products and a sum in fp32 (2^-24 each) the rest is under 2^-20.5 of mscale (|a| + |b|); positions up to
    2^31 add 2 pi 2^-53 2^31 = 2^-19.3."""
    x = x.double()
    y, size = x.clone(), torch.zeros_like(x)
    i = torch.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    c, s = torch.cos(ang)[:, None] * mscale, torch.sin(ang)[:, None] * mscale
    if inverse:
        s = -s
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = abs(mscale) * (a.abs() + b.abs())
    return y, size


def close(got, y, size, dtype, far=False, what=""):
    h = half_step(dtype)
    bound = h * y.abs() * (1 + h) + (2.0 ** -20.5 + (2.0 ** -19.3 if far else 0)) * size * (1 + 2 * h) + \
        torch.finfo(dtype).smallest_normal * h * 2 * (size > 0)
    bad = ~((got.double().cpu() - y).abs() <= bound)
    assert not bad.any(), (what, torch.nonzero(bad)[0].tolist(), float(((got.double().cpu() - y).abs() / bound).nan_to_num().max()))


# -------------------------------------------------------------- on the CPU --

def test_validation(lib):
    def call(x=A, y=A, f=A, p=A, B=2, S=5, H=3, D=128, rot=64, xs=(1920, 384, 128), ys=(1920, 384, 128), inter=0, inv=0,
             m=1.0, dtype=1):
        return lib.fa_rope(x, y, f, p, B, S, H, D, rot, *xs, *ys, inter, inv, m, dtype, None)

    for kw in ("x", "y", "f"):
        assert call(**{kw: None}) == NULL, kw
    assert call(dtype=2) == DTYPE
    for d in (32, 96, 384):
        assert call(D=d) == HEADDIM
    for kw in ({"B": 0}, {"S": -1}, {"S": (1 << 30) + 1}, {"H": 0}, {"H": 1 << 25}, {"rot": 0}, {"rot": 8}, {"rot": 144},
               {"rot": -16}, {"xs": (1920, 384, 4)}, {"ys": (-1920, 384, 128)}, {"xs": (1 << 41, 384, 128)}):
        assert call(**kw) == SHAPE, kw
    for ys in ((0, 384, 128), (1920, 0, 128), (1920, 384, 0)):  # rows of y on one another
        assert call(ys=ys) == SHAPE, ys
    assert call(m=float("nan")) == SCALE
    for kw in ("x", "y"):
        assert call(**{kw: MIS}) == ALIGN, kw
    for kw in ("f", "p"):
        assert call(**{kw: A + 2}) == ALIGN, kw
    assert call(S=0, x=None, y=None, p=None) == OK


def test_no_tokens_of_any_strides(lib):
    """S = 0 does nothing, also where the strides are those of an empty contiguous [B,H,0,D] (0 between heads)."""
    for ys in ((0, 64, 0), (0, 64, 64), (0, 0, 0), (256, 64, 64)):
        assert lib.fa_rope(None, None, A, None, 2, 0, 4, 64, 64, *ys, *ys, 0, 0, 1.0, 1, None) == OK, ys
        for at in (None, A):  # "in place", with strides that mean nothing
            assert lib.fa_rope(at, at, A, None, 2, 0, 4, 64, 64, 512, 128, 64, *ys, 0, 0, 1.0, 1, None) == OK, ys
    for B, H in ((1, 4), (2, 1), (2, 4)):
        x = torch.empty(B, H, 0, 64, dtype=torch.bfloat16)
        st = fa._rows("x", x, x.dtype)
        assert lib.fa_rope(A, A, A, None, B, 0, H, 64, 64, *st, *st, 0, 0, 1.0, 1, None) == OK, (B, H)


def test_in_place_with_other_strides_is_refused(lib):
    """Rows would be written where others are still to be read."""
    def rope(x, y, B, S, H, xs, ys):
        return lib.fa_rope(x, y, A, None, B, S, H, 64, 64, *xs, *ys, 0, 0, 1.0, 1, None)

    for B, S, H, xs, ys in ((1, 5, 3, (0, 192, 64), (0, 64, 320)), (2, 5, 1, (320, 64, 64), (640, 64, 64)),
                            (1, 5, 1, (0, 64, 64), (0, 128, 64)), (1, 1, 3, (0, 0, 64), (0, 0, 128))):
        assert rope(A, A, B, S, H, xs, ys) == SHAPE, (B, S, H)
        if not torch.cuda.is_available():  # elsewhere, or the same strides but in dimensions of one
            assert rope(A, 2 * A, B, S, H, xs, ys) == CUDA
            assert rope(A, A, B, S, H, xs, xs) == CUDA

    def write(q, out, total, stride):
        return lib.fa_rope_kv_write(q, A, A, out, A, A, A, None, A, A, None, 1, total, total, 4, 2, 64, 64, stride, 128, 128,
                                    8, 16, 4, 0, 1.0, 1, None)

    assert write(A, A, 5, 512) == SHAPE
    if not torch.cuda.is_available():
        assert write(A, 2 * A, 5, 512) == write(A, A, 5, 256) == write(A, A, 1, 512) == CUDA
        assert rope(A, A, 1, 1, 1, (64, 64, 64), (8, 8, 8)) == CUDA


def test_write_validation(lib):
    def call(q=A, k=A, v=A, qo=A, kc=A, vc=A, f=A, p=A, bt=A, cu=A, st=A, n=2, total=10, mx=8, H=4, Hkv=2, D=128, rot=64,
             qs=512, ks=256, vs=256, nb=8, bs=16, mb=4, inter=0, m=1.0, dtype=1):
        return lib.fa_rope_kv_write(q, k, v, qo, kc, vc, f, p, bt, cu, st, n, total, mx, H, Hkv, D, rot, qs, ks, vs, nb,
                                    bs, mb, inter, m, dtype, None)

    for kw in ("q", "k", "v", "qo", "kc", "vc", "f", "bt", "cu"):
        assert call(**{kw: None}) == NULL, kw
    assert call(dtype=3) == DTYPE
    for d in (32, 256):
        assert call(D=d) == HEADDIM
    for kw in ({"n": 0}, {"total": -1}, {"mx": 0}, {"H": -1}, {"Hkv": 0}, {"rot": 24}, {"rot": 256}, {"qs": 4},
               {"ks": -8}, {"bs": 24}, {"mb": 0}, {"nb": 0}, {"nb": 1 << 30, "Hkv": 4}, {"H": 1 << 25}):
        assert call(**kw) == SHAPE, kw
    assert call(m=float("inf")) == SCALE
    for kw in ("q", "k", "v", "qo", "kc", "vc"):
        assert call(**{kw: MIS}) == ALIGN, kw
    for kw in ("f", "p", "bt", "cu", "st"):
        assert call(**{kw: A + 2}) == ALIGN, kw
    assert call(total=0, mx=0, q=None, k=None, v=None, qo=None) == OK


def test_binding_refuses():
    x, f = torch.zeros(5, 3, 64, dtype=torch.bfloat16), torch.zeros(16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.flash_rope(x, f)
    with pytest.raises(TypeError, match="unsupported dtype"):
        fa.flash_rope(x.float(), f)
    with pytest.raises(ValueError, match="total,H,D"):
        fa.flash_rope(x[0], f)
    with pytest.raises(TypeError, match="inv_freq"):
        fa.flash_rope(x, f.double())
    with pytest.raises(ValueError, match="positions"):
        fa.flash_rope(x, f, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(TypeError, match="positions"):
        fa.flash_rope(x, f, torch.zeros(5, dtype=torch.int64))
    with pytest.raises(ValueError, match="last dimension"):
        fa.flash_rope(torch.zeros(5, 64, 64, dtype=torch.bfloat16).transpose(1, 2), f)
    with pytest.raises(ValueError, match="multiples of 8"):
        fa.flash_rope(torch.zeros(5, 3, 68, dtype=torch.bfloat16)[..., :64], f)
    with pytest.raises(ValueError, match="y must have"):
        fa.fa_rope(x, x[:4], f)
    k, cu, bt = x, torch.tensor([0, 5], dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    c = torch.zeros(4, 3, 16, 64, dtype=torch.bfloat16)
    call = lambda q=x, k=k, v=k, kc=c, vc=c, cu=cu, bt=bt, **kw: fa.flash_rope_kv_write(q, k, v, kc, vc, bt, cu, 5, f, **kw)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(TypeError, match="v must be"):
        call(v=k.half())
    with pytest.raises(ValueError, match="v must be"):
        call(v=k[:4])
    with pytest.raises(ValueError, match="q must be"):
        call(q=x[:4])
    with pytest.raises(ValueError, match="v_cache"):
        call(vc=c[:, :2])
    with pytest.raises(ValueError, match="heads must be contiguous"):
        call(k=torch.zeros(5, 6, 64, dtype=torch.bfloat16)[:, ::2])
    with pytest.raises(TypeError, match="cu_seqlens"):
        call(cu=cu.long())
    with pytest.raises(ValueError, match="block_table"):
        call(bt=bt[:0])
    with pytest.raises(ValueError, match="q_out"):
        fa.fa_rope_kv_write(None, k, k, x, c, c, bt, cu, 5)


def test_frequencies():
    f, m = fa.rope_frequencies(64, device="cpu")
    assert m == 1.0 and f.dtype == torch.float32
    assert torch.equal(f, (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float())
    g, _ = fa.rope_frequencies(64, scaling="linear", factor=8, device="cpu")
    assert torch.allclose(g, f / 8, rtol=2.0 ** -22)
    g, _ = fa.rope_frequencies(64, scaling="base", factor=8, device="cpu")
    assert g[0] == 1 and math.isclose(float(g[-1]), float(f[-1]) / 8, rel_tol=1e-6)
    g, m = fa.rope_frequencies(64, scaling="parts", factor=8, device="cpu")
    turns = 4096 * f.double() / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32]) and torch.allclose(g[turns < 1], f[turns < 1] / 8, rtol=2.0 ** -22)
    assert m == 0.1 * math.log(8) + 1.0 and (turns > 32).any() and (turns < 1).any()
    for kw in ({"rot_dim": 24}, {"rot_dim": 0}, {"scaling": "other"}, {"factor": 0.0}, {"low": 3.0, "high": 3.0}):
        with pytest.raises(ValueError):
            fa.rope_frequencies(**{"rot_dim": 64, "device": "cpu", **kw})


def test_frequencies_that_are_not_finite_are_refused():
    for kw in ({"base": 1e-300}, {"scaling": "linear", "factor": 1e-45}, {"scaling": "parts", "factor": math.inf},
               {"scaling": "parts", "low": -math.inf}):
        with pytest.raises(ValueError, match="finite"):
            fa.rope_frequencies(64, device="cpu", **kw)
    f, m = fa.rope_frequencies(64, base=math.inf, device="cpu")  # only the first pair turns
    assert f[0] == 1 and (f[1:] == 0).all() and m == 1.0


def test_angles_of_whole_numbers():
    """The oracle's angles against 64-bit floating point, where that is good enough."""
    f, _ = fa.rope_frequencies(32, device="cpu")
    a, b = angles([0, 1, -5, 1000], f), torch.tensor([0.0, 1.0, -5.0, 1000.0], dtype=torch.float64)[:, None] * f.double()
    assert (torch.cos(a) - torch.cos(b)).abs().max() < 1e-12 and (torch.sin(a) - torch.sin(b)).abs().max() < 1e-12


# -------------------------------------------------------------- on the GPU --

FAR = [0, 1, -1, 7, 4096, 131071, 1 << 20, (1 << 24) + 1, -(1 << 30) - 3, (1 << 31) - 1, -(1 << 31)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot,H,S", [(64, 64, 3, 11), (64, 16, 1, 1), (64, 48, 5, 37), (128, 128, 40, 3), (128, 32, 2, 70),
                                       (256, 128, 2, 9), (512, 512, 1, 3), (1024, 1024, 3, 9)])
def test_rope_packed(dtype, inter, D, rot, H, S):
    g = torch.Generator().manual_seed(D + rot + H)
    x = inputs.randn((S, H, D), dtype, g)
    f, m = fa.rope_frequencies(rot, scaling="parts", factor=4, device="cpu")
    pos = [FAR[(3 * i) % len(FAR)] if i % 2 else 17 * i for i in range(S)]
    ang = angles(pos, f)
    p = torch.tensor(pos, dtype=torch.int32).cuda()
    for inverse, fn in ((False, fa.flash_rope), (True, fa.flash_rope_bwd)):
        y = fn(x.cuda(), f.cuda(), p, interleaved=inter, mscale=m)
        ry, size = rotated(x, ang, rot, inter, m, inverse)
        close(y, ry, size, dtype, far=True, what=inverse)
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])  # copied, bit for bit
    fa.fa_check_device_error()


@pytest.mark.gpu
@pytest.mark.parametrize("B,S,H,D", [(1, 1, 1, 64), (3, 130, 2, 64), (2, 33, 7, 128)])
def test_rope_dense_and_strides(B, S, H, D):
    g = torch.Generator().manual_seed(B * S)
    f, _ = fa.rope_frequencies(D, device="cpu")
    x = inputs.randn((B, H, S, D), torch.bfloat16, g)
    ang = angles(range(S), f)
    ry, size = rotated(x.permute(0, 2, 1, 3).reshape(B * S, H, D), ang.repeat(B, 1), D, False, 1.0)
    back = lambda t: t.view(B, S, H, D).permute(0, 2, 1, 3)  # noqa: E731
    xd, fd = x.cuda(), f.cuda()
    y = fa.flash_rope(xd, fd)
    close(y, back(ry), back(size), torch.bfloat16)
    # the same rows as a part of a wider projection [B,S,H+2,D], positions given, in place
    wide = torch.full((B, S, H + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    view = wide[:, :, 1:H + 1].permute(0, 2, 1, 3)
    view.copy_(xd)
    pos = torch.arange(S, dtype=torch.int32).repeat(B, 1).cuda()
    z = fa.flash_rope(view, fd, pos)
    assert z.is_contiguous() and torch.equal(z, y)
    fa.fa_rope(view, view, fd)
    assert torch.equal(view, y) and (wide[:, :, 0] == 7).all() and (wide[:, :, -1] == 7).all()
    # positions of its own for each sequence
    if B > 1:
        pos = pos + 5 * torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
        one = fa.flash_rope(xd[1:2].contiguous(), fd, pos[1:2])
        assert torch.equal(fa.flash_rope(xd, fd, pos.contiguous())[1:2], one) and not torch.equal(one, y[1:2])


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient_against_differences(inter):
    """<dy, (rope(x + e u) - rope(x - e u)) / 2 e> = <rope_bwd(dy), u>, the left side from the 64-bit definition."""
    g = torch.Generator().manual_seed(5)
    S, H, D, rot = 9, 2, 64, 32
    x, u, dy = (inputs.randn((S, H, D), torch.float16, g) for _ in range(3))
    f, m = fa.rope_frequencies(rot, scaling="parts", factor=8, device="cpu")
    ang, e = angles(range(S), f), 1e-3
    def plain(t):
        return rotated(t, ang, rot, inter, m)[0]
    left = (dy.double() * (plain(x.double() + e * u.double()) - plain(x.double() - e * u.double())) / (2 * e)).sum()
    dx = fa.flash_rope_bwd(dy.cuda(), f.cuda(), interleaved=inter, mscale=m).double().cpu()
    right = (dx * u.double()).sum()
    # each element of dx is off by half a step of itself (2^-11) and 2^-20.5 of what meets in it
    room = ((2.0 ** -11 + 2.0 ** -18) * 2 * m * dy.double().abs().max() * u.double().abs()).sum() * 1e-1
    exact = ((2.0 ** -11 + 2.0 ** -17) * (dx.abs() + 1e-3) * u.double().abs()).sum()
    assert abs(left - right) <= min(exact, room) + 1e-9


@pytest.mark.gpu
def test_rope_not_finite_values_stay_in_their_pair():
    x = torch.ones(2, 1, 64, dtype=torch.bfloat16)
    x[0, 0, 3] = math.nan
    x[1, 0, 40] = math.inf
    f, _ = fa.rope_frequencies(32, device="cpu")
    y = fa.flash_rope(x.cuda(), f.cuda()).cpu()
    assert torch.isnan(y[0, 0, 3]) and torch.isnan(y[0, 0, 19]) and y[1, 0, 40] == math.inf
    assert int((~torch.isfinite(y)).sum()) == 3


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_rope_frequencies_that_are_not_finite(bad, inter):
    """An angle of p * inf or p * NaN has no cosine: its pair is NaN, at every position; the others are as without it."""
    g = torch.Generator().manual_seed(3)
    x = inputs.randn((7, 2, 64), torch.bfloat16, g).cuda()
    f, _ = fa.rope_frequencies(48)
    pos = torch.tensor([0, 1, -1, 5, 1 << 20, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32, device="cuda")
    h = f.clone()
    h[5], h[23] = bad, bad
    pair = torch.zeros(64, dtype=torch.bool)
    for i in (5, 23):
        pair[[2 * i, 2 * i + 1] if inter else [i, i + 24]] = True
    c = [torch.zeros(1, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    write = lambda f: fa.flash_rope_kv_write(x, x, x, *c, torch.zeros(1, 1, dtype=torch.int32, device="cuda"),  # noqa: E731
                                             torch.tensor([0, 7], dtype=torch.int32, device="cuda"), 7, f, positions=pos,
                                             interleaved=inter)
    for call in (lambda f: fa.flash_rope(x, f, pos, inter), lambda f: fa.flash_rope_bwd(x, f, pos, inter), write):
        y, z = call(f).cpu(), call(h).cpu()
        assert torch.isnan(z[..., pair]).all() and torch.equal(z[..., ~pair], y[..., ~pair])
    k = c[0][0, :, :7].cpu()
    assert torch.isnan(k[..., pair]).all() and torch.equal(c[1][0, :, :7], x.transpose(0, 1))
    fa.fa_check_device_error()


def cache_rows(cache, table, b, at, block):
    """Rows [n, Hkv, D] of positions ``at`` of sequence b."""
    at = torch.as_tensor(at)
    return cache[table[b][at // block].long(), :, at % block]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,starts,H,Hkv,D,rot,block,inter,dtype", [
    ([1, 1, 1], [0, 15, 16], 4, 2, 64, 64, 16, False, torch.bfloat16),
    ([70, 0, 1, 33], [3, 9, 0, 62], 6, 3, 128, 64, 32, True, torch.float16),
    ([130], [0], 1, 1, 128, 128, 1, False, torch.bfloat16),
    ([5, 200], [1000, 2], 0, 2, 64, 16, 1024, False, torch.float16),
    ([9, 40], [7, 8], 16, 8, 128, 0, 2, False, torch.bfloat16),
])
def test_write(lens, starts, H, Hkv, D, rot, block, inter, dtype):
    g = torch.Generator().manual_seed(sum(lens) + D)
    T, pad = sum(lens), 3  # rows behind the last sequence
    ends = [s + n for s, n in zip(starts, lens)]
    table, nb = inputs.make_paged(len(lens), 1, 1, block, ends, dtype, 3)[3], sum(-(-e // block) for e in ends) + 3
    qkv = inputs.randn((T + pad, H + 2 * Hkv, D), dtype, g)  # a joint projection's rows
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    kc, vc = (torch.full((nb, Hkv, block, D), 9.0, dtype=dtype).cuda() for _ in range(2))
    f = fa.rope_frequencies(rot, device="cpu")[0] if rot else None
    cu = inputs.cu_from_lengths(lens)
    qkvd = qkv.cuda()
    qd, kd, vd = qkvd[:, :H], qkvd[:, H:H + Hkv], qkvd[:, H + Hkv:]
    for pos in (None, [(31 * i * i) % 100003 for i in range(T + pad)]):
        kc.fill_(9.0), vc.fill_(9.0)
        qo = torch.full((T + pad, H, D), 5.0, dtype=dtype).cuda() if H else None
        fa.fa_rope_kv_write(qd if H else None, kd, vd, qo, kc, vc, table.cuda(), cu.cuda(), max(lens), f if f is None else f.cuda(),
                            starts=torch.tensor(starts, dtype=torch.int32).cuda(),
                            positions=None if pos is None else torch.tensor(pos, dtype=torch.int32).cuda(),
                            interleaved=inter, mscale=1.25)
        fa.fa_check_device_error()
        at = pos[:T] if pos else [s + i for s, n in zip(starts, lens) for i in range(n)]
        ang = angles(at, f) if rot else torch.zeros(T, 0, dtype=torch.float64)
        if H:
            y, size = rotated(q[:T], ang, rot, inter, 1.25)
            close(qo[:T], y, size, dtype, what="q")
            assert (qo[T:] == 5).all()
        y, size = rotated(k[:T], ang, rot, inter, 1.25)
        written = torch.zeros(nb, block, dtype=torch.bool)
        for b, n in enumerate(lens):
            rows, t0 = torch.arange(starts[b], starts[b] + n), int(cu[b])
            if n == 0:
                continue
            close(cache_rows(kc.cpu(), table, b, rows, block), y[t0:t0 + n], size[t0:t0 + n], dtype, what="k")
            assert torch.equal(cache_rows(vc.cpu(), table, b, rows, block), v[t0:t0 + n])
            written[table[b][rows // block].long(), rows % block] = True
        rest = ~written[:, None, :, None].expand(-1, Hkv, -1, D)
        assert (kc.cpu()[rest] == 9).all() and (vc.cpu()[rest] == 9).all()
    if H:  # in place, and the allocating form
        ref = fa.flash_rope_kv_write(qd, kd, vd, kc, vc, table.cuda(), cu.cuda(), max(lens), f if f is None else f.cuda(),
                                     starts=torch.tensor(starts, dtype=torch.int32).cuda(), interleaved=inter)
        qc = q.cuda().contiguous()
        fa.fa_rope_kv_write(qc, kd, vd, qc, kc, vc, table.cuda(), cu.cuda(), max(lens), f if f is None else f.cuda(),
                            starts=torch.tensor(starts, dtype=torch.int32).cuda(), interleaved=inter)
        assert torch.equal(qc[:T], ref[:T]) and torch.equal(qc[T:].cpu(), q[T:])


@pytest.mark.gpu
def test_write_checks_on_the_device():
    g = torch.Generator().manual_seed(1)
    k = inputs.randn((8, 2, 64), torch.bfloat16, g).cuda()
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, cu = torch.tensor([[0, 4], [2, -1]], dtype=torch.int32, device="cuda"), i32(0, 4, 8)

    def status(**kw):
        a = {"cu": cu, "mx": 4, "starts": None, **kw}
        kc.zero_(), vc.zero_()
        q = fa.flash_rope_kv_write(k, k, k, kc, vc, table, a["cu"], a["mx"], starts=a["starts"])
        try:
            fa.fa_check_device_error()
        except fa.FAError as e:
            return e.status, q
        return OK, q

    st, q = status()
    assert st == OK and torch.equal(q, k)
    st, q = status(starts=i32(14, 14))  # two tokens of each past page 0: page 4 does not exist, page -1 neither
    assert st == DEV_INDEX and torch.equal(q, k)
    assert torch.equal(kc[0, :, 14:16], k[0:2].transpose(0, 1)) and torch.equal(vc[2, :, 14:16], k[4:6].transpose(0, 1))
    assert int((kc != 0).any(-1).sum()) <= 8
    assert status(starts=i32(30, 0))[0] == DEV_INDEX  # behind the table
    for bad in ({"cu": i32(0, 5, 8)}, {"cu": i32(0, 4, 9)}, {"cu": i32(4, 2, 8)}, {"cu": i32(-1, 4, 8)},
                {"starts": i32(-1, 0)}, {"mx": 3}):
        assert status(**bad)[0] == DEV_SEQLENS, bad
    assert status(cu=i32(0, 0, 0))[0] == OK


@pytest.mark.gpu
def test_streams_and_graphs():
    g = torch.Generator().manual_seed(2)
    x = inputs.randn((300, 4, 64), torch.bfloat16, g).cuda()
    f, _ = fa.rope_frequencies(64)
    ref = fa.flash_rope(x, f)
    side = torch.cuda.Stream()
    y = fa.flash_rope(x, f, stream=side)
    dx = fa.flash_rope_bwd(x, f, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, ref) and torch.equal(dx, fa.flash_rope_bwd(x, f))
    graph, buf = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        out = fa.flash_rope(buf, f)
    buf.copy_(x.flip(0))
    graph.replay()
    assert torch.equal(out, fa.flash_rope(x.flip(0).contiguous(), f))
    empty = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert fa.flash_rope(empty, f).shape == empty.shape


@pytest.mark.gpu
@pytest.mark.parametrize("B,H", [(1, 4), (2, 1), (3, 2)])
def test_dense_of_no_tokens(B, H):
    x = torch.empty(B, H, 0, 64, dtype=torch.bfloat16, device="cuda")
    f, _ = fa.rope_frequencies(64)
    pos = torch.empty(B, 0, dtype=torch.int32, device="cuda")
    for y in (fa.flash_rope(x, f), fa.flash_rope(x, f, pos), fa.flash_rope_bwd(x, f)):
        assert y.shape == x.shape
    fa.fa_check_device_error()


@pytest.mark.gpu
def test_write_of_no_tokens():
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    c = torch.ones(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q = fa.flash_rope_kv_write(k, k, k, c, c, torch.zeros(2, 2, dtype=torch.int32, device="cuda"), i32(0, 0, 0), 0)
    fa.fa_check_device_error()
    assert q.shape == k.shape and (c == 1).all()


@pytest.mark.gpu
def test_one_token_in_each_of_many_sequences():
    """Sequences over two dimensions of the grid (more than 65535)."""
    B = 70000
    g = torch.Generator("cuda").manual_seed(1)
    k = torch.randn(B, 1, 64, generator=g, device="cuda").to(torch.float16)
    kc, vc = (torch.zeros(B, 1, 1, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    table = torch.randperm(B, generator=g, device="cuda").to(torch.int32)[:, None].contiguous()
    f, _ = fa.rope_frequencies(64)
    pos = torch.randint(0, 1 << 20, (B,), generator=g, device="cuda").to(torch.int32)
    q = fa.flash_rope_kv_write(k, k, k, kc, vc, table, torch.arange(B + 1, dtype=torch.int32, device="cuda"), 1, f, positions=pos)
    fa.fa_check_device_error()
    assert torch.equal(q, fa.flash_rope(k, f, pos))
    at = table[:, 0].long()
    assert torch.equal(kc[at, :, 0], q) and torch.equal(vc[at, :, 0], k)
