"""Attention with a sliding window, sinks and shared key heads
(fa_fwd_window, fa_bwd_window and their packed forms) against the definition
in 64 bits."""
import math

import pytest
import torch

import exact_attention_54_gb300 as fa
import plain_ops
from exact_attention_54_gb300 import build as fabuild
from exact_attention_54_gb300 import inputs

NULL, SHAPE, HEADDIM, DTYPE, ALIGN, SCALE, WORKSPACE = -1, -2, -3, -4, -5, -7, -12
A, MIS = 0x10000, 0x10008
LONG = (1 << 29) + 1


@pytest.fixture(scope="module")
def lib():
    fabuild.build()
    return fa.load_library()


# -------------------------------------------------------------- on the CPU --

def _refusals(call, ptrs16, ptrs4, sizes):
    for n in ptrs16 + ptrs4:
        assert call(**{n: None}) == NULL, n
    assert call(dtype=2) == DTYPE
    for d in (32, 96, 256, 512):
        assert call(D=d) == HEADDIM
    for kw in sizes:
        assert call(**kw) == SHAPE, kw
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == SCALE
    for n in ptrs16:
        assert call(**{n: MIS}) == ALIGN, n
    for n in ptrs4:
        assert call(**{n: A + 2}) == ALIGN, n


HEADS = [{"H": 0}, {"Hkv": 0}, {"Hkv": 3}, {"H": 2, "Hkv": 4}, {"W": 0}, {"W": -1}, {"sinks": -1}]


def test_fwd_validation(lib):
    def call(B=1, H=4, Hkv=2, Sq=100, Sk=100, D=128, W=10, sinks=2, scale=0.1, dtype=1, **kw):
        p = [kw.get(n, A) for n in ("q", "k", "v", "o", "lse")]
        return lib.fa_fwd_window(*p, B, H, Hkv, Sq, Sk, D, W, sinks, scale, dtype, None)

    _refusals(call, ["q", "k", "v", "o"], ["lse"],
              HEADS + [{"B": 0}, {"Sq": 0}, {"Sk": 0}, {"Sq": LONG}, {"Sk": LONG}, {"B": 1 << 16, "H": 1 << 16}])


def test_fwd_varlen_validation(lib):
    def call(n=2, Tq=100, Tk=100, mx=60, H=4, Hkv=2, D=64, W=10, sinks=2, scale=0.1, dtype=0, **kw):
        p = [kw.get(x, A) for x in ("q", "k", "v", "o", "lse", "cq", "ck")]
        return lib.fa_fwd_window_varlen(*p, n, Tq, Tk, mx, H, Hkv, D, W, sinks, scale, dtype, None)

    _refusals(call, ["q", "k", "v", "o"], ["lse", "cq", "ck"],
              HEADS + [{"n": 0}, {"Tq": 0}, {"Tk": 0}, {"mx": 0}, {"Tq": LONG}, {"Tk": LONG}, {"mx": LONG}])


def test_bwd_validation(lib):
    names = ["q", "k", "v", "o", "do", "lse", "dq", "dk", "dv", "ws"]

    def call(wsb=1 << 30, B=1, H=4, Hkv=2, Sq=200, Sk=300, D=128, W=10, sinks=2, scale=0.1, dtype=1, **kw):
        return lib.fa_bwd_window(*[kw.get(n, A) for n in names], wsb, B, H, Hkv, Sq, Sk, D, W, sinks, scale, dtype,
                                 None)

    _refusals(call, [n for n in names if n != "lse"], ["lse"],
              HEADS + [{"B": 0}, {"Sq": 0}, {"Sk": 0}, {"Sq": LONG}, {"Sk": LONG}])
    need = lib.fa_bwd_window_workspace_bytes(1, 4, 2, 200, 300, 128, 10, 2)
    assert need >= lib.fa_bwd_workspace_bytes(1, 4, 200, 128) and call(wsb=need - 1) == WORKSPACE
    for bad in ((0, 4, 2, 200, 300, 128, 10, 2), (1, 4, 3, 200, 300, 128, 10, 2), (1, 4, 2, 0, 300, 128, 10, 2),
                (1, 4, 2, 200, LONG, 128, 10, 2), (1, 4, 2, 200, 300, 96, 10, 2), (1, 4, 2, 200, 300, 128, 0, 2)):
        assert lib.fa_bwd_window_workspace_bytes(*bad) == 0


def test_bwd_varlen_validation(lib):
    names = ["q", "k", "v", "o", "do", "lse", "dq", "dk", "dv", "ws"]

    def call(wsb=1 << 30, n=2, Tq=100, Tk=120, mq=60, mk=70, H=4, Hkv=2, D=64, W=10, sinks=2, scale=0.1, dtype=1, **kw):
        return lib.fa_bwd_window_varlen(*[kw.get(x, A) for x in names], wsb, kw.get("cq", A), kw.get("ck", A), n, Tq,
                                        Tk, mq, mk, H, Hkv, D, W, sinks, scale, dtype, None)

    _refusals(call, [x for x in names if x != "lse"], ["lse", "cq", "ck"],
              HEADS + [{"n": 0}, {"Tq": 0}, {"Tk": 0}, {"mq": 0}, {"mk": 0}, {"mq": LONG}, {"mk": LONG}])
    need = lib.fa_bwd_window_varlen_workspace_bytes(2, 100, 60, 70, 4, 2, 64, 10, 2)
    assert need >= lib.fa_bwd_varlen_workspace_bytes(100, 4, 64) and call(wsb=need - 1) == WORKSPACE
    for bad in ((0, 100, 60, 70, 4, 2, 64, 10, 2), (2, 0, 60, 70, 4, 2, 64, 10, 2), (2, 100, 0, 70, 4, 2, 64, 10, 2),
                (2, 100, 60, 70, 4, 2, 32, 10, 2), (2, 100, 60, 70, 4, 2, 64, 10, -1)):
        assert lib.fa_bwd_window_varlen_workspace_bytes(*bad) == 0


def test_binding_refuses():
    q, k = torch.zeros(1, 4, 10, 64, dtype=torch.float16), torch.zeros(1, 2, 10, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.flash_attention_window(q, k, k, 5)
    with pytest.raises(TypeError, match="v must be"):
        fa.flash_attention_window(q, k, k.bfloat16(), 5)
    with pytest.raises(ValueError, match="v must have shape"):
        fa.flash_attention_window(q, k, k[:, :1].contiguous(), 5)
    with pytest.raises(ValueError, match="k must have shape"):
        fa.flash_attention_window(q, k[..., :32].contiguous(), k, 5)
    with pytest.raises(ValueError, match="contiguous"):
        fa.flash_attention_window(q.transpose(2, 3).contiguous().transpose(2, 3), k, k, 5)
    lse = torch.zeros(1, 4, 10)
    with pytest.raises(ValueError, match="dout"):
        fa.flash_attention_window_bwd(q, k, k, q, lse, q[:, :2].contiguous(), 5)
    with pytest.raises(TypeError, match="lse"):
        fa.flash_attention_window_bwd(q, k, k, q, lse.double(), q, 5)
    cu = torch.tensor([0, 10], dtype=torch.int32)
    with pytest.raises(TypeError, match="cu_seqlens_k"):
        fa.flash_attention_window_varlen(q[0].transpose(0, 1).contiguous(), k[0].transpose(0, 1).contiguous(),
                                         k[0].transpose(0, 1).contiguous(), cu, cu.long(), 10, 5)


def test_plain_gradients_are_those_of_differences():
    """The plain form's gradients against central differences of its own forward."""
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn(n, 6, 4, generator=g, dtype=torch.float64) for n in (4, 2, 2, 4))
    r = plain_ops.window_attention(q, k, v, 3, 1, 0.5, do)
    f = lambda: float((plain_ops.window_attention(q, k, v, 3, 1, 0.5)["o"] * do).sum())  # noqa: E731
    for x, name in ((q, "dq"), (k, "dk"), (v, "dv")):
        for at in torch.randint(0, x.numel(), (12,), generator=g).tolist():
            keep = float(x.view(-1)[at])
            x.view(-1)[at] = keep + 1e-5
            up = f()
            x.view(-1)[at] = keep - 1e-5
            down = f()
            x.view(-1)[at] = keep
            assert abs((up - down) / 2e-5 - float(r[name].view(-1)[at])) < 1e-8, (name, at)


# -------------------------------------------------------------- on the GPU --

def draw(B, H, Hkv, Sq, Sk, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (inputs.randn((B, H, Sq, D), dtype, g), inputs.randn((B, Hkv, Sk, D), dtype, g),
            inputs.randn((B, Hkv, Sk, D), dtype, g), inputs.randn((B, H, Sq, D), dtype, g))


CASES = [
    # B, H, Hkv, Sq, Sk, D, dtype, window, sinks
    (1, 1, 1, 1, 1, 64, torch.float16, 1, 0),
    (1, 2, 1, 130, 130, 128, torch.bfloat16, 1, 0),          # the own key only: O = V
    (2, 4, 2, 300, 300, 64, torch.float16, 100, 1),
    (1, 4, 1, 515, 515, 128, torch.bfloat16, 128, 4),         # the window edge on tile borders
    (1, 2, 2, 700, 700, 128, torch.float16, 129, 0),
    (1, 3, 3, 640, 640, 64, torch.bfloat16, 127, 130),        # sinks over two tiles
    (1, 2, 2, 600, 600, 128, torch.bfloat16, 20, 300),        # more sinks than window
    (1, 6, 2, 777, 777, 64, torch.float16, 300, 0),
    (1, 2, 1, 260, 260, 128, torch.bfloat16, 2 ** 31 - 1, 2 ** 31 - 1),
    (1, 2, 1, 100, 400, 128, torch.float16, 30, 2),           # keys no query sees
    (1, 2, 1, 500, 130, 64, torch.bfloat16, 40, 0),           # queries that see nothing
    (1, 2, 2, 700, 100, 128, torch.float16, 50, 0),           # whole tiles of them
    (1, 2, 1, 500, 130, 128, torch.bfloat16, 40, 3),          # and with sinks: those alone
    (3, 8, 1, 257, 257, 128, torch.float16, 64, 16),
    (1, 1, 1, 2050, 2050, 64, torch.bfloat16, 511, 5),
    # few key tiles, each long: cut into segments
    (1, 16, 1, 1000, 1000, 128, torch.bfloat16, 600, 0),
    (1, 16, 1, 900, 900, 128, torch.float16, 400, 130),
    (2, 32, 2, 700, 500, 64, torch.float16, 2000, 3),
    (1, 32, 1, 300, 520, 128, torch.bfloat16, 250, 0),        # and key tiles that no query sees
]


def run_dense(q, k, v, do, window, sinks, **kw):
    qd, kd, vd, dd = (x.cuda() for x in (q, k, v, do))
    o, lse = fa.flash_attention_window(qd, kd, vd, window, sinks, **kw)
    dq, dk, dv = fa.flash_attention_window_bwd(qd, kd, vd, o, lse, dd, window, sinks, **kw)
    fa.fa_check_device_error()
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Hkv,Sq,Sk,D,dtype,window,sinks", CASES)
def test_dense_matches_definition(B, H, Hkv, Sq, Sk, D, dtype, window, sinks):
    q, k, v, do = draw(B, H, Hkv, Sq, Sk, D, dtype, seed=Sq + Sk + H)
    got = run_dense(q, k, v, do, window, sinks)
    for b in range(B):
        ref = plain_ops.window_attention(q[b], k[b], v[b], window, sinks, D ** -0.5, do[b], dtype)
        plain_ops.assert_window_close({n: x[b] for n, x in got.items()}, ref, f"sequence {b}")


PACKED = [
    # query lengths, key lengths, H, Hkv, D, dtype, window, sinks
    ([1], [1], 1, 1, 128, torch.float16, 1, 0),
    ([70, 1, 0, 300], [70, 1, 0, 300], 4, 2, 128, torch.bfloat16, 50, 4),
    ([257, 128, 129], [257, 128, 129], 2, 1, 64, torch.float16, 100, 0),
    ([0, 200, 64, 40], [33, 150, 300, 0], 6, 3, 128, torch.float16, 60, 1),   # lengths that differ; no queries, no keys
    ([300, 10], [100, 500], 4, 1, 64, torch.bfloat16, 33, 0),                 # rows that see nothing
    ([17] * 300, [17] * 300, 2, 2, 64, torch.bfloat16, 5, 2),                 # more sequences than a schedule table
    ([600, 450, 512], [600, 450, 512], 8, 2, 128, torch.bfloat16, 256, 140),
    # segments, some of them with nothing to do
    ([700, 300, 0, 60], [700, 300, 50, 0], 16, 1, 128, torch.bfloat16, 500, 0),
    ([130, 600], [500, 600], 32, 1, 64, torch.float16, 10 ** 6, 200),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk,H,Hkv,D,dtype,window,sinks", PACKED)
def test_packed_matches_definition(lq, lk, H, Hkv, D, dtype, window, sinks):
    g = torch.Generator().manual_seed(sum(lq) + D)
    cq, ck = inputs.cu_from_lengths(lq), inputs.cu_from_lengths(lk)
    Tq, Tk = int(cq[-1]), int(ck[-1])
    q, do = inputs.randn((Tq, H, D), dtype, g), inputs.randn((Tq, H, D), dtype, g)
    k, v = inputs.randn((Tk, Hkv, D), dtype, g), inputs.randn((Tk, Hkv, D), dtype, g)
    qd, kd, vd, dd, cqd, ckd = (x.cuda() for x in (q, k, v, do, cq, ck))
    o, lse = fa.flash_attention_window_varlen(qd, kd, vd, cqd, ckd, max(lq), window, sinks)
    dq, dk, dv = fa.flash_attention_window_varlen_bwd(qd, kd, vd, o, lse, dd, cqd, ckd, max(lq), max(lk), window,
                                                      sinks)
    fa.fa_check_device_error()
    for b in range(len(lq)):
        sq, sk = slice(int(cq[b]), int(cq[b + 1])), slice(int(ck[b]), int(ck[b + 1]))
        t = lambda x: x.transpose(0, 1)  # noqa: E731
        ref = plain_ops.window_attention(t(q[sq]), t(k[sk]), t(v[sk]), window, sinks, D ** -0.5, t(do[sq]), dtype)
        got = {"o": t(o[sq]), "lse": lse[:, sq], "dq": t(dq[sq]), "dk": t(dk[sk]), "dv": t(dv[sk])}
        plain_ops.assert_window_close(got, ref, f"sequence {b}")


def test_long_key_tiles_take_more_workspace(lib):
    """The cases above that are to be cut into segments are."""
    for B, H, Hkv, Sq, Sk, D, _, window, sinks in CASES[-4:]:
        assert lib.fa_bwd_window_workspace_bytes(B, H, Hkv, Sq, Sk, D, window, sinks) >= \
            lib.fa_bwd_workspace_bytes(B, H, Sq, D) + B * Hkv * 2 * 128 * D * 4 * 8
    for lq, lk, H, Hkv, D, _, window, sinks in PACKED[-2:]:
        assert lib.fa_bwd_window_varlen_workspace_bytes(len(lq), sum(lq), max(lq), max(lk), H, Hkv, D, window,
                                                        sinks) >= \
            lib.fa_bwd_varlen_workspace_bytes(sum(lq), H, D) + len(lq) * Hkv * 2 * 128 * D * 4 * 8


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_wide_window_is_causal_attention(D):
    """Forward: bit for bit. The gradients' sums may be cut elsewhere: against the definition."""
    q, k, v, do = draw(2, 3, 3, 600, 600, D, torch.bfloat16, seed=3)
    got = run_dense(q, k, v, do, 600, 0)
    o, lse = fa.flash_attention(*(x.cuda() for x in (q, k, v)), causal=True)
    assert torch.equal(got["o"], o) and torch.equal(got["lse"], lse)
    for b in range(2):
        ref = plain_ops.window_attention(q[b], k[b], v[b], 600, 0, D ** -0.5, do[b])
        plain_ops.assert_window_close({n: x[b] for n, x in got.items()}, ref, f"sequence {b}")


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_shared_heads_are_repeated_heads(D):
    """Forward: equal bit for bit to the same key head given to every query head. Many items and units per CTA."""
    q, k, v, do = draw(4, 24, 3, 500, 500, D, torch.float16, seed=4)
    got = run_dense(q, k, v, do, 200, 4)
    wide = run_dense(q, k.repeat_interleave(8, 1), v.repeat_interleave(8, 1), do, 200, 4)
    assert torch.equal(got["o"], wide["o"]) and torch.equal(got["lse"], wide["lse"])
    again = run_dense(q, k, v, do, 200, 4)
    for n in ("o", "lse", "dk", "dv"):
        assert torch.equal(got[n], again[n]), n
    # gradients of shared heads: the sum, within the roundings of its eight addends and of itself
    for n in ("dk", "dv"):
        parts = wide[n].double().view(4, 3, 8, 500, D)
        bound = 2.0 ** -11 * (parts.abs().sum(2) + parts.sum(2).abs()) * 1.01 + 2.0 ** -16 * parts.abs().amax()
        assert ((got[n].double() - parts.sum(2)).abs() <= bound).all(), n


@pytest.mark.gpu
def test_hidden_tiles_are_never_read():
    """NaN keys and values in tiles that no query sees, NaN queries in tiles behind them."""
    q, k, v, do = draw(1, 2, 1, 1000, 1400, 128, torch.bfloat16, seed=5)
    base = run_dense(q, k, v, do, 100, 4)
    k[:, :, 1024:], v[:, :, 1024:] = math.nan, math.nan  # key tiles past the last query
    got = run_dense(q, k, v, do, 100, 4)
    assert all(torch.equal(got[n], base[n]) for n in ("o", "lse"))
    assert torch.equal(got["dk"][:, :, :1024], base["dk"][:, :, :1024])
    # queries [512, 640) see no key of tiles 1 and 2: NaNs there reach only the queries around them
    q2, k2, v2, do2 = draw(1, 2, 1, 1000, 1000, 128, torch.bfloat16, seed=6)
    base = run_dense(q2, k2, v2, do2, 100, 4)
    k2[:, :, 128:384], v2[:, :, 128:384] = math.nan, math.nan
    o = run_dense(q2, k2, v2, do2, 100, 4)["o"]
    assert torch.equal(o[:, :, 512:], base["o"][:, :, 512:]) and torch.equal(o[:, :, :128], base["o"][:, :, :128])


@pytest.mark.gpu
def test_scale_stream_and_given_workspace():
    q, k, v, do = draw(1, 4, 2, 333, 333, 128, torch.float16, seed=7)
    ref = plain_ops.window_attention(q[0], k[0], v[0], 77, 3, 0.3, do[0], torch.float16)
    qd, kd, vd, dd = (x.cuda() for x in (q, k, v, do))
    ws = torch.full((fa.fa_bwd_window_workspace_bytes(1, 4, 2, 333, 333, 128, 77, 3) // 4,), math.nan, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o, lse = fa.flash_attention_window(qd, kd, vd, 77, 3, scale=0.3)
        dq, dk, dv = fa.flash_attention_window_bwd(qd, kd, vd, o, lse, dd, 77, 3, scale=0.3, workspace=ws)
    fa.fa_check_device_error(s)
    plain_ops.assert_window_close({n: x[0] for n, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv))},
                                  ref)


@pytest.mark.gpu
def test_captured_training_step():
    """Forward and backward captured into a graph, replayed on new inputs."""
    q, k, v, do = (x.cuda() for x in draw(1, 4, 2, 400, 400, 128, torch.bfloat16, seed=8))
    def step():
        o, lse = fa.flash_attention_window(q, k, v, 100, 4)
        return (o, lse, *fa.flash_attention_window_bwd(q, k, v, o, lse, do, 100, 4))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (9, 10):
        for x, y in zip((q, k, v, do), draw(1, 4, 2, 400, 400, 128, torch.bfloat16, seed=seed)):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        ref = plain_ops.window_attention(q[0].cpu(), k[0].cpu(), v[0].cpu(), 100, 4, 128 ** -0.5, do[0].cpu())
        plain_ops.assert_window_close({n: x[0] for n, x in zip(("o", "lse", "dq", "dk", "dv"), out)}, ref)
    fa.fa_check_device_error()


@pytest.mark.gpu
def test_bad_offsets_are_reported():
    g = torch.Generator().manual_seed(11)
    q, k = inputs.randn((100, 2, 64), torch.float16, g).cuda(), inputs.randn((100, 1, 64), torch.float16, g).cuda()
    for cu, mx in (([0, 60, 50], 60), ([0, 60, 101], 60), ([0, 60, 100], 59)):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, lse = torch.full_like(q, 3.0), torch.full((2, 100), 3.0, device="cuda")
        fa.fa_fwd_window_varlen(q, k, k, o, lse, c, c, mx, 20, 1)
        with pytest.raises(fa.FAError) as e:
            fa.fa_check_device_error()
        assert e.value.status == -13 and (o == 3).all() and (lse == 3).all()
        ws = torch.empty(fa.fa_bwd_window_varlen_workspace_bytes(2, 100, mx, mx, 2, 1, 64, 20) // 4, device="cuda")
        dk = torch.full_like(k, 3.0)
        fa.fa_bwd_window_varlen(q, k, k, q, q, lse, torch.empty_like(q), dk, torch.empty_like(k), ws, c, c, mx, mx, 20)
        with pytest.raises(fa.FAError) as e:
            fa.fa_check_device_error()
        assert e.value.status == -13


@pytest.mark.gpu
def test_prefill_write_decode_together():
    """A prompt's windowed prefill, its keys and values into 16-bit pages and the 4-bit cache, then the next
    token: the paged decode gives the row that the prefill of one more token gives."""
    H, Hkv, D, block, n, W, sinks, dtype = 8, 2, 128, 16, 300, 90, 4, torch.bfloat16
    q, k, v, _ = draw(1, H, Hkv, n, n, D, dtype, seed=12)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    ref = plain_ops.window_attention(q[0], k[0], v[0], W, sinks, D ** -0.5, dtype=dtype)
    o, lse = fa.flash_attention_window(qd, kd, vd, W, sinks)
    plain_ops.assert_window_close({"o": o[0], "lse": lse[0]}, ref)
    nb = -(-n // block)
    table = torch.arange(nb, dtype=torch.int32, device="cuda").flip(0).view(1, nb).contiguous()
    pages = [torch.zeros(nb, Hkv, block, D, dtype=dtype, device="cuda") for _ in range(2)]
    pos = torch.arange(n, device="cuda")
    for x, src in zip(pages, (kd, vd)):
        x[table[0].long()[pos // block], :, pos % block] = src[0].transpose(0, 1)
    sl = torch.tensor([n], dtype=torch.int32, device="cuda")
    do, dl = fa.flash_decode_paged_window(qd[:, :, -1:].contiguous(), *pages, table, sl, W, sinks)
    plain_ops.assert_window_close({"o": do[0], "lse": dl[0][:, None]}, {x: y[:, -1:] for x, y in ref.items()})
    # 4 bits: write the prompt, read it back as the next chunk's prefix, decode over it
    cache = fa.kv_cache_q4(nb, Hkv, block, D, dtype)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    kp, vp = kd[0].transpose(0, 1).contiguous(), vd[0].transpose(0, 1).contiguous()
    fa.flash_kv_write_q4(kp, vp, cache, table, cu, n)
    kr, vr = fa.flash_kv_read_q4(cache, table, cu, n, n)
    ref = plain_ops.window_attention(q[0], kr.cpu().transpose(0, 1), vr.cpu().transpose(0, 1), W, sinks, D ** -0.5,
                                     dtype=dtype)
    o, lse = fa.flash_attention_window_varlen(qd[0].transpose(0, 1).contiguous(), kr, vr, cu, cu, n, W, sinks)
    plain_ops.assert_window_close({"o": o.transpose(0, 1), "lse": lse}, ref)
    fa.flash_decode_paged_q4(qd[:, :, -1:].contiguous(), cache, table, sl, W, sinks)
    fa.fa_check_device_error()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("packed", [False, True])
def test_gives_up_on_a_withheld_load_and_the_next_call_is_correct(D, packed):
    """Forward and backward, whose waits run out when one tile load never comes (see fa_test_withhold_load)."""
    q, k, v, do = draw(1, 16, 1, 900, 900, D, torch.bfloat16, seed=30 + D)
    ref = plain_ops.window_attention(q[0], k[0], v[0], 400, 130, D ** -0.5, do[0])
    qd, kd, vd, dd = ((x[0].transpose(0, 1).contiguous() if packed else x).cuda() for x in (q, k, v, do))
    cu = torch.tensor([0, 900], dtype=torch.int32, device="cuda")
    if packed:
        fwd = lambda: fa.flash_attention_window_varlen(qd, kd, vd, cu, cu, 900, 400, 130)  # noqa: E731
        bwd = lambda o, lse: fa.flash_attention_window_varlen_bwd(qd, kd, vd, o, lse, dd, cu, cu, 900, 900, 400, 130)  # noqa: E731
    else:
        fwd = lambda: fa.flash_attention_window(qd, kd, vd, 400, 130)  # noqa: E731
        bwd = lambda o, lse: fa.flash_attention_window_bwd(qd, kd, vd, o, lse, dd, 400, 130)  # noqa: E731
    good = fwd()
    fa.fa_check_device_error()
    try:
        for f, args in ((fwd, ()), (bwd, good)):
            torch.cuda.synchronize()
            fa.fa_test_withhold_load(2, 20_000_000)
            f(*args)
            with pytest.raises(fa.FAError) as e:
                fa.fa_check_device_error()
            assert e.value.status == -9
            fa.fa_test_withhold_load(0, 0)
    finally:
        fa.fa_test_withhold_load(0, 0)
    o, lse = fwd()
    got = {"o": o, "lse": lse, **dict(zip(("dq", "dk", "dv"), bwd(o, lse)))}
    fa.fa_check_device_error()
    plain_ops.assert_window_close({n: x if n == "lse" and packed else x.transpose(0, 1) if packed else x[0]
                                   for n, x in got.items()}, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_a_withheld_load_is_always_missed(packed):
    """D = 128, gradients: CTAs take units from a counter, and some of them none; the load is withheld wherever the
    first unit went."""
    q, k, v, do = draw(1, 16, 1, 900, 900, 128, torch.bfloat16, seed=31)
    qd, kd, vd, dd = ((x[0].transpose(0, 1).contiguous() if packed else x).cuda() for x in (q, k, v, do))
    cu = torch.tensor([0, 900], dtype=torch.int32, device="cuda")
    if packed:
        o, lse = fa.flash_attention_window_varlen(qd, kd, vd, cu, cu, 900, 400, 130)
    else:
        o, lse = fa.flash_attention_window(qd, kd, vd, 400, 130)
    fa.fa_check_device_error()
    try:
        fa.fa_test_withhold_load(2, 2_000_000)
        for i in range(40):
            if packed:
                fa.flash_attention_window_varlen_bwd(qd, kd, vd, o, lse, dd, cu, cu, 900, 900, 400, 130)
            else:
                fa.flash_attention_window_bwd(qd, kd, vd, o, lse, dd, 400, 130)
            with pytest.raises(fa.FAError) as e:
                fa.fa_check_device_error()
            assert e.value.status == -9, i
    finally:
        fa.fa_test_withhold_load(0, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv,D,dtype,W,sinks", [(8, 2, 128, torch.bfloat16, 90, 4), (6, 3, 64, torch.float16, 40, 0)])
def test_decode_behind_a_prefill_and_a_written_prompt(H, Hkv, D, dtype, W, sinks):
    """A prompt prefilled and written to the 4-bit cache, then single tokens one after the other, each written and then
    attended to: every token's o and lse are those of the definition over what the cache stands for, not rounded."""
    block, n, more = 16, 150, 3
    q, k, v, _ = draw(1, H, Hkv, n + more, n + more, D, dtype, seed=14 + D)
    qd, kd, vd = (x[0].transpose(0, 1).contiguous().cuda() for x in (q, k, v))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    o, lse = fa.flash_attention_window_varlen(qd[:n], kd[:n], vd[:n], cu, cu, n, W, sinks)
    ref = plain_ops.window_attention(q[0, :, :n], k[0, :, :n], v[0, :, :n], W, sinks, D ** -0.5, dtype=dtype)
    plain_ops.assert_window_close({"o": o.transpose(0, 1), "lse": lse}, ref)
    nb = -(-(n + more) // block)
    table = torch.arange(nb, dtype=torch.int32, device="cuda").flip(0).view(1, nb).contiguous()
    cache = fa.kv_cache_q4(nb, Hkv, block, D, dtype)
    fa.flash_kv_write_q4(kd[:n], vd[:n], cache, table, cu, n)
    one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    G = H // Hkv
    for t in range(n, n + more):
        at = torch.tensor([t], dtype=torch.int32, device="cuda")
        fa.flash_kv_write_q4(kd[t:t + 1], vd[t:t + 1], cache, table, one, 1, starts=at)
        o, lse = fa.flash_decode_paged_q4(qd[t].view(1, H, 1, D), cache, table, at + 1, W, sinks)
        fa.fa_check_device_error()
        c = [x.cpu() for x in cache]

        def values(page, h):
            return (plain_ops.q4_values(c[0][page, h // G], c[1][page, h // G]),
                    plain_ops.q4_values(c[2][page, h // G], c[3][page, h // G]),
                    c[3][page, h // G].double().repeat_interleave(32, -1))

        ref = plain_ops.decode(q[:, :, t:t + 1], values, table.cpu(), [t + 1], block, W, sinks, D ** -0.5)
        plain_ops.assert_attention_close(o, lse, *ref, dtype, f"token {t}")
