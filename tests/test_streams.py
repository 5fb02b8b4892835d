"""Calls with ``stream=``: what they allocate, clear and launch is in that stream's order, behind the current one's."""
import contextlib
import inspect

import pytest
import torch

import exact_attention_54_gb300 as fa
import plain_ops
from exact_attention_54_gb300 import build as fabuild
from exact_attention_54_gb300 import inputs


def _calls(dev, dtype=torch.float16, seed=0):
    """Every allocating call by name, and the 16-bit inputs they read."""
    g = torch.Generator().manual_seed(seed)
    read = []

    def r(*s):
        read.append(inputs.randn(s, dtype, g).to(dev))
        return read[-1]

    B, H, Hkv, S, D, W, sinks, block = 2, 8, 2, 300, 128, 90, 4, 16
    q, k, v, do, lse = r(B, H, S, D), r(B, Hkv, S, D), r(B, Hkv, S, D), r(B, H, S, D), r(B, H, S).float()
    T = B * S
    qp, kp, vp, dop, lsep = r(T, H, D), r(T, Hkv, D), r(T, Hkv, D), r(T, H, D), r(H, T).float()
    cu = torch.tensor([0, S, T], dtype=torch.int32).to(dev)
    nb = -(-S // block)
    table = torch.arange(B * nb, dtype=torch.int32).view(B, nb).to(dev)
    lens = torch.full((B,), S, dtype=torch.int32).to(dev)
    pages = [r(B * nb, Hkv, block, D) for _ in range(2)]
    cache = fa.kv_cache_q4(B * nb, Hkv, block, D, dtype, device=dev)
    cache = fa.KVCacheQ4(cache.k_codes + 83, r(*cache.k_scales.shape).abs_(), cache.v_codes + 196,
                         r(*cache.v_scales.shape).abs_())
    q1, q2 = r(B, H, 1, D), r(B, Hkv, 1, D)
    return read, {
        "window": lambda **kw: fa.flash_attention_window(q, k, v, W, sinks, **kw),
        "window_bwd": lambda **kw: fa.flash_attention_window_bwd(q, k, v, q, lse, do, W, sinks, **kw),
        "window_varlen": lambda **kw: fa.flash_attention_window_varlen(qp, kp, vp, cu, cu, S, W, sinks, **kw),
        "window_varlen_bwd": lambda **kw: fa.flash_attention_window_varlen_bwd(qp, kp, vp, qp, lsep, dop, cu, cu, S, S, W,
                                                                               sinks, **kw),
        "read": lambda **kw: fa.flash_kv_read_q4(cache, table, cu, T, S, **kw),
        "decode": lambda **kw: fa.flash_decode_paged_window(q1, *pages, table, lens, W, sinks, **kw),
        "dense": lambda **kw: fa.flash_attention(q, q, q, True, **kw),
        "dense_bwd": lambda **kw: fa.flash_attention_bwd(q, q, q, q, lse, do, True, **kw),
        "varlen": lambda **kw: fa.flash_attention_varlen(qp, qp, qp, cu, cu, S, True, **kw),
        "varlen_bwd": lambda **kw: fa.flash_attention_varlen_bwd(qp, qp, qp, qp, lsep, dop, cu, cu, S, S, True, **kw),
        "splitkv": lambda **kw: fa.flash_decode(q1, q, q, 9, **kw),
        "splitkv_fused": lambda **kw: fa.flash_decode(q1, q, q, 9, fused=True, **kw),
        "paged": lambda **kw: fa.flash_decode_paged(q2, *pages, table, lens, 9, **kw),
        "paged_fused": lambda **kw: fa.flash_decode_paged(q2, *pages, table, lens, 9, fused=True, **kw),
        "decode_q4": lambda **kw: fa.flash_decode_paged_q4(q1, cache, table, lens, W, sinks, **kw),
    }


NAMES = ["window", "window_bwd", "window_varlen", "window_varlen_bwd", "read", "decode", "decode_q4", "dense",
         "dense_bwd", "varlen", "varlen_bwd", "splitkv", "splitkv_fused", "paged", "paged_fused"]


# -------------------------------------------------------------- on the CPU --

class _Stream:
    def __init__(self, handle, dev="cuda:0"):
        self.cuda_stream, self.device, self.waited = handle, torch.device(dev), []

    def wait_stream(self, other):
        self.waited.append(other)


@pytest.fixture
def streams(monkeypatch):
    """Streams that only keep account: the current one, and under which one each tensor was made and each kernel
    launched."""
    fabuild.build()
    fa.load_library()
    from torch._subclasses.fake_tensor import FakeTensorMode
    log = {"now": _Stream(0), "made": [], "launched": []}

    @contextlib.contextmanager
    def enter(s):
        before, log["now"] = log["now"], s
        yield
        log["now"] = before

    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: log["now"])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev=None: _Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: _Stream(handle))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)

    def launched(fn, stream, *args, **kw):
        log["launched"].append(log["now"].cuda_stream if stream is None else fa._stream(stream))

    monkeypatch.setattr(fa, "_launch", launched)
    for name in ("fa_fwd", "fa_fwd_varlen", "fa_bwd", "fa_bwd_varlen", "fa_decode_splitkv", "fa_decode_splitkv_fused",
                 "fa_splitkv_merge", "fa_decode_paged_splitkv", "fa_decode_paged_splitkv_fused"):
        at = list(inspect.signature(getattr(fa, name)).parameters).index("stream")
        monkeypatch.setattr(fa, name, lambda *a, _at=at: launched(None, a[_at] if len(a) > _at else None))
    with FakeTensorMode():
        _, calls = _calls("cuda")
        for name in ("empty", "zeros", "empty_like"):
            def made(*a, _f=getattr(torch, name), **kw):
                log["made"].append(log["now"].cuda_stream)
                return _f(*a, **kw)
            monkeypatch.setattr(torch, name, made)
        yield log, calls


@pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("as_handle", [False, True])
def test_allocations_are_the_given_streams(streams, name, as_handle):
    log, calls = streams
    s, outer = _Stream(77), log["now"]
    calls[name](stream=77 if as_handle else s)
    assert log["made"] and set(log["made"]) == {77} and set(log["launched"]) == {77}
    assert as_handle or s.waited == [outer]
    assert log["now"] is outer


@pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
@pytest.mark.parametrize("name", NAMES)
def test_no_stream_is_the_current_one(streams, name):
    log, calls = streams
    calls[name]()
    assert set(log["made"]) == {0} and set(log["launched"]) == {0} and log["now"].waited == []
    calls[name](stream=log["now"])
    assert set(log["launched"]) == {0} and log["now"].waited == []


def test_stream_of_another_device_is_refused(streams):
    log, calls = streams
    with pytest.raises(ValueError, match="stream must be one of cuda:0"):
        calls["decode"](stream=_Stream(5, "cuda:1"))
    assert log["launched"] == []


# -------------------------------------------------------------- on the GPU --

@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_given_stream_without_synchronising(name):
    """Inputs still being made on the current stream, memory of the pool that holds anything, and outputs' and
    workspaces' memory of the current stream's pool written over right after the call."""
    s = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    sizes = (16, 1 << 12, 1 << 20, 1 << 22)
    fill = lambda n: torch.full((n,), 0x7fc00005, dtype=torch.int32, device="cuda")  # noqa: E731
    for seed in (1, 2):
        read, calls = _calls("cuda", seed=seed)
        want = [t.clone() for t in calls[name]()]
        kept = [t.clone() for t in read]
        for t in read:
            t.zero_()
        for n in sizes:
            junk = [fill(n) for _ in range(4)]
            with torch.cuda.stream(s):
                junk += [fill(n) for _ in range(4)]
            del junk
        torch.cuda.synchronize()
        for _ in range(20):  # the current stream is busy for a while, then makes the inputs
            big = big @ big
            big /= big.abs().max()
        for t, x in zip(read, kept):
            t.copy_(x)
        got = calls[name](stream=s)
        for n in sizes:
            for _ in range(4):
                fill(n)
        torch.cuda.synchronize()
        fa.fa_check_device_error()
        for i, (a, b) in enumerate(zip(got, want)):
            # (the LSE given is no forward's: some values pass the 16-bit type's range, in both calls alike)
            a, b = a.double(), b.double()
            close = (a == b) | (torch.isnan(a) & torch.isnan(b))
            if name.endswith("bwd") and i == 0:  # dq: fp32 sums in any order, then one rounding
                h, fine = plain_ops.half_step(got[0].dtype), torch.isfinite(b)
                close |= fine & ((a - b).abs() <= 2 * h * b.abs() + 2.0 ** -13 * b[fine].abs().amax())
            assert bool(close.all()), (seed, i)


def _same(a, b):
    a, b = a.double(), b.double()
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["window", "window_varlen", "read", "decode", "decode_q4", "dense", "splitkv_fused"])
def test_handle_and_default_stream(name):
    """A raw handle in place of the stream, and 0 for the default stream, from inside another one."""
    _, calls = _calls("cuda")
    want = calls[name]()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s.cuda_stream, 0):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = calls[name](stream=handle)
            assert torch.cuda.current_stream() != s
        torch.cuda.synchronize()
        fa.fa_check_device_error()
        assert all(_same(a, b) for a, b in zip(got, want)), handle


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["window", "decode", "decode_q4", "read"])
def test_side_stream_in_a_captured_graph(name):
    """Captured with ``stream=`` another stream than the graph's: it joins the capture, and replays see new inputs."""
    read, calls = _calls("cuda")
    want = [t.clone() for t in calls[name]()]
    kept = [t.clone() for t in read]
    s = torch.cuda.Stream()
    calls[name](stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = calls[name](stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for t in read:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert not all(_same(a, b) for a, b in zip(out, want))
    for t, x in zip(read, kept):
        t.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    fa.fa_check_device_error()
    assert all(_same(a, b) for a, b in zip(out, want))
