"""Packed sequences and their neighbours: infinities and NaNs in one sequence, or in rows of none, reach no other."""
import math

import pytest
import torch

import exact_attention_54_gb300 as fa
from exact_attention_54_gb300 import inputs

CASES = [
    # query lengths, key lengths (None: the same), H, Hkv, D, dtype, window, sinks, rows behind the last sequence
    ([70, 1, 0, 300, 129, 128, 40], None, 4, 2, 128, torch.bfloat16, 50, 4, 200),
    ([257, 128, 129, 5, 64, 63], None, 6, 1, 64, torch.float16, 100, 0, 130),
    ([0, 200, 64, 40, 33], [33, 150, 300, 0, 65], 6, 3, 128, torch.float16, 60, 1, 0),
    ([300, 10, 500, 77], [100, 500, 130, 3], 4, 1, 64, torch.bfloat16, 33, 140, 1),
    ([17] * 300, None, 2, 2, 128, torch.bfloat16, 5, 2, 64),                        # more than a schedule table
    ([700, 300, 60, 450], [700, 300, 60, 450], 16, 1, 128, torch.bfloat16, 500, 130, 90),  # cut into segments
    ([600, 500, 31, 127], None, 32, 1, 64, torch.float16, 10 ** 6, 200, 127),
]


def _make(lq, lk, H, Hkv, D, dtype, pad):
    g = torch.Generator().manual_seed(sum(lq) + D)
    cq, ck = inputs.cu_from_lengths(lq), inputs.cu_from_lengths(lk)
    Tq, Tk = int(cq[-1]) + pad, int(ck[-1]) + pad
    q, do = inputs.randn((Tq, H, D), dtype, g), inputs.randn((Tq, H, D), dtype, g)
    k, v = inputs.randn((Tk, Hkv, D), dtype, g), inputs.randn((Tk, Hkv, D), dtype, g)
    return cq, ck, q, k, v, do


def _spoiled(cu, every, what, x):
    """x with the rows of every second sequence (from `every` on) and those of none replaced."""
    x = x.clone()
    for b in range(every, cu.numel() - 1, 2):
        x[int(cu[b]):int(cu[b + 1])] = what
    x[int(cu[-1]):] = what
    return x


def _whole(cu, every):
    """Rows of the sequences that were left alone."""
    keep = [torch.arange(int(cu[b]), int(cu[b + 1])) for b in range(cu.numel() - 1) if (b - every) % 2]
    return torch.cat(keep).cuda() if keep else torch.zeros(0, dtype=torch.long, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("every", [0, 1])
@pytest.mark.parametrize("lq,lk,H,Hkv,D,dtype,window,sinks,pad", CASES)
def test_forward_keeps_to_its_sequence(lq, lk, H, Hkv, D, dtype, window, sinks, pad, every, what):
    lk = lk or lq
    cq, ck, q, k, v, _ = _make(lq, lk, H, Hkv, D, dtype, pad)
    c, d = cq.cuda(), ck.cuda()
    run = lambda *x: fa.flash_attention_window_varlen(*(t.cuda() for t in x), c, d, max(lq), window, sinks)  # noqa: E731
    o, lse = run(q, k, v)
    o2, lse2 = run(_spoiled(cq, every, what, q), *(_spoiled(ck, every, what, x) for x in (k, v)))
    fa.fa_check_device_error()
    rows = _whole(cq, every)
    assert torch.equal(o[rows], o2[rows]) and torch.equal(lse[:, rows], lse2[:, rows])


@pytest.mark.gpu
@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("every", [0, 1])
@pytest.mark.parametrize("lq,lk,H,Hkv,D,dtype,window,sinks,pad", CASES)
def test_gradients_keep_to_their_sequence(lq, lk, H, Hkv, D, dtype, window, sinks, pad, every, what):
    lk = lk or lq
    cq, ck, q, k, v, do = _make(lq, lk, H, Hkv, D, dtype, pad)
    c, d = cq.cuda(), ck.cuda()

    def run(q, k, v, do):
        q, k, v, do = (t.cuda() for t in (q, k, v, do))
        o, lse = fa.flash_attention_window_varlen(q, k, v, c, d, max(lq), window, sinks)
        if pad:  # rows of no sequence are left as they were made
            o[int(cq[-1]):], lse[:, int(cq[-1]):] = what, what
        return fa.flash_attention_window_varlen_bwd(q, k, v, o, lse, do, c, d, max(lq), max(lk), window, sinks)

    dq, dk, dv = run(q, k, v, do)
    dq2, dk2, dv2 = run(*(_spoiled(u, every, what, x) for u, x in ((cq, q), (ck, k), (ck, v), (cq, do))))
    fa.fa_check_device_error()
    rows, keys = _whole(cq, every), _whole(ck, every)
    assert torch.equal(dk[keys], dk2[keys]) and torch.equal(dv[keys], dv2[keys])
    # dq: fp32 sums in any order (under 2^-13 of the largest: some 20 addends, each off by 2^-24), one rounding each
    a, b = dq[rows].double(), dq2[rows].double()
    if a.numel():
        h = torch.finfo(dtype).eps / 2
        assert bool(((a - b).abs() <= 2 * h * a.abs() * (1 + h) + 2.0 ** -13 * a.abs().amax()).all())
    if pad:
        assert bool((dq2[int(cq[-1]):] == 0).all()) and bool((dq[int(cq[-1]):] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_gives_up_on_a_withheld_load_that_ends_a_sequence(D):
    """The second V tile, and the second step of queries, of a sequence that ends inside them: the call ends with an
    error, and the next one is correct."""
    n, tail = (200, 50) if D == 64 else (100, 50)
    lens = {"fwd": [200, tail], "bwd": [n, tail]}
    for which in ("fwd", "bwd"):
        cq, _, q, k, v, do = _make(lens[which], lens[which], 1, 1, D, torch.bfloat16, 30)
        c = cq.cuda()
        q, k, v, do = (t.cuda() for t in (q, k, v, do))
        mx = max(lens[which])
        fwd = lambda: fa.flash_attention_window_varlen(q, k, v, c, c, mx, 1000, 0)  # noqa: E731
        bwd = lambda o, lse: fa.flash_attention_window_varlen_bwd(q, k, v, o, lse, do, c, c, mx, mx, 1000, 0)  # noqa: E731
        good = fwd()
        want = bwd(*good) if which == "bwd" else good
        fa.fa_check_device_error()
        try:
            fa.fa_test_withhold_load(2, 20_000_000)
            bwd(*good) if which == "bwd" else fwd()
            with pytest.raises(fa.FAError) as e:
                fa.fa_check_device_error()
            assert e.value.status == -9
        finally:
            fa.fa_test_withhold_load(0, 0)
        got = bwd(*good) if which == "bwd" else fwd()
        fa.fa_check_device_error()
        T = int(cq[-1])
        for a, b in list(zip(got, want))[1 if which == "bwd" else 0:]:  # (dq's sums come in any order)
            a, b = (a[:, :T], b[:, :T]) if a.dim() == 2 else (a[:T], b[:T])
            assert torch.equal(a, b)
