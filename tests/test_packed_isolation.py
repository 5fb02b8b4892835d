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
