"""Whole numbers past 32 bits given to the window operators and the 4-bit cache: no wrapping at the C boundary."""
import sys

import pytest
import torch

import exact_attention_54_gb300 as fa
from exact_attention_54_gb300 import build as fabuild

TOP = 2 ** 31 - 1
WIDE = [2 ** 31, 2 ** 32, 2 ** 32 + 10, 2 ** 40 + 3, sys.maxsize, 10 ** 30]


@pytest.fixture
def sent(monkeypatch):
    """Arguments that reach the library, as C takes them: (function, whole numbers)."""
    fabuild.build()
    lib = fa.load_library()
    calls = []

    def launch(fn, stream, tensors, *args, index=None):
        types = getattr(lib, fn).argtypes[len(tensors):len(tensors) + len(args)]
        calls.append((fn, [t(a).value for t, a in zip(types, args)]))

    monkeypatch.setattr(fa, "_launch", launch)
    return calls


def _calls():
    h = dict(dtype=torch.float16)
    q, k = torch.zeros(1, 4, 10, 64, **h), torch.zeros(1, 2, 10, 64, **h)
    qp, kp = torch.zeros(10, 4, 64, **h), torch.zeros(10, 2, 64, **h)
    lse, lsep = torch.zeros(1, 4, 10), torch.zeros(4, 10)
    cu, bt, sl = (torch.zeros(s, dtype=torch.int32) for s in (2, (1, 3), 1))
    pages = torch.zeros(4, 2, 16, 64, **h)
    c = fa.kv_cache_q4(4, 2, 16, 64, torch.float16, device="cpu")
    q1 = torch.zeros(1, 4, 1, 64, **h)
    ws = torch.zeros(1 << 16)
    # name -> call of window and sinks (or of the longest length)
    return {
        "fwd": lambda w, s: fa.flash_attention_window(q, k, k, w, s),
        "bwd": lambda w, s: fa.flash_attention_window_bwd(q, k, k, q, lse, q, w, s, workspace=ws),
        "fwd_varlen": lambda w, s: fa.flash_attention_window_varlen(qp, kp, kp, cu, cu, 10, w, s),
        "bwd_varlen": lambda w, s: fa.flash_attention_window_varlen_bwd(qp, kp, kp, qp, lsep, qp, cu, cu, 10, 10, w, s,
                                                                        workspace=ws),
        "decode": lambda w, s: fa.flash_decode_paged_window(q1, pages, pages, bt, sl, w, s),
        "decode_q4": lambda w, s: fa.flash_decode_paged_q4(q1, c, bt, sl, w, s),
        "write": lambda mx, _: fa.flash_kv_write_q4(kp, kp, c, bt, cu, mx),
        "read": lambda mx, _: fa.flash_kv_read_q4(c, bt, cu, 10, mx),
    }


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("name", ["fwd", "bwd", "fwd_varlen", "bwd_varlen", "decode", "decode_q4"])
def test_wide_windows_and_sinks_are_the_widest(sent, name, wide):
    call = _calls()[name]
    call(wide, wide)
    call(TOP, TOP)
    assert sent[0] == sent[1]
    call(-wide, -wide)  # refused by the library
    window, sinks = sent[2][1][-4:-2]
    assert window < 0 and sinks < 0


@pytest.mark.parametrize("wide", WIDE)
@pytest.mark.parametrize("name", ["write", "read"])
def test_wide_lengths_are_refused(sent, name, wide):
    call = _calls()[name]
    for x in (wide, -wide):
        call(x, 0)
    assert sent[0][1][2] > 1 << 30 and sent[1][1][2] < 0


@pytest.mark.parametrize("wide", WIDE)
def test_wide_arguments_of_the_packed_forms(sent, wide):
    qp, kp, cu = torch.zeros(10, 4, 64).half(), torch.zeros(10, 2, 64).half(), torch.zeros(2, dtype=torch.int32)
    for x in (wide, -wide):
        fa.flash_attention_window_varlen(qp, kp, kp, cu, cu, x, 5)
        fa.flash_attention_window_varlen_bwd(qp, kp, kp, qp, torch.zeros(4, 10), qp, cu, cu, x, x, 5,
                                             workspace=torch.zeros(9))
    assert sent[0][1][3] > 1 << 29 and sent[2][1][3] < 0
    assert all(n > 1 << 29 for n in sent[1][1][6:8]) and all(n < 0 for n in sent[3][1][6:8])


def test_workspaces_and_splits_of_wide_arguments(sent):
    for w in WIDE:
        assert fa.fa_bwd_window_workspace_bytes(1, 16, 1, 900, 900, 128, w, w) == \
            fa.fa_bwd_window_workspace_bytes(1, 16, 1, 900, 900, 128, TOP, TOP)
        assert fa.fa_bwd_window_varlen_workspace_bytes(2, 900, 600, 600, 16, 1, 128, w, w) == \
            fa.fa_bwd_window_varlen_workspace_bytes(2, 900, 600, 600, 16, 1, 128, TOP, TOP)
        assert fa.fa_bwd_window_workspace_bytes(1, 16, 1, 900, 900, 128, -w, 0) == 0
        assert fa.fa_bwd_window_workspace_bytes(1, 16, 1, w, 900, 128, 5, 0) == 0
        assert fa.fa_decode_splits(1, 8, 1, w) == fa.fa_decode_splits(1, 8, 1, TOP)
        assert fa.fa_decode_splits(1, 8, 1, -w) == 1
