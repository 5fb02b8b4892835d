"""Calls that allocate their own workspace name what they refuse, as the library does."""
import pytest
import torch

import exact_attention_54_gb300 as fa
from exact_attention_54_gb300 import build as fabuild

SHAPE, HEADDIM = -2, -3


@pytest.fixture(scope="module", autouse=True)
def lib():
    fabuild.build()
    return fa.load_library()


def _calls(dev, Hkv=3, D=64):
    z = lambda *s: torch.zeros(s, dtype=torch.float16, device=dev)  # noqa: E731
    q, k, lse = z(1, 4, 10, D), z(1, Hkv, 10, D), torch.zeros(1, 4, 10, device=dev)
    qp, kp, lsep = z(10, 4, D), z(10, Hkv, D), torch.zeros(4, 10, device=dev)
    cu = torch.tensor([0, 10], dtype=torch.int32).to(dev)
    return {
        "window_bwd": lambda: fa.flash_attention_window_bwd(q, k, k, q, lse, q, 5),
        "window_varlen_bwd": lambda: fa.flash_attention_window_varlen_bwd(qp, kp, kp, qp, lsep, qp, cu, cu, 10, 10, 5),
        "bwd": lambda: fa.flash_attention_bwd(q, q, q, q, lse, q),
        "varlen_bwd": lambda: fa.flash_attention_varlen_bwd(qp, qp, qp, qp, lsep, qp, cu, cu, 10, 10),
    }


@pytest.mark.parametrize("name", ["window_bwd", "window_varlen_bwd"])
@pytest.mark.parametrize("Hkv,D", [(3, 64), (2, 96)])
def test_a_workspace_is_there_for_sizes_that_are_refused(monkeypatch, name, Hkv, D):
    """(An empty tensor's pointer is NULL: the library would name that.)"""
    seen = []
    monkeypatch.setattr(fa, "_launch", lambda fn, stream, tensors, *a, **kw: seen.append(tensors[9].numel()))
    _calls("cpu", Hkv, D)[name]()
    assert seen[0] > 0


def test_no_sequences_and_a_given_workspace():
    q, pages = torch.zeros(0, 6, 1, 64).half(), torch.zeros(4, 2, 16, 64).half()
    bt, sl = torch.zeros(0, 3, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)
    ws = (torch.zeros(64), torch.zeros(1), torch.zeros(1), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        fa.flash_decode_paged_window(q, pages, pages, bt, sl, 10, workspace=ws)


@pytest.mark.gpu
@pytest.mark.parametrize("name,Hkv,D,status", [("window_bwd", 3, 64, SHAPE), ("window_varlen_bwd", 3, 64, SHAPE),
                                               ("window_bwd", 2, 96, HEADDIM), ("window_varlen_bwd", 2, 96, HEADDIM),
                                               ("bwd", 2, 96, HEADDIM), ("varlen_bwd", 2, 96, HEADDIM)])
def test_the_reason_is_the_librarys(name, Hkv, D, status):
    with pytest.raises(fa.FAError) as e:
        _calls("cuda", Hkv, D)[name]()
    assert e.value.status == status
