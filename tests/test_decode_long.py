"""One-token attention over one long sequence with few key heads: the partitions that fa_decode_splits names."""
import pytest
import torch

import exact_attention_54_gb300 as fa
import plain_ops
from exact_attention_54_gb300 import build as fabuild


@pytest.fixture(scope="module", autouse=True)
def lib():
    fabuild.build()
    return fa.load_library()


@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 1), (16, 1), (16, 2)])
def test_long_sequences_take_more_partitions_than_there_are_sms(H, Hkv):
    units = Hkv
    assert units * fa.fa_decode_splits(1, H, Hkv, 1 << 20) >= 152
    assert units * fa.fa_decode_splits(1, H, Hkv, 1 << 24) >= 3 * 152


def test_partitions_grow_with_the_keys_within_the_limit():
    for B, H, Hkv in ((1, 8, 1), (1, 16, 2), (1, 32, 8), (4, 8, 1), (64, 32, 8)):
        last = 1
        for keys in (1, 100, 1000, 4096, 16384, 65536, 131072, 1 << 18, 1 << 20, 1 << 24, 1 << 30, (1 << 31) - 1):
            n = fa.fa_decode_splits(B, H, Hkv, keys)
            assert 1 <= n <= fa.FA_MAX_SPLITS and n <= max(keys, 1)
            if keys >= 1 << 17 and B * Hkv * (keys // 16 + 16) < 1 << 31:  # (past that, tiles are not dealt out)
                assert n >= last, (B, H, Hkv, keys)
            last = n


def test_sequences_up_to_131072_keys_take_64_at_most():
    """What was measured best there (more partitions cost more to join than they gain)."""
    for keys in (16384, 65536, 131072):
        assert fa.fa_decode_splits(1, 8, 1, keys) == 64 and fa.fa_decode_splits(1, 16, 2, keys) <= 64


# -------------------------------------------------------------- on the GPU --

@pytest.mark.gpu
@pytest.mark.parametrize("q4", [False, True], ids=["16bit", "q4"])
@pytest.mark.parametrize("H,Hkv,D,n,dtype", [(8, 1, 64, 600_001, torch.float16), (4, 2, 128, 300_007, torch.bfloat16)])
def test_many_partitions_match_the_definition(q4, H, Hkv, D, n, dtype):
    block = 256
    nb = -(-n // block)
    g = torch.Generator("cuda").manual_seed(n)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    q, k, v = r(1, H, 1, D), r(n, Hkv, D), r(n, Hkv, D)
    table = torch.randperm(nb, generator=g, device="cuda").to(torch.int32).view(1, nb)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    if q4:
        cache = fa.kv_cache_q4(nb, Hkv, block, D, dtype)
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        fa.flash_kv_write_q4(k, v, cache, table, cu, n)
        o, lse = fa.flash_decode_paged_q4(q, cache, table, lens)
        pos = torch.arange(n, device="cuda")
        at = table[0].long()[pos // block], slice(None), pos % block
        kd, vd = (plain_ops.q4_values(c[at].cpu(), s[at].cpu()).cuda() for c, s in (cache[:2], cache[2:]))
        scales = cache.v_scales[at].double().repeat_interleave(plain_ops.GROUP, -1)
    else:
        pages = []
        for x in (k, v):
            p = torch.zeros(nb * block, Hkv, D, dtype=dtype, device="cuda")
            p[:n] = x
            out = torch.empty(nb, Hkv, block, D, dtype=dtype, device="cuda")
            out[table[0].long()] = p.view(nb, block, Hkv, D).transpose(1, 2)
            pages.append(out)
        o, lse = fa.flash_decode_paged_window(q, *pages, table, lens, 0)
        kd, vd = k.double(), v.double()
    fa.fa_check_device_error()
    assert fa.fa_decode_splits(1, H, Hkv, nb * block) > 64
    G = H // Hkv
    ro, size, low = (torch.zeros(1, H, D, dtype=torch.float64) for _ in range(3))
    rl = torch.zeros(1, H, dtype=torch.float64)
    for h in range(H):
        s = kd[:, h // G] @ q[0, h, 0].double() * D ** -0.5
        rl[0, h] = torch.logsumexp(s, 0)
        p = torch.softmax(s, 0)
        ro[0, h], size[0, h] = (p @ vd[:, h // G]).cpu(), (p @ vd[:, h // G].abs()).cpu()
        if q4:  # as plain_ops.decode
            sc = scales[:, h // G]
            moves = 1 + int(torch.floor(torch.log2(sc.max() / sc[sc > 0].min()) / 8))
            codes = (vd[:, h // G] / torch.where(sc > 0, sc, torch.ones_like(sc))).abs()
            low[0, h] = (2.0 ** (moves - 21) * (p[:, None] * sc).amax(0) * codes.sum(0)).cpu() + 2.0 ** -11 * size[0, h]
        else:
            low[0, h] = plain_ops.half_step(dtype) ** 2 * size[0, h] + (
                2.0 ** -25 * p.max() * vd[:, h // G].abs().sum(0)).cpu()
    plain_ops.assert_attention_close(o, lse, ro, rl, size, low, dtype)
