"""Kernels that are launched before the one ahead of them in the stream has ended
(rotary positions, the paged cache's attention, weights and eviction): each reads
what its predecessor wrote, overwrites what that one read, and can be captured
behind any kind of work, from streams that fork and join."""
import pytest
import torch

import exact_attention_54_gb300 as fa

pytestmark = pytest.mark.gpu

B, H, HKV, D, BS, BLOCKS = 3, 8, 2, 64, 16, 24
LENS, NEW = (300, 17, 129), 5
KEEP = 40


def state(seed):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    s = {"x": rand(B * NEW, H, D), "k": rand(B * NEW, HKV, D), "v": rand(B * NEW, HKV, D),
         "kc": rand(4 * B * BLOCKS, HKV, BS, D), "vc": rand(4 * B * BLOCKS, HKV, BS, D)}
    s["f"] = fa.rope_frequencies(D)[0]
    perm = torch.randperm(4 * B * BLOCKS, generator=g).int()
    s["table"], s["to"] = perm[:B * BLOCKS].view(B, BLOCKS).cuda(), perm[B * BLOCKS:2 * B * BLOCKS].view(B, BLOCKS).cuda()
    s["cu"] = (torch.arange(B + 1) * NEW).int().cuda()
    s["starts"] = torch.tensor(LENS, dtype=torch.int32).cuda()
    s["lens"] = s["starts"] + NEW
    return s


def step(s, between):
    """A step of calls, each of which needs the one before; ``between`` runs between any two of them."""
    fa.fa_rope(s["x"], s["x"], s["f"])                      # in place, twice
    between()
    fa.fa_rope(s["x"], s["x"], s["f"], inverse=True)
    between()
    q = fa.flash_rope_kv_write(s["x"], s["k"], s["v"], s["kc"], s["vc"], s["table"], s["cu"], NEW, s["f"], s["starts"])
    between()
    o, lse = fa.flash_attention_paged(q, s["kc"], s["vc"], s["table"], s["cu"], s["lens"], NEW)
    between()
    w = fa.flash_kv_weights(q, lse, s["kc"], s["table"], s["cu"], s["lens"], NEW)
    between()
    kept, lens, w2 = fa.flash_kv_evict(s["kc"], s["vc"], w, s["table"], s["lens"], s["to"], KEEP, 1, 8)
    between()
    o2, _ = fa.flash_attention_paged(o, s["kc"], s["vc"], s["to"], s["cu"], lens, NEW)
    between()
    s["x"].copy_(o2)                                        # read and overwritten by the next step
    return q, o, lse, w, kept, lens, w2, o2


def same(a, b):
    for n, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), n


def test_chains_without_a_wait():
    apart = state(1)
    expect = [step(apart, torch.cuda.synchronize) for _ in range(4)]
    for _ in range(20):  # (the same again and again: a race need not show at once)
        s = state(1)
        torch.cuda.synchronize()
        got = [step(s, lambda: None) for _ in range(4)]
        for a, b in zip(got, expect):
            same(a, b)
    fa.fa_check_device_error()


def test_large_calls_behind_one_another():
    """Rows of many waves, each call's output the next one's input, and its input the next one's output."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(20000, 8, 128, generator=g).to(torch.float16).cuda()
    f = fa.rope_frequencies(128)[0]

    def run(between):
        a, b = x.clone(), torch.empty_like(x)
        for n in range(6):
            fa.fa_rope(a, b, f, inverse=n % 2 == 1)
            between()
            a, b = b, a
        return a

    assert torch.equal(run(lambda: None), run(torch.cuda.synchronize))


def test_captured_with_streams_that_fork_and_join():
    apart = state(3)
    expect = step(apart, torch.cuda.synchronize)
    s = state(3)
    side, main = torch.cuda.Stream(), torch.cuda.Stream()
    start = {k: v.clone() for k, v in s.items()}
    step(s, lambda: None)  # (attributes of the kernels are set outside the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    extra = []
    with torch.cuda.graph(graph, stream=main):
        for k in ("x", "kc", "vc"):
            s[k].copy_(start[k])                            # behind copies
        flag = torch.zeros(16, device="cuda")               # and a fill
        side.wait_stream(main)
        with torch.cuda.stream(side):                       # a call that only waits for another stream's work
            extra.append(fa.flash_rope(start["x"], s["f"]))
        main.wait_stream(side)                              # one behind two streams
        extra.append(fa.flash_rope(extra[0], s["f"]))
        side.wait_stream(main)
        with torch.cuda.stream(side):
            out = step(s, lambda: None)
        main.wait_stream(side)
        extra.append(fa.flash_rope_bwd(extra[1], s["f"]))
        flag += 1
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        same(out, expect)
        one = fa.flash_rope(start["x"], s["f"])
        torch.cuda.synchronize()
        two = fa.flash_rope(one, s["f"])
        torch.cuda.synchronize()
        same(extra, [one, two, fa.flash_rope_bwd(two, s["f"])])
        assert bool((flag == 1).all())
    fa.fa_check_device_error()
