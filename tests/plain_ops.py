"""Plain 64-bit statements of the window and 4-bit-cache operators (CPU, torch
double, one definition per function, no tiling), and the error bounds that the
tests of their kernels use."""
from __future__ import annotations

import math

import torch

GROUP = 32


def half_step(dtype) -> float:
    """Largest relative error of one rounding to ``dtype``."""
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------ 4-bit cache --

def q4_quantise(x):
    """Rows [..., D] of a 16-bit type -> integers n (int64) [..., D] and scales [..., D/32] (the type of x)."""
    g = x.double().unflatten(-1, (-1, GROUP))
    amax = g.abs().amax(-1)
    fine = torch.isfinite(g).all(-1)
    s = (torch.where(fine, amax, torch.zeros_like(amax)) / 7).to(x.dtype)
    sd = s.double().unsqueeze(-1)
    n = torch.where((sd > 0) & fine.unsqueeze(-1), torch.round(g / torch.where(sd > 0, sd, torch.ones_like(sd))),
                    torch.zeros_like(g))
    s = torch.where(fine, s, torch.full_like(s, math.nan))
    return n.clamp(-7, 7).to(torch.int64).flatten(-2), s


def q4_pack(n):
    """Integers n [..., D] -> code bytes [..., D/2]: column d = 32 w + 4 g + i in nibble i % 2 of byte
    g (D/16) + 2 w + i // 2."""
    D = n.shape[-1]
    out = torch.zeros(n.shape[:-1] + (D // 2,), dtype=torch.int64)
    for d in range(D):
        w, g, i = d // 32, d % 32 // 4, d % 4
        out[..., g * (D // 16) + 2 * w + i // 2] |= (n[..., d] + 8) << (4 * (i % 2))
    return out.to(torch.uint8)


def q4_unpack(codes):
    """Code bytes [..., D/2] -> integers n [..., D]."""
    D = codes.shape[-1] * 2
    c = codes.to(torch.int64)
    cols = []
    for d in range(D):
        w, g, i = d // 32, d % 32 // 4, d % 4
        cols.append(((c[..., g * (D // 16) + 2 * w + i // 2] >> (4 * (i % 2))) & 15) - 8)
    return torch.stack(cols, -1)


def q4_values(codes, scales):
    """What rows of the cache stand for: s * n (double)."""
    return q4_unpack(codes).double() * scales.double().repeat_interleave(GROUP, -1)


# -------------------------------------------------------------- attention --

def visible(nq, nk, window, sinks):
    """[nq, nk] truth values: key j <= query i, and i - j < window (0: no window) or j < sinks."""
    i, j = torch.arange(nq)[:, None], torch.arange(nk)[None, :]
    near = (i - j < window) if window > 0 else torch.ones(nq, nk, dtype=torch.bool)
    return (j <= i) & (near | (j < sinks))


def softmax_attention(q, k, v, seen, scale):
    """One head in double: q [nq,D], k and v [nk,D], seen [nq,nk] -> o, lse, p, and the size of what meets in o
    (sum_j p_j |v_j|). Rows that see nothing: o = 0, lse = -inf."""
    s = (q @ k.t() * scale).masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1) if k.shape[0] else torch.full(q.shape[:1], -math.inf, dtype=torch.float64)
    p = torch.exp(s - lse.masked_fill(torch.isinf(lse), 0.0)[:, None])
    return p @ v, lse, p, p @ v.abs()


def decode(q, values, table, lens, block, window, sinks, scale):
    """q [B,H,1,D]; values(page, head) -> (k, v, s) double [block, D] of one page, s the value's scale (4-bit cache) or
    0; the definition of the paged decode. Returns o [B,H,D], lse [B,H], what meets in o: sum p |v|, and ``low``, what
    the rounding of the weights allows:

    16-bit cache: a weight is the sum of two numbers of its type, off by h^2 relative (h: half a step) and, below
    fp16's normal numbers, 2^-25 of the largest, which is at least 1.

    4-bit cache: p s is rounded to fp16 (2^-11) after a factor r that brings the largest to at least 2^-4, where they
    lose up to 2^-25 each below the normal numbers: 2^-21 max(p s) |n| in o. r follows the running maximum by whole
    powers of two, so the largest may halve with each of its moves by 2^8 or more; after M moves p is under
    2^(8 - 8M), so it is only the largest of p s while s differs by more: M <= 1 + log2(max s / min s) / 8."""
    B, H, _, D = q.shape
    o, size, low = (torch.zeros(B, H, D, dtype=torch.float64) for _ in range(3))
    lse = torch.full((B, H), -math.inf, dtype=torch.float64)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        seen = visible(n, n, window, sinks)[n - 1]
        keys = torch.nonzero(seen).flatten()
        for h in range(H):
            pages = {int(x): values(int(table[b, x]), h) for x in torch.unique(keys // block)}
            k = torch.stack([pages[int(j) // block][0][int(j) % block] for j in keys])
            v = torch.stack([pages[int(j) // block][1][int(j) % block] for j in keys])
            s = torch.stack([pages[int(j) // block][2][int(j) % block] for j in keys])
            r = softmax_attention(q[b, h].double(), k, v, torch.ones(1, len(keys), dtype=torch.bool), scale)
            o[b, h], lse[b, h], size[b, h] = r[0][0], r[1][0], r[3][0]
            if (s > 0).any():
                moves = 1 + math.floor(math.log2(float(s.max() / s[s > 0].min())) / 8)
                n = (v / torch.where(s > 0, s, torch.ones_like(s))).abs()
                low[b, h] = 2.0 ** (moves - 21) * (r[2][0][:, None] * s).amax(0) * n.sum(0) + 2.0 ** -11 * size[b, h]
            else:
                low[b, h] = half_step(q.dtype) ** 2 * size[b, h] + 2.0 ** -25 * v.abs().sum(0)
    return o, lse, size, low


def assert_attention_close(o, lse, ro, rl, size, low, dtype, what=""):
    """O within half a step of its own rounding, ``low`` for its weights (see decode), and 2^-13 of what meets in the
    sum for the rest; LSE within 4e-5 + 2^-21 |LSE|.

    The rest: a score is an fp32 sum of D products, |error| <= 2^-24 * 16 * sum |q k| scale (16: depth of the
    sums), under 2^-24 * 16 * 40 = 2^-14.7 for the inputs here; it enters a weight as a relative error, once in
    the numerator and once in the sum; 2^x and the fp32 sums add a few 2^-22. LSE carries the score's error and
    the rounding of its own value (fp32, two operations)."""
    o, lse = o.double().cpu().reshape(ro.shape), lse.double().cpu().reshape(rl.shape)
    assert torch.equal(torch.isnan(o), torch.isnan(ro)) and torch.equal(torch.isnan(lse), torch.isnan(rl)), what
    h = half_step(dtype)
    tiny = torch.finfo(dtype).smallest_normal * h * 2
    bound = h * ro.abs() * (1 + 2 * h) + 2.0 ** -13 * size + low * (1 + 2 * h) + tiny
    bad = ((o - ro).abs() > bound) & ~torch.isnan(ro)
    assert not bad.any(), (what, "o", float(((o - ro).abs() / bound).nan_to_num().max()), torch.nonzero(bad)[0].tolist())
    empty = torch.isinf(rl)
    assert torch.equal(empty, torch.isinf(lse)) and torch.equal(lse[empty], rl[empty]), what
    off = (lse - rl).abs()[~empty & ~torch.isnan(rl)]
    room = (4e-5 + 2.0 ** -21 * rl.abs())[~empty & ~torch.isnan(rl)]
    assert (off <= room).all(), (what, "lse", float(off.max()))


# ----------------------------------------------------------- window, whole --

def window_attention(q, k, v, window, sinks, scale, dout=None, dtype=torch.bfloat16):
    """One sequence: q [H,Sq,D], k and v [Hkv,Sk,D] -> dict of doubles: o, lse, and with dout [H,Sq,D] also dq, dk,
    dv; each of them but lse with "<name>_bound", the largest error that the kernels' roundings allow.

    Roundings, each by at most h = half a step of the 16-bit type (relative): every output once; P before P V and
    before P^T dO; dS = P (dP - D_i), of the rounded P, before dS^T Q and dS K; O before D_i = dO . O. Beside them P
    carries 2^-13 relative (scores, LSE and 2^x in fp32, as in assert_attention_close), and sums of fp32 products
    2^-18 of what meets in them."""
    H, Sq, D = q.shape
    Hkv, Sk, _ = k.shape
    G, h, e = H // Hkv, half_step(dtype), 2.0 ** -13
    tiny = torch.finfo(dtype).smallest_normal * 2 * h
    q, k, v = q.double(), k.double(), v.double()
    seen = visible(Sq, Sk, window, sinks)
    r = {n: torch.zeros_like(x) for n, x in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
    r.update({n + "_bound": torch.zeros_like(x) for n, x in list(r.items())})
    r["lse"] = torch.zeros(H, Sq, dtype=torch.float64)
    for x in range(H):
        y = x // G
        o, lse, p, size = softmax_attention(q[x], k[y], v[y], seen, scale)
        r["o"][x], r["lse"][x] = o, lse
        o_err = h * o.abs() * (1 + 2 * h) + (h * (1 + h) + e) * size + tiny
        r["o_bound"][x] = o_err
        if dout is None:
            continue
        do = dout[x].double()
        dp, di = do @ v[y].t(), (do * o).sum(-1, keepdim=True)
        ds = p * (dp - di)
        di_err = (do.abs() * o_err).sum(-1, keepdim=True) + 2.0 ** -18 * (do * o).abs().sum(-1, keepdim=True)
        dp_err = 2.0 ** -18 * (do.abs() @ v[y].abs().t())
        # fp16 loses relative precision below its normal numbers: P and dS are off by up to tiny there
        p_err = p * (h + e) * (1 + h) + tiny * seen
        ds_err = (p + p_err) * (di_err + dp_err) + p_err * (dp - di).abs() + h * ds.abs() * (1 + 4 * h) + tiny * seen
        r["dq"][x] = scale * ds @ k[y]
        r["dk"][y] += scale * ds.t() @ q[x]
        r["dv"][y] += p.t() @ do
        r["dq_bound"][x] = scale * (ds_err + 2.0 ** -18 * ds.abs()) @ k[y].abs()
        r["dk_bound"][y] += scale * (ds_err + 2.0 ** -18 * ds.abs()).t() @ q[x].abs()
        r["dv_bound"][y] += (p_err + 2.0 ** -18 * p).t() @ do.abs()
    for n in ("dq", "dk", "dv"):
        r[n + "_bound"] += h * r[n].abs() * (1 + 4 * h) + h * r[n + "_bound"] + tiny
    return r


def assert_window_close(got, ref, what=""):
    """``got``: dict of tensors of one sequence by the names of window_attention."""
    for n, x in got.items():
        x, y = x.double().cpu(), ref[n]
        assert x.shape == y.shape, (what, n, x.shape, y.shape)
        if n == "lse":
            empty = torch.isinf(y)
            assert torch.equal(empty, torch.isinf(x)) and torch.equal(x[empty], y[empty]), (what, n)
            off, room = (x - y).abs()[~empty], (4e-5 + 2.0 ** -21 * y.abs())[~empty]
            assert (off <= room).all(), (what, n, float(off.max()))
            continue
        bad = ~((x - y).abs() <= ref[n + "_bound"])
        assert not bad.any(), (what, n, torch.nonzero(bad)[0].tolist(),
                               float(((x - y).abs() / ref[n + "_bound"]).max()), int(bad.sum()))
