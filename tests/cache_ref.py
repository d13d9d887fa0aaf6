"""Plain float64 forms of the 8-bit cache's operators, on the CPU, written from their definitions, and
the caches and error bounds that the tests use."""
import math

import numpy as np
import torch

QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
E4M3, INT8 = torch.float8_e4m3fn, torch.int8


def need_scale(amax, dtype):
    """The least power of two s >= 2^-60 with amax <= qmax * s, by search."""
    s = 2.0 ** -60
    while amax > QMAX[dtype] * s:
        s *= 2.0
    return s


def round_codes(x, dtype):
    """float64 values in units of their scale -> codes (ties to even, saturated; a NaN is e4m3's NaN, int8's 0)."""
    if dtype == INT8:
        return torch.nan_to_num(x.round().clamp(-127, 127), nan=0.0).to(torch.int8)
    a = x.abs().clamp(max=448.0)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    y = torch.round(a / step) * step          # on the e4m3 grid: the conversion below is exact
    y = torch.copysign(y.clamp(max=448.0), x)
    return torch.where(torch.isnan(x), torch.full_like(x, math.nan), y).to(torch.float32).to(E4M3)


def values(codes, scales):
    """float32 values (code * scale rounded once) of pages [P, H, page, D] as float64."""
    return (codes.to(torch.float32) * scales.to(torch.float32)[..., None, None]).double()


def gather(x, table_row, n, page):
    """[n, H, D] values of a sequence from [P, H, page, D]."""
    if n == 0:
        return x.new_zeros((0, x.shape[1], x.shape[3]))
    ids = table_row[: -(-n // page)].long()
    return x[ids].transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:n]


def gather_scale(s, table_row, n, page):
    """[n, H] scales of a sequence's tokens from [P, H]."""
    return s[table_row[: -(-n // page)].long()].double().repeat_interleave(page, 0)[:n]


def attend(q, kv, vv, *, causal=False, window=0, softcap=0.0, sink=None, off_by_one=False, scale=None, hidden=None, vs=None, terms=1):
    """One sequence: q [Sq, Hq, D], kv / vv [n, Hkv, D] float64.  Returns O, LSE [Hq, Sq], weights [Hkv, n], and for the
    error bounds sum p |v| [Sq, Hq, D] and the largest sum |q k| * scale.

    vs: the values' scales [n, Hkv], for the kernel that rounds its probabilities to fp16.  It rounds p_j vs_j / X with X =
    max_j p_j vs_j (the reference that its exponents subtract is that maximum, or a smaller running one), and multiplies
    v_j / vs_j: where the quotient is below 2^-14, fp16 is subnormal and half a step is 2^-25, not 2^-11 of it.  That adds
    at most 2^-25 X sum_j |v_j| / vs_j to an output; it is returned with sum p |v|, in units of 2^-11.
    terms=2 (float queries): p_j vs_j 2^14 / X is held as the sum of two fp16 numbers; the second is off by half its step, so by
    2^-22 of the whole, or, where it is subnormal, by 2^-25, that is 2^-39 X.  In units of 2^-20, which bounds() has at least."""
    Sq, Hq, D = q.shape
    n, Hkv, _ = kv.shape
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    kk, vx = kv.repeat_interleave(G, 1), vv.repeat_interleave(G, 1)
    t = torch.einsum("ihd,jhd->hij", q, kk) * scale
    mag = float((torch.einsum("ihd,jhd->hij", q.abs(), kk.abs()) * abs(scale)).max()) if n and Sq else 0.0
    if softcap:
        t = softcap * torch.tanh(t / softcap)
    pos = torch.arange(Sq)[:, None] + n - Sq
    j = torch.arange(n)[None]
    see = torch.ones((Sq, n), dtype=torch.bool)
    if causal:
        see &= j <= pos
    if window > 0:
        see &= pos - j < window
    if hidden is not None:
        see &= ~hidden[None]
    t = t.masked_fill(~see[None], -math.inf)
    col = torch.full((Hq, Sq, 1), -math.inf, dtype=torch.float64)
    if sink is not None:
        col[:] = sink.double()[:, None, None]
    elif off_by_one:
        col[:] = 0.0
    both = torch.cat([t, col], 2)
    lse = torch.logsumexp(both, 2)
    p = torch.exp(t - torch.where(torch.isinf(lse), 0.0, lse)[..., None])
    p = torch.where(see[None], p, 0.0)
    clean = torch.where(see.any(0)[:, None, None], vx, 0.0)   # an unseen value may be NaN
    o = torch.einsum("hij,jhd->ihd", p, clean)
    pv = torch.einsum("hij,jhd->ihd", p, clean.abs())
    if vs is not None and n:
        sx = vs.repeat_interleave(G, 1)                                                    # [n, Hq]
        X = (p * sx.T[:, None, :]).amax(2)                                                 # [Hq, Sq]
        units = (clean.abs() / sx[..., None].clamp(min=2.0 ** -60)).sum(0)                 # [Hq, D]
        pv = pv + 2.0 ** (-25 + 11 if terms == 1 else -39 + 20) * torch.einsum("hi,hd->ihd", X, units)
    w = p.sum(1).view(Hkv, G, n).sum(1)
    return o, lse, w, pv, mag


def bounds(D, n, mag, softcap, half):
    """What bounds a result's error, from the arithmetic: returns (logit error, relative error of a sum of
    probabilities times values).

    Logits: a float32 dot product of D terms is off by at most D half steps (2^-24 each) of sum |q k|, times a few
    for the scaling and the change to base 2 (4 half steps of the logit, which is at most sum |q k| or the cap), and
    the cap's tanh by some steps of the cap (8).  Tensor cores may truncate where others round: twice the first term.
    Probabilities: exp2 of a logit off by e is off by e (relative), in the sum above and in the one below: 2 e; exp2
    itself and the rescalings are off by some steps each (16); the sums of n float32 terms by n half steps each; a
    probability rounded to fp16 (half=True) by 2^-11, its half step (attend's vs has what subnormal ones add)."""
    e = (2 * D + 4) * 2.0 ** -24 * mag + 8 * 2.0 ** -24 * softcap
    rel = 2 * e + 16 * 2.0 ** -24 + 2 * n * 2.0 ** -24
    if half:
        rel += 2.0 ** -11
    return e, rel


def make_cache(num_pages, H, page, D, dtype, seed=0, std=1.0, spread=0.5):
    """CPU codes and scales of normal values whose spread differs from page to page, k then v."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        x = torch.randn((num_pages, H, page, D), generator=g, dtype=torch.float64) * std
        x *= torch.exp(spread * torch.randn((num_pages, H, 1, 1), generator=g, dtype=torch.float64))
        s = torch.tensor([[need_scale(float(x[p, h].abs().max()), dtype) for h in range(H)] for p in range(num_pages)])
        out += [round_codes(x / s[..., None, None].double(), dtype), s.float()]
    return out[0], out[2], out[1], out[3]  # k, v, k_scale, v_scale


def append(codes, scales, rows, table, lengths, counts, page):
    """Appends rows [B, S, H, D] (float64) in place, one page and head at a time."""
    dtype = codes.dtype
    for b in range(rows.shape[0]):
        n0, n1 = int(lengths[b]), min(int(lengths[b]) + int(counts[b]), table.shape[1] * page)
        for first in range(n0 // page * page, n1, page):
            lo, hi = max(first, n0), min(first + page, n1)
            if lo >= hi:
                continue
            p, old = int(table[b, first // page]), max(0, n0 - first)
            for h in range(rows.shape[2]):
                x = rows[b, lo - n0:hi - n0, h]
                fin = x[torch.isfinite(x)]
                s = need_scale(float(fin.abs().max()) if fin.numel() else 0.0, dtype)
                was = float(scales[p, h])
                if old and was > s:
                    s = was
                if old and s != was:
                    codes[p, h, :old] = round_codes(codes[p, h, :old].to(torch.float64) * (was / s), dtype)
                codes[p, h, lo - first:hi - first] = round_codes(x / s, dtype)
                scales[p, h] = s


def select(w, n, keep, first, recent):
    """Surviving positions of one head."""
    if n <= keep:
        return list(range(n))
    fixed = list(range(first)) + list(range(n - recent, n))
    key = [math.inf if math.isnan(v) else v for v in w[:n].tolist()]
    nan = [math.isnan(v) for v in w[:n].tolist()]
    mid = sorted(range(first, n - recent), key=lambda i: (not nan[i], -key[i], i))
    return sorted(fixed + mid[: keep - first - recent])


def codes_equal(a, b):
    """Equality of code tensors (e4m3 as bytes, +0 and -0 told apart, any NaN equal to any)."""
    a, b = a.cpu(), b.cpu()
    if a.dtype == INT8:
        return torch.equal(a, b)
    x, y = a.view(torch.uint8), b.view(torch.uint8)
    nan = ((x & 127) == 127) & ((y & 127) == 127)
    return bool(((x == y) | nan).all())


def frac(a):
    return np.asarray(a.detach().cpu().double())
