"""The 8-bit key / value cache's operators as a program calls them: appending tokens to a paged cache
with a scale for each page and head, attention over that cache, and eviction by accumulated weight.

``own`` false: the plain torch forms, in 32 bits.  ``own`` true: the framework's entry points.

A cache is ``k`` and ``v`` [pages, Hkv, page, D] in e4m3 or int8 with float32 scales [pages, Hkv]; a
sequence is a row of ``table`` (its pages in order, -1 past the last) and a length.  A value is
code * scale.  A page's scale is the least power of two that holds its largest magnitude (448 steps
of e4m3, 127 of int8), and at least 2^-60.
"""
import math
import random

import torch

own = False

KINDS = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One decoding step's new tokens, a small server: the smallest call, latency alone.
        dict(name="append_token_small", op="append", B=4, S=1, Hkv=8, D=128, page=64, kind="e4m3", dtype="bf16",
             lo=1, hi=4000, ragged=False, weights=False),
        # The same for a large batch, with the accumulated weights that a cache under eviction carries.
        dict(name="append_token_batch", op="append", B=192, S=1, Hkv=8, D=64, page=32, kind="int8", dtype="bf16",
             lo=0, hi=2048, ragged=False, weights=True),
        # Prompts of a ragged batch, padded to the longest, behind what is cached already.
        dict(name="append_prompts", op="append", B=8, S=4096, Hkv=8, D=128, page=64, kind="e4m3", dtype="bf16",
             lo=0, hi=1000, ragged=True, weights=False),
        # A local layer of a softcapped model, one user: the smallest attention, latency alone.
        dict(name="decode_one_local", op="attend", B=1, Sq=1, Hq=16, Hkv=8, D=256, page=64, kind="e4m3", dtype="bf16",
             lo=1531, hi=1531, window=4096, softcap=50.0, sink=False, causal=True, weights=False),
        # A sink layer decoding for a ragged batch of short and middling rows.
        dict(name="decode_batch_sink", op="attend", B=64, Sq=1, Hq=64, Hkv=8, D=64, page=32, kind="int8", dtype="bf16",
             lo=1, hi=4096, window=0, softcap=0.0, sink=True, causal=True, weights=False),
        # Few users with long contexts: one token each against up to 128k cached ones.
        dict(name="decode_long", op="attend", B=4, Sq=1, Hq=32, Hkv=8, D=128, page=64, kind="e4m3", dtype="bf16",
             lo=98001, hi=131072, window=0, softcap=0.0, sink=False, causal=True, weights=False),
        # Decoding with the weights that the eviction goes by.
        dict(name="decode_weights", op="attend", B=16, Sq=1, Hq=32, Hkv=8, D=128, page=128, kind="int8", dtype="bf16",
             lo=777, hi=16384, window=0, softcap=30.0, sink=False, causal=True, weights=True),
        # Checking a few drafted tokens of each user at once.
        dict(name="verify_drafts", op="attend", B=16, Sq=5, Hq=32, Hkv=8, D=128, page=16, kind="e4m3", dtype="bf16",
             lo=5, hi=8192, window=0, softcap=30.0, sink=False, causal=True, weights=False),
        # A chunk of a long prompt against what is cached of it.
        dict(name="prompt_chunk", op="attend", B=1, Sq=512, Hq=32, Hkv=8, D=128, page=64, kind="e4m3", dtype="bf16",
             lo=16111, hi=16111, window=0, softcap=0.0, sink=False, causal=True, weights=False),
        # float32 queries and one shared kv head, as a reference run wants them.
        dict(name="decode_f32_mqa", op="attend", B=9, Sq=1, Hq=8, Hkv=1, D=128, page=64, kind="int8", dtype="f32",
             lo=1, hi=9001, window=0, softcap=50.0, sink=True, causal=True, weights=True),
        # Shrinking a batch's caches to a quarter.
        dict(name="evict_batch", op="evict", B=16, Hkv=8, D=128, page=64, kind="e4m3", lo=1500, hi=8192,
             keep=2048, recent=256, first=4),
        # Shrinking two long contexts.
        dict(name="evict_long", op="evict", B=2, Hkv=8, D=128, page=64, kind="int8", lo=100003, hi=131072,
             keep=16384, recent=1024, first=64),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm, odd ones as often as even ones."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "evict"])
    c = dict(op=op, kind=rng.choice(["e4m3", "int8"]), page=rng.choice([16, 32, 64, 128]), D=rng.choice([64, 128, 256]))
    if op == "append":
        c |= dict(Hkv=rng.choice([1, 2, 4, 8, 16]), dtype=rng.choice(["bf16", "bf16", "f32"]))
        c["S"] = rng.choice([1, 1, _spread(rng, 2, 4096)])
        rows = 8 * 4096 * 8 * 128 // (c["S"] * c["Hkv"] * c["D"])
        c["B"] = _spread(rng, 1, max(1, min(256, rows)))
        c["lo"] = rng.choice([0, 0, 1, 50])
        c["hi"] = c["lo"] + _spread(rng, 1, 2000)
        c |= dict(ragged=c["S"] > 1 and rng.random() < 0.7, weights=rng.random() < 0.4)
        return c
    if op == "evict":
        c |= dict(Hkv=rng.choice([1, 2, 4, 8, 16]), hi=_spread(rng, 64, 131072))
        c["B"] = _spread(rng, 1, max(1, min(64, 2 * 131072 * 8 * 128 // (c["hi"] * c["Hkv"] * c["D"]))))
        c["lo"] = rng.randint(0, c["hi"])
        c["keep"] = max(8, int(c["hi"] * rng.uniform(0.05, 0.4)))
        c["first"] = rng.choice([0, 0, min(4, c["keep"] // 4), c["keep"] // 8])
        c["recent"] = rng.randint(0, c["keep"] // 2)
        return c
    c |= dict(Hkv=rng.choice([1, 2, 4, 8, 16]), dtype=rng.choice(["bf16"] * 5 + ["f32"]))
    c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 8])
    c["Sq"] = rng.choice([1, 1, 1, _spread(rng, 2, 8), _spread(rng, 2, 512)])
    c["hi"] = _spread(rng, 16, 131072 if c["Sq"] == 1 else 32768)
    at_most = min(4 * 131072 * 8 * 128 // (c["hi"] * c["Hkv"] * c["D"]), 512 * 16111 * 32 // (c["hi"] * c["Sq"] * c["Hq"]),
                  512 * 16111 * 32 * 128 // (c["hi"] * c["Sq"] * c["Hq"] * c["D"]))
    if c["dtype"] == "f32":
        at_most //= 16
    while at_most < 1:
        c["hi"] = max(16, c["hi"] // 2)
        at_most = 2 * at_most + 1
    c["B"] = _spread(rng, 1, max(1, min(128, at_most)))
    c["lo"] = rng.choice([0, 1, c["hi"] // 2, c["hi"]])
    c["window"] = rng.choice([0, 0, 0, _spread(rng, 1, 8192)])
    c["softcap"] = rng.choice([0.0, 0.0, 30.0, 50.0])
    c |= dict(sink=rng.random() < 0.4, causal=rng.random() < 0.8, weights=c["Sq"] <= 8 and rng.random() < 0.4)
    return c


def _lengths(case):
    """The sequences' lengths: the longest is ``hi``; the rest lie between ``lo`` and ``hi``."""
    r = random.Random(case["B"] * 1000003 + case["hi"])
    return [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["B"] - 1)]


def _counts(case):
    r = random.Random(case["B"] * 1000003 + case["S"])
    return [case["S"]] + [r.randint(0, case["S"]) if case["ragged"] else case["S"] for _ in range(case["B"] - 1)]


# ---------------------------------------------------------------- what both sides have in hand

def _need(amax, qmax):
    """The least power of two s >= 2^-60 with amax <= qmax * s."""
    m, e = torch.frexp(amax)
    qm, qe = math.frexp(qmax)
    e = torch.where(amax > 0, e - qe + (m > qm), -60).clamp(min=-60)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(x, kind):
    """Values in units of their scale, rounded to nearest even codes."""
    if kind == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _take(t, index):
    """t[index] over the first axis (8-bit types by their bytes)."""
    return t.view(torch.uint8)[index].view(t.dtype) if t.element_size() == 1 else t[index]


def _cache(g, pages, case, std):
    """Codes and scales of ``pages`` pages of normal values whose spread differs from page to page."""
    dtype, qmax = KINDS[case["kind"]]
    shape = (case["Hkv"], case["page"], case["D"])
    codes = torch.empty((pages, *shape), dtype=torch.uint8, device="cuda").view(dtype)
    scales = torch.empty((pages, case["Hkv"]), device="cuda")
    step = max(1, (1 << 26) // (shape[0] * shape[1] * shape[2]))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn((n, *shape), generator=g, device="cuda")
        x *= std * torch.exp(0.5 * torch.randn((n, case["Hkv"], 1, 1), generator=g, device="cuda"))
        s = _need(x.abs().amax((2, 3)), qmax)
        codes[p:p + n].copy_(_codes(x / s[:, :, None, None], case["kind"]))
        scales[p:p + n].copy_(s)
    return codes, scales


def _sequences(g, lengths, room, page, seed):
    """lengths (in the seed's order) and a table of pages in a random order, with room for ``room`` more tokens."""
    order = list(range(len(lengths)))
    random.Random(seed).shuffle(order)
    lengths = [lengths[i] for i in order]
    need = [-(-(n + room) // page) for n in lengths]
    width = max(1, max(need))
    perm = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    at = torch.tensor(need, device="cuda")
    first = at.cumsum(0) - at
    col = torch.arange(width, device="cuda")[None]
    table = torch.where(col < at[:, None], perm[(first[:, None] + col).clamp(max=max(0, sum(need) - 1))], -1)
    return torch.tensor(lengths, dtype=torch.int32, device="cuda"), table.to(torch.int32).contiguous(), sum(need), order


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    st = dict(case=case)
    B, page, D, Hkv = case["B"], case["page"], case["D"], case["Hkv"]
    room = {"append": case.get("S", 0), "attend": 0, "evict": 0}[case["op"]]
    if case["op"] == "append":  # each sequence's row has all the pages that S more tokens can reach
        room += page
    st["lengths"], st["table"], pages, order = _sequences(g, _lengths(case), room, page, seed)
    if case["op"] == "evict":
        wide = -(-case["keep"] // page)
        st["table_out"] = (pages + torch.randperm(B * wide, generator=g, device="cuda")).view(B, wide).to(torch.int32)
        pages += B * wide
    st["k"], st["k_scale"] = _cache(g, max(1, pages), case, 1.0)
    st["v"], st["v_scale"] = _cache(g, max(1, pages), case, 1.0)
    cap = st["table"].shape[1] * page
    if case["op"] == "append":
        dt = TYPES[case["dtype"]]
        # Keys of a larger spread than what is cached: some pages' scales grow.
        st["k_new"] = (torch.randn((B, case["S"], Hkv, D), generator=g, device="cuda") * 1.5).to(dt)
        st["v_new"] = torch.randn((B, case["S"], Hkv, D), generator=g, device="cuda").to(dt)
        counts = _counts(case)
        st["counts"] = torch.tensor([counts[i] for i in order], dtype=torch.int32, device="cuda")
        st["weights"] = torch.rand((B, Hkv, cap), generator=g, device="cuda") if case["weights"] else None
    elif case["op"] == "attend":
        q = torch.randn((B, case["Sq"], case["Hq"], D), generator=g, device="cuda") * 2.0
        st["q"] = q.to(TYPES[case["dtype"]])
        st["sink"] = torch.randn(case["Hq"], generator=g, device="cuda") * 5.0 if case["sink"] else None
        st["weights"] = st["weights_out"] = None
        if case["weights"]:
            st["weights"] = torch.rand((B, Hkv, cap), generator=g, device="cuda")
            st["weights_out"] = st["weights"].clone()
    else:
        # Accumulated weights have a long tail; zeros (tokens nothing looked at) tie.
        w = torch.randn((B, Hkv, cap), generator=g, device="cuda").mul(2.0).exp()
        st["weights"] = torch.where(torch.rand((B, Hkv, cap), generator=g, device="cuda") < 0.1, 0.0, w)
    return st


# ---------------------------------------------------------------- plain forms

def _plain_append(st):
    case, page, B = st["case"], st["case"]["page"], st["case"]["B"]
    S, kind = case["S"], case["kind"]
    qmax = KINDS[kind][1]
    lengths, counts = st["lengths"].long(), st["counts"].long()
    span = (S + page - 2) // page + 1
    slot = (lengths // page)[:, None] + torch.arange(span, device="cuda")            # [B, span]
    pages = st["table"].long().gather(1, slot)
    pos = slot[:, :, None] * page + torch.arange(page, device="cuda")                # [B, span, page]
    old = pos < lengths[:, None, None]
    new = ~old & (pos < (lengths + counts)[:, None, None])
    touched = new.any(2)                                                             # [B, span]
    row = (pos - lengths[:, None, None]).clamp(0, S - 1)
    m = new[:, :, None, :, None]
    for codes, scales, x in ((st["k"], st["k_scale"], st["k_new"]), (st["v"], st["v_scale"], st["v_new"])):
        x = x.float()[torch.arange(B, device="cuda")[:, None, None], row].transpose(2, 3)  # [B, span, Hkv, page, D]
        need = _need(torch.where(m, x.abs(), 0.0).amax((3, 4)), qmax)
        was, held = scales[pages], _take(codes, pages)
        s = torch.where(old.any(2)[:, :, None], torch.maximum(was, need), need)
        again = _codes(held.float() * (was / s)[..., None, None], kind)
        fresh = _codes(x / s[..., None, None], kind)
        o = old[:, :, None, :, None] & (s != was)[..., None, None]
        t = touched[:, :, None, None, None]
        out = torch.where(t & m, fresh.view(torch.uint8), torch.where(t & o, again.view(torch.uint8), held.view(torch.uint8)))
        codes.view(torch.uint8)[pages] = out
        scales[pages] = torch.where(touched[:, :, None], s, was)
    if st["weights"] is not None:
        at = torch.arange(st["weights"].shape[2], device="cuda")[None]
        added = (at >= lengths[:, None]) & (at < (lengths + counts)[:, None])
        st["weights"].masked_fill_(added[:, None, :], 0.0)
    return (lengths + counts).to(torch.int32)


def _plain_attend(st):
    case = st["case"]
    B, Sq, Hq, D = st["q"].shape
    Hkv, page = case["Hkv"], case["page"]
    G = Hq // Hkv
    pages = st["table"].long().clamp(min=0)
    L = pages.shape[1] * page

    def dense(codes, scales):
        x = _take(codes, pages).float() * scales[pages][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, L, D)

    q = st["q"].float().view(B, Sq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Sq, D)
    s = q @ dense(st["k"], st["k_scale"]).transpose(2, 3) * D ** -0.5
    if case["softcap"]:
        s = case["softcap"] * torch.tanh(s / case["softcap"])
    at = st["lengths"].long()[:, None] - Sq + torch.arange(Sq, device="cuda")        # each query's own position
    j = torch.arange(L, device="cuda")
    seen = (j < st["lengths"][:, None])[:, None, :].expand(B, Sq, L)
    if case["causal"]:
        seen = seen & (j <= at[:, :, None])
    if case["window"]:
        seen = seen & (at[:, :, None] - j < case["window"])
    s = s.view(B, Hkv, G, Sq, L).masked_fill_(~seen[:, None, None], -math.inf)
    lse = s.logsumexp(-1)
    if st["sink"] is not None:
        lse = torch.logaddexp(lse, st["sink"].view(Hkv, G)[None, :, :, None])
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    o = p.view(B, Hkv, G * Sq, L) @ dense(st["v"], st["v_scale"])
    o = o.view(B, Hkv, G, Sq, D).permute(0, 3, 1, 2, 4).reshape(B, Sq, Hq, D).to(st["q"].dtype)
    out = {"o": o, "lse": lse.reshape(B, Hq, Sq)}
    if st["weights"] is not None:
        keep = (j < st["lengths"][:, None])[:, None, :]
        out["weights"] = torch.where(keep, st["weights"] + p.sum((2, 3)), st["weights"])
    return out


def _plain_evict(st):
    case = st["case"]
    B, Hkv, page, keep = case["B"], case["Hkv"], case["page"], case["keep"]
    kind, D = case["kind"], case["D"]
    w, lengths = st["weights"], st["lengths"].long()
    cap = w.shape[2]
    j = torch.arange(cap, device="cuda")
    n = lengths[:, None, None]
    rank = torch.where((j < case["first"]) | (j >= n - case["recent"]), math.inf, w)
    rank = torch.where(j < n, rank, -math.inf)
    picked = torch.sort(rank, dim=2, descending=True, stable=True)[1][:, :, :keep]
    picked = torch.nn.functional.pad(picked, (0, keep - picked.shape[2]), value=cap)
    kept_n = lengths.clamp(max=keep)
    alive = torch.arange(keep, device="cuda") < kept_n[:, None]                      # [B, keep]
    picked = torch.sort(torch.where(alive[:, None, :], picked, cap), dim=2)[0]
    kept = torch.where(alive[:, None, :], picked, -1).to(torch.int32)
    src = picked.clamp(max=cap - 1)
    src_page = st["table"].long().clamp(min=0)[torch.arange(B, device="cuda")[:, None, None], src // page]
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    wide = st["table_out"].shape[1]
    out_pages = st["table_out"].long()                                               # [B, wide]
    pad = wide * page - keep
    live = torch.nn.functional.pad(alive, (0, pad)).view(B, wide, 1, page, 1)
    used = live.any(3, keepdim=True)
    for codes, scales in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
        x = codes.view(torch.uint8)[src_page, head, src % page].view(codes.dtype).float() * scales[src_page, head][..., None]
        x = torch.nn.functional.pad(x, (0, 0, 0, pad)).view(B, Hkv, wide, page, D).transpose(1, 2)
        s = _need(torch.where(live, x.abs(), 0.0).amax((3, 4)), KINDS[kind][1])
        fresh = _codes(x / s[..., None, None], kind).view(torch.uint8)
        codes.view(torch.uint8)[out_pages] = torch.where(live, fresh, _take(codes, out_pages).view(torch.uint8))
        scales[out_pages] = torch.where(used[:, :, :, 0, 0], s, scales[out_pages])
    weights = torch.where(alive[:, None, :], w.gather(2, src), 0.0)
    return kept, kept_n.to(torch.int32), weights


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if own:
        import attention_flash_attn_gb300 as fa
        if "handle" not in state:  # the program's handle of its cache, made once
            state["handle"] = fa.AttnCache(state["k"], state["v"], state["k_scale"], state["v_scale"])
        cache = state["handle"]
        if case["op"] == "append":
            lengths = fa.attn_cache_append(cache, state["k_new"], state["v_new"], state["table"], state["lengths"],
                                           counts=state["counts"], weights=state["weights"])
        elif case["op"] == "attend":
            o, lse = fa.attn_cache_fwd(state["q"], cache, state["table"], state["lengths"], causal=case["causal"],
                                       window=case["window"], softcap=case["softcap"], sink=state["sink"],
                                       weights=state["weights"], weights_out=state["weights_out"])
            out = {"o": o, "lse": lse}
            if state["weights"] is not None:
                out["weights"] = state["weights_out"]
            return out
        else:
            kept, lengths, weights = fa.attn_cache_evict(cache, state["table"], state["lengths"], state["weights"],
                                                         state["table_out"], keep=case["keep"], recent=case["recent"],
                                                         first=case["first"])
    elif case["op"] == "append":
        lengths = _plain_append(state)
    elif case["op"] == "attend":
        return _plain_attend(state)
    else:
        kept, lengths, weights = _plain_evict(state)
    # The cache itself is an output: e4m3 values (int8: whole numbers) in units of their scales.
    out = {"k": state["k"], "v": state["v"], "k_scale": state["k_scale"], "v_scale": state["v_scale"], "lengths": lengths}
    if case["op"] == "append":
        if state["weights"] is not None:
            out["weights"] = state["weights"]
    else:
        out |= {"kept": kept, "weights": weights}
    return out


def work(case):
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    lengths = _lengths(case)
    if case["op"] == "append":
        counts = _counts(case)
        rows = sum(counts)
        each = {"bf16": 2, "f32": 4}[case["dtype"]] + 1
        pages = sum(-(-(n % page + c) // page) for n, c in zip(lengths, counts) if c)
        return {"bytes": 2 * rows * Hkv * D * each + pages * Hkv * 2 * 4 + (4 * rows * Hkv if case["weights"] else 0), "flops": 0}
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lengths)
        return {"bytes": 4 * Hkv * sum(lengths) + kept * Hkv * (4 * D + 12), "flops": 0}
    Sq, Hq, size = case["Sq"], case["Hq"], {"bf16": 2, "f32": 4}[case["dtype"]]
    pairs = keys = 0
    for n in lengths:
        lo = 0 if not case["window"] else max(0, n - Sq - case["window"] + 1)
        keys += n - lo
        for i in range(Sq):
            at = n - Sq + i
            last = min(n, at + 1) if case["causal"] else n
            pairs += max(0, last - (0 if not case["window"] else max(0, at - case["window"] + 1)))
    b = keys * Hkv * (2 * D + 8 / page) + 2 * case["B"] * Sq * Hq * D * size + 4 * case["B"] * Sq * Hq
    if case["weights"]:
        b += 8 * Hkv * sum(lengths)
    return {"bytes": b, "flops": 4 * pairs * Hq * D}


# ---------------------------------------------------------------- from the definition, in 64 bits

def _grid(x, kind):
    """The nearest representable code value of each element (ties to even), in float64."""
    if kind == "int8":
        return torch.round(x).clamp(-127, 127)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.exp2(e - 3)  # three bits behind the leading one; below 2^-6 the step stays
    return (torch.round(x / step) * step).clamp(-448, 448)


def _scale_of(amax, kind):
    """The least 2^e >= 2^-60 with amax <= qmax * 2^e, found by trying the exponents around the logarithm."""
    q = KINDS[kind][1]
    e = math.floor(math.log2(amax / q)) - 1 if amax > 0 else -60
    while e < -60 or amax > q * 2.0 ** e:
        e += 1
    return 2.0 ** e


def exact(case, seed):
    st = prepare(case, seed)
    kind, page, B, Hkv = case["kind"], case["page"], case["B"], case["Hkv"]
    lengths, table = st["lengths"].tolist(), st["table"].tolist()
    whole = lambda t: t if kind == "int8" else t.double()  # noqa: E731
    if case["op"] == "attend":
        return _exact_attend(case, st, lengths, table)
    if case["op"] == "append":
        if B * (case["S"] // page + 2) * Hkv > 30000:
            return None
        counts = st["counts"].tolist()
        for codes, scales, x in (("k", "k_scale", "k_new"), ("v", "v_scale", "v_new")):
            x = st[x].double()
            c, s = st[codes].double(), st[scales].double()
            for b in range(B):
                if not counts[b]:
                    continue
                end = lengths[b] + counts[b]
                for first in range(lengths[b] // page * page, end, page):
                    p = table[b][first // page]
                    o = max(0, lengths[b] - first)
                    last = min(end, first + page)
                    rows = x[b, first + o - lengths[b]:last - lengths[b]].transpose(0, 1)  # [Hkv, n, D]
                    big = rows.abs().amax((1, 2)).tolist()
                    for h in range(Hkv):
                        need = _scale_of(big[h], kind)
                        was = float(s[p, h])
                        now = max(was, need) if o else need
                        if o and now != was:
                            c[p, h, :o] = _grid(c[p, h, :o] * (was / now), kind)
                        s[p, h] = now
                        c[p, h, o:o + rows.shape[1]] = _grid(rows[h] / now, kind)
            st[codes], st[scales] = c.to(torch.int8) if kind == "int8" else c, s
        out = {"k": st["k"], "v": st["v"], "k_scale": st["k_scale"], "v_scale": st["v_scale"],
               "lengths": torch.tensor([n + c for n, c in zip(lengths, counts)], dtype=torch.int32)}
        if st["weights"] is not None:
            w = st["weights"].double()
            for b in range(B):
                w[b, :, lengths[b]:lengths[b] + counts[b]] = 0
            out["weights"] = w
        return out
    if Hkv * sum(-(-min(n, case["keep"]) // page) for n in lengths) > 30000:
        return None
    keep = case["keep"]
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32)
    weights = torch.zeros((B, Hkv, keep), dtype=torch.float64)
    w = st["weights"].cpu()
    codes = {x: st[x].double() for x in ("k", "v")}
    scales = {x: st[x + "_scale"].double() for x in ("k", "v")}
    out_table = st["table_out"].tolist()
    for b in range(B):
        n = lengths[b]
        row = torch.tensor(table[b], device="cuda")
        for h in range(Hkv):
            if n <= keep:
                pick = list(range(n))
            else:
                fixed = set(range(min(case["first"], n))) | set(range(max(0, n - case["recent"]), n))
                vals = w[b, h, :n].tolist()
                free = sorted((i for i in range(n) if i not in fixed), key=lambda i: (-vals[i], i))
                pick = sorted(list(fixed) + free[:keep - len(fixed)])
            at = torch.tensor(pick, dtype=torch.long)
            kept[b, h, :len(pick)] = at.to(torch.int32)
            weights[b, h, :len(pick)] = w[b, h, at].double()
            at = at.cuda()
            for x in ("k", "v"):
                val = codes[x][row[at // page], h, at % page] * scales[x][row[at // page], h][:, None]
                for i in range(0, len(pick), page):
                    blk = val[i:i + page]
                    s = _scale_of(float(blk.abs().max()), kind)
                    p = out_table[b][i // page]
                    codes[x][p, h, :blk.shape[0]] = _grid(blk / s, kind)
                    scales[x][p, h] = s
    return {"k": whole(codes["k"].to(torch.int8) if kind == "int8" else codes["k"]),
            "v": whole(codes["v"].to(torch.int8) if kind == "int8" else codes["v"]),
            "k_scale": scales["k"], "v_scale": scales["v"],
            "lengths": torch.tensor([min(n, keep) for n in lengths], dtype=torch.int32), "kept": kept, "weights": weights}


def _exact_attend(case, st, lengths, table):
    """Sequence by sequence and kv head by kv head, in float64."""
    B, Sq, Hq, D = st["q"].shape
    Hkv, page = case["Hkv"], case["page"]
    G = Hq // Hkv
    o = torch.zeros((B, Sq, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device="cuda")
    weights = st["weights"].double() if st["weights"] is not None else None
    for b in range(B):
        n = lengths[b]
        pages = torch.tensor(table[b][:-(-n // page)], dtype=torch.long, device="cuda")
        qi = torch.arange(Sq, device="cuda")[:, None] + n - Sq
        kj = torch.arange(n, device="cuda")[None]
        hidden = torch.zeros((Sq, n), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= kj > qi
        if case["window"]:
            hidden |= kj <= qi - case["window"]
        for h in range(Hkv):
            kk = (st["k"].view(torch.uint8)[pages, h].view(st["k"].dtype).double() * st["k_scale"][pages, h].double()[:, None, None]).reshape(-1, D)[:n]
            vv = (st["v"].view(torch.uint8)[pages, h].view(st["v"].dtype).double() * st["v_scale"][pages, h].double()[:, None, None]).reshape(-1, D)[:n]
            for r in range(h * G, (h + 1) * G):
                t = st["q"][b, :, r].double() @ kk.T / math.sqrt(D)
                if case["softcap"]:
                    t = torch.tanh(t / case["softcap"]) * case["softcap"]
                t[hidden] = -math.inf
                extra = float(st["sink"][r]) if st["sink"] is not None else -math.inf
                top = torch.cat([t, torch.full((Sq, 1), extra, dtype=torch.float64, device="cuda")], 1).amax(1, keepdim=True)
                top = torch.where(top == -math.inf, 0.0, top)
                e = torch.exp(t - top)
                z = e.sum(1, keepdim=True) + torch.exp(extra - top)
                p = torch.where(z > 0, e / z, 0.0)
                lse[b, r] = (top + torch.log(z))[:, 0]
                o[b, :, r] = p @ vv
                if weights is not None:
                    weights[b, h, :n] += p.sum(0)
    out = {"o": o, "lse": lse}
    if weights is not None:
        out["weights"] = weights
    return out
