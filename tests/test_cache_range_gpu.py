"""Attention over the 8-bit cache where probabilities and values' scales lie far apart: tokens of small probability that make up
the whole output, and pages whose scales differ by more than float32's exponents.  Against float64."""
import math

import pytest
import torch

import cache_ref as ref
from cache_ref import E4M3, INT8
from test_cache_gpu import BF16, F32, Case, fa

pytestmark = pytest.mark.gpu

# Below this power of two of the row's largest p * scale, a rounded probability loses bits (see attn_cache_gb300.h):
# it is held in fp16 (normal down to 2^-14, steps of 2^-24 below) times 2^14, on tcgen05 times 2^11.
SHIFT = {"mma": 14, "tc": 11}


def check(c, O, LSE, W=None, *, path, sink=False, **kw):
    """Case.check's bounds with what subnormal probabilities add taken at the shift above: half a step, 2^-25, times
    2^-shift of X sum |code|, where X is the largest p * scale.  (float queries: two terms, so 2^-14 of that again is
    below what the relative bound has; FFMA: none.)"""
    kf, vf = ref.values(c.k, c.ks), ref.values(c.v, c.vs)
    half = c.q.dtype == BF16
    store = torch.finfo(c.q.dtype).eps / 2
    for b, n in enumerate(c.lengths):
        kk, vv = ref.gather(kf, c.table[b], n, c.page), ref.gather(vf, c.table[b], n, c.page)
        args = dict(sink=c.sink if sink else None, **kw)
        o, lse, w, pv, mag = ref.attend(c.q[b].double(), kk, vv, **args)
        rounded = half and path != "simt"
        e, rel = ref.bounds(c.D, n, mag, kw.get("softcap", 0.0), rounded)
        floor = 0.0
        if path != "simt":
            vs = ref.gather_scale(c.vs, c.table[b], n, c.page)
            with_vs = ref.attend(c.q[b].double(), kk, vv, vs=vs, **args)[3]     # pv + 2^-14 X sum |code|
            floor = (with_vs - pv) * 2.0 ** 14 * 2.0 ** -(25 + (SHIFT[path] if half else 14))
        lim = store * o.abs() + (1 + store) * (rel * pv + floor) + 2.0 ** -24 * pv + 1e-37
        off = (O[b].cpu().double() - o).abs() - lim
        assert torch.isfinite(O[b].float()).all() and off.max() <= 0, (b, float((off + lim).max()), float(off.max()))
        tol = rel + 4 * 2.0 ** -24 * lse.abs()
        assert ((LSE[b].cpu().double() - lse).abs() <= tol).all(), (b, float((LSE[b].cpu().double() - lse).abs().max()))
        if W is not None:
            rows = c.q.shape[1] * (c.q.shape[2] // c.Hkv)
            want = c.w[b, :, :n].double() + w
            tol = (2 * rel + rows * 2.0 ** -24) * w + 2.0 ** -24 * want + 1e-37
            assert ((W[b, :, :n].cpu().double() - want).abs() <= tol).all(), b


def path_of(c):
    t = c.cuda
    return fa().attn_cache_path_name(t["q"], c.cache, t["table"], t["lengths"])


def put(c, **kw):
    for name, x in kw.items():
        setattr(c, name, x)
        c.cuda[name].copy_(x)


FORMS = [(BF16, 64, 8), (BF16, 128, 8), (BF16, 128, 40), (BF16, 256, 8), (BF16, 128, 160), (BF16, 64, 1040), (F32, 128, 8),
         (BF16, 320, 8)]  # dtype, D, Hq over 2 kv heads


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("dtype,D,Hq", FORMS)
@pytest.mark.parametrize("n,gap", [(700, 15.0), (700, 17.5), (9000, 16.25)])
def test_a_first_token_that_takes_the_weight_and_has_no_value(dtype, D, Hq, kind, n, gap):
    """Every other probability is e^-gap of it, and the output is theirs alone."""
    c = Case([n], Hq=Hq, Hkv=2, D=D, kind=kind, dtype=dtype, spread=0.0)
    k, v, q = c.k.clone(), c.v.clone(), torch.zeros_like(c.q)
    ids = c.table[0, : -(-n // 64)].long()
    k.view(torch.uint8)[ids] = 0
    one = torch.ones(1).to(kind) if kind == E4M3 else torch.tensor([1], dtype=torch.int8)
    k[ids[0], :, 0, 0] = one
    v.view(torch.uint8)[ids[0], :, 0] = 0
    q[..., 0] = gap
    ks = c.ks.clone()
    ks[ids] = 1.0
    put(c, k=k, v=v, q=q, ks=ks)
    c.cache = fa().AttnCache(c.cuda["k"], c.cuda["v"], c.cuda["ks"], c.cuda["vs"])
    path = path_of(c)
    O, LSE = c.run(scale=1.0)
    check(c, O, LSE, path=path, scale=1.0)


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("dtype,D,Hq", FORMS)
def test_a_page_of_a_large_scale_and_no_values(dtype, D, Hq, kind):
    """2^18 times the other pages' scales, but codes of 0 in every second column: there the others' values come through."""
    c = Case([640], Hq=Hq, Hkv=2, D=D, kind=kind, dtype=dtype, spread=0.0)
    v, vs = c.v.clone(), c.vs.clone()
    v.view(torch.uint8)[c.table[0, 3].long(), :, :, ::2] = 0
    vs[c.table[0, 3].long()] = 2.0 ** 18 * vs[c.table[0, 0].long()]
    put(c, v=v, vs=vs)
    check(c, *c.run(), path=path_of(c))


# Scales of ten pages of 64 tokens, and what their keys' scales are multiplied by: equal logits, and logits that make up for
# the values' scales.  2^-60 is what append writes for zeros.
FAR = [([67, -60], [1, 1]), ([-60, 67], [1, 1]), ([100, -60, 0, -60, 90, -3, -60, 100, 20, -45], [1] * 10),
       ([-60, -60, 40, 100, -60, 100, -60, -20, 0, 60], [30, 1, 1, 1, 8, 1, 40, 4, 1, 1])]


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("dtype,D,Hq", FORMS)
@pytest.mark.parametrize("powers,louder", FAR)
@pytest.mark.parametrize("sink", [False, True])
def test_pages_whose_scales_are_further_apart_than_floats_exponents(dtype, D, Hq, kind, powers, louder, sink):
    c = Case([64 * len(powers) - 3], Hq=Hq, Hkv=2, D=D, kind=kind, dtype=dtype, spread=0.0, extra_cols=0)
    ids = c.table[0].long()
    vs, ks = c.vs.clone(), c.ks.clone()
    vs[ids] = torch.tensor([2.0 ** x for x in powers])[:, None]
    ks[ids] *= torch.tensor([float(x) for x in louder])[:, None]
    put(c, vs=vs, ks=ks)
    w = c.cuda["w"]
    O, LSE = c.run(sink=c.cuda["sink"] if sink else None, weights=w)
    check(c, O, LSE, w, path=path_of(c), sink=sink)
    O2, LSE2 = c.run(sink=c.cuda["sink"] if sink else None)
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)


@pytest.mark.parametrize("dtype,D,Hq,Hkv,lengths", [(BF16, 128, 32, 8, [20000, 333]), (BF16, 64, 8, 2, [70000]), (BF16, 256, 8, 2, [9001, 5000]),
                                                    (F32, 128, 8, 2, [30000]), (BF16, 128, 160, 2, [5000, 2000]), (BF16, 320, 8, 2, [9000]),
                                                    (BF16, 64, 520, 1, [20000])])
def test_joined_parts_whose_scales_are_far_apart(dtype, D, Hq, Hkv, lengths):
    """Runs of pages of one scale each, so that the parts that a row is split into differ by it."""
    c = Case(lengths, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, spread=0.0, extra_cols=0)
    vs = c.vs.clone()
    for b, n in enumerate(lengths):
        need = -(-n // 64)
        for x in range(need):
            vs[c.table[b, x].long()] = 2.0 ** (-60, 100, 0, 67, -60)[5 * x // need]
    put(c, vs=vs)
    w = c.cuda["w"]
    O, LSE = c.run(weights=w)
    check(c, O, LSE, w, path=path_of(c))


def test_zeros_next_to_large_values_as_append_writes_them():
    """A page of zero values (scale 2^-60) and one of values around 2^75."""
    m = fa()
    cache = m.AttnCache.empty(2, 64, 1, 64)
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn((1, 128, 1, 64), generator=g) for _ in range(2))
    v[:, :64] = 0.0
    v[:, 64:] *= 2.0 ** 75
    table = torch.tensor([[1, 0]], dtype=torch.int32).cuda()
    n = m.attn_cache_append(cache, k.cuda(), v.cuda(), table, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert float(cache.v_scale[1, 0]) == 2.0 ** -60 and float(cache.v_scale[0, 0]) > 2.0 ** 66
    w = torch.zeros((1, 1, 128), device="cuda")
    for dtype in (BF16, F32):
        w.zero_()
        q = torch.randn((1, 1, 4, 64), generator=g).to(dtype)
        O, LSE = m.attn_cache_fwd(q.cuda(), cache, table, n, weights=w)
        kk, vv = (ref.gather(ref.values(x.cpu(), s.cpu()), table[0].cpu(), 128, 64) for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        o, lse, ww, pv, mag = ref.attend(q[0].double(), kk, vv)
        _, rel = ref.bounds(64, 128, mag, 0.0, dtype == BF16)
        eps = torch.finfo(dtype).eps / 2
        assert ((O[0].cpu().double() - o).abs() <= eps * o.abs() + (1 + eps) * (rel + 2.0 ** -24) * pv).all()
        assert ((LSE[0].cpu().double() - lse).abs() <= rel + 4 * 2.0 ** -24 * lse.abs()).all()
        assert ((w[0].cpu().double() - ww).abs() <= (2 * rel + 2.0 ** -20) * ww).all()
