"""Evictions whose weights go on: into rows of the new table's width, and from there into appends, attention and the next eviction."""
import pytest
import torch

import cache_ref as ref
from cache_ref import E4M3, INT8
from test_cache_gpu import BF16, Case, fa, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("keep,page", [(100, 32), (64, 64), (1, 16)])
def test_weights_out_of_any_width(kind, keep, page):
    """The same weights as the dense form's; behind them, and between the rows, nothing is written."""
    m = fa()
    c = Case([700, 0, 1, keep, keep + 1, 499], Hq=4, Hkv=2, D=64, page=page, kind=kind)
    wide = -(-keep // page)
    P, B = c.k.shape[0], 6
    out = (P + torch.arange(B * wide)).view(B, wide).int().cuda()
    grow = lambda t: torch.cat([t, torch.zeros((B * wide, *t.shape[1:]), dtype=t.dtype)])  # noqa: E731
    cache = m.AttnCache(*(grow(t.view(torch.uint8)).view(kind).cuda() for t in (c.k, c.v)), grow(c.ks).cuda(), grow(c.vs).cuda())
    go = lambda **kw: m.attn_cache_evict(cache, c.cuda["table"], c.cuda["lengths"], c.cuda["w"], out, keep=keep, recent=min(17, keep), **kw)  # noqa: E731
    kept, n, dense = go()
    big = torch.full((B, 4, keep + 70), 7.0, device="cuda")
    for view in (big[:, 1:3, 3:], big[:, ::2, : keep], big.transpose(0, 1)[:2].transpose(0, 1)):
        big.fill_(7.0)
        kept2, n2, got = go(weights_out=view)
        assert got is view and torch.equal(kept2, kept) and torch.equal(n2, n) and torch.equal(view[..., :keep], dense)
        assert (view[..., keep:] == 7.0).all() and (big == 7.0).sum() >= big.numel() - B * 2 * keep
    one = c.cuda["w"][:1, :, : keep].contiguous()
    assert torch.equal(m.attn_cache_evict(cache, c.cuda["table"][:1], i32(700).cuda(), c.cuda["w"][:1], out[:1], keep=keep, recent=min(17, keep),
                                          weights_out=one)[2], dense[:1])
    assert m.attn_cache_check_device_status(cache) == 0


def test_weights_out_that_overlaps_weights_is_refused():
    m = fa()
    c = Case([100], Hq=2, Hkv=2, D=32, page=16)
    w = torch.zeros((1, 2, 2 * c.w.shape[2]), device="cuda")
    out = i32(0, 1).cuda()[None]
    for x, y in ((w, w), (w[:, :, : c.w.shape[2]], w[:, :, c.w.shape[2]:])):  # (rows of one between those of the other: not told apart)
        with pytest.raises(m.AttnError):
            m.attn_cache_evict(c.cache, c.cuda["table"], c.cuda["lengths"], x, out, keep=32, weights_out=y)


def test_a_sequence_goes_on_with_its_evicted_weights():
    """Evict, append, attend with weights, evict again, with no copy between: lengths and weights as float64 has them."""
    m = fa()
    g = torch.Generator().manual_seed(5)
    B, H, G, D, page, keep = 2, 2, 4, 64, 32, 50
    cache = m.AttnCache.empty(40, page, H, D)
    new = lambda S: [torch.randn((B, S, H, D), generator=g).bfloat16().cuda() for _ in range(2)]  # noqa: E731
    tables = [torch.arange(x, x + 2 * B, dtype=torch.int32).view(B, 2).cuda() for x in (8, 12)]
    table = torch.arange(0, 8, dtype=torch.int32).view(B, 4).cuda()
    w = torch.zeros((B, H, 4 * page), device="cuda")
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    n = m.attn_cache_append(cache, *new(100), table, n, counts=i32(100, 60).cuda(), weights=w)

    def attend():
        q = torch.randn((B, 1, H * G, D), generator=g).bfloat16()
        before = w.cpu().double()
        m.attn_cache_fwd(q.cuda(), cache, table, n, weights=w)
        for b in range(B):
            L = int(n[b])
            kk, vv = (ref.gather(ref.values(x.cpu(), s.cpu()), table[b].cpu(), L, page) for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
            _, _, ww, _, mag = ref.attend(q[b].double(), kk, vv)
            _, rel = ref.bounds(D, L, mag, 0.0, True)
            want = before[b, :, :L] + ww
            assert ((w[b, :, :L].cpu().double() - want).abs() <= (2 * rel + 2.0 ** -20) * ww + 2.0 ** -24 * want).all()

    attend()
    for to in tables:
        room = torch.full((B, H, 2 * page), 99.0, device="cuda")
        _, n, w = m.attn_cache_evict(cache, table, n, w, to, keep=keep, recent=8, first=2, weights_out=room)
        table = to
        assert w is room and n.tolist() == [keep, keep]
        for _ in range(3):
            n = m.attn_cache_append(cache, *new(1), table, n, weights=w)
            attend()
    assert n.tolist() == [53, 53] and m.attn_cache_check_device_status(cache) == 0
