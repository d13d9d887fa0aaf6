"""The 8-bit paged cache on the GPU against plain float64 forms: attention over the cache (all masks, head layouts, types, odd
lengths, NaN where nothing may look), appending, eviction, and the three together as a serving loop uses them."""
import math

import pytest
import torch

import cache_ref as ref
from cache_ref import E4M3, INT8

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def fa():
    import attention_flash_attn_gb300 as m
    return m


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


class Case:
    """A cache of random pages, sequences over them in random order, and queries.  Everything that no
    sequence may look at is NaN (int8: -128): slots past the last token, pages of nobody, their scales."""

    def __init__(self, lengths, *, Sq=1, Hq=8, Hkv=2, D=128, page=64, kind=E4M3, dtype=BF16, seed=0, q_std=2.0, spread=0.5,
                 extra_cols=1):
        g = torch.Generator().manual_seed(seed + 99)
        self.lengths, self.page, self.kind, self.D, self.Hkv = lengths, page, kind, D, Hkv
        B = len(lengths)
        need = [-(-n // page) for n in lengths]
        P = sum(need) + 3
        self.k, self.v, self.ks, self.vs = ref.make_cache(P, Hkv, page, D, kind, seed, spread=spread)
        perm = torch.randperm(P, generator=g)
        self.table = torch.full((B, max(need) + extra_cols), 2 ** 30, dtype=torch.int32)
        at, used = 0, torch.zeros((P, page), dtype=torch.bool)
        for b, n in enumerate(lengths):
            ids = perm[at:at + need[b]]
            self.table[b, :need[b]] = ids.int()
            at += need[b]
            for x, p in enumerate(ids.tolist()):
                used[p, :min(page, n - x * page)] = True
        bad = 127 if kind == E4M3 else 128
        for c, s in ((self.k, self.ks), (self.v, self.vs)):
            c.view(torch.uint8)[~used[:, None, :, None].expand(c.shape)] = bad
            s[~used.any(1)] = math.nan
        self.q = (torch.randn((B, Sq, Hq, D), generator=g) * q_std).to(dtype)
        self.sink = torch.randn(Hq, generator=g) * 3
        self.w = torch.rand((B, Hkv, self.table.shape[1] * page), generator=g)
        self.cuda = {n: getattr(self, n).cuda() for n in ("k", "v", "ks", "vs", "table", "q", "sink", "w")}
        self.cuda["lengths"] = i32(*lengths).cuda()
        self.cache = fa().AttnCache(self.cuda["k"], self.cuda["v"], self.cuda["ks"], self.cuda["vs"])

    def run(self, q=None, **kw):
        t = self.cuda
        return fa().attn_cache_fwd(t["q"] if q is None else q, self.cache, t["table"], t["lengths"], **kw)

    def check(self, O, LSE, W=None, *, sink=False, hidden=None, rows=None, **kw):
        """Against float64, element by element, within the bounds that the arithmetic gives."""
        kf, vf = ref.values(self.k, self.ks), ref.values(self.v, self.vs)
        O, LSE = O.cpu(), LSE.cpu()
        half = self.q.dtype == BF16
        for b in (range(len(self.lengths)) if rows is None else rows):
            n = self.lengths[b]
            kk, vv = ref.gather(kf, self.table[b], n, self.page), ref.gather(vf, self.table[b], n, self.page)
            hid = None if hidden is None else hidden[b]
            if hid is not None:
                kk, vv = torch.where(hid[:, None, None], 0.0, kk), torch.where(hid[:, None, None], 0.0, vv)
            vs = ref.gather_scale(self.vs, self.table[b], n, self.page) if self.D <= 256 or half else None
            o, lse, w, pv, mag = ref.attend(self.q[b].double(), kk, vv, sink=self.sink if sink else None, hidden=hid, vs=vs,
                                            terms=1 if half else 2, **kw)
            e, rel = ref.bounds(self.D, n, mag, kw.get("softcap", 0.0), half)
            store = torch.finfo(self.q.dtype).eps / 2
            lim = store * o.abs() + (1 + store) * rel * pv + 2.0 ** -24 * pv + 1e-37
            assert torch.isfinite(O[b].float()).all()
            off = (O[b].double() - o).abs() - lim
            assert off.max() <= 0, (b, n, float(off.max()))
            fin = torch.isfinite(lse)
            assert torch.equal(torch.isfinite(LSE[b]), fin) and not torch.isnan(LSE[b]).any()
            tol = rel + 4 * 2.0 ** -24 * lse[fin].abs()
            assert ((LSE[b].double()[fin] - lse[fin]).abs() <= tol).all(), (b, n)
            assert (LSE[b][~fin] == -math.inf).all()
            if W is not None:
                rows_ = self.q.shape[1] * (self.q.shape[2] // self.Hkv)
                want = self.w[b, :, :n].double() + w
                tol = (2 * rel + rows_ * 2.0 ** -24) * w + 2.0 ** -24 * want + 1e-37
                assert ((W[b, :, :n].cpu().double() - want).abs() <= tol).all(), (b, n)


ODD = [1, 777, 0, 64, 65, 31, 130]


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("dtype,D,page", [(BF16, 64, 16), (BF16, 128, 64), (BF16, 256, 32), (F32, 128, 128), (F32, 80, 32), (BF16, 96, 64),
                                          (F32, 512, 16), (F32, 16, 64), (BF16, 320, 32)])
def test_single_tokens(dtype, D, page, kind):
    c = Case(ODD, D=D, page=page, kind=kind, dtype=dtype, seed=D + page)
    c.check(*c.run())
    path = fa().attn_cache_path_name(c.cuda["q"], c.cache, c.cuda["table"], c.cuda["lengths"])
    assert path == ("mma" if D <= 256 else "simt")


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("dtype,D,page,G,Sq", [(BF16, 16, 16, 4, 1), (BF16, 32, 128, 4, 6), (BF16, 48, 32, 5, 1), (BF16, 80, 64, 4, 1),
                                               (BF16, 96, 16, 8, 5), (BF16, 112, 128, 3, 40), (BF16, 144, 16, 4, 1),
                                               (BF16, 160, 64, 2, 9), (BF16, 192, 128, 8, 1), (BF16, 240, 32, 1, 1),
                                               (F32, 48, 64, 4, 1), (F32, 96, 32, 8, 3), (F32, 208, 16, 4, 1)])
def test_head_dims_between_those_compiled(dtype, D, page, G, Sq, kind):
    """One cluster to an item, and (the second case) a split over the grid with the join."""
    for lengths, Hkv in ((ODD, 2), ([9001, 5] + [3000] * 30, 6)):
        c = Case(lengths, Sq=Sq, Hq=G * Hkv, Hkv=Hkv, D=D, page=page, kind=kind, dtype=dtype, seed=D + page)
        w = c.cuda["w"].clone()
        out = c.run(sink=c.cuda["sink"], window=700, softcap=15.0, weights=w)
        c.check(out[0], out[1], w, rows=[0, 1, 4], sink=True, window=700, softcap=15.0)
        c.check(*c.run(), rows=[0, 2])


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (5, 5), (16, 2), (20, 2), (32, 1), (40, 1), (64, 8), (96, 3)])
@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 128)])
def test_head_layouts(Hq, Hkv, dtype, D):
    c = Case([300, 17], Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, seed=Hq)
    c.check(*c.run(softcap=20.0, sink=c.cuda["sink"]), sink=True, softcap=20.0)


MASKS = [dict(), dict(causal=True), dict(causal=True, window=1), dict(causal=True, window=33), dict(window=100),
         dict(causal=True, softcap=15.0), dict(causal=True, off_by_one=True), dict(causal=True, window=64, softcap=50.0, scale=0.3)]


@pytest.mark.parametrize("kw", MASKS, ids=lambda k: "-".join(f"{a}{b}" for a, b in k.items()) or "all")
@pytest.mark.parametrize("dtype,D,kind,page", [(BF16, 64, INT8, 32), (BF16, 128, E4M3, 16), (BF16, 256, E4M3, 64), (F32, 48, E4M3, 32), (F32, 256, INT8, 16),
                                               (F32, 64, E4M3, 64)])
@pytest.mark.parametrize("Sq", [1, 2, 7, 50])
def test_masks(kw, dtype, D, kind, page, Sq):
    """Sequences shorter than Sq among them: causal rows that see nothing."""
    c = Case([200, 3, 0, 129], Sq=Sq, Hq=6, Hkv=2, D=D, kind=kind, page=page, dtype=dtype, seed=Sq)
    O, LSE = c.run(**kw)
    c.check(O, LSE, **kw)
    if Sq == 50 and kw.get("causal") and not kw.get("off_by_one"):
        assert (O[1, :47] == 0).all() and (LSE[1, :, :47] == -math.inf).all()


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_a_sink_takes_rows_that_see_nothing(dtype, D, kind):
    c = Case([0, 2, 90], Sq=4, D=D, kind=kind, dtype=dtype)
    O, LSE = c.run(causal=True, sink=c.cuda["sink"])
    c.check(O, LSE, sink=True, causal=True)
    assert (O[0] == 0).all()
    assert torch.allclose(LSE[0], c.cuda["sink"][:, None].expand(8, 4), rtol=2.0 ** -22)
    none = torch.full_like(c.cuda["sink"], -math.inf)  # a sink of nothing is no sink
    O1, LSE1 = c.run(causal=True, sink=none)
    c.check(O1, LSE1, causal=True)


@pytest.mark.parametrize("lengths,Hq,Hkv,D,kind,page", [([20011, 5], 8, 1, 128, E4M3, 64), ([70001], 4, 2, 64, INT8, 128),
                                                        ([9000, 1, 4097, 0, 333], 16, 8, 256, E4M3, 16)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_long_rows_are_split_and_joined(lengths, Hq, Hkv, D, kind, page, dtype):
    c = Case(lengths, Hq=Hq, Hkv=Hkv, D=D, kind=kind, page=page, dtype=dtype)
    O, LSE = c.run(causal=True, sink=c.cuda["sink"])
    c.check(O, LSE, sink=True, causal=True)
    O2, LSE2 = c.run(causal=True, sink=c.cuda["sink"])
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)  # the split goes by the lengths alone


@pytest.mark.parametrize("kind,D,page", [(E4M3, 128, 64), (INT8, 128, 16), (E4M3, 64, 32), (INT8, 64, 128), (E4M3, 128, 128)])
@pytest.mark.parametrize("lengths,Sq,G,Hkv,kw", [([700, 0, 64, 129, 257], 33, 2, 2, dict(causal=True)), ([5000, 3, 900], 1, 80, 1, {}),
                                                 ([1000, 1001, 200], 100, 4, 2, dict(causal=True, window=77, softcap=30.0)),
                                                 ([3000], 300, 4, 1, dict(causal=True)), ([640, 641], 70, 1, 1, dict(softcap=50.0))])
def test_many_rows(kind, D, page, lengths, Sq, G, Hkv, kw):
    """More than 64 (head dim 64: 512) query rows per kv head: the tcgen05 kernel, partial tiles of rows and keys, whole and split."""
    G = G if D == 128 else 8 * G
    c = Case(lengths, Sq=Sq, Hq=G * Hkv, Hkv=Hkv, D=D, page=page, kind=kind, seed=Sq + page)
    t = c.cuda
    assert fa().attn_cache_path_name(t["q"], c.cache, t["table"], t["lengths"], **kw) == "tc"
    O, LSE = c.run(sink=t["sink"], **kw)
    c.check(O, LSE, sink=True, **kw)
    O2, LSE2 = c.run(sink=t["sink"], **kw)
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    assert fa().attn_cache_check_device_status(c.cache) == 0


def test_many_rows_with_a_table_far_wider_than_the_lengths():
    """Shares of keys that some sequences do not have."""
    c = Case([300, 4000, 0, 65], Sq=40, Hq=4, Hkv=2, page=64, extra_cols=300)
    w = torch.zeros_like(c.cuda["w"])
    c.w.zero_()
    O, LSE = c.run(causal=True, weights=w)
    c.check(O, LSE, w, causal=True)


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("D,G,Sq", [(128, 130, 1), (64, 130, 5), (128, 8, 1), (128, 8, 4), (64, 8, 1), (256, 8, 1), (64, 8, 4)])
def test_the_same_call_gives_the_same_bits(D, G, Sq, kind):
    """The stores of the scores hold up the loads of codes, whose places the next slices' copies take."""
    c = Case([1031, 0, 77, 500], Sq=Sq, Hq=2 * G, Hkv=2, D=D, page=32, kind=kind, seed=D)
    one = None
    for _ in range(200):
        w = c.cuda["w"].clone()
        out = [*c.run(weights=w, softcap=20.0), w]
        one = one or out
        for a, b in zip(one, out):
            assert torch.equal(a, b)
    c.check(*one, softcap=20.0)


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_of_bad_pages(kind, D):
    c = Case([1000, 100], Sq=40, Hq=4 if D == 128 else 32, Hkv=2, D=D, page=32, kind=kind)
    m = fa()
    hidden = [torch.zeros(1000, dtype=torch.bool), torch.zeros(100, dtype=torch.bool)]
    bad = c.cuda["table"].clone()
    for b, col, x in ((0, 1, -1), (0, 13, 2 ** 31 - 1), (0, 31, -5), (1, 0, c.k.shape[0])):
        bad[b, col] = x
        hidden[b][col * 32:(col + 1) * 32] = True
    O, LSE = m.attn_cache_fwd(c.cuda["q"], c.cache, bad, c.cuda["lengths"])
    assert m.attn_cache_check_device_status(c.cache) == 5
    c.table = torch.where((bad.cpu() < 0) | (bad.cpu() >= c.k.shape[0]), 0, bad.cpu())
    c.check(O, LSE, hidden=hidden)


@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_and_nan_in_the_last_tokens(D):
    G = 4 if D == 128 else 32
    c = Case([400], Sq=24, Hq=2 * G, Hkv=2, D=D)   # queries at 376 .. 399
    p, slot = int(c.table[0, 390 // 64]), 390 % 64
    c.v.view(torch.uint8)[p, 0, slot, 3] = 255
    c.k.view(torch.uint8)[p, 1, slot, 5] = 127
    c.cuda["v"].copy_(c.v)
    c.cuda["k"].copy_(c.k)
    assert fa().attn_cache_path_name(c.cuda["q"], c.cache, c.cuda["table"], c.cuda["lengths"]) == "tc"
    O, LSE = (x.cpu().float() for x in c.run(causal=True))
    sees = 390 - 376
    assert torch.isfinite(O[0, :sees]).all() and torch.isfinite(LSE[0, :, :sees]).all()
    assert torch.isnan(O[0, sees:, :G, 3]).all() and torch.isfinite(LSE[0, :G]).all()
    assert torch.isfinite(O[0, sees:, :G][..., [x for x in range(D) if x != 3]]).all()
    assert torch.isnan(O[0, sees:, G:]).all() and torch.isnan(LSE[0, G:, sees:]).all()


@pytest.mark.parametrize("D,G,Sq", [(16, 8, 80), (48, 4, 150), (80, 3, 23), (96, 8, 40), (112, 130, 1)])
@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_many_rows_at_head_dims_between(D, G, Sq, kind):
    for lengths, kw in (([1031, 0, 77, 500], dict(softcap=20.0)), ([9000, 9], dict(causal=True, window=400))):
        c = Case(lengths, Sq=Sq, Hq=2 * G, Hkv=2, D=D, page=32, kind=kind, seed=D)
        t = c.cuda
        assert fa().attn_cache_path_name(t["q"], c.cache, t["table"], t["lengths"], **kw) == "tc"
        w = t["w"].clone()
        out = c.run(sink=t["sink"], weights=w, **kw)
        c.check(out[0], out[1], w, sink=True, **kw)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (F32, 64)])
def test_many_short_sequences(dtype, D):
    g = torch.Generator().manual_seed(1)
    lengths = torch.randint(0, 200, (700,), generator=g).tolist()
    c = Case(lengths, Hq=4, Hkv=2, D=D, page=16, dtype=dtype)
    c.check(*c.run(causal=True), causal=True, rows=list(range(0, 700, 23)) + [699])


@pytest.mark.parametrize("dtype,D,kind", [(BF16, 128, E4M3), (BF16, 256, INT8), (BF16, 64, E4M3), (F32, 128, INT8)])
@pytest.mark.parametrize("Sq,kw", [(1, {}), (1, dict(window=70)), (5, dict(causal=True)), (5, {}), (40, dict(causal=True, window=19, softcap=30.0))])
def test_weights(dtype, D, kind, Sq, kw):
    c = Case([500, 2, 0, 64, 257], Sq=Sq, Hq=8, Hkv=2, D=D, kind=kind, page=32, dtype=dtype, seed=7)
    w, out = c.cuda["w"], c.cuda["w"].clone().fill_(-5.0)
    O, LSE = c.run(sink=c.cuda["sink"], weights=w, weights_out=out, **kw)
    c.check(O, LSE, out, sink=True, **kw)
    for b, n in enumerate(c.lengths):  # behind a sequence's end: as it was
        assert (out[b, :, n:] == -5.0).all()
    assert torch.equal(w.cpu(), c.w)
    O2, LSE2 = c.run(sink=c.cuda["sink"], weights=w, **kw)
    assert torch.equal(O, O2) and torch.equal(LSE, LSE2)
    for b, n in enumerate(c.lengths):
        assert torch.equal(w[b, :, :n], out[b, :, :n]) and torch.equal(w[b, :, n:].cpu(), c.w[b, :, n:])
    O3, _ = c.run(sink=c.cuda["sink"], **kw)
    assert torch.equal(O, O3)


def test_weights_with_a_wider_row_and_every_second_head():
    c = Case([500, 90], Hq=8, Hkv=2)
    wide = torch.full((2, 4, 800), 7.0, device="cuda")
    view = wide[:, ::2, 1:]
    view[..., : c.w.shape[2]] = c.cuda["w"]
    O, LSE = c.run(weights=view)
    c.check(O, LSE, view)
    assert (wide[:, 1::2] == 7.0).all() and (wide[:, :, 0] == 7.0).all()


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (BF16, 256), (F32, 96)])
def test_strided_queries_and_given_outputs(dtype, D):
    c = Case([100, 300, 7], Sq=3, Hq=8, Hkv=2, D=D, dtype=dtype)
    big = torch.full((3, 8, 5, D + 16), math.nan, dtype=dtype, device="cuda")
    q = big[:, :, 1:4, :D].transpose(1, 2)  # [B, Sq, Hq, D], heads before rows in memory
    q.copy_(c.cuda["q"])
    out, lse = torch.empty_like(c.cuda["q"]), torch.empty((3, 8, 3), device="cuda")
    O, LSE = c.run(q=q, causal=True, out=out, lse=lse)
    assert O is out and LSE is lse
    c.check(O, LSE, causal=True)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 128)])
def test_scales_that_differ_by_powers(dtype, D):
    """Pages whose scales lie far apart (as after an outlier), zero values, and a large one nobody looks at."""
    c = Case([640], Hq=4, Hkv=2, D=D, kind=E4M3, dtype=dtype, spread=0.0)
    ids = c.table[0, :10].long()
    c.vs[ids] *= torch.tensor([2.0 ** x for x in (0, -20, 12, -45, 3, 0, 20, -8, 0, 1)])[:, None]
    c.vs[ids[5]] = 0.0
    c.ks[ids[6]] = 2.0 ** -30  # logits of 0, so weight e^-max, on values of 2^20 times the others'
    c.cuda["vs"].copy_(c.vs)
    c.cuda["ks"].copy_(c.ks)
    c.check(*c.run())
    c.vs.zero_()
    c.cuda["vs"].zero_()
    O, LSE = c.run()
    c.check(O, LSE)
    assert (O == 0).all()


@pytest.mark.parametrize("dtype,D,Hq", [(BF16, 64, 8), (BF16, 128, 8), (BF16, 128, 160), (BF16, 256, 8), (F32, 128, 8), (F32, 48, 8)])
@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_scales_that_are_no_powers_of_two(dtype, D, Hq, kind):
    """As another writer may have left them."""
    c = Case([500, 70], Hq=Hq, Hkv=2, D=D, kind=kind, dtype=dtype)
    g = torch.Generator().manual_seed(3)
    for s, name in ((c.ks, "ks"), (c.vs, "vs")):
        s *= torch.rand(s.shape, generator=g) + 0.5
        c.cuda[name].copy_(s)
    c.check(*c.run())


@pytest.mark.parametrize("std", [1e-20, 1e-6, 300.0])
def test_magnitudes_of_queries(std):
    """Far from 1, where fp16 alone would overflow or vanish; the scale brings the logits back."""
    c = Case([90, 200], D=128, q_std=std)
    c.check(*c.run(scale=0.2 / std), scale=0.2 / std)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_elements_of_a_query_far_apart(D):
    c = Case([150], D=D)
    c.q[..., ::3] *= 2.0 ** -20
    c.q[..., 1::7] *= 2.0 ** 10
    c.cuda["q"].copy_(c.q)
    c.check(*c.run(scale=2.0 ** -13), scale=2.0 ** -13)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (BF16, 256), (F32, 128), (BF16, 80), (BF16, 144), (F32, 48)])
def test_nan_in_the_last_tokens_reaches_only_the_rows_that_see_them(dtype, D):
    c = Case([70], Sq=6, Hq=4, Hkv=2, D=D, dtype=dtype)
    p, slot = int(c.table[0, 68 // 64]), 68 % 64
    c.v.view(torch.uint8)[p, 0, slot, 3] = 255   # token 68, kv head 0, column 3: a NaN value
    c.k.view(torch.uint8)[p, 1, slot, 5] = 127   # kv head 1: a NaN key
    c.cuda["v"].copy_(c.v)
    c.cuda["k"].copy_(c.k)
    O, LSE = c.run(causal=True)
    O, LSE = O.cpu().float(), LSE.cpu()
    # Queries stand at 64 .. 69; those at 68 and 69 see token 68.
    assert torch.isfinite(O[0, :4]).all() and torch.isfinite(LSE[0, :, :4]).all()
    assert torch.isnan(O[0, 4:, :2, 3]).all() and torch.isfinite(LSE[0, :2]).all()
    keep = [x for x in range(D) if x != 3]
    assert torch.isfinite(O[0, 4:, :2][..., keep]).all()
    assert torch.isnan(O[0, 4:, 2:]).all() and torch.isnan(LSE[0, 2:, 4:]).all()


def test_a_query_that_is_not_finite_stays_in_its_row():
    for dtype in (BF16, F32):
        c = Case([70], Sq=2, Hq=4, Hkv=2, dtype=dtype)
        q = c.cuda["q"].clone()
        q[0, 0, 1, 5] = math.nan
        q[0, 1, 3, 6] = math.inf
        O, LSE = c.run(q=q)
        bad = torch.zeros(2, 4, dtype=torch.bool)
        bad[0, 1] = bad[1, 3] = True
        assert torch.equal(torch.isnan(O[0]).all(-1).cpu(), bad)
        assert torch.equal(torch.isfinite(O[0]).all(-1).cpu(), ~bad)
        assert torch.isfinite(LSE[0].T[~bad.cuda()]).all()


@pytest.mark.parametrize("dtype,D,page", [(BF16, 128, 16), (BF16, 64, 64), (BF16, 256, 32), (F32, 128, 32)])
def test_bad_page_ids_are_recorded_and_their_tokens_unseen(dtype, D, page):
    c = Case([300, 100], Hq=4, Hkv=2, D=D, page=page, dtype=dtype)
    m = fa()
    c.run()
    assert m.attn_cache_check_device_status(c.cache) == 0
    hidden = [torch.zeros(300, dtype=torch.bool), torch.zeros(100, dtype=torch.bool)]
    bad = c.cuda["table"].clone()
    for b, col, x in ((0, 1, -1), (0, 3, 2 ** 31 - 1), (1, 0, c.k.shape[0])):
        bad[b, col] = x
        hidden[b][col * page:(col + 1) * page] = True
    w = torch.zeros_like(c.cuda["w"])
    O, LSE = m.attn_cache_fwd(c.cuda["q"], c.cache, bad, c.cuda["lengths"], weights=w)
    assert m.attn_cache_check_device_status(c.cache) == 5
    assert m.attn_cache_check_device_status(c.cache) == 0
    c.table = torch.where((bad.cpu() < 0) | (bad.cpu() >= c.k.shape[0]), 0, bad.cpu())
    c.w.zero_()
    c.check(O, LSE, w, hidden=hidden)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_lengths_outside_the_table(dtype):
    c = Case([128, 128], D=128, dtype=dtype, extra_cols=0)
    m = fa()
    O, LSE = m.attn_cache_fwd(c.cuda["q"], c.cache, c.cuda["table"], i32(-3, 129).cuda())
    assert m.attn_cache_check_device_status(c.cache) == 5
    assert (O[0] == 0).all() and (LSE[0] == -math.inf).all()
    c.check(O, LSE, rows=[1])


def test_nothing_to_do():
    c = Case([5])
    m = fa()
    t = c.cuda
    O, LSE = m.attn_cache_fwd(t["q"][:, :0], c.cache, t["table"], t["lengths"])
    assert O.shape == (1, 0, 8, 128) and LSE.shape == (1, 8, 0)
    O, LSE = m.attn_cache_fwd(t["q"][:0], c.cache, t["table"][:0], t["lengths"][:0])
    assert O.shape == (0, 1, 8, 128)
    for dtype in (BF16, F32):  # a table without columns
        O, LSE = m.attn_cache_fwd(t["q"].to(dtype), c.cache, t["table"][:, :0], i32(0).cuda(), weights=t["w"][:, :, :0])
        assert (O == 0).all() and (LSE == -math.inf).all()


def test_host_queries_are_refused():
    c = Case([5])
    with pytest.raises(ValueError, match="every tensor"):
        c.run(q=c.q)


def test_shared_pages_and_two_streams():
    """Two sequences over the same pages, and two calls at once on two streams over one cache."""
    c = Case([5000, 5000], Hq=8, Hkv=2)
    c.table[1] = c.table[0]
    c.cuda["table"].copy_(c.table)
    ref_O, ref_LSE = c.run(causal=True)
    c.check(ref_O, ref_LSE, causal=True)
    q2 = c.cuda["q"].flip(0).contiguous()
    want2 = c.run(q=q2, causal=True)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            a = c.run(causal=True)
        with torch.cuda.stream(s2):
            b = c.run(q=q2, causal=True)
        got.append((a, b))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a[0], ref_O) and torch.equal(b[0], want2[0])


def test_codes_past_32_bits():
    """A cache of more than 2^32 codes: the last pages are read, appended to and moved to."""
    m = fa()
    P, H, page, D = (1 << 32) // (8 * 128 * 128) + 40, 8, 128, 128
    cache = m.AttnCache.empty(P, page, H, D)
    ids = [P - 1, 3, P - 7, P // 2 + 1]
    table = i32(*ids).cuda()[None]
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn((1, 450, H, D), generator=g).bfloat16() for _ in range(2))
    lengths = m.attn_cache_append(cache, k.cuda(), v.cuda(), table, i32(0).cuda())
    q = torch.randn((1, 1, 16, D), generator=g)
    w = torch.zeros((1, H, 512), device="cuda")
    for dtype in (BF16, F32):
        O, LSE = m.attn_cache_fwd(q.to(dtype).cuda(), cache, table, lengths, weights=w)
        kf, vf = (ref.values(c[ids].cpu(), s[ids].cpu()) for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        row = torch.arange(4)
        kk, vv = ref.gather(kf, row, 450, page), ref.gather(vf, row, 450, page)
        vs = ref.gather_scale(cache.v_scale[ids].cpu(), row, 450, page)
        o, lse, _, pv, mag = ref.attend(q[0].to(dtype).double(), kk, vv, vs=vs, terms=1 if dtype == BF16 else 2)
        _, rel = ref.bounds(D, 450, mag, 0.0, dtype == BF16)
        eps = torch.finfo(dtype).eps / 2
        assert ((O[0].cpu().double() - o).abs() <= eps * o.abs() + (1 + eps) * rel * pv).all()
    out = i32(P - 2).cuda()[None]
    kept, n, _ = m.attn_cache_evict(cache, table, lengths, w, out, keep=100, recent=10)
    assert n.tolist() == [100]
    moved = ref.values(cache.k[P - 2:P - 1].cpu(), cache.k_scale[P - 2:P - 1].cpu())
    src = ref.values(cache.k[ids].cpu(), cache.k_scale[ids].cpu())
    for h in range(H):
        at = kept[0, h].long().cpu()
        x = src[at // page, h, at % page]
        assert (moved[0, h, :100] - x).abs().max() <= 2.0 ** -4 * x.abs().max()


# ---------------------------------------------------------------- appending

@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("dtype,D,page,H", [(BF16, 128, 64, 2), (F32, 64, 16, 3), (BF16, 16, 32, 1), (F32, 512, 128, 1), (BF16, 80, 64, 2),
                                            (BF16, 256, 128, 1)])
@pytest.mark.parametrize("S", [1, 5, 200])
def test_append(kind, dtype, D, page, H, S):
    """Behind lengths inside and at the ends of pages, ragged counts, strided rows; every code and scale exact."""
    m = fa()
    g = torch.Generator().manual_seed(S + D)
    lengths = [0, 1, page - 1, page, 3 * page - 2, 77]
    counts = [S, S, 0 if S > 1 else 1, max(1, S // 2), S, S - 1]
    B, cols = len(lengths), (max(lengths) + S) // page + 2
    P = B * cols + 2
    table = torch.randperm(P, generator=g)[: B * cols].view(B, cols).int()
    k, v, ks, vs = ref.make_cache(P, H, page, D, kind, seed=D, spread=1.0)
    cache = m.AttnCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
    x = [(torch.randn((B, H, S + 1, D + 16), generator=g) * 2).to(dtype) for _ in range(2)]
    x[1][0, :, 0] = 0.0
    w = torch.rand((B, H, cols * page), generator=g)
    wc = w.cuda()
    rows = [t.cuda()[:, :, 1:, :D].transpose(1, 2) for t in x]
    n = m.attn_cache_append(cache, *rows, table.cuda(), i32(*lengths).cuda(), counts=i32(*counts).cuda(), weights=wc)
    assert n.tolist() == [a + c for a, c in zip(lengths, counts)]
    for c, s, t in ((k, ks, x[0]), (v, vs, x[1])):
        ref.append(c, s, t[:, :, 1:, :D].transpose(1, 2).double(), table, lengths, counts, page)
    assert ref.codes_equal(cache.k, k) and ref.codes_equal(cache.v, v)
    assert torch.equal(cache.k_scale.cpu(), ks) and torch.equal(cache.v_scale.cpu(), vs)
    for b in range(B):
        w[b, :, lengths[b]:lengths[b] + counts[b]] = 0.0
    assert torch.equal(wc.cpu(), w)
    assert m.attn_cache_check_device_status(cache) == 0


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_append_token_by_token_grows_the_scale(kind):
    """Growing rows, one at a time: the earlier codes are requantised; the values stay within the roundings."""
    m = fa()
    page, H, D = 32, 2, 64
    k, v, ks, vs = ref.make_cache(4, H, page, D, kind)
    cache = m.AttnCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
    table, n = i32(2, 0).cuda()[None], i32(0).cuda()
    g = torch.Generator().manual_seed(1)
    x = torch.randn((1, 40, H, D), generator=g) * torch.exp2(torch.arange(40) / 4.0)[None, :, None, None]
    grown = set()
    for i in range(40):
        n2 = m.attn_cache_append(cache, x[:, i:i + 1].cuda(), -x[:, i:i + 1].cuda(), table, n)
        ref.append(k, ks, x[:, i:i + 1].double(), table.cpu(), [i], [1], page)
        ref.append(v, vs, -x[:, i:i + 1].double(), table.cpu(), [i], [1], page)
        n = n2
        grown.add(float(ks[2, 0]))
    assert len(grown) > 5 and n.tolist() == [40]
    assert ref.codes_equal(cache.k, k) and ref.codes_equal(cache.v, v) and torch.equal(cache.k_scale.cpu(), ks)
    got = ref.gather(ref.values(cache.k.cpu(), cache.k_scale.cpu()), table[0].cpu(), 40, page)
    s = cache.k_scale.cpu().double()[table[0].cpu().long()].repeat_interleave(page, 0)[:40, :, None]
    want = x[0].double()
    if kind == INT8:   # half a step per time the scale grew, each at most half the last one's: one step in all
        assert ((got - want).abs() <= s).all()
    else:              # half of an e4m3 step, and where the codes became subnormal half a step each: one in all
        assert ((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -9 * s).all()


def test_append_values_at_the_scale_rule_s_edges():
    m = fa()
    top = {E4M3: 448.0, INT8: 127.0}
    for kind in (E4M3, INT8):
        cache = m.AttnCache.empty(16, 16, 1, 16, dtype=kind)
        amax = [top[kind], math.nextafter(top[kind], 1e9), 2.0 ** -70, 0.0, 3e38, 2.0 ** -60 * top[kind], 1e-38, 1.0]
        amax[1] = float(torch.nextafter(torch.tensor(top[kind]), torch.tensor(1e9)))
        x = torch.zeros(8, 1, 1, 16)
        x[:, 0, 0, 3] = torch.tensor(amax)
        x[:, 0, 0, 4] = -x[:, 0, 0, 3] / 3
        table = torch.arange(8, dtype=torch.int32)[:, None].contiguous()
        m.attn_cache_append(cache, x.cuda(), -x.cuda(), table.cuda(), torch.zeros(8, dtype=torch.int32, device="cuda"))
        want = [ref.need_scale(float(a), kind) for a in x[:, 0, 0, 3]]
        assert cache.k_scale[:8, 0].tolist() == want
        k = torch.zeros((16, 1, 16, 16), dtype=torch.uint8).view(kind)
        ks = torch.ones((16, 1))
        ref.append(k, ks, x.double(), table, [0] * 8, [1] * 8, 16)
        assert ref.codes_equal(cache.k[:8, :, :1], k[:8, :, :1])


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_append_non_finite_values(kind):
    m = fa()
    cache = m.AttnCache.empty(4, 16, 1, 16, dtype=kind)
    x = torch.ones((1, 2, 1, 16))
    x[0, 0, 0, 1], x[0, 0, 0, 2], x[0, 1, 0, 3] = math.inf, -math.inf, math.nan
    m.attn_cache_append(cache, x.cuda(), torch.ones_like(x).cuda(), i32(1).cuda()[None], i32(0).cuda())
    assert m.attn_cache_check_device_status(cache) == 5
    got = cache.k[1, 0, :2].cpu().float()
    q = ref.QMAX[kind]
    assert cache.k_scale[1, 0].item() == ref.need_scale(1.0, kind)
    assert got[0, 1] == q and got[0, 2] == -q
    assert math.isnan(got[1, 3]) if kind == E4M3 else got[1, 3] == 0
    assert torch.isfinite(got.flatten()[[0, 3, 4, 5, 16, 17]]).all()


def test_append_into_bad_pages_and_past_the_table():
    m = fa()
    cache = m.AttnCache.empty(4, 16, 2, 32)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    x = torch.ones((3, 20, 2, 32), device="cuda")
    table = torch.tensor([[-1, 4], [1 << 30, -7], [2, 3]], dtype=torch.int32).cuda()
    w = torch.ones((3, 2, 32), device="cuda")
    n = m.attn_cache_append(cache, x, x, table, i32(0, 9, 30).cuda(), weights=w)
    assert m.attn_cache_check_device_status(cache) == 5
    assert n.tolist() == [20, 29, 32]
    for t, b in zip((cache.k, cache.v), before):
        assert torch.equal(t.view(torch.uint8)[:3], b.view(torch.uint8)[:3])
        assert torch.equal(t.view(torch.uint8)[3, :, :14], b.view(torch.uint8)[3, :, :14])
    assert (cache.k.float()[3, :, 14:] * cache.k_scale[3, :, None, None] == 1).all()
    assert (w[2, :, 30:] == 0).all() and (w[2, :, :30] == 1).all()
    # Lengths outside the table: nothing is written, nothing read out of place.
    cache2 = m.AttnCache.empty(4, 16, 2, 32)
    n = m.attn_cache_append(cache2, x[:2], x[:2], table[2:].expand(2, 2).contiguous(), i32(33, 1 << 30).cuda())
    assert n.tolist() == [32, 32] and m.attn_cache_check_device_status(cache2) == 5
    assert (cache2.k.float() == 0).all()


def test_append_counts_outside_their_range_and_strides_of_single_rows():
    m = fa()
    cache = m.AttnCache.empty(8, 16, 2, 32)
    table = torch.arange(8, dtype=torch.int32).view(4, 2).cuda()
    big = torch.ones((4, 2, 35), device="cuda")
    x = torch.as_strided(big, (4, 3, 2, 32), (64, 0, 32, 1), 0)    # three equal rows
    n = m.attn_cache_append(cache, x, x, table, torch.zeros(4, dtype=torch.int32, device="cuda"), counts=i32(-3, 0, 2, 99).cuda())
    assert n.tolist() == [0, 0, 2, 3] and m.attn_cache_check_device_status(cache) == 0
    assert (cache.k.float()[0:4] == 0).all() and (cache.k.float()[6, :, :3] * cache.k_scale[6, :, None, None] == 1).all()
    one = torch.as_strided(big, (1, 1, 2, 32), (5, 3, 64, 1), 0)   # odd strides where nothing steps
    assert m.attn_cache_append(cache, one, one, table[:1], i32(7).cuda()).tolist() == [8]
    q = torch.as_strided(big, (1, 1, 2, 32), (7, 1, 32, 1), 0)
    O, _ = m.attn_cache_fwd(q, cache, table[2:3], i32(2).cuda())
    assert torch.equal(O, torch.ones_like(O))


def test_append_on_a_scale_that_is_no_power_of_two():
    m = fa()
    for kind in (E4M3, INT8):
        k, v, ks, vs = ref.make_cache(3, 2, 32, 64, kind, std=4.0)
        ks *= 1.37
        vs *= 0.77
        cache = m.AttnCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
        table = i32(1, 2).cuda()[None]
        x = torch.randn((1, 5, 2, 64), generator=torch.Generator().manual_seed(1)) * 0.1
        m.attn_cache_append(cache, x.cuda(), 500 * x.cuda(), table, i32(20).cuda())
        assert torch.equal(cache.k_scale.cpu(), ks)                    # the present scale holds the new rows
        got = ref.values(cache.k.cpu(), cache.k_scale.cpu())[1, :, 20:25].transpose(0, 1)
        s = ks[1].double()[None, :, None]
        step = s if kind == INT8 else torch.maximum(2.0 ** -9 * s, 2.0 ** -3 * x[0].double().abs())
        assert ((got - x[0].double()).abs() <= 0.5 * step * (1 + 2.0 ** -20)).all()
        assert ((cache.v_scale[1].cpu().log2() % 1) == 0).all()         # the other had to grow, to a power of two
        old = ref.values(v, vs)[1, :, :20]
        now = ref.values(cache.v.cpu(), cache.v_scale.cpu())[1, :, :20]
        s = cache.v_scale[1].cpu().double()[:, None, None]
        assert ((now - old).abs() <= 0.5 * (1 + 2.0 ** -20) * (s if kind == INT8 else torch.maximum(2.0 ** -9 * s, 2.0 ** -3 * old.abs()))).all()


def test_append_no_rows():
    m = fa()
    cache = m.AttnCache.empty(2, 16, 1, 16)
    x = torch.zeros((2, 0, 1, 16), device="cuda")
    assert m.attn_cache_append(cache, x, x, i32(0, 1).cuda()[:, None], i32(3, 4).cuda()).tolist() == [3, 4]
    assert m.attn_cache_append(cache, x[:0], x[:0], torch.zeros((0, 1), dtype=torch.int32, device="cuda"),
                               torch.zeros(0, dtype=torch.int32, device="cuda")).numel() == 0


# ---------------------------------------------------------------- eviction

def evict_case(lengths, *, keep, recent=0, first=0, H=2, page=64, D=64, kind=E4M3, seed=0, weights=None, scales=None):
    m = fa()
    c = Case(lengths, Hq=H, Hkv=H, D=D, page=page, kind=kind, seed=seed)
    if scales is not None:
        c.ks, c.vs = scales(c.ks), scales(c.vs)
    B = len(lengths)
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(c.w.shape, generator=g).exp() if weights is None else weights(c.w.shape, g)
    pages = -(-keep // page)
    P0 = c.k.shape[0]
    out = (P0 + torch.randperm(B * pages + 1, generator=g)[: B * pages]).view(B, pages).int()
    grow = lambda t: torch.cat([t, torch.zeros((B * pages + 1, *t.shape[1:]), dtype=t.dtype)])
    k, v = (grow(t.view(torch.uint8)).view(kind) for t in (c.k, c.v))
    ks, vs = grow(c.ks), grow(c.vs)
    cache = m.AttnCache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())
    kept, n, wo = m.attn_cache_evict(cache, c.cuda["table"], c.cuda["lengths"], w.cuda(), out.cuda(), keep=keep, recent=recent,
                                     first=first)
    kept, n, wo = kept.cpu(), n.cpu(), wo.cpu()
    assert n.tolist() == [min(x, keep) for x in lengths]
    fk, fv = ref.values(k, ks), ref.values(v, vs)
    for b in range(B):
        for h in range(H):
            at = ref.select(w[b, h], lengths[b], keep, first, recent)
            assert kept[b, h, :len(at)].tolist() == at, (b, h)
            assert (kept[b, h, len(at):] == -1).all() and (wo[b, h, len(at):] == 0).all()
            assert torch.equal(wo[b, h, :len(at)].nan_to_num(-9.0), w[b, h, at].nan_to_num(-9.0))
            pos = torch.tensor(at, dtype=torch.long)
            for codes, scales, f in ((k, ks, fk), (v, vs, fv)):
                x = f[c.table[b, pos // page].long(), h, pos % page] if len(at) else f[:0, 0, 0]
                for i in range(0, len(at), page):
                    p, blk = int(out[b, i // page]), x[i:i + page]
                    s = ref.need_scale(float(blk.abs().max()), kind)
                    scales[p, h] = s
                    codes[p, h, :blk.shape[0]] = ref.round_codes(blk / s, kind)
    assert ref.codes_equal(cache.k, k) and ref.codes_equal(cache.v, v)
    same = lambda a, b: torch.equal(a.cpu().nan_to_num(-1.0), b.nan_to_num(-1.0))
    assert same(cache.k_scale, ks) and same(cache.v_scale, vs)
    assert m.attn_cache_check_device_status(cache) == 0


@pytest.mark.parametrize("kind,D,page", [(E4M3, 64, 64), (INT8, 128, 16), (E4M3, 80, 32), (INT8, 512, 128)])
@pytest.mark.parametrize("keep,recent,first", [(1, 0, 0), (64, 0, 0), (100, 17, 5), (100, 100, 0), (100, 60, 40), (129, 0, 129), (500, 33, 3)])
def test_evict(kind, D, page, keep, recent, first):
    evict_case([700, 0, 1, 100, 101, 499], keep=keep, recent=recent, first=first, kind=kind, D=D, page=page, seed=keep)


def test_evict_ties_and_special_weights():
    def ties(shape, g):
        w = torch.randint(0, 4, shape, generator=g).float()
        w[w == 0] *= -1  # -0 and 0 are equal
        w[0, 0] = 0.0
        return w

    def special(shape, g):
        w = torch.randn(shape, generator=g)
        w.view(-1)[::7] = math.nan
        w.view(-1)[1::11] = math.inf
        w.view(-1)[2::13] = -math.inf
        w.view(-1)[3::17] = 1e-42
        return w
    for f in (ties, special):
        for keep, recent, first in ((50, 0, 0), (333, 20, 7), (90, 89, 0)):
            evict_case([600, 340, 334], keep=keep, recent=recent, first=first, weights=f)


@pytest.mark.parametrize("kind", [E4M3, INT8])
def test_evict_scales_that_are_no_powers_of_two_or_far_apart(kind):
    g = torch.Generator().manual_seed(8)
    evict_case([400, 130], keep=90, recent=10, kind=kind, scales=lambda s: s * (torch.rand(s.shape, generator=g) + 0.5))
    evict_case([400, 130], keep=90, recent=10, kind=kind, scales=lambda s: s * torch.exp2(torch.randint(-30, 30, s.shape, generator=g).float()))
    evict_case([400, 130], keep=90, recent=10, kind=kind, scales=lambda s: s * 0.0)


@pytest.mark.parametrize("n,keep", [(70001, 4096), (131072, 1000), (40000, 39999), (33000, 2)])
def test_evict_long(n, keep):
    evict_case([n, n // 3], keep=keep, recent=keep // 8, first=keep // 16, H=1, D=16, page=128,
               weights=lambda s, g: torch.where(torch.rand(s, generator=g) < 0.3, 0.0, torch.randn(s, generator=g).exp()))


def test_evict_bad_pages():
    m = fa()
    c = Case([100, 100], Hq=2, Hkv=2, D=32, page=16)
    P = c.k.shape[0]
    k = torch.zeros((P + 4, 2, 16, 32), dtype=torch.uint8)
    k[:P] = c.k.view(torch.uint8)
    s = torch.ones((P + 4, 2))
    s[:P] = c.ks
    cache = m.AttnCache(k.view(E4M3).cuda(), k.view(E4M3).cuda(), s.cuda(), s.cuda())
    table = c.cuda["table"].clone()
    table[0, 2] = -1
    out = torch.tensor([[P, P + 1], [P + 4, P + 3]], dtype=torch.int32).cuda()
    w = torch.ones_like(c.cuda["w"])
    kept, n, _ = m.attn_cache_evict(cache, table, c.cuda["lengths"], w, out, keep=32, first=20, recent=4)
    assert m.attn_cache_check_device_status(cache) == 5
    assert n.tolist() == [32, 32]
    got = cache.k.float().cpu()
    at = kept[0, 0, 16:].cpu()
    assert (got[P + 1, 0][(at >= 32) & (at < 48)] == 0).all()      # tokens of the bad page: zeros
    assert (cache.k.view(torch.uint8)[P + 2] == 0).all()           # nothing went where nobody asked
    assert cache.k.view(torch.uint8)[P + 3].any()                  # the second row's good page


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("dtype,D,page,window,softcap", [(BF16, 128, 32, 0, 30.0), (BF16, 64, 16, 40, 0.0), (F32, 64, 64, 0, 0.0)])
def test_a_serving_loop(kind, dtype, D, page, window, softcap):
    """Prompts, single tokens, an eviction into fresh pages, and more tokens: at every step the output is that of
    float64 attention over what the cache holds, and what it holds is the tokens within their roundings."""
    m = fa()
    g = torch.Generator().manual_seed(11)
    B, H, G, keep = 3, 2, 4, 96
    counts = [150, 1, 97]
    cols = (150 + 12) // page + 1
    P = B * cols + B * (-(-keep // page) + 1)
    cache = m.AttnCache.empty(P, page, H, D, dtype=kind)
    perm = torch.randperm(P, generator=g).int()
    table = perm[: B * cols].view(B, cols).cuda()
    w = torch.full((B, H, cols * page), 99.0, device="cuda")
    new = lambda S: [torch.randn((B, S, H, D), generator=g).to(dtype).cuda() for _ in range(2)]
    n = torch.zeros(B, dtype=torch.int32, device="cuda")
    hist = [[torch.zeros((0, H, D)) for _ in range(B)] for _ in range(2)]
    sink = torch.randn(H * G, generator=g)

    def step(S, counts, table, w, n):
        kv = new(S)
        n2 = m.attn_cache_append(cache, *kv, table, n, counts=i32(*counts).cuda(), weights=w)
        for x in range(2):
            for b in range(B):
                hist[x][b] = torch.cat([hist[x][b], kv[x][b, :counts[b]].float().cpu()])
        q = torch.randn((B, 1, H * G, D), generator=g).to(dtype)
        before = w.clone()
        O, LSE = m.attn_cache_fwd(q.cuda(), cache, table, n2, causal=True, window=window, softcap=softcap, sink=sink.cuda(), weights=w)
        for b in range(B):
            L = int(n2[b])
            kk, vv = (ref.gather(ref.values(c.cpu(), s.cpu()), table[b].cpu(), L, page)
                      for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
            vs = ref.gather_scale(cache.v_scale.cpu(), table[b].cpu(), L, page)
            o, lse, ww, pv, mag = ref.attend(q[b].double(), kk, vv, causal=True, window=window, softcap=softcap, sink=sink, vs=vs,
                                             terms=1 if dtype == BF16 else 2)
            _, rel = ref.bounds(D, L, mag, softcap, dtype == BF16)
            eps = torch.finfo(dtype).eps / 2
            assert ((O[b].cpu().double() - o).abs() <= eps * o.abs() + (1 + eps) * rel * pv + 1e-37).all()
            want = before[b, :, :L].cpu().double() + ww
            assert ((w[b, :, :L].cpu().double() - want).abs() <= (2 * rel + 2.0 ** -20) * ww + 2.0 ** -24 * want).all()
            if kind == INT8:  # a step of each page's scale bounds any number of growths
                s = cache.k_scale.cpu().double()[table[b].cpu().long()].repeat_interleave(page, 0)[:L, :, None]
                assert ((kk - hist[0][b].double()).abs() <= s).all()
        return n2

    n = step(150, counts, table, w, n)
    for _ in range(6):
        n = step(1, [1] * B, table, w, n)
    assert n.tolist() == [156, 7, 103]
    out = perm[B * cols:].view(B, -1).cuda()
    kept, n, w2 = m.attn_cache_evict(cache, table, n, w, out[:, : -(-keep // page)], keep=keep, recent=16, first=2)
    assert n.tolist() == [96, 7, 96]
    kept = kept.cpu().long()
    for x in range(2):
        for b in range(B):
            hist[x][b] = torch.stack([hist[x][b][kept[b, h, : int(n[b])], h] for h in range(H)], 1)
    room = torch.zeros((B, H, out.shape[1] * page), device="cuda")
    room[:, :, :keep] = w2
    for _ in range(4):
        n = step(1, [1] * B, out.contiguous(), room, n)
    assert n.tolist() == [100, 11, 100]
    assert m.attn_cache_check_device_status(cache) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_decoding_step_in_a_graph(dtype):
    """Append, attention with weights and eviction captured once; replayed with other lengths, tables and tokens, next to another
    graph of the same calls (each has its scratch of its own)."""
    m = fa()
    g = torch.Generator().manual_seed(2)
    B, H, G, D, page, cols = 2, 2, 4, 128, 64, 40
    P = B * cols + 8

    def make(seed):
        k, v, ks, vs = (t.cuda() for t in ref.make_cache(P, H, page, D, E4M3, seed=seed))
        return dict(cache=m.AttnCache(k, v, ks, vs), table=torch.randperm(P, generator=g)[: B * cols].view(B, cols).int().cuda(),
                    lengths=i32(1000, 17).cuda(), kv=[torch.randn((B, 1, H, D), generator=g).to(dtype).cuda() for _ in range(2)],
                    q=torch.randn((B, 1, H * G, D), generator=g).to(dtype).cuda(), w=torch.rand((B, H, cols * page), generator=g).cuda(),
                    w_out=torch.zeros((B, H, cols * page), device="cuda"), out=torch.arange(P - 8, P, dtype=torch.int32).view(2, 4).cuda())

    def step(s):
        n = m.attn_cache_append(s["cache"], *s["kv"], s["table"], s["lengths"], weights=s["w"])
        O, LSE = m.attn_cache_fwd(s["q"], s["cache"], s["table"], n, causal=True, weights=s["w"], weights_out=s["w_out"])
        return (O, LSE, *m.attn_cache_evict(s["cache"], s["table"], n, s["w_out"], s["out"], keep=200, recent=5))

    states, graphs, outs = [make(1), make(2)], [], []
    for s in states:
        s["out"] = torch.tensor(sorted(set(range(P)) - set(s["table"].flatten().tolist()))[:8], dtype=torch.int32).view(2, 4).cuda()
        step(s)
    torch.cuda.synchronize()
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(s))
        graphs.append(graph)
    for lengths in ((1001, 18), (0, 2500), (64, 63)):
        for s in states:
            s["lengths"].copy_(i32(*lengths))
            s["q"].copy_(torch.randn(s["q"].shape, generator=g))
            for x in s["kv"]:
                x.copy_(torch.randn(x.shape, generator=g))
        before = [[t.clone() for t in (s["cache"].k.view(torch.uint8), s["cache"].v.view(torch.uint8), s["cache"].k_scale,
                                       s["cache"].v_scale, s["w"])] for s in states]
        st = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for x in range(2):
            with torch.cuda.stream(st[x]):
                graphs[x].replay()
        torch.cuda.synchronize()
        for x, s in enumerate(states):
            got = [t.clone() for t in outs[x]]
            for t, old in zip((s["cache"].k.view(torch.uint8), s["cache"].v.view(torch.uint8), s["cache"].k_scale, s["cache"].v_scale,
                               s["w"]), before[x]):
                t.copy_(old)
            want = step(s)
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_tensors_of_another_stream():
    """A call on a side stream whose inputs were made on the default one, and results used on a third."""
    c = Case([3000], Hq=8, Hkv=2)
    want = c.run(causal=True)
    torch.cuda.synchronize()
    side, third = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        O, LSE = c.run(causal=True)
    third.wait_stream(side)
    with torch.cuda.stream(third):
        twice = O * 2
    torch.cuda.synchronize()
    assert torch.equal(O, want[0]) and torch.equal(twice, want[0] * 2)
