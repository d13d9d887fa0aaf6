"""Host-side tests of the 8-bit cache: refusals of the C ABI and of the binding before anything
launches, and the arithmetic by which attention's work is shared out, on the CPU.  No CUDA call
is made here."""
import ctypes
import random

import pytest
import torch

import attention_flash_attn_gb300 as fa


@pytest.fixture(scope="module")
def capi():
    from attention_flash_attn_gb300 import build as b
    b.build()
    from attention_flash_attn_gb300 import _capi
    return _capi


FAKE = 0x10000  # never dereferenced: only validation runs in these tests


def cache_args(capi, **kw):
    c = capi.AttnCacheArgs(capi.ATTN_CACHE_E4M3, 8, 64, 2, 128, FAKE, FAKE, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def seq_args(capi, **kw):
    s = capi.AttnCacheSeqs(2, 4, FAKE, 4, FAKE)
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def fwd_args(capi, **kw):
    a = capi.AttnCacheFwdArgs(1, 1, 4, FAKE, 512, 512, 128, 1, 0, 0.0, 0.1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def append_args(capi, **kw):
    a = capi.AttnCacheAppendArgs(1, 3, FAKE, FAKE, 768, 256, 128, 768, 256, 128, None, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def evict_args(capi, **kw):
    a = capi.AttnCacheEvictArgs(100, 4, 10, FAKE, 512, 256, FAKE, 2, FAKE, FAKE + 256, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_CACHE = [("kind", 0, 1), ("kind", 3, 1), ("num_pages", 0, 1), ("page_size", 8, 2), ("page_size", 48, 2),
             ("page_size", 256, 2), ("Hkv", 0, 1), ("Hkv", 70000, 1), ("D", 0, 1), ("D", 72, 2), ("D", 528, 2), ("k", None, 1),
             ("v", FAKE + 8, 1), ("k_scale", None, 1), ("v_scale", FAKE + 2, 1), ("status", None, 1)]
BAD_SEQS = [("B", -1, 1), ("max_pages", -1, 1), ("max_pages", 1 << 19, 2), ("table", None, 1), ("table_stride", 3, 1),
            ("lengths", None, 1), ("lengths", FAKE + 2, 1)]
BAD_FWD = [("dtype", 3, 1), ("Sq", -1, 1), ("Hq", 3, 1), ("Hq", 0, 1), ("softcap", -1.0, 1), ("softcap", float("nan"), 1),
           ("scale", float("inf"), 1), ("q", None, 1), ("q", FAKE + 8, 1), ("q_stride_s", 12, 1), ("q_stride_b", -8, 1),
           ("softmax_type", 2, 1), ("weights", FAKE, 1), ("weights_out", FAKE, 1), ("sink", FAKE + 1, 1)]
BAD_APPEND = [("dtype", 0, 1), ("S", -1, 1), ("k", None, 1), ("v", FAKE + 4, 1), ("k_stride_s", 4, 1), ("v_stride_h", -8, 1),
              ("counts", FAKE + 1, 1), ("lengths_out", FAKE, 1), ("weights", FAKE + 2, 1)]
BAD_EVICT = [("keep", 0, 1), ("keep", 13, 1), ("first", -1, 1), ("recent", -1, 1), ("weights", None, 1), ("table_out", None, 1),
             ("table_out_stride", 1, 1), ("kept", None, 1), ("lengths_out", None, 1), ("lengths_out", FAKE, 1),
             ("weights_out", None, 1), ("weights_stride_h", -4, 1)]


def calls(capi, c, s, f=None, a=None, e=None):
    L = capi.lib()
    r = ctypes.byref
    f, a, e = f or fwd_args(capi), a or append_args(capi, lengths_out=FAKE + 512), e or evict_args(capi)
    return (lambda: L.attn_cache_fwd(r(c), r(s), r(f), FAKE, FAKE, FAKE, 1 << 40, None),
            lambda: L.attn_cache_append(r(c), r(s), r(a), None),
            lambda: L.attn_cache_evict(r(c), r(s), r(e), None),
            lambda: L.attn_cache_fwd_workspace_size(r(c), r(s), r(f)))


@pytest.mark.parametrize("field,value,status", BAD_CACHE)
def test_bad_caches_are_refused_by_every_call(capi, field, value, status):
    n = capi.lib().attn_launch_counter()
    fwd, app, ev, size = calls(capi, cache_args(capi, **{field: value}), seq_args(capi))
    assert (fwd(), app(), ev(), size()) == (status, status, status, 0)
    assert capi.lib().attn_launch_counter() == n


@pytest.mark.parametrize("field,value,status", BAD_SEQS)
def test_bad_sequences_are_refused_by_every_call(capi, field, value, status):
    n = capi.lib().attn_launch_counter()
    fwd, app, ev, size = calls(capi, cache_args(capi), seq_args(capi, **{field: value}))
    assert (fwd(), app(), ev(), size()) == (status, status, status, 0)
    assert capi.lib().attn_launch_counter() == n


@pytest.mark.parametrize("field,value,status", BAD_FWD)
def test_bad_attention_arguments_are_refused(capi, field, value, status):
    n = capi.lib().attn_launch_counter()
    a = fwd_args(capi, **{field: value})
    fwd, _, _, size = calls(capi, cache_args(capi), seq_args(capi), f=a)
    assert (fwd(), size()) == (status, 0)
    r = ctypes.byref
    assert capi.lib().attn_cache_path_name(r(cache_args(capi)), r(seq_args(capi)), r(a)) == b""
    assert capi.lib().attn_launch_counter() == n


def test_sink_and_off_by_one_exclude_each_other(capi):
    a = fwd_args(capi, softmax_type=capi.ATTN_SOFTMAX_OFF_BY_ONE)
    assert calls(capi, cache_args(capi), seq_args(capi), f=a)[3]() > 0
    a.sink = FAKE
    assert calls(capi, cache_args(capi), seq_args(capi), f=a)[0]() == 1


@pytest.mark.parametrize("field,value,status", BAD_APPEND)
def test_bad_append_arguments_are_refused(capi, field, value, status):
    n = capi.lib().attn_launch_counter()
    assert calls(capi, cache_args(capi), seq_args(capi), a=append_args(capi, **{field: value}))[1]() == status
    assert capi.lib().attn_launch_counter() == n


@pytest.mark.parametrize("field,value,status", BAD_EVICT)
def test_bad_eviction_arguments_are_refused(capi, field, value, status):
    n = capi.lib().attn_launch_counter()
    assert calls(capi, cache_args(capi), seq_args(capi), e=evict_args(capi, **{field: value}))[2]() == status
    assert capi.lib().attn_launch_counter() == n


def test_outputs_and_workspace_are_checked(capi):
    L, r = capi.lib(), ctypes.byref
    c, s, a = cache_args(capi), seq_args(capi), fwd_args(capi)
    need = L.attn_cache_fwd_workspace_size(r(c), r(s), r(a))
    assert need >= 256 and need % 256 == 0
    n = L.attn_launch_counter()
    call = lambda O=FAKE, LSE=FAKE, ws=FAKE, size=need: L.attn_cache_fwd(r(c), r(s), r(a), O, LSE, ws, size, None)
    assert call(O=None) == 1 and call(LSE=None) == 1 and call(O=FAKE + 8) == 1
    assert call(ws=None) == 3 and call(size=need - 1) == 3 and call(ws=FAKE + 16) == 3
    assert L.attn_launch_counter() == n


def test_rows_of_written_weights_that_overlap_are_refused(capi):
    s = seq_args(capi)
    room = s.max_pages * 64
    for sb, sh, ok in ((2 * room, room, True), (room, 2 * room, True), (0, room, False), (room, 0, False), (2 * room - 1, room, False),
                       (room, room, False)):
        f = fwd_args(capi, weights=FAKE, weights_out=FAKE, weights_stride_b=sb, weights_stride_h=sh)
        assert (calls(capi, cache_args(capi), s, f=f)[3]() > 0) == ok, (sb, sh)
        if not ok:
            a = append_args(capi, weights=FAKE, weights_stride_b=sb, weights_stride_h=sh)
            assert calls(capi, cache_args(capi), s, f=f, a=a)[0]() == 1 and calls(capi, cache_args(capi), s, f=f, a=a)[1]() == 1


def test_scores_are_part_of_the_workspace_only_with_weights(capi):
    L, r = capi.lib(), ctypes.byref
    c, s = cache_args(capi), seq_args(capi)
    plain = L.attn_cache_fwd_workspace_size(r(c), r(s), r(fwd_args(capi)))
    with_w = L.attn_cache_fwd_workspace_size(r(c), r(s), r(fwd_args(capi, weights=FAKE, weights_out=FAKE, weights_stride_b=512,
                                                                               weights_stride_h=256)))
    assert with_w - plain == 4 * 2 * 4 * 1 * 4 * 64  # 4 * B * Hq * Sq * max_pages * page_size


def test_nothing_to_do(capi):
    n = capi.lib().attn_launch_counter()
    fwd, app, ev, size = calls(capi, cache_args(capi), seq_args(capi, B=0, table=None, lengths=None))
    assert (fwd(), app(), ev(), size()) == (0, 0, 0, 256)
    assert calls(capi, cache_args(capi), seq_args(capi), f=fwd_args(capi, Sq=0, q=None))[0]() == 0
    assert capi.lib().attn_launch_counter() == n


# ---------------------------------------------------------------- binding

def tensors(P=4, H=2, page=64, D=128, dtype=torch.float8_e4m3fn):
    k = torch.zeros((P, H, page, D), dtype=torch.uint8).view(dtype)
    return k, k.clone(), torch.ones(P, H), torch.ones(P, H)


def test_the_handle_checks_its_tensors():
    k, v, ks, vs = tensors()
    with pytest.raises(ValueError, match="CUDA"):
        fa.AttnCache(k, v, ks, vs)
    with pytest.raises(TypeError, match="dtype"):
        fa.AttnCache(k.float(), v.float(), ks, vs)
    with pytest.raises(TypeError, match="dtype"):
        fa.AttnCache(k, v.view(torch.int8), ks, vs)
    with pytest.raises(ValueError, match="both"):
        fa.AttnCache(k, v[:2], ks, vs)
    with pytest.raises(ValueError, match="k_scale"):
        fa.AttnCache(k, v, ks[:, :1], vs)
    with pytest.raises(ValueError, match="v_scale"):
        fa.AttnCache(k, v, ks, vs.double())
    with pytest.raises(ValueError, match="page_size"):
        fa.AttnCache(*tensors(page=48))
    with pytest.raises(ValueError, match="multiple of 16"):
        fa.AttnCache(*tensors(D=72))
    with pytest.raises(ValueError, match="contiguous"):
        fa.AttnCache(k.transpose(0, 1), v.transpose(0, 1), ks, vs)
    with pytest.raises(TypeError, match="dtype"):
        fa.AttnCache.empty(4, 64, 2, 128, dtype=torch.bfloat16, device="cpu")


class HostCache(fa.AttnCache):
    """A handle over host tensors, for the checks that come before any launch."""

    def __init__(self):
        from attention_flash_attn_gb300._capi import AttnCacheArgs
        self.k, self.v, self.k_scale, self.v_scale = tensors()
        self.num_pages, self.Hkv, self.page_size, self.D, self.device = 4, 2, 64, 128, torch.device("cpu")
        self.status = torch.zeros(256, dtype=torch.uint8)
        self._c = AttnCacheArgs(1, 4, 64, 2, 128, FAKE, FAKE, FAKE, FAKE, FAKE)
        self._addr = ctypes.addressof(self._c)


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_attention_arguments_of_the_binding():
    c = HostCache()
    q = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16)
    table, lengths = torch.zeros(2, 2, dtype=torch.int32), ints(1, 2)
    go = lambda q=q, table=table, lengths=lengths, **kw: fa.attn_cache_path_name(q, c, table, lengths, **kw)
    assert go() in ("simt", "mma")
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        go(q=q.half())
    with pytest.raises(ValueError, match="D = 128"):
        go(q=q[..., :64])
    with pytest.raises(ValueError, match="contiguous"):
        go(q=torch.zeros(2, 1, 128, 128, dtype=torch.bfloat16).transpose(2, 3))
    with pytest.raises(ValueError, match="multiple of the cache's"):
        go(q=q[:, :, :3])
    with pytest.raises(ValueError, match="table"):
        go(table=table.long())
    with pytest.raises(ValueError, match="table"):
        go(table=table[:1])
    with pytest.raises(ValueError, match="overlap"):
        go(table=torch.zeros(3, dtype=torch.int32).as_strided((2, 2), (1, 1)))
    with pytest.raises(ValueError, match="lengths"):
        go(lengths=lengths.long())
    with pytest.raises(ValueError, match="lengths"):
        go(lengths=ints(1, 2, 3))
    with pytest.raises(ValueError, match="sink"):
        go(sink=torch.zeros(2))
    with pytest.raises(ValueError, match="sink"):
        go(sink=torch.zeros(4, dtype=torch.bfloat16))
    w = torch.zeros(2, 2, 128)
    assert go(weights=w)
    with pytest.raises(ValueError, match="weights"):
        go(weights=w[:, :, :127])
    with pytest.raises(ValueError, match="weights"):
        go(weights=w.double())
    with pytest.raises(ValueError, match="needs weights"):
        go(weights_out=w)
    with pytest.raises(ValueError, match="strides"):
        go(weights=w, weights_out=torch.zeros(2, 2, 130)[:, :, :128])
    for bad in (torch.zeros(1, 2, 128).expand(2, 2, 128), torch.zeros(2, 1, 128).expand(2, 2, 128),
                torch.zeros(500).as_strided((2, 2, 128), (200, 100, 1)), torch.zeros(500).as_strided((2, 2, 128), (130, 130, 1))):
        with pytest.raises(ValueError, match="weights.* must not overlap"):
            go(weights=bad)
    for good in (torch.zeros(2, 2, 128).transpose(0, 1), torch.zeros(600).as_strided((2, 2, 128), (128, 300, 1))):
        assert go(weights=good)
    for kw, what in ((dict(out=torch.zeros(2, 1, 4, 128)), "out"), (dict(lse=torch.zeros(2, 4)), "lse")):
        with pytest.raises(ValueError, match=what):
            fa.attn_cache_fwd(q, c, table, lengths, **kw)


def test_append_arguments_of_the_binding():
    c = HostCache()
    k = torch.zeros(2, 3, 2, 128)
    table, lengths = torch.zeros(2, 2, dtype=torch.int32), ints(1, 2)
    with pytest.raises(ValueError, match="heads"):
        fa.attn_cache_append(c, k[:, :, :1], k[:, :, :1], table, lengths)
    with pytest.raises(ValueError, match="v must be"):
        fa.attn_cache_append(c, k, k[:, :2], table, lengths)
    with pytest.raises(TypeError, match="share a dtype"):
        fa.attn_cache_append(c, k, k.bfloat16(), table, lengths)
    with pytest.raises(ValueError, match="counts"):
        fa.attn_cache_append(c, k, k, table, lengths, counts=ints(1))
    with pytest.raises(ValueError, match="counts"):
        fa.attn_cache_append(c, k, k, table, lengths, counts=torch.tensor([1, 1]))
    with pytest.raises(ValueError, match="weights"):
        fa.attn_cache_append(c, k, k, table, lengths, weights=torch.zeros(2, 2, 64))
    with pytest.raises(ValueError, match="must not overlap"):
        fa.attn_cache_append(c, k, k, table, lengths, weights=torch.zeros(1, 2, 128).expand(2, 2, 128))


def test_eviction_arguments_of_the_binding():
    c = HostCache()
    table, lengths, w = torch.zeros(2, 2, dtype=torch.int32), ints(1, 2), torch.zeros(2, 2, 128)
    out = torch.zeros(2, 1, dtype=torch.int32)
    go = lambda w=w, out=out, **kw: fa.attn_cache_evict(c, table, lengths, w, out, **{"keep": 64, **kw})
    for kw in (dict(keep=0), dict(recent=-1), dict(first=-1), dict(recent=60, first=5)):
        with pytest.raises(ValueError, match="keep"):
            go(**kw)
    with pytest.raises(ValueError, match="weights"):
        go(w=w[:, :1])
    with pytest.raises(ValueError, match="table_out"):
        go(keep=65)
    with pytest.raises(ValueError, match="table_out"):
        go(out=out.long())
    with pytest.raises(ValueError, match="kept"):
        go(kept=torch.zeros(2, 2, 63, dtype=torch.int32))
    with pytest.raises(ValueError, match="weights_out"):
        go(weights_out=torch.zeros(2, 2, 64, dtype=torch.float64))


# ---------------------------------------------------------------- shares of work

def test_every_unit_has_one_owner_and_every_split_item_its_parts():
    """U units over C CTAs: U // C each and one more for the first U % C.  The join finds an item's CTAs by the inverse, and a
    CTA's second partial by where the item begins.  Here the same arithmetic, against a walk over the shares."""
    rng = random.Random(3)
    for _ in range(400):
        items = [rng.choice([0, 0, 1, 2, 3, 17, rng.randint(0, 200)]) for _ in range(rng.randint(1, 40))]
        U, most = sum(items), rng.choice([1, 2, 5, 152, 456])
        C = min(U, most)
        if U == 0:
            continue
        each, extra = divmod(U, C)
        begin = [c * each + min(c, extra) for c in range(C + 1)]
        big = extra * (each + 1)
        owner = lambda u: u // (each + 1) if u < big else extra + (u - big) // each  # noqa: E731
        assert begin[C] == U and all(begin[owner(u)] <= u < begin[owner(u) + 1] for u in range(U))
        parts, slots = {}, set()
        for c in range(C):
            assert begin[c] < begin[c + 1]
            u, first, it = begin[c], 0, 0
            while u < begin[c + 1]:
                while u >= first + items[it]:
                    first += items[it]
                    it += 1
                cnt = min(items[it] - (u - first), begin[c + 1] - u)
                if cnt < items[it]:
                    slot = 2 * c + (1 if first > begin[c] else 0)
                    assert slot not in slots
                    slots.add(slot)
                    parts.setdefault(it, []).append(slot)
                u += cnt
        first = 0
        for it, n in enumerate(items):
            if n:
                c0, c1 = owner(first), owner(first + n - 1)
                want = [] if c0 == c1 else [2 * c + (1 if c == c0 and first > begin[c0] else 0) for c in range(c0, c1 + 1)]
                assert parts.get(it, []) == want
            first += n
