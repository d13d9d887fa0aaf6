"""Accumulated weights where windows and causality leave most keys, most queries or whole blocks of keys unseen."""
import pytest
import torch

from cache_ref import E4M3, INT8
from test_cache_gpu import BF16, F32, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,kind", [(BF16, 64, E4M3), (BF16, 128, INT8), (F32, 64, E4M3), (BF16, 320, INT8)])
@pytest.mark.parametrize("lengths,Sq,Hq,kw", [([9000, 4096, 513, 512, 0, 1], 1, 6, dict(window=700)), ([5000, 511], 1, 8, dict(causal=True, window=1)),
                                              ([3000, 700, 30], 300, 2, dict(causal=True, window=65)), ([3000, 40], 50, 4, dict(window=513)),
                                              ([2000, 1999], 1200, 2, dict(causal=True)), ([1025, 600], 64, 40, dict(causal=True, window=512))])
def test_weights_of_keys_that_few_queries_see(dtype, D, kind, lengths, Sq, Hq, kw):
    """Out of place, where unseen keys keep their weights, and in place; and the same bits from both."""
    c = Case(lengths, Sq=Sq, Hq=Hq, Hkv=2, D=D, kind=kind, dtype=dtype, seed=Sq)
    w, out = c.cuda["w"], torch.full_like(c.cuda["w"], -5.0)
    O, LSE = c.run(sink=c.cuda["sink"], weights=w, weights_out=out, **kw)
    c.check(O, LSE, out, sink=True, **kw)
    for b, n in enumerate(lengths):
        assert (out[b, :, n:] == -5.0).all()
        first = n - Sq - kw.get("window", n) + 1        # keys before it are behind every query's window
        if first > 0:
            assert torch.equal(out[b, :, :first].cpu(), c.w[b, :, :first])
    assert torch.equal(w.cpu(), c.w)
    c.run(sink=c.cuda["sink"], weights=w, **kw)
    for b, n in enumerate(lengths):
        assert torch.equal(w[b, :, :n], out[b, :, :n]) and torch.equal(w[b, :, n:].cpu(), c.w[b, :, n:])
