"""Which kernel a batch of many rows at small head dims takes, and that both give float64's results where the choice changes."""
import pytest

from cache_ref import E4M3, INT8
from test_cache_gpu import Case, fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("D,B,Hkv,G,Sq,path", [(64, 16, 8, 4, 24, "tc"), (64, 16, 8, 4, 16, "mma"), (48, 13, 8, 8, 9, "tc"), (64, 12, 8, 8, 9, "mma"),
                                               (64, 64, 1, 5, 28, "tc"), (64, 1, 8, 4, 64, "mma"), (32, 40, 4, 13, 5, "tc")])
def test_batches_at_small_head_dims(D, B, Hkv, G, Sq, path, kind):
    """Tiles of 32 rows in one wave of two CTAs to an SM, and more than that."""
    c = Case([300, 0, 7, 129] + [Sq + 64 * (b % 3) for b in range(4, B)] if B > 4 else [300], Sq=Sq, Hq=G * Hkv, Hkv=Hkv, D=D, page=32, kind=kind)
    t = c.cuda
    assert fa().attn_cache_path_name(t["q"], c.cache, t["table"], t["lengths"]) == path
    w = t["w"].clone()
    O, LSE = c.run(causal=True, softcap=20.0, sink=t["sink"], weights=w)
    c.check(O, LSE, w, causal=True, softcap=20.0, sink=True, rows=list(range(min(B, 6))))
    assert fa().attn_cache_check_device_status(c.cache) == 0
