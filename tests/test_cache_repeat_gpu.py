"""Equal calls of attention over the 8-bit cache give equal bits, for the forms whose ring of codes is refilled while stores of
scores are queued in the same unit: float queries, tiles of 32 rows, items in one cluster and items split over the grid."""
import pytest
import torch

from cache_ref import E4M3, INT8
from test_cache_gpu import BF16, F32, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [E4M3, INT8])
@pytest.mark.parametrize("lengths", [[1031, 0, 77, 500], [20011, 4000]])
@pytest.mark.parametrize("dtype,D,G,Sq", [(F32, 64, 8, 1), (F32, 128, 8, 1), (F32, 256, 8, 1), (F32, 96, 4, 4), (BF16, 64, 5, 5),
                                          (BF16, 128, 20, 1), (BF16, 112, 6, 5), (BF16, 256, 8, 4)])
def test_equal_calls_give_equal_bits(dtype, D, G, Sq, lengths, kind):
    c = Case(lengths, Sq=Sq, Hq=2 * G, Hkv=2, D=D, page=32, kind=kind, dtype=dtype, seed=D)
    one = None
    for _ in range(100):
        w = c.cuda["w"].clone()
        out = [*c.run(weights=w, softcap=20.0), w]
        one = one or out
        for a, b in zip(one, out):
            assert torch.equal(a, b)
    c.check(*one, softcap=20.0)
