"""NaN values among the codes of long rows, whose keys are split over the grid: they reach the rows that see them, and no others."""
import pytest
import torch

from cache_ref import E4M3
from test_cache_gpu import BF16, F32, Case, fa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D,Sq", [(BF16, 64, 4), (BF16, 48, 4), (BF16, 64, 8), (BF16, 128, 4), (BF16, 256, 4), (F32, 64, 4)])
@pytest.mark.parametrize("window", [0, 20001])
def test_nan_in_long_rows_reaches_only_the_rows_that_see_them(dtype, D, Sq, window):
    """A NaN value near the end, and with a window one at the first key that only the first query sees."""
    n, G = 40000, 4
    c = Case([n], Sq=Sq, Hq=2 * G, Hkv=2, D=D, dtype=dtype)
    at = {n - 2: 3}                                     # position: column, of kv head 0
    if window:
        at[n - Sq - window + 1] = 17
    for pos, col in at.items():
        c.v.view(torch.uint8)[int(c.table[0, pos // 64]), 0, pos % 64, col] = 255
    c.cuda["v"].copy_(c.v)
    want = torch.zeros((Sq, 2 * G, D), dtype=torch.bool)
    for i in range(Sq):
        p = n - Sq + i
        for pos, col in at.items():
            if pos <= p and (not window or p - pos < window):
                want[i, :G, col] = True
    assert want.any() and not want.all(-1).any()
    for _ in range(20):
        O, LSE = c.run(causal=True, window=window)
        assert torch.equal(torch.isnan(O[0]).cpu(), want)
        assert torch.isfinite(LSE).all()
    assert fa().attn_cache_check_device_status(c.cache) == 0
