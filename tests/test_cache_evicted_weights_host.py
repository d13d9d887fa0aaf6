"""Refusals of evicted weights' rows: those that overlap one another or the weights they come from.  No CUDA call is made here."""
import pytest
import torch

import attention_flash_attn_gb300 as fa
from test_cache_host import FAKE, HostCache, cache_args, calls, capi, evict_args, ints, seq_args  # noqa: F401


def test_rows_of_evicted_weights_of_the_c_call(capi):  # noqa: F811
    s = seq_args(capi)                      # 2 sequences of 4 pages of 64 tokens, 2 kv heads; weights [2, 2, 256] dense at FAKE
    far = FAKE + (1 << 20)
    n = capi.lib().attn_launch_counter()
    refused = lambda **kw: calls(capi, cache_args(capi), s, e=evict_args(capi, **kw))[2]() == 1  # noqa: E731
    for sb, sh in ((99, 200), (100, 100), (200, 0), (0, 100), (199, 100), (-400, 200), (100, 150)):
        assert refused(weights_out=far, weights_out_stride_b=sb, weights_out_stride_h=sh), (sb, sh)
    for at in (FAKE, FAKE + 4 * 1023, FAKE - 4):  # weights' first and last element, and a row that ends behind the first
        assert refused(weights_out=at, weights_out_stride_b=512, weights_out_stride_h=256), at
        assert refused(weights_out=at)
    assert capi.lib().attn_launch_counter() == n


def test_rows_of_evicted_weights_of_the_binding():
    c = HostCache()
    table, lengths, w = torch.zeros(2, 2, dtype=torch.int32), ints(1, 2), torch.zeros(2, 2, 128)
    go = lambda out: fa.attn_cache_evict(c, table, lengths, w, torch.zeros(2, 1, dtype=torch.int32), keep=64, weights_out=out)  # noqa: E731
    for bad in (torch.zeros(2, 2, 63), torch.zeros(2, 1, 64), torch.zeros(2, 2, 64, dtype=torch.float64), torch.zeros(2, 2, 128)[:, :, ::2],
                torch.zeros(1, 2, 64).expand(2, 2, 64), torch.zeros(400).as_strided((2, 2, 64), (64, 63, 1))):
        with pytest.raises(ValueError, match="weights_out"):
            go(bad)
    for good in (torch.zeros(2, 2, 64), torch.zeros(2, 2, 200), torch.zeros(2, 2, 200).transpose(0, 1), torch.zeros(2, 3, 80)[:, 1:, 5:]):
        with pytest.raises(ValueError, match="CUDA device"):  # (all that is wrong with it)
            go(good)
