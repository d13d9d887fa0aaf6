"""Strides of dimensions of size 1 say nothing: the binding does not compare them.  No CUDA call is made here."""
import pytest
import torch

import attention_flash_attn_gb300 as fa
from test_cache_host import HostCache, ints


def rows(shape, strides):
    return torch.zeros(4000).as_strided(shape, strides)


def test_weights_and_their_output_may_differ_in_the_stride_of_a_single_sequence():
    c = HostCache()                                                            # 2 kv heads
    go = lambda B, w, o: fa.attn_cache_path_name(torch.zeros(B, 1, 4, 128, dtype=torch.bfloat16), c, torch.zeros(B, 2, dtype=torch.int32),  # noqa: E731
                                                 ints(*range(B)), weights=w, weights_out=o)
    for sb in (0, 1, 256, 999):
        assert go(1, rows((1, 2, 128), (256, 128, 1)), rows((1, 2, 128), (sb, 128, 1)))
        assert go(1, rows((1, 2, 128), (sb, 128, 1)), rows((1, 2, 128), (256, 128, 1)))
    with pytest.raises(ValueError, match="strides"):
        go(1, rows((1, 2, 128), (256, 128, 1)), rows((1, 2, 128), (256, 130, 1)))
    with pytest.raises(ValueError, match="strides"):
        go(2, rows((2, 2, 128), (256, 128, 1)), rows((2, 2, 128), (260, 128, 1)))
