"""The cache operators without a GPU: arguments at the ends of their ranges."""
import pytest
import torch

import hierarchical_sparse_attention_block_b200 as hs
from test_cache_cpu import _OnGpu, _p


@pytest.mark.parametrize("first,recent", [(1 << 32, 0), (0, 1 << 32), ((1 << 32) + 4, 8), (-(1 << 32), 0), (-1, 0)])
def test_counts_beyond_32_bits_are_refused(first, recent):
    """The library takes 32 bits: what they would lose is refused, not cut off."""
    i32 = torch.int32
    with pytest.raises(hs.HisaError) as err:
        hs.hisa_cache_keep(_p(), _OnGpu((2, 512), torch.float32), _OnGpu((2,), i32), 64, _OnGpu((2, 64), i32),
                           _OnGpu((2,), i32), first, recent, workspace=_OnGpu((16,), torch.uint8))
    assert err.value.status == hs.HISA_ERR_INVALID_ARG and "n_first" in str(err.value)


@pytest.mark.parametrize("n", [513, (1 << 32) + 5])
def test_lists_longer_than_the_cache_are_refused(n):
    with pytest.raises(hs.HisaError) as err:
        hs.hisa_cache_compact(_p(), _OnGpu((2, n), torch.int32), [_OnGpu((2, 512, 4), torch.float32)])
    assert err.value.status == hs.HISA_ERR_INVALID_ARG and "n <= n_kv" in str(err.value)
