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


@pytest.mark.parametrize("T,G,rows", [(1, 1, 16), (4, 4, 16), (16, 1, 16), (17, 1, 128), (32, 4, 128), (43, 3, 256),
                                      (256, 8, 256)])
@pytest.mark.parametrize("d", [64, 128])
def test_partial_results_have_the_rows_of_an_item(T, G, rows, d):
    """Scratch of a call without weights: two partial results for each of 148 CTAs, of 16, 128 or 256 query rows of
    d + 2 numbers, the lengths' sums, and at most 256 bytes of padding for each of the three."""
    b = 3
    need = hs.hisa_tree_attn_workspace_size(_p(batch=b, n_q=T, n_kv=4096, n_heads=2 * G, n_kv_heads=2, d_head=d))
    least = 148 * 2 * rows * (d + 2) * 4 + 8 * (b + 2)
    assert least <= need <= least + 3 * 256


@pytest.mark.parametrize("T,G,kept", [(1, 1, True), (8, 1, True), (2, 4, True), (9, 1, False), (4, 4, False)])
def test_scratch_of_a_call_with_weights(T, G, kept):
    """Up to 8 query rows a KV head the scores are kept: 4 bytes a query row and key tile row; above, a sum a key and
    head group at most."""
    b, n_kv, Hk = 3, 4000, 2
    p = _p(batch=b, n_q=T, n_kv=n_kv, n_heads=Hk * G, n_kv_heads=Hk, d_head=64)
    more = hs.hisa_tree_attn_workspace_size(p, True) - hs.hisa_tree_attn_workspace_size(p, False)
    scores = 4 * b * T * Hk * G * 4096
    assert (scores <= more <= scores + 4 * b * T * Hk * G + 512) == kept
    assert kept or more <= 4 * b * n_kv * Hk + 4 * b * T * Hk * G + 512
