"""The workspace of attention over the paged cache: a portion of work leaves two parts at most, however many
sequences there are (no GPU needed)."""
import itertools

import pytest


def _workspace(*sizes):
    import quantized_weight_gemv_amd as q
    return q.lib().qattn_decode_workspace(*sizes)


@pytest.mark.parametrize("cache", [1, 2, 3])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_it_does_not_grow_with_the_sequences(cache, dim):
    """Work is cut for 4 workgroups a compute unit at most, over the key heads and groups of rows; each has up to 32
    rows of dim accumulators, a maximum and a sum in two parts.  Beyond that only what 16 tokens of 1024 heads have."""
    most = 2 * max(4 * 256 * 32, 16 * 1024) * (dim + 2) * 4
    for B, M, kv, share, places in itertools.product((1, 2, 63, 512, 65536), (1, 5, 16), (1, 8, 48, 1024), (1, 4, 16),
                                                     (64, 4096, 1 << 17, 1 << 20)):
        if kv * share > 1024 or B * M * kv * share > 1 << 23 or B * places > 1 << 36:
            continue
        assert _workspace(B, M, kv * share, kv, dim, cache, 64, places // 64) <= most, (B, M, kv, share, places)


def test_it_does_not_grow_with_the_sequences_that_a_table_of_any_width_has():
    few, many = (_workspace(B, 1, 32, 8, 128, 3, 64, 4096) for B in (128, 65536))
    assert 0 < few == many
