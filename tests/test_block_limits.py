"""Sizes at the limits of the block operators' C ABI, on the host: refused before anything is launched."""

import pytest

from bit_weight_only_awq_gb300 import build as awq_build

EINVAL = -1
FAKE = 1 << 40  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    awq_build.build()
    from bit_weight_only_awq_gb300 import awq
    return awq.lib


def test_query_rows_are_counted_in_32_bits(lib):
    """Query rows of a cache head: min(T, max_q) * heads / kv_heads is at most 2^30."""
    def call(T, max_q, heads, kv_heads):
        return lib.kv4_attention(FAKE, heads * 64, FAKE, FAKE, 64, FAKE, FAKE, FAKE, None, T, 1, max_q, heads, kv_heads, 64,
                                 100, 64, 64, 0.1, 0, 0, None, 0, None)

    for args in ((2 ** 31 - 1, 2 ** 31 - 1, 1, 1), (2 ** 27 + 1, 2 ** 31 - 1, 8, 1), (2 ** 31 - 1, 2 ** 20 + 1, 1024, 1)):
        assert call(*args) == EINVAL, args
        assert lib.kv4_attention_workspace_bytes(args[0], 1, args[1], args[2], args[3], 64) == 0
    for args in ((2 ** 30, 2 ** 31 - 1, 8, 8), (2 ** 27, 2 ** 31 - 1, 8, 1), (2 ** 31 - 1, 2 ** 20, 1024, 1), (5, 2 ** 31 - 1, 32, 8)):
        assert call(*args) != EINVAL, args
