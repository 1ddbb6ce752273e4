"""The limit of attention's waits, which has to outlast the longest of them."""
import pytest

from fp4_gemm_nvfp4_gb300 import build as libbuild
from fp4_gemm_nvfp4_gb300 import capi


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return capi.load()


@pytest.mark.parametrize("tokens", [1, 8192, 10_000_000, 2 ** 31 - 257])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (24, 12), (24, 1), (128, 2)])
def test_a_wait_outlasts_the_longest_item(tokens, q_heads, kv_heads):
    """A wait can last as long as an item: one tile per 128 tokens, in the
    backward pass for every query head of a group, 1.5 us each (measured: 0.5 to
    1.5 us for a tile of 128 dims)."""
    tiles = (tokens + 127) // 128
    for backward, item in ((0, tiles), (1, tiles * (q_heads // kv_heads))):
        limit = capi.nvfp4_testing_attention_wait_limit_us(backward, tokens, q_heads, kv_heads)
        assert limit >= 2_000_000 and limit >= 3 * 1.5 * item


def test_no_limit_for_a_refused_shape():
    for tokens, q_heads, kv_heads in ((-1, 1, 1), (2 ** 31, 1, 1), (1, 0, 1), (1, 1, 0)):
        assert capi.nvfp4_testing_attention_wait_limit_us(1, tokens, q_heads, kv_heads) == 0
