"""The 8-bit KV cache at the ends of its argument ranges, without a GPU: what is
refused before anything reaches a device."""
import pytest

from transformer_attention_gb300 import _lib as L
from transformer_attention_gb300.build import build

P = 1 << 20            # stands for a device pointer; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build()
    return L.lib()


def test_more_blocks_than_a_launch_has_ctas(lib):
    """65535 rows of 65535 kv heads fit the byte limit at S = 1, but are 2^33
    (block, head, K' or V) units."""
    big = 65535
    assert lib.gemma3_kv_cache8_write(P, P, big * 128, P, None, big, 1, 1, 0, big, 128, P, P, P, P, P,
                                      None) == -1
    assert lib.gemma3_kv_cache8_evict(1 << 44, 2 << 44, 3 << 44, 4 << 44, 5 << 44, 6 << 44, big, 1, 1,
                                      big, 128, 1, 0, 7 << 44, 8 << 44, 9 << 44, 10 << 44, 11 << 44,
                                      12 << 44, 13 << 44, 1, None) == -1
