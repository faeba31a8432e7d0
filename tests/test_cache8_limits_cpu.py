"""The 8-bit KV cache at the ends of its argument ranges, without a GPU: what is
refused before anything reaches a device."""
import pytest
import torch

import transformer_attention_gb300 as G3
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


def _cache(B=2, S=100, H_kv=2, d_h=128):
    return list(G3.new_kv_cache8(B, S, H_kv, d_h, "cpu")), torch.zeros(B, S)


def test_evict_into_a_cache_of_other_sizes():
    """A cache that does not fit the one it is filled from, or is no plain
    layout, is refused by shape."""
    cache, w = _cache()
    for into in (_cache(B=1), _cache(H_kv=1), _cache(d_h=256)):
        with pytest.raises(ValueError, match="K8"):
            G3.evict_kv_cache8(cache, w, 90, 40, 8, into=into)
    dst, w_dst = _cache(S=64)
    with pytest.raises(ValueError, match="weight_sum"):
        G3.evict_kv_cache8(cache, w, 90, 40, 8, into=(dst, w_dst[:, :50]))
    with pytest.raises(ValueError, match="weight_sum"):
        G3.evict_kv_cache8(cache, w.double(), 90, 40, 8, into=(dst, w_dst))
    wide, _ = _cache(S=128)
    wide[0] = wide[0][:, :64]
    wide[1] = wide[1][:, :64]
    wide[4] = wide[4][:, :64].contiguous()
    wide[2] = wide[3] = torch.zeros(2, 1, 2)
    with pytest.raises(ValueError, match="contiguous"):
        G3.evict_kv_cache8(cache, w, 90, 40, 8, into=(wide, torch.zeros(2, 64)))
    short, _ = _cache()
    short[2] = short[2][:, :1].contiguous()
    with pytest.raises(ValueError, match="K_scale"):
        G3.evict_kv_cache8(short, w, 90, 40, 8, into=(dst, w_dst))


def test_layer_with_another_cache():
    x = torch.zeros(2, 3, 256, dtype=torch.bfloat16)
    seg = torch.zeros(2, 3, dtype=torch.int32)
    gamma = torch.zeros(128, dtype=torch.bfloat16)
    kw = dict(H=4, H_kv=2, attn_type=0, window=0, rope_base=1e4, rope_scale=1.0, query_scale=1.0)
    for cache, w in (_cache(B=1), _cache(H_kv=4), _cache(d_h=256)):
        with pytest.raises(ValueError, match="K8"):
            G3.attention_forward_cached8(x, seg, None, cache, 0, x, x, x, gamma, gamma, **kw)
    cache, w = _cache()
    with pytest.raises(ValueError, match="weight_sum"):
        G3.attention_forward_cached8(x, seg, None, cache, 0, x, x, x, gamma, gamma, weight_sum=w[:1], **kw)
    cache[0] = cache[0].view(torch.int8)
    with pytest.raises(ValueError, match="K8"):
        G3.attention_forward_cached8(x, seg, None, cache, 0, x, x, x, gamma, gamma, **kw)


def test_a_tensor_that_is_not_on_the_gpu(monkeypatch):
    """The wrappers take addresses: a tensor elsewhere is refused."""
    monkeypatch.setattr(L, "_device", lambda: 0)
    t = torch.zeros(4)
    with pytest.raises(ValueError, match="current GPU"):
        L.gemma3_kv_cache8_read(P, P, P, t, 1, 64, 0, 1, 2, 128, P, P, 256, 0)
    with pytest.raises(ValueError, match="current GPU"):
        L.gemma3_kv_cache8_evict(P, P, P, P, P, t, 1, 64, 1, 2, 128, 1, 0, P, P, P, P, P, P, P, 64, 0)
