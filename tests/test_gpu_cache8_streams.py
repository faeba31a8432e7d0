"""The wrappers that allocate, called with a stream other than the current
one: what they allocate and fill belongs to the stream that they launch on."""
import pytest
import torch

from tests import test_gpu_cache8 as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_attention_gb300.build import build
    build()
    import transformer_attention_gb300 as G3
    G3.lib()


def _bits(result):
    cache, w, kept = result
    return [t.view(torch.uint8) for t in (*cache, w, kept)]


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_evict_on_another_stream(handle):
    """The current stream is busy when the eviction runs on another one: the
    new cache's fills do not land on what was moved into it."""
    import transformer_attention_gb300 as G3
    B, S, end, keep = 2, 300, 290, 100
    src = C._to_dev(C._random_cache(B, S, 2, 128, 5))
    w = torch.rand((B, S), generator=C._gen(6)).cuda()
    want = G3.evict_kv_cache8(src, w, end, keep, 16, S=128)
    side = torch.cuda.Stream()
    spare = G3.evict_kv_cache8(src, w, end, keep, 16, S=128)   # its memory is reused
    del spare
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    got = G3.evict_kv_cache8(src, w, end, keep, 16, S=128,
                             stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert G3.gemma3_attn_check_status() == 0
    for a, b in zip(_bits(got), _bits(want)):
        assert torch.equal(a, b)


def test_evict_on_the_null_stream():
    import transformer_attention_gb300 as G3
    src = C._to_dev(C._random_cache(1, 200, 1, 256, 7))
    w = torch.rand((1, 200), generator=C._gen(8)).cuda()
    want = G3.evict_kv_cache8(src, w, 200, 70, 5)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        got = G3.evict_kv_cache8(src, w, 200, 70, 5, stream=0)
    torch.cuda.synchronize()
    for a, b in zip(_bits(got), _bits(want)):
        assert torch.equal(a, b)
