"""The wrappers that allocate, called with a stream other than the current
one: what they allocate and fill belongs to the stream that they launch on."""
import pytest
import torch

from tests import test_gpu_cache8 as C
from transformer_attention_gb300 import workloads as WL

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


def _layer():
    w = WL.small(WL.WORKLOADS["tiny_local"], name="streams", B=2, T=64, D=256, H=4, H_kv=2, d_h=256,
                 attn_type="local", window=24)
    p = {k: v.cuda() for k, v in WL.weights(w).items()}
    x = WL.x_full(w).cuda()
    seg = torch.arange(w.T, dtype=torch.int32, device="cuda").repeat(w.B, 1)
    args = [p[k] for k in ("Wq", "Wkv", "Wo", "gamma_q", "gamma_k")]
    kw = dict(H=w.H, H_kv=w.H_kv, window=w.window, rope_base=w.rope_base, rope_scale=w.rope_scale,
              query_scale=w.query_scale)
    return w, x, seg, args, kw


def _call(G3, name, stream):
    w, x, seg, args, kw = _layer()
    kw["attn_type"] = G3.GEMMA3_LOCAL_SLIDING
    weight = None
    if name == "attention_forward_cached8":
        cache = G3.new_kv_cache8(w.B, 80, w.H_kv, w.d_h, "cuda")
        weight = torch.zeros((w.B, 80), device="cuda")
        run = lambda: G3.attention_forward_cached8(  # noqa: E731
            x, seg, None, cache, 0, *args, weight_sum=weight, stream=stream, **kw)
    elif name == "attention_forward_cached":
        cache = G3.new_kv_cache(w.B, 80, w.H_kv, w.d_h, "cuda")
        run = lambda: G3.attention_forward_cached(x, seg, None, cache, 0, *args, stream=stream, **kw)  # noqa: E731
    elif name == "attention_forward":
        run = lambda: G3.attention_forward(x, seg, None, *args, stream=stream, **kw)  # noqa: E731
    else:
        g = torch.zeros(w.D, dtype=torch.bfloat16, device="cuda")
        wg = torch.full((2, 128, w.D), 0.01, dtype=torch.bfloat16, device="cuda")
        wd = torch.full((w.D, 128), 0.01, dtype=torch.bfloat16, device="cuda")
        if name == "block_forward":
            run = lambda: G3.block_forward(x, seg, None, *args, g, g, g, g, wg, wd, stream=stream, **kw)  # noqa: E731
        else:
            run = lambda: G3.block_attention_forward(x, seg, None, *args, g, g, stream=stream, **kw)  # noqa: E731
    torch.cuda.synchronize()
    return run(), weight


@pytest.mark.parametrize("name", ["attention_forward_cached8", "attention_forward_cached", "attention_forward",
                                  "block_attention_forward", "block_forward"])
def test_workspace_of_another_stream(name, monkeypatch):
    """A workspace made for a call on another stream is not handed out again on
    the current one, which does not wait for that call."""
    import transformer_attention_gb300 as G3
    want, w_want = _call(G3, name, None)
    made = []
    real = G3._empty_ws

    def empty_ws(nbytes, device):
        t = real(nbytes, device)
        made.append((t.data_ptr(), t.numel()))
        return t

    monkeypatch.setattr(G3, "_empty_ws", empty_ws)
    side = torch.cuda.Stream()
    got, w_got = _call(G3, name, side)
    (at, n), = made
    again = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert G3.gemma3_attn_check_status() == 0
    assert torch.equal(got, want)
    assert w_want is None or torch.equal(w_got, w_want)
    assert all(not (t.data_ptr() < at + n and at < t.data_ptr() + n) for t in again)
