"""The 8-bit cache after an error that another call recorded (a bad token id),
before anybody has read it: calls whose own work is not lost give what they
always give, and where the projections stop, a layer leaves its cache and its
slot weights as they were."""
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


def _record_bad_token(G3):
    """A token id outside the vocabulary, which the kernel's own check records."""
    E = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
    x = torch.empty((1, 64), dtype=torch.float32, device="cuda")
    G3.gemma3_embed(torch.tensor([9], dtype=torch.int32, device="cuda"), E, 8, 64, 1, 1.0, x)
    torch.cuda.synchronize()


def _read_bad_token(G3):
    with pytest.raises(G3.Gemma3Error) as e:
        G3.gemma3_attn_check_status()
    assert e.value.status == G3.GEMMA3_ERR_BAD_INPUT


@pytest.mark.parametrize("T,window", [(1, 0), (3, 50), (200, 0), (200, 50), (40, 0)])
@pytest.mark.parametrize("d_h", [128, 256])
def test_attention_after_a_recorded_error(T, window, d_h):
    import transformer_attention_gb300 as G3
    B, S, end, H, H_kv = 2, 700, 450, 8, 4
    c, Q, seg = C._stage(B, T, S, end, H, H_kv, d_h, None, "plain", 3 + T)
    dev = C._to_dev(c)
    w0 = torch.rand((B, S), generator=C._gen(4))

    def call():
        w = w0.cuda()
        return C._attend(G3, Q, dev, seg, None, T, end, H, H_kv, d_h, window, torch.bfloat16, w), w

    want = call()
    assert G3.gemma3_attn_check_status() == 0
    _record_bad_token(G3)
    got = call()
    _read_bad_token(G3)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [1, 16, 64])
def test_layer_after_a_recorded_error(T):
    """Few tokens are unharmed.  Where the projections stop at a recorded
    error (T = 16 and 64: more than 16 rows), the tokens are not written, so
    that the block's scale and older numbers stay, and no weight is added; the
    call made again gives what it would have given."""
    import transformer_attention_gb300 as G3
    w = WL.small(WL.WORKLOADS["tiny_local"], name="errors", B=2, T=128, D=256, H=4, H_kv=1, d_h=256,
                 attn_type="global", window=0)
    p = {k: v.cuda() for k, v in WL.weights(w).items()}
    x = WL.x_full(w).cuda()
    B, S, T0 = w.B, 200, 40
    n = G3.gemma3_attn_cached8_workspace_size((B, 64, w.D, w.H, w.H_kv, w.d_h), S, True)

    def layer(a, z, cache, weights):
        ws = torch.full((n,), 0x7B, dtype=torch.uint8, device="cuda")     # 61280 in fp16
        seg = torch.arange(a, z, dtype=torch.int32, device="cuda").repeat(B, 1)
        out = torch.full((B, z - a, w.D), 5.0, dtype=torch.bfloat16, device="cuda")
        return G3.attention_forward_cached8(
            x[:, a:z].contiguous(), seg, None, cache, a, p["Wq"], p["Wkv"], p["Wo"], p["gamma_q"],
            p["gamma_k"], H=w.H, H_kv=w.H_kv, attn_type=G3.GEMMA3_GLOBAL, window=0,
            rope_base=w.rope_base, rope_scale=w.rope_scale, query_scale=w.query_scale,
            weight_sum=weights, out=out, workspace=ws)

    def state():
        cache, weights = G3.new_kv_cache8(B, S, w.H_kv, w.d_h, "cuda"), torch.zeros((B, S), device="cuda")
        layer(0, T0, cache, weights)
        return cache, weights

    def bits(cache, weights):
        return [t.view(torch.uint8).clone() for t in (*cache, weights)]

    clean = state()
    want = layer(T0, T0 + T, *clean)
    assert G3.gemma3_attn_check_status() == 0
    mine = state()
    before = bits(*mine)
    _record_bad_token(G3)
    got = layer(T0, T0 + T, *mine)
    _read_bad_token(G3)
    if B * T > 16:
        for a, b in zip(bits(*mine), before):
            assert torch.equal(a, b)
        got = layer(T0, T0 + T, *mine)
        assert G3.gemma3_attn_check_status() == 0
    assert torch.equal(got, want)
    for a, b in zip(bits(*mine), bits(*clean)):
        assert torch.equal(a, b)
