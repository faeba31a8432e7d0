"""The 8-bit cache after an error that another call recorded (a bad token id),
before anybody has read it: calls whose own work is not lost give what they
always give."""
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
