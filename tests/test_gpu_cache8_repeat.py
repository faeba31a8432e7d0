"""Calls of the 8-bit cache attention that follow one another without a gap, as
a model's layers do: every one gives the same bits as a call on its own."""
import pytest
import torch

from tests import test_gpu_cache8 as C

pytestmark = pytest.mark.gpu

CASES = [
    # B, T, S, end, H, H_kv, d_h, window
    (2, 1024, 4096, 2000, 32, 16, 128, 0),     # whole query tiles and cut ones
    (1, 1024, 9000, 7900, 32, 16, 128, 0),     # all cut
    (1, 2432, 9000, 6500, 8, 4, 256, 0),       # one round of whole ones
    (2, 515, 4096, 3001, 16, 8, 256, 1024),
    (1, 100, 30000, 29000, 8, 8, 128, 0),      # one query tile per kv head
    (1, 1, 60000, 59990, 16, 8, 128, 0),       # few rows: splits and a merge
    (3, 4, 20000, 19000, 8, 2, 256, 0),
    (4, 2, 9000, 8000, 8, 4, 256, 512),        # a cluster's
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "B{}T{}S{}e{}H{}/{}d{}W{}".format(*c))
def test_calls_back_to_back(case):
    import transformer_attention_gb300 as G3
    B, T, S, end, H, H_kv, d_h, W = case
    g = torch.Generator(device="cuda").manual_seed(S + T)
    cache = G3.new_kv_cache8(B, S, H_kv, d_h, "cuda")
    for t in cache[:2]:
        t.view(torch.uint8).copy_((torch.randn(t.shape, generator=g, device="cuda") * 60)
                                  .to(torch.float8_e4m3fn).view(torch.uint8))
    for t in cache[2:4]:
        t.copy_(2.0 ** torch.randint(-8, -5, t.shape, generator=g, device="cuda"))
    cache[4][:, :end + T] = torch.arange(end + T, device="cuda", dtype=torch.int32)
    seg = torch.arange(end, end + T, device="cuda", dtype=torch.int32).repeat(B, 1)
    Q = (torch.randn((B, T, H, d_h), generator=g, device="cuda") / 8).half()
    n = G3.gemma3_cached8_attention_workspace_size(B, T, S, H, H_kv, d_h, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(O, w):
        G3.gemma3_cached8_attention(Q, *cache, seg, None, O, G3.GEMMA3_BF16, w, B, T, S, end, H, H_kv,
                                    d_h, W, ws, n)

    def outputs():
        return torch.empty_like(Q, dtype=torch.bfloat16), torch.zeros((B, S), device="cuda")

    want = outputs()
    torch.cuda.synchronize()
    call(*want)
    torch.cuda.synchronize()
    outs = [outputs() for _ in range(8)]
    torch.cuda.synchronize()
    for o in outs:
        call(*o)
    torch.cuda.synchronize()
    assert G3.gemma3_attn_check_status() == 0
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
    # without weights, where the attention's launches follow one another alone
    for o in outs:
        call(o[0], None)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0])
    assert G3.gemma3_attn_check_status() == 0
