"""Steps of the 8-bit cache whose positions and padding are advanced in place
between calls without a gap: each call sees what was there when it was made."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_attention_gb300.build import build
    build()
    import transformer_attention_gb300 as G3
    G3.lib()


@pytest.mark.parametrize("T,d_h,window", [(1, 128, 0), (2, 256, 40), (1, 256, 40), (20, 128, 40), (20, 256, 0)])
def test_positions_advanced_in_place(T, d_h, window):
    import transformer_attention_gb300 as G3
    B, S, H, H_kv, steps = 3, 1500, 8, 4, 30
    kvd = H_kv * d_h
    g = torch.Generator(device="cuda").manual_seed(T + d_h)
    rows = torch.randn((steps, B * T, 2 * kvd), generator=g, device="cuda").half()
    Q = (torch.randn((steps, B, T, H, d_h), generator=g, device="cuda") / 16).half()
    pads = torch.randint(0, T, (steps, B), generator=g, device="cuda", dtype=torch.int32)
    n = G3.gemma3_cached8_attention_workspace_size(B, T, S, H, H_kv, d_h, True)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")

    def run(sync):
        cache = G3.new_kv_cache8(B, S, H_kv, d_h, "cuda")
        w = torch.zeros((B, S), device="cuda")
        seg = torch.arange(T, device="cuda", dtype=torch.int32).repeat(B, 1)
        pad = torch.zeros(B, device="cuda", dtype=torch.int32)
        outs = [torch.empty((B, T, H, d_h), dtype=torch.float16, device="cuda") for _ in range(steps)]
        torch.cuda.synchronize()
        for i in range(steps):
            pad.copy_(pads[i])
            if sync:
                torch.cuda.synchronize()
            G3.gemma3_kv_cache8_write(rows[i], rows[i][:, kvd:], 2 * kvd, seg, pad, B, T, S, i * T, H_kv,
                                      d_h, *cache)
            G3.gemma3_cached8_attention(Q[i], *cache, seg, pad, outs[i], G3.GEMMA3_F16, w, B, T, S, i * T, H,
                                        H_kv, d_h, window, ws, ws.numel())
            if sync:
                torch.cuda.synchronize()
            seg += T
        torch.cuda.synchronize()
        return outs + [w, cache[4]] + [t.view(torch.uint8) for t in cache[:4]]

    want = run(True)
    assert int(want[steps + 1].max()) == steps * T - 1 - int(pads[-1].min())
    for _ in range(5):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
    assert G3.gemma3_attn_check_status() == 0
