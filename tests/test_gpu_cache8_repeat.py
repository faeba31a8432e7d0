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


@pytest.mark.parametrize("H,H_kv,d_h,T", [(32, 16, 128, 1), (16, 8, 256, 2), (16, 16, 128, 20)])
def test_steps_that_grow_scales(H, H_kv, d_h, T):
    """Write and attend in turn without a gap, every step with larger values in
    some heads, so that the block's scales of those grow: each step sees the
    scales that its own write left."""
    import transformer_attention_gb300 as G3
    B, S, steps = 6, 2000, 40
    g = torch.Generator(device="cuda").manual_seed(d_h + T)
    kvd = H_kv * d_h
    rows = (torch.randn((steps, B * T, 2, H_kv, d_h), generator=g, device="cuda") * 2.0 ** -6)
    grow = torch.rand((steps, 1, 2, H_kv, 1), generator=g, device="cuda") < 0.3
    rows *= 2.0 ** torch.cumsum(grow.float(), 0).clamp(max=18)
    rows = rows.half().view(steps, B * T, 2 * kvd)
    Q = (torch.randn((steps, B, T, H, d_h), generator=g, device="cuda") / 64).half()
    n = G3.gemma3_cached8_attention_workspace_size(B, T, S, H, H_kv, d_h, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    seg = [torch.arange(300 + i * T, 300 + (i + 1) * T, device="cuda", dtype=torch.int32).repeat(B, 1)
           for i in range(steps)]

    def run(sync):
        cache = G3.new_kv_cache8(B, S, H_kv, d_h, "cuda")
        cache[4][:, :300] = torch.arange(300, device="cuda", dtype=torch.int32)
        cache[2].fill_(2.0 ** -15)
        cache[3].fill_(2.0 ** -15)
        w = torch.zeros((B, S), device="cuda")
        outs = [torch.empty((B, T, H, d_h), dtype=torch.float16, device="cuda") for _ in range(steps)]
        torch.cuda.synchronize()
        for i in range(steps):
            end = 300 + i * T
            G3.gemma3_kv_cache8_write(rows[i], rows[i][:, kvd:], 2 * kvd, seg[i], None, B, T, S, end,
                                      H_kv, d_h, *cache)
            if sync:
                torch.cuda.synchronize()
            G3.gemma3_cached8_attention(Q[i], *cache, seg[i], None, outs[i], G3.GEMMA3_F16, w, B, T, S,
                                        end, H, H_kv, d_h, 0, ws, n)
            if sync:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs + [w] + list(cache[2:4])

    want = run(True)
    for _ in range(6):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
    assert G3.gemma3_attn_check_status() == 0


@pytest.mark.parametrize("T,d_h", [(1, 128), (3, 256), (200, 128), (200, 256)])
def test_two_inputs_in_turn(T, d_h):
    """Two inputs in turn through one workspace, without a gap."""
    import transformer_attention_gb300 as G3
    B, S, end, H, H_kv = 2, 9000, 8000, 16, 8
    g = torch.Generator(device="cuda").manual_seed(T)
    ins = []
    for _ in range(2):
        cache = G3.new_kv_cache8(B, S, H_kv, d_h, "cuda")
        for t in cache[:2]:
            t.view(torch.uint8).copy_((torch.randn(t.shape, generator=g, device="cuda") * 60)
                                      .to(torch.float8_e4m3fn).view(torch.uint8))
        for t in cache[2:4]:
            t.copy_(2.0 ** torch.randint(-8, -5, t.shape, generator=g, device="cuda"))
        cache[4][:, :end + T] = torch.arange(end + T, device="cuda", dtype=torch.int32)
        ins.append(((torch.randn((B, T, H, d_h), generator=g, device="cuda") / 8).half(), cache))
    seg = torch.arange(end, end + T, device="cuda", dtype=torch.int32).repeat(B, 1)
    n = G3.gemma3_cached8_attention_workspace_size(B, T, S, H, H_kv, d_h, True)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def call(i, O, w):
        G3.gemma3_cached8_attention(ins[i][0], *ins[i][1], seg, None, O, G3.GEMMA3_BF16, w, B, T, S, end,
                                    H, H_kv, d_h, 0, ws, n)

    def outputs():
        return (torch.empty((B, T, H, d_h), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((B, S), device="cuda"))

    want = [outputs(), outputs()]
    for i in (0, 1):
        torch.cuda.synchronize()
        call(i, *want[i])
    torch.cuda.synchronize()
    outs = [outputs() for _ in range(20)]
    torch.cuda.synchronize()
    for k, o in enumerate(outs):
        call(k % 2, *o)
    torch.cuda.synchronize()
    for k, o in enumerate(outs):
        assert torch.equal(o[0], want[k % 2][0]) and torch.equal(o[1], want[k % 2][1])
    assert G3.gemma3_attn_check_status() == 0


CUT = [
    (4, 256, 4300, 4000, 12, 12, 256, 0),      # 96 units: a large part each and small ones
    (4, 256, 4300, 4000, 24, 24, 256, 0),      # 192: one round of whole ones, then equal parts
    (4, 256, 4300, 4000, 31, 31, 256, 0),      # 248: then large and small ones
    (4, 256, 4300, 4000, 24, 24, 128, 0),
    (5, 512, 9000, 8300, 48, 24, 128, 0),      # 480
]


@pytest.mark.parametrize("case", CUT, ids=lambda c: "B{}T{}S{}e{}H{}/{}d{}W{}".format(*c))
def test_cut_units_back_to_back(case):
    test_calls_back_to_back(case)
