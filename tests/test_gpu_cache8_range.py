"""The 8-bit cache attention over the range of its probabilities: keys far
above many equal ones; of query positions: negative ones; and of stored
values: beyond fp16's largest.

Bounds as in test_gpu_cache8.py, with a tighter absolute term: probabilities
are rounded to fp16 times 2^15 (few rows) or 2^7 at least (many), so that
below fp16's normal range they are off by 2^-25 / 2^7 of the row's largest.
"""
import pytest
import torch

from oracle import cache8_oracle as C8
from tests import test_gpu_cache8 as C

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_attention_gb300.build import build
    build()
    import transformer_attention_gb300 as G3
    G3.lib()


FORMS = [(1, 4, 2, 128), (3, 4, 1, 256), (40, 4, 2, 128), (300, 4, 2, 128), (70, 4, 2, 256)]


@pytest.mark.parametrize("apart", [8, 64, 5000])
@pytest.mark.parametrize("gap", [12.0, 16.0, 18.0, 20.0])
@pytest.mark.parametrize("T,H,H_kv,d_h", FORMS)
def test_sinks_far_above_equal_keys(T, H, H_kv, d_h, gap, apart):
    """Every apart-th slot, of value zero, is e^gap times as likely as the
    others, whose small shares still add up."""
    import transformer_attention_gb300 as G3
    B, S, end = 1, 5000, 4500
    c, Q, seg = C._stage(B, T, S, end, H, H_kv, d_h, None, "plain", 7, (0, 0))
    v = 100.0 + 30.0 * torch.randn(c["v8"].shape, generator=C._gen(5))
    c["v8"][:, :end + T] = C8.encode(v.to(F64))[:, :end + T]
    c["v8"][:, :end:apart] = 0
    c["k8"][:, :end + T] = 0
    c["k8"][:, :end:apart, :, 0] = C8.encode(torch.tensor(gap, dtype=F64))
    Q = torch.zeros_like(Q)
    Q[..., 0] = 1.0
    ref, w, A, PV = C8.attend(Q, c, seg, None, end, 0)
    wsum = torch.zeros((B, S), device="cuda")
    O = C._attend(G3, Q, C._to_dev(c), seg, None, T, end, H, H_kv, d_h, 0, torch.float16, wsum)
    assert G3.gemma3_attn_check_status() == 0
    # (the largest probability is 1 / sinks: each of the others' is off by that share)
    vmax = float(C8.values(c, "v").nan_to_num(0.0).abs().max())
    sinks = -(-end // apart)
    d = (d_h / 16 + 4) * 2.0 ** -22 * A + 2.0 ** -21
    tol = ((2.0 ** -11 + 2 * d + 2.0 ** -18)[..., None] * PV + (end + T) / sinks * 2.0 ** -32 * vmax) * (
        1 + 2.0 ** -11) + 2.0 ** -11 * ref.abs() + 2.0 ** -25
    err = (O.cpu().to(F64) - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())
    dw = 2 * ((d_h / 16 + 4) * 2.0 ** -22 * float(A.max()) + 2.0 ** -21)
    assert ((wsum.cpu().to(F64) - w).abs() <= (dw + (T * H + 2) * 2.0 ** -23) * w).all()


@pytest.mark.parametrize("T,H,H_kv,d_h", FORMS)
def test_queries_at_negative_positions(T, H, H_kv, d_h):
    """A query's own position may be negative: on a local layer it sees the
    slots within its window, and they receive its weight."""
    import transformer_attention_gb300 as G3
    B, S, end, W = 2, 700, 350, 60
    for shift in (-30, -T // 2 - 5, -2 ** 31):
        c, Q, seg = C._stage(B, T, S, end, H, H_kv, d_h, None, "plain", 8)
        seg = torch.arange(T).repeat(B, 1) + shift
        c["pos"][:, end:end + T] = -1
        ref, w, A, PV = C8.attend(Q, c, seg, None, end, W)
        wsum = torch.zeros((B, S), device="cuda")
        O = C._attend(G3, Q, C._to_dev(c), seg, None, T, end, H, H_kv, d_h, W, torch.float16, wsum)
        assert G3.gemma3_attn_check_status() == 0
        C._check_o(O, ref, A, PV, float(C8.values(c, "v").nan_to_num(0.0).abs().max()), end + T, d_h,
                   torch.float16)
        assert (w > 0).any() == (shift > -2 ** 31)
        got = wsum.cpu().to(F64)
        dw = 2 * ((d_h / 16 + 4) * 2.0 ** -22 * float(A.max()) + 2.0 ** -21)
        assert ((got - w).abs() <= (dw + (T * H + 2) * 2.0 ** -23) * w).all()


@pytest.mark.parametrize("T,H,H_kv,d_h", FORMS)
def test_stored_values_beyond_fp16(T, H, H_kv, d_h):
    """A number that stands for 65536 or, from an infinity, for 114688 counts
    as that in every form, in K and in V."""
    import transformer_attention_gb300 as G3
    B, S, end = 1, 700, 300
    g = C._gen(9)
    k = torch.zeros((B, end + T, H_kv, d_h)).half()
    v = torch.zeros_like(k)
    # K: 65504 (stored as 65536), an infinity or 57344 in one channel
    pick = torch.randint(0, 3, (B, end + T, H_kv), generator=g)
    top = torch.tensor([65504.0, float("inf"), 57344.0]).half()
    k[..., 0] = top[pick]
    sign = torch.randint(0, 2, v.shape, generator=g) * 2.0 - 1.0
    v[:] = (top[torch.randint(0, 3, v.shape, generator=g)].float() * sign).half()
    c = C8.write(C8.empty(B, S, H_kv, d_h), k, v, torch.arange(end + T)[None], None, 0)
    assert float(C8.values(c, "k").max()) == 114688.0
    Q = torch.zeros((B, T, H, d_h)).half()
    Q[..., 0] = 2.0 ** -15
    seg = torch.arange(end, end + T)[None]
    ref, w, A, PV = C8.attend(Q, c, seg, None, end, 0)
    wsum = torch.zeros((B, S), device="cuda")
    O = C._attend(G3, Q, C._to_dev(c), seg, None, T, end, H, H_kv, d_h, 0, torch.bfloat16, wsum)
    assert G3.gemma3_attn_check_status() == 0
    C._check_o(O, ref, A, PV, 114688.0, end + T, d_h, torch.bfloat16)
    dw = 2 * ((d_h / 16 + 4) * 2.0 ** -22 * float(A.max()) + 2.0 ** -21)
    assert ((wsum.cpu().to(F64) - w).abs() <= (dw + (T * H + 2) * 2.0 ** -23) * w).all()


@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("T,H,H_kv,d_h", FORMS + [(600, 2, 1, 128), (200, 2, 2, 256)])
def test_large_values_in_some_blocks(T, H, H_kv, d_h, window):
    """Blocks of the largest scale, for K, for V or for both, next to others."""
    import transformer_attention_gb300 as G3
    B, S, end = 2, 1500, 800
    n = end + T
    g = C._gen(10 + T)
    k = torch.randn((B, n, H_kv, d_h), generator=g)
    v = 3000 * torch.randn((B, n, H_kv, d_h), generator=g)
    kind = (torch.arange(n)[:, None] // 64 * 7 + torch.arange(H_kv)[None] * 3) % 5   # of a block and head
    top = torch.tensor([65504.0, float("inf"), 57344.0])
    pick = top[torch.randint(0, 3, (B, n, H_kv), generator=g)]
    k[..., 0] = torch.where((kind % 2 == 0)[None], pick, k[..., 0])
    sign = torch.randint(0, 2, v.shape, generator=g) * 2.0 - 1.0
    big = top[torch.randint(0, 3, v.shape, generator=g)] * sign
    v = torch.where((kind >= 2)[None, :, :, None] & (torch.rand(v.shape, generator=g) < 0.3), big, v)
    c = C8.write(C8.empty(B, S, H_kv, d_h), k.half(), v.half(), torch.arange(n).repeat(B, 1), None, 0)
    for w in ("ks", "vs"):
        assert 256.0 in c[w] and 0 < float((c[w] == 256.0).double().mean()) < 1
    Q = (torch.randn((B, T, H, d_h), generator=g) * 0.02).half()
    Q[..., 0] = 2.0 ** -15
    seg = torch.arange(end, n).repeat(B, 1)
    ref, w, A, PV = C8.attend(Q, c, seg, None, end, window)
    wsum = torch.zeros((B, S), device="cuda")
    O = C._attend(G3, Q, C._to_dev(c), seg, None, T, end, H, H_kv, d_h, window, torch.bfloat16, wsum)
    assert G3.gemma3_attn_check_status() == 0
    C._check_o(O, ref, A, PV, 114688.0, n, d_h, torch.bfloat16)
    dw = 2 * ((d_h / 16 + 4) * 2.0 ** -22 * float(A.max()) + 2.0 ** -21)
    assert ((wsum.cpu().to(F64) - w).abs() <= (dw + (T * H + 2) * 2.0 ** -23) * w).all()
