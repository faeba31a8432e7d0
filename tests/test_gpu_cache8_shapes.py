"""The 8-bit cache attention where its launches change form: few and many
rows on either side of the limit, splits merged in a cluster or by a second
launch, query tiles cut into equal and unequal parts, windows over long
caches with gaps, every head grouping; against the fp64 oracle with the
bounds of test_gpu_cache8.py.  And the calls that its documentation allows at
the ends of their ranges.
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


def _check(case, dtype=torch.float16, weights=True, exps=(-2, 2), seed=3):
    import transformer_attention_gb300 as G3
    B, T, S, end, H, H_kv, d_h, W, pads, layout = case
    c, Q, seg = C._stage(B, T, S, end, H, H_kv, d_h, pads, layout, seed + S + T, exps)
    ref, w, A, PV = C8.attend(Q, c, seg, pads, end, W)
    vmax = float(C8.values(c, "v").nan_to_num(0.0).abs().max())
    dev = C._to_dev(c)
    wsum = torch.zeros((B, S), device="cuda") if weights else None
    O = C._attend(G3, Q, dev, seg, pads, T, end, H, H_kv, d_h, W, dtype, wsum)
    assert G3.gemma3_attn_check_status() == 0
    C._check_o(O, ref, A, PV, vmax, end + T, d_h, dtype)
    if weights:
        d = 2 * ((d_h / 16 + 4) * 2.0 ** -22 * float(A.max()) + 2.0 ** -21)
        tol = (d + (T * H + 2) * 2.0 ** -23) * w
        got = wsum.cpu().to(F64)
        assert ((got - w).abs() <= tol).all()
        # every token and head with something to see hands out a weight of one
        total = sum(T - (pads[b] if pads else 0) for b in range(B)) * H
        if W == 0:
            assert abs(float(got.sum()) / max(total, 1) - 1) < 1e-5 or total == 0


FORMS = [
    # one row, long: a second launch merges many splits
    (1, 1, 20000, 19999, 2, 2, 128, 0, None, "plain"),
    (1, 1, 20000, 19990, 4, 1, 256, 0, None, "gaps"),
    # short: one to eight CTAs of a cluster
    (2, 1, 70, 63, 4, 2, 128, 0, None, "plain"),
    (8, 1, 1100, 1050, 8, 4, 256, 0, None, "gaps"),
    (1, 2, 600, 555, 4, 1, 256, 0, [1], "stale"),
    (3, 1, 2200, 2100, 8, 8, 128, 0, None, "plain"),
    # windows: late slots only, early slots found behind a jump of positions
    (2, 1, 9000, 8990, 8, 4, 256, 512, None, "gaps"),
    (2, 3, 9000, 8900, 4, 2, 128, 300, [0, 1], "plain"),
    (1, 16, 5000, 4900, 1, 1, 128, 1000, None, "gaps"),
    # the last few-row call and the first many-row one, each grouping
    (1, 16, 300, 200, 3, 3, 128, 0, None, "plain"),
    (1, 17, 300, 200, 3, 3, 128, 0, None, "plain"),
    (1, 8, 300, 200, 6, 3, 256, 0, [2], "stale"),
    (1, 9, 300, 200, 6, 3, 256, 0, [2], "stale"),
    (2, 4, 900, 800, 12, 3, 256, 50, None, "gaps"),
    (2, 5, 900, 800, 12, 3, 256, 50, None, "gaps"),
    # query tiles: one row over, one token, exactly full
    (1, 64, 400, 336, 4, 1, 128, 0, None, "plain"),
    (1, 65, 400, 300, 4, 1, 128, 0, None, "plain"),
    (1, 256, 300, 0, 2, 2, 128, 0, None, "plain"),
    (1, 128, 4000, 3800, 2, 2, 256, 0, [7], "gaps"),
    (1, 33, 4000, 3800, 8, 2, 256, 700, [30], "gaps"),
    # 96 and 100 units: large parts and small ones
    (4, 700, 900, 200, 8, 8, 128, 0, [0, 3, 700, 1], "plain"),
    (5, 600, 1100, 450, 4, 4, 256, 0, None, "gaps"),
    # more units than SMs, the rest of them cut
    (3, 1000, 1000, 0, 6, 6, 256, 0, [0, 500, 999], "plain"),
    (2, 900, 2000, 1000, 10, 10, 256, 300, [0, 1], "gaps"),
]


@pytest.mark.parametrize("case", FORMS, ids=C.IDS)
def test_forms(case):
    _check(case)


@pytest.mark.parametrize("T", [1, 12, 40])
def test_window_behind_a_jump_back_of_positions(T):
    """Stored positions need not grow with the slot: early slots that hold the
    positions just before the queries' are seen, late ones far away are not."""
    import transformer_attention_gb300 as G3
    B, S, end, H, H_kv, d_h, W = 2, 6000, 5000, 4, 2, 128, 200
    c, Q, seg = C._stage(B, T, S, end, H, H_kv, d_h, None, "plain", 9)
    for b in range(B):
        p = torch.arange(end + T)
        p[:end] += 100000
        p[300 + 700 * b:420 + 700 * b] = torch.arange(4900, 5020)   # around the queries'
        p[2777] = 5001
        p[end:] = torch.arange(5000, 5000 + T)
        c["pos"][b, :end + T] = p
        seg[b] = p[end:]
    ref, w, A, PV = C8.attend(Q, c, seg, None, end, W)
    dev = C._to_dev(c)
    wsum = torch.zeros((B, S), device="cuda")
    O = C._attend(G3, Q, dev, seg, None, T, end, H, H_kv, d_h, W, torch.float16, wsum)
    assert G3.gemma3_attn_check_status() == 0
    C._check_o(O, ref, A, PV, float(C8.values(c, "v").nan_to_num(0.0).abs().max()), end + T, d_h, torch.float16)
    got = wsum.cpu().to(F64)
    assert torch.equal(got > 0, w > 0)
    assert float((got - w).abs().max()) < 1e-4


@pytest.mark.parametrize("T", [1, 5, 70])
def test_rows_that_see_nothing(T):
    """A batch row of padding only, and one whose cache holds no token that a
    query sees: zeros, and no weight for any slot."""
    import transformer_attention_gb300 as G3
    B, S, end, H, H_kv, d_h = 3, 500, 300, 4, 2, 256
    c, Q, seg = C._stage(B, T, S, end, H, H_kv, d_h, None, "plain", 2)
    pads = [0, T, 0]
    c["pos"][1, end:end + T] = -1
    c["pos"][2, :] = -1
    dev = C._to_dev(c)
    for W in (0, 100):
        wsum = torch.full((B, S), 0.5, device="cuda")
        O = C._attend(G3, Q, dev, seg, pads, T, end, H, H_kv, d_h, W, torch.bfloat16, wsum)
        assert G3.gemma3_attn_check_status() == 0
        assert (O[1:] == 0).all() and (O[0] != 0).any()
        assert (wsum[1:] == 0.5).all() and (wsum[0] > 0.5).any()


@pytest.mark.parametrize("T", [2, 100])
def test_extreme_windows_and_positions(T):
    """Windows and positions near 2^31 do not overflow."""
    import transformer_attention_gb300 as G3
    B, S, end, H, H_kv, d_h = 1, 400, 250, 2, 2, 128
    top = 2 ** 31 - 1
    for W, shift in ((top, 0), (top, top - 400), (60, top - 400), (1, 0)):
        c, Q, seg = C._stage(B, T, S, end, H, H_kv, d_h, None, "plain", 6)
        c["pos"][0, :end + T] += shift
        seg += shift
        ref, w, A, PV = C8.attend(Q, c, seg, None, end, W)
        wsum = torch.zeros((B, S), device="cuda")
        O = C._attend(G3, Q, C._to_dev(c), seg, None, T, end, H, H_kv, d_h, W, torch.float16, wsum)
        assert G3.gemma3_attn_check_status() == 0
        C._check_o(O, ref, A, PV, float(C8.values(c, "v").nan_to_num(0.0).abs().max()), end + T, d_h,
                   torch.float16)
        assert torch.equal(wsum.cpu() > 0, w.float() > 0)


@pytest.mark.parametrize("T", [1, 10, 60])
def test_nan_in_a_seen_slot_reaches_only_its_head(T):
    """A NaN number of a slot that is seen makes that kv head's rows NaN, and
    no other head's or batch row's."""
    import transformer_attention_gb300 as G3
    B, S, end, H, H_kv, d_h = 2, 300, 200, 4, 2, 128
    c, Q, seg = C._stage(B, T, S, end, H, H_kv, d_h, None, "plain", 8)
    c["v8"][0, 57, 1, 3] = 0x7F
    O = C._attend(G3, Q, C._to_dev(c), seg, None, T, end, H, H_kv, d_h, 0, torch.float16, None)
    assert G3.gemma3_attn_check_status() == 0
    assert torch.isnan(O[0, :, 2:, 3]).all()
    assert not torch.isnan(O[0, :, :2]).any() and not torch.isnan(O[1]).any()


def test_values_beyond_fp16():
    """Numbers that stand for 65536 count as fp16's largest in every form."""
    import transformer_attention_gb300 as G3
    B, S, H, H_kv, d_h = 1, 200, 2, 2, 128
    for T, end in ((1, 150), (40, 100)):
        c = C8.empty(B, S, H_kv, d_h)
        x = torch.full((B, end + T, H_kv, d_h), 65504.0).half()
        k = torch.zeros_like(x)
        c = C8.write(c, k, x, torch.arange(end + T)[None], None, 0)
        assert float(C8.values(c, "v").max()) == 65536.0
        Q = torch.zeros((B, T, H, d_h)).half()
        seg = torch.arange(end, end + T)[None]
        O = C._attend(G3, Q, C._to_dev(c), seg, None, T, end, H, H_kv, d_h, 0, torch.bfloat16, None)
        assert G3.gemma3_attn_check_status() == 0
        assert ((O.float() - 65536.0).abs() <= 65536.0 * 2.0 ** -8).all()


def test_longest_offsets():
    """A cache whose bytes pass 2^32: the last slots of the last row."""
    import transformer_attention_gb300 as G3
    B, S, H_kv, d_h, H = 3, 500000, 16, 256, 16
    n = 40
    end = S - n
    dev = list(G3.new_kv_cache8(B, S, H_kv, d_h, "cuda"))
    assert dev[0].numel() > 2 ** 32
    kvd = H_kv * d_h
    x = C._rows((B * n, 2 * kvd), 5)
    seg = torch.arange(end, end + n).repeat(B, 1)
    C._write(G3, x.cuda(), H_kv, d_h, 2 * kvd, seg, None, B, n, S, end, dev)
    back = torch.empty((B * n, 2 * kvd), dtype=torch.float16, device="cuda")
    G3.gemma3_kv_cache8_read(dev[0], dev[1], dev[2], dev[3], B, S, end, n, H_kv, d_h, back,
                             back[:, kvd:], 2 * kvd)
    small = C8.write(C8.empty(B, 128, H_kv, d_h), x[:, :kvd].reshape(B, n, H_kv, d_h),
                     x[:, kvd:].reshape(B, n, H_kv, d_h), seg, None, end % 64)
    want = torch.cat([C8.values(small, k)[:, end % 64:end % 64 + n].reshape(B * n, kvd)
                      for k in "kv"], 1)
    assert torch.equal(back.cpu().to(F64), want)
    Q = (torch.randn((B, 1, H, d_h), generator=C._gen(4)) / 16).half()
    O = C._attend(G3, Q, dev, seg[:, -1:], None, 1, S - 1, H, H_kv, d_h, 0, torch.float16, None)
    ref, _, A, PV = C8.attend(Q, small, seg[:, -1:], None, end % 64 + n - 1, 0)
    C._check_o(O, ref, A, PV, float(C8.values(small, "v").nan_to_num(0.0).abs().max()), n, d_h, torch.float16)
    w = torch.rand((B, S), device="cuda")
    got, w_got, kept = G3.evict_kv_cache8(tuple(dev), w, S, 30, 10, S=64)
    assert G3.gemma3_attn_check_status() == 0
    for b in range(B):
        held = list(range(end, S))
        late = held[-10:]
        rank = sorted(held[:-10], key=lambda s: -float(w[b, s]))[:20]
        assert kept[b].cpu().tolist() == sorted(late + rank)


def test_tensors_elsewhere_are_refused():
    import transformer_attention_gb300 as G3
    dev = G3.new_kv_cache8(1, 70, 2, 128, "cuda")
    out = torch.zeros((1, 512), dtype=torch.float16)
    with pytest.raises(ValueError):
        G3.gemma3_kv_cache8_read(dev[0], dev[1], dev[2], dev[3], 1, 70, 0, 1, 2, 128, out,
                                 out[:, 256:], 512)
