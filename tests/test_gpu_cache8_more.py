"""The 8-bit cache in longer runs: prompts of uneven query tiles, an eviction
whose keys exceed a CTA's shared memory, calls that repeat, graphs that share
a workspace, keys beyond fp16's largest."""
import pytest
import torch

from oracle import cache8_oracle as C8
from tests import test_gpu_cache8 as C
from tests.test_gpu_cache8_shapes import _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_attention_gb300.build import build
    build()
    import transformer_attention_gb300 as G3
    G3.lib()


PROMPTS = [
    # more query tiles than SMs, the first tokens' far shorter than the last's
    (2, 1500, 1500, 0, 12, 6, 256, 0, [0, 700], "plain"),
    (5, 1100, 1200, 64, 8, 8, 128, 0, [0, 1100, 1, 550, 0], "plain"),
    (2, 1300, 1400, 10, 8, 8, 256, 200, [3, 0], "gaps"),
]


@pytest.mark.parametrize("case", PROMPTS, ids=C.IDS)
def test_long_prompts(case):
    _check(case)


@pytest.mark.parametrize("equal", [False, True])
def test_evict_keys_beyond_shared_memory(equal):
    """Runs of more than 40960 slots per CTA (S > 327680) read their keys again."""
    import transformer_attention_gb300 as G3
    B, S, end, H_kv, d_h, keep, recent = 2, 340000, 339001, 1, 128, 20001, 333
    g = C._gen(12)
    cache = G3.new_kv_cache8(B, S, H_kv, d_h, "cuda")
    pos = torch.arange(S, dtype=torch.int32).repeat(B, 1)
    pos[torch.rand((B, S), generator=g) < 0.05] = -1
    cache[4].copy_(pos.cuda())
    w = torch.full((B, S), 2.0) if equal else torch.round(torch.rand((B, S), generator=g) * 5e4)
    got, w_got, kept = G3.evict_kv_cache8(cache, w.cuda(), end, keep, recent, S=keep)
    assert G3.gemma3_attn_check_status() == 0
    for b in range(B):
        key = w[b, :end].double()
        key[end - recent:] = float("inf")
        key[pos[b, :end] < 0] = -1
        order = torch.sort(key, descending=True, stable=True)[1][:keep]
        want = torch.sort(order[key[order] >= 0])[0]
        assert len(want) == keep
        assert torch.equal(kept[b].cpu().long(), want)
        assert torch.equal(got[4][b].cpu(), pos[b][want])
        assert torch.equal(w_got[b].cpu(), w[b][want])


def test_graphs_that_share_a_workspace():
    """A decode step, a chunk and a windowed step, all with weights, captured
    with one workspace and replayed in turn, give what eager calls give, every
    time the same bits."""
    import transformer_attention_gb300 as G3
    calls = []
    for T, end, window in ((2, 900, 0), (150, 700, 0), (3, 900, 128)):
        c, Q, seg = C._stage(2, T, 1000, end, 8, 4, 256, [0, 1], "plain", T)
        calls.append((T, end, window, Q.cuda(), C._to_dev(c), seg.int().cuda()))
    pads = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    n = max(G3.gemma3_cached8_attention_workspace_size(2, T, 1000, 8, 4, 256, True)
            for T, *_ in calls)

    def run(call, O, w, ws):
        T, end, window, Q, dev, seg = call
        w.zero_()
        G3.gemma3_cached8_attention(Q, *dev, seg, pads, O, G3.GEMMA3_BF16, w, 2, T, 1000, end, 8, 4,
                                    256, window, ws, ws.numel())

    def outputs(call):
        return (torch.empty((2, call[0], 8, 256), dtype=torch.bfloat16, device="cuda"),
                torch.empty((2, 1000), device="cuda"))

    want = []
    for call in calls:
        o = outputs(call)
        run(call, *o, torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda"))
        want.append(o)
    shared = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    torch.cuda.synchronize()
    for call in calls:
        g, o = torch.cuda.CUDAGraph(), outputs(call)
        with torch.cuda.graph(g):
            run(call, *o, shared)
        graphs.append(g)
        outs.append(o)
    for i in (0, 1, 2, 1, 0, 2, 2, 1):
        outs[i][0].fill_(7)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
    assert G3.gemma3_attn_check_status() == 0


@pytest.mark.parametrize("T,end", [(1, 150), (40, 100)])
def test_keys_beyond_fp16(T, end):
    """Keys that stand for 65536: equal keys share the weight equally."""
    import transformer_attention_gb300 as G3
    B, S, H, H_kv, d_h = 1, 200, 2, 2, 128
    k = torch.full((B, end + T, H_kv, d_h), 65504.0).half()
    v = torch.randn((B, end + T, H_kv, d_h), generator=C._gen(3)).half()
    c = C8.write(C8.empty(B, S, H_kv, d_h), k, v, torch.arange(end + T)[None], None, 0)
    assert float(C8.values(c, "k").max()) == 65536.0
    Q = torch.full((B, T, H, d_h), 2.0 ** -12).half()
    seg = torch.arange(end, end + T)[None]
    w = torch.zeros((B, S), device="cuda")
    O = C._attend(G3, Q, C._to_dev(c), seg, None, T, end, H, H_kv, d_h, 0, torch.float16, w)
    assert G3.gemma3_attn_check_status() == 0
    vals = C8.values(c, "v").double()
    for t in range(T):
        mean = vals[0, :end + t + 1].mean(0)
        # p is exactly 1, O's sum in fp32 (n 2^-24 of the magnitudes), one rounding to fp16
        tol = 2.0 ** -11 * mean.abs() + (end + T) * 2.0 ** -24 * vals[0].abs().max() + 2.0 ** -25
        assert ((O[0, t].cpu().double() - mean).abs() <= tol).all()
    want = torch.zeros(S, dtype=torch.float64)
    for t in range(T):
        want[:end + t + 1] += H / (end + t + 1)
    assert ((w[0].cpu().double() - want).abs() <= (T * H + 4) * 2.0 ** -23 * want).all()


@pytest.mark.parametrize("T,d_h,stride", [(70, 128, 3), (150, 256, 2), (70, 256, 0), (9, 128, 3)])
def test_windows_over_positions_that_skip(T, d_h, stride):
    """Positions stride * slot (0: shuffled): neither a tile's slots nor its
    tokens are at consecutive positions."""
    import transformer_attention_gb300 as G3
    B, S, end, H, H_kv, W = 2, 1500, 1200, 4, 2, 300
    c, Q, seg = C._stage(B, T, S, end, H, H_kv, d_h, None, "plain", 21)
    for b in range(B):
        n = torch.arange(end + T)
        p = n * stride + 5 if stride else torch.randperm(end + T, generator=C._gen(b))
        c["pos"][b, :end + T] = p
        seg[b] = p[end:]
    ref, w, A, PV = C8.attend(Q, c, seg, None, end, W)
    wsum = torch.zeros((B, S), device="cuda")
    O = C._attend(G3, Q, C._to_dev(c), seg, None, T, end, H, H_kv, d_h, W, torch.float16, wsum)
    assert G3.gemma3_attn_check_status() == 0
    C._check_o(O, ref, A, PV, float(C8.values(c, "v").nan_to_num(0.0).abs().max()), end + T, d_h,
               torch.float16)
    d = 2 * ((d_h / 16 + 4) * 2.0 ** -22 * float(A.max()) + 2.0 ** -21)
    assert ((wsum.cpu().double() - w).abs() <= (d + (T * H + 2) * 2.0 ** -23) * w).all()


CUT = [
    (4, 256, 4300, 4000, 12, 12, 256, 0, [0, 256, 100, 1], "gaps"),
    (4, 256, 4300, 4000, 24, 24, 256, 0, None, "plain"),
    (4, 256, 4300, 4000, 31, 31, 256, 0, None, "stale"),
    (4, 250, 4300, 4040, 24, 24, 128, 0, [0, 3, 200, 0], "gaps"),
]


@pytest.mark.parametrize("case", CUT, ids=C.IDS)
def test_cut_units(case):
    """Query tiles over slots enough to be cut into parts: 96, 192 and 248
    units on 152 SMs, in equal parts and in large and small ones."""
    _check(case)


@pytest.mark.parametrize("where", [0, 20000, 59000])
@pytest.mark.parametrize("T", [40, 600])
def test_window_behind_many_slots(T, where):
    """A local layer far into a cache: the first visible slot lies early (a run
    of slots at the queries' positions), in the middle, or just before."""
    import transformer_attention_gb300 as G3
    B, S, end, H, H_kv, d_h, W = 1, 61000, 60000, 2, 1, 128, 500
    c, Q, seg = C._stage(B, T, S, end, H, H_kv, d_h, None, "plain", 33)
    p = torch.arange(end + T) + 100000
    p[where:where + 64] = torch.arange(end + 100000 - 100, end + 100000 - 36)
    c["pos"][0, :end + T] = p
    seg[0] = p[end:]
    ref, w, A, PV = C8.attend(Q, c, seg, None, end, W)
    wsum = torch.zeros((B, S), device="cuda")
    O = C._attend(G3, Q, C._to_dev(c), seg, None, T, end, H, H_kv, d_h, W, torch.float16, wsum)
    assert G3.gemma3_attn_check_status() == 0
    C._check_o(O, ref, A, PV, float(C8.values(c, "v").nan_to_num(0.0).abs().max()), end + T, d_h,
               torch.float16)
    d = 2 * ((d_h / 16 + 4) * 2.0 ** -22 * float(A.max()) + 2.0 ** -21)
    assert ((wsum.cpu().double() - w).abs() <= (d + (T * H + 2) * 2.0 ** -23) * w).all()
