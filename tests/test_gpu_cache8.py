"""GPU parity of the 8-bit KV cache against its fp64 oracle.

- write: codes, scales and positions equal, other slots and blocks untouched;
- read: every value equal;
- attention: elementwise error bounds derived below; weights received;
- evict: the kept slots, their codes, scales, positions and weights equal;
- the layer entry equal to its stages; a run of prompt, steps, eviction and
  more steps; two streams; a captured graph; guard bytes.

Bounds of the attention test, for one row with probabilities p and values v:
a logit is a sum of exact products accumulated in fp32 in steps of 16
channels, off by at most (d_h / 16 + 4) 2^-22 A with A = max_s sum_c |q_c k_c|
(each step rounds or truncates at 2^-23 of a partial sum <= A, the last adds
scale it); exp2 adds 2^-21 relative.  A probability is rounded once to fp16,
2^-11 relative, or 2^-25 of the largest below fp16's normal range; on the
tensor cores the sums of p v are fp32 steps again, within 2^-18 of sum p |v|
for the lengths here.  So an output is within
  (2^-11 + 2 d + 2^-18) sum p |v| + n 2^-25 max |v| + its own half step,
d the relative error of a probability (and, once more, of the sum they are
divided by).
"""
import pytest
import torch

from oracle import cache8_oracle as C8
from tests import helpers as Hh
from transformer_attention_gb300 import workloads as WL

pytestmark = pytest.mark.gpu

F64 = torch.float64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_attention_gb300.build import build
    build()
    import transformer_attention_gb300 as G3
    G3.lib()


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rows(shape, seed, spread=2):
    g = _gen(seed)
    x = torch.randn(shape, generator=g)
    return (x * torch.exp2(torch.randint(-spread, spread + 1, shape[:-1] + (1,), generator=g))).half()


def _to_dev(c):
    """An oracle cache as the library's five tensors."""
    f8 = torch.float8_e4m3fn
    return (c["k8"].cuda().view(f8), c["v8"].cuda().view(f8), c["ks"].float().cuda(),
            c["vs"].float().cuda(), c["pos"].int().cuda())


def _from_dev(dev):
    k8, v8, ks, vs, pos = (t.cpu() for t in dev)
    return {"k8": k8.view(torch.uint8), "v8": v8.view(torch.uint8), "ks": ks.to(F64),
            "vs": vs.to(F64), "pos": pos.to(torch.int64)}


def _same(a, b):
    for k in ("pos", "ks", "vs", "k8", "v8"):
        assert torch.equal(a[k], b[k]), (k, int((a[k] != b[k]).sum()))


def _random_cache(B, S, H_kv, d_h, seed, exps=(-3, 3)):
    """A cache with every slot filled: any finite codes, scales 2^exps."""
    g = _gen(seed)
    c = C8.empty(B, S, H_kv, d_h)
    for k in ("k8", "v8"):
        x = torch.randn(c[k].shape, generator=g, dtype=torch.float32)
        c[k] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    for k in ("ks", "vs"):
        c[k] = torch.exp2(torch.randint(exps[0], exps[1] + 1, c[k].shape, generator=g).to(F64))
    c["pos"] = torch.arange(S).repeat(B, 1)
    return c


# ---------------------------------------------------------------- write and read
WRITE = [
    # B, T, S, end, H_kv, d_h, pads, extra elements between rows
    (1, 1, 1, 0, 1, 128, None, 0),
    (2, 1, 200, 131, 4, 256, None, 0),
    (3, 5, 40, 17, 2, 128, [0, 2, 5], 64),
    (2, 130, 300, 61, 2, 256, [0, 7], 8),
    (1, 64, 128, 64, 3, 128, None, 0),
    (2, 65, 129, 64, 1, 256, [65, 0], 0),
    (1, 700, 1000, 299, 2, 128, [100], 16),
]


def _write(G3, rows, H_kv, d_h, ld, seg, pad, B, T, S, end, dev):
    kvd = H_kv * d_h
    G3.gemma3_kv_cache8_write(rows, rows[:, kvd:], ld, seg.int().cuda(),
                              None if pad is None else torch.tensor(pad, dtype=torch.int32).cuda(),
                              B, T, S, end, H_kv, d_h, *dev)


@pytest.mark.parametrize("case", WRITE, ids=lambda c: "B{}T{}S{}e{}H{}d{}".format(*c[:6]))
@pytest.mark.parametrize("kind", ["spread", "small", "large", "zeros", "nonfinite"])
def test_write_and_read(case, kind):
    import transformer_attention_gb300 as G3
    B, T, S, end, H_kv, d_h, pad, extra = case
    kvd, ld = H_kv * d_h, 2 * H_kv * d_h + extra
    x = _rows((B, T, ld // 8, 8), 5 + T).reshape(B * T, ld)
    if kind == "small":         # below the smallest scale's normal numbers, fp16 subnormals
        x = x * 2.0 ** -15
    elif kind == "large":       # up to fp16's largest
        x = (x.float() * 9000).clamp(-65504, 65504).half()
    elif kind == "zeros":
        x = x * 0
    elif kind == "nonfinite":
        at = torch.randint(0, x.numel(), (max(3, x.numel() // 500),), generator=_gen(9))
        x.view(-1)[at] = torch.tensor([float("inf"), float("-inf"), float("nan")]).half()[
            torch.arange(at.numel()) % 3]
    c = _random_cache(B, S, H_kv, d_h, 11 + S, (-6, -2))
    c["pos"][:, end:] = -1
    seg = torch.randint(0, 5000, (B, T), generator=_gen(3))
    dev = _to_dev(c)
    rows = x.cuda()
    _write(G3, rows, H_kv, d_h, ld, seg, pad, B, T, S, end, dev)
    assert G3.gemma3_attn_check_status() == 0
    K = x[:, :kvd].reshape(B, T, H_kv, d_h)
    V = x[:, kvd:2 * kvd].reshape(B, T, H_kv, d_h)
    want = C8.write(c, K, V, seg, pad, end)
    _same(_from_dev(dev), want)
    # read back from inside a block, into strided rows
    first, n = max(0, end - 3), min(T + 3, S - max(0, end - 3))
    back = torch.full((B * n, ld), 3.0, dtype=torch.float16, device="cuda")
    G3.gemma3_kv_cache8_read(dev[0], dev[1], dev[2], dev[3], B, S, first, n, H_kv, d_h, back,
                             back[:, kvd:], ld)
    got = back.cpu().to(F64).reshape(B, n, ld)
    for i, w in enumerate(("k", "v")):
        ref = C8.values(want, w)[:, first:first + n].reshape(B, n, kvd).clamp(-65504, 65504)
        g = got[..., i * kvd:(i + 1) * kvd]
        assert torch.equal(torch.isnan(g), torch.isnan(ref))
        assert torch.equal(g.nan_to_num(0.0), ref.nan_to_num(0.0))
    assert (got[..., 2 * kvd:] == 3.0).all()


def test_write_token_by_token_equals_oracle():
    """Scales that grow several times within a block, one token per call."""
    import transformer_attention_gb300 as G3
    B, S, H_kv, d_h, n = 2, 150, 2, 128, 140
    kvd = H_kv * d_h
    x = _rows((B, n, 2 * kvd // 8, 8), 21, 1).reshape(B, n, 2 * kvd)
    x = (x * torch.exp2(torch.arange(n) / 9.0 % 8)[None, :, None]).half()
    c = C8.empty(B, S, H_kv, d_h)
    dev = _to_dev(c)
    for t in range(n):
        row = x[:, t].contiguous().cuda()
        seg = torch.full((B, 1), t)
        _write(G3, row, H_kv, d_h, 2 * kvd, seg, None, B, 1, S, t, dev)
        K = x[:, t:t + 1, :kvd].reshape(B, 1, H_kv, d_h)
        V = x[:, t:t + 1, kvd:].reshape(B, 1, H_kv, d_h)
        c = C8.write(c, K, V, seg, None, t)
    _same(_from_dev(dev), c)


def test_read_of_nothing():
    import transformer_attention_gb300 as G3
    dev = G3.new_kv_cache8(1, 70, 2, 128, "cuda")
    out = torch.full((1, 512), 2.0, dtype=torch.float16, device="cuda")
    G3.gemma3_kv_cache8_read(dev[0], dev[1], dev[2], dev[3], 1, 70, 70, 0, 2, 128, out, out[:, 256:],
                             512)
    torch.cuda.synchronize()
    assert (out == 2.0).all()


# ---------------------------------------------------------------- attention
STAGE = [
    # B, T, S, end, H, H_kv, d_h, window, pads, layout
    (1, 1, 1, 0, 4, 2, 128, 0, None, "plain"),
    (2, 1, 1000, 999, 4, 1, 256, 0, None, "plain"),
    (2, 1, 3000, 2500, 8, 4, 256, 64, None, "gaps"),
    (1, 1, 5000, 4999, 4, 2, 128, 0, None, "gaps"),
    (2, 3, 700, 600, 2, 2, 128, 100, [0, 1], "gaps"),
    (3, 2, 300, 10, 4, 1, 256, 0, [0, 0, 1], "stale"),
    (2, 5, 100, 50, 4, 4, 256, 7, None, "stale"),
    (4, 4, 600, 555, 4, 1, 128, 0, [0, 4, 1, 2], "gaps"),
    (1, 16, 400, 300, 2, 2, 256, 0, None, "plain"),
    (1, 17, 400, 300, 2, 2, 128, 0, [3], "gaps"),
    (2, 20, 200, 100, 4, 2, 256, 33, [0, 3], "gaps"),
    (1, 130, 130, 0, 8, 2, 128, 0, [5], "plain"),
    (2, 129, 500, 333, 4, 2, 128, 0, [0, 129], "stale"),
    (1, 200, 700, 450, 4, 4, 256, 90, [1], "gaps"),
    (1, 257, 1025, 700, 4, 1, 256, 0, [0], "stale"),
    (1, 1, 40000, 39999, 8, 4, 256, 1024, None, "plain"),
]
IDS = lambda c: "B{}T{}S{}e{}H{}/{}d{}W{}{}".format(*c[:8], "-pad" if c[8] else "") + "-" + c[9]  # noqa: E731


def _stage(B, T, S, end, H, H_kv, d_h, pads, layout, seed, exps=(-2, 2)):
    c = _random_cache(B, S, H_kv, d_h, seed, exps)
    Q = (torch.randn((B, T, H, d_h), generator=_gen(seed + 1)) * d_h ** -0.5).half()
    seg = torch.zeros((B, T), dtype=torch.int64)
    for b in range(B):
        p = torch.arange(end + T)
        if layout == "gaps":        # an empty stretch (a padded prompt) and a jump of positions
            e0, e1 = end // 3, end // 3 + max(1, end // 10)
            p[e1:] += 50 - (e1 - e0)
            p[e0:e1] = -1
        c["pos"][b, :end + T] = p
        c["pos"][b, end + T:] = torch.arange(S - end - T) if layout == "stale" else -1
        seg[b] = c["pos"][b, end:end + T]
        v = T - (pads[b] if pads else 0)
        c["pos"][b, end + v:end + T] = -1
    # every hidden slot holds NaN, and blocks nobody sees have a NaN scale
    for k, s in (("k8", "ks"), ("v8", "vs")):
        hidden = c["pos"] < 0
        hidden[:, end + T:] = True
        c[k][hidden] = 0x7F
        whole = torch.nn.functional.pad(hidden, (0, C8.blocks(S) * 64 - S), value=True)
        c[s][whole.view(B, -1, 64).all(2)] = float("nan")
    return c, Q, seg


def _attend(G3, Q, dev, seg, pads, T, end, H, H_kv, d_h, W, out_dtype, wsum, ws=None, stream=None):
    B, S = dev[4].shape
    if ws is None:
        n = G3.gemma3_cached8_attention_workspace_size(B, T, S, H, H_kv, d_h, wsum is not None)
        ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")
    O = torch.empty((B, T, H, d_h), dtype=out_dtype, device="cuda")
    pad = None if pads is None else torch.tensor(pads, dtype=torch.int32).cuda()
    G3.gemma3_cached8_attention(
        Q.cuda(), *dev, seg.int().cuda(), pad, O,
        G3.GEMMA3_F16 if out_dtype == torch.float16 else G3.GEMMA3_BF16, wsum, B, T, S, end, H,
        H_kv, d_h, W, ws, ws.numel(), stream)
    return O


def _check_o(O, ref, A, PV, vmax, n, d_h, dtype):
    d = (d_h / 16 + 4) * 2.0 ** -22 * A + 2.0 ** -21
    tol = ((2.0 ** -11 + 2 * d + 2.0 ** -18)[..., None] * PV + n * 2.0 ** -25 * vmax) * (
        1 + HALF_STEP[dtype]) + HALF_STEP[dtype] * ref.abs() + 2.0 ** -25
    err = (O.cpu().to(F64) - ref).abs()
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))


@pytest.mark.parametrize("case", STAGE, ids=IDS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_attention_stage(case, dtype):
    import transformer_attention_gb300 as G3
    B, T, S, end, H, H_kv, d_h, W, pads, layout = case
    c, Q, seg = _stage(B, T, S, end, H, H_kv, d_h, pads, layout, 10 + S + T)
    ref, w, A, PV = C8.attend(Q, c, seg, pads, end, W)
    vmax = float(C8.values(c, "v").nan_to_num(0.0).abs().max())
    dev = _to_dev(c)
    w0 = torch.rand((B, S), generator=_gen(77))
    wsum = w0.cuda()
    O = _attend(G3, Q, dev, seg, pads, T, end, H, H_kv, d_h, W, dtype, None)
    assert G3.gemma3_attn_check_status() == 0
    _check_o(O, ref, A, PV, vmax, end + T, d_h, dtype)
    Ow = _attend(G3, Q, dev, seg, pads, T, end, H, H_kv, d_h, W, dtype, wsum)
    assert G3.gemma3_attn_check_status() == 0
    assert torch.equal(O, Ow)
    for b in range(B):
        v = T - (pads[b] if pads else 0)
        assert (O[b, v:] == 0).all()
    # a weight is off by the relative error of its probabilities, and by the
    # fp32 sums over tokens and heads and onto what was there
    got = wsum.cpu().to(F64)
    d = 2 * ((d_h / 16 + 4) * 2.0 ** -22 * float(A.max()) + 2.0 ** -21)
    tol = (d + (T * H + 2) * 2.0 ** -23) * w + 2.0 ** -23 * (w0.to(F64) + w)
    assert ((got - w0.to(F64) - w).abs() <= tol).all()
    assert torch.equal(got[w == 0], w0.to(F64)[w == 0])
    # the same calls again: the same bits
    wsum2 = w0.cuda()
    assert torch.equal(_attend(G3, Q, dev, seg, pads, T, end, H, H_kv, d_h, W, dtype, wsum2), Ow)
    assert torch.equal(wsum2, wsum)


@pytest.mark.parametrize("T,H,H_kv,d_h", [(1, 4, 2, 128), (3, 4, 1, 256), (140, 2, 1, 128),
                                          (140, 2, 1, 256)])
def test_attention_over_scales_far_apart(T, H, H_kv, d_h):
    """Blocks whose V scales span the whole range, one key far above the rest."""
    import transformer_attention_gb300 as G3
    B, S, end = 1, 1000, 850
    c, Q, seg = _stage(B, T, S, end, H, H_kv, d_h, None, "plain", 4, (-2, 1))
    c["vs"] = torch.exp2((torch.arange(C8.blocks(S)) * 7 % 24 - 15).to(F64))[None, :, None].expand_as(
        c["vs"]).clone()
    c["k8"][0, 100] = C8.encode(Q[0, 0, 0].to(F64) * 200)      # a sink for the first query head
    ref, w, A, PV = C8.attend(Q, c, seg, None, end, 0)
    dev = _to_dev(c)
    O = _attend(G3, Q, dev, seg, None, T, end, H, H_kv, d_h, 0, torch.float16, None)
    assert G3.gemma3_attn_check_status() == 0
    vmax = float(C8.values(c, "v").nan_to_num(0.0).abs().max())
    # outputs near fp16's largest are compared below it
    keep = ref.abs() < 60000
    d = (d_h / 16 + 4) * 2.0 ** -22 * A + 2.0 ** -21
    tol = ((2.0 ** -11 + 2 * d + 2.0 ** -18)[..., None] * PV + (end + T) * 2.0 ** -25 * vmax) * (
        1 + 2.0 ** -11) + 2.0 ** -11 * ref.abs() + 2.0 ** -25
    err = (O.cpu().to(F64) - ref).abs()
    assert (err <= tol)[keep].all()


def test_attention_in_place():
    """O may take Q's place when no weights are asked for."""
    import transformer_attention_gb300 as G3
    for T in (1, 3, 150):
        c, Q, seg = _stage(2, T, 900, 700, 4, 2, 128, None, "plain", 5)
        dev = _to_dev(c)
        ref = _attend(G3, Q, dev, seg, None, T, 700, 4, 2, 128, 0, torch.float16, None)
        q = Q.cuda()
        n = G3.gemma3_cached8_attention_workspace_size(2, T, 900, 4, 2, 128)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        G3.gemma3_cached8_attention(q, *dev, seg.int().cuda(), None, q, G3.GEMMA3_F16, None, 2, T, 900,
                                    700, 4, 2, 128, 0, ws, ws.numel())
        assert torch.equal(q, ref)


# ---------------------------------------------------------------- evict
EVICT = [
    # B, S, end, S_dst, H_kv, d_h, keep, recent, weights
    (1, 1, 1, 1, 1, 128, 1, 0, "plain"),
    (2, 100, 0, 70, 2, 128, 65, 10, "plain"),
    (2, 300, 290, 128, 2, 256, 100, 16, "ties"),
    (1, 500, 499, 500, 1, 128, 499, 0, "odd"),
    (3, 700, 650, 300, 1, 256, 65, 65, "plain"),
    (1, 1500, 1300, 400, 2, 128, 333, 0, "equal"),
    (2, 9000, 8999, 3000, 1, 128, 2777, 100, "ties"),
    (1, 40000, 40000, 9000, 1, 128, 8000, 64, "odd"),
]


@pytest.mark.parametrize("case", EVICT, ids=lambda c: "B{}S{}e{}D{}H{}d{}k{}r{}-{}".format(*c))
def test_evict(case):
    import transformer_attention_gb300 as G3
    B, S, end, S_dst, H_kv, d_h, keep, recent, kind = case
    g = _gen(S + keep)
    c = _random_cache(B, S, H_kv, d_h, 31 + S, (-15, 6))
    c["pos"][torch.rand((B, S), generator=g) < 0.1] = -1
    w = torch.exp(2 * torch.randn((B, S), generator=g))
    if kind == "ties":
        w = torch.round(w)
    elif kind == "equal":
        w = torch.full_like(w, 0.25)
    elif kind == "odd":
        w = torch.round(2 * torch.randn((B, S), generator=g)) / 2
        u = torch.rand((B, S), generator=g)
        w[u < 0.02] = float("nan")
        w[(u > 0.02) & (u < 0.03)] = float("inf")
        w[(u > 0.03) & (u < 0.05)] = float("-inf")
        w[(u > 0.05) & (u < 0.2)] = -0.0
    dst = _random_cache(B, S_dst, H_kv, d_h, 41 + S, (-3, 3))
    w_dst = torch.rand((B, S_dst), generator=g)
    want, w_want, kept = C8.evict(c, w, end, keep, recent, dst, w_dst)
    into = (_to_dev(dst), w_dst.cuda())
    src = _to_dev(c)
    got, w_got, k_got = G3.evict_kv_cache8(src, w.cuda(), end, keep, recent, into=into)
    assert G3.gemma3_attn_check_status() == 0
    assert torch.equal(k_got.cpu().to(torch.int64), kept)
    _same(_from_dev(got), want)
    w_got = w_got.cpu()
    assert torch.equal(torch.isnan(w_got), torch.isnan(w_want))
    assert torch.equal(w_got.nan_to_num(0.5), w_want.nan_to_num(0.5))
    _same(_from_dev(src), c)


# ---------------------------------------------------------------- together
def _layer(**kw):
    return WL.small(WL.WORKLOADS["tiny_local"], name="cache8", **kw)


LAYERS = [
    dict(B=2, T=64, D=256, H=4, H_kv=2, d_h=256, attn_type="local", window=24),
    dict(B=2, T=64, D=384, H=4, H_kv=1, d_h=128, attn_type="global", window=0, rope_base=1e6,
         rope_scale=8.0, query_scale=168 ** -0.5),
]


@pytest.mark.parametrize("kw", LAYERS, ids=["local-d256", "global-d128"])
def test_layer_prompt_steps_evict_steps(kw):
    """A padded prompt, decode steps with the weights kept, an eviction and
    more steps: every call bitwise the composition of its stages, and the
    attention stage within its bounds of the oracle over the cache it read."""
    import transformer_attention_gb300 as G3
    w = _layer(**kw)
    B, D, H, H_kv, d_h = w.B, w.D, w.H, w.H_kv, w.d_h
    kvd, S, T0 = H_kv * d_h, 96, 40
    p = {k: v.cuda() for k, v in WL.weights(w).items()}
    x_all = WL.x_full(w).cuda()
    kind = G3.GEMMA3_LOCAL_SLIDING if w.attn_type == "local" else G3.GEMMA3_GLOBAL
    pads = [0, 5]
    cache = G3.new_kv_cache8(B, S, H_kv, d_h, "cuda")
    wsum = torch.zeros((B, S), device="cuda")

    def call(x, seg, pad, end, cache, wsum):
        M, T = B * x.shape[1], x.shape[1]
        xs = x.contiguous()
        segd = seg.int().cuda()
        padd = None if pad is None else torch.tensor(pad, dtype=torch.int32).cuda()
        twin, wtwin = tuple(t.clone() for t in cache), wsum.clone()
        got = G3.attention_forward_cached8(
            xs, segd, padd, cache, end, p["Wq"], p["Wkv"], p["Wo"], p["gamma_q"], p["gamma_k"], H=H,
            H_kv=H_kv, attn_type=kind, window=w.window, rope_base=w.rope_base,
            rope_scale=w.rope_scale, query_scale=w.query_scale, weight_sum=wsum)
        Q = torch.empty((M, H * d_h), dtype=torch.float16, device="cuda")
        KV = torch.empty((M, 2 * kvd), dtype=torch.float16, device="cuda")
        G3.gemma3_qkv_proj_norm_rope(xs, D, p["Wq"], p["Wkv"], Q, KV, M, D, H, H_kv, d_h,
                                     G3.GEMMA3_BF16, p["gamma_q"], p["gamma_k"], segd, w.rope_base,
                                     w.rope_scale, w.query_scale)
        G3.gemma3_kv_cache8_write(KV, KV[:, kvd:], 2 * kvd, segd, padd, B, T, twin[4].shape[1], end,
                                  H_kv, d_h, *twin)
        Qv = Q.view(B, T, H, d_h)
        O = _attend(G3, Qv, twin, seg, pad, T, end, H, H_kv, d_h, w.window, torch.bfloat16, wtwin)
        ref = G3.linear(O.view(M, H * d_h), p["Wo"]).view(B, T, D)
        assert G3.gemma3_attn_check_status() == 0
        assert torch.equal(got, ref) and torch.equal(wsum, wtwin)
        for a, b in zip(cache, twin):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        c = _from_dev(twin)
        r, _, A, PV = C8.attend(Qv.cpu(), c, seg, pad, end, w.window)
        _check_o(O, r, A, PV, float(C8.values(c, "v").abs().max()), end + T, d_h, torch.bfloat16)
        return got

    call(x_all[:, :T0], torch.arange(T0).repeat(B, 1), pads, 0, cache, wsum)
    end = T0
    for i in range(3):
        seg = torch.tensor([[T0 - q + i] for q in pads])
        call(x_all[:, end:end + 1], seg, None, end, cache, wsum)
        end += 1
    live = wsum.sum(1).cpu()
    if w.attn_type == "global":        # each token and head hands out a weight of one
        assert torch.allclose(live, torch.tensor([float((T0 - q + 3) * H) for q in pads]), rtol=1e-5)
    keep = 20
    small, w_small, kept = G3.evict_kv_cache8(cache, wsum, end, keep, 6, S=40)
    assert torch.equal(small[4][:, :keep].cpu(), cache[4].cpu().gather(1, kept.cpu().to(torch.int64)))
    end, used = keep, end
    for i in range(3, 6):
        seg = torch.tensor([[T0 - q + i] for q in pads])
        call(x_all[:, used:used + 1], seg, None, end, small, w_small)
        end, used = end + 1, used + 1
    # a chunk of tokens, one of them padding
    seg = torch.stack([torch.arange(T0 - q + 6, T0 - q + 13) for q in pads])
    call(x_all[:, used:used + 7], seg, [1, 0], end, small, w_small)


def test_two_streams_and_a_captured_graph():
    """Steps on two streams at once with workspaces of their own, and the
    same step captured and replayed on changed inputs."""
    import transformer_attention_gb300 as G3
    args = dict(T=2, S=2000, end=1500, H=8, H_kv=4, d_h=128)
    cs = [_stage(2, 2, 2000, 1500, 8, 4, 128, None, "gaps", s) for s in (1, 2)]
    n = G3.gemma3_cached8_attention_workspace_size(2, 2, 2000, 8, 4, 128, True)
    ins = [(Q.cuda(), _to_dev(c), seg.int().cuda()) for c, Q, seg in cs]

    def step(i, O, wsum, ws, stream=None):
        Q, dev, seg = ins[i]
        G3.gemma3_cached8_attention(Q, *dev, seg, None, O, G3.GEMMA3_F16, wsum, 2, args["T"],
                                    args["S"], args["end"], 8, 4, 128, 0, ws, ws.numel(), stream)

    def buffers():
        return (torch.zeros((2, 2, 8, 128), dtype=torch.float16, device="cuda"),
                torch.zeros((2, 2000), device="cuda"),
                torch.empty(max(n, 256), dtype=torch.uint8, device="cuda"))

    refs = []
    for i in (0, 1):
        b = buffers()
        step(i, *b)
        refs.append(b)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream(), torch.cuda.Stream()], [buffers(), buffers()]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                outs[i][1].zero_()
                step(i, *outs[i])
    torch.cuda.synchronize()
    for i in (0, 1):
        assert torch.equal(outs[i][0], refs[i][0]) and torch.equal(outs[i][1], refs[i][1])
    g, b = torch.cuda.CUDAGraph(), buffers()
    with torch.cuda.graph(g):
        b[1].zero_()
        step(0, *b)
    for i in (1, 0, 1):
        q, dev, seg = ins[i]
        q0, dev0, seg0 = [t.clone() for t in (ins[0][0],)][0], [t.clone() for t in ins[0][1]], ins[0][2].clone()
        ins[0][0].copy_(q)
        for a, s in zip(ins[0][1], dev):
            a.view(torch.uint8).copy_(s.view(torch.uint8))
        ins[0][2].copy_(seg)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b[0], refs[i][0]) and torch.equal(b[1], refs[i][1])
        ins[0][0].copy_(q0)
        for a, s in zip(ins[0][1], dev0):
            a.view(torch.uint8).copy_(s.view(torch.uint8))
        ins[0][2].copy_(seg0)
    assert G3.gemma3_attn_check_status() == 0


# ---------------------------------------------------------------- guard bytes
def test_only_outputs_and_workspace_are_written():
    """Every output between guard bytes; a cache only in the new slots' bytes."""
    import transformer_attention_gb300 as G3
    from tests.test_gpu_guards import Guarded
    B, S, H, H_kv, d_h, end = 2, 333, 4, 2, 128, 131
    kvd = H_kv * d_h
    for T in (1, 3, 170):
        c, Q, seg = _stage(B, T, S, end, H, H_kv, d_h, None, "plain", T)
        bufs = [Guarded(t.numel() * t.element_size(), t) for t in _to_dev(c)]
        dev = [g.inner for g in bufs]
        x = _rows((B * T, 2 * kvd), 8).cuda()
        G3.gemma3_kv_cache8_write(x, x[:, kvd:], 2 * kvd, seg.int().cuda(), None, B, T, S, end, H_kv,
                                  d_h, *dev)
        need = G3.gemma3_cached8_attention_workspace_size(B, T, S, H, H_kv, d_h, True)
        ws, O, wsum = Guarded(max(need, 256)), Guarded(B * T * H * d_h * 2), Guarded(B * S * 4)
        wsum.inner.zero_()
        G3.gemma3_cached8_attention(Q.cuda(), *dev, seg.int().cuda(), None, O.inner, G3.GEMMA3_BF16,
                                    wsum.inner, B, T, S, end, H, H_kv, d_h, 0, ws.inner, ws.n)
        keep, S_dst, n = 70, 90, end + T
        outs = [Guarded(B * S_dst * kvd), Guarded(B * S_dst * kvd), Guarded(B * 2 * H_kv * 4),
                Guarded(B * 2 * H_kv * 4), Guarded(B * S_dst * 4), Guarded(B * S_dst * 4),
                Guarded(B * keep * 4)]
        G3.gemma3_kv_cache8_evict(*dev, wsum.inner, B, S, n, H_kv, d_h, keep, 9,
                                  *[g.inner for g in outs], S_dst)
        back = Guarded(B * keep * 2 * kvd * 2)
        rows = back.view(torch.float16, (B * keep, 2 * kvd))
        G3.gemma3_kv_cache8_read(*[g.inner for g in outs[:4]], B, S_dst, 0, keep, H_kv, d_h, rows,
                                 rows[:, kvd:], 2 * kvd)
        assert G3.gemma3_attn_check_status() == 0
        assert all(g.guards_intact() for g in bufs + outs + [ws, O, wsum, back])
        # places behind `keep` are left as they were
        assert (outs[4].view(torch.uint8, (B, S_dst, 4))[:, keep:] == 0xA5).all()
        assert (outs[0].view(torch.uint8, (B, S_dst, kvd))[:, keep:] == 0xA5).all()
