"""Cases of the 8-bit KV cache: its write and read-back, the attention over it
(with the weight each slot received), and the eviction by that weight.

A cache of S slots per batch row holds K' and V [B, S, H_kv, d_h] as e4m3
numbers and, for each block of 64 slots and kv head, one scale each for K' and
V (fp32, a power of two), [B, ceil(S / 64), H_kv]; a slot's value is its
e4m3 number times its block's scale.  pos_cache [B, S] holds the position of
each slot's token, negative where the slot holds none.

  write   tokens' fp16 rows go to slots [end, end + T); a block's scale is the
          smallest 2^e >= 2^-15 whose 448 * 2^e covers its values, and where a
          block already holds tokens its scale only grows, its older numbers
          being rounded again to the larger one.
  attend  softmax attention of T tokens per row over the slots each may see
          (slot s <= end + t, a token in it, on a local layer a position closer
          than the window); with `weights`, the probabilities that every slot
          received are added to weight_sum [B, S].
  evict   of the slots [0, end), the last `recent` and the heaviest others, keep
          in all, move in order to the front of another cache.
"""
import torch

own = False

BLOCK = 64
E4M3_MAX = 448.0
MIN_EXP = -15


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step's append, 4B-shaped local layer (two rows)
        dict(name="write_step", op="write", B=2, T=1, S=32768, end=32767, H_kv=4, d_h=256, pads=False),
        # a chunk of ragged prompts that starts and ends inside a block
        dict(name="write_ragged", op="write", B=3, T=1333, S=9001, end=4001, H_kv=8, d_h=256, pads=True),
        # a long prompt of the 27B-shaped global layer
        dict(name="write_prompt", op="write", B=1, T=65536, S=65536, end=0, H_kv=16, d_h=128, pads=False),
        # decode step, 4B-shaped local layer: the window of a long cache
        dict(name="step_local", op="attend", B=2, T=1, S=32768, end=32767, H=8, H_kv=4, d_h=256, window=1024,
             out="bf16", weights=False, pads=False, gaps=False),
        # decode step, 27B-shaped global layer over the whole long cache
        dict(name="step_global", op="attend", B=1, T=1, S=131072, end=131071, H=32, H_kv=16, d_h=128, window=0,
             out="bf16", weights=False, pads=False, gaps=False),
        # a decode batch, 12B-shaped global layer, rows with padded prompts, weights kept for a later eviction
        dict(name="step_batch_weights", op="attend", B=16, T=1, S=8192, end=7777, H=16, H_kv=8, d_h=256, window=0,
             out="bf16", weights=True, pads=False, gaps=True),
        # four drafted tokens checked at once, 1B-shaped global layer
        dict(name="draft_global", op="attend", B=4, T=4, S=6000, end=5003, H=4, H_kv=1, d_h=256, window=0,
             out="f16", weights=True, pads=True, gaps=True),
        # a prompt's later chunk, 27B-shaped global layer
        dict(name="chunk_global", op="attend", B=1, T=1024, S=32768, end=31744, H=32, H_kv=16, d_h=128, window=0,
             out="bf16", weights=False, pads=False, gaps=False),
        # a padded chunk, 12B-shaped local layer, weights kept
        dict(name="chunk_local_weights", op="attend", B=2, T=515, S=8192, end=3001, H=16, H_kv=8, d_h=256, window=1024,
             out="bf16", weights=True, pads=True, gaps=True),
        # a small cache halved, 1B-shaped
        dict(name="evict_small", op="evict", B=1, S=1024, end=1000, S_dst=1024, H_kv=1, d_h=256, keep=500, recent=64),
        # an odd number of slots kept, 4B-shaped batch
        dict(name="evict_batch", op="evict", B=8, S=20000, end=17777, S_dst=6000, H_kv=4, d_h=256, keep=5003, recent=256),
        # the long cache of the 27B-shaped layer brought down to a quarter
        dict(name="evict_long", op="evict", B=2, S=131072, end=131072, S_dst=32768, H_kv=16, d_h=128, keep=32768, recent=1024),
    ]


SHAPES = [(4, 1, 256), (8, 4, 256), (16, 8, 256), (32, 16, 128), (8, 8, 128), (8, 2, 128)]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    H, H_kv, d_h = rng.choice(SHAPES)
    row = H_kv * d_h
    op = rng.choice(["write", "attend", "attend", "attend", "evict"])
    if op == "write":
        B = _log(rng, 1, 16)
        T = _log(rng, 1, min(65536, (65536 * 2048) // (B * row)))
        end = rng.choice([0, _log(rng, 1, 16384)])
        return dict(op=op, B=B, T=T, S=end + T + rng.randrange(200), end=end, H_kv=H_kv, d_h=d_h,
                    pads=rng.random() < 0.5)
    if op == "evict":
        B = _log(rng, 1, 8)
        end = _log(rng, 300, min(131072, (2 * 131072 * 2048) // (B * row)))
        keep = max(1, int(end * rng.uniform(0.1, 0.25)))
        return dict(op=op, B=B, S=end + rng.randrange(100), end=end, S_dst=keep + rng.randrange(100), H_kv=H_kv,
                    d_h=d_h, keep=keep, recent=rng.randrange(keep + 1))
    long = rng.random() < 0.35
    T = _log(rng, 17, 1024) if long else rng.choice([1, 1, 1, 2, 3, 4, 8])
    B = _log(rng, 1, 4 if long else 16)
    most = 131072 * 2048 // (B * row)
    if long:
        most = min(most, (1000 * 32 * 32768 * 128) // (B * T * H * d_h), 32768)
    end = _log(rng, 200, max(201, min(131071, most) - T))
    return dict(op=op, B=B, T=T, S=end + T + rng.randrange(100), end=end, H=H, H_kv=H_kv, d_h=d_h,
                window=rng.choice([0, 0, 512, 1024]), out=rng.choice(["bf16", "f16"]), weights=rng.random() < 0.4,
                pads=T > 1 and rng.random() < 0.5, gaps=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _scale_exponent(amax):
    """Smallest e >= -15 with amax <= 448 * 2^e (448 = 0.875 * 2^9; amax = m * 2^x, 0.5 <= m < 1)."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)


def _two_to(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e).float()


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _filled(g, B, S, used, H_kv, d_h):
    """A cache's e4m3 numbers and scales with values in slots [0, used): the spread of K' and V over tokens and heads varies by block."""
    nb = _blocks(S)
    num = torch.zeros((B, S, H_kv, d_h), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.zeros((B, nb, H_kv), dtype=torch.float32, device="cuda")
    ub = _blocks(used)
    if ub:
        spread = torch.exp2(torch.randint(-1, 2, (B, ub, H_kv), generator=g, device="cuda").float())
        for b in range(B):
            x = torch.randn((ub * BLOCK, H_kv, d_h), generator=g, device="cuda")
            x[used:] = 0
            x = x.view(ub, BLOCK, H_kv, d_h) * spread[b][:, None, :, None]
            s = _two_to(_scale_exponent(x.abs().amax((1, 3))))
            scale[b, :ub] = s
            num[b, :used] = (x / s[:, None, :, None]).view(ub * BLOCK, H_kv, d_h)[:used].to(torch.float8_e4m3fn)
    return num, scale


def _positions(g, B, S, used, gaps):
    """Stored positions of slots [0, used): counting up; with gaps, each row's prompt ended in padding (negative positions)."""
    pos = torch.full((B, S), -1, dtype=torch.int32, device="cuda")
    slot = torch.arange(used, device="cuda", dtype=torch.int64)[None].expand(B, used)
    hole = torch.zeros((B, 1), dtype=torch.int64, device="cuda")
    if gaps and used > 8:
        hole = torch.randint(0, used // 4 + 1, (B, 1), generator=g, device="cuda")
    first = used // 3
    inside = (slot >= first) & (slot < first + hole)
    p = torch.where(slot >= first, slot - hole, slot)
    pos[:, :used] = torch.where(inside, torch.full_like(p, -1), p).int()
    return pos, hole


def _pads(g, case):
    B, T = case["B"], case["T"]
    if not case["pads"]:
        return None
    return torch.randint(0, (T + 1) // 2 + 1, (B,), generator=g, device="cuda", dtype=torch.int32).clamp(max=T)


def prepare(case, seed):
    g = _gen(seed)
    B, S, end, H_kv, d_h = (case[k] for k in ("B", "S", "end", "H_kv", "d_h"))
    st = dict(case)
    if case["op"] == "write":
        T, kvd = case["T"], H_kv * d_h
        st["K8"], st["K_scale"] = _filled(g, B, S, end, H_kv, d_h)
        st["V8"], st["V_scale"] = _filled(g, B, S, end, H_kv, d_h)
        st["pos"], hole = _positions(g, B, S, end, False)
        # [K'|V] rows as the projections leave them, of varying size over tokens
        size = torch.exp2(torch.randint(-1, 3, (B * T, 1), generator=g, device="cuda").float())
        st["rows"] = (torch.randn((B * T, 2 * kvd), generator=g, device="cuda") * size).half()
        st["seg"] = (end + torch.arange(T, device="cuda", dtype=torch.int32)).repeat(B, 1)
        st["pad"] = _pads(g, case)
        st["first"] = end // BLOCK * BLOCK
        st["n"] = end + T - st["first"]
        st["back"] = torch.empty((B * st["n"], 2 * kvd), dtype=torch.float16, device="cuda")
        return st
    if case["op"] == "evict":
        st["K8"], st["K_scale"] = _filled(g, B, S, end, H_kv, d_h)
        st["V8"], st["V_scale"] = _filled(g, B, S, end, H_kv, d_h)
        st["pos"], _ = _positions(g, B, S, end, True)
        # a few slots hold most of the weight; some tie exactly, some got none at all
        w = torch.exp(2 * torch.randn((B, S), generator=g, device="cuda"))
        u = torch.rand((B, S), generator=g, device="cuda")
        w = torch.where(u < 0.1, torch.zeros_like(w), torch.where(u < 0.4, torch.round(w * 8) / 8, w))
        st["wsum"] = w
        keep, S_dst = case["keep"], case["S_dst"]
        for n in ("K8", "V8"):
            st[n + "_dst"] = torch.zeros((B, S_dst, H_kv, d_h), dtype=torch.float8_e4m3fn, device="cuda")
        for n in ("K_scale", "V_scale"):
            st[n + "_dst"] = torch.zeros((B, _blocks(S_dst), H_kv), dtype=torch.float32, device="cuda")
        st["pos_dst"] = torch.full((B, S_dst), -1, dtype=torch.int32, device="cuda")
        st["wsum_dst"] = torch.zeros((B, S_dst), dtype=torch.float32, device="cuda")
        st["kept"] = torch.empty((B, keep), dtype=torch.int32, device="cuda")
        st["back"] = torch.empty((B * keep, 2 * H_kv * d_h), dtype=torch.float16, device="cuda")
        return st
    T, H = case["T"], case["H"]
    used = end + T
    st["K8"], st["K_scale"] = _filled(g, B, S, used, H_kv, d_h)
    st["V8"], st["V_scale"] = _filled(g, B, S, used, H_kv, d_h)
    st["pos"], hole = _positions(g, B, S, end, case["gaps"])
    st["seg"] = (end - hole + torch.arange(T, device="cuda", dtype=torch.int64)[None]).int().contiguous()
    st["pad"] = _pads(g, case)
    valid = torch.full((B, 1), T, device="cuda")
    if st["pad"] is not None:
        valid = T - st["pad"][:, None]
    st["pos"][:, end:used] = torch.where(torch.arange(T, device="cuda")[None] < valid, st["seg"],
                                         torch.full_like(st["seg"], -1))
    # Q' with the query scale in it: logits of a spread of about 1.5
    st["Q"] = (torch.randn((B, T, H, d_h), generator=g, device="cuda") * (1.5 * d_h ** -0.5)).half()
    st["wsum"] = torch.rand((B, S), generator=g, device="cuda") if case["weights"] else None
    st["O"] = torch.empty((B, T, H, d_h), dtype=torch.float16 if case["out"] == "f16" else torch.bfloat16,
                          device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    if st["op"] == "write":
        return _run_write(st)
    if st["op"] == "evict":
        return _run_evict(st)
    return _run_attend(st)


def _run_write(st):
    B, T, S, end, H_kv, d_h = (st[k] for k in ("B", "T", "S", "end", "H_kv", "d_h"))
    kvd = H_kv * d_h
    if own:
        import transformer_attention_gb300 as G3
        G3.gemma3_kv_cache8_write(st["rows"], st["rows"][:, kvd:], 2 * kvd, st["seg"], st["pad"], B, T, S, end, H_kv,
                                  d_h, st["K8"], st["V8"], st["K_scale"], st["V_scale"], st["pos"])
        G3.gemma3_kv_cache8_read(st["K8"], st["V8"], st["K_scale"], st["V_scale"], B, S, st["first"], st["n"], H_kv,
                                 d_h, st["back"], st["back"][:, kvd:], 2 * kvd)
        return {"values": st["back"], "K_scale": st["K_scale"], "V_scale": st["V_scale"], "pos": st["pos"]}
    first, n = st["first"], st["n"]
    t = torch.arange(T, device="cuda")
    live = torch.ones((B, T), dtype=torch.bool, device="cuda") if st["pad"] is None else t[None] < T - st["pad"][:, None]
    rows = st["rows"].view(B, T, 2, H_kv, d_h)
    back = []
    for i, name in enumerate(("K", "V")):
        num, scale = st[name + "8"], st[name + "_scale"]
        x = torch.where(live[..., None, None], rows[:, :, i].float(), 0.0)
        nb = _blocks(n)
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, end - first, nb * BLOCK - n))
        s = _two_to(_scale_exponent(x.view(B, nb, BLOCK, H_kv, d_h).abs().amax((2, 4))))
        b0 = first // BLOCK
        if end > first:  # a block that holds tokens already: its scale only grows
            s[:, 0] = torch.maximum(s[:, 0], scale[:, b0])
            x[:, :end - first] = num[:, first:end].float() * scale[:, b0, None, :, None]
        q = (x.view(B, nb, BLOCK, H_kv, d_h) / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
        num[:, first:first + n] = q.view(B, nb * BLOCK, H_kv, d_h)[:, :n]
        scale[:, b0:b0 + nb] = s
        v = q.float() * s[:, :, None, :, None]
        back.append(v.view(B, nb * BLOCK, kvd)[:, :n])
    st["pos"][:, end:end + T] = torch.where(live, st["seg"], -1)
    return {"values": torch.cat(back, 2).view(B * n, 2 * kvd).half(), "K_scale": st["K_scale"],
            "V_scale": st["V_scale"], "pos": st["pos"]}


def _values(num, scale, n):
    """The first n slots' values, fp32 [B, H_kv, n, d_h]."""
    s = scale.repeat_interleave(BLOCK, 1)[:, :n]
    return (num[:, :n].float() * s[..., None]).transpose(1, 2)


def _seen(st):
    """[B, T, hi]: the slots that each token sees."""
    B, T, end = st["B"], st["T"], st["end"]
    hi = end + T
    t = torch.arange(T, device="cuda")
    pos = st["pos"][:, None, :hi]
    seen = (pos >= 0) & (torch.arange(hi, device="cuda")[None] <= end + t[:, None])[None]
    if st["window"] > 0:
        seen = seen & ((st["seg"][:, :, None] - pos).abs() < st["window"])
    if st["pad"] is not None:
        seen = seen & (t[None] < T - st["pad"][:, None])[:, :, None]
    return seen


def _run_attend(st):
    B, T, S, end, H, H_kv, d_h = (st[k] for k in ("B", "T", "S", "end", "H", "H_kv", "d_h"))
    if own:
        import transformer_attention_gb300 as G3
        if "ws" not in st:
            st["ws_bytes"] = G3.gemma3_cached8_attention_workspace_size(B, T, S, H, H_kv, d_h,
                                                                        st["wsum"] is not None)
            st["ws"] = torch.empty(max(256, st["ws_bytes"]), dtype=torch.uint8, device="cuda")
        G3.gemma3_cached8_attention(st["Q"], st["K8"], st["V8"], st["K_scale"], st["V_scale"], st["pos"], st["seg"],
                                    st["pad"], st["O"], G3.GEMMA3_F16 if st["out"] == "f16" else G3.GEMMA3_BF16,
                                    st["wsum"], B, T, S, end, H, H_kv, d_h, st["window"], st["ws"], st["ws_bytes"])
        return {"O": st["O"], "weight_sum": st["wsum"]}
    hi, G = end + T, H // H_kv
    k, v = _values(st["K8"], st["K_scale"], hi), _values(st["V8"], st["V_scale"], hi)
    q = st["Q"].float().view(B, T, H_kv, G, d_h).permute(0, 2, 1, 3, 4).reshape(B, H_kv, T * G, d_h)
    seen = _seen(st)[:, None, :, None, :]                                   # [B, 1, T, 1, hi]
    x = torch.matmul(q, k.transpose(2, 3)).view(B, H_kv, T, G, hi)
    x = torch.where(seen, x, float("-inf"))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)                           # a row that sees nothing stays all zero
    p = torch.exp(x - m)
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.view(B, H_kv, T * G, hi), v).view(B, H_kv, T, G, d_h)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, H, d_h).to(st["O"].dtype)
    if st["wsum"] is not None:
        st["wsum"][:, :hi] += p.sum((1, 2, 3))
    return {"O": o, "weight_sum": st["wsum"]}


def _run_evict(st):
    B, S, end, H_kv, d_h, keep, recent, S_dst = (st[k] for k in ("B", "S", "end", "H_kv", "d_h", "keep", "recent", "S_dst"))
    kvd = H_kv * d_h
    out = {"K_scale": st["K_scale_dst"], "V_scale": st["V_scale_dst"], "pos": st["pos_dst"],
           "weight_sum": st["wsum_dst"]}
    if own:
        import transformer_attention_gb300 as G3
        G3.gemma3_kv_cache8_evict(st["K8"], st["V8"], st["K_scale"], st["V_scale"], st["pos"], st["wsum"], B, S, end,
                                  H_kv, d_h, keep, recent, st["K8_dst"], st["V8_dst"], st["K_scale_dst"],
                                  st["V_scale_dst"], st["pos_dst"], st["wsum_dst"], st["kept"], S_dst)
        G3.gemma3_kv_cache8_read(st["K8_dst"], st["V8_dst"], st["K_scale_dst"], st["V_scale_dst"], B, S_dst, 0, keep,
                                 H_kv, d_h, st["back"], st["back"][:, kvd:], 2 * kvd)
        return dict(out, values=st["back"], kept=st["kept"])
    slot = torch.arange(end, device="cuda")[None]
    w, held = st["wsum"][:, :end], st["pos"][:, :end] >= 0
    key = torch.where(held, torch.where(slot >= end - recent, float("inf"), w), float("-inf"))
    order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :keep]
    order = torch.nn.functional.pad(order, (0, keep - order.shape[1]))
    ok = (torch.arange(keep, device="cuda")[None] < held.sum(1, keepdim=True))
    kept = torch.sort(torch.where(ok, order, S), dim=1)[0]
    have = kept < S
    src = torch.where(have, kept, 0)
    nb = _blocks(keep)
    back = []
    for name in ("K", "V"):
        at = src[:, :, None, None].expand(B, keep, H_kv, d_h)
        s = st[name + "_scale"].gather(1, (src // BLOCK)[..., None].expand(B, keep, H_kv))
        x = st[name + "8"].view(torch.uint8).gather(1, at).view(torch.float8_e4m3fn).float() * s[..., None]
        x = torch.where(have[..., None, None], x, 0.0)
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, nb * BLOCK - keep)).view(B, nb, BLOCK, H_kv, d_h)
        s = _two_to(_scale_exponent(x.abs().amax((2, 4))))
        q = (x / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
        st[name + "8_dst"][:, :keep] = q.view(B, nb * BLOCK, H_kv, d_h)[:, :keep]
        st[name + "_scale_dst"][:, :nb] = s
        back.append((q.float() * s[:, :, None, :, None]).view(B, nb * BLOCK, kvd)[:, :keep])
    st["pos_dst"][:, :keep] = torch.where(have, st["pos"].gather(1, src), -1)
    st["wsum_dst"][:, :keep] = torch.where(have, st["wsum"].gather(1, src), 0.0)
    return dict(out, values=torch.cat(back, 2).view(B * keep, 2 * kvd).half(),
                kept=torch.where(have, kept, -1).int())


# ------------------------------------------------------------------ least work
def work(case):
    B, end, H_kv, d_h = (case[k] for k in ("B", "end", "H_kv", "d_h"))
    row = 2 * H_kv * d_h                                        # K' and V of one slot, in numbers
    if case["op"] == "write":
        T = case["T"]
        n = end + T - end // BLOCK * BLOCK
        # fp16 rows in, 8-bit slots out; 8-bit slots in, fp16 values out; a block's scale is far less
        return {"bytes": B * row * (T * 3 + n * 3) + 8 * B * T, "flops": 4 * B * T * row}
    if case["op"] == "evict":
        keep = case["keep"]
        # positions and weights of every slot, the kept slots moved, then read back
        return {"bytes": B * (8 * end + keep * (2 * row + 3 * row + 12)), "flops": 4 * B * keep * row}
    T, H = case["T"], case["H"]
    hi = end + T
    seen = min(hi, case["window"] + T) if case["window"] else hi   # slots that some token sees, at most
    pairs = T * hi - T * (T - 1) // 2
    if case["window"]:
        pairs = min(pairs, T * case["window"])
    nbytes = B * (seen * row + 4 * seen + 4 * T * H * d_h + (8 * seen if case["weights"] else 0))
    return {"bytes": nbytes, "flops": B * 4 * pairs * H * d_h}


# ------------------------------------------------------------------ in 64 bits
def _table():
    """The 256 numbers of e4m3: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    code = torch.arange(256, device="cuda")
    e, m = (code >> 3) & 15, (code & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * _power(e - 7))
    mag = torch.where((code & 127) == 127, float("nan"), mag)
    return torch.where(code >= 128, -mag, mag)


def _power(e):
    """2^e in 64 bits, without the last bit that a device's pow may be off by."""
    return torch.pow(2.0, e.double()).float().double()


def _rounded(x):
    """x to the nearest e4m3 number, ties to the even one (|x| <= 448)."""
    # frexp: |x| = m * 2^e with 0.5 <= m < 1, so the numbers around x are 2^(e - 4) apart, and 2^-9 below 2^-6
    step = _power(torch.frexp(x.abs().clamp(min=2.0 ** -6))[1] - 4)
    return torch.round(x / step) * step


def _covering(amax):
    """The smallest 2^e >= 2^-15 with amax <= 448 * 2^e, by trying them all."""
    tries = _power(torch.arange(-15, 17, device="cuda"))
    fits = amax[..., None] <= 448.0 * tries
    return tries[fits.double().argmax(-1)]


def exact(case, seed):
    st = prepare(case, seed)
    B, end, H_kv, d_h = (case[k] for k in ("B", "end", "H_kv", "d_h"))
    table = _table()

    def slot(name, b, at):
        """Values [len(at), H_kv, d_h] of row b's slots `at` in 64 bits."""
        v = table[st[name + "8"][b].view(torch.uint8)[at].long()]
        return v * st[name + "_scale"][b][at // 64].double()[..., None]

    def stored(x):
        """Values as a cache holds them when `x` [n, H_kv, d_h] fills blocks from their start; and the blocks' scales."""
        n = x.shape[0]
        nb = -(-n // 64)
        full = torch.zeros((nb * 64, H_kv, d_h), dtype=torch.float64, device="cuda")
        full[:n] = x
        s = _covering(full.view(nb, 64, H_kv, d_h).abs().amax((1, 3)))
        each = s.repeat_interleave(64, 0)[:n, :, None]
        return _rounded(x / each) * each, s

    if case["op"] == "write":
        T, first, n = case["T"], st["first"], st["n"]
        vals = torch.empty((B, n, 2, H_kv, d_h), dtype=torch.float64, device="cuda")
        scales = {}
        for b in range(B):
            live = T - (0 if st["pad"] is None else int(st["pad"][b]))
            for i, name in enumerate(("K", "V")):
                new = st["rows"].view(B, T, 2, H_kv, d_h)[b, :, i].double()
                new[live:] = 0
                old = slot(name, b, torch.arange(first, end, device="cuda"))
                sc = scales.setdefault(name, st[name + "_scale"].double().clone())
                held = sc[b, first // 64].clone()
                v, s = stored(torch.cat([torch.zeros_like(old), new]))
                if end > first:
                    s[0] = torch.maximum(s[0], held)
                    top = min(64, n)
                    x = torch.cat([old, new])[:top]
                    v[:top] = _rounded(x / s[0][None, :, None]) * s[0][None, :, None]
                vals[b, :, i] = v
                sc[b, first // 64:first // 64 + s.shape[0]] = s
        return {"values": vals.view(B * n, 2 * H_kv * d_h), "K_scale": scales["K"], "V_scale": scales["V"], "pos": None}

    if case["op"] == "evict":
        keep, recent, S_dst = case["keep"], case["recent"], case["S_dst"]
        vals = torch.zeros((B, keep, 2, H_kv, d_h), dtype=torch.float64, device="cuda")
        scales = {n: torch.zeros((B, -(-S_dst // 64), H_kv), dtype=torch.float64, device="cuda") for n in ("K", "V")}
        wd = torch.zeros((B, S_dst), dtype=torch.float64, device="cuda")
        for b in range(B):
            held = torch.nonzero(st["pos"][b, :end] >= 0).view(-1)
            late, early = held[held >= end - recent], held[held < end - recent]
            w = st["wsum"][b].double()
            heavy = early[torch.sort(-w[early], stable=True)[1]][:keep - late.numel()]
            at = torch.sort(torch.cat([late, heavy]))[0]
            wd[b, :at.numel()] = w[at]
            for i, name in enumerate(("K", "V")):
                x = torch.zeros((keep, H_kv, d_h), dtype=torch.float64, device="cuda")
                x[:at.numel()] = slot(name, b, at)
                vals[b, :, i], s = stored(x)
                scales[name][b, :s.shape[0]] = s
        return {"K_scale": scales["K"], "V_scale": scales["V"], "pos": None, "weight_sum": wd,
                "values": vals.view(B * keep, 2 * H_kv * d_h), "kept": None}

    T, H, hi = case["T"], case["H"], end + case["T"]
    G = H // H_kv
    if 4 * B * H * T * hi * d_h > 1.2e13:
        return None
    O = torch.zeros((B, T, H, d_h), dtype=torch.float64, device="cuda")
    wsum = None if st["wsum"] is None else st["wsum"].double()
    slots = torch.arange(hi, device="cuda")
    for b in range(B):
        live = T - (0 if st["pad"] is None else int(st["pad"][b]))
        for j in range(H_kv):
            k = table[st["K8"][b, :hi, j].view(torch.uint8).long()] * st["K_scale"][b, slots // 64, j].double()[:, None]
            v = table[st["V8"][b, :hi, j].view(torch.uint8).long()] * st["V_scale"][b, slots // 64, j].double()[:, None]
            for t0 in range(0, live, 256):
                t = torch.arange(t0, min(t0 + 256, live), device="cuda")
                p = st["pos"][b, :hi].long()
                see = (p >= 0)[None] & (slots[None] <= end + t[:, None])
                if case["window"]:
                    q_at = st["seg"][b, t].long()[:, None]
                    see = see & (p[None] > q_at - case["window"]) & (p[None] < q_at + case["window"])
                for g in range(G):
                    x = st["Q"][b, t, j * G + g].double() @ k.T
                    x = x.masked_fill(~see, float("-inf"))
                    w = torch.softmax(x, -1).nan_to_num(0.0)
                    O[b, t, j * G + g] = w @ v
                    if wsum is not None:
                        wsum[b, :hi] += w.sum(0)
    return {"O": O, "weight_sum": wsum}
