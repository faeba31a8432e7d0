"""Cases of the paged KV cache operators: the append with norm and rotation, the
attention of drafted trees, single tokens and prompt chunks over the pages, and
the commit of the accepted tokens.

A layer's cache is a pool of pages, K_pages and V_pages [n_pages, P, H_kv, d_h]
fp16.  Slot s of sequence b lies in page page_table[b, s / P]; lens[b] slots are
filled and a filled slot's position is its number.  A call's new tokens are rows
row_start[b] .. row_start[b + 1] of packed arrays.  Token i of sequence b goes to
slot lens[b] + i; its parent is another of the sequence's new tokens, earlier than
itself, or -1: the filled slots.  Without parents each token follows the one
before it.  A token's position is lens[b] + its depth.

  append  Q and K rows get RMSNorm over d_h with (1 + gamma), RoPE at the token's
          position, Q the query scale; K' and V rows go to the tokens' slots.
  attend  softmax attention of every token over the filled slots (on a local
          layer those closer than the window), its ancestors and itself.
  commit  of each sequence's new tokens, the accepted ones move in order to the
          slots from lens[b] on, in every layer; the new length is lens[b] + count.
"""
import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------ cases
def listed():
    return [
        # drafted trees of a decode batch, 12B-shaped global layer, small pages
        dict(name="append_trees", op="append", B=16, n_lo=5, n_hi=12, tree=True, len_lo=0, len_hi=700, P=16, H=16,
             H_kv=8, d_h=256, base=1e6, scale=8.0),
        # prompts of uneven lengths packed into one call, 27B-shaped global layer
        dict(name="append_prompts", op="append", B=5, n_lo=1201, n_hi=6007, tree=False, len_lo=0, len_hi=2000, P=64,
             H=32, H_kv=16, d_h=128, base=1e6, scale=8.0),
        # decode step of two sequences, 4B-shaped local layer: the window of a long cache
        dict(name="step_local", op="attend", B=2, n_lo=1, n_hi=1, tree=False, len_lo=32767, len_hi=32767, P=64, H=8,
             H_kv=4, d_h=256, window=1024, out="bf16"),
        # decode step, 27B-shaped global layer over a long cache
        dict(name="step_global", op="attend", B=1, n_lo=1, n_hi=1, tree=False, len_lo=131071, len_hi=131071, P=64,
             H=32, H_kv=16, d_h=128, window=0, out="bf16"),
        # decode batch of sequences of very uneven lengths, 12B-shaped global layer, small pages
        dict(name="step_batch", op="attend", B=32, n_lo=1, n_hi=1, tree=False, len_lo=100, len_hi=16000, P=16, H=16,
             H_kv=8, d_h=256, window=0, out="bf16"),
        # one sequence's small tree of drafted tokens, 1B-shaped global layer
        dict(name="tree_small", op="attend", B=1, n_lo=7, n_hi=7, tree=True, len_lo=5003, len_hi=5003, P=32, H=4,
             H_kv=1, d_h=256, window=0, out="f16"),
        # large trees of a batch, 27B-shaped global layer
        dict(name="tree_batch", op="attend", B=8, n_lo=33, n_hi=64, tree=True, len_lo=1000, len_hi=16384, P=16, H=32,
             H_kv=16, d_h=128, window=0, out="bf16"),
        # trees on a local layer, 12B-shaped, large pages
        dict(name="tree_local", op="attend", B=6, n_lo=15, n_hi=33, tree=True, len_lo=300, len_hi=9000, P=128, H=16,
             H_kv=8, d_h=256, window=1024, out="bf16"),
        # a prompt's later chunk, 27B-shaped global layer
        dict(name="chunk_global", op="attend", B=1, n_lo=1024, n_hi=1024, tree=False, len_lo=31744, len_hi=31744,
             P=64, H=32, H_kv=16, d_h=128, window=0, out="bf16"),
        # chunks of some sequences beside single tokens of others, 4B-shaped global layer
        dict(name="mixed", op="attend", B=10, n_lo=1, n_hi=1500, tree=False, len_lo=1, len_hi=9000, P=32, H=8, H_kv=4,
             d_h=256, window=0, out="bf16"),
        # a few accepted tokens a sequence, six 12B-shaped layers
        dict(name="commit_step", op="commit", B=4, n_lo=3, n_hi=8, len_lo=10, len_hi=400, P=16, H_kv=8, d_h=256,
             layers=6),
        # a large batch's accepted paths, six 27B-shaped layers
        dict(name="commit_batch", op="commit", B=64, n_lo=17, n_hi=64, len_lo=10, len_hi=500, P=64, H_kv=16, d_h=128,
             layers=6),
    ]


SHAPES = [(4, 1, 256), (8, 4, 256), (16, 8, 256), (32, 16, 128), (8, 8, 128), (8, 2, 128)]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    H, H_kv, d_h = rng.choice(SHAPES)
    P = rng.choice([16, 32, 64, 128, 256])
    op = rng.choice(["append", "attend", "attend", "attend", "commit"])
    c = dict(op=op, P=P, H_kv=H_kv, d_h=d_h)
    if op == "commit":
        hi = _log(rng, 2, 64)
        return dict(c, B=_log(rng, 1, 48), n_lo=rng.randint(1, hi), n_hi=hi, len_lo=0, len_hi=_log(rng, 10, 500),
                    layers=_log(rng, 1, 6))
    c["H"] = H
    tree = rng.random() < 0.4
    if op == "append":
        hi = _log(rng, 1, 64 if tree else 6000)
        return dict(c, B=_log(rng, 1, 32 if tree else 4), n_lo=_log(rng, 1, hi), n_hi=hi, tree=tree, len_lo=0,
                    len_hi=_log(rng, 10, 2000), base=rng.choice([1e4, 1e6]), scale=rng.choice([1.0, 8.0]))
    kind = "tree" if tree else rng.choice(["step", "step", "chunk", "mixed"])
    B = 1 if kind == "chunk" else _log(rng, 2, 12) if kind == "mixed" else _log(rng, 1, 32)
    most = max(300, min(131071 if kind == "step" else 16384 if kind == "tree" else 9000, 131072 * 2048 // (B * H_kv * d_h)))
    top = _log(rng, 200, most)
    hi = {"tree": _log(rng, 2, 64), "step": 1, "chunk": _log(rng, 17, 1024), "mixed": _log(rng, 20, 1000)}[kind]
    return dict(c, B=B, n_lo=1 if kind in ("step", "mixed") else _log(rng, 1, hi), n_hi=hi, tree=tree,
                len_lo=_log(rng, 1, top), len_hi=top, window=rng.choice([0, 0, 512, 1024]),
                out=rng.choice(["bf16", "f16"]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 31)


def _spread(lo, hi, B):
    """B whole numbers of [lo, hi], spread over their logarithm; the last is hi."""
    return [hi if k == B - 1 else min(hi, max(lo, round((lo + 1) * ((hi + 1) / (lo + 1)) ** ((k + 0.5) / B) - 1)))
            for k in range(B)]


def prepare(case, seed):
    g = _gen(seed)
    B, P, H_kv, d_h = case["B"], case["P"], case["H_kv"], case["d_h"]
    L = case.get("layers", 1)
    st = dict(case)
    # which sequence has which length, and how many new tokens, goes by the seed
    lens, n = (torch.tensor(_spread(case[x + "_lo"], case[x + "_hi"], B), device="cuda")[
        torch.randperm(B, generator=g, device="cuda")] for x in ("len", "n"))
    st["lens"] = lens.int()
    st["row_start"] = torch.nn.functional.pad(n.cumsum(0), (1, 0)).int()
    st["M"], st["T_max"], st["S_max"] = int(n.sum()), int(n.max()), int((lens + n).max())
    st["max_pages"] = -(-(case["len_hi"] + case["n_hi"]) // P)
    # pages in no order; entries behind a sequence's last page hold nothing
    need = (lens + n + P - 1) // P
    st["n_pages"] = int(((lens + P - 1) // P + (n + P - 1) // P).sum()) + 3
    table = torch.full((B, st["max_pages"]), -1, dtype=torch.int32, device="cuda")
    at = torch.arange(st["max_pages"], device="cuda")[None] < need[:, None]
    table[at] = torch.randperm(st["n_pages"], generator=g, device="cuda")[:int(need.sum())].int()
    st["page_table"] = table
    shape = (L, st["n_pages"], P, H_kv, d_h)
    for name in ("K_pages", "V_pages"):
        pool = torch.empty(shape, dtype=torch.float16, device="cuda")
        for layer in range(L):
            pool[layer] = torch.randn(shape[1:], generator=g, device="cuda", dtype=torch.float16)
        st[name] = pool if case["op"] == "commit" else pool[0]
    st["parents"] = None
    if case["op"] == "commit" or case["tree"]:
        i = (torch.arange(st["M"], device="cuda") -
             st["row_start"][:-1].long().repeat_interleave(n))          # a token's number in its sequence
        back = torch.randint(1, 5, (st["M"],), generator=g, device="cuda")
        st["parents"] = (i - back).clamp(min=-1).int()                   # drafted breadth first: parents a little earlier
    if case["op"] == "commit":
        # an accepted path of some depth: numbers of tokens, ascending
        T = st["T_max"]
        keep = (torch.rand((B, T), generator=g, device="cuda") < 0.4) & (torch.arange(T, device="cuda")[None] < n[:, None])
        st["counts"] = keep.sum(1).int()
        st["accepted"] = torch.sort(torch.where(keep, torch.arange(T, device="cuda")[None], T), 1)[0].int()
        st["accepted"] = torch.where(st["accepted"] == T, -1, st["accepted"]).contiguous()
        st["new_lens"] = torch.zeros_like(st["lens"])
        return st
    M, H = st["M"], case["H"]
    if case["op"] == "append":
        size = torch.exp2(torch.randint(-1, 3, (M, 1), generator=g, device="cuda").float())
        st["Q"] = (torch.randn((M, H * d_h), generator=g, device="cuda") * size).half()
        st["KV"] = (torch.randn((M, 2 * H_kv * d_h), generator=g, device="cuda") * size).half()
        for name in ("gamma_q", "gamma_k"):
            st[name] = (torch.randn(d_h, generator=g, device="cuda") * 0.1 ** 0.5).bfloat16()
        st["Q_out"] = torch.empty_like(st["Q"])
        return st
    # Q' with the query scale in it: logits of a spread of about 1.5
    st["Q"] = (torch.randn((M, H, d_h), generator=g, device="cuda") * (1.5 * d_h ** -0.5)).half()
    st["O"] = torch.empty((M, H, d_h), dtype=torch.float16 if case["out"] == "f16" else torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _run_own(st)
    return {"append": _run_append, "attend": _run_attend, "commit": _run_commit}[st["op"]](st)


def _run_own(st):
    import transformer_attention_gb300 as G3
    if "batch" not in st:
        st["batch"] = G3.paged_batch(st["lens"], st["row_start"], st["page_table"], rows=st["M"], T_max=st["T_max"],
                                     page_size=st["P"], n_pages=st["n_pages"],
                                     parents=None if st["op"] == "commit" else st["parents"])
    batch = st["batch"]
    if st["op"] == "append":
        kvd = st["H_kv"] * st["d_h"]
        G3.gemma3_paged_append(batch, st["Q"], st["H"] * st["d_h"], st["Q_out"], st["H"] * st["d_h"], st["KV"],
                               st["KV"][:, kvd:], 2 * kvd, st["gamma_q"], st["gamma_k"], st["H"], st["H_kv"],
                               st["d_h"], st["base"], st["scale"], st["d_h"] ** -0.5, st["K_pages"], st["V_pages"])
        return {"Q": st["Q_out"], "K_pages": st["K_pages"], "V_pages": st["V_pages"]}
    if st["op"] == "commit":
        G3.gemma3_paged_commit(batch, st["accepted"], st["counts"], st["layers"], st["H_kv"], st["d_h"],
                               st["K_pages"], st["V_pages"], st["new_lens"])
        return {"K_pages": st["K_pages"], "V_pages": st["V_pages"], "lens": st["new_lens"]}
    if "ws" not in st:
        st["ws_bytes"] = G3.gemma3_paged_attention_workspace_size(batch, st["H"], st["H_kv"], st["d_h"])
        st["ws"] = torch.empty(max(256, st["ws_bytes"]), dtype=torch.uint8, device="cuda")
    G3.gemma3_paged_attention(batch, st["Q"], st["K_pages"], st["V_pages"], st["O"],
                              G3.GEMMA3_F16 if st["out"] == "f16" else G3.GEMMA3_BF16, st["H"], st["H_kv"], st["d_h"],
                              st["window"], st["ws"], st["ws_bytes"])
    return {"O": st["O"]}


def _tokens(st):
    """Of each row: its sequence, its number there and its slot's row of the pool."""
    row = torch.arange(st["M"], device="cuda")
    start = st["row_start"].long()
    b = torch.searchsorted(start, row, right=True) - 1
    i = row - start[b]
    return b, i, _pool_row(st, b, st["lens"].long()[b] + i)


def _pool_row(st, b, slot):
    P = st["P"]
    page = st["page_table"][b, (slot // P).clamp(max=st["max_pages"] - 1)].long().clamp(min=0)
    return page * P + slot % P


def _closure(st, b, i):
    """[B, T, T]: whether the second token is the first or an ancestor of it."""
    B, T = st["B"], st["T_max"]
    step = torch.eye(T, device="cuda").repeat(B, 1, 1)
    step[b, i, st["parents"].long().clamp(min=0)] += (st["parents"] >= 0).float()
    return torch.linalg.matrix_power(step, T) > 0     # paths of at most T steps


def _run_append(st):
    H, H_kv, d_h, M = st["H"], st["H_kv"], st["d_h"], st["M"]
    b, i, at = _tokens(st)
    depth = i
    if st["parents"] is not None:
        depth = _closure(st, b, i).sum(2)[b, i] - 1
    pos = (st["lens"].long()[b] + depth).double()
    freq = torch.tensor(st["base"], dtype=torch.float64, device="cuda") ** (
        -2.0 * torch.arange(d_h // 2, device="cuda", dtype=torch.float64) / d_h)
    angle = (pos / st["scale"])[:, None, None] * freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()

    def heads(rows, n, gamma):
        x = rows.float().view(M, n, d_h)
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (1 + gamma.float())
        a, c = x[..., :d_h // 2], x[..., d_h // 2:]
        return torch.cat([a * cos - c * sin, c * cos + a * sin], -1)

    st["Q_out"].copy_((heads(st["Q"], H, st["gamma_q"]) * d_h ** -0.5).reshape(M, H * d_h))
    kvd = H_kv * d_h
    st["K_pages"].view(-1, H_kv, d_h)[at] = heads(st["KV"][:, :kvd], H_kv, st["gamma_k"]).half()
    st["V_pages"].view(-1, H_kv, d_h)[at] = st["KV"][:, kvd:].reshape(M, H_kv, d_h)
    return {"Q": st["Q_out"], "K_pages": st["K_pages"], "V_pages": st["V_pages"]}


def _run_attend(st):
    B, T, S, M, H, H_kv, d_h = (st[k] for k in ("B", "T_max", "S_max", "M", "H", "H_kv", "d_h"))
    G = H // H_kv
    b, i, _ = _tokens(st)
    lens = st["lens"].long()
    n = st["row_start"].long().diff()
    slot = torch.arange(S, device="cuda")
    first = 0
    if st["window"]:   # slots below every token's window are not looked at
        first = max(0, int(st["len_lo"]) - st["window"] + 1)
        slot = slot[first:]
    rows = _pool_row(st, torch.arange(B, device="cuda")[:, None], slot[None])
    held = (slot[None] < (lens + n)[:, None])[..., None, None]
    k, v = (torch.where(held, st[x].view(-1, H_kv, d_h)[rows].float(), 0.0).permute(0, 2, 1, 3)
            for x in ("K_pages", "V_pages"))                                           # [B, H_kv, S, d_h]
    q = torch.zeros((B, T, H, d_h), device="cuda")
    q[b, i] = st["Q"].float()
    q = q.view(B, T, H_kv, G, d_h).permute(0, 2, 1, 3, 4).reshape(B, H_kv, T * G, d_h)
    number = slot[None] - lens[:, None]                                                # of a new token, where >= 0
    t = torch.arange(T, device="cuda")
    if st["parents"] is None:
        depth = t.expand(B, T)
        new = (number >= 0)[:, None] & (number[:, None] <= t[:, None])
    else:
        closure = _closure(st, b, i)
        depth = closure.sum(2) - 1
        new = torch.gather(closure, 2, number.clamp(0, T - 1)[:, None].expand(B, T, slot.numel()))
        new = new & (number >= 0)[:, None] & (number < T)[:, None]
    seen = new | (number < 0)[:, None]
    if st["window"]:
        at = torch.where(number < 0, slot[None],
                         lens[:, None] + torch.gather(depth, 1, number.clamp(0, T - 1)))
        seen = seen & (at[:, None] > (lens[:, None] + depth)[:, :, None] - st["window"])
    x = torch.matmul(q, k.transpose(2, 3)).view(B, H_kv, T, G, slot.numel())
    x = torch.where(seen[:, None, :, None], x, float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-3e38))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.view(B, H_kv, T * G, slot.numel()), v).view(B, H_kv, T, G, d_h)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, H, d_h)
    st["O"].copy_(o[b, i])
    return {"O": st["O"]}


def _run_commit(st):
    B, T, L, H_kv, d_h = (st[k] for k in ("B", "T_max", "layers", "H_kv", "d_h"))
    b = torch.arange(B, device="cuda")[:, None].expand(B, T)
    to = torch.arange(T, device="cuda")[None].expand(B, T)
    lens = st["lens"].long()[:, None]
    ok = to < st["counts"][:, None]
    src = _pool_row(st, b, lens + st["accepted"].long().clamp(min=0))
    dst = _pool_row(st, b, lens + to)
    src, dst = src[ok], dst[ok]
    for_layers = lambda x: x.view(L, -1, H_kv, d_h)  # noqa: E731
    for_layers(st["K_pages"])[:, dst] = for_layers(st["K_pages"])[:, src]
    for_layers(st["V_pages"])[:, dst] = for_layers(st["V_pages"])[:, src]
    st["new_lens"].copy_(st["lens"] + st["counts"])
    return {"K_pages": st["K_pages"], "V_pages": st["V_pages"], "lens": st["new_lens"]}


# ------------------------------------------------------------------ least work
def work(case):
    B, H_kv, d_h = case["B"], case["H_kv"], case["d_h"]
    row = 4 * H_kv * d_h                                        # bytes of a slot's K' and V
    n = sum(_spread(case["n_lo"], case["n_hi"], B))
    if case["op"] == "commit":
        return {"bytes": 2 * 0.4 * n * row * case["layers"] + 8 * B, "flops": 0}
    H = case["H"]
    if case["op"] == "append":
        return {"bytes": n * (4 * H * d_h + 2 * row), "flops": 12 * n * (H + H_kv) * d_h}
    lens = _spread(case["len_lo"], case["len_hi"], B)
    seen = [min(x, case["window"]) if case["window"] else x for x in lens]   # filled slots that a token sees
    # which sequence has how many new tokens goes by the seed: the mean; a token sees half of the new ones
    pairs = n * (sum(seen) + 0.5 * (n - B)) / B + n
    return {"bytes": (sum(seen) + n) * row + 4 * n * H * d_h, "flops": 4 * H * d_h * pairs}


# ------------------------------------------------------------------ in 64 bits
def _ancestors(parents):
    """For each of a sequence's new tokens the set of its ancestors and itself."""
    found = []
    for i, p in enumerate(parents):
        found.append({i} | (found[p] if p >= 0 else set()))
    return found


def exact(case, seed):
    st = prepare(case, seed)
    P, H_kv, d_h = case["P"], case["H_kv"], case["d_h"]
    lens, start, table = st["lens"].tolist(), st["row_start"].tolist(), st["page_table"].long()

    def places(b, slots):
        """Page and offset of a sequence's slots."""
        s = torch.as_tensor(slots, device="cuda", dtype=torch.long)
        return table[b].index_select(0, torch.div(s, P, rounding_mode="floor")), torch.remainder(s, P)

    if case["op"] == "commit":
        pools = {x: st[x].clone() for x in ("K_pages", "V_pages")}
        for b, count in enumerate(st["counts"].tolist()):
            pick = st["accepted"][b, :count].tolist()
            sp, so = places(b, [lens[b] + a for a in pick])
            dp, do = places(b, [lens[b] + a for a in range(count)])
            for x in pools:
                pools[x][:, dp, do] = st[x][:, sp, so]
        return dict(pools, lens=None)

    H = case["H"]
    G = H // H_kv
    families = []
    for b in range(case["B"]):
        n = start[b + 1] - start[b]
        if st["parents"] is None:
            families.append(None)
        else:
            families.append(_ancestors(st["parents"][start[b]:start[b + 1]].tolist()))
        if families[b] is not None and len(families[b]) != n:
            raise ValueError("parents")

    if case["op"] == "append":
        out = {"Q": torch.empty((st["M"], H, d_h), dtype=torch.float64, device="cuda"),
               "K_pages": st["K_pages"].double(), "V_pages": st["V_pages"].double()}
        half = d_h // 2
        for b in range(case["B"]):
            r0, r1 = start[b], start[b + 1]
            if families[b] is None:
                deep = list(range(r1 - r0))
            else:
                deep = [len(f) - 1 for f in families[b]]
            pos = torch.tensor([lens[b] + x for x in deep], dtype=torch.float64, device="cuda") / case["scale"]
            turn = torch.polar(torch.ones((r1 - r0, 1, half), dtype=torch.float64, device="cuda"),
                               torch.stack([pos * case["base"] ** (-2.0 * c / d_h) for c in range(half)], -1)[:, None])

            def rotated(x, gamma):
                x = x.double() / (x.double().pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * (1 + gamma.double())
                z = torch.complex(x[..., :half], x[..., half:]) * turn
                return torch.cat([z.real, z.imag], -1)

            out["Q"][r0:r1] = rotated(st["Q"][r0:r1].view(-1, H, d_h), st["gamma_q"]) / d_h ** 0.5
            page, off = places(b, list(range(lens[b], lens[b] + r1 - r0)))
            kv = st["KV"][r0:r1].view(-1, 2, H_kv, d_h)
            out["K_pages"][page, off] = rotated(kv[:, 0], st["gamma_k"])
            out["V_pages"][page, off] = kv[:, 1].double()
        out["Q"] = out["Q"].view(st["M"], H * d_h)
        return out

    pairs = sum((start[b + 1] - start[b]) * (lens[b] + start[b + 1] - start[b]) for b in range(case["B"]))
    if 4 * H * d_h * pairs > 6e12:
        return None
    O = torch.zeros((st["M"], H, d_h), dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        r0, n, used = start[b], start[b + 1] - start[b], lens[b]
        page, off = places(b, list(range(used + n)))
        at = torch.arange(used + n, device="cuda")
        mine = torch.tril(torch.ones((n, n), dtype=torch.bool, device="cuda"))
        deep = list(range(n))
        if families[b] is not None:
            mine = torch.tensor([[j in f for j in range(n)] for f in families[b]], device="cuda").view(n, n)
            deep = [len(f) - 1 for f in families[b]]
        deep = torch.tensor(deep, device="cuda")
        at[used:] = used + deep
        for t0 in range(0, n, 256):
            t = torch.arange(t0, min(n, t0 + 256), device="cuda")
            see = torch.cat([torch.ones((t.numel(), used), dtype=torch.bool, device="cuda"), mine[t]], 1)
            if case["window"]:
                see = see & ((used + deep[t])[:, None] - at[None] < case["window"])
            for j in range(H_kv):
                k, v = st["K_pages"][page, off, j].double(), st["V_pages"][page, off, j].double()
                for h in range(j * G, j * G + G):
                    x = (st["Q"][r0 + t, h].double() @ k.T).masked_fill(~see, float("-inf"))
                    O[r0 + t, h] = torch.softmax(x, -1) @ v
    return {"O": O}
