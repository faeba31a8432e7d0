"""The paged KV cache in plain fp64: what gemma3_paged_positions, _append,
_attention and _commit compute, written from their definitions (CPU).

A batch is a dict: "lens" [B], "row_start" [B + 1], "parents" [M] or None,
"table" [B, max_pages] (lists or CPU tensors), "P" slots per page.  Pools are
[n_pages, P, H_kv, d_h].
"""
from __future__ import annotations

import torch

F64 = torch.float64


def sequences(batch):
    """(b, first row, new tokens, length) of every sequence."""
    rs = [int(x) for x in batch["row_start"]]
    return [(b, rs[b], rs[b + 1] - rs[b], int(batch["lens"][b])) for b in range(len(rs) - 1)]


def families(batch, row0, n):
    """Each new token's ancestors and itself, as sets of their numbers."""
    out = []
    for i in range(n):
        p = i - 1 if batch["parents"] is None else int(batch["parents"][row0 + i])
        out.append({i} | (out[p] if p >= 0 else set()))
    return out


def place(batch, b, s):
    """(page, row of the page) of slot s."""
    return int(batch["table"][b][s // batch["P"]]), s % batch["P"]


def slots(batch, pool, b, n):
    """The first n slots of sequence b, [n, H_kv, d_h] fp64."""
    at = [place(batch, b, s) for s in range(n)]
    return pool[[a for a, _ in at], [r for _, r in at]].to(F64)


def positions(batch, M):
    pos = torch.zeros(M, dtype=torch.int64)
    for _, row0, n, length in sequences(batch):
        for i, f in enumerate(families(batch, row0, n)):
            pos[row0 + i] = length + len(f) - 1
    return pos


def norm_rope(x, gamma, pos, base, scale):
    """x [M, heads, d_h]: RMSNorm, (1 + gamma), rotation of (c, c + d_h / 2)."""
    d = x.shape[-1]
    x = x.to(F64)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (1 + gamma.to(F64))
    c = torch.arange(d // 2, dtype=F64)
    angle = (pos.to(F64) / scale)[:, None] * torch.pow(torch.tensor(base, dtype=F64), -2 * c / d)
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    a, b = y[..., :d // 2], y[..., d // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1), y


def attention(batch, Q, K_pages, V_pages, window):
    """O [M, H, d_h] fp64 (rows of no sequence NaN), and for the error bounds of
    each row: sum p |v| [M, H, d_h], the largest sum |q k| and the number of
    visible slots [M, H], the largest |v| seen [M, H]."""
    M, H, d = Q.shape
    H_kv = K_pages.shape[2]
    G = H // H_kv
    O = torch.full((M, H, d), float("nan"), dtype=F64)
    mag = torch.zeros((M, H, d), dtype=F64)
    big, seen, vmax = (torch.zeros((M, H), dtype=F64) for _ in range(3))
    for b, row0, n, length in sequences(batch):
        if n == 0:
            continue
        fam = families(batch, row0, n)
        k, v = slots(batch, K_pages, b, length + n), slots(batch, V_pages, b, length + n)
        at = torch.cat([torch.arange(length), torch.tensor([length + len(f) - 1 for f in fam])])
        for i, f in enumerate(fam):
            see = torch.zeros(length + n, dtype=torch.bool)
            see[:length] = True
            see[[length + x for x in f]] = True
            if window > 0:
                see &= at > length + len(f) - 1 - window
            ks, vs = k[see], v[see]
            for h in range(H):
                q = Q[row0 + i, h].to(F64)
                kk, vv = ks[:, h // G], vs[:, h // G]
                p = torch.softmax(kk @ q, 0)
                O[row0 + i, h] = p @ vv
                mag[row0 + i, h] = p @ vv.abs()
                big[row0 + i, h] = (kk.abs() @ q.abs()).max()
                seen[row0 + i, h] = len(ks)
                vmax[row0 + i, h] = vv.abs().max()
    return O, mag, big, seen, vmax


def commit(batch, pools, accepted, counts):
    """The pools after the move (copies, whatever their dtype), and the new lengths."""
    out = [p.clone() for p in pools]
    new = []
    for b, _, n, length in sequences(batch):
        count = n if counts is None else int(counts[b])
        new.append(length + count)
        for i in range(count):
            src = i if accepted is None else int(accepted[b][i])
            sp, so = place(batch, b, length + src)
            dp, do = place(batch, b, length + i)
            for o, p in zip(out, pools):
                o[..., dp, do, :, :] = p[..., sp, so, :, :]
    return out, torch.tensor(new)
