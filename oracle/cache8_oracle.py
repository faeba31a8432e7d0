"""The 8-bit KV cache in plain fp64: what gemma3_kv_cache8_write, _read,
_evict and gemma3_cached8_attention compute, written from their definitions.

A cache is a dict: "k8", "v8" [B, S, H_kv, d_h] uint8 (e4m3 codes), "ks", "vs"
[B, ceil(S/64), H_kv] float64 scales, "pos" [B, S] int64 positions.
"""
from __future__ import annotations

import torch

F64 = torch.float64
BLOCK = 64
MAX = 448.0


def _table() -> torch.Tensor:
    """Value of each e4m3 code: sign, 4 exponent bits of bias 7, 3 mantissa
    bits, subnormals of step 2^-9, codes 0x7f and 0xff NaN."""
    out = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if code & 127 == 127:
            v = float("nan")
        out.append(-v if code >= 128 else v)
    return torch.tensor(out, dtype=F64)


TABLE = _table()


def decode(codes: torch.Tensor) -> torch.Tensor:
    return TABLE[codes.to(torch.int64)]


def encode(x: torch.Tensor) -> torch.Tensor:
    """Codes of the nearest e4m3 numbers, ties to the even code; beyond 448
    the largest number, NaN the code 0x7f."""
    mags = TABLE[:127]                                  # ascending magnitudes, codes 0 .. 126
    a = x.abs().clamp(max=MAX)
    hi = torch.searchsorted(mags, a.nan_to_num(0.0)).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - mags[lo], mags[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = torch.where(up, hi, lo)
    code = torch.where(torch.isnan(x), torch.tensor(127), code)
    neg = (torch.signbit(x)) & ~torch.isnan(x)
    return (code + 128 * neg.to(code.dtype)).to(torch.uint8)


def scale_for(amax: float) -> float:
    """Smallest 2^e, e >= -15, with amax <= 448 * 2^e."""
    e = -15
    while amax > MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def _amax(x: torch.Tensor) -> float:
    a = x[torch.isfinite(x)].abs()
    return float(a.max()) if a.numel() else 0.0


def blocks(S: int) -> int:
    return -(-S // BLOCK)


def empty(B: int, S: int, H_kv: int, d_h: int) -> dict:
    return {"k8": torch.zeros(B, S, H_kv, d_h, dtype=torch.uint8),
            "v8": torch.zeros(B, S, H_kv, d_h, dtype=torch.uint8),
            "ks": torch.zeros(B, blocks(S), H_kv, dtype=F64),
            "vs": torch.zeros(B, blocks(S), H_kv, dtype=F64),
            "pos": torch.full((B, S), -1, dtype=torch.int64)}


def clone(cache: dict) -> dict:
    return {k: v.clone() for k, v in cache.items()}


def write(cache: dict, K, V, segment_pos, pad_lens, end: int) -> dict:
    """K, V [B, T, H_kv, d_h] into slots [end, end + T); returns a new cache."""
    out = clone(cache)
    B, T, H_kv, _ = K.shape
    for b in range(B):
        valid = T - int(pad_lens[b]) if pad_lens is not None else T
        for t in range(T):
            out["pos"][b, end + t] = int(segment_pos[b, t]) if t < valid else -1
        for codes, scales, x in (("k8", "ks", K), ("v8", "vs", V)):
            x = x[b].to(F64).clone()
            x[valid:] = 0.0
            for blk in range(end // BLOCK, (end + T - 1) // BLOCK + 1):
                s0, s1 = max(end, blk * BLOCK), min(end + T, (blk + 1) * BLOCK)
                for j in range(H_kv):
                    new = x[s0 - end:s1 - end, j]
                    s = scale_for(_amax(new))
                    if blk * BLOCK < end:
                        old = float(out[scales][b, blk, j])
                        s = max(old, s)
                        held = slice(blk * BLOCK, end)
                        if s != old:
                            out[codes][b, held, j] = encode(decode(out[codes][b, held, j]) * old / s)
                    out[codes][b, s0:s1, j] = encode(new / s)
                    out[scales][b, blk, j] = s
    return out


def values(cache: dict, which: str) -> torch.Tensor:
    """All values [B, S, H_kv, d_h] of "k" or "v"."""
    S = cache["pos"].shape[1]
    return decode(cache[which + "8"]) * cache[which + "s"].repeat_interleave(BLOCK, 1)[:, :S, :, None]


def visible(cache: dict, b: int, segment_pos, valid: int, T: int, end: int, window: int):
    """[T, S] mask of batch row b."""
    S = cache["pos"].shape[1]
    t, s = torch.arange(T)[:, None], torch.arange(S)[None]
    p = cache["pos"][b][None]
    see = (t < valid) & (s <= end + t) & (p >= 0)
    if window > 0:
        q = segment_pos[b].to(torch.int64)[:, None]
        see = see & (p > q - window) & (p < q + window)
    return see


def attend(Q, cache: dict, segment_pos, pad_lens, end: int, window: int):
    """O [B, T, H, d_h], the weights every slot received [B, S], and for error
    bounds the largest sum_c |q_c k_c| over visible slots and sum_s p_s |v_s|."""
    B, T, H, d_h = Q.shape
    H_kv = cache["k8"].shape[2]
    G = H // H_kv
    S = cache["pos"].shape[1]
    K, V = values(cache, "k"), values(cache, "v")
    O = torch.zeros(B, T, H, d_h, dtype=F64)
    A = torch.zeros(B, T, H, dtype=F64)
    PV = torch.zeros(B, T, H, d_h, dtype=F64)
    w = torch.zeros(B, S, dtype=F64)
    for b in range(B):
        valid = T - int(pad_lens[b]) if pad_lens is not None else T
        see = visible(cache, b, segment_pos, valid, T, end, window)
        used = see.any(0)
        k, v = K[b][used], V[b][used]
        m = see[:, used]
        for h in range(H):
            q = Q[b, :, h].to(F64)
            x = (q @ k[:, h // G].T).masked_fill(~m, float("-inf"))
            p = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300)) if x.shape[1] else x
            p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
            O[b, :, h] = p @ v[:, h // G]
            PV[b, :, h] = p @ v[:, h // G].abs()
            if x.shape[1]:
                A[b, :, h] = (q.abs() @ k[:, h // G].abs().T).masked_fill(~m, 0.0).amax(1)
            w[b, used] += p.sum(0)
    return O, w, A, PV


def evict(cache: dict, weight_sum, end: int, keep: int, recent: int, dst: dict, w_dst):
    """Returns (cache, weight_sum, kept) of the other cache after the move."""
    out, w_out = clone(dst), w_dst.clone()
    B, _, H_kv, d_h = cache["k8"].shape
    kept = torch.full((B, keep), -1, dtype=torch.int64)
    for b in range(B):
        held = [s for s in range(end) if int(cache["pos"][b, s]) >= 0]
        late = [s for s in held if s >= end - recent]
        rank = []
        for s in held:
            if s < end - recent:
                x = float(weight_sum[b, s])
                rank.append((1, 0.0, s) if x != x else (0, -x, s))
        stay = sorted(late + [s for _, _, s in sorted(rank)[:keep - len(late)]])
        n = len(stay)
        kept[b, :n] = torch.tensor(stay, dtype=torch.int64)
        out["pos"][b, :keep] = -1
        w_out[b, :keep] = 0.0
        out["pos"][b, :n] = cache["pos"][b, stay]
        w_out[b, :n] = weight_sum[b, stay]
        for codes, scales in (("k8", "ks"), ("v8", "vs")):
            for blk in range(blocks(keep)):
                d0, d1 = blk * BLOCK, min(keep, (blk + 1) * BLOCK)
                src = stay[d0:min(n, d1)]
                for j in range(H_kv):
                    x = torch.zeros(d1 - d0, d_h, dtype=F64)
                    if src:
                        s_in = cache[scales][b, [s // BLOCK for s in src], j]
                        x[:len(src)] = decode(cache[codes][b, src, j]) * s_in[:, None]
                    s = scale_for(_amax(x))
                    out[codes][b, d0:d1, j] = encode(x / s)
                    out[scales][b, blk, j] = s
    return out, w_out, kept
