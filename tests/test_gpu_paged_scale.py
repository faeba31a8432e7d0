"""The paged KV cache over more sequences than a CTA has threads (384 in the
attention's plan) or the append keeps starts of in shared memory (1024), and guard
bytes around everything that the paged calls write.

Bounds: those of tests/test_gpu_paged.py."""
import pytest
import torch

from oracle import paged_oracle as PO
from tests import test_gpu_paged as T
from tests.test_gpu_guards import Guarded
from tests.test_gpu_paged_more import _weights

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_attention_gb300.build import build
    build()
    import transformer_attention_gb300 as G3
    G3.lib()


def _crowd(B, seed, top=3):
    """Lengths and new tokens of B short sequences, a third of them without any."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, 40, (B,), generator=g).tolist()
    new = [max(0, n) for n in torch.randint(-1, top, (B,), generator=g).tolist()]
    return lens, new


# ---------------------------------------------------------------- many sequences
@pytest.mark.parametrize("B", [384, 385, 1100])
@pytest.mark.parametrize("kind", ["steps", "trees", "chunk", "chunk at the end"])
@pytest.mark.parametrize("d_h", [128, 256])
@pytest.mark.parametrize("window", [0, 500])
def test_attention(B, kind, d_h, window):
    """Several sequences per thread of the plan: steps and trees in equal shares,
    and beside a chunk whose units take whole shares of several CTAs."""
    lens, new = _crowd(B, 160 + B)
    if kind.startswith("chunk"):
        at = B - 1 if kind != "chunk" else B // 3
        lens[at], new[at] = 6000, 300
    elif kind == "trees":
        new = [4 * n for n in new]
    T.check(T.make_batch(lens, new, 16, 161, tree=kind == "trees", behind=2), 2, 1, d_h, window, torch.float16, 162)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B", [1023, 1024, 1025, 2500])
@pytest.mark.parametrize("norm", [False, True])
def test_append(B, tree, norm):
    """Rows find their sequence in shared memory, and beyond 1024 in global memory."""
    import transformer_attention_gb300 as G3
    H, H_kv, d_h, kvd = 4, 2, 128, 256
    lens, new = _crowd(B, 163, top=6)
    b = T.make_batch(lens, new, 16, 164, tree=tree, behind=3)
    Q, KV, gq, gk = T.append_args(b, H, H_kv, d_h, 165)
    M, used = b["M"], sum(new)
    kv, out = KV.cuda(), torch.full((M, H * d_h), 9.0, dtype=torch.float16, device="cuda")
    dev = [torch.full((b["n_pages"], 16, H_kv, d_h), 3.0 + i, dtype=torch.float16, device="cuda") for i in range(2)]
    q, g1, g2 = (Q.cuda(), gq.cuda(), gk.cuda()) if norm else (None, None, None)
    G3.gemma3_paged_append(T.dev_batch(b), q, H * d_h, out if norm else None, H * d_h, kv, kv[:, kvd:], 2 * kvd, g1, g2,
                           H, H_kv, d_h, 1e6, 8.0, 0.17, *dev)
    assert T._status() == 0
    pos = PO.positions(b, M)[:used]
    got = out.cpu()
    assert bool((got[used:] == 9.0).all())
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(new))
    slot = torch.cat([torch.arange(a, a + n) for a, n in zip(lens, new)])
    at = b["table"].long()[seq, slot // 16] * 16 + slot % 16
    k, v = (d.cpu().flatten(0, 1) for d in dev)
    new_k = KV[:used, :kvd].reshape(used, H_kv, d_h)
    if norm:
        refq, yq = PO.norm_rope(Q[:used].view(used, H, d_h), gq, pos, 1e6, 8.0)
        T.near(got[:used].view(used, H, d_h), refq * 0.17, yq, 0.17)
        T.near(k[at], *PO.norm_rope(new_k, gk, pos, 1e6, 8.0))
    else:
        assert bool((got == 9.0).all()) and torch.equal(k[at], new_k)
    assert torch.equal(v[at], KV[:used, kvd:].view(used, H_kv, d_h))
    rest = torch.ones(len(k), dtype=torch.bool)
    rest[at] = False
    assert bool((k[rest] == 3.0).all()) and bool((v[rest] == 4.0).all())


def test_commit():
    """A sequence per CTA row, many of them without accepted tokens."""
    import transformer_attention_gb300 as G3
    B = 2500
    lens, new = _crowd(B, 166, top=6)
    b = T.make_batch(lens, new, 16, 167)
    g = torch.Generator().manual_seed(168)
    pools = [torch.randn((2, b["n_pages"], 16, 1, 128), generator=g).half() for _ in range(2)]
    accepted = torch.full((B, b["T_max"]), -7, dtype=torch.int32)
    counts = torch.zeros(B, dtype=torch.int32)
    for s, n in enumerate(new):
        path = (torch.rand(n, generator=g) < 0.6).nonzero()[:, 0].int()
        counts[s], accepted[s, :len(path)] = len(path), path
    dev = [p.cuda() for p in pools]
    got = G3.commit_paged_cache(T.dev_batch(b), dev, accepted.cuda(), counts.cuda())
    assert T._status() == 0
    ref, new_lens = PO.commit(b, pools, accepted, counts)
    assert torch.equal(got.cpu().long(), new_lens)
    assert all(torch.equal(a.cpu(), r) for a, r in zip(dev, ref))


# ---------------------------------------------------------------- guard bytes
SHARES = [
    (4, 2, 128, [3000], [300], False),        # whole shares, cut units and their merge
    (16, 16, 128, [300, 0, 700, 40, 129, 128], [260, 300, 1, 150, 33, 128], False),   # more units than CTAs
    (8, 4, 256, [200, 0, 1000, 640], [260, 300, 100, 1], False),
    (4, 1, 256, [20000], [1], False),         # a step in many parts
    (4, 1, 128, [700, 300], [7, 33], True),   # a cluster per unit
    (2, 2, 128, [9000, 4, 2500], [64, 5, 64], True),
]


@pytest.mark.parametrize("H,H_kv,d_h,lens,new,tree", SHARES)
@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_attention_writes_only_its_rows_and_workspace(H, H_kv, d_h, lens, new, tree, window, dtype):
    import transformer_attention_gb300 as G3
    b = T.make_batch(lens, new, 32, 170, tree=tree, behind=3)
    pools = T.make_pools(b, H_kv, d_h, 171)
    Q, db = T.queries(b["M"], H, d_h, 172), T.dev_batch(b)
    q, dev = Q.cuda(), [p.cuda() for p in pools]
    n = G3.gemma3_paged_attention_workspace_size(db, H, H_kv, d_h)
    start = torch.full((b["M"], H, d_h), 7.0, dtype=dtype, device="cuda")
    ws, out = Guarded(n, torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")), Guarded(Q.numel() * 2, start)
    code = G3.GEMMA3_F16 if dtype == torch.float16 else G3.GEMMA3_BF16
    G3.gemma3_paged_attention(db, q, *dev, out.inner, code, H, H_kv, d_h, window, ws.inner, n)
    assert T._status() == 0
    assert ws.guards_intact() and out.guards_intact()
    assert torch.equal(q.cpu(), Q)
    assert all(torch.equal(a.view(torch.int16).cpu(), p.view(torch.int16)) for a, p in zip(dev, pools))
    used = sum(new)
    got = out.view(dtype, (b["M"], H, d_h)).cpu()
    assert bool((got[used:] == 7.0).all())
    ref = PO.attention(b, Q[:used], *pools, window)
    assert float(((got[:used].to(F64) - ref[0]).abs() / T.bound(ref, dtype, d_h)).max()) <= 1.0


@pytest.mark.parametrize("H,H_kv,d_h,lens,new,tree", SHARES)
def test_the_other_calls_write_only_what_they_say(H, H_kv, d_h, lens, new, tree):
    """Positions, append and commit: what is inside is the other tests'."""
    import transformer_attention_gb300 as G3
    b = T.make_batch(lens, new, 32, 173, tree=tree, behind=3)
    db, kvd, M = T.dev_batch(b), H_kv * d_h, b["M"]
    Q, KV, gq, gk = (t.cuda() for t in T.append_args(b, H, H_kv, d_h, 174))
    pos, out, lens_out = Guarded(M * 4), Guarded(M * H * d_h * 2), Guarded(len(lens) * 4)
    pools = [Guarded(b["n_pages"] * 32 * kvd * 2) for _ in range(2)]
    G3.gemma3_paged_positions(db, pos.inner)
    G3.gemma3_paged_append(db, Q, H * d_h, out.inner, H * d_h, KV, KV[:, kvd:], 2 * kvd, gq, gk, H, H_kv, d_h, 1e6, 8.0,
                           0.17, pools[0].inner, pools[1].inner)
    accepted = torch.zeros((len(lens), b["T_max"]), dtype=torch.int32)
    for s, n in enumerate(new):
        accepted[s, :n // 2] = torch.arange(n // 2) * 2 + 1
    G3.gemma3_paged_commit(db, accepted.cuda(), torch.tensor([n // 2 for n in new], dtype=torch.int32, device="cuda"), 1,
                           H_kv, d_h, pools[0].inner, pools[1].inner, lens_out.inner)
    assert T._status() == 0
    assert all(g.guards_intact() for g in (pos, out, lens_out, *pools))
    assert lens_out.view(torch.int32, (len(lens),)).tolist() == [a + n // 2 for a, n in zip(lens, new)]


@pytest.mark.parametrize("new,tree", [([3, 1], False), ([60, 64], True), ([300, 40], False)])
@pytest.mark.parametrize("H,H_kv,d_h", [(4, 2, 128), (4, 1, 128), (4, 1, 256)])
def test_layer_writes_only_out_pages_and_workspace(new, tree, H, H_kv, d_h):
    import transformer_attention_gb300 as G3
    D = 256
    w = {k: v.cuda() for k, v in _weights(D, H, H_kv, d_h, 175).items()}
    b = T.make_batch([3000, 10], new, 32, 176, tree=tree, behind=3)
    db, M = T.dev_batch(b), b["M"]
    x = torch.randn((M, D), generator=torch.Generator().manual_seed(177)).bfloat16().cuda()
    pools = [p.cuda() for p in T.make_pools(b, H_kv, d_h, 178, fill=0.0)]
    n = G3.gemma3_attn_paged_workspace_size(db, D, H, H_kv, d_h)

    def call(out, ws, K, V):
        G3.gemma3_attn_forward_paged(db, D, H, H_kv, d_h, x, w["Wq"], w["Wkv"], w["Wo"], w["gamma_q"], w["gamma_k"],
                                     G3.GEMMA3_GLOBAL, 0, 1e6, 8.0, 0.1, K, V, out, ws, n)
        assert T._status() == 0

    kept = x.clone()
    mine = [Guarded(p.numel() * 2, p) for p in pools]
    ws, out = Guarded(n), Guarded(M * D * 2)
    call(out.inner, ws.inner, *(g.inner for g in mine))
    assert all(g.guards_intact() for g in (ws, out, *mine)) and torch.equal(x, kept)
    want, plain = [p.clone() for p in pools], torch.empty((M, D), dtype=torch.bfloat16, device="cuda")
    call(plain, torch.empty(n, dtype=torch.uint8, device="cuda"), *want)
    assert torch.equal(out.view(torch.bfloat16, (M, D)), plain)
    assert all(torch.equal(g.view(torch.float16, p.shape), p) for g, p in zip(mine, want))
