"""GPU parity of the paged KV cache against its fp64 oracle.

- positions: equal; append: elementwise bounds, other slots and rows untouched;
- attention: elementwise bounds derived below, over steps, trees and chunks;
- commit: every number equal;
- the layer entry equal to its stages; a run of prompt, trees and commits.

Bounds of the attention, for one row with probabilities p and values v: a
logit is a sum of exact products accumulated in fp32 in steps of 16 channels,
off by at most (d_h / 16 + 4) 2^-22 A with A = max_s sum_c |q_c k_c| (each step
rounds or truncates at 2^-23 of a partial sum <= A; the scaling to base 2 adds
to it); exp2 adds 2^-21 relative.  A probability is rounded once to fp16:
2^-11 relative, or 2^-32 of the row's largest below fp16's normal range.  The
sums of p v and of p are fp32 steps, within 2^-18 of sum p |v| for the lengths
here, and so are the parts' sums.  So an output is within
  (2^-11 + 2 d + 2^-18) sum p |v| + n 2^-32 max |v| + its own half step,
d the relative error of a probability (and, once more, of the sum they are
divided by).

Bounds of the append: RMS and (1 + gamma) in fp32 are within 2^-20 relative;
an angle is within 2^-19 (reduced from p f in two fp32 parts, p < 2^24, plus
the hardware sine's 2^-21), which moves a rotated value by at most that times
the pair's |a| + |b|; the result is rounded to fp16 (half a step 2^-11, 2^-25
below its normal range).
"""
import pytest
import torch

from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu

F64 = torch.float64
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
SHAPES = [(4, 1, 256), (8, 4, 256), (4, 4, 256), (4, 1, 128), (4, 2, 128), (3, 3, 128)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_attention_gb300.build import build
    build()
    import transformer_attention_gb300 as G3
    G3.lib()


def _status():
    import transformer_attention_gb300 as G3
    return G3.gemma3_attn_check_status()


def make_batch(lens, new, P, seed, tree=False, behind=0, spare=2, extra_pages=1):
    """A batch (CPU dict) of these lengths and new tokens, pages in random
    order, -1 in the table's unused entries, `behind` rows of no sequence."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(a + n) // P) for a, n in zip(lens, new)]
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=g).tolist()
    width = max(max(need), 1) + extra_pages
    table, k = torch.full((len(lens), width), -1, dtype=torch.int32), 0
    for b, c in enumerate(need):
        table[b, :c] = torch.tensor(perm[k:k + c], dtype=torch.int32)
        k += c
    rs = torch.tensor([0] + new).cumsum(0).int()
    M = int(rs[-1]) + behind
    parents = None
    if tree:
        parents = torch.zeros(M, dtype=torch.int32)
        for b, n in enumerate(new):
            for i in range(n):
                back = int(torch.randint(1, 6, (1,), generator=g))
                parents[int(rs[b]) + i] = max(-1, i - back)
    return dict(lens=torch.tensor(lens, dtype=torch.int32), row_start=rs, parents=parents,
                table=table, P=P, n_pages=n_pages, M=M, T_max=max(max(new), 1))


def dev_batch(batch):
    import transformer_attention_gb300 as G3
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    return G3.paged_batch(up(batch["lens"]), up(batch["row_start"]), up(batch["table"]),
                          rows=batch["M"], T_max=batch["T_max"], page_size=batch["P"],
                          n_pages=batch["n_pages"], parents=up(batch["parents"]))


def make_pools(batch, H_kv, d_h, seed, fill=float("nan")):
    """Pools with numbers in the slots of the sequences and `fill` elsewhere."""
    g = torch.Generator().manual_seed(seed)
    pools = []
    for _ in range(2):
        x = torch.full((batch["n_pages"], batch["P"], H_kv, d_h), fill, dtype=torch.float16)
        for b, _, n, length in PO.sequences(batch):
            for s in range(length + n):
                p, r = PO.place(batch, b, s)
                x[p, r] = torch.randn((H_kv, d_h), generator=g).half()
        pools.append(x)
    return pools


def queries(M, H, d_h, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((M, H, d_h), generator=g) * spread * d_h ** -0.5).half()


def bound(ref, dtype, d_h):
    O, mag, big, seen, vmax = ref
    d = ((d_h / 16 + 4) * 2.0 ** -22 * big + 2.0 ** -21)[..., None]
    return ((2.0 ** -11 + 2 * d + 2.0 ** -18) * mag + (seen * 2.0 ** -32 * vmax)[..., None]
            + HALF_STEP[dtype] * (O.abs() + mag * 2.0 ** -10) + 2.0 ** -25)


def attend(batch, Q, pools, window, dtype=torch.bfloat16, O=None):
    import transformer_attention_gb300 as G3
    M, H, d_h = Q.shape
    H_kv = pools[0].shape[2]
    db = dev_batch(batch)
    ws_n = G3.gemma3_paged_attention_workspace_size(db, H, H_kv, d_h)
    ws = torch.full((ws_n,), 0xFF, dtype=torch.uint8, device="cuda")
    if O is None:
        O = torch.full((M, H, d_h), 7.0, dtype=dtype, device="cuda")
    code = G3.GEMMA3_F16 if dtype == torch.float16 else G3.GEMMA3_BF16
    G3.gemma3_paged_attention(db, Q.cuda(), pools[0].cuda(), pools[1].cuda(), O, code, H, H_kv, d_h,
                              window, ws, ws_n)
    assert _status() == 0
    return O.cpu()


def check(batch, H, H_kv, d_h, window, dtype, seed, spread=1.5):
    pools = make_pools(batch, H_kv, d_h, seed)
    Q = queries(batch["M"], H, d_h, seed + 1, spread)
    used = int(batch["row_start"][-1])
    got = attend(batch, Q, pools, window, dtype)
    assert bool((got[used:] == 7.0).all())           # rows behind the last sequence
    ref = PO.attention(batch, Q[:used], *pools, window)
    err = (got[:used].to(F64) - ref[0]).abs()
    worst = float((err / bound(ref, dtype, d_h)).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("H,H_kv,d_h", SHAPES)
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("window", [0, 40])
def test_steps(H, H_kv, d_h, P, window):
    """One token after lengths around pages, tiles and none at all."""
    lens = [0, 1, 15, 16, 127, 128, 129, 300]
    check(make_batch(lens, [1] * len(lens), P, 1, behind=2), H, H_kv, d_h, window, torch.bfloat16, 2)


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d_h", [128, 256])
def test_pages(P, d_h):
    check(make_batch([700, 3, 255, 511], [2, 5, 1, 3], P, 3), 4, 2, d_h, 0, torch.float16, 4)


@pytest.mark.parametrize("H,H_kv,d_h", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 3, 100])
def test_trees(H, H_kv, d_h, window):
    """Trees of one to 64 tokens, some sequences without new tokens."""
    check(make_batch([130, 0, 77, 60, 250], [64, 33, 0, 1, 17], 16, 5, tree=True, behind=1), H, H_kv, d_h,
          window, torch.float16, 6)


@pytest.mark.parametrize("H,H_kv,d_h", SHAPES)
@pytest.mark.parametrize("window", [0, 60])
def test_chunks(H, H_kv, d_h, window):
    """Chunks of several query tiles beside steps."""
    check(make_batch([0, 190, 5, 64], [301, 129, 1, 70], 32, 7, behind=3), H, H_kv, d_h, window,
          torch.bfloat16, 8)


@pytest.mark.parametrize("d_h", [128, 256])
@pytest.mark.parametrize("new", [1, 9, 300])
def test_many_sequences(d_h, new):
    """More sequences than a warp, most without new tokens."""
    n = [new if b % 7 == 3 else 0 for b in range(75)]
    check(make_batch([(b * 37) % 200 for b in range(75)], n, 16, 9), 2, 1, d_h, 0, torch.float16, 10)


@pytest.mark.parametrize("d_h", [128, 256])
@pytest.mark.parametrize("spread", [1e-3, 30.0])
def test_flat_and_sharp(d_h, spread):
    """Probabilities all alike, and one that takes everything."""
    check(make_batch([900, 2000], [3, 40], 64, 11, tree=True), 4, 2, d_h, 0, torch.float16, 12, spread)


def test_nothing_to_do():
    b = make_batch([5, 0], [0, 0], 16, 13, behind=4)
    pools = make_pools(b, 2, 128, 14)
    assert bool((attend(b, queries(4, 4, 128, 15), pools, 0) == 7.0).all())


# ---------------------------------------------------------------- append, positions, commit
def append_args(batch, H, H_kv, d_h, seed):
    g = torch.Generator().manual_seed(seed)
    M = batch["M"]
    size = torch.exp2(torch.randint(-6, 4, (M, 1), generator=g).float())
    Q = (torch.randn((M, H * d_h), generator=g) * size).half()
    KV = (torch.randn((M, 2 * H_kv * d_h), generator=g) * size).half()
    gq, gk = ((torch.randn(d_h, generator=g) * 0.3).bfloat16() for _ in range(2))
    return Q, KV, gq, gk


def near(got, ref, y, scale=1.0):
    half = y.shape[-1] // 2
    pair = y[..., :half].abs() + y[..., half:].abs()
    pair = torch.cat([pair, pair], -1) * scale
    tol = 2.0 ** -11 * ref.abs() + (2.0 ** -19 + 2.0 ** -20) * (1 + 2.0 ** -11) * pair + 2.0 ** -25
    worst = float(((got.to(F64) - ref).abs() / tol).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("H,H_kv,d_h", SHAPES)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_append(H, H_kv, d_h, tree, inplace):
    import transformer_attention_gb300 as G3
    b = make_batch([0, 100000, 31, 5], [3, 40, 0, 9], 16, 21, tree=tree, behind=2, extra_pages=0)
    Q, KV, gq, gk = append_args(b, H, H_kv, d_h, 22)
    kvd, M, used = H_kv * d_h, b["M"], int(b["row_start"][-1])
    pools = [torch.full((b["n_pages"], 16, H_kv, d_h), 3.0 + i, dtype=torch.float16) for i in range(2)]
    dev = [p.cuda() for p in pools]
    q, kv = Q.cuda(), KV.cuda()
    out = q if inplace else torch.full((M, H * d_h + 8), 9.0, dtype=torch.float16, device="cuda")
    db = dev_batch(b)
    pos = torch.empty(M, dtype=torch.int32, device="cuda")
    G3.gemma3_paged_positions(db, pos)
    G3.gemma3_paged_append(db, q, H * d_h, out, out.shape[1], kv, kv[:, kvd:], 2 * kvd, gq.cuda(),
                           gk.cuda(), H, H_kv, d_h, 1e6, 8.0, 0.17, *dev)
    assert _status() == 0
    ref_pos = PO.positions(b, M)
    assert torch.equal(pos.cpu().long(), ref_pos)
    refq, yq = PO.norm_rope(Q[:used].view(used, H, d_h), gq, ref_pos[:used], 1e6, 8.0)
    refk, yk = PO.norm_rope(KV[:used, :kvd].reshape(used, H_kv, d_h), gk, ref_pos[:used], 1e6, 8.0)
    got = out.cpu()
    near(got[:used, :H * d_h].view(used, H, d_h), refq * 0.17, yq, 0.17)
    if inplace:
        assert torch.equal(got[used:], Q[used:])
    else:
        assert bool((got[used:] == 9.0).all()) and bool((got[:, H * d_h:] == 9.0).all())
    assert torch.equal(kv.cpu(), KV)
    new_k, new_v = (d.cpu() for d in dev)
    written = torch.zeros(b["n_pages"], 16, dtype=torch.bool)
    for s, row0, n, length in PO.sequences(b):
        for i in range(n):
            p, r = PO.place(b, s, length + i)
            written[p, r] = True
            near(new_k[p, r], refk[row0 + i], yk[row0 + i])
            assert torch.equal(new_v[p, r], KV[row0 + i, kvd:].view(H_kv, d_h))
    assert bool((new_k[~written] == 3.0).all()) and bool((new_v[~written] == 4.0).all())


@pytest.mark.parametrize("M", [1, 700])
def test_append_without_norm(M):
    """Finished rows go to the pages bit by bit."""
    import transformer_attention_gb300 as G3
    b = make_batch([13], [M], 32, 23, behind=1)
    _, KV, _, _ = append_args(b, 2, 2, 128, 24)
    dev = [torch.zeros((b["n_pages"], 32, 2, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    kv = KV.cuda()
    G3.gemma3_paged_append(dev_batch(b), None, 0, None, 0, kv, kv[:, 256:], 512, None, None, 0, 2, 128,
                           0.0, 0.0, 0.0, *dev)
    assert _status() == 0
    for d, rows in zip(dev, (KV[:, :256], KV[:, 256:])):
        d = d.cpu()
        for i in range(M):
            p, r = PO.place(b, 0, 13 + i)
            assert torch.equal(d[p, r].reshape(-1), rows[i])
        assert int((d != 0).any(-1).any(-1).sum()) == M


@pytest.mark.parametrize("H_kv,d_h", [(1, 128), (3, 256), (16, 128)])
@pytest.mark.parametrize("layers", [1, 3])
def test_commit(H_kv, d_h, layers):
    import transformer_attention_gb300 as G3
    lens, new = [0, 17, 250, 9, 40, 63], [5, 64, 33, 0, 7, 300]
    b = make_batch(lens, new, 16, 31)
    g = torch.Generator().manual_seed(32)
    pools = [torch.randn((layers, b["n_pages"], 16, H_kv, d_h), generator=g).half() for _ in range(2)]
    accepted = torch.full((6, 300), -7, dtype=torch.int32)
    paths = [[0, 1, 2, 3, 4], list(range(1, 64, 2)), [32], [], [], list(range(3, 290))]
    for i, p in enumerate(paths):
        accepted[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
    counts = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    dev = [p.cuda() for p in pools]
    got = G3.commit_paged_cache(dev_batch(b), dev, accepted.cuda(), counts.cuda())
    assert _status() == 0
    ref, new_lens = PO.commit(b, pools, accepted, counts)
    assert torch.equal(got.cpu().long(), new_lens)
    for a, r in zip(dev, ref):
        assert torch.equal(a.cpu(), r)


def test_commit_without_path():
    """The first tokens, or all, stay where they are."""
    import transformer_attention_gb300 as G3
    b = make_batch([3, 20], [5, 2], 16, 33)
    pools = [torch.randn((1, b["n_pages"], 16, 1, 128)).half().cuda() for _ in range(2)]
    before = [p.clone() for p in pools]
    assert G3.commit_paged_cache(dev_batch(b), pools).tolist() == [8, 22]
    counts = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    assert G3.commit_paged_cache(dev_batch(b), pools, None, counts).tolist() == [3, 21]
    assert _status() == 0
    assert all(torch.equal(a, c) for a, c in zip(pools, before))
