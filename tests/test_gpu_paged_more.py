"""The paged KV cache where a call can go wrong: batches that do not fit
themselves, NaN in hidden slots, aliases, repeated and captured calls, streams,
pools beyond 2^32 bytes, and the layer over a run of prompt, trees and commits."""
import pytest
import torch

from oracle import gemma3_oracle as O
from oracle import paged_oracle as PO
from tests import helpers as Hh
from tests import test_gpu_paged as T

pytestmark = pytest.mark.gpu

F64 = torch.float64
H, H_KV = 4, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_attention_gb300.build import build
    build()
    import transformer_attention_gb300 as G3
    G3.lib()


def expect_bad_input():
    import transformer_attention_gb300 as G3
    with pytest.raises(G3.Gemma3Error) as e:
        G3.gemma3_attn_check_status()
    assert e.value.status == G3.GEMMA3_ERR_BAD_INPUT
    assert G3.gemma3_last_device_status() == 0x4000
    assert G3.gemma3_attn_check_status() == 0


def attend(db, Q, dev, O_, window=0, ws=None, stream=None):
    """gemma3_paged_attention on device tensors; no synchronisation."""
    import transformer_attention_gb300 as G3
    _, heads, d_h = Q.shape
    H_kv = dev[0].shape[2]
    n = G3.gemma3_paged_attention_workspace_size(db, heads, H_kv, d_h)
    if ws is None:
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    code = G3.GEMMA3_F16 if O_.dtype == torch.float16 else G3.GEMMA3_BF16
    G3.gemma3_paged_attention(db, Q, dev[0], dev[1], O_, code, heads, H_kv, d_h, window, ws, n, stream)
    return O_


def check_rows(got, batch, Q, pools, window, dtype, skip=()):
    """The rows of the sequences not in `skip` against the oracle; 7.0 elsewhere."""
    ref = PO.attention(batch, Q, *pools, window)
    bound = T.bound(ref, dtype, Q.shape[2])
    for b, row0, n, _ in PO.sequences(batch):
        rows = slice(row0, row0 + n)
        if b in skip:
            continue
        worst = float(((got[rows].to(F64) - ref[0][rows]).abs() / bound[rows]).max()) if n else 0.0
        assert worst <= 1.0, (b, worst)


# ---------------------------------------------------------------- batches that do not fit
LENS, NEW = [40, 130, 5, 77], [3, 2, 4, 1]


@pytest.mark.parametrize("what", ["row beyond M", "more than T_max", "negative length", "beyond the table"])
@pytest.mark.parametrize("d_h", [128, 256])
def test_sequences_that_do_not_fit(what, d_h):
    """Such a sequence counts as one without new tokens."""
    b = T.make_batch(LENS, NEW, 16, 1)
    pools = T.make_pools(b, H_KV, d_h, 2)
    Q = T.queries(b["M"], H, d_h, 3)
    bad = dict(b, lens=b["lens"].clone(), row_start=b["row_start"].clone())
    skip = {3}
    if what == "row beyond M":
        bad["row_start"][4] = b["M"] + 1
    elif what == "more than T_max":
        bad["T_max"], skip = 3, {2}
    elif what == "negative length":
        bad["lens"][3] = -1
    else:
        bad["lens"][3] = 16 * b["table"].shape[1]
    db, dev = T.dev_batch(bad), [p.cuda() for p in pools]
    got = attend(db, Q.cuda(), dev, torch.full((b["M"], H, d_h), 7.0, dtype=torch.float16, device="cuda"))
    expect_bad_input()
    check_rows(got.cpu(), b, Q, pools, 0, torch.float16, skip)
    for s in skip:
        assert bool((got[int(b["row_start"][s]):int(b["row_start"][s + 1])] == 7.0).all())
    # the append: neither their rows nor their slots are written
    import transformer_attention_gb300 as G3
    q, kv, gq, gk = (t.cuda() for t in T.append_args(b, H, H_KV, d_h, 4))
    out = torch.full_like(q, 9.0)
    pages = [torch.full_like(p, 3.0) for p in dev]
    kvd = H_KV * d_h
    G3.gemma3_paged_append(db, q, H * d_h, out, H * d_h, kv, kv[:, kvd:], 2 * kvd, gq, gk, H, H_KV, d_h, 1e4, 1.0,
                           1.0, *pages)
    expect_bad_input()
    written = torch.zeros(b["n_pages"], 16, dtype=torch.bool)
    for s, row0, n, length in PO.sequences(b):
        assert bool((out[row0:row0 + n] == 9.0).all()) == (s in skip)
        for i in range(n if s not in skip else 0):
            written[PO.place(b, s, length + i)] = True
    for p in pages:
        assert torch.equal((p != 3.0).flatten(2).any(2).cpu(), written)
    pos = torch.full((b["M"],), -5, dtype=torch.int32, device="cuda")
    G3.gemma3_paged_positions(db, pos)
    expect_bad_input()
    want = PO.positions(b, b["M"])
    for s in skip:
        want[int(b["row_start"][s]):int(b["row_start"][s + 1])] = 0
    assert torch.equal(pos.cpu().long(), want)


def test_row_start_that_falls():
    """Which rows have a sequence is open then; only slots of the batch are written."""
    import transformer_attention_gb300 as G3
    b = T.make_batch(LENS, NEW, 16, 1)
    bad = dict(b, row_start=torch.tensor([0, 3, 5, 9, 8], dtype=torch.int32))
    db = T.dev_batch(bad)
    q, kv, gq, gk = (t.cuda() for t in T.append_args(b, H, H_KV, 128, 4))
    pages = [torch.full((b["n_pages"], 16, H_KV, 128), 3.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    G3.gemma3_paged_append(db, q, H * 128, torch.empty_like(q), H * 128, kv, kv[:, 256:], 512, gq, gk, H, H_KV, 128, 1e4,
                           1.0, 1.0, *pages)
    expect_bad_input()
    G3.gemma3_paged_positions(db, torch.empty(b["M"], dtype=torch.int32, device="cuda"))
    expect_bad_input()
    attend(db, q.view(-1, H, 128), pages, torch.empty_like(q).view(-1, H, 128))
    expect_bad_input()
    slots = torch.zeros(b["n_pages"], 16, dtype=torch.bool)
    for s, _, n, length in PO.sequences(b):
        for i in range(n):
            slots[PO.place(b, s, length + i)] = True
    for p in pages:
        assert not bool(((p != 3.0).flatten(2).any(2).cpu() & ~slots).any())


@pytest.mark.parametrize("page", [-1, -2 ** 31, 2 ** 31 - 1, "n_pages"])
@pytest.mark.parametrize("d_h", [128, 256])
def test_pages_outside_the_pool(page, d_h):
    """They are neither read nor written; the other sequences do not notice."""
    import transformer_attention_gb300 as G3
    b = T.make_batch(LENS, NEW, 16, 5)
    pools = T.make_pools(b, H_KV, d_h, 6)
    Q = T.queries(b["M"], H, d_h, 7)
    bad = dict(b, table=b["table"].clone())
    bad["table"][1, 8] = b["n_pages"] if page == "n_pages" else page       # of its last slots, the new ones
    db, dev = T.dev_batch(bad), [p.cuda() for p in pools]
    got = attend(db, Q.cuda(), dev, torch.full((b["M"], H, d_h), 7.0, dtype=torch.float16, device="cuda"))
    expect_bad_input()
    check_rows(got.cpu(), b, Q, pools, 0, torch.float16, {1})
    q, kv, gq, gk = (t.cuda() for t in T.append_args(b, H, H_KV, d_h, 8))
    pages = [torch.full_like(p, 3.0) for p in dev]
    kvd = H_KV * d_h
    G3.gemma3_paged_append(db, q, H * d_h, q, H * d_h, kv, kv[:, kvd:], 2 * kvd, gq, gk, H, H_KV, d_h, 1e4, 1.0,
                           1.0, *pages)
    expect_bad_input()
    written = torch.zeros(b["n_pages"], 16, dtype=torch.bool)
    for s, row0, n, length in PO.sequences(b):
        for i in range(n if s != 1 else 0):
            written[PO.place(b, s, length + i)] = True
    for p in pages:
        assert torch.equal((p != 3.0).flatten(2).any(2).cpu(), written)
    # entries behind a sequence's last slot are not looked at (-1 here), nor those before a window
    far = dict(b, table=b["table"].clone())
    far["table"][1, 0] = 2 ** 30
    hidden = attend(T.dev_batch(far), Q.cuda(), dev, torch.empty((b["M"], H, d_h), dtype=torch.float16, device="cuda"), 2)
    assert G3.gemma3_attn_check_status() == 0
    check_rows(hidden.cpu(), b, Q, pools, 2, torch.float16)


@pytest.mark.parametrize("value", [-2, 2, 5, 2 ** 31 - 1, -2 ** 31])
def test_parents_that_are_no_earlier_token(value):
    """They count as -1."""
    import transformer_attention_gb300 as G3
    b = T.make_batch([20, 60], [5, 9], 16, 9, tree=True)
    b["parents"][7] = -1                                  # sequence 1, token 2
    pools = T.make_pools(b, H_KV, 128, 10)
    Q = T.queries(b["M"], H, 128, 11)
    bad = dict(b, parents=b["parents"].clone())
    bad["parents"][7] = value
    got = attend(T.dev_batch(bad), Q.cuda(), [p.cuda() for p in pools],
                 torch.empty((b["M"], H, 128), dtype=torch.float16, device="cuda"))
    expect_bad_input()
    check_rows(got.cpu(), b, Q, pools, 0, torch.float16)
    pos = torch.empty(b["M"], dtype=torch.int32, device="cuda")
    G3.gemma3_paged_positions(T.dev_batch(bad), pos)
    expect_bad_input()
    assert torch.equal(pos.cpu().long(), PO.positions(b, b["M"]))


@pytest.mark.parametrize("path,count", [([2, 2], 2), ([3, 1], 2), ([-1, 2], 2), ([0, 4], 2), ([0, 1], 5), ([0], -1)])
def test_commit_of_what_does_not_ascend(path, count):
    """That sequence is left as it is, the others move."""
    import transformer_attention_gb300 as G3
    b = T.make_batch([30, 14, 3], [6, 4, 5], 16, 12)
    g = torch.Generator().manual_seed(13)
    pools = [torch.randn((2, b["n_pages"], 16, 1, 128), generator=g).half() for _ in range(2)]
    accepted = torch.full((3, 6), 5, dtype=torch.int32)
    accepted[0, :2], accepted[2, :2] = torch.tensor([1, 4]), torch.tensor([2, 3])
    accepted[1, :len(path)] = torch.tensor(path)
    dev = [p.cuda() for p in pools]
    got = G3.commit_paged_cache(T.dev_batch(b), dev, accepted.cuda(),
                                torch.tensor([2, count, 2], dtype=torch.int32, device="cuda"))
    expect_bad_input()
    ref, lens = PO.commit(b, pools, accepted, [2, 0, 2])
    assert got.tolist() == lens.tolist()
    assert all(torch.equal(a.cpu(), r) for a, r in zip(dev, ref))


def test_after_a_recorded_error():
    """A bad token id that another call recorded changes nothing here."""
    import transformer_attention_gb300 as G3
    b = T.make_batch([300, 20], [5, 7], 16, 14, tree=True)
    pools = [p.cuda() for p in T.make_pools(b, H_KV, 128, 15)]
    Q, db = T.queries(b["M"], H, 128, 16).cuda(), T.dev_batch(b)
    want = attend(db, Q, pools, torch.empty_like(Q))
    E = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
    G3.gemma3_embed(torch.tensor([9], dtype=torch.int32, device="cuda"), E, 8, 64, 1, 1.0,
                    torch.empty((1, 64), device="cuda"))
    got = attend(db, Q, pools, torch.empty_like(Q))
    with pytest.raises(G3.Gemma3Error):
        G3.gemma3_attn_check_status()
    assert torch.equal(got, want)


# ---------------------------------------------------------------- what slots hold
@pytest.mark.parametrize("d_h", [128, 256])
@pytest.mark.parametrize("tree", [False, True])
def test_nan_before_the_window(d_h, tree):
    """Slots that no new token's window reaches may hold anything."""
    W = 50
    b = T.make_batch([400, 200, 30], [6, 1, 3], 16, 17, tree=tree)
    pools = T.make_pools(b, H_KV, d_h, 18)
    Q = T.queries(b["M"], H, d_h, 19)
    clean = [p.clone() for p in pools]
    for s, row0, n, length in PO.sequences(b):
        for slot in range(0, length - W + 1):
            for p, fill in zip(pools, (float("inf"), float("nan"))):
                p[PO.place(b, s, slot)] = fill
    got = attend(T.dev_batch(b), Q.cuda(), [p.cuda() for p in pools],
                 torch.empty((b["M"], H, d_h), dtype=torch.float16, device="cuda"), W)
    check_rows(got.cpu(), b, Q, clean, W, torch.float16)


@pytest.mark.parametrize("d_h,new", [(128, 3), (128, 200), (256, 3), (256, 100)])
def test_a_nan_query_stays_in_its_row(d_h, new):
    b = T.make_batch([150, 10], [new, 2], 16, 20)
    pools = T.make_pools(b, H_KV, d_h, 21)
    Q = T.queries(b["M"], H, d_h, 22)
    Q[1, 2] = float("nan")
    Q[2, 0] = 60000.0                                      # logits far apart
    got = attend(T.dev_batch(b), Q.cuda(), [p.cuda() for p in pools],
                 torch.empty((b["M"], H, d_h), dtype=torch.bfloat16, device="cuda")).cpu()
    assert bool(torch.isnan(got[1, 2]).all())
    rest = torch.ones(b["M"], H, dtype=torch.bool)
    rest[1, 2] = False
    assert bool(torch.isfinite(got[rest]).all())
    ref = PO.attention(b, Q, *pools, 0)[0]
    assert torch.allclose(got[rest].to(F64), ref[rest], rtol=2.0 ** -6, atol=2.0 ** -6)


@pytest.mark.parametrize("d_h,new", [(128, 1), (128, 300), (256, 40)])
def test_output_over_the_queries(d_h, new):
    b = T.make_batch([700, 1, 90], [new, 3, 2], 32, 23)
    pools = [p.cuda() for p in T.make_pools(b, H_KV, d_h, 24)]
    Q, db = T.queries(b["M"], H, d_h, 25).cuda(), T.dev_batch(b)
    want = attend(db, Q, pools, torch.empty_like(Q))
    got = attend(db, Q, pools, Q)
    assert got.data_ptr() == Q.data_ptr() and torch.equal(got, want)


# ---------------------------------------------------------------- repeated, captured, side by side
def _many():
    """Batches whose calls take different forms."""
    return [(T.make_batch([1500, 40, 3000], [1, 1, 1], 16, 30), 128), (T.make_batch([900, 31], [64, 20], 64, 31, tree=True), 128),
            (T.make_batch([200, 700], [400, 1], 32, 32), 128), (T.make_batch([2500], [7], 16, 33, tree=True), 256),
            (T.make_batch([50, 800, 9], [300, 1, 70], 128, 34), 256), (T.make_batch([3000], [300], 64, 35), 128)]


def test_the_same_bits_without_a_gap():
    """Calls that follow one another, of other batches between them, give what
    each gives alone."""
    calls = []
    for k, (b, d_h) in enumerate(_many()):
        pools = [p.cuda() for p in T.make_pools(b, H_KV, d_h, 40 + k, fill=0.5)]
        calls.append((T.dev_batch(b), T.queries(b["M"], H, d_h, 50 + k).cuda(), pools))
    alone = []
    for db, Q, pools in calls:
        alone.append(attend(db, Q, pools, torch.empty_like(Q)))
        assert T._status() == 0
    import transformer_attention_gb300 as G3
    need = max(G3.gemma3_paged_attention_workspace_size(db, H, H_KV, Q.shape[2]) for db, Q, _ in calls)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(30):
        outs = [attend(db, Q, pools, torch.empty_like(Q), ws=ws) for db, Q, pools in calls]
        torch.cuda.synchronize()
        for o, a in zip(outs, alone):
            assert torch.equal(o, a)
    assert T._status() == 0


def test_captured_and_replayed():
    """Two graphs that share a workspace, replayed with other lengths, rows and
    pages than at their capture."""
    import transformer_attention_gb300 as G3
    first = T.make_batch([500, 60, 7], [4, 2, 1], 16, 60, behind=1)
    other = T.make_batch([33, 300, 0], [1, 0, 3], 16, 61)
    width = max(first["table"].shape[1], other["table"].shape[1])
    n_pages = max(first["n_pages"], other["n_pages"])
    M, T_max = first["M"], 4
    lens, rs = first["lens"].cuda(), first["row_start"].cuda()
    table = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    db = G3.paged_batch(lens, rs, table, rows=M, T_max=T_max, page_size=16, n_pages=n_pages)
    dev = [torch.zeros((n_pages, 16, H_KV, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    Q = torch.zeros((M, H, 128), dtype=torch.float16, device="cuda")
    outs = [torch.empty((M, H, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    n = G3.gemma3_paged_attention_workspace_size(db, H, H_KV, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def fill(b, seed):
        pools, q = T.make_pools(b, H_KV, 128, seed), T.queries(M, H, 128, seed + 1)
        lens.copy_(b["lens"])
        rs.copy_(b["row_start"])
        table.fill_(-1)
        table[:, :b["table"].shape[1]] = b["table"].cuda()
        for d, p in zip(dev, pools):
            d.zero_()
            d[:p.shape[0]] = p.cuda()
        Q.copy_(q)
        return pools, q

    fill(first, 62)
    attend(db, Q, dev, outs[0], 0, ws)
    torch.cuda.synchronize()
    graphs = []
    for out, window in zip(outs, (0, 30)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attend(db, Q, dev, out, window, ws)
        graphs.append(g)
    for b, seed in ((first, 62), (other, 64), (first, 66)):
        pools, q = fill(b, seed)
        for o in outs:
            o.fill_(7.0)
        for g in graphs * 2:
            g.replay()
        assert T._status() == 0
        for o, window in zip(outs, (0, 30)):
            got, used = o.cpu(), int(b["row_start"][-1])
            assert bool((got[used:] == 7.0).all())
            check_rows(got, b, q, pools, window, torch.float16)


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own."""
    calls = []
    for k, (b, d_h) in enumerate(_many()):
        pools = [p.cuda() for p in T.make_pools(b, H_KV, d_h, 70 + k, fill=0.25)]
        Q = T.queries(b["M"], H, d_h, 80 + k).cuda()
        calls.append((T.dev_batch(b), Q, pools, attend(T.dev_batch(b), Q, pools, torch.empty_like(Q))))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        outs = []
        for k, (db, Q, pools, want) in enumerate(calls):
            for s in streams if k % 2 else streams[::-1]:
                with torch.cuda.stream(s):
                    out = torch.empty_like(Q)
                    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
                    outs.append((attend(db, Q, pools, out, ws=ws, stream=s), want))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in outs)
    assert T._status() == 0


# ---------------------------------------------------------------- far offsets
@pytest.mark.parametrize("d_h", [128, 256])
def test_a_pool_beyond_32_bits(d_h):
    """Pages whose bytes lie behind 2^32, written and read."""
    import transformer_attention_gb300 as G3
    H_kv, P = 8, 64
    n_pages = (5 << 30) // (P * H_kv * d_h * 2)
    pools = [torch.empty((n_pages, P, H_kv, d_h), dtype=torch.float16, device="cuda") for _ in range(2)]
    b = T.make_batch([100, 200], [9, 70], P, 90, spare=0, extra_pages=0)
    small, Q = T.make_pools(b, H_kv, d_h, 91), T.queries(b["M"], 8, d_h, 92)
    far = dict(b, table=torch.where(b["table"] >= 0, n_pages - 1 - b["table"], b["table"]), n_pages=n_pages)
    for p, s in zip(pools, small):
        p[n_pages - b["n_pages"]:] = s.flip(0).cuda()
    db = T.dev_batch(far)
    got = attend(db, Q.cuda(), pools, torch.empty((b["M"], 8, d_h), dtype=torch.float16, device="cuda"))
    assert T._status() == 0
    check_rows(got.cpu(), b, Q, small, 0, torch.float16)
    kv = T.append_args(b, 8, H_kv, d_h, 93)[1].cuda()
    kvd = H_kv * d_h
    G3.gemma3_paged_append(db, None, 0, None, 0, kv, kv[:, kvd:], 2 * kvd, None, None, 0, H_kv, d_h, 0.0, 0.0, 0.0,
                           *pools)
    accepted = torch.full((2, 70), -1, dtype=torch.int32)
    accepted[0, :2], accepted[1, :3] = torch.tensor([2, 8]), torch.tensor([0, 33, 69])
    lens = G3.commit_paged_cache(db, [p[None] for p in pools], accepted.cuda(),
                                 torch.tensor([2, 3], dtype=torch.int32, device="cuda"))
    assert T._status() == 0 and lens.tolist() == [102, 203]
    for s, row0, path in ((0, 0, [2, 8]), (1, 9, [0, 33, 69])):
        for i, a in enumerate(path):
            page, r = PO.place(far, s, int(b["lens"][s]) + i)
            for p, rows in zip(pools, (kv[:, :kvd], kv[:, kvd:])):
                assert torch.equal(p[page, r].reshape(-1), rows[row0 + a])


def test_a_long_sequence():
    """300001 slots of one kv head, in pages of 16 in random order."""
    length, d_h = 300000, 128
    b = T.make_batch([length], [1], 16, 94)
    g = torch.Generator(device="cuda").manual_seed(95)
    pools = [torch.randn((b["n_pages"], 16, 1, d_h), generator=g, device="cuda").half() for _ in range(2)]
    Q = T.queries(1, 4, d_h, 96)
    got = attend(T.dev_batch(b), Q.cuda(), pools, torch.empty((1, 4, d_h), dtype=torch.float16, device="cuda"))
    rows = (b["table"][0].long().cuda().clamp(min=0)[:, None] * 16 + torch.arange(16, device="cuda")).view(-1)[:length + 1]
    k, v = (p.view(-1, d_h)[rows].double() for p in pools)
    p = torch.softmax(Q[0].double().cuda() @ k.T, -1)
    O_, mag = p @ v, p @ v.abs()
    big = (Q[0].double().cuda().abs() @ k.abs().T).amax(1)
    ref = (O_.cpu()[None], mag.cpu()[None], big.cpu()[None], torch.full((1, 4), length + 1.0, dtype=F64),
           torch.full((1, 4), float(v.abs().max()), dtype=F64))
    worst = float(((got.cpu().to(F64) - ref[0]).abs() / T.bound(ref, torch.float16, d_h)).max())
    assert worst <= 1.0, worst


# ---------------------------------------------------------------- the layer
def _weights(D, heads, H_kv, d_h, seed):
    g = torch.Generator().manual_seed(seed)
    w = lambda *s: (torch.randn(s, generator=g) * D ** -0.5).bfloat16()  # noqa: E731
    gam = lambda: (torch.randn(d_h, generator=g) * 0.3).bfloat16()  # noqa: E731
    return dict(Wq=w(heads * d_h, D), Wkv=w(2, H_kv * d_h, D), Wo=w(D, heads * d_h), gamma_q=gam(), gamma_k=gam())


def _run_layer(b, x, cache, w, kw, stream=None):
    import transformer_attention_gb300 as G3
    return G3.attention_forward_paged(x.cuda(), T.dev_batch(b), cache, *(w[k].cuda() for k in (
        "Wq", "Wkv", "Wo", "gamma_q", "gamma_k")), stream=stream, **kw)


@pytest.mark.parametrize("heads,H_kv,d_h", [(4, 2, 128), (4, 1, 256), (2, 1, 128)])
@pytest.mark.parametrize("window", [0, 20])
def test_layer_run(heads, H_kv, d_h, window):
    """A prompt, two trees of drafted tokens with their commits, and a step:
    every token's output is that of the layer over the path to it."""
    import transformer_attention_gb300 as G3
    D, P, B = 512, 16, 2
    w = _weights(D, heads, H_kv, d_h, 100)
    base = dict(rope_base=1e4, rope_scale=2.0, query_scale=d_h ** -0.5, H=heads, H_kv=H_kv)
    kind = G3.GEMMA3_LOCAL_SLIDING if window else G3.GEMMA3_GLOBAL
    kw = dict(base, attn_type=kind, window=window)
    okw = dict(base, attn_type=O.LOCAL_SLIDING if window else O.GLOBAL, window=window, d_h=d_h)
    width, n_pages = 8, 16
    table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(101)).int().view(B, width)
    cache = G3.new_paged_cache(1, n_pages, P, H_kv, d_h, "cuda")
    g = torch.Generator().manual_seed(102)
    tokens = [torch.zeros((0, D), dtype=torch.bfloat16) for _ in range(B)]     # the accepted ones
    lens = torch.zeros(B, dtype=torch.int32)
    # (new tokens, a tree's parents, accepted)
    plan = [([50, 33], None, None), ([7, 3], [[-1, 0, 0, 1, -1, 4, 3], [-1, -1, 0]], [[0, 1, 3], []]),
            ([20, 12], [[max(-1, i - 2) for i in range(20)], [i - 1 for i in range(12)]], [[1, 3, 5, 7], list(range(12))]),
            ([1, 1], None, None)]
    for step, (new, parents, accepted) in enumerate(plan):
        rs = torch.tensor([0] + new).cumsum(0).int()
        M = int(rs[-1]) + 2
        x = torch.randn((M, D), generator=g).bfloat16()
        par = None
        if parents is not None:
            par = torch.tensor(parents[0] + parents[1] + [0, 0], dtype=torch.int32)
        b = dict(lens=lens, row_start=rs, parents=par, table=table, P=P, n_pages=n_pages, M=M, T_max=max(new))
        out = _run_layer(b, x, (cache[0][0], cache[1][0]), w, kw).cpu()
        assert T._status() == 0
        assert bool((out[int(rs[-1]):] == 0).all())
        for s in range(B):
            mine = x[int(rs[s]):int(rs[s + 1])]
            got, ref = [], []
            if parents is None:
                seq = torch.cat([tokens[s], mine])
                n = len(seq)
                ref = O.attention_layer(seq[None], torch.arange(n)[None], None, **{k: w[k] for k in w}, **okw)[0][-len(mine):]
                got = out[int(rs[s]):int(rs[s + 1])]
            else:
                for i in range(len(mine)):
                    path, q = [], i
                    while q >= 0:
                        path.insert(0, q)
                        q = parents[s][q]
                    seq = torch.cat([tokens[s], mine[path]])
                    n = len(seq)
                    ref.append(O.attention_layer(seq[None], torch.arange(n)[None], None, **{k: w[k] for k in w}, **okw,
                                                 rows=[[n - 1]])[0])
                    got.append(out[int(rs[s]) + i:int(rs[s]) + i + 1])
                ref, got = torch.cat(ref), torch.cat(got)
            Hh.assert_close(got, ref, f"paged layer {heads}/{H_kv}/{d_h} W{window} step {step} seq {s}")
            keep = list(range(len(mine))) if accepted is None else accepted[s]
            tokens[s] = torch.cat([tokens[s], mine[keep]])
        if accepted is None:
            lens = G3.commit_paged_cache(T.dev_batch(b), cache).cpu()
        else:
            ac = torch.zeros((B, max(new)), dtype=torch.int32)
            for s in range(B):
                ac[s, :len(accepted[s])] = torch.tensor(accepted[s], dtype=torch.int32)
            counts = torch.tensor([len(a) for a in accepted], dtype=torch.int32)
            lens = G3.commit_paged_cache(T.dev_batch(b), cache, ac.cuda(), counts.cuda()).cpu()
        assert lens.tolist() == [len(t) for t in tokens]


@pytest.mark.parametrize("M", [5, 40])
def test_layer_is_its_stages(M):
    """The layer against its calls one by one, on a side stream, in a padded batch."""
    import transformer_attention_gb300 as G3
    heads, H_kv, d_h, D = 4, 2, 128, 256
    w = _weights(D, heads, H_kv, d_h, 110)
    b = T.make_batch([70, 3], [M - 4, 2], 16, 111, behind=2)
    x = torch.randn((M, D), generator=torch.Generator().manual_seed(112)).bfloat16()
    x[M - 2:] = float("nan")                               # rows of no sequence
    start = [p.cuda() for p in T.make_pools(b, H_kv, d_h, 113, fill=0.0)]
    kw = dict(H=heads, H_kv=H_kv, attn_type=G3.GEMMA3_GLOBAL, window=0, rope_base=1e6, rope_scale=8.0, query_scale=0.1)
    side = torch.cuda.Stream()
    pools = [p.clone() for p in start]
    torch.cuda.synchronize()
    out = _run_layer(b, x, pools, w, kw, stream=side)
    torch.cuda.synchronize()
    assert T._status() == 0 and bool((out[M - 2:] == 0).all())
    db, kvd, dev = T.dev_batch(b), H_kv * d_h, {k: v.cuda() for k, v in w.items()}
    mine = [p.clone() for p in start]
    pos = torch.empty(M, dtype=torch.int32, device="cuda")
    G3.gemma3_paged_positions(db, pos)
    Q = torch.empty((M, heads * d_h), dtype=torch.float16, device="cuda")
    KV = torch.empty((M, 2 * kvd), dtype=torch.float16, device="cuda")
    G3.gemma3_qkv_proj_norm_rope(x.cuda(), D, dev["Wq"], dev["Wkv"], Q, KV, M, D, heads, H_kv, d_h, G3.GEMMA3_BF16,
                                 dev["gamma_q"], dev["gamma_k"], pos, 1e6, 8.0, 0.1)
    G3.gemma3_paged_append(db, None, 0, None, 0, KV, KV[:, kvd:], 2 * kvd, None, None, 0, H_kv, d_h, 0.0, 0.0, 0.0, *mine)
    O_ = torch.zeros((M, heads, d_h), dtype=torch.bfloat16, device="cuda")
    attend(db, Q.view(M, heads, d_h), mine, O_)
    want = G3.linear(O_.view(M, heads * d_h), dev["Wo"])
    assert T._status() == 0
    for a, c in zip(pools, mine):
        assert float((a.float() - c.float()).abs().max()) <= (0.0 if M > 16 else 2.0 ** -9)
    assert float((out[:M - 2].float() - want[:M - 2].float()).abs().max()) <= (0.0 if M > 16 else 2.0 ** -6)


@pytest.mark.parametrize("M", [4, 40])
def test_layer_after_a_recorded_error(M):
    """With more than 16 rows the projections stop at it, and the pages stay as
    they were; the call can be made again."""
    import transformer_attention_gb300 as G3
    heads, H_kv, d_h, D = 4, 2, 128, 256
    w = _weights(D, heads, H_kv, d_h, 120)
    b = T.make_batch([70, 3], [M - 2, 2], 16, 121)
    x = torch.randn((M, D), generator=torch.Generator().manual_seed(122)).bfloat16()
    start = [p.cuda() for p in T.make_pools(b, H_kv, d_h, 123, fill=0.0)]
    kw = dict(H=heads, H_kv=H_kv, attn_type=G3.GEMMA3_GLOBAL, window=0, rope_base=1e6, rope_scale=8.0, query_scale=0.1)
    want = [p.clone() for p in start]
    out = _run_layer(b, x, want, w, kw)
    assert T._status() == 0
    pools = [p.clone() for p in start]
    E = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
    G3.gemma3_embed(torch.tensor([9], dtype=torch.int32, device="cuda"), E, 8, 64, 1, 1.0, torch.empty((1, 64), device="cuda"))
    _run_layer(b, x, pools, w, kw)
    with pytest.raises(G3.Gemma3Error):
        G3.gemma3_attn_check_status()
    if M > 16:
        assert all(torch.equal(a, s) for a, s in zip(pools, start))
    again = _run_layer(b, x, pools, w, kw)
    assert T._status() == 0 and torch.equal(again, out)
    assert all(torch.equal(a, c) for a, c in zip(pools, want))


# ---------------------------------------------------------------- how the work is shared out
@pytest.mark.parametrize("H_,H_kv,d_h,lens,new,tree", [
    (4, 2, 128, [3000], [300], False),        # units longer than a share, a few
    (4, 4, 128, [5000, 10], [257, 1], False),
    (4, 2, 256, [4000], [200], False),
    (4, 1, 128, [6000], [64], True),          # a tree of two query tiles
    (16, 16, 128, [300, 0, 700, 40, 129, 128], [260, 300, 1, 150, 33, 128], False),   # more units than CTAs
    (8, 4, 256, [200, 0, 1000, 640], [260, 300, 100, 1], False),
    (4, 1, 256, [20000], [1], False),         # a step over many CTAs
    (2, 2, 128, [9000, 4, 2500], [64, 5, 64], True),
])
@pytest.mark.parametrize("window", [0, 700])
def test_shares(H_, H_kv, d_h, lens, new, tree, window):
    T.check(T.make_batch(lens, new, 32, 130, tree=tree), H_, H_kv, d_h, window, torch.float16, 131)


# ---------------------------------------------------------------- what a call may leave out
@pytest.mark.parametrize("P", [16, 256])
@pytest.mark.parametrize("H_kv,d_h,lens,new,tree", [
    (2, 128, [700, 1300, 30], [6, 1, 3], True),
    (2, 256, [700, 1300, 30], [6, 1, 3], False),
    (4, 128, [1500, 700], [300, 1], False),
    (2, 256, [1500, 700], [300, 1], False),
])
def test_pages_given_back(P, H_kv, d_h, lens, new, tree):
    """Pages before every window may be gone from the table."""
    import transformer_attention_gb300 as G3
    W = 50
    b = T.make_batch(lens, new, P, 70, tree=tree)
    pools = T.make_pools(b, H_kv, d_h, 71)
    Q = T.queries(b["M"], 2 * H_kv, d_h, 72)
    gone = dict(b, table=b["table"].clone())
    for s, length in enumerate(lens):
        gone["table"][s, :max(0, length - W + 1) // P] = [-1, 2 ** 31 - 1, b["n_pages"]][s]
    got = attend(T.dev_batch(gone), Q.cuda(), [p.cuda() for p in pools],
                 torch.empty((b["M"], 2 * H_kv, d_h), dtype=torch.float16, device="cuda"), W)
    assert G3.gemma3_attn_check_status() == 0
    check_rows(got.cpu(), b, Q, pools, W, torch.float16)


@pytest.mark.parametrize("what", ["row beyond M", "negative length", "beyond the table"])
@pytest.mark.parametrize("count", [0, 1, None])
def test_commit_of_sequences_that_do_not_fit(what, count):
    """Their length and slots stay as they were, the others' tokens move."""
    import transformer_attention_gb300 as G3
    b = T.make_batch([30, 14, 3], [6, 4, 5], 16, 73)
    g = torch.Generator().manual_seed(74)
    pools = [torch.randn((2, b["n_pages"], 16, 1, 128), generator=g).half() for _ in range(2)]
    bad = dict(b, lens=b["lens"].clone(), row_start=b["row_start"].clone())
    if what == "row beyond M":
        bad["row_start"][3] = b["M"] + 1
    else:
        bad["lens"][2] = -4 if what == "negative length" else 16 * b["table"].shape[1]
    accepted = torch.tensor([[1, 4, 0, 0, 0, 0], [0, 2, 0, 0, 0, 0], [1, 2, 0, 0, 0, 0]], dtype=torch.int32)
    dev = [p.cuda() for p in pools]
    counts = None if count is None else torch.tensor([2, 2, count], dtype=torch.int32, device="cuda")
    got = G3.commit_paged_cache(T.dev_batch(bad), dev, None if count is None else accepted.cuda(), counts)
    expect_bad_input()
    ref, lens = PO.commit(b, pools, None if count is None else accepted, [6, 4, 0] if count is None else [2, 2, 0])
    assert got.tolist() == lens.tolist()[:2] + [int(bad["lens"][2])]
    assert all(torch.equal(a.cpu(), r) for a, r in zip(dev, ref))


@pytest.mark.parametrize("window", [2 ** 30, 2 ** 30 + 1, 2 ** 31 - 1])
@pytest.mark.parametrize("new,tree", [(3, True), (300, False)])
def test_the_widest_windows(window, new, tree):
    """They hide nothing."""
    b = T.make_batch([700, 9], [new, 2], 32, 75, tree=tree)
    pools = T.make_pools(b, H_KV, 128, 76)
    Q = T.queries(b["M"], H, 128, 77)
    got = attend(T.dev_batch(b), Q.cuda(), [p.cuda() for p in pools],
                 torch.empty((b["M"], H, 128), dtype=torch.float16, device="cuda"), window)
    check_rows(got.cpu(), b, Q, pools, 0, torch.float16)


@pytest.mark.parametrize("T_max", [10 ** 9, 2 ** 31 - 1])
@pytest.mark.parametrize("d_h", [128, 256])
def test_t_max_beyond_the_rows(T_max, d_h):
    b = dict(T.make_batch([700, 9, 40], [1, 30, 2], 32, 78), T_max=T_max)
    pools = T.make_pools(b, H_KV, d_h, 79)
    Q = T.queries(b["M"], H, d_h, 80)
    for window in (0, 33):
        got = attend(T.dev_batch(b), Q.cuda(), [p.cuda() for p in pools],
                     torch.empty((b["M"], H, d_h), dtype=torch.float16, device="cuda"), window)
        check_rows(got.cpu(), b, Q, pools, window, torch.float16)


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("B", [31, 32, 33, 1025, 2500])
def test_many_sequences(B, tree):
    """Rows find their sequence among many, some of them without new tokens."""
    import transformer_attention_gb300 as G3
    g = torch.Generator().manual_seed(81)
    new = [0, 0] + torch.randint(0, 5, (B - 2,), generator=g).tolist()
    lens = torch.randint(0, 40, (B,), generator=g).tolist()
    b = T.make_batch(lens, new, 16, 82, tree=tree, behind=3)
    pos = torch.full((b["M"],), -5, dtype=torch.int32, device="cuda")
    G3.gemma3_paged_positions(T.dev_batch(b), pos)
    assert G3.gemma3_attn_check_status() == 0
    assert torch.equal(pos.cpu().long(), PO.positions(b, b["M"]))


# ---------------------------------------------------------------- appends of many rows
@pytest.mark.parametrize("H_,H_kv,d_h,new", [
    (4, 1, 256, [1999, 1, 800]), (4, 2, 256, [2500, 33]), (8, 2, 128, [700, 1900]), (3, 3, 128, [2600]),
    (1, 1, 128, [2432]), (3, 3, 256, [30, 2411]), (8, 4, 256, [2500, 2]), (4, 1, 256, [12000, 8001]), (16, 4, 128, [2500]),
])
def test_append_of_prompts(H_, H_kv, d_h, new):
    """Few heads: a row's vectors in one piece; many rows: several rounds of a CTA."""
    import transformer_attention_gb300 as G3
    lens = [17 * i + 5 for i in range(len(new))]
    b = T.make_batch(lens, new, 64, 83, behind=3)
    Q, KV, gq, gk = T.append_args(b, H_, H_kv, d_h, 84)
    M, used, kvd = b["M"], sum(new), H_kv * d_h
    q, kv, out = Q.cuda(), KV.cuda(), torch.full((b["M"], H_ * d_h + 8), 9.0, dtype=torch.float16, device="cuda")
    dev = [torch.full((b["n_pages"], 64, H_kv, d_h), 3.0 + i, dtype=torch.float16, device="cuda") for i in range(2)]
    G3.gemma3_paged_append(T.dev_batch(b), q, H_ * d_h, out, H_ * d_h + 8, kv, kv[:, kvd:], 2 * kvd, gq.cuda(), gk.cuda(),
                           H_, H_kv, d_h, 1e6, 8.0, 0.17, *dev)
    assert G3.gemma3_attn_check_status() == 0
    pos = torch.cat([torch.arange(n) + length for n, length in zip(new, lens)])
    refq, yq = PO.norm_rope(Q[:used].view(used, H_, d_h), gq, pos, 1e6, 8.0)
    refk, yk = PO.norm_rope(KV[:used, :kvd].reshape(used, H_kv, d_h), gk, pos, 1e6, 8.0)
    got = out.cpu()
    T.near(got[:used, :H_ * d_h].view(used, H_, d_h), refq * 0.17, yq, 0.17)
    assert bool((got[used:] == 9.0).all()) and bool((got[:, H_ * d_h:] == 9.0).all())
    seq = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new))
    at = b["table"].long()[seq, pos // 64] * 64 + pos % 64
    k, v = (d.cpu().flatten(0, 1) for d in dev)
    T.near(k[at], refk, yk)
    assert torch.equal(v[at], KV[:used, kvd:].view(used, H_kv, d_h))
    rest = torch.ones(len(k), dtype=torch.bool)
    rest[at] = False
    assert bool((k[rest] == 3.0).all()) and bool((v[rest] == 4.0).all())
