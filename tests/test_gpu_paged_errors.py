"""Errors that kernels record while a paged batch is at work: a batch that does
not fit itself costs its own sequence alone, whatever else is computed until the
status is read, and a wait that gave up is reported beside errors of the input.

What the layer writes to the pages is compared bit by bit with a batch that fits:
projections and append compute a row alone.  Its output is compared within the
layer tests' tolerance: where the units of the attention are cut follows from the
whole batch, so the parts' fp32 sums (within 2^-18) may round the other way.
"""
import pytest
import torch

from oracle import paged_oracle as PO
from tests import helpers as Hh
from tests import test_gpu_paged as T
from tests.test_gpu_paged_more import _run_layer, _weights, expect_bad_input

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_attention_gb300.build import build
    build()
    import transformer_attention_gb300 as G3
    G3.lib()


def spoil(b, what):
    """The batch with sequence 1 made not to fit, and the sequences that take no
    part or whose output is open."""
    bad = dict(b, lens=b["lens"].clone(), row_start=b["row_start"].clone(), table=b["table"].clone())
    if what == "more than T_max":       # (the others have fewer tokens)
        bad["T_max"] = int(b["row_start"][2] - b["row_start"][1]) - 1
    elif what == "negative length":
        bad["lens"][1] = -3
    elif what == "beyond the table":
        bad["lens"][1] = b["P"] * b["table"].shape[1]
    elif what == "page outside the pool":
        bad["table"][1, int(b["lens"][1]) // b["P"]] = b["n_pages"]
    else:                               # a parent that is not earlier
        bad["parents"] = b["parents"].clone()
        bad["parents"][int(b["row_start"][1])] = 1
    return bad


# few rows; more than 16, norm and rotation in the projection (H_kv d_h a
# multiple of 256) or in the append; several rows for each of the append's CTAs
@pytest.mark.parametrize("new,heads,H_kv,d_h", [
    ([3, 6, 1, 2], 4, 2, 128), ([3, 6, 1, 2], 4, 1, 256), ([13, 30, 1, 9], 4, 2, 128), ([13, 30, 1, 9], 4, 1, 128),
    ([13, 30, 1, 9], 4, 1, 256), ([900, 1600, 1, 700], 4, 2, 128), ([900, 1600, 1, 700], 2, 1, 128),
])
@pytest.mark.parametrize("what", ["more than T_max", "negative length", "beyond the table", "page outside the pool",
                                  "parent not earlier"])
def test_layer_with_a_sequence_that_does_not_fit(new, heads, H_kv, d_h, what):
    """The other sequences' output and pages are what they always are."""
    import transformer_attention_gb300 as G3
    tree, D = what == "parent not earlier", 256
    if tree and max(new) > G3.GEMMA3_TREE_MAX:
        new = [60, 64, 1, 50]
    w = _weights(D, heads, H_kv, d_h, 140)
    b = T.make_batch([40, 130, 5, 77], new, 16, 141, tree=tree, behind=2)
    bad = spoil(b, what)
    x = torch.randn((b["M"], D), generator=torch.Generator().manual_seed(142)).bfloat16()
    start = [p.cuda() for p in T.make_pools(b, H_kv, d_h, 143, fill=0.0)]
    kw = dict(H=heads, H_kv=H_kv, attn_type=G3.GEMMA3_GLOBAL, window=0, rope_base=1e6, rope_scale=8.0, query_scale=0.1)
    want = [p.clone() for p in start]
    out = _run_layer(b, x, want, w, kw).cpu()
    assert T._status() == 0
    pools = [p.clone() for p in start]
    got = _run_layer(bad, x, pools, w, kw).cpu()
    expect_bad_input()
    for s, row0, n, length in PO.sequences(b):
        if s != 1:
            Hh.assert_close(got[row0:row0 + n], out[row0:row0 + n], f"beside one that does not fit, seq {s}")
        elif what not in ("page outside the pool", "parent not earlier"):
            assert bool((got[row0:row0 + n] == 0).all())
    assert bool((got[b["M"] - 2:] == 0).all())
    # every slot holds what it did, or the other sequences' new K' and V
    if tree:        # (the sequence's own rows may have another position)
        for s, _, n, length in PO.sequences(b):
            for i in range(length, length + n):
                at = PO.place(b, s, i)
                assert all(torch.equal(p[at], a[at]) for p, a in list(zip(pools, want))[0 if s != 1 else 1:])
                for p, a in zip(pools, want):
                    p[at] = a[at]
    else:
        gone = range(int(b["lens"][1]), int(b["lens"][1]) + new[1])
        if what == "page outside the pool":
            gone = [i for i in gone if i // 16 == int(b["lens"][1]) // 16]
        for i in gone:
            at = PO.place(b, 1, i)
            for p, a in zip(want, start):
                p[at] = a[at]
    assert all(torch.equal(p, a) for p, a in zip(pools, want))


def _record_bad_paged(G3):
    """A sequence of negative length, which the positions' own check records."""
    b = T.make_batch([5], [2], 16, 150)
    b["lens"][0] = -1
    G3.gemma3_paged_positions(T.dev_batch(b), torch.empty(2, dtype=torch.int32, device="cuda"))


def _record_bad_token(G3):
    E = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
    G3.gemma3_embed(torch.tensor([9], dtype=torch.int32, device="cuda"), E, 8, 64, 1, 1.0,
                    torch.empty((1, 64), device="cuda"))


@pytest.mark.parametrize("H,H_kv,d_h", [(4, 1, 256), (4, 2, 128)])
def test_other_layers_run_after_a_paged_error(H, H_kv, d_h):
    """A batch that did not fit is no reason for a layer without pages to stop."""
    import transformer_attention_gb300 as G3
    B, n, D = 2, 200, 256
    w = {k: v.cuda() for k, v in _weights(D, H, H_kv, d_h, 151).items()}
    x = torch.randn((B, n, D), generator=torch.Generator().manual_seed(152)).bfloat16().cuda()
    pos = torch.arange(n, dtype=torch.int32, device="cuda").repeat(B, 1)

    def layer():
        return G3.attention_forward(x, pos, None, *(w[k] for k in ("Wq", "Wkv", "Wo", "gamma_q", "gamma_k")), H=H,
                                    H_kv=H_kv, attn_type=G3.GEMMA3_GLOBAL, window=0, rope_base=1e4, rope_scale=1.0,
                                    query_scale=0.1, out=torch.full((B, n, D), 5.0, dtype=torch.bfloat16, device="cuda"))

    want = layer()
    assert T._status() == 0
    _record_bad_paged(G3)
    got = layer()
    expect_bad_input()
    assert torch.equal(got, want)


@pytest.mark.parametrize("paged,token", [(True, False), (False, True), (True, True), (False, False)])
def test_a_lost_wait_is_reported_beside_bad_input(paged, token):
    """What was recorded first does not hide that a kernel gave up on a wait."""
    import transformer_attention_gb300 as G3
    from transformer_attention_gb300 import _lib as L
    if paged:
        _record_bad_paged(G3)
    if token:
        _record_bad_token(G3)
    assert G3.gemma3_selftest_wait_timeout(50_000_000) == L.GEMMA3_ERR_TIMEOUT      # 50 ms
    assert G3.gemma3_last_device_status() == (0x4000 if paged else 0) + (0x2000 if token else 0) + 0x1000 + 99
    assert G3.gemma3_attn_check_status() == 0


def test_both_kinds_of_bad_input():
    import transformer_attention_gb300 as G3
    for first, second in ((_record_bad_paged, _record_bad_token), (_record_bad_token, _record_bad_paged)):
        first(G3)
        second(G3)
        with pytest.raises(G3.Gemma3Error) as e:
            G3.gemma3_attn_check_status()
        assert e.value.status == G3.GEMMA3_ERR_BAD_INPUT
        assert G3.gemma3_last_device_status() == 0x6000
        assert G3.gemma3_attn_check_status() == 0
