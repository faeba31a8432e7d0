"""The paged KV cache without a GPU: what is refused before anything reaches a
device, the oracle against direct forms, and how the attention counts work."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

import transformer_attention_gb300 as G3
from oracle import gemma3_oracle as O
from oracle import paged_oracle as PO
from transformer_attention_gb300 import _lib as L
from transformer_attention_gb300.build import CSRC, INCLUDE, _nvcc, build

P = 1 << 40            # stands for a device pointer; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build()
    return L.lib()


def batch(**kw):
    d = dict(B=3, M=40, T_max=20, page_size=16, n_pages=100, max_pages=10, lens=P, row_start=2 * P,
             parents=None, page_table=3 * P)
    d.update(kw)
    return ctypes.byref(L.gemma3_paged_batch(**d))


def attend(lib, b, *, Q=4 * P, K=5 * P, V=6 * P, Out=7 * P, o_dtype=0, H=8, H_kv=4, d_h=128, window=0,
           ws=8 * P, nbytes=1 << 40):
    return lib.gemma3_paged_attention(b, Q, K, V, Out, o_dtype, H, H_kv, d_h, window, ws, nbytes, None)


BAD_SIZES = [
    (dict(B=0), -1), (dict(B=65536), -1), (dict(M=0), -1), (dict(M=(1 << 30) + 1), -1),
    (dict(T_max=0), -1), (dict(page_size=8), -3), (dict(page_size=48), -3), (dict(page_size=512), -3),
    (dict(n_pages=0), -1), (dict(n_pages=1 << 27), -1), (dict(max_pages=0), -1),
    (dict(max_pages=1 << 27), -1), (dict(parents=P, T_max=65), -3),
]


@pytest.mark.parametrize("change,code", BAD_SIZES)
def test_sizes(lib, change, code):
    n = ctypes.c_size_t()
    b = batch(**change)
    assert lib.gemma3_paged_attention_workspace_size(b, 8, 4, 128, ctypes.byref(n)) == code
    assert lib.gemma3_attn_paged_workspace_size(b, 512, 8, 4, 128, ctypes.byref(n)) == code
    assert attend(lib, b) == code
    assert lib.gemma3_paged_positions(b, P, None) == code
    assert lib.gemma3_paged_append(b, P, 1024, P, 1024, 2 * P, 2 * P, 512, P, P, 8, 4, 128, 1e4, 1.0, 1.0, P,
                                   P, None) == code
    assert lib.gemma3_paged_commit(b, None, None, 1, 4, 128, P, 2 * P, 9 * P, None) == code


@pytest.mark.parametrize("name", ["lens", "row_start", "page_table", "parents"])
def test_arrays(lib, name):
    if name != "parents":
        assert attend(lib, batch(**{name: None})) == -1
    assert attend(lib, batch(**{name: P + 2})) == -2


@pytest.mark.parametrize("change,code", [
    (dict(H=6, H_kv=4), -1), (dict(H=8, H_kv=1), -3), (dict(d_h=64), -3), (dict(H=0), -1),
    (dict(Q=None), -1), (dict(Out=None), -1), (dict(K=None), -1), (dict(V=None), -1), (dict(ws=None), -1),
    (dict(Q=4 * P + 8), -2), (dict(K=5 * P + 8), -2), (dict(Out=7 * P + 4), -2), (dict(ws=8 * P + 16), -2),
    (dict(o_dtype=2), -1), (dict(nbytes=1000), -6), (dict(Out=4 * P + 16), -1),
])
def test_attention_arguments(lib, change, code):
    assert attend(lib, batch(), **change) == code


def append(lib, *, Q=4 * P, ldq=1024, Qo=5 * P, ldqo=1024, K=6 * P, V=7 * P, ldkv=512, gq=P, gk=P, H=8,
           H_kv=4, d_h=128, base=1e4, scale=1.0, Kp=8 * P, Vp=9 * P):
    return lib.gemma3_paged_append(batch(), Q, ldq, Qo, ldqo, K, V, ldkv, gq, gk, H, H_kv, d_h, base, scale, 1.0,
                                   Kp, Vp, None)


@pytest.mark.parametrize("change,code", [
    (dict(Q=None), -1), (dict(Qo=None), -1), (dict(K=None), -1), (dict(V=None), -1), (dict(Kp=None), -1),
    (dict(gq=None), -1), (dict(gk=None), -1), (dict(ldq=1023), -1), (dict(ldqo=1016), -1), (dict(ldkv=504), -1),
    (dict(ldq=1028), -2), (dict(ldkv=516), -2), (dict(K=6 * P + 8), -2), (dict(gq=P + 4), -2),
    (dict(base=0.0), -1), (dict(base=float("inf")), -1), (dict(scale=float("nan")), -1), (dict(scale=-1.0), -1),
    (dict(Qo=4 * P, ldqo=1032), -1), (dict(Qo=4 * P + 2048), -1), (dict(d_h=96), -3), (dict(H=7), -1),
])
def test_append_arguments(lib, change, code):
    assert append(lib, **change) == code


@pytest.mark.parametrize("change,code", [
    (dict(layers=0), -1), (dict(layers=32768), -1), (dict(new=None), -1), (dict(K=None), -1),
    (dict(new=9 * P + 2), -2), (dict(new=P), -1), (dict(new=P + 8), -1), (dict(accepted=4 * P + 1), -2),
    (dict(counts=9 * P), -1), (dict(accepted=9 * P - 100), -1),
])
def test_commit_arguments(lib, change, code):
    a = dict(accepted=4 * P, counts=5 * P, layers=2, K=6 * P, V=7 * P, new=9 * P)
    a.update(change)
    assert lib.gemma3_paged_commit(batch(), a["accepted"], a["counts"], a["layers"], 4, 128, a["K"], a["V"],
                                   a["new"], None) == code


def test_layer_arguments(lib):
    def call(b=None, D=512, H=8, H_kv=4, d_h=128, out=P, kind=1, window=0, nbytes=1 << 40, base=1e4, x=P, ws=8 * P):
        return lib.gemma3_attn_forward_paged(b or batch(), D, H, H_kv, d_h, x, P, P, P, P, P, kind, window, base,
                                             1.0, 1.0, P, P, out, ws, nbytes, None)
    assert call(b=batch(lens=None)) == -1
    assert call(D=508) == -1 and call(H=7) == -1 and call(d_h=64) == -3
    assert call(out=None) == -1 and call(out=P + 8) == -2 and call(x=None) == -1
    assert call(kind=2) == -1 and call(kind=0, window=0) == -1 and call(base=-1.0) == -1
    assert call(ws=8 * P + 128) == -2


def test_workspace_sizes(lib):
    n = ctypes.c_size_t()
    sizes = []
    for t in (1, 2, 64, 100000):
        assert lib.gemma3_paged_attention_workspace_size(batch(T_max=t), 8, 4, 128, ctypes.byref(n)) == 0
        sizes.append(n.value)
        m = ctypes.c_size_t()
        assert lib.gemma3_attn_paged_workspace_size(batch(T_max=t), 512, 8, 4, 128, ctypes.byref(m)) == 0
        assert m.value >= n.value + 40 * (8 + 2 * 4) * 128 * 2
    assert sizes == sorted(sizes) and sizes[-1] < 1 << 28


# ---------------------------------------------------------------- the Python side
def tensors(B=2, pages=4, rows=6):
    i = torch.int32
    return (torch.zeros(B, dtype=i), torch.zeros(B + 1, dtype=i), torch.zeros(B, pages, dtype=i)), dict(
        rows=rows, T_max=3, page_size=16, n_pages=9)


@pytest.mark.parametrize("at,bad", [
    (0, torch.zeros(2)), (0, torch.zeros(2, 1, dtype=torch.int32)), (1, torch.zeros(2, dtype=torch.int32)),
    (2, torch.zeros(3, 4, dtype=torch.int32)), (2, torch.zeros(2, 8, dtype=torch.int32)[:, ::2]),
    (2, torch.zeros(8, dtype=torch.int32)),
])
def test_batch_tensors(at, bad):
    t, kw = tensors()
    G3.paged_batch(*t, **kw)
    t = list(t)
    t[at] = bad
    with pytest.raises(ValueError, match=("lens", "row_start", "page_table")[at] + "|row_start"):
        G3.paged_batch(*t, **kw)


def test_batch_parents_and_caches():
    t, kw = tensors()
    with pytest.raises(ValueError, match="parents"):
        G3.paged_batch(*t, **kw, parents=torch.zeros(5, dtype=torch.int32))
    b = G3.paged_batch(*t, **kw, parents=torch.zeros(6, dtype=torch.int32))
    cache = G3.new_paged_cache(2, 9, 16, 2, 128, "cpu")
    assert cache[0].shape == cache[1].shape == (2, 9, 16, 2, 128)
    gamma = torch.zeros(128, dtype=torch.bfloat16)
    x = torch.zeros(6, 256, dtype=torch.bfloat16)
    kw = dict(H=2, H_kv=2, attn_type=1, window=0, rope_base=1e4, rope_scale=1.0, query_scale=1.0)
    with pytest.raises(ValueError, match="rows"):
        G3.attention_forward_paged(x[:5], b, (cache[0][0], cache[1][0]), x, x, x, gamma, gamma, **kw)
    for bad in (cache, (cache[0][0], cache[1][0].float()), (cache[0][0, :, :8], cache[1][0])):
        with pytest.raises(ValueError, match="pages"):
            G3.attention_forward_paged(x, b, bad, x, x, x, gamma, gamma, **kw)
    with pytest.raises(ValueError, match="accepted"):
        G3.commit_paged_cache(b, cache, torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="counts"):
        G3.commit_paged_cache(b, cache, None, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="V_pages"):
        G3.commit_paged_cache(b, (cache[0], cache[1][:1]))


def test_another_device(monkeypatch):
    t, kw = tensors()
    b = G3.paged_batch(*t, **kw)              # (on the CPU: device -1)
    monkeypatch.setattr(L, "_device", lambda: 0)
    with pytest.raises(ValueError, match="current GPU"):
        L.gemma3_paged_positions(b, P, 0)
    monkeypatch.setattr(b, "device", 0)
    with pytest.raises(ValueError, match="current GPU"):
        L.gemma3_paged_positions(b, torch.zeros(6, dtype=torch.int32), 0)


# ---------------------------------------------------------------- oracle pins
def pages_of(K, P_):
    """Dense [S, H_kv, d_h] as pages in reversed order, and their table."""
    n = -(-K.shape[0] // P_)
    pool = torch.zeros((n, P_) + tuple(K.shape[1:]), dtype=K.dtype)
    pool.view(n * P_, *K.shape[1:])[:K.shape[0]] = K
    return pool.flip(0), torch.arange(n - 1, -1, -1)[None]


@pytest.mark.parametrize("window", [0, 7])
def test_oracle_chunk_is_the_contiguous_cache(window):
    """Tokens of a chunk over pages attend as the contiguous cache's oracle."""
    g = torch.Generator().manual_seed(1)
    S, n, H, H_kv, d = 37, 5, 4, 2, 16
    K, V = (torch.randn((S, H_kv, d), generator=g) for _ in range(2))
    Q = torch.randn((n, H, d), generator=g)
    kp, table = pages_of(K, 16)
    vp, _ = pages_of(V, 16)
    b = dict(lens=[S - n], row_start=[0, n], parents=None, table=table, P=16)
    got = PO.attention(b, Q, kp, vp, window)[0]
    pos = torch.arange(S)
    for t in range(n):
        see = (pos <= S - n + t) & ((window == 0) | (pos > S - n + t - window))
        for h in range(H):
            p = torch.softmax(K[see, h // 2].double() @ Q[t, h].double(), 0)
            assert torch.allclose(got[t, h], p @ V[see, h // 2].double(), rtol=0, atol=1e-12)


def test_oracle_tree_is_its_paths():
    """A token of a tree attends as the last token of the path to it would."""
    g = torch.Generator().manual_seed(2)
    parents = [-1, 0, 0, 1, -1, 2, 5]
    length, n, d = 9, len(parents), 8
    K, V = (torch.randn((length + n, 1, d), generator=g) for _ in range(2))
    Q = torch.randn((n, 2, d), generator=g)
    kp, table = pages_of(K, 16)
    vp, _ = pages_of(V, 16)
    b = dict(lens=[length], row_start=[0, n], parents=torch.tensor(parents), table=table, P=16)
    tree = PO.attention(b, Q, kp, vp, 4)[0]
    assert PO.positions(b, n).tolist() == [9, 10, 10, 11, 9, 11, 12]
    for i in range(n):
        path, q = [], i
        while q >= 0:
            path.insert(0, q)
            q = parents[q]
        rows = list(range(length)) + [length + x for x in path]
        ck, tb = pages_of(K[rows], 16)
        cv, _ = pages_of(V[rows], 16)
        chain = dict(lens=[length], row_start=[0, len(path)], parents=None, table=tb, P=16)
        ref = PO.attention(chain, Q[path], ck, cv, 4)[0][-1]
        assert torch.allclose(tree[i], ref, rtol=0, atol=1e-12)


def test_oracle_norm_rope_is_the_layers():
    g = torch.Generator().manual_seed(3)
    x, gamma = torch.randn((5, 2, 16), generator=g), torch.randn(16, generator=g)
    pos = torch.tensor([0, 1, 7, 1000, 16000000])
    got, y = PO.norm_rope(x, gamma, pos, 1e6, 8.0)
    ref = O.rope(O.rms_norm(x.double(), gamma.double()), pos, 1e6, 8.0)
    assert torch.allclose(got, ref, rtol=0, atol=1e-9)
    assert torch.allclose(got.norm(dim=-1), y.norm(dim=-1))


def test_oracle_commit():
    pool = torch.arange(4 * 16).view(4, 16, 1, 1)
    b = dict(lens=[14], row_start=[0, 6], parents=None, table=torch.tensor([[2, 0]]), P=16)
    (out,), new = PO.commit(b, [pool], torch.tensor([[1, 2, 5, -1, -1, -1]]), torch.tensor([3]))
    assert new.tolist() == [17]
    at = lambda t, s: t[PO.place(b, 0, s)].item()  # noqa: E731
    assert [at(out, s) for s in (14, 15, 16)] == [at(pool, s) for s in (15, 16, 19)]
    assert [at(out, s) for s in (13, 17, 18, 19)] == [at(pool, s) for s in (13, 17, 18, 19)]


# ---------------------------------------------------------------- the work units
SOURCE = r"""
#include "paged.cuh"
#include <cstdio>
int main() {
  int len, n, w, tree, ts, q;
  while (scanf("%d %d %d %d %d %d", &len, &n, &w, &tree, &ts, &q) == 6) {
    const g3::PagedUnit u = g3::paged_unit(len, n, w, tree, ts, q);
    printf("%d %d %d %d %lld\n", u.lo, u.hi, u.tile0, u.tiles, g3::paged_prefix(len, n, w, tree, ts, q));
  }
}
"""


def test_units_against_the_masks(tmp_path):
    """A unit's slots and tiles, and the closed form of their sums, against the
    visible slots of its tokens one by one."""
    src, exe = tmp_path / "units.cu", tmp_path / "units"
    src.write_text(SOURCE)
    subprocess.run([_nvcc(), "-std=c++17", "-I", CSRC, "-I", INCLUDE, "-o", str(exe), str(src)], check=True,
                   capture_output=True, env=dict(os.environ))
    rng = random.Random(4)
    cases = []
    for _ in range(400):
        tree = rng.random() < 0.3
        n = rng.randint(1, 64) if tree else rng.choice([1, 5, 64, 128, 129, 500, 3001])
        cases.append((rng.choice([0, 1, 127, 128, 129, 1000, 40000]) + rng.randint(0, 3), n,
                      rng.choice([0, 0, 1, 2, 100, 128, 1024]), int(tree), rng.randint(5, 8)))
    asked = [(*c, q) for c in cases for q in range(-(-c[1] // (1 << c[4])) + 1)]
    out = subprocess.run([str(exe)], input="\n".join(" ".join(map(str, a)) for a in asked), text=True,
                         capture_output=True, check=True).stdout.split("\n")
    k = 0
    for length, n, w, tree, ts in cases:
        total = 0
        for q in range(-(-n // (1 << ts)) + 1):
            lo, hi, tile0, tiles, prefix = map(int, out[k].split())
            k += 1
            assert prefix == total
            tokens = range(q << ts, min(n, (q + 1) << ts))
            if not tokens:
                continue
            # a tree's tokens may have any depth, a chain's have their number
            first = min((length + (0 if tree else i) - w + 1 for i in tokens), default=0) if w else 0
            assert lo == max(0, first) and hi == length + tokens[-1] + 1
            assert tile0 == lo // 128 and tiles == -(-hi // 128) - tile0 >= 1
            total += tiles


WHOLE = r"""
#include "paged.cuh"
#include <cstdio>
#include <vector>
int main() {   // a batch per line: CTAs, kv heads, window, tree, ts, a unit's cost, sequences, their lengths and new tokens
  int grid, heads, w, tree, ts, unit_cost, B;
  while (scanf("%d %d %d %d %d %d %d", &grid, &heads, &w, &tree, &ts, &unit_cost, &B) == 7) {
    std::vector<int> len(B), n(B);
    long long all = 0, exact = 0, taken = 0;
    int units = 0, longest = 0;
    for (int b = 0; b < B; ++b) {
      if (scanf("%d %d", &len[b], &n[b]) != 2) return 1;
      if (n[b] == 0) continue;
      const int nq = g3::paged_units(n[b], ts);
      all += heads * (g3::kTileCost * g3::paged_prefix(len[b], n[b], w, tree, ts, nq) + (long long)unit_cost * nq);
      exact += (long long)heads * nq;
      units += g3::paged_count_units(n[b], ts, heads);
      const int t = g3::paged_most_tiles(len[b], n[b], w, tree, ts);
      if (t > longest) longest = t;
    }
    const g3::PagedWhole p = g3::paged_whole(all, units, longest, grid, w);
    for (int b = 0; b < B; ++b)
      taken += (long long)heads * g3::paged_units(n[b], ts) * g3::paged_whole_shares(p, len[b], n[b], w, tree, ts);
    printf("%d %lld %lld %d\n", p.uncut, taken, exact, g3::kMaxCtas);
  }
}
"""


def test_whole_shares_fit_the_ctas(tmp_path):
    """What CTAs take whole is no more than there are CTAs: all units where they
    stay uncut, and else shares that leave a CTA for the rest."""
    src, exe = tmp_path / "whole.cu", tmp_path / "whole"
    src.write_text(WHOLE)
    subprocess.run([_nvcc(), "-std=c++17", "-I", CSRC, "-I", INCLUDE, "-o", str(exe), str(src)], check=True,
                   capture_output=True, env=dict(os.environ))
    rng = random.Random(5)
    lines, grids = [], []
    for grid in (1, 7, 132, 152, 159, 160):
        # one sequence of many units, beside ones without new tokens
        for n in (64 * k + d for k in (1, 9, 10, 11, 32, 200) for d in (-1, 0, 1)):
            for window in (0, 100):
                lines.append(f"{grid} 16 {window} 0 6 5 3 0 0 5 {n} 9 0")
                grids.append(grid)
        for _ in range(300):
            tree, B = rng.random() < 0.2, rng.choice([1, 2, 5, 40])
            top = 64 if tree else rng.choice([1, 60, 300, 5000])
            lens = [rng.choice([0, 100, 4000, 60000]) + rng.randint(0, 300) for _ in range(B)]
            new = [rng.choice([0, 1, rng.randint(1, top)]) for _ in range(B)]
            lines.append(f"{grid} {rng.choice([1, 4, 16])} {rng.choice([0, 0, 1, 700])} {int(tree)} {rng.randint(5, 8)} "
                         f"5 {B} " + " ".join(f"{a} {c}" for a, c in zip(lens, new)))
            grids.append(grid)
    out = subprocess.run([str(exe)], input="\n".join(lines), text=True, capture_output=True,
                         check=True).stdout.splitlines()
    assert len(out) == len(lines)
    seen = set()
    for line, grid, got in zip(lines, grids, out):
        uncut, taken, units, most = map(int, got.split())
        assert grid <= most
        assert taken == units <= grid if uncut else taken < grid, line
        seen.add((uncut, taken > 0))
    assert seen >= {(1, True), (0, True), (0, False)}


@pytest.mark.parametrize("name", ["rows", "T_max", "page_size", "n_pages"])
def test_sizes_beyond_32_bits_are_refused(name):
    sizes = dict(rows=3, T_max=2, page_size=16, n_pages=8)
    lens, starts, table = torch.zeros(2).int(), torch.zeros(3).int(), torch.zeros((2, 4)).int()
    assert G3.paged_batch(lens, starts, table, **sizes).sizes == (2, 3, 2, 16, 8, 4)
    sizes[name] += 1 << 32                    # the same lower 32 bits
    with pytest.raises(ValueError, match="32 bits"):
        G3.paged_batch(lens, starts, table, **sizes)
