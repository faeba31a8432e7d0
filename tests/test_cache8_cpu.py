"""The 8-bit KV cache without a GPU: the oracle's e4m3 against torch's, its
scale rule, and the refusals of the entry points (arguments are checked before
anything reaches a device)."""
import ctypes

import pytest
import torch

from oracle import cache8_oracle as C8
from transformer_attention_gb300 import _lib as L
from transformer_attention_gb300.build import build

P = 1 << 20            # stands for a device pointer; never dereferenced
FAR = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build()
    return L.lib()


def test_oracle_e4m3_matches_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).to(torch.float64)
    got = C8.decode(codes)
    assert torch.equal(torch.isnan(ref), torch.isnan(got))
    assert torch.equal(ref.nan_to_num(7.0), got.nan_to_num(7.0))
    x = torch.cat([torch.randn(4000, dtype=torch.float64) * 2.0 ** k for k in range(-10, 7)])
    x = x.to(torch.float32).to(torch.float64).clamp(-448, 448)
    ties = (C8.TABLE[:126] + C8.TABLE[1:127]) / 2
    x = torch.cat([x, ties, -ties, C8.TABLE[:127], torch.tensor([0.0, -0.0])])
    want = x.to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(C8.encode(x), want)
    far = C8.encode(torch.tensor([float("inf"), float("-inf"), float("nan")], dtype=torch.float64))
    assert far.tolist() == [126, 254, 127]


def test_oracle_scale_rule():
    assert C8.scale_for(0.0) == 2.0 ** -15
    assert C8.scale_for(448.0) == 1.0
    assert C8.scale_for(448.0 + 2.0 ** -10) == 2.0
    assert C8.scale_for(447.0) == 1.0 and C8.scale_for(224.0) == 0.5
    assert C8.scale_for(65504.0) == 256.0


def test_oracle_growth_is_exact_for_normal_numbers():
    """A block's scale that grows by 2^k leaves numbers that stay normal as they were."""
    c = C8.empty(1, 64, 1, 128)
    x = torch.randn(1, 8, 1, 128, generator=torch.Generator().manual_seed(1)).half()
    seg = torch.arange(64)[None]
    c1 = C8.write(c, x, x, seg, None, 0)
    big = torch.full((1, 1, 1, 128), 20.0).half()
    c2 = C8.write(c1, big, big, seg, None, 8)
    assert float(c2["ks"][0, 0, 0]) > float(c1["ks"][0, 0, 0])
    a, b = C8.values(c1, "k")[0, :8], C8.values(c2, "k")[0, :8]
    normal = a.abs() >= 2.0 ** -6 * float(c2["ks"][0, 0, 0])
    assert torch.equal(a[normal], b[normal])
    assert (a - b).abs().max() <= 2.0 ** -10 * float(c2["ks"][0, 0, 0])


# ---------------------------------------------------------------- refusals
#            K  V  ld   seg pad B  T  S   end Hkv dh  K8  V8  ks vs pos stream
WRITE = dict(K=P, V=P, ld=512, seg=P, pad=None, B=1, T=4, S=100, end=0, H_kv=2, d_h=256, K8=P, V8=P,
             ks=P, vs=P, pos=P, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(K=None), -1), (dict(V=None), -1), (dict(seg=None), -1), (dict(K8=None), -1),
    (dict(V8=None), -1), (dict(ks=None), -1), (dict(vs=None), -1), (dict(pos=None), -1),
    (dict(T=0), -1), (dict(B=0), -1), (dict(H_kv=0), -1), (dict(S=0), -1), (dict(end=-1), -1),
    (dict(end=97), -1), (dict(end=2 ** 31 - 1), -1), (dict(S=2 ** 30 + 1), -1), (dict(B=65536), -1),
    (dict(B=60000, S=2 ** 30), -1), (dict(ld=504), -1), (dict(d_h=64), -3), (dict(ld=516), -2),
    (dict(K=P + 8), -2), (dict(V=P + 2), -2), (dict(K8=P + 8), -2), (dict(V8=P + 1), -2),
    (dict(ks=P + 2), -2), (dict(vs=P + 1), -2), (dict(pos=P + 2), -2), (dict(seg=P + 2), -2),
    (dict(pad=P + 1), -2),
])
def test_write_refusals(lib, change, code):
    assert lib.gemma3_kv_cache8_write(*dict(WRITE, **change).values()) == code


READ = dict(K8=P, V8=P, ks=P, vs=P, B=1, S=100, first=0, n=4, H_kv=2, d_h=256, K=P, V=P, ld=512,
            stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(K8=None), -1), (dict(vs=None), -1), (dict(K=None), -1), (dict(V=None), -1),
    (dict(first=-1), -1), (dict(n=-1), -1), (dict(first=97), -1), (dict(n=101), -1),
    (dict(ld=511), -1), (dict(d_h=192), -3), (dict(ld=513), -2), (dict(K=P + 4), -2),
    (dict(K8=P + 4), -2),
])
def test_read_refusals(lib, change, code):
    assert lib.gemma3_kv_cache8_read(*dict(READ, **change).values()) == code


ATTEND = dict(Q=P, K8=P, V8=P, ks=P, vs=P, pos=P, seg=P, pad=None, O=FAR, dt=0, w=None, B=1, T=4, S=100,
              end=0, H=4, H_kv=2, d_h=256, window=0, ws=P, nbytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(Q=None), -1), (dict(O=None), -1), (dict(K8=None), -1), (dict(ks=None), -1),
    (dict(pos=None), -1), (dict(seg=None), -1), (dict(ws=None), -1), (dict(dt=2), -1),
    (dict(H=5), -1), (dict(H=16), -3), (dict(H=6), -3), (dict(d_h=64), -3), (dict(T=0), -1),
    (dict(end=97), -1), (dict(end=-1), -1), (dict(S=0), -1), (dict(Q=P + 8), -2), (dict(O=P + 8), -2),
    (dict(K8=P + 8), -2), (dict(vs=P + 2), -2), (dict(ws=P + 128), -2), (dict(w=P + 2), -2),
    (dict(nbytes=16), -6), (dict(w=P, O=P), -1), (dict(w=P, O=P + 4096), -1), (dict(B=65536), -1),
])
def test_attention_refusals(lib, change, code):
    assert lib.gemma3_cached8_attention(*dict(ATTEND, **change).values()) == code


EVICT = dict(K8=1 << 30, V8=2 << 30, ks=3 << 30, vs=4 << 30, pos=5 << 30, w=6 << 30, B=1, S=100, end=90,
             H_kv=2, d_h=256, keep=40, recent=8, K8d=7 << 30, V8d=8 << 30, ksd=9 << 30, vsd=10 << 30,
             posd=11 << 30, wd=12 << 30, kept=13 << 30, S_dst=64, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(K8=None), -1), (dict(w=None), -1), (dict(pos=None), -1), (dict(K8d=None), -1),
    (dict(wd=None), -1), (dict(posd=None), -1), (dict(kept=None), -1), (dict(keep=0), -1),
    (dict(keep=65), -1), (dict(recent=41), -1), (dict(recent=-1), -1), (dict(end=101), -1),
    (dict(end=-1), -1), (dict(S_dst=0), -1), (dict(d_h=64), -3), (dict(K8d=(7 << 30) + 8), -2),
    (dict(kept=(13 << 30) + 2), -2), (dict(wd=(12 << 30) + 1), -2),
    # the caches must not overlap, nor the outputs one another
    (dict(K8d=1 << 30), -1), (dict(V8d=(1 << 30) + 1024), -1), (dict(posd=5 << 30), -1),
    (dict(wd=6 << 30), -1), (dict(kept=5 << 30), -1), (dict(V8d=7 << 30), -1),
    (dict(wd=11 << 30), -1), (dict(ksd=3 << 30), -1),
])
def test_evict_refusals(lib, change, code):
    assert lib.gemma3_kv_cache8_evict(*dict(EVICT, **change).values()) == code


def test_workspace_sizes(lib):
    n = L.gemma3_cached8_attention_workspace_size(2, 1, 4096, 8, 4, 256)
    w = L.gemma3_cached8_attention_workspace_size(2, 1, 4096, 8, 4, 256, True)
    assert n % 256 == 0 and w >= n
    dims = (2, 1, 2560, 8, 4, 256)
    assert L.gemma3_attn_cached8_workspace_size(dims, 4096) >= n
    b = ctypes.c_size_t()
    assert lib.gemma3_cached8_attention_workspace_size(1, 1, 0, 8, 4, 256, 0, ctypes.byref(b)) == -1
    assert lib.gemma3_cached8_attention_workspace_size(1, 1, 64, 8, 4, 64, 0, ctypes.byref(b)) == -3
    assert lib.gemma3_cached8_attention_workspace_size(1, 1, 64, 8, 4, 256, 0, None) == -1


def test_layer_refusals(lib):
    d = L.gemma3_attn_dims(1, 1, 256, 4, 2, 256)
    base = dict(d=ctypes.byref(d), S=100, end=0, x=P, seg=P, pad=None, Wq=P, Wkv=P, Wo=P, gq=P, gk=P, t=0,
                window=8, base=1e4, scale=1.0, qs=1.0, K8=P, V8=P, ks=P, vs=P, pos=P, w=None, out=P,
                ws=P, nbytes=1 << 40, stream=None)
    for change in (dict(x=None), dict(S=0), dict(end=100), dict(K8=None), dict(vs=None),
                   dict(pos=None), dict(out=None), dict(window=0), dict(base=-1.0)):
        assert lib.gemma3_attn_forward_cached8(*dict(base, **change).values()) < 0, change
