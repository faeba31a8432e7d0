"""Errors that kernels record while a paged batch is at work: a wait that gave up
is reported beside errors of the input."""
import pytest
import torch

from tests import test_gpu_paged as T

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from transformer_attention_gb300.build import build
    build()
    import transformer_attention_gb300 as G3
    G3.lib()


def _record_bad_paged(G3):
    """A sequence of negative length, which the positions' own check records."""
    b = T.make_batch([5], [2], 16, 150)
    b["lens"][0] = -1
    G3.gemma3_paged_positions(T.dev_batch(b), torch.empty(2, dtype=torch.int32, device="cuda"))


def _record_bad_token(G3):
    E = torch.ones((8, 64), dtype=torch.bfloat16, device="cuda")
    G3.gemma3_embed(torch.tensor([9], dtype=torch.int32, device="cuda"), E, 8, 64, 1, 1.0,
                    torch.empty((1, 64), device="cuda"))


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
