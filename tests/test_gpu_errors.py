"""Several device-side errors before one check: mobi_sync_check names each of them."""
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def mobi():
    import token_adaptive_mixed_b200 as m
    from token_adaptive_mixed_b200 import build
    build.build()
    m.lib()
    return m


def _bad_target(mobi):
    mobi.mobi_logprobs(torch.zeros(2, 100, device=DEV), torch.tensor([5, 100], device=DEV))


def _bad_activation(mobi):
    w, sz = mobi.mobi_pack(torch.zeros(64, 256, device=DEV).half())
    x = torch.zeros(4, 256, device=DEV).bfloat16()
    x[1, 5] = 2.0 ** 31
    mobi.mobi_linear(x, torch.zeros(256, 3, device=DEV), None, w, sz, 64)


def _timeout(mobi):
    g = torch.Generator().manual_seed(1)
    x, xs = ref.operand(8, 4096, 1, g, device=DEV)
    w, ws = ref.operand(1024, 4096, 128, g, device=DEV)
    mobi.mobi_debug_set_wait_limit(1)
    try:
        mobi.mobi_fp8_gemm(x, xs, w, ws)
        torch.cuda.synchronize()
    finally:
        mobi.mobi_debug_set_wait_limit(0)


@pytest.mark.parametrize("target_first", [False, True])
def test_a_target_is_reported_beside_an_activation(mobi, target_first):
    mobi.mobi_sync_check()
    for call in (_bad_target, _bad_activation)[::1 if target_first else -1]:
        call(mobi)
    with pytest.raises(mobi.MobiError) as e:
        mobi.mobi_sync_check()
    assert e.value.status == 1 and "vocabulary" in str(e.value) and "2^31" in str(e.value)
    mobi.mobi_sync_check()


@pytest.mark.parametrize("target_first", [False, True])
def test_a_target_is_reported_beside_a_timeout(mobi, target_first):
    """The timeout keeps its status and its own wait site."""
    mobi.mobi_sync_check()
    for call in (_bad_target, _timeout)[::1 if target_first else -1]:
        call(mobi)
    with pytest.raises(mobi.MobiError) as e:
        mobi.mobi_sync_check()
    assert e.value.status == 6 and "vocabulary" in str(e.value) and "wait site 0x5" in str(e.value)
    mobi.mobi_sync_check()


def test_each_error_alone(mobi):
    mobi.mobi_sync_check()
    for call, status, text in ((_bad_target, 1, "vocabulary"), (_bad_activation, 1, "2^31"), (_timeout, 6, "wait site")):
        call(mobi)
        with pytest.raises(mobi.MobiError) as e:
            mobi.mobi_sync_check()
        assert e.value.status == status and text in str(e.value) and ";" not in str(e.value)
        mobi.mobi_sync_check()
