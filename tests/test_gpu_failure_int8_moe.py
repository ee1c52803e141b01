"""The failure path of the bounded waits of the mixture-of-experts and W8A8
kernels, without a fault: test hooks (include/aq_testing.h) shorten the waits
to 2 ms and hold one role back for 50 ms.  The kernel must set bit 0 of
aq_device_errors() and return, the context stays usable, and later calls on the
same scratch are right."""
import contextlib

import pytest
import torch

from group_wise_affine_quant_b200 import api
from group_wise_affine_quant_b200._lib import AQ_OK, lib
from tests.gpu_util import DEV
from tests.test_gpu_int8 import codes, mm_ref, scales
from tests.test_gpu_moe import Layer

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def waits_run_out():
    torch.cuda.synchronize()
    assert lib().aq_device_errors() == 0
    try:
        lib().aq_testing_set_wait_limit_ns(2_000_000)
        lib().aq_testing_set_start_delay_ns(50_000_000)
        yield
        torch.cuda.synchronize()
    finally:
        lib().aq_testing_set_wait_limit_ns(0)
        lib().aq_testing_set_start_delay_ns(0)
    assert lib().aq_device_errors() & 1, "the bounded waits did not report running out"
    assert lib().aq_testing_clear_device_errors() == AQ_OK
    assert lib().aq_device_errors() == 0


@pytest.mark.parametrize("own_workspace", [True, False])
@pytest.mark.parametrize("router", [True, False])
def test_moe_scratch_serves_again(router, own_workspace):
    """With a router the other CTAs give up at the first barrier and the late one
    at the second; without, at what is then the first."""
    L = Layer(8, 512, 256, gs=32, seed=41)
    x = L.x(9)
    want, indices, weights = api.aq_moe(x, L.router, *L.m, 2, True, **L.kw)
    space = api.Workspace() if own_workspace else None

    def call():
        if router:
            return api.aq_moe(x, L.router, *L.m, 2, True, workspace=space, **L.kw)[0]
        return api.aq_moe_experts(x, indices, weights, *L.m, workspace=space, **L.kw)
    for _ in range(2):
        with waits_run_out():
            call()
        if space:
            assert int(space.get(x.device, 1)[:65536].count_nonzero()) == 0
        got = [call() for _ in range(3)]
        assert all(torch.equal(y, want) for y in got)
    torch.cuda.synchronize()
    assert lib().aq_device_errors() == 0


@pytest.mark.parametrize("tokens,pair,splits", [(16, 0, 1), (32, 0, 4), (64, 0, 8), (128, 0, 1), (128, 1, 1),
                                                (256, 1, 1)])
@pytest.mark.parametrize("M,N,K", [(40, 300, 272), (600, 1000, 4096)])
def test_int8_mm_returns_and_serves_again(tokens, pair, splits, M, N, K):
    """The products' and the stores' waits run out while the TMA warp is held back;
    it then finds the flag.  K = 272: all copies fit the ring, so that the warp
    ends with copies in flight; 4096: it gives up on its own wait."""
    xq, wq, xs, ws = codes(M, K, 1), codes(N, K, 2), scales(M, 1), scales(N, 2)
    want = mm_ref(xq, xs, wq, ws, torch.bfloat16)
    room = torch.full((M * N + 128,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = room[64:64 + M * N].view(M, N)
    try:
        lib().aq_testing_set_int8_plan(tokens, pair, splits)
        with waits_run_out():
            api.aq_int8_mm(xq, xs, wq, ws, out=out)
        for _ in range(2):
            assert torch.equal(api.aq_int8_mm(xq, xs, wq, ws, out=out), want)
    finally:
        lib().aq_testing_set_int8_plan(0, 0, 0)
    assert (room[:64] == 7).all() and (room[64 + M * N:] == 7).all()
    assert lib().aq_device_errors() == 0


def test_qqmm_int8_after_a_time_out():
    x = torch.randn((9, 1024), device=DEV).to(torch.bfloat16)
    wq, ws = api.aq_quantize_int8(torch.randn((512, 1024), device=DEV).to(torch.bfloat16))
    want = api.aq_qqmm_int8(x, wq, ws)
    with waits_run_out():
        api.aq_qqmm_int8(x, wq, ws)
    assert torch.equal(api.aq_qqmm_int8(x, wq, ws), want)
    torch.cuda.synchronize()
    assert lib().aq_device_errors() == 0
