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
