"""The mixture-of-experts layer at the ends of its ranges: every pair at one
expert, slots with gaps, and the widest rows in either product."""
import pytest
import torch

from group_wise_affine_quant_b200 import api
from tests.gpu_util import DEV
from tests.test_gpu_moe import Layer, errors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("low", [0, -2])
def test_most_pairs_at_few_experts(low, dt):
    """64 tokens of 16 slots, all at expert 0; then at either of two or at none."""
    L = Layer(2, 128, 96, gs=32, dt=dt, seed=51)
    x = L.x(64)
    high = 1 if low == 0 else 4
    indices = torch.randint(low, high, (64, 16), dtype=torch.int32, device=DEV)
    weights = torch.rand((64, 16), device=DEV) * 0.1
    L.check_experts(x, indices, weights, api.aq_moe_experts(x, indices, weights, *L.m, **L.kw))
    errors()


@pytest.mark.parametrize("H,I", [(65536, 32), (32, 65536)])
@pytest.mark.parametrize("T", [1, 6, 64])
def test_widest_rows(H, I, T):
    L = Layer(2, H, I, gs=32, seed=52)
    x = L.x(T)
    indices = torch.randint(0, 2, (T, 1), dtype=torch.int32, device=DEV)
    weights = torch.ones((T, 1), device=DEV)
    L.check_experts(x, indices, weights, api.aq_moe_experts(x, indices, weights, *L.m, **L.kw))
    errors()


def test_router_of_the_widest_rows():
    L = Layer(3, 65536, 64, "affine", 5, 64, seed=53)
    x = L.x(33)
    L.check_moe(x, 2, True, api.aq_moe(x, L.router, *L.m, 2, True, **L.kw))
    errors()
