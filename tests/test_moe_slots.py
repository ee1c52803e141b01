"""Numbers of slots that aq_moe refuses, without a GPU: the tensors are small and
the outputs' allocation and the C call are stood in for."""
import ctypes

import pytest
import torch

from group_wise_affine_quant_b200 import api


@pytest.mark.parametrize("top_k", [17, 1 << 40, (1 << 64) + 2, -3])
def test_refused_before_the_outputs_are_allocated(monkeypatch, top_k):
    T, H, I, E = 2, 64, 64, 4
    dev = torch.device("cpu")
    sizes = []
    empty = torch.empty

    def small(*size, **kw):
        assert all(n <= 64 for n in size)
        sizes.append(size)
        return empty(*size, **kw)
    seen = {}

    def call(*args):
        seen["top_k"] = args[12]
        return 1
    monkeypatch.setattr(api, "_moe_stacks", lambda *a: (0, (0,) * 9))
    monkeypatch.setattr(api, "_fits", lambda *a: True)
    monkeypatch.setattr(api, "_current_device", lambda: -1)
    monkeypatch.setattr(api, "_stream_of", lambda d: 0)
    monkeypatch.setattr(api, "_workspace", lambda *a: (None, None, 0))
    monkeypatch.setattr(api, "_by_address", lambda name: call)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=dev)
    gate = (torch.zeros((E, I, H // 2), dtype=torch.uint8),)
    router = torch.zeros((E, H), dtype=torch.bfloat16)
    monkeypatch.setattr(torch, "empty", small)
    with pytest.raises(api.AqError):
        api.aq_moe(x, router, gate, gate, gate, top_k)
    assert not 1 <= ctypes.c_int64(seen["top_k"]).value <= 16 and sizes
