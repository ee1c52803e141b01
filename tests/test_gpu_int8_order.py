"""The product of aq_qqmm_int8 reads its weights before the quantizer of x has
ended: never before a kernel that writes them, also one that lets its
successors start while it runs."""
import pytest
import torch

from group_wise_affine_quant_b200 import api
from group_wise_affine_quant_b200.inputs import gen, normal
from tests.gpu_util import to_dev
from tests.test_gpu_int8 import mm_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("between", [False, True])
def test_weights_quantized_just_before(between):
    """Two weights in turn through one buffer, quantized (some 20 us) right before
    the call, or before a short product on other tensors."""
    N, K = 8192, 4096
    x = to_dev(normal((4, K), 1.0, 1, gen(3)))
    w = [to_dev(normal((N, K), 0.02, 1, gen(s))) for s in (4, 5)]
    plain = [api.aq_quantize_int8(v) for v in w]
    xq, xs = api.aq_quantize_int8(x)
    other = api.aq_quantize_int8(to_dev(normal((32, 64), 1.0, 1, gen(6))))
    want = [mm_ref(xq, xs, *p, x.dtype) for p in plain]
    wq, ws = torch.empty_like(plain[0][0]), torch.empty_like(plain[0][1])
    space = api.Workspace()
    api.aq_qqmm_int8(x, *plain[0], workspace=space)
    torch.cuda.synchronize()
    got = []
    for i in range(20):
        api.aq_quantize_int8(w[i % 2], out=(wq, ws))
        if between:
            api.aq_int8_mm(*other, *other)
        got.append(api.aq_qqmm_int8(x, wq, ws, workspace=space))
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])


def test_operands_quantized_just_before():
    """aq_int8_mm on what two quantizers write right before it."""
    N, K = 4096, 4096
    x = [to_dev(normal((512, K), 1.0, 1, gen(s))) for s in (7, 8)]
    w = [to_dev(normal((N, K), 0.02, 1, gen(s))) for s in (9, 10)]
    plain = [(*api.aq_quantize_int8(a), *api.aq_quantize_int8(b)) for a, b in zip(x, w)]
    want = [mm_ref(*p, x[0].dtype) for p in plain]
    xo, wo = [torch.empty_like(t) for t in plain[0][:2]], [torch.empty_like(t) for t in plain[0][2:]]
    torch.cuda.synchronize()
    got = []
    for i in range(20):
        api.aq_quantize_int8(x[i % 2], out=xo)
        api.aq_quantize_int8(w[i % 2], out=wo)
        got.append(api.aq_int8_mm(*xo, *wo))
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])
