"""Host threads that share the default stream and leave the scratch to the
binding: aq_qqmm_int8 (two launches a call) and aq_moe, in different sizes, so
that one thread's scratch grows while the other's calls are under way."""
import threading

import pytest
import torch

from group_wise_affine_quant_b200 import api
from group_wise_affine_quant_b200.inputs import gen, normal
from tests.gpu_util import to_dev
from tests.test_gpu_moe import Layer

pytestmark = pytest.mark.gpu


def _product(M, N, K, seed):
    x = to_dev(normal((M, K), 1.0, 1, gen(seed)))
    wq, ws = api.aq_quantize_int8(to_dev(normal((N, K), 0.02, 1, gen(seed + 1))))
    return lambda space=None: (api.aq_qqmm_int8(x, wq, ws, workspace=space),)


def _layer(T, H, I, k, seed):
    L = Layer(8, H, I, gs=32, seed=seed)
    x = L.x(T)
    return lambda space=None: api.aq_moe(x, L.router, *L.m, k, True, workspace=space, **L.kw)


def test_two_threads_on_the_default_stream():
    calls = [[_product(64, 512, 1024, 1), _layer(3, 512, 256, 2, 31), _product(5, 300, 2048, 3)],
             [_layer(2, 256, 512, 3, 32), _product(48, 512, 1024, 5), _product(700, 128, 2048, 7),
              _layer(20, 512, 512, 4, 33), _product(1500, 64, 4096, 9)]]
    want = [[f(api.Workspace()) for f in mine] for mine in calls]
    torch.cuda.synchronize()
    assert api.lib().aq_device_errors() == 0
    got, errs, meet = [[], []], [], threading.Barrier(2)

    def run(j):
        try:
            meet.wait()
            for _ in range(40):
                got[j].append([f() for f in calls[j]])
        except Exception as e:          # reported by the main thread
            errs.append(e)
    threads = [threading.Thread(target=run, args=(j,)) for j in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errs, errs
    torch.cuda.synchronize()
    assert api.lib().aq_device_errors() == 0
    for j in range(2):
        for outs in got[j]:
            for o, w in zip(outs, want[j]):
                assert all(torch.equal(a, b) for a, b in zip(o, w))
