"""Host-side refusals of the W8A8 and mixture-of-experts entry points (no GPU:
the addresses are never dereferenced)."""
import pytest

from group_wise_affine_quant_b200 import _lib

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA, WORKSPACE = range(6)
A = 0x10000


def L():
    return _lib.lib()


def test_quantize_int8():
    q = L().aq_quantize_int8
    assert q(A, A, A, 4, 64, 2, None) == UNSUPPORTED
    assert q(A, A, A, 4, 24, 1, None) == INVALID
    assert q(A, A, A, -1, 64, 1, None) == INVALID
    assert q(A, A, A, (1 << 30) + 1, 16, 1, None) == INVALID
    assert q(A + 8, A, A, 4, 64, 1, None) == MISALIGNED
    assert q(A, A + 8, A, 4, 64, 1, None) == MISALIGNED
    assert q(A, A, A + 2, 4, 64, 1, None) == MISALIGNED
    assert q(None, A, A, 4, 64, 1, None) == INVALID
    assert q(A, A, None, 4, 64, 1, None) == INVALID
    assert q(None, None, None, 0, 64, 1, None) == OK


def test_int8_mm():
    def f(**kw):
        a = dict(x=A, xs=A, w=A, ws=A, y=A, M=4, N=8, K=64, dt=1)
        a.update(kw)
        return L().aq_int8_mm(a["x"], a["xs"], a["w"], a["ws"], a["y"], a["M"], a["N"], a["K"], a["dt"], None)
    assert f(dt=2) == UNSUPPORTED
    assert f(K=72) == INVALID and f(K=131072) == INVALID
    assert b"131071" in L().aq_last_error()
    assert f(M=-1) == INVALID and f(N=(1 << 30) + 1) == INVALID
    for name in ("x", "xs", "w", "ws", "y"):
        assert f(**{name: None}) == INVALID
    for name in ("x", "w", "y"):
        assert f(**{name: A + 8}) == MISALIGNED
    for name in ("xs", "ws"):
        assert f(**{name: A + 2}) == MISALIGNED
    assert f(M=0, x=None, y=None) == OK and f(N=0, w=None, y=None) == OK


def test_qqmm_int8():
    q = L().aq_qqmm_int8
    size = lambda M, N, K: L().aq_workspace_size(5, M, N, K, 8, 16, 0, 1)
    assert size(4, 8, 64) == 65536 + 256 + 256
    assert size(1000, 8, 4096) == 65536 + 1000 * 4096 + 4096
    assert size(0, 8, 64) == 0 and size(4, 8, 131072) == 0
    assert q(A, A, A, A, 4, 8, 64, 1, None, 0, None) == WORKSPACE
    assert q(A, A, A, A, 4, 8, 64, 1, A, 65536 + 511, None) == WORKSPACE
    assert q(A, A, A, A, 4, 8, 64, 1, A + 16, 1 << 20, None) == MISALIGNED
    assert q(A + 2, A, A, A, 4, 8, 64, 1, A, 1 << 20, None) == MISALIGNED
    assert q(None, A, A, A, 4, 8, 64, 1, A, 1 << 20, None) == INVALID
    assert q(A, A, None, A, 4, 8, 64, 1, A, 1 << 20, None) == INVALID
    assert q(A, A, A, A, 4, 8, 40, 1, A, 1 << 20, None) == INVALID
    assert q(A, A, A, A, 0, 8, 64, 1, None, 0, None) == OK


def _m(**kw):
    f = dict(w_q=A, scales=A, biases=A)
    f.update(kw)
    return _lib.MoeMatrix(f["w_q"], f["scales"], f["biases"])


def _moe(router=True, **kw):
    a = dict(x=A, r=A, g=_m(), u=_m(), d=_m(), y=A, i=A, w=A, T=4, H=128, I=64, E=8, k=2, norm=1, bits=4,
             gs=64, mode=0, dt=1, ws=A, wsb=1 << 30)
    a.update(kw)
    tail = (a["bits"], a["gs"], a["mode"], a["dt"], a["ws"], a["wsb"], None)
    sizes = (a["T"], a["H"], a["I"], a["E"], a["k"])
    if router:
        return L().aq_moe(a["x"], a["r"], a["g"], a["u"], a["d"], a["y"], a["i"], a["w"], *sizes, a["norm"], *tail)
    return L().aq_moe_experts(a["x"], a["i"], a["w"], a["g"], a["u"], a["d"], a["y"], *sizes, *tail)


@pytest.mark.parametrize("router", [True, False])
def test_moe(router):
    f = lambda **kw: _moe(router, **kw)
    assert f(bits=7) == UNSUPPORTED and f(dt=2) == UNSUPPORTED and f(gs=16) == UNSUPPORTED
    assert f(T=65) == INVALID and f(T=-1) == INVALID
    assert f(E=0) == INVALID and f(E=513) == INVALID
    assert f(k=0) == INVALID and f(k=17) == INVALID
    assert f(H=96) == INVALID and f(I=32) == INVALID and f(H=0) == INVALID and f(H=65600) == INVALID
    assert f(mode=1, gs=16, H=48, g=_m(biases=None), u=_m(biases=None), d=_m(biases=None)) == INVALID
    for name in ("g", "u", "d"):
        assert f(**{name: _m(w_q=None)}) == INVALID
        assert f(**{name: _m(biases=None)}) == INVALID
        assert f(**{name: _m(scales=A + 8)}) == MISALIGNED
        assert f(**{name: None}) == INVALID
    assert b"down" in L().aq_last_error()
    assert f(mode=1, gs=32) == INVALID                          # FP4 takes no biases
    for name in ("x", "y", "i", "w"):
        assert f(**{name: None}) == INVALID
    for name in ("x", "y"):
        assert f(**{name: A + 8}) == MISALIGNED
    assert f(i=A + 2) == MISALIGNED
    need = L().aq_moe_workspace_size(4, 128, 64, 8, 2)
    assert f(ws=None) == WORKSPACE and f(wsb=need - 1) == WORKSPACE
    assert f(ws=A + 16) == MISALIGNED
    assert f(T=0, ws=None, wsb=0) == OK


def test_moe_router_only():
    assert _moe(r=None) == INVALID
    assert _moe(r=A + 8) == MISALIGNED
    assert _moe(k=9) == INVALID                                 # more slots than experts
    assert b"top_k" in L().aq_last_error()


def test_moe_workspace():
    ws = L().aq_moe_workspace_size
    # counters, logits, h and the results of each pair
    assert ws(4, 128, 64, 8, 2) == 65536 + 256 + 4 * 2 * 64 * 4 + 4 * 2 * 128 * 4
    assert ws(0, 128, 64, 8, 2) == 0 and ws(65, 128, 64, 8, 2) == 0
    assert ws(4, 128, 64, 513, 2) == 0 and ws(4, 128, 64, 8, 17) == 0


def test_binding_refuses_tensors_off_the_gpu():
    import torch

    from group_wise_affine_quant_b200 import api
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    q, s = torch.zeros((3, 64), dtype=torch.int8), torch.zeros((3,))
    with pytest.raises(ValueError, match="CUDA"):
        api.aq_quantize_int8(x)
    with pytest.raises(ValueError, match="CUDA"):
        api.aq_qqmm_int8(x, q, s)
    with pytest.raises(ValueError, match="dimensions"):
        api.aq_qqmm_int8(x[0], q, s)
    with pytest.raises(TypeError):
        api.aq_quantize_int8(x.float())
