"""GPU tests of the W8A8 operators: the row quantizer bit for bit against numpy's
fp32, the integer product bit for bit against a 64-bit integer sum with the
documented roundings, every tile the launcher may choose, and the two in one
call."""
import numpy as np
import pytest
import torch

from group_wise_affine_quant_b200 import api
from group_wise_affine_quant_b200.inputs import gen, normal
from tests.gpu_util import DEV, TDT, dev_u16, to_dev
from tests.util import u16_to_f64

pytestmark = pytest.mark.gpu


def quantize_ref(x_u16, dt):
    """The definition in numpy fp32 (IEEE division, rint to even)."""
    x = u16_to_f64(x_u16, dt).astype(np.float32)
    with np.errstate(all="ignore"):
        s = np.abs(x).max(1) / np.float32(127)
        s = np.where(np.isnan(x).any(1), np.float32(np.nan), s)
        q = np.rint(x / s[:, None])
        q = np.where((s[:, None] > 0) & np.isfinite(s[:, None]), np.clip(q, -127, 127), 0)
    return q.astype(np.int8), s.astype(np.float32)


def check_quantize(x, dt):
    q, s = api.aq_quantize_int8(x)
    torch.cuda.synchronize()
    rq, rs = quantize_ref(dev_u16(x), dt)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("R,K", [(1, 16), (3, 496), (9, 512), (17, 528), (8, 1024), (5, 2048), (2, 2064),
                                 (3, 4096), (2, 4112), (2, 8192), (2, 16384), (2, 16400), (1, 131056)])
def test_quantize(R, K, dt):
    check_quantize(to_dev(normal((R, K), 1.0, dt, gen(R + K))), dt)


@pytest.mark.parametrize("dt", [0, 1])
def test_quantize_edges(dt):
    """Zeros, -0, one value, ties, the type's largest and smallest, infinities
    and NaN, each in a row of its own, in the warp and the block form."""
    big, tiny = float(torch.finfo(TDT[dt]).max), float(torch.finfo(TDT[dt]).smallest_normal)
    sub = tiny * float(torch.finfo(TDT[dt]).eps)
    for K in (64, 2064):
        x = normal((12, K), 1.0, dt, gen(K)).clone()
        x[0] = 0
        x[1] = -0.0
        x[2] = 0
        x[2, K - 1] = -3.0
        x[3] = torch.arange(K, dtype=torch.float32).remainder(255).sub(127).mul(0.5).to(TDT[dt])  # ties
        x[3, 0] = 127.0
        x[4] = big
        x[4, ::2] = -big
        x[5] = sub
        x[5, 3] = -3 * sub
        x[6] = tiny
        x[7, 7] = float("inf")
        x[8, 9] = float("-inf")
        x[9, K - 1] = float("nan")
        x[10, 0], x[10, 1] = float("nan"), float("inf")
        check_quantize(to_dev(x), dt)


@pytest.mark.parametrize("dt", [0, 1])
def test_quantize_every_pattern(dt):
    """Every finite value of the type against several row maxima."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(TDT[dt])
    v = v[torch.isfinite(v)]
    for top in (1.0, 127.0, 3.3, float(torch.finfo(TDT[dt]).max)):
        x = v[v.abs() <= top]
        x = torch.cat([x, torch.full((-(-(x.numel() + 1) // 16) * 16 - x.numel(),), top, dtype=TDT[dt])])
        check_quantize(to_dev(x[None]), dt)


@pytest.mark.parametrize("dt", [0, 1])
def test_quantize_every_maximum(dt):
    """A row for every finite magnitude of the type, which is its largest."""
    top = torch.arange(32768, dtype=torch.int32).to(torch.int16).view(TDT[dt])
    top = top[torch.isfinite(top)]
    x = top[:, None] * torch.linspace(-1, 1, 16).to(TDT[dt])[None, :]
    x[:, 0] = -top
    check_quantize(to_dev(x), dt)


def codes(M, K, seed):
    return torch.randint(-128, 128, (M, K), dtype=torch.int8, generator=gen(seed)).to(DEV)


def scales(n, seed):
    return (torch.rand((n,), generator=gen(seed)) * 0.01 + 1e-4).to(DEV)


def mm_ref(xq, xs, wq, ws, dtype):
    """The documented steps: an exact sum, then three fp32 roundings and the cast."""
    s = xq.double() @ wq.double().T             # exact: below 2^53
    return ((s.float() * xs[:, None]) * ws[None, :]).to(dtype)


def check_mm(M, N, K, dt, seed=0):
    xq, wq, xs, ws = codes(M, K, seed), codes(N, K, seed + 1), scales(M, seed), scales(N, seed + 1)
    y = api.aq_int8_mm(xq, xs, wq, ws, dtype=TDT[dt])
    torch.cuda.synchronize()
    assert torch.equal(y, mm_ref(xq, xs, wq, ws, TDT[dt]))
    assert api.lib().aq_device_errors() == 0


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 7, 48), (2, 129, 144), (3, 2048, 2048), (16, 512, 8192),
                                   (17, 300, 1040), (64, 1000, 512), (65, 257, 256), (200, 131, 2064),
                                   (333, 1001, 1040), (1, 5000, 128), (2048, 640, 384), (1000, 2000, 304)])
@pytest.mark.parametrize("dt", [0, 1])
def test_int8_mm(M, N, K, dt):
    check_mm(M, N, K, dt, seed=M + N + K)


@pytest.mark.parametrize("tokens,pair,splits", [(16, 0, 1), (16, 0, 8), (32, 0, 1), (32, 0, 3), (64, 0, 1),
                                                (64, 0, 5), (128, 0, 1), (128, 0, 7), (128, 1, 1), (256, 1, 1)])
@pytest.mark.parametrize("M,N,K", [(1, 100, 128), (40, 130, 1040), (300, 520, 1296), (257, 513, 16)])
def test_int8_mm_tiles(tokens, pair, splits, M, N, K):
    """Each tile and split on sizes that leave every edge ragged."""
    try:
        api.lib().aq_testing_set_int8_plan(tokens, pair, splits)
        check_mm(M, N, K, 1, seed=tokens + splits)
    finally:
        api.lib().aq_testing_set_int8_plan(0, 0, 0)


def test_int8_mm_many_tiles():
    """More tiles than the GPU holds at once: each CTA and pair takes several."""
    for plan in ((256, 1, 1), (128, 1, 1), (128, 0, 1), (16, 0, 1)):
        try:
            api.lib().aq_testing_set_int8_plan(*plan)
            check_mm(1100, 5000, 272, 1, seed=plan[0])
        finally:
            api.lib().aq_testing_set_int8_plan(0, 0, 0)


def sample(n, seed):
    at = torch.randint(0, n, (40,), generator=gen(seed))
    at[:2] = torch.tensor([0, n - 1])
    return at.to(DEV)


@pytest.mark.parametrize("N", [32768, 32769])
def test_int8_mm_past_32_bits(N):
    """More than 2^31 elements of y, and codes of x beyond 2^31 bytes; rows of y
    by TMA and by the warps.  Checked at a sample of rows."""
    for M, n, K in ((70000, N, 64), (140000, 64 + N % 2, 16384)):
        xq = torch.randint(-128, 128, (M, K), dtype=torch.int8, device=DEV)
        wq, xs, ws = codes(n, K, 3), scales(M, 3), scales(n, 4)
        y = api.aq_int8_mm(xq, xs, wq, ws)
        rows = sample(M, M)
        assert torch.equal(y[rows], mm_ref(xq[rows], xs[rows], wq, ws, y.dtype))
        del xq, y
    assert api.lib().aq_device_errors() == 0


def test_quantize_past_32_bits():
    R, K = 70000, 32768
    x = torch.randn((R, K), dtype=TDT[1], device=DEV)
    q, s = api.aq_quantize_int8(x)
    rows = sample(R, 9)
    rq, rs = quantize_ref(dev_u16(x[rows]), 1)
    assert np.array_equal(q[rows].cpu().numpy(), rq) and np.array_equal(s[rows].cpu().numpy(), rs)


def test_int8_mm_largest_sum():
    """The longest K with the largest products: the 32-bit sum just fits."""
    K = 131056
    for v in (-128, 127):
        xq = torch.full((2, K), v, dtype=torch.int8, device=DEV)
        wq = torch.full((3, K), -128, dtype=torch.int8, device=DEV)
        one = torch.ones((3,), device=DEV)
        y = api.aq_int8_mm(xq, one[:2] * 2.0 ** -10, wq, one)
        assert torch.equal(y, torch.full_like(y, -128.0 * v * K * 2.0 ** -10))


def test_int8_mm_scales_not_finite():
    xq, wq = codes(3, 64, 1), codes(5, 64, 2)
    xs, ws = scales(3, 1), scales(5, 2)
    xs[1], ws[2] = float("nan"), float("inf")
    y = api.aq_int8_mm(xq, xs, wq, ws)
    assert torch.isnan(y[1]).all() and torch.isinf(y[[0, 2], 2]).all()
    keep = [0, 1, 3, 4]
    assert torch.equal(y[[0, 2]][:, keep], mm_ref(xq, xs, wq, ws, y.dtype)[[0, 2]][:, keep])


def test_empty_sizes():
    y = api.aq_int8_mm(codes(0, 32, 1), scales(0, 1), codes(4, 32, 2), scales(4, 2))
    assert y.shape == (0, 4)
    y = api.aq_int8_mm(codes(3, 0, 1), scales(3, 1), codes(4, 0, 2), scales(4, 2))
    assert y.shape == (3, 4) and int(y.count_nonzero()) == 0
    q, s = api.aq_quantize_int8(torch.empty((2, 0), dtype=torch.float16, device=DEV))
    assert q.shape == (2, 0) and s.tolist() == [0.0, 0.0]
    y = api.aq_qqmm_int8(torch.empty((2, 0), dtype=torch.float16, device=DEV), codes(4, 0, 2), scales(4, 2))
    assert y.shape == (2, 4) and int(y.count_nonzero()) == 0


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("M,N,K", [(1, 512, 2048), (5, 2048, 8192), (40, 600, 528), (700, 1024, 1024)])
def test_qqmm_int8(M, N, K, dt):
    """The same bits as the two calls, and the workspace's counters untouched."""
    x = to_dev(normal((M, K), 1.0, dt, gen(M)))
    wq, ws = api.aq_quantize_int8(to_dev(normal((N, K), 0.02, dt, gen(N))))
    space = api.Workspace()
    for _ in range(3):
        y = api.aq_qqmm_int8(x, wq, ws, workspace=space)
    xq, xs = api.aq_quantize_int8(x)
    want = mm_ref(xq, xs, wq, ws, TDT[dt])
    assert torch.equal(y, want)
    assert torch.equal(api.aq_int8_mm(xq, xs, wq, ws, dtype=TDT[dt]), want)
    assert int(space.get(x.device, 1)[:65536].count_nonzero()) == 0
    assert api.lib().aq_device_errors() == 0


def test_chain_on_a_stream_and_in_a_graph():
    """Dependent calls (each reads the last one's y) eagerly on a stream of
    their own, and captured and replayed on a new input."""
    K = 512
    ws = [api.aq_quantize_int8(to_dev(normal((K, K), 0.06, 1, gen(s)))) for s in range(4)]
    space = api.Workspace()

    def chain(x):
        for wq, s in ws:
            x = api.aq_qqmm_int8(x, wq, s, workspace=space)
        return x

    def plain(x):
        for wq, s in ws:
            xq, xs = api.aq_quantize_int8(x)
            torch.cuda.synchronize()
            x = mm_ref(xq, xs, wq, s, x.dtype)
        return x
    x = to_dev(normal((9, K), 1.0, 1, gen(77)))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = chain(x)
    torch.cuda.synchronize()
    assert torch.equal(got, plain(x))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = chain(x)
    x.copy_(to_dev(normal((9, K), 1.0, 1, gen(78))))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, plain(x))
    assert api.lib().aq_device_errors() == 0


def test_weights_written_just_before():
    """The product of aq_qqmm_int8 reads its weights early, yet after a kernel
    that writes them on the same stream."""
    K, N = 4096, 2048
    x = to_dev(normal((4, K), 1.0, 1, gen(3)))
    a = api.aq_quantize_int8(to_dev(normal((N, K), 0.02, 1, gen(4))))
    b = api.aq_quantize_int8(to_dev(normal((N, K), 0.02, 1, gen(5))))
    xq, xs = api.aq_quantize_int8(x)
    wq, ws = torch.empty_like(a[0]), torch.empty_like(a[1])
    got = []
    for i in range(20):
        src = (a, b)[i % 2]
        wq.copy_(src[0])
        ws.copy_(src[1])
        got.append(api.aq_qqmm_int8(x, wq, ws))
    for i, y in enumerate(got):
        src = (a, b)[i % 2]
        assert torch.equal(y, mm_ref(xq, xs, *src, y.dtype))


def test_two_streams_with_the_default_scratch():
    K = 1024
    wq, ws = api.aq_quantize_int8(to_dev(normal((512, K), 0.02, 1, gen(6))))
    x = [to_dev(normal((64, K), 1.0, 1, gen(s))) for s in (7, 8)]
    want = [mm_ref(*api.aq_quantize_int8(v), wq, ws, v.dtype) for v in x]
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(30):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                got[j].append(api.aq_qqmm_int8(x[j], wq, ws))
    torch.cuda.synchronize()
    for j in range(2):
        assert all(torch.equal(y, want[j]) for y in got[j])


def test_weight_prefetch_setting():
    """With the thread's weight prefetch on, after a kernel that writes x only."""
    wq, ws = api.aq_quantize_int8(to_dev(normal((4096, 2048), 0.02, 1, gen(1))))
    x = to_dev(normal((4, 2048), 1.0, 1, gen(2)))
    torch.cuda.synchronize()
    try:
        api.aq_set_weight_prefetch(True)
        for _ in range(5):
            xq, xs = api.aq_quantize_int8(x)
            y = api.aq_int8_mm(xq, xs, wq, ws)
    finally:
        api.aq_set_weight_prefetch(False)
    assert torch.equal(y, mm_ref(xq, xs, wq, ws, y.dtype))


def test_out_and_neighbours():
    """y of odd row length goes into `out`, and nothing around it changes."""
    M, N, K = 21, 333, 272
    room = torch.full((M * N + 128,), 7.0, dtype=TDT[0], device=DEV)
    out = room[64:64 + M * N].view(M, N)
    xq, wq, xs, ws = codes(M, K, 5), codes(N, K, 6), scales(M, 5), scales(N, 6)
    api.aq_int8_mm(xq, xs, wq, ws, out=out)
    assert torch.equal(out, mm_ref(xq, xs, wq, ws, TDT[0]))
    assert (room[:64] == 7).all() and (room[64 + M * N:] == 7).all()


def test_refuses_what_the_kernel_cannot_take():
    xq, wq, xs, ws = codes(4, 64, 1), codes(8, 64, 2), scales(4, 1), scales(8, 2)
    with pytest.raises(ValueError, match="contiguous"):
        api.aq_int8_mm(codes(8, 64, 1)[::2], xs, wq, ws)
    with pytest.raises(TypeError, match="w_q"):
        api.aq_int8_mm(xq, xs, wq.to(torch.uint8), ws)
    with pytest.raises(ValueError, match="x_scales"):
        api.aq_int8_mm(xq, ws, wq, ws)
    with pytest.raises(ValueError, match="CUDA"):
        api.aq_int8_mm(xq.cpu(), xs.cpu(), wq.cpu(), ws.cpu())
    with pytest.raises(ValueError, match="device"):
        api.aq_int8_mm(xq, xs.cpu(), wq, ws)
    with pytest.raises(TypeError):
        api.aq_int8_mm(xq, xs, wq, ws, dtype=torch.float32)
    with pytest.raises(api.AqError, match="multiple of 16"):
        api.aq_quantize_int8(torch.ones((2, 24), dtype=torch.float16, device=DEV))
    with pytest.raises(api.AqError, match="131071"):
        api.aq_int8_mm(codes(1, 131072, 1), xs[:1], codes(2, 131072, 2), ws[:2])
    with pytest.raises(api.AqError, match="aligned"):
        room = torch.empty((4 * 64 + 8,), dtype=torch.int8, device=DEV)
        api.aq_int8_mm(room[8:].view(4, 64), xs, wq, ws)
