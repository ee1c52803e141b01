"""GPU tests of the mixture-of-experts layer (aq_moe, aq_moe_experts) against
its formula in 64 bits: every weight format, group size and type, one token to
64, odd group counts per row, slots without an expert, an expert named twice,
ties and NaN among the logits, captured replays, streams and workspaces, and
the layer among W8A8 projections."""
import numpy as np
import pytest
import torch

from group_wise_affine_quant_b200 import api
from group_wise_affine_quant_b200.inputs import gen, normal
from tests import moe_ref
from tests.gpu_util import DEV, TDT, dev_u16, dev_u8, to_dev
from tests.util import u16_to_f64

pytestmark = pytest.mark.gpu


def stack(E, N, K, fmt, bits, gs, dt, seed, std=0.05):
    w = to_dev(normal((E * N, K), std, dt, gen(seed)))
    if fmt == "fp4":
        codes, scales = api.aq_quantize_fp4(w, gs)
        return codes.view(E, N, -1), scales.view(E, N, -1), None
    q, s, b = api.aq_quantize(w, bits, gs)
    return q.view(E, N, -1), s.view(E, N, -1), b.view(E, N, -1)


def host(m):
    q, s, b = m
    if b is None:
        return dev_u8(q), dev_u8(s), None
    return dev_u8(q), dev_u16(s), dev_u16(b)


class Layer:
    def __init__(self, E, H, I, fmt="affine", bits=4, gs=64, dt=1, seed=0):
        self.f = (bits, gs, dt)
        self.kw = dict(bits=bits, group_size=gs)
        self.E, self.H, self.I, self.dt = E, H, I, dt
        self.m = [stack(E, n, k, fmt, bits, gs, dt, seed * 10 + j)
                  for j, (n, k) in enumerate(((I, H), (I, H), (H, I)))]
        self.h = [host(m) for m in self.m]
        self.router = to_dev(normal((E, H), 2 / H ** 0.5, dt, gen(seed * 10 + 5)))

    def x(self, T, seed=1):
        return to_dev(normal((T, self.H), 1.0, self.dt, gen(1000 + seed)))

    def x64(self, x):
        return u16_to_f64(dev_u16(x), self.dt)

    def check_experts(self, x, indices, weights, y, what="y"):
        ref, tol = moe_ref.experts(self.x64(x), indices.cpu().numpy(),
                                   weights.cpu().double().numpy(), *self.h, *self.f)
        moe_ref.check(dev_u16(y), ref, tol, self.dt, what)

    def check_moe(self, x, k, normalize, out):
        y, indices, weights = out
        r64 = u16_to_f64(dev_u16(self.router), self.dt)
        at, w = moe_ref.route(self.x64(x), r64, k, normalize)
        assert np.array_equal(indices.cpu().numpy(), at)
        # expf (2 ulp), sums over E <= 512 in fp32, a division: below 2^-19 together
        assert np.all(np.abs(weights.cpu().double().numpy() - w) <= 2.0 ** -19 * w + 1e-37)
        self.check_experts(x, indices, weights, y)


def errors():
    torch.cuda.synchronize()
    assert api.lib().aq_device_errors() == 0


FORMATS = [("affine", b, g) for b in (2, 3, 4, 5, 6, 8) for g in (32, 64, 128)] + \
          [("fp4", 4, 16), ("fp4", 4, 32)]


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("fmt,bits,gs", FORMATS)
def test_formats(fmt, bits, gs, dt):
    """Each format with row lengths that end inside a stage and an odd number
    of groups in a row (scale rows of any alignment)."""
    unit = max(gs, 32)
    L = Layer(5, unit * (9 if gs <= 32 else 7), unit * 3, fmt, bits, gs, dt, seed=bits + gs)
    x = L.x(6)
    L.check_moe(x, 2, True, api.aq_moe(x, L.router, *L.m, 2, True, **L.kw))
    errors()


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 17, 33, 64])
@pytest.mark.parametrize("E,k", [(1, 1), (3, 2), (40, 8)])
def test_tokens_and_experts(T, E, k):
    """From one pair to tiles of one expert that hold all tokens."""
    L = Layer(E, 256, 192, seed=E)
    x = L.x(T, T)
    L.check_moe(x, k, T % 2 == 0, api.aq_moe(x, L.router, *L.m, k, T % 2 == 0, **L.kw))
    errors()


def test_largest_counts():
    """512 experts, 16 slots, 64 tokens: the most pairs there can be."""
    L = Layer(512, 64, 64, gs=32, seed=3)
    x = L.x(64)
    L.check_moe(x, 16, True, api.aq_moe(x, L.router, *L.m, 16, True, **L.kw))
    errors()


@pytest.mark.parametrize("H,I", [(2048, 768), (4096, 64), (64, 4096), (32, 32)])
@pytest.mark.parametrize("dt", [0, 1])
def test_widths(H, I, dt):
    """Long and short rows in either product (teams of warps share long ones)."""
    L = Layer(4, H, I, gs=32, dt=dt, seed=H + I)
    x = L.x(3)
    L.check_moe(x, 2, False, api.aq_moe(x, L.router, *L.m, 2, False, **L.kw))
    errors()


@pytest.mark.parametrize("fmt,bits,gs,H,I", [
    ("affine", 4, 64, 8256, 64),        # gate and up rows in three pieces, the last a single group
    ("affine", 4, 32, 64, 4128),        # down
    ("affine", 8, 64, 4160, 2112),      # both, 8-bit rows
    ("affine", 3, 64, 4160, 2112),      # rows that start at any 4 bytes
    ("affine", 6, 32, 2080, 2080),
    ("affine", 2, 128, 8320, 128),
    ("fp4", 4, 32, 4128, 2080),         # scale rows of odd length
    ("fp4", 4, 16, 8224, 4128)])
@pytest.mark.parametrize("T", [2, 7])
def test_rows_in_several_passes(fmt, bits, gs, H, I, T):
    """Rows longer than a CTA's warps hold at once, with token tiles of up to 4
    (T = 2) and of up to 8 pairs (T = 7, all at one expert)."""
    L = Layer(2, H, I, fmt, bits, gs, 1, seed=bits + T)
    x = L.x(T)
    indices = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    if T == 2:
        indices[1] = 1
    weights = torch.full((T, 1), 0.25, device=DEV)
    y = api.aq_moe_experts(x, indices, weights, *L.m, **L.kw)
    L.check_experts(x, indices, weights, y)
    errors()


@pytest.mark.parametrize("counts", [[4, 4, 4], [5, 1, 1], [8, 1, 0], [9, 9, 0], [12, 3, 1], [20, 2, 2], [33, 0, 1]])
def test_pairs_per_expert(counts):
    """Token tiles of 4 and of 8 pairs, full and cut off."""
    L = Layer(len(counts), 192, 96, gs=32, seed=sum(counts))
    order = [e for e, c in enumerate(counts) for _ in range(c)]
    T = len(order)
    indices = torch.tensor(order, dtype=torch.int32)[torch.randperm(T, generator=gen(T))].view(T, 1).to(DEV)
    weights = torch.rand((T, 1), device=DEV)
    x = L.x(T)
    L.check_experts(x, indices, weights, api.aq_moe_experts(x, indices, weights, *L.m, **L.kw))
    errors()


def test_slots_without_an_expert():
    """-1 and other indices outside the stack skip their slot whatever its
    weight; a token with none gives zeros; the same expert twice counts twice."""
    L = Layer(4, 128, 128, seed=8)
    x = L.x(6)
    indices = torch.tensor([[0, 1, 2], [-1, 3, -1], [-1, -7, 4], [2, 2, 1], [1 << 30, 0, 0],
                            [3, -2147483648, 3]], dtype=torch.int32, device=DEV)
    weights = torch.rand((6, 3), device=DEV)
    bad = (indices < 0) | (indices >= 4)
    L.check_experts(x, indices, weights, api.aq_moe_experts(x, indices, weights, *L.m, **L.kw))
    for v in (float("nan"), float("inf"), -3.4e38):
        w = torch.where(bad, torch.full_like(weights, v), weights)
        y = api.aq_moe_experts(x, indices, w, *L.m, **L.kw)
        assert int(y[2].count_nonzero()) == 0
        L.check_experts(x, indices, torch.where(bad, 0.0, w), y)
    none = torch.full_like(indices, -1)
    assert int(api.aq_moe_experts(x, none, weights, *L.m, **L.kw).count_nonzero()) == 0
    errors()


def test_more_slots_than_experts():
    L = Layer(2, 64, 64, gs=32, seed=9)
    x = L.x(5)
    indices = torch.randint(0, 2, (5, 7), dtype=torch.int32, device=DEV)
    weights = torch.randn((5, 7), device=DEV)          # negative weights too
    L.check_experts(x, indices, weights, api.aq_moe_experts(x, indices, weights, *L.m, **L.kw))
    errors()


def test_ties_go_to_the_lower_index():
    L = Layer(40, 64, 64, gs=32, seed=10)
    x = L.x(3)
    router = L.router[:1].repeat(40, 1).contiguous()
    _, indices, weights = api.aq_moe(x, router, *L.m, 4, False, **L.kw)
    assert indices.tolist() == [[0, 1, 2, 3]] * 3
    assert torch.allclose(weights, torch.full_like(weights, 1 / 40), rtol=1e-6)
    zero = torch.zeros_like(router)                    # +0 and -0 are equal
    zero[::2] = -0.0
    assert api.aq_moe(x, zero, *L.m, 4, False, **L.kw)[1].tolist() == [[0, 1, 2, 3]] * 3
    errors()


def test_not_finite():
    """A NaN in a token or in one expert's router row shows in the weights and
    y of the tokens it meets, in no other token, and every index stays valid."""
    L = Layer(8, 64, 64, gs=32, seed=11)
    x = L.x(4)
    x[1, 5] = float("nan")
    y, indices, weights = api.aq_moe(x, L.router, *L.m, 3, True, **L.kw)
    assert torch.isnan(y[1]).all() and torch.isnan(weights[1]).all()
    assert sorted(indices[1].tolist()) == [0, 1, 2]
    ok = [0, 2, 3]
    L.check_moe(x[ok].contiguous(), 3, True, (y[ok].contiguous(), indices[ok], weights[ok]))
    router = L.router.clone()
    router[6, 0] = float("nan")
    _, indices, weights = api.aq_moe(L.x(4), router, *L.m, 3, True, **L.kw)
    assert torch.isnan(weights).all() and not (indices == 6).any()
    for row in indices.tolist():
        assert len(set(row)) == 3 and all(0 <= e < 8 for e in row)
    errors()


def test_large_h_in_fp16():
    """h far above fp16's range inside, y back in it."""
    L = Layer(2, 64, 64, gs=32, dt=0, seed=12)
    x = L.x(2) * 200
    d = list(L.m[2])
    d[1], d[2] = d[1] / 256, d[2] / 256
    L.m[2] = tuple(d)
    L.h[2] = host(L.m[2])
    L.m[1] = (L.m[1][0], L.m[1][1] * 16, L.m[1][2] * 16)
    L.h[1] = host(L.m[1])
    indices = torch.tensor([[0, 1], [1, 0]], dtype=torch.int32, device=DEV)
    weights = torch.full((2, 2), 0.01, device=DEV)
    y = api.aq_moe_experts(x, indices, weights, *L.m, **L.kw)
    assert torch.isfinite(y).all()
    L.check_experts(x, indices, weights, y)
    errors()


def test_same_bits_twice_and_counters():
    L = Layer(16, 512, 256, seed=13)
    x = L.x(20)
    ws = api.Workspace()
    outs = [api.aq_moe(x, L.router, *L.m, 4, True, workspace=ws, **L.kw) for _ in range(3)]
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    assert int(ws.get(x.device, 1)[:65536].count_nonzero()) == 0
    y = api.aq_moe_experts(x, outs[0][1], outs[0][2], *L.m, **L.kw)
    assert torch.equal(y, outs[0][0])
    errors()


def test_out_and_neighbours():
    """y goes into `out`, and nothing around it changes."""
    L = Layer(3, 96, 64, gs=32, seed=14)
    x = L.x(5)
    room = torch.full((7, 96), 7.0, dtype=TDT[1], device=DEV)
    out = room[1:6]
    indices = torch.zeros((5, 1), dtype=torch.int32, device=DEV)
    weights = torch.ones((5, 1), device=DEV)
    got = api.aq_moe_experts(x, indices, weights, *L.m, out=out, **L.kw)
    assert got.data_ptr() == out.data_ptr()
    L.check_experts(x, indices, weights, out)
    assert (room[0] == 7).all() and (room[6] == 7).all()
    errors()


def test_offsets_past_32_bits():
    """Experts that lie beyond 2^31 bytes of their stacks."""
    E, H, I = 512, 4096, 2176
    g = torch.Generator(device=DEV)
    g.manual_seed(1)

    def big(N, K):
        q = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device=DEV, generator=g)
        s = torch.rand((E, N, K // 128), device=DEV, generator=g).mul(0.01).to(TDT[1])
        return q, s, (-8 * s.float()).to(TDT[1])
    m = [big(I, H), big(I, H), big(H, I)]
    assert m[0][0].numel() > 1 << 31
    x = to_dev(normal((2, H), 1.0, 1, gen(2)))
    indices = torch.tensor([[510, 0], [511, 7]], dtype=torch.int32, device=DEV)
    weights = torch.full((2, 2), 0.5, device=DEV)
    y = api.aq_moe_experts(x, indices, weights, *m, bits=4, group_size=128)
    few = [tuple(t[[510, 0, 511, 7]].contiguous() for t in w) for w in m]
    small = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV)
    ref, tol = moe_ref.experts(u16_to_f64(dev_u16(x), 1), small.cpu().numpy(), weights.cpu().double().numpy(),
                               *[host(w) for w in few], 4, 128, 1)
    moe_ref.check(dev_u16(y), ref, tol, 1)
    errors()


def test_no_tokens():
    L = Layer(3, 64, 64, gs=32, seed=15)
    y, indices, weights = api.aq_moe(L.x(1)[:0], L.router, *L.m, 2, True, **L.kw)
    assert y.shape == (0, 64) and indices.shape == (0, 2) and weights.shape == (0, 2)


def test_graph_replays():
    """Captured once, replayed on other tokens and other routing."""
    L = Layer(6, 128, 128, seed=16)
    x, ws = L.x(4), api.Workspace()
    api.aq_moe(x, L.router, *L.m, 2, True, workspace=ws, **L.kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = api.aq_moe(x, L.router, *L.m, 2, True, workspace=ws, **L.kw)
    for seed in (31, 32):
        x.copy_(L.x(4, seed))
        g.replay()
        torch.cuda.synchronize()
        L.check_moe(x, 2, True, out)
    errors()


def test_two_streams_at_once():
    """Calls in flight on two streams, a workspace each."""
    L = Layer(8, 512, 512, seed=17)
    xs = [L.x(3, s) for s in (41, 42)]
    streams, spaces = [torch.cuda.Stream() for _ in xs], [api.Workspace() for _ in xs]
    want = [api.aq_moe(x, L.router, *L.m, 2, True, **L.kw) for x in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                got[j].append(api.aq_moe(xs[j], L.router, *L.m, 2, True, workspace=spaces[j], **L.kw))
    errors()
    for j in range(2):
        for o in got[j]:
            assert all(torch.equal(a, b) for a, b in zip(o, want[j]))


def test_two_streams_with_the_default_scratch():
    L = Layer(8, 512, 256, seed=19)
    xs = [L.x(3, s) for s in (51, 52)]
    streams = [torch.cuda.Stream() for _ in xs]
    want = [api.aq_moe(x, L.router, *L.m, 2, True, **L.kw) for x in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                got[j].append(api.aq_moe(xs[j], L.router, *L.m, 2, True, **L.kw))
    errors()
    for j in range(2):
        for o in got[j]:
            assert all(torch.equal(a, b) for a, b in zip(o, want[j]))


def test_two_graphs_with_the_default_scratch():
    """Each captured call has scratch of its own: replays on two streams at once
    and eager calls beside them."""
    L = Layer(8, 512, 256, seed=20)
    xs = [L.x(3, s) for s in (61, 62)]
    want = [api.aq_moe(x, L.router, *L.m, 2, True, **L.kw) for x in xs]
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph() for _ in xs], []
    for g, x in zip(graphs, xs):
        with torch.cuda.graph(g):
            outs.append(api.aq_moe(x, L.router, *L.m, 2, True, **L.kw))
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(10):
        for j in range(2):
            with torch.cuda.stream(streams[j]):
                graphs[j].replay()
        eager = api.aq_moe(xs[0], L.router, *L.m, 2, True, **L.kw)
    errors()
    for j in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[j], want[j]))
    assert all(torch.equal(a, b) for a, b in zip(eager, want[0]))


def test_linear_layers_of_a_block():
    """The operators together, as a decoder block's linear layers use them: an
    8-bit projection, the mixture of experts, a second projection, two tokens
    in decode and then five; eagerly, and captured once per count."""
    H, E = 256, 6
    L = Layer(E, H, 128, seed=21)
    proj = [api.aq_quantize_int8(to_dev(normal((H, H), 0.06, 1, gen(s)))) for s in (71, 72)]

    def block(x):
        a = api.aq_qqmm_int8(x, *proj[0])
        y, indices, weights = api.aq_moe(a, L.router, *L.m, 2, True, **L.kw)
        return a, y, indices, weights, api.aq_qqmm_int8(y, *proj[1])

    def check(x, out):
        a, y, indices, weights, z = out
        L.check_moe(a, 2, True, (y, indices, weights))
        for src, (wq, ws), got in ((x, proj[0], a), (y, proj[1], z)):
            xq, xs = api.aq_quantize_int8(src)
            exact = (xq.double() @ wq.double().T).float()
            assert torch.equal(got, ((exact * xs[:, None]) * ws[None, :]).to(got.dtype))
    for T in (2, 5):
        x = L.x(T)
        check(x, block(x))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = block(x)
        for seed in (81, 82):
            x.copy_(L.x(T, seed))
            g.replay()
            torch.cuda.synchronize()
            check(x, out)
    errors()


def test_refuses_what_the_kernel_cannot_take():
    L = Layer(3, 64, 64, gs=32, seed=18)
    x = L.x(2)
    idx, w = torch.zeros((2, 1), dtype=torch.int32, device=DEV), torch.ones((2, 1), device=DEV)
    with pytest.raises(ValueError, match="contiguous"):
        api.aq_moe_experts(L.x(4)[::2], idx, w, *L.m, **L.kw)
    with pytest.raises(TypeError, match="indices"):
        api.aq_moe_experts(x, idx.long(), w, *L.m, **L.kw)
    with pytest.raises(ValueError, match="shape"):
        api.aq_moe_experts(x, idx, w[:1], *L.m, **L.kw)
    with pytest.raises(ValueError, match="CUDA"):
        api.aq_moe_experts(x.cpu(), idx, w, *L.m, **L.kw)
    with pytest.raises(ValueError, match="device"):
        api.aq_moe_experts(x, idx.cpu(), w, *L.m, **L.kw)
    with pytest.raises(ValueError, match="up w_q"):
        api.aq_moe_experts(x, idx, w, L.m[0], tuple(t[:2] for t in L.m[1]), L.m[2], **L.kw)
    with pytest.raises(TypeError, match="w_router"):
        api.aq_moe(x, L.router.float(), *L.m, 1, **L.kw)
    with pytest.raises(api.AqError, match="top_k"):
        api.aq_moe(x, L.router, *L.m, 4, **L.kw)
    with pytest.raises(api.AqError, match="tokens"):
        api.aq_moe(L.x(65), L.router, *L.m, 1, **L.kw)
