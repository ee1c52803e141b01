"""Thin Python binding over the C ABI (include/aq.h), one function per entry
point with the same name.  It only marshals arguments: torch tensors supply
device memory and the current CUDA stream; every step of the computation runs
in libaq.so's kernels.

Tensors: x / w / y are fp16 or bf16 CUDA tensors; w_q is uint8 [N, K*bits/8];
affine scales / biases are T [N, K/group_size]; FP4 scales are uint8.  The
W8A8 functions take int8 codes and fp32 scales; the mixture-of-experts ones
take stacks [E, ...] of the same weights.
"""
import ctypes
import functools
import threading

import torch

from . import _lib
from ._lib import (AQ_BF16, AQ_F16, AQ_MODE_AFFINE, AQ_MODE_FP4, AQ_OP_QCONV2D, AQ_OP_QMM,
                   AQ_OP_QMM_NT, AQ_OP_QMV, AQ_OP_QQMM, AQ_OP_QQMM_INT8, AqError, check, lib)

__all__ = ["aq_quantize", "aq_quantize_fp4", "aq_quantize_dequantize_fp", "aq_qqmm", "aq_dequantize", "aq_qmv", "aq_qmv_batched", "aq_qmm", "aq_qmm_nt", "aq_gather_qmm", "aq_qconv2d_nhwc",
           "aq_quantize_int8", "aq_int8_mm", "aq_qqmm_int8", "aq_moe", "aq_moe_experts",
           "aq_workspace_size", "aq_qmv_noalloc", "aq_last_error", "aq_set_weight_prefetch",
           "aq_get_weight_prefetch", "aq_set_input_prefetch", "aq_get_input_prefetch", "AqError", "AQ_MODE_AFFINE", "AQ_MODE_FP4", "Workspace"]

_DT = {torch.float16: AQ_F16, torch.bfloat16: AQ_BF16}
_TORCH_DT = {AQ_F16: torch.float16, AQ_BF16: torch.bfloat16}


def _dt(t):
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError("expected an fp16 or bf16 tensor, got %s" % t.dtype) from None


def _ptr(t):
    return None if t is None else t.data_ptr()


# torch.cuda.current_stream builds an object for each call (2.3 us of a call's
# 10); the handle alone takes 0.1.
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(device):
    if device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _stream_of(device.index)


def _mode(scales):
    return AQ_MODE_FP4 if scales.dtype == torch.uint8 else AQ_MODE_AFFINE


class Workspace:
    """Per-device zero-initialised scratch buffer for the ABI's workspace
    argument, grown on demand (a grown buffer is zero-filled again).  The
    tensor-core qmv kernels keep split-K partials and counters there and leave
    it zero-filled after every call; one Workspace serves calls issued on one
    stream at a time."""

    def __init__(self):
        self._bufs = {}

    def get(self, device, nbytes):
        if nbytes == 0:
            return None
        buf = self._bufs.get(device)
        if buf is None or buf.numel() < nbytes:
            buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
            self._bufs[device] = buf
        return buf


_default_ws = Workspace()


def aq_set_weight_prefetch(enable):
    """Stream weights before waiting on the previous kernel (see include/aq.h)."""
    lib().aq_set_weight_prefetch(1 if enable else 0)


def aq_get_weight_prefetch():
    return bool(lib().aq_get_weight_prefetch())


def aq_set_input_prefetch(enable):
    """Read x before waiting on the previous kernel (see include/aq.h)."""
    lib().aq_set_input_prefetch(1 if enable else 0)


def aq_get_input_prefetch():
    return bool(lib().aq_get_input_prefetch())


def aq_last_error():
    return lib().aq_last_error().decode()


def aq_workspace_size(op, M, N, K, bits, group_size, mode=AQ_MODE_AFFINE, groups=1):
    return lib().aq_workspace_size(op, M, N, K, bits, group_size, mode, groups)


def aq_quantize(w, bits=4, group_size=64, out=None):
    """w [N, K] T -> (w_q uint8 [N, K*bits/8], scales T [N, G], biases T [N, G])."""
    N, K = w.shape
    if out is None:
        G = K // group_size if group_size > 0 else 0
        out = (torch.empty((N, K * bits // 8), dtype=torch.uint8, device=w.device),
               torch.empty((N, G), dtype=w.dtype, device=w.device),
               torch.empty((N, G), dtype=w.dtype, device=w.device))
    w_q, s, b = out
    check(lib().aq_quantize(_ptr(w), _ptr(w_q), _ptr(s), _ptr(b), N, K, bits, group_size, _dt(w),
                            _stream(w.device)), "aq_quantize")
    return w_q, s, b


def aq_quantize_fp4(w, group_size=32, out=None):
    """w [N, K] fp16/bf16 -> (codes [N, K/2] uint8, scales [N, K/group_size]
    uint8): E2M1 codes with E8M0 (group 32) or E4M3 (group 16) scales."""
    N, K = w.shape
    if out is None:
        out = (torch.empty((N, K // 2), dtype=torch.uint8, device=w.device),
               torch.empty((N, K // group_size), dtype=torch.uint8, device=w.device))
    check(lib().aq_quantize_fp4(_ptr(w), _ptr(out[0]), _ptr(out[1]), N, K, group_size, _dt(w),
                                _stream(w.device)), "aq_quantize_fp4")
    return out


def aq_quantize_dequantize_fp(x, bits=4, group_size=32, out=None):
    """Fake quantization of x [N, K] fp16/bf16: E2M1 (bits 4) or E4M3 (bits 8)
    elements under E8M0 (group 32) or E4M3 (group 16) scales, back in T."""
    N, K = x.shape
    if out is None:
        out = torch.empty_like(x)
    check(lib().aq_quantize_dequantize_fp(_ptr(x), _ptr(out), N, K, bits, group_size, _dt(x),
                                          _stream(x.device)), "aq_quantize_dequantize_fp")
    return out


def aq_qqmm(x, w_q, scales, group_size=32, out=None, workspace=None):
    """W4A4: y = fq(x) . dequant(w)^T with FP4 weights and x fake-quantized to
    the weights' FP4 format."""
    M, K = x.shape
    N = w_q.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
    ws_bytes = aq_workspace_size(AQ_OP_QQMM, M, N, K, 4, group_size, AQ_MODE_FP4)
    ws = (workspace or _default_ws).get(x.device, ws_bytes)
    check(lib().aq_qqmm(_ptr(x), _ptr(w_q), _ptr(scales), _ptr(out), M, N, K, group_size, _dt(x),
                        _ptr(ws), 0 if ws is None else ws.numel(), _stream(x.device)), "aq_qqmm")
    return out


def aq_dequantize(w_q, scales, biases, K, bits=4, group_size=64, dtype=None, out=None):
    """-> w_out T [N, K].  dtype defaults to the affine scales' dtype (bf16 for FP4)."""
    mode = _mode(scales)
    N = w_q.shape[0]
    if dtype is None:
        dtype = scales.dtype if mode == AQ_MODE_AFFINE else torch.bfloat16
    if out is None:
        out = torch.empty((N, K), dtype=dtype, device=w_q.device)
    check(lib().aq_dequantize(_ptr(w_q), _ptr(scales), _ptr(biases), _ptr(out), N, K, bits,
                              group_size, mode, _DT[dtype], _stream(w_q.device)), "aq_dequantize")
    return out


def _mm(fn_name, op, x, w_q, scales, biases, bits, group_size, out, workspace):
    M, K = x.shape
    N = w_q.shape[0]
    mode = _mode(scales)
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
    ws_bytes = aq_workspace_size(op, M, N, K, bits, group_size, mode)
    ws = (workspace or _default_ws).get(x.device, ws_bytes)
    fn = getattr(lib(), fn_name)
    check(fn(_ptr(x), _ptr(w_q), _ptr(scales), _ptr(biases), _ptr(out), M, N, K, bits,
             group_size, mode, _dt(x), _ptr(ws), 0 if ws is None else ws.numel(),
             _stream(x.device)), fn_name)
    return out


def aq_qmv(x, w_q, scales, biases, bits=4, group_size=64, out=None, workspace=None):
    """y = x . dequant(w)^T for 1 <= M <= 16 rows of x."""
    return _mm("aq_qmv", AQ_OP_QMV, x, w_q, scales, biases, bits, group_size, out, workspace)


def aq_qmv_noalloc(x, w_q, scales, biases, bits=4, group_size=64, out=None):
    """aq_qmv on the library's fixed scratch (no workspace; the C call
    allocates nothing).  `out` is allocated here by torch if not given."""
    M, K = x.shape
    N = w_q.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
    check(lib().aq_qmv_noalloc(_ptr(x), _ptr(w_q), _ptr(scales), _ptr(biases), _ptr(out), M, N,
                               K, bits, group_size, _mode(scales), _dt(x), _stream(x.device)),
          "aq_qmv_noalloc")
    return out


def aq_qmv_batched(xs, w_qs, scales, biases, bits=4, group_size=64, outs=None, workspace=None):
    """Independent problems y_i = x_i . dequant(w_i)^T (all x_i with the same
    M <= 16, one dtype, one format) in one call; biases is a list (or None for
    FP4).  Returns the list of outputs."""
    n = len(xs)
    if not (len(w_qs) == len(scales) == n) or (biases is not None and len(biases) != n):
        raise ValueError("one w_q, scales (and biases) per x")
    if n == 0:
        return []
    M = xs[0].shape[0]
    mode = _mode(scales[0])
    if outs is None:
        outs = [torch.empty((M, w.shape[0]), dtype=x.dtype, device=x.device) for x, w in zip(xs, w_qs)]
    arr = (_lib.QmvProblem * n)()
    for i in range(n):
        arr[i] = _lib.QmvProblem(_ptr(xs[i]), _ptr(w_qs[i]), _ptr(scales[i]),
                                 None if biases is None else _ptr(biases[i]), _ptr(outs[i]),
                                 w_qs[i].shape[0], xs[i].shape[1])
    L = lib()
    ws_bytes = L.aq_qmv_batched_workspace_size(arr, n, M, bits, group_size, mode)
    ws = (workspace or _default_ws).get(xs[0].device, ws_bytes)
    check(L.aq_qmv_batched(arr, n, M, bits, group_size, mode, _dt(xs[0]), _ptr(ws),
                           0 if ws is None else ws.numel(), _stream(xs[0].device)),
          "aq_qmv_batched")
    return outs


def aq_gather_qmm(x, w_q, scales, biases, lhs_indices=None, rhs_indices=None, bits=4,
                  group_size=64, out=None, workspace=None):
    """Pair i: y[i] = x[lhs[i]] . dequant(w[rhs[i]])^T, with x [Bx, M, K],
    w_q [E, N, K*bits/8], scales / biases [E, N, K/group_size]; the index
    lists are host sequences of int (None: 0, 1, ...).  Returns [P, M, N]."""
    import ctypes
    Bx, M, K = x.shape
    E, N = w_q.shape[0], w_q.shape[1]
    n = len(lhs_indices) if lhs_indices is not None else (
        len(rhs_indices) if rhs_indices is not None else min(Bx, E))
    mode = _mode(scales)

    def arr(ix):
        if ix is None:
            return None
        return (ctypes.c_int32 * n)(*[int(v) for v in ix])
    if out is None:
        out = torch.empty((n, M, N), dtype=x.dtype, device=x.device)
    L = lib()
    ws_bytes = L.aq_gather_qmm_workspace_size(n, M, N, K, bits, group_size, mode)
    ws = (workspace or _default_ws).get(x.device, ws_bytes)
    check(L.aq_gather_qmm(_ptr(x), _ptr(w_q), _ptr(scales), _ptr(biases), arr(lhs_indices),
                          arr(rhs_indices), _ptr(out), n, M, N, K, Bx, E, bits, group_size, mode,
                          _dt(x), _ptr(ws), 0 if ws is None else ws.numel(),
                          _stream(x.device)), "aq_gather_qmm")
    return out


def aq_qmm(x, w_q, scales, biases, bits=4, group_size=64, out=None, workspace=None):
    """y = x . dequant(w)^T for any M."""
    return _mm("aq_qmm", AQ_OP_QMM, x, w_q, scales, biases, bits, group_size, out, workspace)


def aq_qmm_nt(x, w_q, scales, biases, bits=4, group_size=64, out=None, workspace=None):
    """y [M, K] = x [M, N] . dequant(w) with the weight stored [N, K] as for
    aq_qmv / aq_qmm (the transpose = false product)."""
    M, N = x.shape
    K = w_q.shape[1] * 8 // bits
    mode = _mode(scales)
    if out is None:
        out = torch.empty((M, K), dtype=x.dtype, device=x.device)
    ws_bytes = aq_workspace_size(AQ_OP_QMM_NT, M, N, K, bits, group_size, mode)
    ws = (workspace or _default_ws).get(x.device, ws_bytes)
    check(lib().aq_qmm_nt(_ptr(x), _ptr(w_q), _ptr(scales), _ptr(biases), _ptr(out), M, N, K, bits,
                          group_size, mode, _dt(x), _ptr(ws), 0 if ws is None else ws.numel(),
                          _stream(x.device)), "aq_qmm_nt")
    return out


def conv_out_hw(H, W, kh, kw, stride, pad):
    return (H + 2 * pad[0] - kh) // stride[0] + 1, (W + 2 * pad[1] - kw) // stride[1] + 1


def aq_qconv2d_nhwc(x, w_q, scales, biases, Cout, kh, kw, stride=(1, 1), pad=(0, 0), groups=1,
                    bits=4, group_size=64, out=None, workspace=None):
    """x [B, H, W, Cin] T -> y [B, Ho, Wo, Cout] T (weights as aq_qconv2d_nhwc documents)."""
    B, H, W, Cin = x.shape
    Ho, Wo = conv_out_hw(H, W, kh, kw, stride, pad)
    if out is None:
        out = torch.empty((B, Ho, Wo, Cout), dtype=x.dtype, device=x.device)
    Cg = Cin // groups if groups > 0 else 0
    Kp = -(-kh * kw * Cg // group_size) * group_size if group_size > 0 else 0
    ws_bytes = aq_workspace_size(AQ_OP_QCONV2D, B * Ho * Wo, Cout // max(groups, 1), Kp, bits,
                                 group_size, AQ_MODE_AFFINE, groups)
    ws = (workspace or _default_ws).get(x.device, ws_bytes)
    check(lib().aq_qconv2d_nhwc(_ptr(x), _ptr(w_q), _ptr(scales), _ptr(biases), _ptr(out), B, H,
                                W, Cin, Cout, kh, kw, stride[0], stride[1], pad[0], pad[1],
                                groups, bits, group_size, _dt(x), _ptr(ws),
                                0 if ws is None else ws.numel(), _stream(x.device)),
          "aq_qconv2d_nhwc")
    return out


def _fits(t, dtype, shape, dev):
    """Whether the C call can take the tensor as it is (it sees only the address)."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev


def _refuse(x, *checks):
    """Raise what is wrong with the first (name, tensor, dtype, shape) that does not fit."""
    for name, t, dtype, shape in checks:
        if not t.is_cuda:
            if x.is_cuda:
                raise ValueError("all tensors must be on one device, got %s and %s" % (x.device, t.device))
            raise ValueError("%s must be a CUDA tensor" % name)
        if t.device != x.device:
            raise ValueError("all tensors must be on one device, got %s and %s" % (x.device, t.device))
        if t.dtype is not dtype:
            raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
        if t.shape != shape:
            raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    raise ValueError("tensors on %s" % x.device)


def _matrix_shape(name, t):
    if t.dim() != 2:
        raise ValueError("%s must have 2 dimensions, got %d" % (name, t.dim()))
    return t.shape


class _Scratch(threading.local):
    """Default scratch of the calling host thread, a buffer per device and
    stream.  Threads do not share one, though they share the default stream: a
    call may be several launches, and another thread's may come between them."""

    def __init__(self):
        self.bufs = {}


_scratch = _Scratch()


def _workspace(workspace, x, nbytes, counters):
    """(buffer, address, bytes) of the caller's Workspace, or of a buffer of this
    host thread, device and stream (calls on two streams may overlap); a call
    that is being captured gets one of its own, which lives in the graph's
    memory.  The caller holds the buffer until it has launched: the address alone
    does not keep it from the allocator."""
    if nbytes == 0:
        return None, None, 0
    if workspace is not None:
        buf = workspace.get(x.device, nbytes)
    elif torch.cuda.is_current_stream_capturing():
        buf = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        if counters:
            buf[:_COUNTER_BYTES].zero_()
    else:
        dev = x.get_device()
        key = (dev, _stream_of(dev))
        bufs = _scratch.bufs
        buf = bufs.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = bufs[key] = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=x.device)
    return buf, buf.data_ptr(), buf.numel()


_COUNTER_BYTES = 65536           # at a workspace's start, zero between calls (include/aq.h)


@functools.lru_cache(maxsize=4096)
def _qqmm_int8_bytes(M, N, K):
    return lib().aq_workspace_size(AQ_OP_QQMM_INT8, M, N, K, 8, 16, AQ_MODE_AFFINE, 1)


@functools.lru_cache(maxsize=4096)
def _moe_bytes(T, H, I, E, k):
    return lib().aq_moe_workspace_size(T, H, I, E, k)


# The functions below launch on the current device: they call themselves with it
# changed where x is on another.  (torch.empty is faster with the sizes as
# arguments than with a tuple or as a method.)


def aq_quantize_int8(x, out=None):
    """x [R, K] fp16/bf16 -> (codes int8 [R, K], scales fp32 [R]): a symmetric
    scale per row (a token, or a channel of a weight)."""
    R, K = _matrix_shape("x", x)
    dt, dev = _dt(x), x.get_device()
    if dev < 0 or not x.is_contiguous():
        _refuse(x, ("x", x, x.dtype, x.shape))
    if out is None:
        q, s = torch.empty_like(x, dtype=torch.int8), torch.empty(R, dtype=torch.float32, device=x.device)
    else:
        q, s = out
        if not (_fits(q, torch.int8, (R, K), dev) and _fits(s, torch.float32, (R,), dev)):
            _refuse(x, ("codes", q, torch.int8, (R, K)), ("scales", s, torch.float32, (R,)))
    if dev != _current_device():
        with torch.cuda.device(dev):
            return aq_quantize_int8(x, (q, s))
    st = lib().aq_quantize_int8(x.data_ptr(), q.data_ptr(), s.data_ptr(), R, K, dt, _stream_of(dev))
    if st:
        check(st, "aq_quantize_int8")
    return q, s


def aq_int8_mm(x_q, x_scales, w_q, w_scales, dtype=torch.bfloat16, out=None):
    """y [M, N] = dtype(x_q . w_q^T * x_scales[:, None] * w_scales[None, :]) for
    int8 x_q [M, K], w_q [N, K] and fp32 scales per token and channel."""
    xshape, wshape = x_q.shape, w_q.shape
    if len(xshape) != 2 or len(wshape) != 2:
        _matrix_shape("x_q", x_q), _matrix_shape("w_q", w_q)
    (M, K), N = xshape, wshape[0]
    dev = x_q.get_device()
    if out is not None:
        dtype = out.dtype
    dt = _DT.get(dtype)
    if dt is None:
        raise TypeError("expected fp16 or bf16 as the result's type, got %s" % dtype)
    i8, f32 = torch.int8, torch.float32
    # _fits of the four, written out
    if not (dev >= 0 and wshape[1] == K and x_scales.shape == (M,) and w_scales.shape == (N,)
            and x_q.dtype is i8 and w_q.dtype is i8 and x_scales.dtype is f32 and w_scales.dtype is f32
            and x_q.is_contiguous() and w_q.is_contiguous() and x_scales.is_contiguous()
            and w_scales.is_contiguous() and w_q.get_device() == dev and x_scales.get_device() == dev
            and w_scales.get_device() == dev):
        _refuse(x_q, ("x_q", x_q, i8, (M, K)), ("x_scales", x_scales, f32, (M,)),
                ("w_q", w_q, i8, (N, K)), ("w_scales", w_scales, f32, (N,)))
    if out is None:
        out = torch.empty(M, N, dtype=dtype, device=x_q.device)
    elif not _fits(out, dtype, (M, N), dev):
        _refuse(x_q, ("out", out, dtype, (M, N)))
    if dev != _current_device():
        with torch.cuda.device(dev):
            return aq_int8_mm(x_q, x_scales, w_q, w_scales, dtype, out)
    st = lib().aq_int8_mm(x_q.data_ptr(), x_scales.data_ptr(), w_q.data_ptr(), w_scales.data_ptr(),
                          out.data_ptr(), M, N, K, dt, _stream_of(dev))
    if st:
        check(st, "aq_int8_mm")
    return out


def aq_qqmm_int8(x, w_q, w_scales, out=None, workspace=None):
    """W8A8: y [M, N] = x . w^T with the rows of x [M, K] fp16/bf16 quantized on
    the way and an int8 weight w_q [N, K] with fp32 scales per channel.  A
    `workspace` passed in serves one host thread and stream at a time."""
    xshape, wshape = x.shape, w_q.shape
    if len(xshape) != 2 or len(wshape) != 2:
        _matrix_shape("x", x), _matrix_shape("w_q", w_q)
    (M, K), N = xshape, wshape[0]
    dt, dev = _dt(x), x.get_device()
    # _fits of the three, written out
    if not (dev >= 0 and wshape[1] == K and w_scales.shape == (N,) and w_q.dtype is torch.int8
            and w_scales.dtype is torch.float32 and x.is_contiguous() and w_q.is_contiguous()
            and w_scales.is_contiguous() and w_q.get_device() == dev and w_scales.get_device() == dev):
        _refuse(x, ("x", x, x.dtype, (M, K)), ("w_q", w_q, torch.int8, (N, K)),
                ("w_scales", w_scales, torch.float32, (N,)))
    if out is None:
        out = torch.empty(M, N, dtype=x.dtype, device=x.device)
    elif not _fits(out, x.dtype, (M, N), dev):
        _refuse(x, ("out", out, x.dtype, (M, N)))
    if dev != _current_device():
        with torch.cuda.device(dev):
            return aq_qqmm_int8(x, w_q, w_scales, out, workspace)
    buf, ws, nbytes = _workspace(workspace, x, _qqmm_int8_bytes(M, N, K), False)
    st = lib().aq_qqmm_int8(x.data_ptr(), w_q.data_ptr(), w_scales.data_ptr(), out.data_ptr(), M, N, K, dt,
                            ws, nbytes, _stream_of(dev))
    if st:
        check(st, "aq_qqmm_int8")
    return out


def _moe_stacks(x, H, I, E, gate, up, down, bits, group_size):
    """Check three stacks (w_q, scales, biases) -> (mode, the C structs' nine
    addresses).  E and I come from gate."""
    (gq, gs, gb), (uq, us, ub), (dq, ds, db) = gate, up, down
    unit = group_size if group_size > 0 else 1
    wide, deep = (E, I, H * bits // 8), (E, H, I * bits // 8)        # codes
    wscale, dscale = (E, I, H // unit), (E, H, I // unit)
    dtype, dev, u8 = x.dtype, x.get_device(), torch.uint8
    mode = AQ_MODE_FP4 if gs.dtype is u8 else AQ_MODE_AFFINE
    stype = u8 if mode else dtype
    if (dev >= 0 and _fits(gq, u8, wide, dev) and _fits(uq, u8, wide, dev) and _fits(dq, u8, deep, dev)
            and _fits(gs, stype, wscale, dev) and _fits(us, stype, wscale, dev)
            and _fits(ds, stype, dscale, dev)):
        if gb is None and ub is None and db is None:
            return mode, (gq.data_ptr(), gs.data_ptr(), 0, uq.data_ptr(), us.data_ptr(), 0,
                          dq.data_ptr(), ds.data_ptr(), 0)
        if (gb is not None and ub is not None and db is not None and _fits(gb, dtype, wscale, dev)
                and _fits(ub, dtype, wscale, dev) and _fits(db, dtype, dscale, dev)):
            return mode, (gq.data_ptr(), gs.data_ptr(), gb.data_ptr(), uq.data_ptr(), us.data_ptr(),
                          ub.data_ptr(), dq.data_ptr(), ds.data_ptr(), db.data_ptr())
    checks = [("x", x, dtype, x.shape)]
    for name, (w_q, scales, biases), w, s in (("gate", gate, wide, wscale), ("up", up, wide, wscale),
                                              ("down", down, deep, dscale)):
        if _mode(scales) != mode or (biases is None) != (gb is None):
            raise ValueError("gate, up and down must have one format")
        checks += [(name + " w_q", w_q, u8, w), (name + " scales", scales, stype, s)]
        if biases is not None:
            checks.append((name + " biases", biases, dtype, s))
    _refuse(x, *checks)


def _moe_sizes(x, gate):
    T, H = _matrix_shape("x", x)
    if gate[0].dim() != 3:
        raise ValueError("gate w_q must have 3 dimensions, got %d" % gate[0].dim())
    E, I = gate[0].shape[:2]
    if not x.is_contiguous():
        _refuse(x, ("x", x, x.dtype, (T, H)))
    return T, H, I, E


def _moe_out(x, out, T, H):
    if out is None:
        return torch.empty_like(x)
    if not _fits(out, x.dtype, (T, H), x.get_device()):
        _refuse(x, ("out", out, x.dtype, (T, H)))
    return out


_Nine = ctypes.c_uint64 * 9
_MAX_TOP_K = 16


def aq_moe(x, w_router, gate, up, down, top_k, normalize=True, bits=4, group_size=64, out=None,
           workspace=None):
    """A mixture-of-experts layer for T <= 64 tokens: x [T, H], w_router [E, H],
    gate / up (w_q [E, I, H*bits/8], scales and biases [E, I, H/group_size],
    biases None for FP4), down likewise [E, H, I...].  Returns (y [T, H],
    indices int32 [T, top_k], weights fp32 [T, top_k])."""
    T, H, I, E = _moe_sizes(x, gate)
    dt, dev = _dt(x), x.get_device()
    mode, at = _moe_stacks(x, H, I, E, gate, up, down, bits, group_size)
    if not _fits(w_router, x.dtype, (E, H), dev):
        _refuse(x, ("w_router", w_router, x.dtype, (E, H)))
    out = _moe_out(x, out, T, H)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return aq_moe(x, w_router, gate, up, down, top_k, normalize, bits, group_size, out, workspace)
    top_k = max(min(int(top_k), 1 << 62), -1)   # what a 64-bit argument holds
    k = min(max(top_k, 0), _MAX_TOP_K)          # more are refused below, not allocated first
    indices = torch.empty(T, k, dtype=torch.int32, device=x.device)
    weights = torch.empty(T, k, dtype=torch.float32, device=x.device)
    buf, ws, nbytes = _workspace(workspace, x, _moe_bytes(T, H, I, E, k), True)
    m = _Nine(*at)
    a = ctypes.addressof(m)
    st = _by_address("aq_moe")(x.data_ptr(), w_router.data_ptr(), a, a + 24, a + 48, out.data_ptr(),
                               indices.data_ptr(), weights.data_ptr(), T, H, I, E, top_k,
                               1 if normalize else 0, bits, group_size, mode, dt, ws, nbytes, _stream_of(dev))
    if st:
        check(st, "aq_moe")
    return out, indices, weights


def aq_moe_experts(x, indices, weights, gate, up, down, bits=4, group_size=64, out=None,
                   workspace=None):
    """The experts of aq_moe for given routing: indices int32 [T, k] and weights
    fp32 [T, k] on the device (an index outside 0..E-1 skips its slot)."""
    T, H, I, E = _moe_sizes(x, gate)
    dt, dev = _dt(x), x.get_device()
    mode, at = _moe_stacks(x, H, I, E, gate, up, down, bits, group_size)
    k = _matrix_shape("indices", indices)[1]
    if not (_fits(indices, torch.int32, (T, k), dev) and _fits(weights, torch.float32, (T, k), dev)):
        _refuse(x, ("indices", indices, torch.int32, (T, k)), ("weights", weights, torch.float32, (T, k)))
    out = _moe_out(x, out, T, H)
    if dev != _current_device():
        with torch.cuda.device(dev):
            return aq_moe_experts(x, indices, weights, gate, up, down, bits, group_size, out, workspace)
    buf, ws, nbytes = _workspace(workspace, x, _moe_bytes(T, H, I, E, k), True)
    m = _Nine(*at)
    a = ctypes.addressof(m)
    st = _by_address("aq_moe_experts")(x.data_ptr(), indices.data_ptr(), weights.data_ptr(), a, a + 24, a + 48,
                                       out.data_ptr(), T, H, I, E, k, bits, group_size, mode, dt, ws, nbytes,
                                       _stream_of(dev))
    if st:
        check(st, "aq_moe_experts")
    return out


@functools.lru_cache(maxsize=None)
def _by_address(name):
    """The function with its structs given by address."""
    f = lib()[name]
    res, args = _lib.SIGNATURES[name]
    f.restype = res
    f.argtypes = [ctypes.c_void_p if a is _lib.MoeMatrixPtr else a for a in args]
    return f
