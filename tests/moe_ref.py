"""A mixture-of-experts layer in 64 bits (numpy), with a bound on the error of
a kernel that keeps fp32 sums: the reference of tests/test_gpu_moe.py.

Bound.  A gate / up / down product adds terms s (c + q) x per group, c the
offset an operand may carry beside its code (at most 128), and at most 32
fp32 roundings reach each term (16 products and their additions in an MMA, up
to 8 MMAs per group, the group sums, the K-slices): its error is at most
32 * 2^-23 times sum |s| (c + 2^bits) |x|, for FP4 (no offset) sum |w x|.  h has
16 bits of significand (2^-17) and a few roundings of 2^-23 from exp and the
division (2^-20 in all), plus what its factors bring: |silu'| <= 1.1.  The
weighted sum adds at most 2^-20 of its terms, and y half a step of T."""
import numpy as np

from tests.util import np_unpack, u16_to_f64, ulp_t

LUT = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def fp4_scale(byte, gs, dt):
    """Scale bytes -> the value in T (E8M0 for 32, E4M3 for 16)."""
    import torch
    if gs == 16:
        v = torch.from_numpy(byte.copy()).view(torch.float8_e4m3fn).float()
    else:
        v = torch.from_numpy(np.where(byte == 0, 2.0 ** -127, 2.0 ** (byte.astype(np.float64) - 127)))
    return v.to(torch.float16 if dt == 0 else torch.bfloat16).double().numpy()


def matrix(w_q, scales, biases, K, bits, gs, dt):
    """One expert matrix: (w [N, K], the magnitudes its rounding errors go by)."""
    N = w_q.shape[0]
    q = np_unpack(w_q, N, K, bits).astype(np.float64)
    if biases is None:
        w = LUT[q.astype(int)] * np.repeat(fp4_scale(scales, gs, dt), gs, axis=1)
        return w, np.abs(w)
    s = np.repeat(u16_to_f64(scales, dt), gs, axis=1)
    b = np.repeat(u16_to_f64(biases, dt), gs, axis=1)
    return s * q + b, np.abs(s) * (128 + 2.0 ** bits) + np.abs(b)


def route(x, w_router, k, normalize):
    """(indices, weights) of the k largest logits, ties to the lower index."""
    l = x @ w_router.T
    at = np.argsort(-l, axis=1, kind="stable")[:, :k]
    p = np.exp(l - l.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    w = np.take_along_axis(p, at, 1)
    return at, w / w.sum(1, keepdims=True) if normalize else w


def experts(x, indices, weights, gate, up, down, bits, gs, dt):
    """x [T, H] float64, stacks of (w_q, scales, biases) numpy arrays ->
    (y [T, H], bound [T, H] without the rounding of y)."""
    T, H = x.shape
    I = gate[0].shape[1]
    E = gate[0].shape[0]
    y, tol = np.zeros((T, H)), np.zeros((T, H))

    def at(m, e, K):
        return matrix(m[0][e], m[1][e], None if m[2] is None else m[2][e], K, bits, gs, dt)
    eps = 32 * 2.0 ** -23
    for e in sorted(set(int(v) for v in indices.ravel() if 0 <= v < E)):
        wg, ag = at(gate, e, H)
        wu, au = at(up, e, H)
        wd, ad = at(down, e, I)
        for t, j in np.argwhere(indices == e):
            g, u = wg @ x[t], wu @ x[t]
            eg, eu = eps * (ag @ np.abs(x[t])), eps * (au @ np.abs(x[t]))
            sig = 1 / (1 + np.exp(-g))
            h = g * sig * u
            eh = 1.1 * eg * np.abs(u) + np.abs(g * sig) * eu + 1.1 * eg * eu + 2.0 ** -16 * np.abs(h)
            o = wd @ h
            eo = np.abs(wd) @ eh + eps * (ad @ (np.abs(h) + eh))
            wt = float(weights[t, j])
            y[t] += wt * o
            tol[t] += abs(wt) * (eo + 2.0 ** -20 * np.abs(o))
    return y, tol


def check(y_u16, ref, tol, dt, what="y"):
    y = u16_to_f64(y_u16, dt)
    full = tol + 0.5 * ulp_t(np.abs(ref) + tol, dt)
    bad = ~(np.abs(y - ref) <= full)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d outside; first at %s: y=%r ref=%r bound=%r"
                             % (what, bad.sum(), y.size, i, y[i], ref[i], full[i]))
