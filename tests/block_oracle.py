"""Plain 64-bit forms of the operators around the 4-bit linear layer (8-bit
linear, layer norm, rotary positions) for the tests, and error bounds counted
in roundings. Everything here runs on the CPU in numpy."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24                      # half a step of fp32, relative
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
SUBNORMAL = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def np64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def rounding(y, dtype):
    """Error of rounding a value within a few fp32 steps of y to dtype."""
    return HALF_STEP[dtype] * np.abs(y) * (1 + 2.0 ** -10) + SUBNORMAL[dtype]


def within(got, want, bound, what=""):
    d = np.abs(np64(got) - want)
    bad = ~(d <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, d - bound, -np.inf)), d.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} values off, worst at {i}: "
                             f"{np64(got)[i]!r} for {want[i]!r}, bound {np.broadcast_to(bound, d.shape)[i]:.3g}")


def int8_codes(x, mult=None):
    """(codes, scales) of fp32 values x [M][K]: v = fp32(x mult), s = fp32(max|v| fp32(1/127))."""
    v = x.astype(np.float32)
    if mult is not None:
        v = v * mult.astype(np.float32)
    s = (np.abs(v).max(axis=1) * (np.float32(1) / np.float32(127))).astype(np.float32)
    safe = np.where(s > 0, s, 1).astype(np.float64)
    q = np.clip(np.rint(v.astype(np.float64) / safe[:, None]), -127, 127)
    return np.where(s[:, None] > 0, q, 0).astype(np.int64), s


def int8_linear(qx, sx, qw, sw, bias):
    """(Y, bound on the error before Y's own rounding): the sum to fp32, two products, one addition."""
    p = (qx.astype(np.float64) @ qw.astype(np.float64).T) * sx.astype(np.float64)[:, None] * sw.astype(np.float64)
    b = np.zeros(qw.shape[0]) if bias is None else bias.astype(np.float64)
    return p + b, 4 * U * (np.abs(p) + np.abs(b))


def group_rows(w, M, C, rows, default):
    if w is None:
        return np.full((M, C), default)
    w = w.reshape(-1, C)
    return w[np.arange(M) // (rows or max(M, 1))]


# fp32 additions that any one term of a row's sum passes: at most 32 in a thread, 5 in a warp, 5 across warps
DEPTH = 44


def layernorm(x, w, b, eps, rows, add_one):
    """(y, mean, rstd, bounds of the three before y's rounding) of fp64 x [M][C], w and b [groups][C] or None."""
    M, C = x.shape
    g = group_rows(w, M, C, rows, 0.0 if add_one else 1.0) + (1.0 if add_one else 0.0)
    o = group_rows(b, M, C, rows, 0.0)
    mean = x.mean(1)
    d = x - mean[:, None]
    var = (d * d).mean(1)
    rstd = 1 / np.sqrt(var + eps)
    xh = d * rstd[:, None]
    y = xh * g + o
    dmean = (DEPTH + 2) * U * np.abs(x).mean(1)
    # each (x - mean)^2 is off by its difference's rounding and by the mean's error; the sum by its depth
    dvar = (DEPTH + 4) * U * var + 2 * np.sqrt(var) * U * np.abs(x).max(1) + dmean ** 2 + 2 * dmean * DEPTH * U * np.sqrt(var)
    rel = 0.5 * dvar / (var + eps) * 1.01 + 4 * U
    dxh = rstd[:, None] * (dmean[:, None] + U * (np.abs(x) + np.abs(mean)[:, None])) + np.abs(xh) * (rel[:, None] + 2 * U)
    dy = dxh * np.abs(g) + 3 * U * (np.abs(xh * g) + np.abs(o))
    return y, mean, rstd, dy, dmean, rel * rstd


def layernorm_backward(dy, x, w, mean, rstd, rows, add_one):
    """(dx, dw, db, bounds) with the forward pass's own statistics."""
    M, C = x.shape
    n = rows or max(M, 1)
    G = max(1, -(-M // n))
    g = group_rows(w, M, C, rows, 0.0 if add_one else 1.0) + (1.0 if add_one else 0.0)
    r, mu = rstd[:, None], mean[:, None]
    xh = (x - mu) * r
    h = dy * g
    m1, m2 = h.mean(1, keepdims=True), (h * xh).mean(1, keepdims=True)
    dx = r * (h - m1 - xh * m2)
    dxh = U * (np.abs(x) + np.abs(mu)) * r + 2 * U * np.abs(xh)
    dh = 2 * U * np.abs(h)
    dm1 = (DEPTH + 4) * U * np.abs(h).mean(1, keepdims=True)
    dm2 = (DEPTH + 6) * U * np.abs(h * xh).mean(1, keepdims=True) + (np.abs(h) * dxh).mean(1, keepdims=True)
    bdx = r * (dh + dm1 + np.abs(xh) * dm2 + np.abs(m2) * dxh + 4 * U * (np.abs(h) + np.abs(m1) + np.abs(xh * m2)))
    dw, db, bdw, bdb = (np.zeros((G, C)) for _ in range(4))
    for k in range(G if M else 0):
        s = slice(k * n, min(M, (k + 1) * n))
        depth = min(n, M) + 24                 # at worst every row is added in turn
        dw[k], db[k] = (dy[s] * xh[s]).sum(0), dy[s].sum(0)
        bdw[k] = depth * U * np.abs(dy[s] * xh[s]).sum(0) + (np.abs(dy[s]) * dxh[s]).sum(0)
        bdb[k] = depth * U * np.abs(dy[s]).sum(0)
    return dx, dw, db, bdx, bdw, bdb


def rope(x, pos, axis_dims, freqs, interleaved, inverse):
    """(y, bound before y's rounding) for x [T][H][D], pos [P][axes]. The angle's fp32 form in half turns is off by
    2^-25, that is pi 2^-25 < 2 U radians; sincospif by two of its steps (2 U); a turn has three roundings."""
    T = x.shape[0]
    pos = pos[np.arange(T) % pos.shape[0]]
    axis = np.repeat(np.arange(len(axis_dims)), [d // 2 for d in axis_dims])
    angle = pos[:, axis] * freqs * (-1.0 if inverse else 1.0)
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    R = sum(axis_dims)
    y = x.copy()
    bound = np.zeros_like(x)
    i, j = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    bound[..., i] = bound[..., j] = 8 * U * (np.abs(a) + np.abs(b))
    return y, bound
