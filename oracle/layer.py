"""The linear-attention layer with a decay per head and the norms around it in
64 bits, straight from their definitions (numpy, CPU): what the tests compare
the kernels with. Token arrays are [tokens, heads, d] for one sequence."""
import numpy as np


def linattn(q, k, v, log_decay, scale, s0=None):
    """(o [T, H, dv], final state [H, dk, dv]) by the recurrence."""
    T, H, dk = q.shape
    G, dv = k.shape[1], v.shape[2]
    lam = np.exp(np.asarray(log_decay, dtype=np.float64))
    S = np.zeros((H, dk, dv)) if s0 is None else np.array(s0, dtype=np.float64)
    o = np.zeros((T, H, dv))
    g = np.arange(H) // (H // G)
    for t in range(T):
        S = lam[:, None, None] * S + k[t, g][:, :, None] * v[t, g][:, None, :]
        o[t] = scale * np.einsum("hd,hde->he", q[t], S)
    return o, S


def linattn_bwd(q, k, v, log_decay, scale, do, s0=None, dfinal=None):
    """(dq, dk, dv, dinitial) of linattn by the adjoint recurrence."""
    T, H, dk = q.shape
    G, dv = k.shape[1], v.shape[2]
    lam = np.exp(np.asarray(log_decay, dtype=np.float64))
    S = np.zeros((H, dk, dv)) if s0 is None else np.array(s0, dtype=np.float64)
    g = np.arange(H) // (H // G)
    dq, dkh, dvh = np.zeros((T, H, dk)), np.zeros((T, H, dk)), np.zeros((T, H, dv))
    for t in range(T):
        S = lam[:, None, None] * S + k[t, g][:, :, None] * v[t, g][:, None, :]
        dq[t] = scale * np.einsum("hde,he->hd", S, do[t])
    R = np.zeros((H, dk, dv)) if dfinal is None else np.array(dfinal, dtype=np.float64)
    for t in range(T - 1, -1, -1):
        R = R + scale * q[t][:, :, None] * do[t][:, None, :]
        dkh[t] = np.einsum("hde,he->hd", R, v[t, g])
        dvh[t] = np.einsum("hde,hd->he", R, k[t, g])
        R = lam[:, None, None] * R
    shared = lambda x: x.reshape(T, G, H // G, x.shape[2]).sum(2)  # noqa: E731
    return dq, shared(dkh), shared(dvh), R


def _silu(z):
    s = np.exp(-np.logaddexp(0.0, -z))  # sigmoid, at any z
    return z * s, s * (1.0 + z * (1.0 - s))


def _norm(a, groups, eps):
    g = a.reshape(a.shape[0], groups, -1)
    inv = 1.0 / np.sqrt(np.mean(g * g, axis=2, keepdims=True) + eps)
    return (g * inv).reshape(a.shape), np.broadcast_to(inv, g.shape).reshape(a.shape)


def _norm_bwd(hat, inv, dh, groups):
    m = np.mean((dh * hat).reshape(hat.shape[0], groups, -1), axis=2, keepdims=True)
    m = np.broadcast_to(m, (hat.shape[0], groups, hat.shape[1] // groups)).reshape(hat.shape)
    return inv * (dh - hat * m)


def gated_norm(x, z, w, groups, eps, gate_first):
    gate = 1.0 if z is None else _silu(z)[0]
    hat, _ = _norm(x * gate if gate_first else x, groups, eps)
    y = hat * (1.0 if w is None else w)
    return y if gate_first else y * gate


def gated_norm_bwd(x, z, w, dy, groups, eps, gate_first):
    """(dx, dz or None, dw)"""
    gate, slope = (1.0, 0.0) if z is None else _silu(z)
    ww = 1.0 if w is None else w
    hat, inv = _norm(x * gate if gate_first else x, groups, eps)
    up = dy if gate_first else dy * gate
    da = _norm_bwd(hat, inv, up * ww, groups)
    dw = np.sum(up * hat, axis=0)
    if gate_first:
        return da * gate, (None if z is None else da * x * slope), dw
    return da, (None if z is None else dy * hat * ww * slope), dw


def residual_norm(x, res, w, cs, scale, eps):
    """(y, the sum)"""
    r = scale * x * (1.0 if cs is None else cs) + (0.0 if res is None else res)
    return _norm(r, 1, eps)[0] * (1.0 if w is None else w), r


def residual_norm_bwd(r, w, dy, dr, x, cs, scale, eps):
    """(dx, dresidual, dw, dc or None)"""
    hat, inv = _norm(r, 1, eps)
    d = (0.0 if dr is None else dr) + _norm_bwd(hat, inv, dy * (1.0 if w is None else w), 1)
    dc = None if x is None or cs is None else np.sum(scale * x * d, axis=0)
    return scale * d * (1.0 if cs is None else cs), d, np.sum(dy * hat, axis=0), dc
