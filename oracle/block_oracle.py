"""CPU oracle of the operators around the MoE layer: MXFP4 values and the norms
in front of and behind the block with their gradients.

TEST INFRASTRUCTURE ONLY, like moe_oracle: float64 NumPy, written from the
formulas, sharing no code with the HIP library.
"""
from __future__ import annotations

import numpy as np

from .moe_oracle import _f64

# ------------------------------------------------------------------ MXFP4
MX_LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mxfp4_quantize(x) -> tuple:
    """x [rows, n] (bf16 bits or float32) -> codes [rows, n / 2], scales [rows, n / 32].
    Every step is exact in float64 (powers of two and comparisons)."""
    v = _f64(x)
    rows, n = v.shape
    v = v.reshape(rows, n // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    with np.errstate(invalid="ignore"):
        top = np.where(bad, 0.0, np.abs(v).max(-1))
    exp = np.frexp(top)[1] - 1  # floor(log2 top), top > 0
    e = np.where(top > 0, np.clip(exp - 2, -127, 127), -127)
    with np.errstate(invalid="ignore"):
        a = np.abs(v) / np.exp2(e.astype(np.float64))[..., None]
    # nearest level, ties to the even code, saturating: a tie between codes c and
    # c + 1 goes up only where c + 1 is even
    code = np.zeros(v.shape, dtype=np.uint8)
    for c in range(7):
        mid = (MX_LEVELS[c] + MX_LEVELS[c + 1]) / 2
        with np.errstate(invalid="ignore"):
            code += (a > mid) | ((a == mid) & ((c + 1) % 2 == 0))
    code |= np.signbit(v).astype(np.uint8) << 3
    code[bad] = 0
    code = code.reshape(rows, n)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), scales


def mxfp4_decode(codes, scales) -> np.ndarray:
    """codes [..., n / 2], scales [..., n / 32] -> float64 [..., n]."""
    codes = np.asarray(codes)
    both = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)
    v = MX_LEVELS[both & 7] * np.where(both & 8, -1.0, 1.0)
    s = np.exp2(np.asarray(scales).astype(np.float64) - 127)
    s = np.where(np.asarray(scales) == 255, np.nan, s)
    return v * np.repeat(s, 32, -1)


# ------------------------------------------------------------------ norms
def rms_norm(x, w=None, eps=1e-6):
    """(xn, rstd): xn = x r w, r = 1 / sqrt(mean x^2 + eps)."""
    x = _f64(x)
    r = 1.0 / np.sqrt((x * x).mean(-1) + eps)
    xn = x * r[:, None]
    return (xn if w is None else xn * _f64(w)), r


def rms_norm_backward(d_xn, x, w=None, eps=1e-6, d_residual=None):
    """(d_x, d_w) of rms_norm."""
    g, x = _f64(d_xn), _f64(x)
    r = 1.0 / np.sqrt((x * x).mean(-1) + eps)[:, None]
    n = x * r
    gw = g if w is None else g * _f64(w)
    d_x = r * (gw - n * (gw * n).mean(-1, keepdims=True))
    if d_residual is not None:
        d_x = d_x + _f64(d_residual)
    return d_x, (g * n).sum(0)


def _rows_of(y, slot_of, topk_w, T):
    """The k rows and weights of every token: ([T, k, d], [T, k])."""
    y = _f64(y)
    if slot_of is None:
        return y[:, None, :], np.ones((T, 1))
    g = _f64(topk_w)
    return y[np.asarray(slot_of)].reshape(T, g.shape[1], -1), g


def combine_norm(y, slot_of, topk_w, residual, w=None, gate=None, eps=1e-6, scale=1.0, T=None):
    """(out, rstd): out = scale residual + gate (y r w), y the weighted sum of a
    token's expert rows (or y itself in token order)."""
    T = len(_f64(y)) if slot_of is None else _f64(topk_w).shape[0]
    rows, g = _rows_of(y, slot_of, topk_w, T)
    s = (rows * g[..., None]).sum(1)
    n, r = rms_norm(s, w, eps)
    if gate is not None:
        gate = _f64(gate)
        n = n * np.repeat(gate, T // gate.shape[0], 0)
    return (n if residual is None else n + scale * _f64(residual)), r


def combine_norm_backward(d_out, y, slot_of, topk_w, w=None, gate=None, eps=1e-6, scale=1.0):
    """Gradients of combine_norm: dict d_y, d_topk_w, d_residual, d_weight, d_gate."""
    g_out = _f64(d_out)
    T, d = g_out.shape
    rows, g = _rows_of(y, slot_of, topk_w, T)
    s = (rows * g[..., None]).sum(1)
    r = 1.0 / np.sqrt((s * s).mean(-1) + eps)[:, None]
    n = s * r
    wf = np.ones(d) if w is None else _f64(w)
    n_gate = 1 if gate is None else _f64(gate).shape[0]
    gf = np.ones((T, d)) if gate is None else np.repeat(_f64(gate), T // n_gate, 0)
    dn = gf * wf * g_out
    dy = r * (dn - n * (dn * n).mean(-1, keepdims=True))
    d_rows = g[..., None] * dy[:, None]
    if slot_of is None:
        d_y = dy
    else:
        d_y = np.zeros((rows.shape[0] * rows.shape[1], d))
        d_y[np.asarray(slot_of)] = d_rows.reshape(-1, d)
    return dict(d_y=d_y, d_topk_w=(rows * dy[:, None]).sum(-1), d_residual=scale * g_out,
                d_weight=(gf * g_out * n).sum(0),
                d_gate=(wf * g_out * n).reshape(n_gate, T // n_gate, d).sum(1))
