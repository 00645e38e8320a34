"""Float64 CPU oracle of the dense 8-bit operators (row norm with quantised output, 8-bit
product, gated product, dense decoder layer).

TEST INFRASTRUCTURE, as oracle/moe_oracle.py: numpy arrays in, numpy arrays out, no code
shared with the library.  A dense layer stands beside the MoE blocks in the stack that
TensorFold issue #1247 describes (config paragraph: 24 layers, a dense layer 0); its 8-bit
form is the usual one of int8 codes with a scale per token and per output channel.

Nothing is rounded except what the operators store: the residual sum, rows and outputs in the
activation type, and the codes.
"""
from __future__ import annotations

import numpy as np

from oracle import moe_oracle as mo


def summed_rows(x, residual=None, act="bf16") -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    return x if residual is None else mo.round_act(x + np.asarray(residual, dtype=np.float64), act)


def norm_rows(x, gamma=None, residual=None, eps=mo.RMS_EPS, act="bf16") -> np.ndarray:
    """The values that are stored as rows or codes, before that rounding."""
    s = summed_rows(x, residual, act)
    return s if gamma is None else mo.rms_norm(s, gamma, eps)


def quant_i8(v):
    """(codes, scales): scale = amax / 127 per row (1 for a zero row, not finite where the row is
    not), code = rint(v / scale)."""
    v = np.asarray(v, dtype=np.float64)
    amax = np.abs(v).max(axis=1)
    scale = np.where(amax == 0, 1.0, amax / 127.0)
    return np.clip(np.rint(v / scale[:, None]), -127, 127), scale


def product(x_codes, x_scales, w_codes, w_scales) -> np.ndarray:
    """float64 holds every sum of the codes' products exactly (|sum| <= 2^30)."""
    acc = np.asarray(x_codes, dtype=np.float64) @ np.asarray(w_codes, dtype=np.float64).T
    return acc * np.asarray(x_scales, dtype=np.float64)[:, None] * np.asarray(w_scales, dtype=np.float64)


def glu(x_codes, x_scales, w_gate, s_gate, w_up, s_up) -> np.ndarray:
    g = product(x_codes, x_scales, w_gate, s_gate)
    return g * mo.sigmoid(g) * product(x_codes, x_scales, w_up, s_up)


def dense_layer(x, gamma, w, act="bf16", eps=mo.RMS_EPS) -> np.ndarray:
    """x + down(i8(glu(i8(norm(x))))), before the store's rounding.  `w`: codes w_gate,
    w_up, w_down and scales s_gate, s_up, s_down."""
    xq, sx = quant_i8(norm_rows(x, gamma, None, eps, act))
    h = glu(xq, sx, w["w_gate"], w["s_gate"], w["w_up"], w["s_up"])
    return np.asarray(x, dtype=np.float64) + product(*quant_i8(h), w["w_down"], w["s_down"])
