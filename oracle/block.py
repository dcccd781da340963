"""What stands around a quantised projection in a block (oracle), in fp64.

The pages describe the projection; these are the elementary definitions of the
operators next to it, written from their formulas:

  residual_norm: u = N_post(y) act(gate); r_out = residual_scale r + branch_scale u;
                 h = N_pre(r_out), with N an RMS or a layer norm.
  lora_add: y[t] = y_in[t] + scale[g] B_g (A_g x[t]) with g = adapter[t], over the first
                 ranks[g] rows of A_g and columns of B_g; y_in[t] where there is no adapter.
"""
from __future__ import annotations

import numpy as np

from ._checks import require_finite


def norm(v, kind, weight=None, bias=None, eps=1e-6, weight_offset=0.0):
    require_finite("norm", v, weight, bias)
    v = np.asarray(v, dtype=np.float64)
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    elif kind != "rms":
        raise ValueError(kind)
    v = v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    if weight is not None:
        v = v * (np.asarray(weight, dtype=np.float64) + weight_offset)
    if bias is not None:
        v = v + np.asarray(bias, dtype=np.float64)
    return v


def activate(gate, act):
    require_finite("activate", gate)
    g = np.asarray(gate, dtype=np.float64)
    if act == "linear":
        return g
    s = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
    return {"sigmoid": s, "silu": g * s}[act]


def residual_norm(y, r=None, post="none", post_weight=None, post_bias=None, gate=None, gate_act="linear",
                  residual_scale=1.0, branch_scale=1.0, pre="none", pre_weight=None, pre_bias=None, eps=1e-6,
                  weight_offset=0.0):
    """(u, r_out, h) as fp64 [rows, d]."""
    require_finite("residual_norm", y, r, gate)
    u = norm(y, post, post_weight, post_bias, eps, weight_offset)
    if gate is not None:
        u = u * activate(gate, gate_act)
    out = branch_scale * u
    if r is not None:
        out = out + residual_scale * np.asarray(r, dtype=np.float64)
    return u, out, norm(out, pre, pre_weight, pre_bias, eps, weight_offset)


def lora_add(x, adapter, a, b, y_in=None, ranks=None, scale=None):
    """(y, size) fp64 [tokens, d_out]; ``size`` bounds the magnitudes behind y's adapter
    part: the largest over j of sum_i |x_i a_ji|, times sum_j |b_oj|, times |scale|."""
    x, adapter = np.asarray(x, dtype=np.float64), np.asarray(adapter)
    require_finite("lora_add", x, y_in, scale)
    n, d_out, rank = b.shape
    y = np.zeros((x.shape[0], d_out)) if y_in is None else np.array(y_in, dtype=np.float64)
    size = np.zeros_like(y)
    for g in set(adapter.tolist()):
        if not 0 <= g < n:
            continue
        k = rank if ranks is None else min(max(int(ranks[g]), 0), rank)
        rows = np.flatnonzero(adapter == g)
        ag, bg = np.asarray(a[g, :k], dtype=np.float64), np.asarray(b[g, :, :k], dtype=np.float64)
        require_finite("lora_add", ag, bg)
        sc = 1.0 if scale is None else float(scale[g])
        y[rows] += sc * ((x[rows] @ ag.T) @ bg.T)
        if k:
            size[rows] = abs(sc) * np.outer((np.abs(x[rows]) @ np.abs(ag).T).max(1), np.abs(bg).sum(1))
    return y, size
