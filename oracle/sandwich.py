"""Sandwich norm: a plain fp64 CPU statement of what the library's
monarch_sandwich_* entry points compute. TEST INFRASTRUCTURE ONLY (same rules
as monarch_oracle; it shares no code with the HIP path).

What is computed, for rows h, y [rows, features]:

    u     = norm_post(y) * post_w + post_b
    h_out = skip * h + branch * gate * u
    n     = norm_pre(h_out) * pre_w + pre_b

norm(v) = (v - mu) / sqrt(mean((v - mu)^2) + eps) with mu the row's mean ("layer")
or 0 ("rms"), and v itself for "none". gate [gates, features]: row i takes gate row
i // (rows / gates).

The backward pass is written from the Jacobian of the norm, row by row as a
matrix: with c = v - mu and rho the reciprocal root,
    d norm_i / d v_j = rho (delta_ij - [layer] 1/d) - rho^3 c_i c_j / d
(the rows of the centring sum to zero, so c_j needs none of its own). It is
pinned against finite differences in tests/test_sandwich_oracle.py.
"""
from __future__ import annotations

import numpy as np


def norm(v, kind, eps):
    """(norm(v), centred rows, rho) of [rows, d]."""
    v = np.asarray(v, dtype=np.float64)
    if kind == "none":
        return v, v, np.ones((v.shape[0], 1))
    c = v - v.mean(axis=1, keepdims=True) if kind == "layer" else v
    rho = 1.0 / np.sqrt((c * c).mean(axis=1, keepdims=True) + eps)
    return c * rho, c, rho


def norm_grad(dq, v, kind, eps):
    """Gradient by v of sum(dq * norm(v)), through each row's Jacobian."""
    dq = np.asarray(dq, dtype=np.float64)
    if kind == "none":
        return dq
    _, c, rho = norm(v, kind, eps)
    d = c.shape[1]
    out = rho * dq - rho ** 3 * c * (c * dq).sum(axis=1, keepdims=True) / d
    if kind == "layer":
        out = out - rho * dq.sum(axis=1, keepdims=True) / d
    return out


def _gate_rows(gate, rows):
    if gate is None:
        return 1.0
    gate = np.asarray(gate, dtype=np.float64)
    return np.repeat(gate, rows // gate.shape[0], axis=0)


def _or(v, default):
    return default if v is None else np.asarray(v, dtype=np.float64)


def forward(h, y, post_w=None, post_b=None, gate=None, pre_w=None, pre_b=None, post="rms",
            pre="rms", skip=1.0, branch=1.0, eps=1e-5):
    """(h_out, n); n is None for pre == "none", h_out is h without y."""
    h = np.asarray(h, dtype=np.float64)
    if y is None:
        h_out = h
    else:
        u = norm(y, post, eps)[0] * _or(post_w, 1.0) + _or(post_b, 0.0)
        h_out = skip * h + branch * _gate_rows(gate, h.shape[0]) * u
    if pre == "none":
        return h_out, None
    return h_out, norm(h_out, pre, eps)[0] * _or(pre_w, 1.0) + _or(pre_b, 0.0)


def backward(dh_out, dn, h, y, post_w=None, post_b=None, gate=None, pre_w=None, pre_b=None,
             post="rms", pre="rms", skip=1.0, branch=1.0, eps=1e-5):
    """dict of the gradients of sum(dh_out * h_out) + sum(dn * n)."""
    h_out, _ = forward(h, y, post_w, post_b, gate, pre_w, pre_b, post, pre, skip, branch, eps)
    rows, d = h_out.shape
    D = np.zeros((rows, d)) if dh_out is None else np.asarray(dh_out, dtype=np.float64)
    g = {}
    if pre != "none":
        dn = np.asarray(dn, dtype=np.float64)
        g["dpre_w"] = (dn * norm(h_out, pre, eps)[0]).sum(axis=0)
        g["dpre_b"] = dn.sum(axis=0)
        D = D + norm_grad(dn * _or(pre_w, 1.0), h_out, pre, eps)
    if y is None:
        g["dh"] = D
        return g
    g["dh"] = skip * D
    yhat = norm(y, post, eps)[0]
    u = yhat * _or(post_w, 1.0) + _or(post_b, 0.0)
    e = branch * _gate_rows(gate, rows) * D
    if gate is not None:
        per = branch * D * u
        g["dgate"] = per.reshape(np.asarray(gate).shape[0], -1, d).sum(axis=1)
    g["dpost_w"] = (e * yhat).sum(axis=0)
    g["dpost_b"] = e.sum(axis=0)
    g["dy"] = norm_grad(e * _or(post_w, 1.0), y, post, eps)
    return g
