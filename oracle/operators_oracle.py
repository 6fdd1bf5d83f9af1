"""fp64 NumPy statement of the operators next to the fused projections: the
projection back into the residual stream, the mixture-of-experts layer, and
token log probabilities with their gradient.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Definitions:

    project:    act(x @ W + b) + residual; gelu(z) = z Phi(z), gelu_tanh its
                tanh form, silu(z) = z / (1 + e^-z)
    moe_route:  l = RMSNorm(x; g) @ R^T; s = softmax(l) or sigmoid(l); the top k
                by l (or by s + bias where a bias is given), ties to the lower
                index, NaN below every number; weights s (/ their sum) * scale
    moe_swiglu: residual + sum_j w_j (silu(h G_e) * (h U_e)) D_e
    token_logprobs: z = scale * logits; lse, z_t - lse, -sum p log p, top k
    token_logprobs_grad: scale * (gl (1[v = t] - p) - gh p (log p + H))
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import numpy as np

from .flashnorm_oracle import rms_inv, silu, to_f64

__all__ = ["project", "moe_route", "moe_swiglu", "token_logprobs", "token_logprobs_grad"]

_erf = np.vectorize(math.erf, otypes=[np.float64])


def project(x, W, bias=None, act: str = "none", residual=None) -> np.ndarray:
    z = to_f64(x) @ to_f64(W)
    if bias is not None:
        z = z + to_f64(bias)[None, :]
    if act == "relu":
        z = np.where(z < 0, 0.0, z)
    elif act == "gelu":
        z = 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0))) if z.size else z
    elif act == "gelu_tanh":
        z = 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    elif act == "silu":
        z = silu(z)
    elif act != "none":
        raise ValueError(act)
    return z if residual is None else z + to_f64(residual)


def moe_route(x, g, router, k: int, eps: float, score: str = "softmax", select_bias=None, renorm: bool = True,
              route_scale: float = 1.0) -> Tuple[np.ndarray, np.ndarray]:
    """(ids [M, k], weights [M, k])."""
    x = to_f64(x)
    with np.errstate(all="ignore"):
        l = rms_inv(x, eps)[:, None] * ((x * to_f64(g)[None, :]) @ to_f64(router).T)
        if score == "softmax":
            e = np.exp(l - l.max(axis=1, keepdims=True))
            s = e / e.sum(axis=1, keepdims=True)
        else:
            s = 1.0 / (1.0 + np.exp(-l))
        key = l if select_bias is None else s + to_f64(select_bias)[None, :]
        key = np.where(np.isnan(key), -np.inf, key)
        ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
        w = np.take_along_axis(s, ids, axis=1)
        if renorm:
            w = w / w.sum(axis=1, keepdims=True)
    return ids, w * route_scale


def moe_swiglu(x, g, router, W_gate, W_up, W_down, k: int, eps: float, residual=None, **route):
    """(y [M, d], ids, weights); W_gate, W_up [E, d, I] with the gain folded in,
    W_down [E, I, d]."""
    ids, w = moe_route(x, g, router, k, eps, **route)
    x = to_f64(x)
    with np.errstate(all="ignore"):
        h = x * rms_inv(x, eps)[:, None]
        y = np.zeros_like(x) if residual is None else to_f64(residual).copy()
        for e in range(len(W_gate)):
            rows, slot = np.nonzero(ids == e)
            if rows.size:
                a = silu(h[rows] @ to_f64(W_gate[e])) * (h[rows] @ to_f64(W_up[e]))
                y[rows] += w[rows, slot][:, None] * (a @ to_f64(W_down[e]))
    return y, ids, w


def token_logprobs(logits, targets=None, top_k: int = 0, scale: float = 1.0):
    """(logprob [M] or None, entropy [M], lse [M], top_ids [M, k], top_logprobs [M, k])."""
    raw = to_f64(logits)
    M, V = raw.shape
    z = raw * float(np.float32(scale))
    lp = np.zeros(M) if targets is not None else None
    H, lse = np.zeros(M), np.zeros(M)
    ids, top = np.zeros((M, top_k), np.int64), np.zeros((M, top_k))
    for i in range(M):
        # largest first, ties to the lower index, NaN before every number
        order = np.lexsort((np.arange(V), -np.where(np.isnan(raw[i]), 0.0, raw[i]), ~np.isnan(raw[i])))[:top_k]
        ids[i] = order
        if np.isnan(z[i]).any() or np.isposinf(z[i]).any():
            H[i] = lse[i] = np.nan
            top[i] = np.nan
            v = np.nan
        elif np.isneginf(z[i]).all():
            lse[i], v = -np.inf, -np.inf
            top[i] = -np.inf
        else:
            m = z[i].max()
            s = np.exp(z[i] - m).sum()
            lse[i] = m + math.log(s)
            q = (z[i] - m) - math.log(s)
            p = np.exp(q)
            H[i] = -np.sum(p[p > 0] * q[p > 0])
            top[i] = q[order]
            v = None
        if lp is not None:
            t = int(targets[i])
            lp[i] = 0.0 if t < 0 else np.nan if t >= V else (v if v is not None else q[t])
    return lp, H, lse, ids, top


def token_logprobs_grad(logits, targets, grad_logprob=None, grad_entropy=None, scale: float = 1.0) -> np.ndarray:
    """Gradient of sum(gl * logprob + gh * entropy) with respect to the logits."""
    raw = to_f64(logits)
    M, V = raw.shape
    sc = float(np.float32(scale))
    out = np.zeros((M, V))
    for i in range(M):
        z = raw[i] * sc
        if np.isneginf(z).all():
            continue
        m = z.max()
        q = (z - m) - math.log(np.exp(z - m).sum())
        p = np.exp(q)
        if grad_logprob is not None and targets[i] >= 0:
            out[i] -= float(grad_logprob[i]) * p
            out[i, targets[i]] += float(grad_logprob[i])
        if grad_entropy is not None:
            safe = np.where(p > 0, q, 0.0)
            H = -np.sum(p * safe)
            out[i] -= float(grad_entropy[i]) * p * (safe + H)
    return out * sc
