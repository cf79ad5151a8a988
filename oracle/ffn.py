"""FFN block around the FP8 linears, in float64: the linear with bias,
activation and residual, the MoE router, and the whole MoE FFN of a few tokens.

Definitions (the source pages name the linears alone; these are the common ones):
    linear_epilogue  act((P * s_x) * s_w + bias) + residual
    route            the k largest logits of a token, ties to the lower expert,
                     NaN below -inf; softmax weights; rows by (expert, token)
    moe_layer        per (token, choice): quantize, up, activation (gated:
                     act(z[:F]) * z[F:]), fp16, quantize, down; weighted sum
Results that the device rounds to fp16 at the end are returned unrounded in
float64, with the sum of the product's absolute terms where a caller bounds an
fp32 accumulation by it.
"""
from __future__ import annotations

import math

import numpy as np

from .e4m3 import e4m3_decode
from .e5m2 import e5m2_decode
from .quant import quant_rows

_DECODERS = {"e4m3": e4m3_decode, "e5m2": e5m2_decode}
_erfc = np.frompyfunc(math.erfc, 1, 1)


def activation_ref(z: np.ndarray, name) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    if name in (None, "none"):
        return z
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0)).astype(np.float64)
    if name == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z * 0.5 * (1.0 + np.tanh(0.5 * z))   # z / (1 + exp(-z)) without overflow
    raise ValueError(name)


def product_terms(Xq, s_x, Wq, s_w, x_fmt: str = "e4m3") -> tuple[np.ndarray, np.ndarray]:
    """The dequantized product [M,N] and the sum of its terms' absolute values, float64."""
    x, w = _DECODERS[x_fmt](Xq), e4m3_decode(Wq)
    scale = np.asarray(s_x, dtype=np.float64)[:, None] * np.asarray(s_w, dtype=np.float64)[None, :]
    return (x @ w.T) * scale, (np.abs(x) @ np.abs(w).T) * scale


def linear_epilogue_ref(Xq, s_x, Wq, s_w, bias=None, activation=None, residual=None, x_fmt: str = "e4m3"):
    """-> (unrounded result [M,N], sum of absolute product terms [M,N]), float64."""
    z, terms = product_terms(Xq, s_x, Wq, s_w, x_fmt)
    if bias is not None:
        z = z + np.asarray(bias, dtype=np.float64)[None, :]
    y = activation_ref(z, activation)
    if residual is not None:
        y = y + np.asarray(residual, dtype=np.float64)
    return y, terms


def route_ref(logits, topk: int, renormalize: bool = True) -> dict:
    """Router on fp16 logits [T,E], by a plain sort per token and plain loops."""
    L = np.asarray(logits).astype(np.float64)
    T, E = L.shape
    experts = np.zeros((T, topk), dtype=np.int32)
    weights = np.zeros((T, topk), dtype=np.float64)
    rows = []
    for t in range(T):
        def rank(e):
            v = L[t, e]
            return (1, 0.0, e) if math.isnan(v) else (0, -v, e)
        best = sorted(range(E), key=rank)[:topk]
        m = L[t, best[0]]
        for j, e in enumerate(best):
            experts[t, j] = e
            rows.append((e, t, j))
        if math.isnan(m) or m == -math.inf:
            continue   # no usable logit: weights 0
        def term(v):
            return 0.0 if math.isnan(v) else 1.0 if v == m else math.exp(v - m)
        total = math.fsum(term(L[t, e]) for e in (best if renormalize else range(E)))
        for j, e in enumerate(best):
            weights[t, j] = term(L[t, e]) / total
    rows.sort()
    offsets = np.zeros(E + 1, dtype=np.int32)
    token_rows = np.zeros((T, topk), dtype=np.int32)
    for r, (e, t, j) in enumerate(rows):
        offsets[e + 1] += 1
        token_rows[t, j] = r
    return {"experts": experts, "weights": weights, "offsets": np.cumsum(offsets).astype(np.int32),
            "row_token": np.array([t for _, t, _ in rows], dtype=np.int32),
            "row_weight": np.array([weights[t, j] for _, t, j in rows], dtype=np.float64), "token_rows": token_rows}


def moe_hidden_ref(X, experts, Wq_up, s_up, activation, gated: bool):
    """Unrounded hidden rows [T*topk, F] (zero where the expert is -1) and a bound's
    ingredients: the absolute product terms of both halves, [T*topk, F] or [T*topk, 2F]."""
    T, topk = np.asarray(experts).shape
    xq, s_x = quant_rows(np.asarray(X))
    up = Wq_up.shape[1]
    F = up // 2 if gated else up
    z = np.zeros((T * topk, up))
    terms = np.zeros((T * topk, up))
    flat = np.asarray(experts).reshape(-1)
    for e in sorted(set(flat.tolist()) - {-1}):
        at = np.nonzero(flat == e)[0]
        z[at], terms[at] = product_terms(xq[at // topk], s_x[at // topk], Wq_up[e], s_up[e])
    h = activation_ref(z[:, :F], activation) * z[:, F:] if gated else activation_ref(z, activation)
    return h, z, terms


def moe_out_ref(hidden_f16, experts, weights, Wq_down, s_down, residual=None):
    """Unrounded output [T,N] from fp16 hidden rows [T*topk, F], and the weighted
    sum of absolute product terms, float64."""
    T, topk = np.asarray(experts).shape
    N = Wq_down.shape[1]
    flat = np.asarray(experts).reshape(-1)
    y = np.zeros((T * topk, N))
    terms = np.zeros((T * topk, N))
    for e in sorted(set(flat.tolist()) - {-1}):
        at = np.nonzero(flat == e)[0]
        hq, s_h = quant_rows(np.asarray(hidden_f16)[at])
        y[at], terms[at] = product_terms(hq, s_h, Wq_down[e], s_down[e])
    w = np.where(flat >= 0, np.asarray(weights, dtype=np.float64).reshape(-1), 0.0)[:, None]
    out = (y * w).reshape(T, topk, N).sum(1)
    terms = (terms * np.abs(w)).reshape(T, topk, N).sum(1)
    if residual is not None:
        out = out + np.asarray(residual, dtype=np.float64)
    return out, terms


def moe_layer_ref(X, experts, weights, Wq_up, s_up, Wq_down, s_down, activation, gated=False, residual=None):
    """The whole layer: -> (unrounded output [T,N] float64, hidden rows fp16)."""
    h, _, _ = moe_hidden_ref(X, experts, Wq_up, s_up, activation, gated)
    h16 = h.astype(np.float16)
    return moe_out_ref(h16, experts, weights, Wq_down, s_down, residual)[0], h16
