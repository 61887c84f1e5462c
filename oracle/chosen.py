"""Float64 restatement of the operators whose weights are chosen for each token.

TEST INFRASTRUCTURE ONLY (see the package docstring): the product path never
imports this module.

* ``moe_route``: top-k of the router's logits, softmax weights;
* ``moe_awq_w4a16``: a mixture-of-experts layer on AWQ W4A16 experts, out_t =
  sum over t's slots of weight * (silu(x Wg^T) * (x Wu^T)) Wd^T;
* ``lora_add``: y + scale[a] * ((x A[a]^T) B[a]^T), a = ids[m].

Readings: a logit of -inf or NaN is not live and is never chosen; equal logits
go to the lowest index; where the largest logit is +inf, the +inf logits share
the weight equally; a slot without a live logit has id -1 and weight 0; ids
outside the range choose nothing.
"""

from __future__ import annotations

import numpy as np

from .convrot import awq_dequantize


def moe_route(logits, k: int, renormalize: bool):
    """(T, E) -> (weights (T, k) float64, ids (T, k) int32)."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    w = np.zeros((T, k))
    ids = np.full((T, k), -1, dtype=np.int32)
    for t in range(T):
        live = [e for e in range(E) if logits[t, e] > -np.inf]          # False for NaN
        live.sort(key=lambda e: (-logits[t, e], e))
        chosen = live[:k]
        if not chosen:
            continue
        m = logits[t, chosen[0]]
        p = {e: 1.0 if logits[t, e] == m else float(np.exp(logits[t, e] - m)) for e in live}
        total = sum(p[e] for e in (chosen if renormalize else live))
        for j, e in enumerate(chosen):
            ids[t, j] = e
            w[t, j] = p[e] / total
    return w, ids


def silu(v):
    v = np.asarray(v, dtype=np.float64)
    e = np.exp(-np.abs(v))
    return v * np.where(v >= 0, 1.0, e) / (1.0 + e)


def moe_awq_w4a16(x, ids, weights, gate_up, down, G: int):
    """x (T, K); ids, weights (T, k); gate_up and down: (bytes, scales, zeros) of all experts."""
    x = np.asarray(x, dtype=np.float64)
    T, K = x.shape
    E = gate_up[0].shape[0]
    I = gate_up[0].shape[1] // 2
    out = np.zeros((T, K))
    for e in sorted({int(i) for i in np.asarray(ids).ravel() if 0 <= i < E}):
        wgu = awq_dequantize(gate_up[0][e], gate_up[1][e], gate_up[2][e], G)
        wd = awq_dequantize(down[0][e], down[1][e], down[2][e], G)
        share = np.where(np.asarray(ids) == e, weights, 0.0).sum(axis=1)
        for t in np.nonzero((np.asarray(ids) == e).any(axis=1))[0]:
            gu = wgu @ x[t]
            out[t] += share[t] * (wd @ (silu(gu[:I]) * gu[I:]))
    return out


def lora_add(y, x, a, b, ids, scales=None):
    out = np.array(y, dtype=np.float64)
    x, a, b = (np.asarray(v, dtype=np.float64) for v in (x, a, b))
    for m, i in enumerate(np.asarray(ids)):
        if 0 <= i < a.shape[0]:
            out[m] += (1.0 if scales is None else float(scales[i])) * (b[i] @ (a[i] @ x[m]))
    return out
