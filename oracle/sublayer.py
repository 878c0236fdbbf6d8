"""Float64 CPU oracle of the sublayer operators (test infrastructure only):
routing to experts, the permutation by expert, the linear product with its
epilogue, the experts' products.

Representation as in the boundary's oracle: bf16 tensors are float64 arrays of
bf16-exact values, roundings are explicit. Index outputs are int64 arrays.
"""

from __future__ import annotations

import math

import numpy as np

from .mhc import bf16_round

__all__ = ["moe_route", "moe_permute", "linear", "moe_experts", "activation"]


def moe_route(logits, top_k, bias=None, scoring="softmax", num_groups=1, top_groups=1, group_top=1, renormalize=True,
              weight_scale=1.0):
    """(weights [R, k], ids [R, k]) of logits [R, E], row by row from the definition.

    An expert whose logit or bias is -inf or NaN is not available. Without a
    bias, choices order as the logits (the scores' own order, where scores that
    are equal in floating point stand for different logits)."""
    logits = np.asarray(logits, dtype=np.float64)
    R, E = logits.shape
    weights = np.zeros((R, top_k))
    ids = np.full((R, top_k), -1, dtype=np.int64)
    size = E // num_groups
    for r in range(R):
        l = [v if v == v else -math.inf for v in logits[r].tolist()]
        if scoring == "softmax":
            top = max(l)
            if top == math.inf:
                s = [1.0 if v == math.inf else 0.0 for v in l]
            else:
                s = [0.0 if v == -math.inf else math.exp(v - top) for v in l]
            total = math.fsum(s)
            s = [v / total if total > 0 else 0.0 for v in s]
        else:
            s = [1.0 / (1.0 + math.exp(-v)) if v > -700 else math.exp(max(v, -2000.0)) for v in l]
        free, value = [], {}
        for e in range(E):
            v = s[e] + (0.0 if bias is None else float(bias[e]))
            if l[e] != -math.inf and v > -math.inf:
                free.append(e)
                value[e] = v
        if num_groups > 1:
            worth = []
            for g in range(num_groups):
                best = sorted((value[e] for e in free if e // size == g), reverse=True)[:group_top]
                if best:
                    worth.append((-sum(best), g))
            kept = {g for _, g in sorted(worth)[:top_groups]}
            free = [e for e in free if e // size in kept]
        key = (lambda e: (-value[e], e)) if bias is not None else (lambda e: (-l[e], e))
        chosen = sorted(free, key=key)[:top_k]
        w = [s[e] for e in chosen]
        if renormalize and chosen:
            if scoring == "softmax" and max(l) != math.inf:  # ratios of the exponentials, free of underflow
                m = max(l[e] for e in chosen)
                w = [math.exp(l[e] - m) for e in chosen]
            total = math.fsum(w)
            w = [v / total if total > 0 else 0.0 for v in w]
        ids[r, : len(chosen)] = chosen
        weights[r, : len(chosen)] = [v * weight_scale for v in w]
    return weights, ids


def moe_permute(ids, experts):
    """(e2p [R*k], permuted_rows [R*k], offsets [E+1]) of the stable sort of the
    pairs (row, slot) by expert; a slot without an expert (id < 0) has place -1,
    places behind the last pair have row -1."""
    R, k = ids.shape
    e2p = np.full(R * k, -1, dtype=np.int64)
    rows = np.full(R * k, -1, dtype=np.int64)
    offsets = np.zeros(experts + 1, dtype=np.int64)
    place = 0
    flat = ids.reshape(-1)
    for e in range(experts):
        for i in np.nonzero(flat == e)[0]:
            e2p[i] = place
            rows[place] = i // k
            place += 1
        offsets[e + 1] = place
    return e2p, rows, offsets


def activation(name, v):
    if name == "none":
        return v
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "silu":
        return v / (1.0 + np.exp(-v))
    if name == "gelu":
        return v * 0.5 * (1.0 + np.vectorize(math.erf)(v / math.sqrt(2.0)))
    raise ValueError(name)


def linear(x, weight, bias=None, act="none", residual=None):
    """act(x weight^T + bias) + residual, unrounded; "swiglu": the first half of
    the features gates the second."""
    y = np.asarray(x, np.float64) @ np.asarray(weight, np.float64).T
    if bias is not None:
        y = y + bias
    if act == "swiglu":
        g, u = np.split(y, 2, axis=1)
        y = activation("silu", g) * u
    else:
        y = activation(act, y)
    return y if residual is None else y + residual


def moe_experts(x, w13, w2, permuted_rows, offsets):
    """gemm2_permuted [P, H], unrounded, the intermediate rounded to bf16; rows
    behind the last expert's are NaN."""
    out = np.full((len(permuted_rows), x.shape[1]), np.nan)
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a < b:
            inner = bf16_round(linear(x[permuted_rows[a:b]], w13[e], act="swiglu"))
            out[a:b] = inner @ w2[e].T
    return out
