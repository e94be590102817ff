"""CPU oracle of the plain MXFP4 product and of expert routing (NumPy, float64).

The product is the dense one that the two-path GEMM decomposes:
Y = deq(A) @ deq(W)^T. Routing follows the definition in include/sharq.h one
token at a time, in Python: scores, ordering keys, groups, the k best with
ties to the lower index, weights, and a stable sort of the pairs by expert.
"""

from __future__ import annotations

import math

import numpy as np

from .sharq_ref import mxfp4_dequantize, unpack_nibbles

__all__ = ["linear_mxfp4_ref", "moe_route_ref"]


def _values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    return mxfp4_dequantize(unpack_nibbles(np.asarray(codes)), np.asarray(scales).astype(np.int64) - 127)


def linear_mxfp4_ref(a_codes, a_scales, w_codes, w_scales):
    """(Y, B): the product in float64 from row-major codes [R, K/2] and scale
    bytes [R, K/32], and B = |A| @ |W|^T, the sum of |a_k w_k| per output."""
    a = np.asarray(_values(a_codes, a_scales), dtype=np.float64)
    w = np.asarray(_values(w_codes, w_scales), dtype=np.float64)
    return a @ w.T, np.abs(a) @ np.abs(w).T


def moe_route_ref(logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_score="max",
                  renormalize=True, scale=1.0, num_tokens=None):
    """dict of expert [T, k], weight float64 [T, k], seg_offsets [E+1],
    a_rows [T k], pair_index [T, k]."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    top_groups = groups if top_groups is None else top_groups
    num_tokens = T if num_tokens is None else num_tokens
    expert = np.full((T, k), -1, np.int32)
    weight = np.zeros((T, k))
    for t in range(min(T, num_tokens)):
        x = [min(v, float(np.finfo(np.float32).max)) for v in logits[t].tolist()]
        live = [e for e in range(E) if x[e] > -math.inf]  # False for NaN as well
        s = {}
        if live and score == "softmax":
            top = max(x[e] for e in live)
            total = math.fsum(math.exp(x[e] - top) for e in live)
            s = {e: math.exp(x[e] - top) / total for e in live}
        elif live:
            s = {e: 1 / (1 + math.exp(-x[e])) if x[e] > -700 else 0.0 for e in live}
        value = {e: x[e] if bias is None else s[e] + float(bias[e]) for e in live}
        value = {e: v for e, v in value.items() if v > -math.inf}
        if groups > 1:
            size = E // groups
            rated = []
            for g in range(groups):
                members = sorted((value[e] if group_score == "max" or bias is not None else s[e]
                                  for e in range(g * size, (g + 1) * size) if e in value), reverse=True)
                if not members:
                    rated.append((math.inf, g))
                else:
                    rated.append((-(sum(members[:2]) if group_score == "sum2" else members[0]), g))
            kept = {g for _, g in sorted(rated)[:top_groups]}
            value = {e: v for e, v in value.items() if e // size in kept}
        best = sorted(value, key=lambda e: (-value[e], e))[:k]
        share = {e: s[e] for e in best}
        if renormalize and best:  # ratios of the scores: a common factor keeps them away from underflow
            top = max(x[e] for e in best)
            if score == "softmax":
                share = {e: math.exp(x[e] - top) for e in best}
            elif top < 0:
                share = {e: math.exp(x[e] - top) / (1 + math.exp(x[e])) for e in best}
            total = math.fsum(share.values())
            share = {e: v / total for e, v in share.items()}
        for j, e in enumerate(best):
            expert[t, j] = e
            weight[t, j] = scale * share[e]
    pairs = sorted((int(expert[t, j]), t, j) for t in range(T) for j in range(k) if expert[t, j] >= 0)
    seg = np.zeros(E + 1, np.int32)
    a_rows = np.full(T * k, -1, np.int32)
    pair_index = np.full((T, k), -1, np.int32)
    for p, (e, t, j) in enumerate(pairs):
        seg[e + 1] += 1
        a_rows[p] = t
        pair_index[t, j] = p
    return {"expert": expert, "weight": weight, "seg_offsets": np.cumsum(seg, dtype=np.int32), "a_rows": a_rows,
            "pair_index": pair_index}
