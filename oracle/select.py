"""Selection of experts from router scores (fp64, plain loops).

TEST INFRASTRUCTURE ONLY (see the package docstring).

Scores are sigmoids or the softmax over all experts; a bias is added for the
choice alone; experts in consecutive groups of equal size, whose value is the sum
of their one or two largest choices, are kept by the best groups; the largest
choices of the kept groups are taken.  Equal values go to the lower index, NaN
comes before every number.  A logit of -inf takes its expert out of service:
score 0, choice -inf, nothing for its group.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import numpy as np


def _best(values: list, n: int) -> list:
    """Indices of the n largest values, NaN first, ties to the lower index."""
    def key(i):
        v = values[i]
        return (0, 0.0, i) if math.isnan(v) else (1, -v, i)

    return sorted(range(len(values)), key=key)[:n]


def _scores_row(z: list, scores: str) -> list:
    if scores == "sigmoid":
        def sig(v):
            if math.isnan(v):
                return math.nan
            return 1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 if v == -math.inf else math.exp(v)

        return [sig(v) for v in z]
    live = [v for v in z if v != -math.inf]
    if any(math.isnan(v) or v == math.inf for v in live):
        return [0.0 if v == -math.inf else math.nan for v in z]
    if not live:
        return [0.0] * len(z)
    top = max(live)
    p = [0.0 if v == -math.inf else math.exp(v - top) for v in z]
    s = math.fsum(p)
    return [v / s for v in p]


def route_select(logits: np.ndarray, k: int, scores: str = "sigmoid",
                 bias: Optional[np.ndarray] = None, groups: int = 1, top_groups: int = 1,
                 group_top: int = 2, renormalise: bool = True,
                 scale: float = 1.0) -> Tuple[np.ndarray, np.ndarray]:
    """topk_ids int32 [T, k] and gates fp32 [T, k] from logits [T, E]."""
    lg = np.asarray(logits, dtype=np.float64)
    T, E = lg.shape
    per = E // groups
    ids = np.zeros((T, k), np.int32)
    gates = np.zeros((T, k), np.float32)
    for t in range(T):
        z = lg[t].tolist()
        s = _scores_row(z, scores)
        c = [-math.inf if z[e] == -math.inf else s[e] + (0.0 if bias is None else float(bias[e]))
             for e in range(E)]
        if groups > 1:
            value = []
            for g in range(groups):
                own = c[g * per:(g + 1) * per]
                first = [own[i] for i in _best(own, group_top)]
                value.append(first[0] if len(first) == 1 or first[1] == -math.inf else first[0] + first[1])
            kept = set(_best(value, top_groups))
            c = [v if e // per in kept else -math.inf for e, v in enumerate(c)]
        sel = _best(c, k)
        w = [0.0 if c[e] == -math.inf else s[e] for e in sel]
        if renormalise:
            total = 0.0
            for v in w:
                total += v
            w = [0.0 if total == 0 else v / total for v in w]
        ids[t] = sel
        gates[t] = np.array([v * float(np.float32(scale)) for v in w]).astype(np.float32)
    return ids, gates
