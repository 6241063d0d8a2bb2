"""Oracle: sampling from given random numbers, and the acceptance walk under sampling.

The pages verify greedily ([JF] technical summary section 1); under sampling the target's token at a node is a draw
from its distribution instead of the argmax, and the rest of the walk (:mod:`oracle.accept`) is unchanged.

Readings: the filters apply in the order temperature, min-p, top-k, top-p, each to what the one before kept; candidates
are ordered by (logit descending, token id ascending); min-p keeps x - m >= T ln(min_p) with m the row maximum; top-p
keeps the shortest non-empty prefix that holds at least that share of the weight kept so far; the drawn token is the
lowest kept id at which the running weight in id order exceeds u times the kept weight; temperature 0 is greedy.
-inf and NaN logits are no candidates; a row without candidates gives token -1 and log-probability -inf; equal maxima
of +inf share the weight.

Pinned by tests/test_oracle_sampling.py: closed forms on uniform and geometric rows, a hand-worked example, numpy's
choice of a sorted CDF without filters, greedy limits, and the interval of u that draws each token.
"""
from __future__ import annotations

import numpy as np


def kept_ids(x, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """Ids kept by the filters, ascending, and their weights exp((x - m) / T); float64 logits x."""
    x = np.asarray(x, dtype=np.float64)
    cand = np.flatnonzero(x > -np.inf)  # NaN compares false
    if cand.size == 0:
        return cand, np.zeros(0)
    m = x[cand].max()
    gap = np.zeros(cand.size)
    below = x[cand] != m
    gap[below] = x[cand][below] - m
    w = np.exp(gap / temperature)
    keep = np.ones(cand.size, bool) if min_p <= 0 else gap >= temperature * np.log(min_p)
    cand, w = cand[keep], w[keep]
    order = np.lexsort((cand, -x[cand]))
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1:
        c = np.cumsum(w[order])
        order = order[:max(1, int(np.sum(c < top_p * c[-1])) + 1)]
    order = np.sort(order)  # positions in cand, so ids ascend
    return cand[order], w[order]


def sample_row(x, u, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log-probability) of one row."""
    x = np.asarray(x, dtype=np.float64)
    if temperature == 0:
        cand = np.flatnonzero(x > -np.inf)
        if cand.size == 0:
            return -1, -np.inf
        return int(cand[np.argmax(x[cand])]), 0.0
    ids, w = kept_ids(x, temperature, top_k, top_p, min_p)
    if ids.size == 0:
        return -1, -np.inf
    c = np.cumsum(w)
    j = int(np.sum(c <= u * c[-1]))
    return int(ids[j]), float(np.log(w[j] / c[-1]))


def accept_sampled(token, parent, target_logits, u, max_depth, temperature, top_k=None, top_p=None, min_p=None):
    """token, parent int [B, N]; target_logits [B, N, V]; u [B, max_depth + 1]; parameters [B].  Returns
    (accepted_len, path, bonus, logprob)."""
    B, N = token.shape
    acc, bonus = np.zeros(B, np.int32), np.zeros(B, np.int32)
    path = np.full((B, max_depth + 1), -1, np.int32)
    logprob = np.zeros((B, max_depth + 1))
    for b in range(B):
        cur = L = 0
        path[b, 0] = 0
        how = [0 if top_k is None else int(top_k[b]), 1.0 if top_p is None else float(top_p[b]),
               0.0 if min_p is None else float(min_p[b])]
        while True:
            a, logprob[b, L] = sample_row(target_logits[b, cur], float(u[b, L]), float(temperature[b]), *how)
            if L == max_depth or a < 0:
                break
            kids = [c for c in range(N) if parent[b, c] == cur and token[b, c] == a]
            if not kids:
                break
            L += 1
            cur = path[b, L] = kids[0]
        acc[b], bonus[b] = L, a
    return acc, path, bonus, logprob
