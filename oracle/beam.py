"""Beam search's selection, oracle side (test infrastructure; shares no code with
the CUDA-side library).

The pages name beam search only as a sharer of a prompt's blocks ("PagedAttention:
The vLLM Paper", "Implementation Essentials", prefix sharing). Reading taken, the
plain definition: score[k][v] = beam_score[k] + x[k][v] - log sum_u exp(x[k][u]),
in float64; the best candidates over all (k, v), ties to the smaller k V + v;
-inf scores are no candidates, a beam with a NaN or +inf among its logits or as
its score has none; places left over are (-inf, -1, -1).
"""

import math

import numpy as np


def all_scores(logits, beam_scores):
    """float64 [K, V] scores of one sequence, and whether a beam was rejected."""
    x = np.asarray(logits, np.float64)
    out = np.full(x.shape, -math.inf)
    bad = False
    for k in range(len(x)):
        b = float(beam_scores[k])
        if np.isnan(x[k]).any() or (x[k] == math.inf).any() or b != b or b == math.inf:
            bad = True
            continue
        top = x[k].max()
        if top == -math.inf or b == -math.inf:
            continue
        # x - top first: a row of values near the type's largest magnitude keeps its log V
        out[k] = (x[k] - top) + (b - math.log(np.exp(x[k] - top).sum()))
    return out, bad


def select(logits, beam_scores, n):
    """(scores, parents, tokens) of one sequence."""
    s, _ = all_scores(logits, beam_scores)
    flat = s.reshape(-1)
    order = np.argsort(-flat, kind="stable")[:n]
    order = order[flat[order] > -math.inf]
    scores = np.full(n, -math.inf)
    parents, tokens = np.full(n, -1), np.full(n, -1)
    scores[:len(order)] = flat[order]
    parents[:len(order)], tokens[:len(order)] = np.divmod(order, s.shape[1])
    return scores, parents, tokens
