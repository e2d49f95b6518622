"""Mixture-of-experts layer for given dequantized experts (oracle, fp64).

  l = x router^T; p = softmax(l); the top_k experts of the largest l, ties to
  the lowest index; optionally their p divided by their sum;
  y = sum_j p_j down_e (silu(gate_e x) * (up_e x)).

A logit of -inf masks its expert (p = 0, chosen last); a token with every
expert masked has p = 0 throughout.
"""

import numpy as np


def route(logits, top_k, renormalize):
    """(ids int32 [t][top_k], probs fp64 [t][top_k]), in order of decreasing logit."""
    l = np.asarray(logits, np.float64)
    t, e = l.shape
    ids = np.zeros((t, top_k), np.int32)
    probs = np.zeros((t, top_k))
    for i in range(t):
        order = sorted(range(e), key=lambda j: (-l[i, j], j))[:top_k]
        ids[i] = order
        if l[i, order[0]] == -np.inf:
            continue
        w = np.exp(l[i] - l[i, order[0]])
        p = w / w.sum()
        probs[i] = p[order] / (p[order].sum() if renormalize else 1.0)
    return ids, probs


def experts(x, ids, probs, gate, up, down):
    """y fp64 [t][h] for gate, up [e][i][h] and down [e][h][i]."""
    x = np.asarray(x, np.float64)
    y = np.zeros_like(x)
    for t in range(x.shape[0]):
        for e, p in zip(ids[t], probs[t]):
            if p == 0:
                continue
            g, u = gate[e] @ x[t], up[e] @ x[t]
            y[t] += down[e] @ (p * (g / (1.0 + np.exp(-g)) * u))
    return y
