"""Scores of given tokens, their gradients, and embedding rows, in fp64.

The definitions behind dspark_logprobs, dspark_logprobs_grad, dspark_embed and
dspark_embed_grad, one function each, on numpy arrays.
"""
from __future__ import annotations

import numpy as np


def row_scores(x: np.ndarray, token: int, top_k: int = 0) -> dict:
    """One row of logits: log probability of `token`, entropy, the largest
    logit and the sum of exponentials under it, and the alternatives. Bounds
    on first-order errors go by the moments E|x-m| and E|x-m|^2 (mean1, mean2)."""
    x = np.asarray(x, dtype=np.float64)
    ids, lps = np.full(top_k, -1, dtype=np.int32), np.full(top_k, -np.inf)
    seen = np.where(np.isnan(x), -np.inf, x)
    order = np.lexsort((np.arange(x.size), -seen))[:top_k]
    order = order[seen[order] > -np.inf]
    ids[:order.size] = order
    if np.any(np.isnan(x)) or np.any(x == np.inf):
        return {"logprob": np.nan, "entropy": np.nan, "m": np.nan, "s": np.nan, "top_tokens": ids,
                "top_logprobs": np.full(top_k, np.nan), "mean1": 0.0, "mean2": 0.0}
    m = x.max()
    if m == -np.inf:
        return {"logprob": -np.inf, "entropy": 0.0, "m": m, "s": 0.0, "top_tokens": ids, "top_logprobs": lps,
                "mean1": 0.0, "mean2": 0.0}
    d = x - m
    e = np.exp(d)
    s = e.sum()
    p = e / s
    dp = np.where(p > 0, d, 0.0)
    mean1, mean2 = float((p * -dp).sum()), float((p * dp * dp).sum())
    lps[:order.size] = x[order] - m - np.log(s)
    return {"logprob": x[token] - m - np.log(s), "entropy": np.log(s) + mean1, "m": m, "s": s, "top_tokens": ids,
            "top_logprobs": lps, "mean1": mean1, "mean2": mean2}


def row_scores_grad(x: np.ndarray, token: int, g_logprob: float, g_entropy: float = 0.0) -> np.ndarray:
    """Gradient of g_logprob * logprob + g_entropy * entropy with respect to x;
    0 at masked logits, and everywhere if nothing is left or token is -1."""
    x = np.asarray(x, dtype=np.float64)
    if token < 0 or np.all(x == -np.inf):
        return np.zeros_like(x)
    if np.any(np.isnan(x)) or np.any(x == np.inf):
        return np.full_like(x, np.nan)
    left = x > -np.inf
    d = x - x.max()
    e = np.exp(d)
    p = e / e.sum()
    lp = np.where(p > 0, d - np.log(e.sum()), 0.0)
    H = -(p * lp).sum()
    hit = np.arange(x.size) == token
    return np.where(left, g_logprob * (hit - p) - g_entropy * p * (lp + H), 0.0)


def embed(table: np.ndarray, tokens: np.ndarray, scale: float) -> np.ndarray:
    """scale * table[tokens], zeros for a token of -1."""
    rows = np.asarray(table, dtype=np.float64)[np.maximum(tokens, 0)] * scale
    return np.where((tokens >= 0)[:, None], rows, 0.0)


def embed_grad(dout: np.ndarray, tokens: np.ndarray, scale: float, dtable: np.ndarray | None, V: int) -> np.ndarray:
    """scale * the sum of dout's rows of each token, added to dtable (None: 0)."""
    dout = np.asarray(dout, dtype=np.float64)
    g = np.zeros((V, dout.shape[1])) if dtable is None else np.asarray(dtable, dtype=np.float64).copy()
    for i in np.argsort(tokens, kind="stable"):
        if tokens[i] >= 0:
            g[tokens[i]] += scale * dout[i]
    return g
