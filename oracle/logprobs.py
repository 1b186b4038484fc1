"""Oracle: log probabilities of tokens, entropies and alternatives, a row at a time in fp64 (test infrastructure only).

A row x of finite or -inf logits, over the temperature: log p(v) = x[v] - ln sum exp x, entropy = -sum p ln p over the
tokens with p > 0.  Alternatives: the tokens with a logit above -inf, by logit (the given one, not the quotient), equal
ones by index; missing ones are id -1 with -inf.  A row with no finite logit gives log p = -inf, entropy 0.
"""
from __future__ import annotations

import math

import numpy as np


def row(x, temperature=1.0):
    """log p of every token of a row, and the entropy."""
    x = np.asarray(x, np.float64)
    seen = x > -np.inf
    if not seen.any():
        return np.full(x.shape, -np.inf), 0.0
    y = x / temperature
    top = y[seen].max()
    logp = np.full(x.shape, -np.inf)
    logp[seen] = y[seen] - top - math.log(math.fsum(np.exp(y[seen] - top)))
    p = np.exp(logp[seen])
    return logp, -math.fsum(np.where(p > 0, p * logp[seen], 0.0))


def score(logits, tokens, rows=None, temperature=1.0, top=0):
    """logits [M, V], tokens [R], rows [R] -> logprob [R], entropy [R], ids [R, top], values [R, top]; an output whose row is
    out of range is NaN (id -2) throughout."""
    logits = np.asarray(logits)
    R = len(tokens)
    lp, ent = np.full(R, np.nan), np.full(R, np.nan)
    ids, alt = np.full((R, top), -2, np.int64), np.full((R, top), np.nan)
    for r in range(R):
        m = r if rows is None else int(rows[r])
        if not 0 <= m < len(logits):
            continue
        x = logits[m].astype(np.float64)
        logp, ent[r] = row(x, temperature)
        t = int(tokens[r])
        lp[r] = logp[t] if 0 <= t < len(x) else 0.0 if t == -1 else np.nan
        seen = np.flatnonzero(x > -np.inf)
        order = seen[np.argsort(-x[seen], kind="stable")][:top]
        ids[r], alt[r] = -1, -np.inf
        ids[r, :len(order)], alt[r, :len(order)] = order, logp[order]
    return lp, ent, ids, alt
