"""Beam selection, beam reordering and routing from their definitions in 64 bits
(numpy). Shares no code with the package. Error bounds as in logits_ref."""
import numpy as np

import logits_ref as ref


def beam_totals(x, scores, ended=None, end_token=0, temp=1.0):
    """[beams, vocab (+ end)] totals of one item's continuations: -inf where there is none; None where
    what is looked at holds a NaN or +inf. An ended beam's continuation is named by the last column."""
    beams, cols = x.shape
    out = np.full((beams, cols + 1), -np.inf)
    for b in range(beams):
        s = float(scores[b])
        if s == -np.inf:
            continue
        if not np.isfinite(s):
            return None
        if ended is not None and ended[b]:
            out[b, cols] = s
            continue
        lp = ref.log_probs(x[b:b + 1], temp)[0]
        if np.isnan(lp).any():
            return None
        out[b, :cols] = s + lp
    return out


def beam_select(x, scores, count, ended=None, end_token=0, scale=None, temp=1.0):
    """One item: (tokens, parents, scores, ranks of the places, the next rank that was left out)."""
    beams, cols = x.shape
    totals = beam_totals(x, scores, ended, end_token, temp)
    w = np.ones(beams) if scale is None else scale.astype(np.float64)
    live = scores != -np.inf
    if totals is None or not (np.isfinite(w[live]) & (w[live] > 0)).all():
        return np.full(count, -1), np.full(count, -1), np.full(count, np.nan), None, None
    with np.errstate(invalid="ignore"):
        ranks = np.where(totals > -np.inf, totals * np.where(live, w, 1.0)[:, None], -np.inf)
    order = np.argsort(-ranks.ravel(), kind="stable")
    chosen = order[:count]
    good = ranks.ravel()[chosen] > -np.inf
    token = np.where(chosen % (cols + 1) == cols, end_token, chosen % (cols + 1))
    after = ranks.ravel()[order[count]] if len(order) > count else -np.inf
    return (np.where(good, token, -1), np.where(good, chosen // (cols + 1), -1),
            np.where(good, totals.ravel()[chosen], -np.inf), ranks.ravel()[chosen], after)


def reorder(state, parents, lengths=None, dim=None):
    """state [batch, beams, ...]; dim counts the state's own dimensions."""
    out = state.copy()
    for i, row in enumerate(parents):
        for j, p in enumerate(row):
            if not 0 <= p < parents.shape[1]:
                continue
            at = [slice(None)] * (state.ndim - 2)
            if lengths is not None:
                at[dim - 2] = slice(0, max(0, int(lengths[i])))
            out[(i, j, *at)] = state[(i, p, *at)]
    return out


def route(x, k, normalize=True, valid=None):
    """(weights, ids, lse, counts, rows that take part, balance) for [rows, experts] float64 x."""
    rows, experts = x.shape
    weights, ids = np.zeros((rows, k)), np.full((rows, k), -1)
    lse = np.full(rows, -np.inf)
    counts, total, n = np.zeros(experts, int), np.zeros(experts), 0
    for r in range(rows):
        if (valid is not None and not valid[r]) or (x[r] == -np.inf).all():
            continue
        n += 1
        lp = ref.log_probs(x[r:r + 1], 1.0)[0]
        order = [e for e in np.lexsort((np.arange(experts), -np.where(np.isnan(x[r]), -np.inf, x[r]))) if x[r, e] > -np.inf][:k]
        ids[r, :len(order)] = order
        counts[order] += 1
        if np.isnan(lp).any():
            weights[r], lse[r], total[:] = np.nan, np.nan, np.nan
            continue
        lse[r] = ref.logprobs(x[r:r + 1])["lse"][0]
        p = np.exp(lp)
        weights[r, :len(order)] = np.exp(lp[order] - np.logaddexp.reduce(lp[order]) if normalize else lp[order])
        total += p
    balance = experts * (counts / (k * max(n, 1)) * (total / max(n, 1))).sum()
    return weights, ids, lse, counts, n, balance


def route_grad(x, ids, counts, n, k, g, h, b, normalize=True, valid=None):
    """(gradient, sum of the absolute values of the terms of each element), from the formula."""
    rows, experts = x.shape
    out, size = np.zeros_like(x), np.zeros_like(x)
    c = b * experts * counts / (k * max(n, 1) ** 2)
    for r in range(rows):
        if (valid is not None and not valid[r]) or (x[r] == -np.inf).all():
            continue
        lp = ref.log_probs(x[r:r + 1], 1.0)[0]
        if np.isnan(lp).any():
            out[r] = np.nan
            continue
        p = np.exp(lp)
        at = ids[r][ids[r] >= 0]
        gr = g[r][ids[r] >= 0]
        w = np.exp(lp[at] - np.logaddexp.reduce(lp[at])) if normalize and len(at) else p[at]
        along = (gr * w).sum()
        out[r] = p * (c - (c * p).sum() + h[r] - (0 if normalize else along))
        out[r, at] += w * (gr - (along if normalize else 0))
        size[r] = p * (np.abs(c) + np.abs(c * p).sum() + np.abs(h[r]) + np.abs(gr * w).sum())
        size[r, at] += w * (np.abs(gr) + np.abs(gr * w).sum())
    return out, size
