"""The vocabulary-row operators from their definitions in 64 bits (numpy), and
the error bounds that the kernels are held to. Shares no code with the package."""
import numpy as np

U32 = 2.0 ** -24  # unit roundoff of binary32


def _masked(x, temp):
    """z = x / T, with the row maxima and the sums of exponentials."""
    z = x.astype(np.float64) / temp
    with np.errstate(invalid="ignore", divide="ignore"):
        m = np.fmax.reduce(z, axis=-1) if z.shape[-1] else z
        ref = np.where(np.isfinite(m), m, 0.0)
        e = np.exp(z - ref[:, None])
        e[np.isposinf(z)] = np.nan
        s = e.sum(-1)
    return z, ref, e, s


def log_probs(x, temp):
    z, ref, e, s = _masked(x, temp)
    with np.errstate(invalid="ignore", divide="ignore"):
        lp = z - ref[:, None] - np.log(s)[:, None]
    lp[s == 0] = -np.inf
    lp[np.isnan(s)] = np.nan
    return lp


def logprobs(x, tokens=None, k=0, temp=1.0):
    """Dict of logprob, entropy, lse, top_ids, top_logprobs for [rows, cols] float64 x."""
    rows, cols = x.shape
    z, ref, _, s = _masked(x, temp)
    lp = log_probs(x, temp)
    p = np.exp(lp)
    out = {}
    with np.errstate(invalid="ignore", divide="ignore"):
        terms = np.where(p > 0, p * lp, 0.0)
        terms[np.isnan(lp)] = np.nan
        out["entropy"] = -terms.sum(-1)
        out["lse"] = np.where(s == 0, -np.inf, ref + np.log(s))
    if tokens is not None:
        got = np.zeros(rows)
        for r, t in enumerate(tokens):
            got[r] = 0.0 if t < 0 else np.nan if t >= cols else lp[r, t]
        out["logprob"] = got
    if k:
        # larger first, equal ones by index, NaNs last
        order = [np.lexsort((np.arange(cols), np.where(np.isnan(v), 0, -v), np.isnan(v)))[:k] for v in x]
        out["top_ids"] = np.stack(order)
        out["top_logprobs"] = np.take_along_axis(lp, out["top_ids"], 1)
    return out


def logprobs_grad(x, tokens, g, h, c, temp=1.0):
    """Gradient of sum(g logprob + h entropy + c lse) to x."""
    rows, cols = x.shape
    lp = log_probs(x, temp)
    p = np.exp(lp)
    ent = logprobs(x, temp=temp)["entropy"]
    out = np.zeros_like(p)
    for r in range(rows):
        if (x[r] == -np.inf).all():
            continue
        gr = 0.0 if tokens is None or tokens[r] < 0 else g[r]
        if tokens is not None and tokens[r] >= cols:
            gr = np.nan
        d = c[r] * p[r] - gr * p[r] - h[r] * p[r] * (np.where(p[r] > 0, lp[r], 0.0) + ent[r])
        if gr != 0 and 0 <= tokens[r] < cols:
            d[tokens[r]] += gr
        out[r] = d / temp
    return out


def teacher(ids, val, cols, temp, tail):
    """(q, ln q, rest) of one row's slots; None where an id is past the row."""
    if (ids >= cols).any():
        return None
    here = ids >= 0
    val = val.astype(np.float64)
    if tail:
        q = np.where(here, np.exp(np.where(here, val, 0.0)), 0.0)
        lnq = np.where(here, val, 0.0)
        return q, lnq, (max(0.0, 1.0 - q.sum()) if here.any() else 0.0)
    v = np.where(here, val / temp, -np.inf)
    if not (v > -np.inf).any():
        return np.zeros(len(ids)), np.zeros(len(ids)), 0.0
    v = v - v.max()
    q = np.exp(v) / np.exp(v).sum()
    return q, np.where(q > 0, v - np.log(np.exp(v).sum()), 0.0), 0.0


def distill(x, ids, val, temp=1.0, tail=False, grad_loss=None):
    """(loss, gradient or None) in 64 bits."""
    rows, cols = x.shape
    lp = log_probs(x, temp)
    p = np.exp(lp)
    loss = np.zeros(rows)
    grad = np.zeros_like(p) if grad_loss is not None else None
    for r in range(rows):
        t = teacher(ids[r], val[r], cols, temp, tail)
        if t is None:
            loss[r] = np.nan
            if grad is not None:
                grad[r] = np.nan
            continue
        q, lnq, rest = t
        used = q > 0
        if not used.any() and rest == 0.0:
            continue
        here = ids[r] >= 0
        other = np.ones(cols, bool)
        other[ids[r][here]] = False
        mass = p[r][other].sum()
        with np.errstate(invalid="ignore", divide="ignore"):
            loss[r] = (q[used] * (lnq[used] - lp[r][ids[r][used]])).sum()
            if np.isnan(lp[r]).any():
                loss[r] = np.nan
            if rest > 0 and (mass > 0 or np.isnan(mass)):
                loss[r] += rest * (np.log(rest) - np.log(mass))
            else:
                rest = 0.0
        if grad is not None:
            if (x[r] == -np.inf).all():
                continue
            d = (q.sum() + rest) * p[r]
            d[ids[r][here]] -= q[here]
            if rest > 0:
                d[other] -= rest * p[r][other] / mass
            grad[r] = d * grad_loss[r] / temp
    return loss, grad


# ---------------------------------------------------------------------------
# Error bounds. A sum of n positive terms is off by a share of at most about
# 6 sqrt(n) u (the probabilistic bound of Higham and Mary, "A new approach to
# probabilistic rounding error analysis", 2019, with lambda = 6); a thread adds
# at most cols / 32 of them. Each term exp2(y) carries the rounding of y (four
# roundings of |y| <= 24 or so where the term matters, each |y| ln 2 u) and the two
# units in the last place of the exponential: below 100 u.
# ---------------------------------------------------------------------------
def sum_error(cols):
    return U32 * (6.0 * np.sqrt(max(1.0, cols / 32)) + 100.0)


def logprob_bound(ref, cols):
    """|error| of a log probability, lse or loss of this value."""
    return sum_error(cols) + 8 * U32 * np.abs(np.where(np.isfinite(ref), ref, 0.0))


def entropy_bound(ref, lnv, cols):
    """entropy = ln s - ln 2 t / s, both sums off by sum_error (t by twice that), |ln 2 t / s| <= ln s + entropy <= 2 lnv."""
    return 3 * sum_error(cols) * (1.0 + 2 * lnv) + 8 * U32 * np.abs(np.where(np.isfinite(ref), ref, 0.0))


ROUND = {"f32": (2.0 ** -24, 0.0), "f16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 0.0)}


def grad_bound(ref, terms, cols, dtype):
    """|error| of a gradient element: the rounding to its type and, for the sum
    of terms that it is (`terms`, their absolute values), sum_error of them."""
    rel, least = ROUND[dtype]
    fine = np.abs(np.where(np.isfinite(ref), ref, 0.0))
    return rel * fine + least + (2 * sum_error(cols)) * terms + 1e-37
