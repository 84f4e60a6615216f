"""Cases of the selections over rows of scores: a beam search's step over beams and vocabulary, the
reordering of what its beams keep, and a router's choice of experts with per-expert counts, the
balance loss and their gradients.

``run`` computes a case in its plain form (elementary torch operations, rounded once at the end) or,
where ``own`` is true, through the framework's kernels. ``exact`` is the definition in 64 bits,
written apart from the plain form.

* select: for each item, beams with totals s_b and logits x_b. Every continuation (b, v) has the
  total s_b + log softmax(x_b / T)_v; an ended beam has one, (b, end token), with the total s_b. The
  ``count`` continuations of the largest w_b * total (w_b a scale for the length, 1 without) come
  first to last, ties to the lowest (b, v): their tokens, beams and totals. Places that no
  continuation above -inf is left for have token and beam -1 and total -inf. Totals are taken in 64
  bits, since continuations of different beams lie close together.
* reorder: beam j of an item takes over what beam parents[j] kept (-1: it keeps its own), in every
  cache, for the item's first ``lengths`` positions; later positions stay as they were. In place.
* route: for each row of expert logits, the k largest (ties to the lowest index; what is not above
  -inf is not chosen: id -1, weight 0), their softmax weights over the chosen ones (normalize) or over
  all experts, the row's log-sum-exp, how many rows chose each expert, the number N of rows that
  took part (rows that are padding or wholly -inf do not), and the balance loss
  E * sum_e counts_e / (k N) * (sum of the softmax's e over the rows) / N.
* route_grad: the gradient of sum(g * weights) + sum(h * lse) + b * balance to the logits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i64": torch.int64}
ES = {"f32": 4, "f16": 2, "bf16": 2, "i64": 8}
END = 2  # the token that an ended beam goes on with


def listed():
    return [
        # a single request's first step: one beam has begun, the others wait (total -inf). Latency alone
        select("beam_first", 1, 4, 32000, "f32", 8, begun=1),
        # a server's batch of requests, twice as many continuations as beams, as some of them end
        select("beam_batch", 16, 4, 202048, "bf16", 8),
        # answers held to a grammar: nearly every logit is -inf; an odd vocabulary, ended beams that
        # compete by a scale for their length
        select("beam_grammar", 9, 5, 100003, "f16", 10, allowed=0.001, ended=0.2, scaled=True),
        # translating a corpus: many requests, many beams
        select("beam_wide", 64, 16, 202048, "bf16", 32, ended=0.05),
        # the token histories of a few requests: latency alone
        reorder("reorder_tokens", 4, 4, 1, 1, 513, 1, "i64"),
        # a batch's key and value caches over 16 layers, requests of different lengths
        reorder("reorder_caches", 16, 4, 32, 8, 1024, 128, "bf16"),
        # recurrent states of odd sizes, 5 beams
        reorder("reorder_odd", 9, 5, 12, 3, 77, 129, "f32"),
        # the tokens of one decoding step: latency alone
        route("route_decode", "route", 8, 64, "f32", 6, balance=False),
        # a training batch, padded positions among it
        route("route_train", "route", 65536, 256, "f32", 8, padded=0.1),
        # few experts, as many rows
        route("route_few", "route", 65536, 8, "bf16", 2),
        # the gradients of both batches, the second with an odd number of experts and weights over all
        route("route_grad_train", "route_grad", 65536, 256, "f32", 8, padded=0.1),
        route("route_grad_odd", "route_grad", 20001, 60, "bf16", 4, normalize=False),
    ]


def select(name, items, beams, cols, dtype, count, temp=1.0, begun=0, allowed=1.0, ended=0.0, scaled=False, pad=0):
    """begun: how many beams have begun (0: all); allowed: share of the logits that are not -inf;
    ended: share of the beams that have ended; pad: elements between the end of a row and the next."""
    c = {"op": "select", "items": items, "beams": beams, "cols": cols, "dtype": dtype, "count": count, "temp": temp,
         "begun": begun, "allowed": allowed, "ended": ended, "scaled": scaled, "pad": pad}
    return dict(c, name=name) if name else c


def reorder(name, items, beams, caches, heads, positions, width, dtype, ragged=True):
    c = {"op": "reorder", "items": items, "beams": beams, "caches": caches, "heads": heads, "positions": positions,
         "width": width, "dtype": dtype, "ragged": ragged}
    return dict(c, name=name) if name else c


def route(name, op, rows, experts, dtype, k, normalize=True, balance=True, padded=0.0, pad=0):
    """padded: share of the rows that are padding; pad: elements between the end of a row and the next."""
    c = {"op": op, "rows": rows, "experts": experts, "dtype": dtype, "k": k, "normalize": normalize,
         "balance": balance, "padded": padded, "pad": pad}
    return dict(c, name=name) if name else c


def log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """Requests from 1 to 64 with 1 to 16 beams over vocabularies of 1000 to 262144; caches up to 2 GiB;
    rows from 1 to 65536 over 2 to 512 experts; every direction, type and option."""
    op = rng.choice(["select", "select", "reorder", "route", "route_grad"])
    if op == "select":
        dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
        cols = log_int(rng, 1000, 262144)
        beams = rng.randint(1, 16)
        most = max(1, min(64, 1024 * 202048 * 2 // (beams * cols * ES[dtype])))
        return select(None, log_int(rng, 1, most), beams, cols, dtype, rng.randint(1, 2 * beams),
                      temp=rng.choice([1.0, 1.0, 0.8]), begun=1 if rng.random() < 0.15 else 0,
                      allowed=0.002 if rng.random() < 0.2 else 1.0, ended=rng.choice([0.0, 0.1, 0.3]),
                      scaled=rng.random() < 0.3, pad=rng.choice([0, 0, rng.randint(1, 128)]))
    if op == "reorder":
        dtype = rng.choice(["f32", "f16", "bf16", "i64"])
        beams, heads, width = rng.randint(1, 16), rng.randint(1, 16), rng.choice([1, 64, 128, rng.randint(2, 256)])
        row = heads * width * ES[dtype]
        positions = log_int(rng, 1, 2048)
        ragged = rng.random() < 0.7
        most = max(1, (1 + ragged) * 2**30 // (row * positions * beams))
        items = log_int(rng, 1, min(64, most))
        return reorder(None, items, beams, log_int(rng, 1, min(32, max(1, most // items))), heads, positions, width,
                       dtype, ragged=ragged)
    experts = log_int(rng, 2, 512)
    rows = log_int(rng, 1, min(65536, 65536 * 256 // experts))
    return route(None, op, rows, experts, rng.choice(["f32", "f32", "f16", "bf16"]),
                 log_int(rng, 1, min(16, experts)), normalize=rng.random() < 0.7, balance=rng.random() < 0.8,
                 padded=rng.choice([0.0, 0.1, 0.4]), pad=rng.choice([0, 0, rng.randint(1, 64)]))


def prepare(c, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    make = {"select": prepare_select, "reorder": prepare_reorder}.get(c["op"], prepare_route)
    return dict(make(c, gen), case=c)


def rand(gen, *shape):
    return torch.rand(*shape, device="cuda", generator=gen)


def prepare_select(c, gen):
    items, beams, cols = c["items"], c["beams"], c["cols"]
    store = torch.empty(items, beams, cols + c["pad"], device="cuda")
    store.normal_(0.0, 3.0, generator=gen)
    if c["allowed"] < 1.0:
        store.masked_fill_(rand(gen, *store.shape) >= c["allowed"], -math.inf)
        store[0, :, 3:] = -math.inf  # the grammar leaves the first item three tokens at most
        store[:, :, 1] = 0.5  # and every beam one
    # totals of some twenty tokens, best first, as the step before left them
    scores = (-20.0 - 3.0 * rand(gen, items, beams)).sort(-1, descending=True)[0]
    if c["begun"]:
        scores[:, c["begun"]:] = -math.inf
        store[:, c["begun"]:] = math.nan  # and what the model gave for them is not looked at
    s = {"x": store.to(DTYPES[c["dtype"]])[..., :cols], "scores": scores.contiguous(), "ended": None, "scale": None}
    if c["ended"]:
        s["ended"] = rand(gen, items, beams) < c["ended"]
    if c["scaled"]:
        length = torch.randint(5, 40, (items, beams), device="cuda", generator=gen)
        s["scale"] = (6.0 / (5.0 + length)) ** 0.6
    return s


def prepare_reorder(c, gen):
    items, beams = c["items"], c["beams"]
    shape = (items * beams, c["heads"], c["positions"], c["width"])
    dtype = DTYPES[c["dtype"]]
    if dtype.is_floating_point:
        caches = [torch.randn(shape, device="cuda", generator=gen, dtype=dtype) for _ in range(c["caches"])]
    else:
        caches = [torch.randint(0, 32000, shape, device="cuda", generator=gen) for _ in range(c["caches"])]
    # a step's survivors: about half the beams go on from themselves, the better ones have more successors
    parents = (rand(gen, items, beams) ** 2 * beams).long().clamp(max=beams - 1)
    stay = rand(gen, items, beams) < 0.4
    parents = torch.where(stay, torch.arange(beams, device="cuda"), parents)
    parents = torch.where(rand(gen, items, beams) < 0.03, -1, parents)  # a place that nothing was left for
    lengths = torch.randint(0, c["positions"] + 1, (items,), device="cuda", generator=gen) if c["ragged"] else None
    return {"caches": caches, "parents": parents, "lengths": lengths}


def prepare_route(c, gen):
    rows, experts, k = c["rows"], c["experts"], c["k"]
    store = torch.empty(rows, experts + c["pad"], device="cuda")
    store.normal_(0.0, 1.0, generator=gen)
    store += torch.randn(store.shape[1], device="cuda", generator=gen) * 0.5  # some experts are liked better
    s = {"valid": None}
    if c["padded"]:
        s["valid"] = rand(gen, rows) >= c["padded"]
        store[~s["valid"]] = math.nan  # nothing is promised about padding
    s["x"] = store.to(DTYPES[c["dtype"]])[:, :experts]
    if c["op"] == "route_grad":
        weights, ids, lse, counts, taken, _ = route_forward(s["x"], s["valid"], k, c["normalize"])
        s.update(weights=weights, ids=ids, lse=lse, counts=counts, rows=taken)
        s["grad_weights"] = torch.randn(rows, k, device="cuda", generator=gen)
        s["grad_lse"] = torch.randn(rows, device="cuda", generator=gen) * 1e-3
        s["grad_balance"] = rand(gen, 1)[0] * rows * 0.01 if c["balance"] else None  # sums over rows, not means
    return s


def work(c):
    if c["op"] == "select":
        live = c["items"] * (c["begun"] or c["beams"]) * (1.0 - c["ended"])
        return {"bytes": live * c["cols"] * ES[c["dtype"]] + c["items"] * (c["beams"] * 9 + c["count"] * 20),
                "flops": live * c["cols"] * 4}
    if c["op"] == "reorder":
        # about half of the beams move; each distinct parent of theirs is read, each of them written
        beams = c["beams"]
        moved = sum(0.58 * (1.0 - math.sqrt((j + 1) / beams) + math.sqrt(j / beams)) for j in range(beams))
        read = sum(1.0 - (1.0 - 0.58 * (math.sqrt((j + 1) / beams) - math.sqrt(j / beams))) ** (beams - 1)
                   for j in range(beams))
        row = c["heads"] * c["positions"] * c["width"] * ES[c["dtype"]] * (0.5 if c["ragged"] else 1.0)
        return {"bytes": c["items"] * (c["caches"] * row * (moved + read) + 8 * beams + 8), "flops": 0}
    rows, experts, k, es = c["rows"], c["experts"], c["k"], ES[c["dtype"]]
    live = rows * (1.0 - c["padded"])
    if c["op"] == "route":
        return {"bytes": live * experts * es + rows * (12 * k + 4 + (1 if c["padded"] else 0)) + 8 * experts,
                "flops": live * experts * (4 + k)}
    return {"bytes": (live + rows) * experts * es + rows * (16 * k + 8 + (1 if c["padded"] else 0)) + 8 * experts,
            "flops": live * experts * 8}


# ---------------------------------------------------------------------------------------------
# the framework's kernels
# ---------------------------------------------------------------------------------------------
def run(s):
    if not own:
        return plain(s)
    import row_wise_arg_gb300 as A
    c = s["case"]
    if c["op"] == "select":
        r = A.beam_select(s["x"], s["scores"], c["count"], ended=s["ended"], end_token=END, scale=s["scale"],
                          temperature=c["temp"])
        return {"tokens": r.tokens, "parents": r.parents, "scores": r.scores}
    if c["op"] == "reorder":
        return A.beam_reorder(s["caches"], s["parents"], s["lengths"], dim=2)
    if c["op"] == "route":
        r = A.route_topk(s["x"], c["k"], valid=s["valid"], normalize=c["normalize"], counts=True,
                         balance=c["balance"])
        return route_out(c, r.weights, r.ids, r.lse, r.counts, r.rows, r.balance)
    return {"grad": A.route_topk_backward(s["x"], s["weights"], s["ids"], s["lse"], s["counts"], s["rows"],
                                          grad_weights=s["grad_weights"], grad_lse=s["grad_lse"],
                                          grad_balance=s["grad_balance"], normalize=c["normalize"])}


def route_out(c, weights, ids, lse, counts, rows, balance):
    out = {"weights": weights, "ids": ids, "lse": lse, "counts": counts, "rows": rows}
    return dict(out, balance=balance) if c["balance"] else out


# ---------------------------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------------------------
def plain(s):
    c = s["case"]
    if c["op"] == "select":
        return plain_select(s)
    if c["op"] == "reorder":
        return [plain_reorder(s, cache) for cache in s["caches"]]
    if c["op"] == "route":
        return route_out(c, *route_forward(s["x"], s["valid"], c["k"], c["normalize"]))
    return {"grad": plain_route_grad(s)}


def plain_select(s):
    c, x, scores = s["case"], s["x"], s["scores"].double()
    k = min(c["count"], c["cols"])
    z = (x.double() - x.amax(-1, keepdim=True).double()) / c["temp"]
    best = torch.sort(x, dim=-1, descending=True, stable=True)[1][..., :k]
    total = scores[..., None] + (z.gather(-1, best) - z.exp().sum(-1, keepdim=True).log())
    total = torch.where(scores[..., None] > -math.inf, total, -math.inf)
    if s["ended"] is not None:
        first = torch.where(torch.arange(k, device=x.device) == 0, scores[..., None], -math.inf)
        total = torch.where(s["ended"][..., None], first, total)
        best = torch.where(s["ended"][..., None], END, best)
    ranks = total if s["scale"] is None else total * s["scale"].double()[..., None]
    order = torch.sort(ranks.flatten(1), dim=-1, descending=True, stable=True)[1][:, : c["count"]]
    total = total.flatten(1).gather(1, order)
    left = total > -math.inf
    return {"tokens": torch.where(left, best.flatten(1).gather(1, order), -1),
            "parents": torch.where(left, order // k, -1), "scores": total.float()}


def plain_reorder(s, cache):
    c, parents, lengths = s["case"], s["parents"], s["lengths"]
    beams = torch.arange(c["items"] * c["beams"], device=cache.device)
    source = torch.where(parents.flatten() >= 0, beams // c["beams"] * c["beams"] + parents.flatten(), beams)
    new = cache[source]
    if lengths is not None:
        at = torch.arange(c["positions"], device=cache.device)
        live = at < lengths[beams // c["beams"]][:, None]
        new = torch.where(live[:, None, :, None], new, cache)
    return cache.copy_(new)


def softmax_of(x, valid):
    """(x in 32 bits, -inf where a row is padding; which rows take part; softmax, 0 elsewhere; lse)."""
    x = x.float()
    if valid is not None:
        x = torch.where(valid[:, None], x, -math.inf)
    m = x.amax(-1)
    live = m > -math.inf
    e = (x - torch.where(live, m, 0.0)[:, None]).exp()
    total = e.sum(-1)
    return x, live, e / torch.where(live, total, 1.0)[:, None], torch.where(live, m + total.log(), -math.inf)


def route_forward(x, valid, k, normalize):
    experts = x.shape[1]
    x, live, p, lse = softmax_of(x, valid)
    best = torch.sort(x, dim=-1, descending=True, stable=True)[1][:, :k]
    chosen = x.gather(1, best) > -math.inf
    weights = torch.where(chosen, p.gather(1, best), 0.0)
    if normalize:
        e = torch.where(chosen, (x.gather(1, best) - x.gather(1, best[:, :1])).exp(), 0.0)
        weights = e / torch.where(live, e.sum(-1), 1.0)[:, None]
    ids = torch.where(chosen, best, -1)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=x.device)
    counts.index_add_(0, torch.where(chosen, best, experts).flatten(), torch.ones_like(ids).flatten())
    counts, rows = counts[:-1], live.sum()
    share = p.sum(0, dtype=torch.float64) / rows.clamp(min=1)
    balance = experts * (counts.double() / (k * rows.clamp(min=1)) * share).sum()
    return weights, ids, lse, counts, rows, balance.float()


def plain_route_grad(s):
    c, ids, w, g = s["case"], s["ids"], s["weights"], s["grad_weights"]
    live = s["lse"] > -math.inf
    p = torch.where(live[:, None], (s["x"].float() - s["lse"][:, None]).exp(), 0.0)
    along = (g * w).sum(-1)  # the chosen weights' part that every expert has
    rest = s["grad_lse"] if c["normalize"] else s["grad_lse"] - along
    grad = p * rest[:, None]
    if s["grad_balance"] is not None:
        rows = s["rows"].clamp(min=1).double()
        pull = (s["grad_balance"].double() * c["experts"] * s["counts"] / (c["k"] * rows * rows)).float()
        grad = grad + p * (pull - (p * pull).sum(-1, keepdim=True))
    at_ids = w * (g - along[:, None] if c["normalize"] else g)
    grad.scatter_add_(1, ids.clamp(min=0), torch.where(ids >= 0, at_ids, 0.0))
    return torch.where(live[:, None], grad, 0.0).to(s["x"].dtype)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "reorder":  # nothing is computed: the values themselves, beam by beam
        return [exact_cache(c, s, cache) for cache in s["caches"]]
    if c["op"] == "select":
        parts = [exact_item(c, s, i) for i in range(c["items"])]
        return {n: torch.stack([p[n] for p in parts]) for n in parts[0]}
    return exact_route(c, s) if c["op"] == "route" else exact_route_grad(c, s)


def exact_cache(c, s, cache):
    new = cache.clone()
    parents = s["parents"].tolist()
    lengths = [c["positions"]] * c["items"] if s["lengths"] is None else s["lengths"].tolist()
    for i, (row, n) in enumerate(zip(parents, lengths)):
        for j, parent in enumerate(row):
            if parent >= 0:
                new[i * c["beams"] + j, :, :n] = cache[i * c["beams"] + parent, :, :n]
    return new


def exact_item(c, s, i):
    """One item: the best continuation that is left, `count` times."""
    beams, cols = c["beams"], c["cols"]
    totals = torch.full((beams, cols), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(beams):
        if s["scores"][i, b] == -math.inf:
            continue
        if s["ended"] is not None and s["ended"][i, b]:
            totals[b, END] = s["scores"][i, b].double()
        else:
            totals[b] = s["scores"][i, b].double() + torch.log_softmax(s["x"][i, b].double() / c["temp"], 0)
    weight = torch.ones(beams, dtype=torch.float64, device="cuda") if s["scale"] is None else s["scale"][i].double()
    left = (totals * weight[:, None]).flatten()
    place = torch.arange(beams * cols, device="cuda")
    found = []
    for _ in range(c["count"]):
        best = left.amax()
        at = torch.where(left == best, place, beams * cols).amin()
        found.append(torch.where(best > -math.inf, at, -1))
        left[at] = -math.inf
    at = torch.stack(found)
    scores = torch.where(at >= 0, totals.flatten()[at.clamp(min=0)], -math.inf)
    return {"tokens": torch.where(at >= 0, at % cols, -1), "parents": torch.where(at >= 0, at // cols, -1), "scores": scores}


def exact_rows(s):
    """(rows that take part, their indices, their logits)."""
    x = s["x"].double()
    ok = torch.isfinite(x).any(-1) if s["valid"] is None else s["valid"] & (x > -math.inf).any(-1)
    at = ok.nonzero()[:, 0]
    return ok, at, x[at]


def exact_route(c, s):
    rows, experts, k = c["rows"], c["experts"], c["k"]
    ok, at, x = exact_rows(s)
    p = torch.softmax(x, -1)
    left, order = x.clone(), torch.arange(experts, device=x.device)
    ids = torch.full((rows, k), -1, device=x.device)
    weights = torch.zeros(rows, k, dtype=torch.float64, device=x.device)
    for j in range(k):
        best = left.amax(-1, keepdim=True)
        first = torch.where(left == best, order, experts).amin(-1)
        first = torch.where(best[:, 0] > -math.inf, first, -1)
        ids[at, j] = first
        weights[at, j] = torch.where(first >= 0, p.gather(1, first.clamp(min=0)[:, None])[:, 0], 0.0)
        left.scatter_(1, first.clamp(min=0)[:, None], -math.inf)
    if c["normalize"]:
        weights = weights / weights.sum(-1, keepdim=True).clamp(min=1e-300)
    lse = torch.full((rows,), -math.inf, dtype=torch.float64, device=x.device)
    lse[at] = torch.logsumexp(x, -1)
    counts = torch.bincount(ids[ids >= 0], minlength=experts)
    n = max(len(at), 1)
    balance = experts * torch.dot(counts.double() / (k * n), p.sum(0) / n)
    return route_out(c, weights, ids, lse, counts, ok.sum(), balance)


def exact_route_grad(c, s):
    """As automatic differentiation in 64 bits gives it, the choice and the counts held fixed."""
    ok, at, x = exact_rows(s)
    x = x.requires_grad_()
    p = torch.softmax(x, -1)
    ids = s["ids"][at]
    chosen = torch.where(ids >= 0, p.gather(1, ids.clamp(min=0)), 0.0)
    if c["normalize"]:
        chosen = chosen / chosen.sum(-1, keepdim=True)
    goal = (s["grad_weights"].double()[at] * chosen).sum() + (s["grad_lse"].double()[at] * torch.logsumexp(x, -1)).sum()
    if s["grad_balance"] is not None:
        n = max(len(at), 1)
        f = s["counts"].double() / (c["k"] * n)
        goal = goal + s["grad_balance"].double() * c["experts"] * torch.dot(f, p.sum(0) / n)
    goal.backward()
    grad = torch.zeros(s["x"].shape, dtype=torch.float64, device=x.device)
    grad[at] = x.grad
    return {"grad": grad}
