"""Cases of the vocabulary-row operators: log probabilities of given tokens with entropy and top
alternatives, the distillation loss from a teacher's top logits, and the gradients of both.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded once at
the end) or, where ``own`` is true, through the framework's kernels. ``exact`` is the definition in
64 bits, written apart from the plain form.

With z = x / T, lse = log sum_j exp(z_j) and p = exp(z - lse), for each row x of the logits:

* logprobs: log p_t of the row's token t (0 where t < 0, a position without one), the entropy
  -sum_j p_j log p_j, lse, and the k largest logits' indices (ties to the lowest) with their log p.
  A row of -inf alone has lse = -inf, log p = -inf, entropy 0.
* logprobs_grad: the gradient of sum(g * log p_t) + sum(h * entropy) with respect to x.
* distill: sum_i q_i (log q_i - log p_{id_i}) over the row's slots, those with id < 0 left out.
  tail false: q is the softmax of the teacher's logits / T over the slots. tail true: q_i =
  exp(teacher_i), log probabilities, and what is left of 1 is one more outcome, held against the
  student's probability of every index that no slot names.
* distill_grad: the gradient of sum(g * loss) with respect to x.
* distill_step: the loss and that gradient.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one sequence being decoded, its token's log probability with five alternatives: latency alone
        case("answer_one", "logprobs", 1, 32000, "f32", k=5),
        # a sampler's batch with the twenty alternatives that a client may ask for
        case("answer_batch", "logprobs", 32, 202048, "bf16", k=20, temp=0.7),
        # answers held to a grammar: nearly every logit is -inf, in some rows all but a few, and
        # the vocabulary's size is odd, so that rows start at any address
        case("answer_grammar", "logprobs", 9, 100003, "f16", k=20, allowed=0.001),
        # scoring given text: no alternatives but the best, an odd vocabulary
        case("score_text", "logprobs", 1500, 65537, "f32", k=1),
        # the teacher's pass over a training batch: its top 64 are what a student is taught from
        case("teacher_pass", "logprobs", 2048, 202048, "bf16", k=64),
        # policy gradient on a few short answers, an odd vocabulary
        case("policy_small", "logprobs_grad", 48, 32001, "f32", ignored=0.1),
        # policy gradient with an entropy bonus on a full batch, padded positions among it
        case("policy_batch", "logprobs_grad", 2048, 202048, "bf16", ignored=0.1),
        # evaluating a student on a handful of positions
        case("distill_few", "distill", 4, 32000, "f32", k=16, temp=2.0),
        # evaluating a student against log probabilities kept for the likeliest 32, fewer in some rows
        case("distill_eval", "distill", 512, 100003, "f16", k=32, tail=True, ignored=0.25),
        # the gradient alone, as automatic differentiation asks for it
        case("distill_backward", "distill_grad", 1024, 262144, "bf16", k=64, temp=2.0),
        # a training step of the student: the loss and its gradient
        case("distill_train", "distill_step", 1024, 202048, "bf16", k=64, tail=True),
        # the same in 32 bits, an odd vocabulary cut from padded rows, many slots, some of them empty
        case("distill_train_odd", "distill_step", 333, 50021, "f32", k=100, pad=43, ignored=0.25),
    ]


def case(name, op, rows, cols, dtype, k=0, temp=1.0, tail=False, allowed=1.0, ignored=0.0, pad=0):
    """allowed: share of the logits that are not -inf; ignored: share of the positions without a
    token (of the slots without an id); pad: elements between the end of a row and the next."""
    c = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "k": k, "temp": temp, "tail": tail,
         "allowed": allowed, "ignored": ignored, "pad": pad}
    return dict(c, name=name) if name else c


def draw(rng):
    """Rows from 1 to 2048, vocabularies from 1000 to 262144, every direction, type and option."""
    op = rng.choice(["logprobs", "logprobs", "logprobs_grad", "distill", "distill_grad", "distill_step"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    cols = int(round(math.exp(rng.uniform(math.log(1000), math.log(262144)))))
    most = min(2048, 2048 * 202048 * 2 // (cols * ES[dtype]))
    rows = int(round(math.exp(rng.uniform(0.0, math.log(most)))))
    if op.startswith("logprobs"):
        k = 0 if op == "logprobs_grad" else int(round(math.exp(rng.uniform(0.0, math.log(65))))) - 1
    else:
        k = int(round(math.exp(rng.uniform(0.0, math.log(128)))))
    return case(None, op, rows, cols, dtype, k=k, temp=rng.choice([1.0, 1.0, 0.7, 2.0]),
                tail=op.startswith("distill") and rng.random() < 0.5,
                allowed=0.002 if op == "logprobs" and rng.random() < 0.2 else 1.0,
                ignored=rng.choice([0.0, 0.1, 0.25]), pad=rng.choice([0, 0, rng.randint(1, 128)]))


def prepare(c, seed):
    rows, cols, k, temp = c["rows"], c["cols"], c["k"], c["temp"]
    gen = torch.Generator("cuda").manual_seed(seed)
    store = torch.empty(rows, cols + c["pad"], device="cuda")
    store.normal_(0.0, 3.0, generator=gen)
    if c["allowed"] < 1.0:
        cut = torch.rand(store.shape, device="cuda", generator=gen) >= c["allowed"]
        cut[0, 3:] = True  # the grammar leaves the first row three tokens at most
        store.masked_fill_(cut, -math.inf)
        store[:, 1] = 0.5  # and every row one
        del cut
    x = store.to(DTYPES[c["dtype"]])[:, :cols]
    s = {"case": c, "x": x}
    if c["op"].startswith("logprobs"):
        noise = torch.rand(rows, cols, device="cuda", generator=gen).clamp_(1e-9, 1.0 - 1e-7)
        s["tokens"] = (x.float() / temp - noise.log_().neg_().log_()).argmax(-1)  # drawn from the softmax
        gone = torch.rand(rows, device="cuda", generator=gen) < c["ignored"]
        s["tokens"] = torch.where(gone, -100, s["tokens"])
        if c["op"] == "logprobs_grad":
            m, logsum, lp = log_softmax(x, temp)
            entropy = -(lp.exp() * lp).sum(-1)
            s["stats"] = torch.stack((m, logsum, entropy, torch.zeros_like(m)), 1)
            s["grad_logprob"] = torch.randn(rows, device="cuda", generator=gen)  # advantages
            s["grad_entropy"] = torch.full((rows,), 0.01, device="cuda")
    else:
        # the teacher agrees with the student up to a disturbance
        y = store[:, :cols] + torch.randn(rows, cols, device="cuda", generator=gen)
        top, s["ids"] = y.topk(min(k, cols), -1)
        s["teacher"] = (top / temp - (y / temp).logsumexp(-1, keepdim=True)) if c["tail"] else top
        s["teacher"] = s["teacher"].contiguous()
        gone = torch.rand(s["ids"].shape, device="cuda", generator=gen) < c["ignored"]
        s["ids"] = torch.where(gone, -1, s["ids"]).contiguous()
        if c["op"] != "distill":
            s["grad_loss"] = torch.rand(rows, device="cuda", generator=gen)
        if c["op"] == "distill_grad":
            m, logsum, lp = log_softmax(x, temp)
            s["stats"] = torch.stack((m, logsum, torch.log(tail_mass(s, lp)) + logsum, torch.zeros_like(m)), 1)
    return s


def work(c):
    rows, cols, k, es = c["rows"], c["cols"], c["k"], ES[c["dtype"]]
    n = rows * cols
    per_row = {"logprobs": 8 + 12 + 12 * k, "logprobs_grad": 8 + 16 + 8, "distill": 12 * k + 4,
               "distill_grad": 12 * k + 16 + 4, "distill_step": 12 * k + 4 + 4}[c["op"]]
    passes = 1 if c["op"] in ("logprobs", "distill") else 2
    # a subtraction, a scaling, an exponential and the sums (or the products with the gradients)
    return {"bytes": passes * n * es + rows * per_row, "flops": n * (8 if c["op"] == "distill_step" else 5)}


# ---------------------------------------------------------------------------------------------
# the framework's kernels
# ---------------------------------------------------------------------------------------------
def run(s):
    if not own:
        return plain(s)
    import row_wise_arg_gb300 as A
    c, x = s["case"], s["x"]
    if c["op"] == "logprobs":
        r = A.token_logprobs(x, s["tokens"], c["k"], temperature=c["temp"])
        return logprobs_out(c, r.logprob, r.entropy, r.lse, r.top_ids, r.top_logprobs)
    if c["op"] == "logprobs_grad":
        return {"grad": A.token_logprobs_backward(x, s["tokens"], s["stats"], s["grad_logprob"], s["grad_entropy"],
                                                  temperature=c["temp"])}
    if c["op"] == "distill":
        return {"loss": A.distill_topk(x, s["ids"], s["teacher"], temperature=c["temp"], tail=c["tail"]).loss}
    if c["op"] == "distill_grad":
        return {"grad": A.distill_topk_backward(x, s["ids"], s["teacher"], s["stats"], s["grad_loss"],
                                                temperature=c["temp"], tail=c["tail"])}
    loss, grad = A.distill_topk_step(x, s["ids"], s["teacher"], s["grad_loss"], temperature=c["temp"], tail=c["tail"])
    return {"loss": loss, "grad": grad}


def logprobs_out(c, logprob, entropy, lse, top_ids, top_logprobs):
    out = {"logprob": logprob, "entropy": entropy, "lse": lse}
    return dict(out, top_ids=top_ids, top_logprobs=top_logprobs) if c["k"] else out


# ---------------------------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------------------------
def log_softmax(x, temp):
    """Row maxima of x, log sum exp((x - max) / T), and log p."""
    x = x.float()
    m = x.amax(-1)
    d = (x - torch.where(torch.isinf(m), 0.0, m)[:, None]) / temp
    logsum = d.exp().sum(-1).log()
    return m, logsum, torch.where(torch.isinf(m)[:, None], -math.inf, d - logsum[:, None])


def present(s):
    """For each slot whether it names an index, and the index (0 where it names none)."""
    return s["ids"] >= 0, s["ids"].clamp(min=0)


def in_slots(s):
    """For each index of each row whether a slot names it."""
    here, at = present(s)
    named = torch.zeros(s["x"].shape, dtype=torch.int32, device=at.device)
    return named.scatter_add_(1, at, here.int()) > 0


def tail_mass(s, lp):
    """The student's probability of every index that no slot names."""
    return torch.where(in_slots(s), 0.0, lp.exp()).sum(-1)


def teacher_probs(s):
    """The slots' q and log q (0 and 0 where a slot is empty), and what is left of 1."""
    c, (here, _) = s["case"], present(s)
    logq = s["teacher"]
    if not c["tail"]:
        u = torch.where(here, logq / c["temp"], -math.inf)
        top = u.amax(-1, keepdim=True).clamp(min=-3e38)
        logq = u - top - (u - top).exp().sum(-1, keepdim=True).log()
    q = torch.where(here, logq.exp(), 0.0)
    rest = (1.0 - q.sum(-1)).clamp(min=0.0) if c["tail"] else torch.zeros_like(q[:, 0])
    return q, torch.where(q > 0, logq, 0.0), torch.where(here.any(-1), rest, 0.0)


def plain_loss(s, lp):
    here, at = present(s)
    q, logq, rest = teacher_probs(s)
    loss = torch.where(q > 0, q * (logq - lp.gather(1, at)), 0.0).sum(-1)
    if s["case"]["tail"]:
        mass = tail_mass(s, lp)
        loss = loss + torch.where((rest > 0) & (mass > 0), rest * (rest.log() - mass.log()), 0.0)
    return loss


def plain_distill_grad(s, lp, mass):
    """g / T * (total * p - q over the slots - rest * p / mass over the other indices)."""
    c, x = s["case"], s["x"]
    here, at = present(s)
    q, _, rest = teacher_probs(s)
    p = lp.exp()
    rest = torch.where(mass > 0, rest, 0.0)
    share = torch.where(rest > 0, rest / mass, 0.0)
    grad = p * ((q.sum(-1) + rest)[:, None] - torch.where(in_slots(s), 0.0, share[:, None]))
    grad.scatter_add_(1, at, -q)
    return (grad * (s["grad_loss"] / c["temp"])[:, None]).to(x.dtype)


def from_stats(s):
    """log p from the row's saved maximum and log sum."""
    x, temp = s["x"].float(), s["case"]["temp"]
    return (x - s["stats"][:, 0:1]) / temp - s["stats"][:, 1:2]


def plain(s):
    c, x = s["case"], s["x"]
    if c["op"] == "logprobs":
        m, logsum, lp = log_softmax(x, c["temp"])
        entropy = -torch.where(lp > -math.inf, lp.exp() * lp, 0.0).sum(-1)
        tokens = s["tokens"]
        logprob = torch.where(tokens < 0, 0.0, lp.gather(1, tokens.clamp(min=0)[:, None])[:, 0])
        top_ids = torch.sort(x, dim=-1, descending=True, stable=True)[1][:, : c["k"]] if c["k"] else None
        top = lp.gather(1, top_ids) if c["k"] else None
        return logprobs_out(c, logprob, entropy, m / c["temp"] + logsum, top_ids, top)
    if c["op"] == "logprobs_grad":
        lp, tokens = from_stats(s), s["tokens"]
        g, h = torch.where(tokens < 0, 0.0, s["grad_logprob"]), s["grad_entropy"]
        grad = -lp.exp() * (g[:, None] + h[:, None] * (lp + s["stats"][:, 2:3]))
        grad.scatter_add_(1, tokens.clamp(min=0)[:, None], g[:, None])
        return {"grad": (grad / c["temp"]).to(x.dtype)}
    if c["op"] == "distill_grad":
        mass = torch.exp(s["stats"][:, 2] - s["stats"][:, 1])
        return {"grad": plain_distill_grad(s, from_stats(s), mass)}
    _, _, lp = log_softmax(x, c["temp"])
    if c["op"] == "distill":
        return {"loss": plain_loss(s, lp)}
    return {"loss": plain_loss(s, lp), "grad": plain_distill_grad(s, lp, tail_mass(s, lp) if c["tail"] else plain_ones(x))}


def plain_ones(x):
    return torch.ones(x.shape[0], device=x.device)


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits, some rows at a time
# ---------------------------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    at_once = max(1, (1 << 26) // c["cols"])
    parts = [exact_rows(c, {n: v[r:r + at_once] for n, v in s.items() if n != "case"})
             for r in range(0, c["rows"], at_once)]
    return {n: torch.cat([p[n] for p in parts]) for n in parts[0]}


def exact_rows(c, s):
    z = s["x"].double() / c["temp"]
    lse = torch.logsumexp(z, -1)
    rows = torch.arange(len(z), device=z.device)
    if c["op"] == "logprobs":
        logp = z - lse[:, None]
        p = logp.exp()
        out = {"entropy": -torch.xlogy(p, p).sum(-1), "lse": lse,
               "logprob": torch.where(s["tokens"] >= 0, logp[rows, s["tokens"]], 0.0)}
        left, ids = z.clone(), []
        order = torch.arange(c["cols"], device=z.device)
        taken = torch.zeros_like(z, dtype=torch.bool)
        for _ in range(c["k"]):  # the largest that is left, the first of equals
            best = left.amax(-1, keepdim=True)
            first = torch.where((left == best) & ~taken, order, c["cols"]).amin(-1)
            ids.append(first)
            left[rows, first] = -math.inf
            taken[rows, first] = True
        if c["k"]:
            out["top_ids"] = torch.stack(ids, 1)
            out["top_logprobs"] = logp.gather(1, out["top_ids"])
        return out
    if c["op"] == "logprobs_grad":
        m, logsum, entropy = (s["stats"][:, i].double()[:, None] for i in range(3))
        logp = (s["x"].double() - m) / c["temp"] - logsum
        g = torch.where(s["tokens"] >= 0, s["grad_logprob"].double(), 0.0)
        chosen = torch.zeros_like(z)
        chosen[rows, s["tokens"].clamp(min=0)] = 1.0
        p = logp.exp()
        grad = g[:, None] * (chosen - p) - s["grad_entropy"].double()[:, None] * p * (logp + entropy)
        return {"grad": grad / c["temp"]}
    # each row's slots spread over the vocabulary
    here = s["ids"] >= 0
    teacher = s["teacher"].double()
    q = teacher.exp() if c["tail"] else torch.softmax(torch.where(here, teacher / c["temp"], -math.inf), -1)
    q = torch.where(here, q, 0.0)
    slot_of = torch.where(here, s["ids"], c["cols"])  # empty slots go to a column of their own
    wide = torch.zeros(len(z), c["cols"] + 1, dtype=torch.float64, device=z.device).scatter_(1, slot_of, q)[:, :-1]
    other = torch.ones(len(z), c["cols"] + 1, device=z.device).scatter_(1, slot_of, 0.0)[:, :-1] > 0
    logp = z - lse[:, None]
    if c["op"] == "distill_grad":
        logp = (s["x"].double() - s["stats"][:, 0:1].double()) / c["temp"] - s["stats"][:, 1:2].double()
    p = logp.exp()
    rest = (1.0 - q.sum(-1)).clamp(min=0.0) if c["tail"] else torch.zeros_like(lse)
    rest = torch.where(here.any(-1), rest, 0.0)
    mass = torch.where(other, p, 0.0).sum(-1)
    if c["op"] == "distill_grad":
        mass = (s["stats"][:, 2].double() - s["stats"][:, 1].double()).exp()
    rest = torch.where(mass > 0, rest, 0.0)
    out = {}
    if c["op"] != "distill_grad":
        kept = torch.where(rest > 0, rest * (rest / mass).log(), 0.0)
        out["loss"] = torch.xlogy(q, q).sum(-1) - torch.where(wide > 0, wide * logp, 0.0).sum(-1) + kept
    if c["op"] != "distill":
        share = torch.where(rest > 0, rest / mass, 0.0)
        grad = (wide.sum(-1) + rest)[:, None] * p - wide - torch.where(other, share[:, None] * p, 0.0)
        out["grad"] = grad * (s["grad_loss"].double() / c["temp"])[:, None]
    return out
