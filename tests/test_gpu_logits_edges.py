"""Vocabulary-row operators on the GPU where their inner workings meet: hand-overs between warps, plans
larger than the problem, streams, ranges of numbers, ties across segments, repeated slots. Against the
definitions in 64 bits, with the bounds of logits_ref and the checks of test_gpu_logits."""
import numpy as np
import pytest

import logits_ref as ref

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import row_wise_arg_gb300 as A  # noqa: E402
from test_gpu_logits import (DT, check_distill, check_logprobs, close, forward_plan, grad_plan, slots_for,  # noqa: E402
                             step_plan, stream_plan)


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_wise_arg_gb300.build import build
    build()


@pytest.mark.parametrize("finishers", [1, 2, 3])
def test_many_short_rows_per_persistent_cta(finishers):
    """Rows that end so soon that finishers and streamers meet all the time; 100 and more rows per CTA."""
    rng = np.random.default_rng(finishers)
    for rows, cols, block, grid in ((301, 70, 512, 2), (200, 3, 160, 1), (403, 1000, 256, 4)):
        x = rng.normal(0, 3, (rows, cols)).astype(np.float32)
        plan = stream_plan(finishers, block, grid)
        for k in (0, 3):
            check_logprobs(x, "bf16", rng.integers(-1, cols, rows), k, plan=plan)
        for tail in (False, True):
            ids, val = slots_for(rng, rows, cols, 5, tail, 0.2)
            check_distill(x, "f32", ids, val, 1.0, tail, plan=plan)


@pytest.mark.parametrize("cluster,block,grid", [(1, 128, 700), (4, 64, 40), (2, 512, 9)])
def test_plans_with_more_row_slots_than_rows(cluster, block, grid):
    """CTAs without a row do nothing, a prefetch included: it would be of addresses past the logits."""
    rng = np.random.default_rng(grid)
    x = rng.normal(0, 3, (5, 30011)).astype(np.float32)
    ids, val = slots_for(rng, 5, 30011, 9, True, 0.2)
    for dtype in DT:
        plan = forward_plan(cluster, block, grid, grid)
        check_logprobs(x, dtype, rng.integers(-1, 30011, 5), 7, plan=plan)
        check_distill(x, dtype, ids, val, 1.0, True, plan=plan, grad_plan=grad_plan(3, 128, grid),
                      step_plan=step_plan(max(cluster, 2), min(block, 256), grid))
        check_logprobs(x, dtype, None, 7, plan=stream_plan(2, 512, grid))


def busy():
    """Some milliseconds of work on the current stream."""
    a = torch.full((4096, 4096), 1.0 / 4096, device="cuda")
    for _ in range(20):
        a = a @ a
    return a.sum() * 0.0


def stream_kinds():
    side = torch.cuda.Stream()
    return [side, side.cuda_stream, torch.cuda.ExternalStream(side.cuda_stream)]


def test_gradients_of_calls_on_another_stream():
    """Gradients that are made late reach a backward pass whose forward pass ran on another stream, and its own are used
    at once on this one; the forward pass's tensors are dropped as soon as they can be."""
    g = torch.Generator("cuda").manual_seed(31)
    x = torch.randn(300, 20011, device="cuda", generator=g)
    tok = torch.randint(0, 20011, (300,), device="cuda", generator=g)
    ids = torch.stack([torch.randperm(20011, device="cuda", generator=g)[:8] for _ in range(300)])
    val = torch.log_softmax(torch.randn(300, 9, device="cuda", generator=g), -1)[:, :8].contiguous()
    weights = torch.rand(300, device="cuda", generator=g)

    def as_stream(s):
        return s if not isinstance(s, int) else torch.cuda.ExternalStream(s) if s else torch.cuda.default_stream()

    def pass_(how, stream):
        leaf = x.clone().requires_grad_()
        scaled = leaf * 1.5  # the operator's own input is dropped after the backward pass
        if stream is not None:
            as_stream(stream).wait_stream(torch.cuda.current_stream())
        if how == "logprobs":
            r = A.token_logprobs(scaled, tok, 5, stream=stream)
            parts = (r.logprob, r.entropy, r.lse)
        else:
            parts = (A.distill_topk(scaled, ids, val, tail=True, stream=stream).loss,)
        del scaled
        if stream is not None:
            torch.cuda.current_stream().wait_stream(as_stream(stream))
        late = weights + busy()
        sum((p * late * (i + 1)).sum() for i, p in enumerate(parts)).backward()
        used = leaf.grad * 2.0
        junk = [torch.full((300, 20011), 7.0, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert all((j == 7.0).all() for j in junk)
        return used

    for how in ("logprobs", "distill"):
        want = pass_(how, None)
        assert want.abs().sum() > 0
        for stream in stream_kinds() * 2:
            assert torch.equal(pass_(how, stream), want)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):  # from a side stream to the default one, by its handle
            assert torch.equal(pass_(how, 0), want)


def test_memory_of_calls_on_another_stream():
    """What a call makes for itself, and what it returns and is dropped at once, is not handed out while the other stream
    still writes it."""
    g = torch.Generator("cuda").manual_seed(32)
    x = torch.randn(2000, 3001, device="cuda", generator=g)
    ids = torch.stack([torch.randperm(3001, device="cuda", generator=g)[:4] for _ in range(2000)])
    val = torch.log_softmax(torch.randn(2000, 5, device="cuda", generator=g), -1)[:, :4].contiguous()
    w = torch.rand(2000, device="cuda", generator=g)
    want = A.distill_topk_step(x, ids, val, w, tail=True)
    tok = ids[:, 0].contiguous()
    stats = A.token_logprobs(x, tok, with_stats=True).stats
    torch.cuda.synchronize()
    for stream in stream_kinds():
        s = torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream
        for _ in range(3):
            with torch.cuda.stream(s):
                busy()
            late = w.clone()  # an input that is dropped at once, too
            s.wait_stream(torch.cuda.current_stream())
            got = A.distill_topk_step(x, ids, val, w, tail=True, stream=stream)
            A.token_logprobs(x, tok, 3, with_stats=True, stream=stream)
            A.token_logprobs_backward(x, tok, stats, late, stream=stream)
            del late
            junk = [torch.full((2000, n), 7.0, device="cuda") for n in (1, 2, 3, 4, 3001) for _ in range(4)]
            s.synchronize()
            torch.cuda.synchronize()
            assert all((j == 7.0).all() for j in junk)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---------------------------------------------------------------------------
# Ranges of numbers.
# ---------------------------------------------------------------------------
def tail_in_logs(x, ids, val, temp, g):
    """(loss, gradient, bounds of both) with the tail, in 64 bits, the tail's mass as a logarithm. Every row's slots
    are filled, its tail is neither empty nor masked.

    Bounds: a sum is off by a share of sum_error (logits_ref), an exponential's argument y by 8 |y| u, what is left of 1
    by sum_error itself; ln p_rest multiplies that, and the weight of a tail element is its share of the tail."""
    rows, cols = x.shape
    loss, grad = np.zeros(rows), np.zeros((rows, cols))
    lbound, terms = np.zeros(rows), np.zeros((rows, cols))
    for r in range(rows):
        z = x[r] / temp
        named = np.zeros(cols, bool)
        named[ids[r]] = True
        lse = np.logaddexp.reduce(z)
        lse_rest = np.logaddexp.reduce(z[~named])
        q = np.exp(val[r].astype(np.float64))
        rest = 1.0 - q.sum()
        lp = z - lse
        used = q > 0
        loss[r] = (q[used] * (val[r][used] - lp[ids[r]][used])).sum() + rest * (np.log(rest) - (lse_rest - lse))
        share = np.where(named, 0.0, np.exp(np.minimum(z - lse_rest, 0.0)))
        d = (q.sum() + rest) * np.exp(lp) - rest * share
        np.subtract.at(d, ids[r], q)
        grad[r] = d * g[r] / temp
        far = abs(lse_rest - lse)
        lbound[r] = ref.logprob_bound(loss[r], cols) + ref.sum_error(cols) * (
            2 * np.abs(lp[ids[r]][used]).max() + np.log(len(q)) + 3 + far + abs(np.log(rest)) + 8)
        t = np.exp(lp) * (1 + np.abs(lp)) + share * (1 + np.abs(np.where(named, 0.0, lp)) + far)
        np.add.at(t, ids[r], q * (2 + np.abs(np.where(used, val[r], 0.0))))
        terms[r] = t * abs(g[r]) / temp
    return loss, grad, lbound, terms


TAIL_PLANS = [(forward_plan(1, 128, 2, 2), step_plan(1, 128, 2)), (forward_plan(4, 64, 5, 5), step_plan(4, 64, 3)),
              (stream_plan(1, 128, 2), step_plan(2, 32, 1)), (stream_plan(2, 256, 3), None), (None, None)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("gap,temp", [(20, 1.0), (60, 1.0), (80, 1.0), (84, 1.0), (86, 1.0), (87, 1.0), (88, 1.0),
                                      (90, 1.0), (100, 1.0), (150, 1.0), (700, 1.0), (26, 0.3), (27, 0.3), (200, 0.3),
                                      (300, 3.0)])
def test_a_tail_far_below_the_row(gap, temp, dtype):
    """A student that gives the tail next to nothing is told so: its logarithm is finite however small it is."""
    rng = np.random.default_rng(gap)
    rows, cols, slots = 5, 3001, 64
    x = np.round(rng.normal(-gap, 0.5, (rows, cols)) * 8) / 8
    ids = np.stack([rng.permutation(cols)[:slots] for _ in range(rows)]).astype(np.int64)
    for r in range(rows):
        x[r, ids[r]] = np.round(rng.normal(0, 0.5, slots) * 8) / 8 if r else 0.0
    x[0, np.setdiff1d(np.arange(cols), ids[0])[1:]] -= gap  # a lone element leads the tail
    t = torch.from_numpy(x).to(DT[dtype])
    x64, xd = t.double().numpy(), t.cuda()
    val = np.log(rng.dirichlet(np.full(slots, 2.0), rows) * rng.uniform(0.5, 0.95, (rows, 1))).astype(np.float32)
    g = rng.normal(size=rows).astype(np.float32)
    loss, grad, lbound, terms = tail_in_logs(x64, ids, val, temp, g)
    gbound = ref.grad_bound(grad, terms, cols, dtype)
    i, v, w = (torch.from_numpy(a).cuda() for a in (ids, val, g))
    kw = dict(temperature=temp, tail=True)
    for plan, splan in TAIL_PLANS:
        r = A.distill_topk(xd, i, v, plan=plan, with_stats=True, **kw)
        close(r.loss, loss, lbound, "loss")
        close(A.distill_topk_backward(xd, i, v, r.stats, w, **kw), grad, gbound, "grad")
        both = A.distill_topk_step(xd, i, v, w, plan=splan, **kw)
        close(both[0], loss, lbound, "step's loss")
        close(both[1], grad, gbound, "step's grad")


def test_a_tail_that_is_masked_is_left_out():
    """By -inf, or so low that its probability is 0 in binary64 as well: finite, and as without the term."""
    rng = np.random.default_rng(4)
    ids = np.stack([rng.permutation(3001)[:64] for _ in range(3)]).astype(np.int64)
    val = np.log(rng.dirichlet(np.full(64, 2.0), 3) * 0.9).astype(np.float32)
    for dtype in DT:
        for low in (-np.inf, -1e4, -6e4):
            x = np.full((3, 3001), low)
            for r in range(3):
                x[r, ids[r]] = rng.normal(0, 1, 64)
            for plan, splan in TAIL_PLANS:
                check_distill(x.astype(np.float32), dtype, ids, val, 1.0, True, plan=plan, step_plan=splan)


# ---------------------------------------------------------------------------
# Ties across the segments of a CTA's part (8192 groups of 64 bytes).
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", list(DT))
def test_ties_in_a_later_segment(dtype):
    """Many equal values that come after a segment of smaller ones, with fewer larger ones than alternatives."""
    seg = 8192 * (16 if dtype == "f32" else 32)
    cols = 2 * seg + 777
    for first, later in ((-1.0, 0.0), (-np.inf, -5.0), (-5.0, -5.0), (np.nan, -5.0)):
        x = np.full((2, cols), later, np.float32)
        x[:, :seg + 100] = first
        x[1, seg + 300:] = first  # a few of them only
        x[:, seg + 5000:seg + 5003] = 2.0
        x[:, 70] = 1.0
        x[:, 2 * seg + 500] = 1.0
        for k in (1, 5, 20, 128):
            for plan in (forward_plan(1, 512, 2, 2), forward_plan(1, 64, 2, 2), None):
                check_logprobs(x, dtype, None, k, plan=plan)
    # the planner's own choice of a CTA per row
    rows = 90
    assert A.argreduce_logits_plan("logprobs", rows, cols, dtype, 20, A.make_caps(152)).cluster == 1
    t = torch.full((rows, cols), -1.0, dtype=DT[dtype], device="cuda")
    t[:, seg + 100:] = 0.0
    got = A.token_logprobs(t, None, 20).top_ids
    assert torch.equal(got, torch.arange(seg + 100, seg + 120, device="cuda").expand(rows, 20))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_teacher_logits_of_any_size(dtype):
    """Their softmax does not depend on what they have in common; differences come before the temperature."""
    rng = np.random.default_rng(12)
    rows, cols, slots = 6, 2003, 33
    x = rng.normal(0, 2, (rows, cols)).astype(np.float32)
    ids, val = slots_for(rng, rows, cols, slots, False)
    top = 3.4028234663852886e38
    for shift, temp in ((0.0, 1.0), (1e3, 1.0), (-1e4, 1.0), (1e4, 0.5), (1e6, 0.7)):
        check_distill(x, dtype, ids, (val + np.float32(shift)).astype(np.float32), temp, False)
    low = np.full_like(val, -top)
    high = np.full_like(val, top)
    one = low.copy()
    one[:, 4] = 1.0
    for v in (low, high, one):
        for temp in (0.5, 1.0, 2.0):
            check_distill(x, dtype, ids, v, temp, False)
            check_distill(x, dtype, ids, v, temp, False, plan=stream_plan(1, 128, 2))


def test_forward_mode_is_refused():
    """A tangent would be dropped without a word."""
    import torch.autograd.forward_ad as fwd
    x = torch.randn(3, 50, device="cuda")
    tok = torch.zeros(3, dtype=torch.int64, device="cuda")
    ids, val, one = tok[:, None].contiguous(), torch.zeros(3, 1, device="cuda"), torch.ones(3, device="cuda")
    s = A.token_logprobs(x, tok, with_stats=True).stats
    with fwd.dual_level():
        dual = fwd.make_dual(x, torch.ones_like(x))
        for call in (lambda: A.token_logprobs(dual, tok), lambda: A.token_logprobs_backward(dual, tok, s, one),
                     lambda: A.distill_topk(dual, ids, val), lambda: A.distill_topk_step(dual, ids, val, one),
                     lambda: A.distill_topk_backward(dual, ids, val, s, one)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        A.token_logprobs(x, tok)  # without a tangent all is well


def test_gradients_written_over_tensors_are_seen_by_autograd():
    """A graph that saved logits which a gradient has since overwritten says so; inference tensors have no such count."""
    g = torch.Generator("cuda").manual_seed(7)
    leaf = torch.randn(4, 300, device="cuda", generator=g, requires_grad=True)
    tok = torch.randint(0, 300, (4,), device="cuda", generator=g)
    ids, val, one = tok[:, None].contiguous(), torch.zeros(4, 1, device="cuda"), torch.ones(4, device="cuda")
    for how in ("logprobs", "distill", "step"):
        x = leaf * 2.0
        loss = A.token_logprobs(x, tok).logprob.sum()
        over = x.detach()
        if how == "logprobs":
            A.token_logprobs_backward(over, tok, A.token_logprobs(over, tok, with_stats=True).stats, one, grad=over)
        elif how == "distill":
            s = A.distill_topk(over, ids, val, with_stats=True).stats
            A.distill_topk_backward(over, ids, val, s, one, grad=over)
        else:
            A.distill_topk_step(over, ids, val, one, grad=over)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    with torch.inference_mode():
        x = torch.randn(4, 300, device="cuda", generator=g)
        want = A.distill_topk_step(x, ids, val, one)[1]
        assert torch.equal(A.distill_topk_step(x, ids, val, one, grad=x)[1], want)
