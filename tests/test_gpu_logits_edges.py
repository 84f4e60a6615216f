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
                      step_plan=step_plan(cluster, min(block, 256), grid))
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
