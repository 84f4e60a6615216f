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
from test_gpu_logits import (DT, check_distill, check_logprobs, forward_plan, grad_plan, slots_for, step_plan,  # noqa: E402
                             stream_plan)


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
