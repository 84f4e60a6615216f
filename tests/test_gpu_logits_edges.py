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
