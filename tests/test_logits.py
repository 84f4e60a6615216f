"""Vocabulary-row operators without a GPU: the 64-bit reference's gradients
against differences of its own losses, the refusals of the C entry points, and
the planner."""
import ctypes

import numpy as np
import pytest

import logits_ref as ref
import row_wise_arg_gb300 as A
from row_wise_arg_gb300 import _lib
from row_wise_arg_gb300.build import build

CAPS = A.make_caps(152)
X = 0x10000  # a fake, never dereferenced address, 16-byte aligned


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def differences(f, x, step=1e-5):
    d = np.zeros_like(x)
    for at in np.ndindex(x.shape):
        hi, lo = x.copy(), x.copy()
        hi[at] += step
        lo[at] -= step
        d[at] = (f(hi) - f(lo)) / (2 * step)
    return d


@pytest.mark.parametrize("temp", [1.0, 0.7, 3.0])
def test_reference_logprob_gradient_against_differences(temp):
    rng = np.random.default_rng(1)
    x = rng.normal(0, 2, (3, 9))
    tokens = np.array([4, -1, 8])
    g, h, c = rng.normal(size=(3, 3))

    def f(v):
        o = ref.logprobs(v, tokens, 0, temp)
        return (g * o["logprob"] + h * o["entropy"] + c * o["lse"]).sum()
    np.testing.assert_allclose(ref.logprobs_grad(x, tokens, g, h, c, temp), differences(f, x), atol=1e-8)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("temp", [1.0, 2.5])
def test_reference_distill_gradient_against_differences(temp, tail):
    rng = np.random.default_rng(2)
    x = rng.normal(0, 2, (4, 11))
    ids = np.stack([rng.permutation(11)[:4] for _ in range(4)])
    ids[1, 2] = -1
    ids[2] = -1
    val = np.log(rng.dirichlet(np.ones(5), 4)[:, :4]) if tail else rng.normal(0, 2, (4, 4))
    g = rng.normal(size=4)
    _, grad = ref.distill(x, ids, val, temp, tail, g)
    np.testing.assert_allclose(grad, differences(lambda v: (g * ref.distill(v, ids, val, temp, tail)[0]).sum(), x),
                               atol=1e-8)
    assert (grad[2] == 0).all()


def codes(f, good, bad):
    """Each entry of `bad` changes some arguments of the call `good` and names the status it must give."""
    for change, want in bad:
        args = dict(good, **change)
        assert f(*args.values()) == want, change


def test_logprobs_refusals_before_any_device_work():
    lib = _lib.load()
    good = dict(x=X, dtype=0, rows=3, cols=100, stride=100, temp=1.0, tokens=X, k=5, logprob=X, entropy=X, lse=X,
                ids=X, top=X, stats=X, plan=None, stream=None)
    inval, unsup, ok = _lib.ARGR_EINVAL, _lib.ARGR_EUNSUPPORTED, _lib.ARGR_OK
    codes(lib.argreduce_logprobs, good, [
        ({"rows": 0}, ok), ({"rows": 0, "x": None}, ok), ({"rows": -1}, inval), ({"x": None}, inval),
        ({"x": X + 2}, inval), ({"dtype": 1, "x": X + 1}, inval), ({"cols": 0}, inval), ({"cols": 2 ** 31}, inval),
        ({"stride": -1}, inval), ({"stride": 2 ** 62}, inval), ({"rows": 2 ** 62}, inval),
        ({"temp": 0.0}, inval), ({"temp": -1.0}, inval), ({"temp": float("inf")}, inval),
        ({"temp": float("nan")}, inval), ({"temp": 1e-40}, inval),
        ({"dtype": _lib.ARGR_F64}, unsup), ({"dtype": _lib.ARGR_I32}, unsup), ({"dtype": _lib.ARGR_I64}, unsup),
        ({"dtype": 17}, inval), ({"k": -1}, inval), ({"k": 129}, inval), ({"k": 101}, inval),
        ({"tokens": None}, inval), ({"tokens": X + 4}, inval), ({"logprob": X + 2}, inval), ({"stats": X + 8}, inval),
        ({"ids": X + 4}, inval), ({"top": X + 1}, inval), ({"entropy": X + 1}, inval), ({"lse": X + 1}, inval)])


def test_logprobs_backward_refusals():
    lib = _lib.load()
    inval = _lib.ARGR_EINVAL
    far = X + (1 << 30)
    good = dict(x=X, dtype=0, rows=3, cols=100, stride=100, temp=1.0, tokens=X, stats=X, g=X, h=X, c=X, grad=far,
                gstride=100, plan=None, stream=None)
    codes(lib.argreduce_logprobs_backward, good, [
        ({"rows": 0}, _lib.ARGR_OK), ({"stats": None}, inval), ({"tokens": None}, inval), ({"grad": None}, inval),
        ({"grad": far + 2}, inval), ({"gstride": 99}, inval), ({"gstride": -100}, inval), ({"stats": X + 4}, inval),
        ({"g": X + 2}, inval), ({"h": X + 2}, inval), ({"c": X + 2}, inval),
        # the gradient may be x itself, but not overlap it otherwise
        ({"grad": X + 4}, inval), ({"grad": X, "gstride": 101}, inval), ({"grad": X + 4 * 299}, inval),
        ({"grad": X, "stride": 0}, inval),
        ({"dtype": _lib.ARGR_F64}, _lib.ARGR_EUNSUPPORTED)])


def test_distill_refusals():
    lib = _lib.load()
    inval, ok = _lib.ARGR_EINVAL, _lib.ARGR_OK
    far = X + (1 << 30)
    good = dict(x=X, dtype=2, rows=3, cols=100, stride=100, temp=1.0, ids=X, val=X, slots=8, tail=1, loss=X, stats=X,
                plan=None, stream=None)
    codes(lib.argreduce_distill, good, [
        ({"rows": 0}, ok), ({"slots": -1}, inval), ({"slots": 1025}, inval), ({"ids": None}, inval),
        ({"val": None}, inval), ({"ids": X + 4}, inval), ({"val": X + 2}, inval), ({"loss": X + 2}, inval),
        ({"stats": X + 4}, inval), ({"x": X + 1}, inval), ({"temp": 0.0}, inval)])
    good = dict(x=X, dtype=2, rows=3, cols=100, stride=100, temp=1.0, ids=X, val=X, slots=8, tail=1, stats=X, g=X,
                grad=far, gstride=100, plan=None, stream=None)
    codes(lib.argreduce_distill_backward, good, [
        ({"rows": 0}, ok), ({"stats": None}, inval), ({"g": None}, inval), ({"grad": None}, inval),
        ({"grad": far + 1}, inval), ({"grad": X + 2}, inval), ({"gstride": 10}, inval), ({"slots": 2000}, inval)])
    good = dict(x=X, dtype=2, rows=3, cols=100, stride=100, temp=1.0, ids=X, val=X, slots=8, tail=1, g=X, loss=X,
                stats=X, grad=far, gstride=100, plan=None, stream=None)
    codes(lib.argreduce_distill_step, good, [
        ({"rows": 0}, ok), ({"stats": None}, inval), ({"g": None}, inval), ({"grad": None}, inval),
        ({"grad": X + 2}, inval), ({"ids": None}, inval), ({"loss": X + 2}, inval)])


OPS = ["logprobs", "logprobs_backward", "distill", "distill_backward", "distill_step"]


@pytest.mark.parametrize("what", OPS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_plans_hold_for_every_shape(what, dtype):
    for sms in (1, 16, 148, 152):
        for rows in (1, 2, 31, 152, 1000, 65536, 2 ** 40):
            for cols in (1, 31, 1000, 32001, 202048, 10 ** 7, 2 ** 31 - 1):
                for k in (0, 1, 20, 128):
                    p = A.argreduce_logits_plan(what, rows, cols, dtype, k, A.make_caps(sms))
                    assert p.block % 32 == 0 and 32 <= p.block <= 1024
                    assert 1 <= p.cluster <= 16 and p.grid_rows >= 1


def test_plan_refusals():
    for bad in (dict(what=7), dict(cols=0), dict(cols=2 ** 31), dict(rows=-1), dict(k=-1), dict(k=5000)):
        args = dict(what=0, rows=3, cols=100, dtype="f32", k=0)
        args.update(bad)
        with pytest.raises(A.ArgreduceError):
            A.argreduce_logits_plan(args["what"], args["rows"], args["cols"], args["dtype"], args["k"], CAPS)
    with pytest.raises(A.ArgreduceError) as e:
        A.argreduce_logits_plan("logprobs", 3, 100, "f64", 0, CAPS)
    assert e.value.status == _lib.ARGR_EUNSUPPORTED
    assert _lib.load().argreduce_logits_plan(0, 3, 100, 0, 0, ctypes.byref(CAPS), None) == _lib.ARGR_EINVAL


def test_cpu_tensors_are_refused():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 5)
    with pytest.raises(ValueError, match="CUDA"):
        A.token_logprobs(x, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        A.distill_topk(x, torch.zeros(2, 1, dtype=torch.int64), torch.zeros(2, 1))
