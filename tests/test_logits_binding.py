"""The vocabulary-row operators' binding without a GPU: import, refusals before any device work."""
import ctypes
import os
import subprocess
import sys

import pytest

import row_wise_arg_gb300 as A
from row_wise_arg_gb300 import _lib
from row_wise_arg_gb300.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
X = 0x10000  # a fake, never dereferenced address, 16-byte aligned


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def python(code):
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_star_import_needs_no_torch():
    python("import sys; sys.modules['torch'] = None\n"
           "from row_wise_arg_gb300 import *\n"
           "assert callable(argreduce) and callable(argreduce_logits_plan)")


@pytest.mark.parametrize("lacking", ["sys.modules['torch'] = None",
                                     "_lib.load = lambda: (_ for _ in ()).throw(RuntimeError('not built'))"])
def test_operators_are_absent_where_they_cannot_be_loaded(lacking):
    """As attributes are: hasattr says so, and the reason is named."""
    python("import sys\nimport row_wise_arg_gb300 as A\nfrom row_wise_arg_gb300 import _lib\n" + lacking + "\n"
           "assert not hasattr(A, 'token_logprobs')\n"
           "try:\n    A.distill_topk\nexcept AttributeError as e:\n    assert e.__cause__ is not None and 'distill_topk' in str(e)\n"
           "else:\n    raise SystemExit('no error')")


def test_temperature_whose_scale_overflows():
    """log2(e) / T multiplies every difference of logits: infinite, it would turn 0 * inf into NaN."""
    lib = _lib.load()
    t = ctypes.c_float(4e-39)  # 1 / t is finite, log2(e) / t is not
    rows = (X, 0, 3, 100, 100, t)
    far = X + (1 << 30)
    assert lib.argreduce_logprobs(*rows, X, 0, X, X, X, None, None, None, None, None) == _lib.ARGR_EINVAL
    assert lib.argreduce_logprobs_backward(*rows, X, X, X, None, None, far, 100, None, None) == _lib.ARGR_EINVAL
    assert lib.argreduce_distill(*rows, X, X, 4, 0, X, None, None, None) == _lib.ARGR_EINVAL
    assert lib.argreduce_distill_backward(*rows, X, X, 4, 0, X, X, far, 100, None, None) == _lib.ARGR_EINVAL
    assert lib.argreduce_distill_step(*rows, X, X, 4, 0, X, X, X, far, 100, None, None) == _lib.ARGR_EINVAL


class Elsewhere:
    """What the binding looks at of logits that lie on another GPU than the current one."""
    is_cuda, requires_grad, shape = True, False, (4, 100)

    def get_device(self):
        return 1

    def __getattr__(self, name):
        raise AssertionError(f"{name} was used of logits on another device")


def test_logits_of_another_device_are_refused(monkeypatch):
    """The library plans and launches on the current device."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = Elsewhere()
    for call in (lambda: A.token_logprobs(x), lambda: A.token_logprobs_backward(x, None, None),
                 lambda: A.distill_topk(x, None, None), lambda: A.distill_topk_backward(x, None, None, None, None),
                 lambda: A.distill_topk_step(x, None, None, None)):
        with pytest.raises(ValueError, match="current device"):
            call()
