"""Beam selection, reordering and routing without a GPU: refusals before any device
work, the geometry of states, and the definitions that the GPU tests hold the kernels to."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import row_wise_arg_gb300 as A
import select_ref as ref
from row_wise_arg_gb300 import _lib
from row_wise_arg_gb300.build import build

X = 0x10000  # fake, never dereferenced addresses, 16-byte aligned
FAR = X + (1 << 40)
EINVAL, OK = _lib.ARGR_EINVAL, _lib.ARGR_OK


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


def select(**kw):
    a = dict(x=X, dtype=0, items=2, beams=3, cols=100, stride=100, temp=1.0, scores=FAR, ended=None, end=0, scale=None, count=4,
             tokens=FAR, parents=FAR, out=FAR, scratch=None, bytes=0, stream=None)
    a.update(kw)
    return _lib.load().argreduce_beam_select(*a.values())


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=X + 2), dict(items=-1), dict(items=1 << 40), dict(beams=0), dict(beams=65), dict(cols=0), dict(cols=1 << 31),
    dict(stride=-1), dict(temp=0.0), dict(temp=float("nan")), dict(scores=None), dict(scores=FAR + 1), dict(scale=FAR + 2),
    dict(count=0), dict(count=129), dict(tokens=None), dict(tokens=FAR + 4), dict(parents=None), dict(out=None), dict(out=FAR + 1),
    dict(dtype=7), dict(stride=1 << 62)])
def test_select_refuses(bad):
    assert select(**bad) == EINVAL


def test_select_other_returns():
    assert select(items=0, x=None, scores=None, tokens=None, parents=None, out=None) == OK
    assert select(dtype=3) == _lib.ARGR_EUNSUPPORTED


def reorder(states=(X,), **kw):
    a = dict(n=len(states), items=2, beams=3, item_stride=300, beam_stride=100, outer=2, outer_stride=50, positions=10, bytes=5,
             parents=FAR, lengths=None, stream=None)
    a.update(kw)
    return _lib.load().argreduce_beam_reorder((ctypes.c_void_p * len(states))(*states), *a.values())


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(n=1025), dict(items=-1), dict(beams=0), dict(beams=65), dict(outer=-1), dict(positions=-1), dict(bytes=0),
    dict(item_stride=-300), dict(parents=None), dict(parents=FAR + 4), dict(lengths=FAR + 1), dict(parents=X + 8), dict(lengths=X + 592),
    dict(beam_stride=99), dict(item_stride=299), dict(outer_stride=49), dict(beam_stride=0), dict(positions=1 << 62),
    dict(item_stride=(1 << 63) - 1, items=1 << 30)])
def test_reorder_refuses(bad):
    assert reorder(**bad) == EINVAL


def test_reorder_refuses_states_that_overlap():
    assert reorder(states=(X, None)) == EINVAL
    assert reorder(states=(X, X)) == EINVAL
    assert reorder(states=(X, FAR * 2, X + 599)) == EINVAL
    # one beam: nothing can move, so these calls end before the device is asked for
    one = dict(beams=1, items=4, item_stride=200, outer=2, outer_stride=60, positions=10, bytes=3)
    assert reorder(states=(X,), **one) == OK
    assert reorder(states=(X, X + 30), **one) == OK       # columns of the same rows
    assert reorder(states=(X, X + 110), **one) == OK      # behind the row's last segment
    assert reorder(states=(X, X + 29), **one) == EINVAL
    assert reorder(states=(X, X + 60), **one) == EINVAL   # its first segment is the other's second
    assert reorder(states=(X, X + 200), **one) == EINVAL  # its first item is the other's second
    assert reorder(states=(X, X + 171), **one) == EINVAL  # reaches into the next item
    assert reorder(states=(X, X + 170), **one) == OK
    assert reorder(states=(X, X + 800), **one) == OK
    assert reorder(states=(X + 30, X, X + 800), **one) == OK
    assert reorder(states=(), **one) == OK


@pytest.mark.parametrize("seed", range(30))
def test_overlaps_are_found_exactly(seed):
    """Against the bytes themselves, for nested layouts of every kind."""
    rng = np.random.Generator(np.random.PCG64(seed))
    seg = int(rng.integers(1, 6))
    counts = rng.integers(1, 4, 2)
    strides, extent = [], seg
    for n in counts:
        strides.append(extent + int(rng.integers(0, 7)))
        extent += strides[-1] * (int(n) - 1)
    order = rng.permutation(2)
    items, outer = int(counts[order[0]]), int(counts[order[1]])
    si, so = strides[order[0]], strides[order[1]]
    mine = {i * si + o * so + b for i in range(items) for o in range(outer) for b in range(seg)}
    for d in range(0, extent + 3):
        meets = any(b + d in mine for b in mine)
        got = reorder(states=(X, X + d), beams=1, items=items, item_stride=si, outer=outer, outer_stride=so, positions=seg, bytes=1)
        assert got == (EINVAL if meets else OK), (d, seg, counts, strides)


def route(**kw):
    a = dict(x=X, dtype=0, rows=4, experts=10, stride=10, k=2, normalize=1, valid=None, weights=FAR, ids=FAR, lse=FAR, counts=None,
             taken=None, balance=None, scratch=None, bytes=0, stream=None)
    a.update(kw)
    return _lib.load().argreduce_route(*a.values())


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(rows=-1), dict(experts=0), dict(experts=1025), dict(k=0), dict(k=11), dict(k=33, experts=64), dict(weights=None),
    dict(ids=None), dict(lse=None), dict(ids=FAR + 4), dict(counts=FAR), dict(taken=FAR), dict(balance=FAR), dict(weights=FAR + 1),
    dict(counts=FAR + 4, taken=FAR), dict(stride=-1)])
def test_route_refuses(bad):
    assert route(**bad) == EINVAL


def route_backward(**kw):
    a = dict(x=X, dtype=0, rows=4, experts=10, stride=10, k=2, normalize=1, weights=FAR, ids=FAR, lse=FAR, counts=FAR, taken=FAR,
             gw=FAR, gl=FAR, gb=FAR, grad=FAR, grad_stride=10, stream=None)
    a.update(kw)
    return _lib.load().argreduce_route_backward(*a.values())


@pytest.mark.parametrize("bad", [
    dict(lse=None), dict(weights=None), dict(ids=None), dict(counts=None), dict(taken=None), dict(grad=None), dict(grad=X + 4),
    dict(grad_stride=9), dict(grad=X, grad_stride=11), dict(gb=FAR + 2), dict(k=0), dict(experts=1025)])
def test_route_backward_refuses(bad):
    assert route_backward(**bad) == EINVAL


def test_route_nothing_to_do():
    assert route(rows=0, x=None, weights=None, ids=None, lse=None) == OK
    assert route(rows=0, x=None, dtype=3) == _lib.ARGR_EUNSUPPORTED
    assert route_backward(rows=0, x=None, grad=None, lse=None) == OK


# -- the plan of a step ------------------------------------------------------------------------
PLANNER = """
#include "select.h"
extern "C" int plan(int64_t items, int beams, int64_t cols, int dtype, int k, int max_cluster, int placed, int* out) {
    argr_caps caps = {};
    caps.sm_count = 152;
    caps.max_threads_per_sm = 2048;
    caps.max_cluster = max_cluster;
    argr::BeamPlan p;
    int asked = 0;
    const auto fits = [&](const argr::BeamPlan& b, bool* ok) {
        ++asked;
        *ok = b.cluster <= placed;
        return placed < 0 ? cudaErrorInvalidValue : cudaSuccess;
    };
    const cudaError_t e = argr::fitting_beam_plan(items, beams, cols, dtype, k, caps, fits, &p);
    out[0] = p.cluster;
    out[1] = p.shift;
    out[2] = p.block;
    out[3] = p.stream;
    out[4] = asked;
    return e;
}
"""


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    """The planner, with a device of which the caller says what clusters it places."""
    from row_wise_arg_gb300 import build as b
    at = tmp_path_factory.mktemp("planner")
    (at / "planner.cpp").write_text(PLANNER)
    so = str(at / "planner.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(b.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + b.INCLUDE, "-I" + b.CSRC, "-I" + cuda, str(at / "planner.cpp"),
                    _lib.LIB_PATH, "-Wl,-rpath," + os.path.dirname(_lib.LIB_PATH), "-o", so], check=True)
    lib = ctypes.CDLL(so)

    def plan(items, beams, cols, dtype=0, k=8, max_cluster=16, placed=16):
        out = (ctypes.c_int * 5)()
        st = lib.plan(ctypes.c_int64(items), beams, ctypes.c_int64(cols), dtype, k, max_cluster, placed, out)
        return (st, *out)
    return plan


def test_a_step_without_room_for_its_cluster(planner):
    """Clusters that a device does not place are made smaller, then done without (rows, and a merge that needs scratch)."""
    assert planner(1, 4, 202048, 2)[:3] == (0, 16, 2) and planner(1, 4, 202048, 2, placed=8)[:3] == (0, 8, 1)
    assert planner(1, 1, 202048, 2)[:3] == (0, 4, 2)
    assert planner(1, 1, 202048, 2, placed=2)[:3] == (0, 2, 1)
    assert planner(1, 1, 202048, 2, placed=1)[:3] == (0, 1, 0)
    assert planner(1, 4, 202048, 2, placed=4)[:3] == (0, 4, 0)
    for beams in range(1, 17):
        for items, cols in ((1, 1000), (2, 300000), (9, 32000)):
            for placed in (1, 2, 3, 4, 7, 8, 12, 15, 16):
                st, cluster, shift, block, stream, asked = planner(items, beams, cols, placed=placed)
                assert st == 0 and asked <= 5 and 32 <= block <= 512 and not stream
                if beams <= placed:
                    assert cluster == beams << shift and cluster <= placed
                    assert planner(items, beams, cols, placed=16)[1] <= placed or cluster * 2 > placed
                else:
                    assert cluster == 0 and shift == 0
                # a device that says so by itself gives the same plan
                assert planner(items, beams, cols, max_cluster=placed)[:5] == (0, cluster, shift, block, stream)
    assert planner(1, 17, 1000)[1] == 0 and planner(1, 17, 1000)[5] == 0
    assert planner(1, 4, 1000, placed=-1)[0] != 0  # an error is handed on


# -- the geometry of states ------------------------------------------------------------------
def test_geometry():
    torch = pytest.importorskip("torch")
    from row_wise_arg_gb300.beam import _geometry
    t = torch.empty(6, 5, 20, 8, dtype=torch.float16)  # 2 items of 3 beams
    row = 5 * 20 * 8 * 2
    assert _geometry(t, 2, 3, 2) == (3 * row, row, 5, 320, 20, 16)
    assert _geometry(t, 2, 3, -2) == (3 * row, row, 5, 320, 20, 16)
    assert _geometry(t, 2, 3, None) == (3 * row, row, 1, 0, 1, row)
    assert _geometry(t.view(2, 3, 5, 20, 8), 2, 3, 3) == (3 * row, row, 5, 320, 20, 16)
    assert _geometry(t[:, 1:3], 2, 3, 2) == (3 * row, row, 2, 320, 20, 16)
    assert _geometry(t[:, :, :7], 2, 3, None) == (3 * row, row, 5, 320, 1, 7 * 16)
    assert _geometry(t[..., 0, 0], 2, 3, None)[2:] == (5, 320, 1, 2)
    assert _geometry(torch.empty(6), 2, 3, None) == (12, 4, 1, 0, 1, 4)
    for bad, dim in ((t.transpose(1, 2), 1), (t, 0), (t, 4), (t[..., :4], 2), (t[:, :, ::2], 2), (t[:5], 2)):
        with pytest.raises(ValueError):
            _geometry(bad, 2, 3, dim)


def test_geometry_of_one_item():
    """A lone item's stride says nothing: columns of the same rows are apart whatever it is."""
    torch = pytest.importorskip("torch")
    from row_wise_arg_gb300.beam import _apart, _geometry
    rows = torch.empty(4, 10)
    a = rows.as_strided((1, 4, 3), (7, 10, 1))
    b = rows.as_strided((1, 4, 5), (1, 10, 1), 3)
    ga, gb = _geometry(a, 1, 4, None), _geometry(b, 1, 4, None)
    assert ga == (160, 40, 1, 0, 1, 12) and gb == (160, 40, 1, 0, 1, 20)
    assert _apart(a.data_ptr(), ga, b.data_ptr(), gb, 1, 4)


class Elsewhere:
    """What the binding looks at of logits that lie on another GPU than the current one."""
    is_cuda, requires_grad, shape = True, False, (4, 100)

    def get_device(self):
        return 1

    def __getattr__(self, name):
        raise AssertionError(f"{name} was used of logits on another device")


def test_logits_of_another_device_are_refused(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x = Elsewhere()
    for call in (lambda: A.beam_select(x, None, 3), lambda: A.route_topk(x, 2),
                 lambda: A.route_topk_backward(x, None, None, None)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_what_lies_on_the_cpu_is_refused():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 10)
    p = torch.zeros(1, 4, dtype=torch.int64)
    for call in (lambda: A.beam_select(x, x[:, 0], 3), lambda: A.route_topk(x, 2), lambda: A.beam_reorder(x, p),
                 lambda: A.beam_reorder([x], p)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_an_argument_with_a_tangent_is_refused():
    torch = pytest.importorskip("torch")
    from torch.autograd import forward_ad
    from row_wise_arg_gb300.logits import _arg
    t = torch.ones(3, 2)
    arg = lambda v, dtype: _arg(v, "scores", dtype, (3, 2), t.device)  # noqa: E731
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(t, torch.ones(3, 2))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            arg(dual, torch.float32)
        assert arg(t, torch.float32) == t.data_ptr() and arg(t > 0, torch.bool)
    assert arg(t, torch.float32) == t.data_ptr() and arg(None, torch.float32) is None


def test_apart():
    pytest.importorskip("torch")
    from row_wise_arg_gb300.beam import _apart
    a, b = (300, 100, 1, 0, 10, 4), (300, 100, 1, 0, 5, 12)  # 40 and 60 bytes of rows of 100
    assert _apart(1000, a, 1040, b, 2, 3) and not _apart(1000, a, 1039, b, 2, 3) and not _apart(1000, a, 1041, b, 2, 3)
    assert _apart(1000, a, 1540, b, 2, 3) and not _apart(1000, b, 1550, a, 2, 3) and _apart(1000, b, 1560, a, 2, 3)
    assert not _apart(1000, a, 1040, (600, 200, 1, 0, 5, 12), 2, 3)


@pytest.mark.parametrize("seed", range(20))
def test_apart_is_never_wrong(seed):
    """Against the bytes themselves: states that share one are never taken to be apart."""
    pytest.importorskip("torch")
    from row_wise_arg_gb300.beam import _apart
    rng = np.random.Generator(np.random.PCG64(seed))
    seen = set()
    for _ in range(300):
        unit = int(rng.integers(6, 13))  # what segments lie apart, one item and beam of which take `per` or more
        per = int(rng.integers(1, 4))
        items, beams = int(rng.integers(1, 3)), int(rng.integers(1, 3))

        def geometry():
            outer, size = int(rng.integers(1, per + 1)), int(rng.integers(1, 7))
            beam = unit * (per + int(rng.integers(0, 2)) if rng.random() < 0.3 else per) + (int(rng.integers(0, 2)) if rng.random() < 0.3 else 0)
            item = beam * beams + (unit * int(rng.integers(0, 3)) if rng.random() < 0.3 else 0)
            return (item, beam, outer, unit if outer > 1 else 0, size, 1)

        def touched(at, g):
            return {at + i * g[0] + j * g[1] + o * g[3] + p for i in range(items) for j in range(beams) for o in range(g[2])
                    for p in range(g[4])}
        ga, gb, d = geometry(), geometry(), int(rng.integers(0, 40))
        apart, meet = _apart(1000, ga, 1000 + d, gb, items, beams), not touched(1000, ga).isdisjoint(touched(1000 + d, gb))
        assert not (apart and meet), (ga, gb, d, items, beams)
        seen.add((apart, meet))
    assert seen == {(True, False), (False, True), (False, False)}


def test_apart_by_segments():
    """[2, 3, 5, 10 | 6] int8 cut along the last dimension: segments of 10 and of 6 bytes, 16 apart."""
    pytest.importorskip("torch")
    from row_wise_arg_gb300.beam import _apart
    a, b = (240, 80, 5, 16, 1, 10), (240, 80, 5, 16, 1, 6)
    assert _apart(1000, a, 1010, b, 2, 3) and not _apart(1000, a, 1009, b, 2, 3) and not _apart(1000, a, 1011, b, 2, 3)
    assert not _apart(1000, a, 1010, (240, 80, 5, 15, 1, 5), 2, 3)


def test_beam_definition():
    """The 64-bit step against sorting every continuation by hand."""
    x = np.log(np.array([[0.5, 0.3, 0.2], [0.1, 0.8, 0.1]]))
    t, p, s, _, _ = ref.beam_select(x, np.array([-1.0, -1.2]), 4)
    assert t.tolist() == [1, 0, 1, 2] and p.tolist() == [1, 0, 0, 0]
    assert np.allclose(s, [np.log(0.8) - 1.2, np.log(0.5) - 1, np.log(0.3) - 1, np.log(0.2) - 1])
    t, p, s, _, _ = ref.beam_select(x, np.array([-np.inf, -1.2]), 5, ended=np.array([False, True]), end_token=7)
    assert t.tolist() == [7, -1, -1, -1, -1] and p.tolist() == [1, -1, -1, -1, -1] and s[0] == -1.2 and np.isinf(s[1:]).all()


def test_route_gradient_against_differences():
    rng = np.random.Generator(np.random.PCG64(2))
    x = rng.normal(size=(5, 6))
    for normalize in (True, False):
        w, ids, lse, counts, n, _ = ref.route(x, 2, normalize)
        g, h, b = rng.normal(size=w.shape), rng.normal(size=5), 1.7
        grad, _ = ref.route_grad(x, ids, counts, n, 2, g, h, b, normalize)
        for r in range(5):
            for e in range(6):
                f = []
                for s in (1e-6, -1e-6):
                    z = x.copy()
                    z[r, e] += s
                    w, i, lse, _, _, balance = ref.route(z, 2, normalize)
                    assert (i == ids).all()
                    f.append((g * w).sum() + (h * lse).sum() + b * balance)
                assert abs((f[0] - f[1]) / 2e-6 - grad[r, e]) < 1e-7
