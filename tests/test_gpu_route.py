"""Routing on the GPU against its definition in 64 bits: weights, ids, counts, the
balance loss and the gradients, at the sizes, strides and masks where they can go wrong."""
import numpy as np
import pytest

import logits_ref
import select_ref as ref

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import row_wise_arg_gb300 as A  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LOWEST = {"f32": -3.4028234663852886e38, "f16": -65504.0, "bf16": -3.3895313892515355e38}
U = logits_ref.U32


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_wise_arg_gb300.build import build
    build()


def on_gpu(x, dtype, pad=0, offset=0):
    rows, cols = x.shape
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype])
    buf = torch.full((offset + rows * (cols + pad) + 64,), float("nan"), dtype=DT[dtype], device="cuda")
    view = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t.cuda())
    return view, t.double().numpy()


def close(got, want, bound, what):
    got, want = got.detach().double().cpu().numpy(), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    assert (np.isnan(got) == np.isnan(want)).all(), f"{what}: NaNs"
    inf = np.isinf(want)
    assert (got[inf] == want[inf]).all(), f"{what}: infinities"
    ok = np.isfinite(want)
    off = (np.abs(got - np.where(ok, want, 0.0)) / np.broadcast_to(bound, want.shape))[ok]
    assert off.size == 0 or off.max() <= 1.0, f"{what}: {off.max():.2f} times the bound"


def check(x, dtype, k, normalize=True, valid=None, pad=0, offset=0, seed=1, grads="whb"):
    rows, experts = x.shape
    xd, x64 = on_gpu(x, dtype, pad, offset)
    v = None if valid is None else torch.from_numpy(valid).cuda()
    r = A.route_topk(xd, k, valid=v, normalize=normalize, counts=True, balance=True)
    w, ids, lse, counts, n, balance = ref.route(x64, k, normalize, valid)
    e = logits_ref.sum_error(experts)
    assert (r.ids.cpu().numpy() == ids).all()
    assert (r.counts.cpu().numpy() == counts).all() and r.rows.item() == n
    # a quotient of two sums of exponentials
    close(r.weights, w, 2 * e * w + 1e-37, "weights")
    close(r.lse, lse, logits_ref.logprob_bound(lse, experts), "lse")
    # positive terms: each p off by 2 e, their sums over the rows by 6 sqrt(rows) u, the last rounding
    close(r.balance, balance, (2 * e + U * (6 * np.sqrt(rows) + 4)) * np.abs(balance) + 1e-37, "balance")
    plain = A.route_topk(xd, k, valid=v, normalize=normalize)
    assert plain.counts is None and plain.rows is None and plain.balance is None
    assert torch.equal(plain.ids, r.ids) and torch.equal(plain.weights.nan_to_num(7), r.weights.nan_to_num(7))
    # gradients
    rng = np.random.Generator(np.random.PCG64(seed))
    g = rng.normal(size=(rows, k)).astype(np.float32) * ("w" in grads)
    h = rng.normal(size=rows).astype(np.float32) * ("h" in grads)
    b = np.float32(rng.normal() * rows * ("b" in grads))
    want, size = ref.route_grad(x64, ids, counts, n, k, g.astype(np.float64), h.astype(np.float64), float(b), normalize, valid)
    cuda = lambda a, on: torch.from_numpy(np.asarray(a)).cuda() if on in grads else None  # noqa: E731
    given = dict(grad_weights=cuda(g, "w"), grad_lse=cuda(h, "h"), grad_balance=cuda(b, "b"))
    got = A.route_topk_backward(xd, r.weights, r.ids, r.lse, r.counts, r.rows, normalize=normalize, **given)
    bound = logits_ref.grad_bound(want, 2 * size, experts, dtype) + 16 * U * size * np.abs(np.where(np.isfinite(lse), lse, 0))[:, None]
    close(got, want, bound, "gradient")
    # by automatic differentiation, and written over the logits
    leaf = xd.detach().clone().requires_grad_()
    t = A.route_topk(leaf, k, valid=v, normalize=normalize, counts="b" in grads, balance="b" in grads)
    parts = [(o, i) for o, i in ((t.weights, given["grad_weights"]), (t.lse, given["grad_lse"]), (t.balance, given["grad_balance"])) if i is not None]
    torch.autograd.backward([o for o, _ in parts], [i for _, i in parts])
    assert torch.equal(leaf.grad.nan_to_num(7), got.nan_to_num(7))
    A.route_topk_backward(xd, r.weights, r.ids, r.lse, r.counts, r.rows, normalize=normalize, grad=xd, **given)
    assert torch.equal(xd.nan_to_num(7), got.nan_to_num(7))
    return r


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,experts,k,normalize,pad,offset", [
    (1, 1, 1, True, 0, 0), (1, 8, 2, True, 0, 0), (3, 2, 2, False, 0, 1), (7, 60, 6, True, 0, 0), (300, 64, 8, False, 0, 0),
    (1000, 129, 5, True, 0, 0), (257, 256, 8, True, 0, 0), (33, 1024, 32, True, 0, 0), (5, 1023, 17, False, 3, 1),
    (2000, 8, 2, True, 0, 0), (3, 33, 32, False, 0, 0), (64, 31, 31, True, 5, 3), (100, 500, 4, True, 0, 0), (9, 4, 4, True, 12, 1),
    (501, 16, 1, False, 0, 0), (130, 384, 8, True, 8, 0), (40, 160, 6, True, 0, 8),
    (700, 256, 32, True, 0, 0), (90, 200, 20, False, 0, 0), (50, 512, 32, True, 0, 0), (333, 12, 12, True, 4, 0), (70, 32, 32, False, 0, 0)])
def test_sizes(dtype, rows, experts, k, normalize, pad, offset):
    rng = np.random.Generator(np.random.PCG64(rows + experts))
    x = rng.normal(size=(rows, experts)) + rng.normal(size=experts) * 0.5
    check(x, dtype, k, normalize, pad=pad, offset=offset)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("experts,k", [(20, 6), (8, 8), (200, 12)])
def test_masks(dtype, normalize, experts, k):
    rng = np.random.Generator(np.random.PCG64(3))
    x = rng.normal(size=(60, experts)) * 3
    valid = rng.random(60) < 0.7
    x[~valid] = np.nan  # not looked at
    x[5:9], valid[5:9] = -np.inf, True  # nothing left
    x[9, 3:], valid[9] = -np.inf, True  # fewer than k
    x[10, :], valid[10] = LOWEST[dtype], True
    x[11, 1:], valid[11] = LOWEST[dtype], True
    x[12, 1:], valid[12] = 40.0, True
    x[:, 2] = -np.inf  # an expert that is gone
    check(x, dtype, k, normalize, valid)
    check(x[:0], dtype, k, normalize, valid[:0])
    check(x[5:9], dtype, k, normalize)
    check(x[5:13], dtype, k, normalize, np.zeros(8, bool))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("experts,k", [(8, 2), (16, 3), (20, 6), (60, 4), (100, 5), (200, 12), (500, 8), (1000, 4)])
def test_gradient_of_rows_far_from_zero(dtype, normalize, experts, k):
    """Rows whose lse, a binary32 number, says little or nothing of their sum: a large common offset, the type's
    lowest value throughout, its largest. Each p is still exp(x - m) / s, so the bound has no part that grows with lse."""
    rng = np.random.Generator(np.random.PCG64(experts))
    high = {"f32": 3e7, "f16": 60000.0, "bf16": 1e5}[dtype]
    offsets = np.array([0.0, 1000.0, -1000.0, 30000.0, -30000.0, high, -high])
    x = rng.normal(size=(40, experts)) + offsets[np.arange(40) % len(offsets)][:, None]
    x[5] = LOWEST[dtype]
    x[6] = -LOWEST[dtype]
    x[7, 1:] = LOWEST[dtype]
    x[8] = LOWEST[dtype]
    x[8, experts // 2:] = -np.inf
    xd, x64 = on_gpu(x, dtype)
    r = A.route_topk(xd, k, normalize=normalize, balance=True)
    w, ids, lse, counts, n, _ = ref.route(x64, k, normalize)
    assert (r.ids.cpu().numpy() == ids).all() and (r.counts.cpu().numpy() == counts).all() and r.rows.item() == n
    for on in ("w", "h", "b", "whb"):
        g = rng.normal(size=(40, k)).astype(np.float32) * ("w" in on)
        h = rng.normal(size=40).astype(np.float32) * ("h" in on)
        b = np.float32(rng.normal() * 40 * ("b" in on))
        want, size = ref.route_grad(x64, ids, counts, n, k, g.astype(np.float64), h.astype(np.float64), float(b), normalize)
        cuda = lambda a, name: torch.from_numpy(np.asarray(a)).cuda() if name in on else None  # noqa: E731
        got = A.route_topk_backward(xd, r.weights, r.ids, r.lse, r.counts, r.rows, normalize=normalize,
                                    grad_weights=cuda(g, "w"), grad_lse=cuda(h, "h"), grad_balance=cuda(b, "b"))
        close(got, want, logits_ref.grad_bound(want, 2 * size, experts, dtype), f"gradient of {on}")


@pytest.mark.parametrize("what", [np.nan, np.inf])
def test_rows_with_a_mistake(what):
    rng = np.random.Generator(np.random.PCG64(4))
    x = rng.normal(size=(40, 24))
    x[7, 5] = what
    r = check(x, "f32", 4)
    assert torch.isnan(r.balance) and torch.isnan(r.weights[7]).all() and not torch.isnan(r.weights[:7]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties(dtype):
    """Few values: the lowest index first."""
    rng = np.random.Generator(np.random.PCG64(5))
    for experts in (8, 40, 256, 700):
        check(rng.integers(0, 3, (200, experts)) * 1.0, dtype, min(8, experts))
    check(np.zeros((50, 64)), dtype, 32)
    check(np.where(rng.random((50, 64)) < 0.5, 0.0, -0.0), dtype, 7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_close_values(dtype):
    """Neighbours in the type: the order is exact."""
    rng = np.random.Generator(np.random.PCG64(6))
    step = 2.0 ** (-23 if dtype == "f32" else -7)
    check(1.0 + step * rng.integers(0, 100, (300, 256)), dtype, 8)
    check(-1.0 - step * rng.integers(0, 20, (300, 16)), dtype, 8)


@pytest.mark.parametrize("grads", ["w", "h", "b", "wb", "hb"])
def test_each_gradient(grads):
    rng = np.random.Generator(np.random.PCG64(7))
    x = rng.normal(size=(333, 48))
    check(x, "f32", 6, True, rng.random(333) < 0.8, grads=grads)
    check(x, "f16", 6, False, grads=grads)


def test_many_rows():
    """More rows than a wave of CTAs takes at once, wide and narrow."""
    rng = np.random.Generator(np.random.PCG64(8))
    for experts, rows in ((8, 70001), (64, 40003), (256, 9001)):
        x = rng.normal(size=(rows, experts)).astype(np.float32)
        xd = torch.from_numpy(x).cuda()
        r = A.route_topk(xd, 4, counts=True, balance=True)
        z = torch.from_numpy(x).double()
        order = torch.sort(z, dim=-1, descending=True, stable=True)[1][:, :4]
        assert torch.equal(r.ids.cpu(), order)
        counts = torch.bincount(order.flatten(), minlength=experts)
        assert torch.equal(r.counts.cpu(), counts) and r.rows.item() == rows
        want = experts * (counts.double() / (4 * rows) * torch.softmax(z, -1).mean(0)).sum()
        assert abs(r.balance.item() - want.item()) <= (2 * logits_ref.sum_error(experts) + U * (6 * np.sqrt(rows) + 4)) * want.item()
        again = A.route_topk(xd, 4, counts=True, balance=True)
        assert torch.equal(again.balance, r.balance)


def test_offsets_past_32_bits():
    """Rows that begin beyond 2^31 elements, and their gradient over them."""
    stride = (1 << 30) + 64
    buf = torch.empty(3 * stride + 64, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((4, 60), (stride, 1))
    near = torch.randn(4, 60, device="cuda").bfloat16()
    x.copy_(near)
    r, want = (A.route_topk(t, 5, counts=True, balance=True) for t in (x, near))
    assert all(torch.equal(a, b) for a, b in zip(r, want))
    g = dict(grad_weights=torch.randn(4, 5, device="cuda"), grad_lse=torch.randn(4, device="cuda"),
             grad_balance=torch.tensor(2.0, device="cuda"))
    want = A.route_topk_backward(near, *want[:5], **g)
    A.route_topk_backward(x, *r[:5], grad=x, **g)
    assert torch.equal(x, want)


def test_calls_at_once():
    """Routes of many rows (with scratch) and of few, and gradients, on two streams at a time."""
    given = [torch.randn(n, e, device="cuda") for n, e in ((60000, 64), (5000, 256), (30, 64), (20001, 60))]
    want = [A.route_topk(x, 6, counts=True, balance=True) for x in given]
    g = [torch.randn(x.shape[0], 6, device="cuda") for x in given]
    grads = [A.route_topk_backward(x, *r[:5], grad_weights=w) for x, r, w in zip(given, want, g)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for turn in range(8):
        for i, x in enumerate(given):
            s = streams[(i + turn) % 2]
            r = A.route_topk(x, 6, counts=True, balance=True, stream=s)
            got.append((i, r, A.route_topk_backward(x, *r[:5], grad_weights=g[i], stream=s)))
    torch.cuda.synchronize()
    for i, r, d in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want[i])) and torch.equal(d, grads[i]), i


def test_gradient_against_differences():
    """The 64-bit formula that the kernel is held to, against differences of the definition (the choice fixed)."""
    rng = np.random.Generator(np.random.PCG64(9))
    x = rng.normal(size=(7, 9))
    k, step = 3, 1e-6
    g, h, b = rng.normal(size=(7, k)), rng.normal(size=7), 2.5
    for normalize in (True, False):
        w, ids, lse, counts, n, _ = ref.route(x, k, normalize)
        grad, _ = ref.route_grad(x, ids, counts, n, k, g, h, b, normalize)
        def goal(z):
            w, i, lse, c, n, balance = ref.route(z, k, normalize)
            assert (i == ids).all()
            return (g * w).sum() + (h * lse).sum() + b * balance
        for r in range(7):
            for e in range(9):
                up, down = x.copy(), x.copy()
                up[r, e] += step
                down[r, e] -= step
                # differences of order step^2, roundings of 1e-16 / step
                assert abs((goal(up) - goal(down)) / (2 * step) - grad[r, e]) < 1e-7


def test_shapes_streams_and_graphs():
    x = torch.randn(3, 5, 16, device="cuda")
    r = A.route_topk(x, 2, counts=True, balance=True)
    assert r.weights.shape == (3, 5, 2) and r.lse.shape == (3, 5) and r.counts.shape == (16,) and r.balance.shape == ()
    one = A.route_topk(x[1, 2], 2)
    assert torch.equal(one.ids, r.ids[1, 2]) and torch.equal(one.weights, r.weights[1, 2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = A.route_topk(x, 2, counts=True, balance=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(s, r))
    # two graphs, replayed beside one another: each has scratch of its own
    many = [torch.randn(4000, 100, device="cuda") for _ in range(2)]
    want = [A.route_topk(m, 4, counts=True, balance=True) for m in many]
    graphs, got, sides = [], [], [torch.cuda.Stream() for _ in range(2)]
    for m, st in zip(many, sides):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            got.append(A.route_topk(m, 4, counts=True, balance=True))
    for _ in range(20):
        for g, st in zip(graphs, sides):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("rows,experts", [(1, 8), (256, 1024), (257, 1024), (5000, 64)])
def test_scratch_is_what_the_library_asks_for(monkeypatch, rows, experts):
    """Also for few rows: which routes need scratch is the library's plan alone."""
    from row_wise_arg_gb300 import route
    given = []

    class Library:
        def __getattr__(self, name):
            return getattr(lib, name)

        def argreduce_route_scratch_bytes(self, *a):
            return lib.argreduce_route_scratch_bytes(*a) + 4096

        def argreduce_route(self, *a):
            given.append(a[-3:-1])
            return lib.argreduce_route(*a)

    lib = route._LIB
    x = torch.randn(rows, experts, device="cuda")
    want = A.route_topk(x, 4, balance=True)
    route._scratch_bytes.cache_clear()
    monkeypatch.setattr(route, "_LIB", Library())
    got, plain = A.route_topk(x, 4, balance=True), A.route_topk(x, 4)
    route._scratch_bytes.cache_clear()
    assert given[0][0] and given[0][1] == lib.argreduce_route_scratch_bytes(rows, experts) + 4096
    assert given[1] == (None, 0)  # nothing is counted
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(plain.ids, want.ids)


@pytest.mark.parametrize("rows,experts,k", [(1, 8, 2), (300, 64, 4), (4000, 8, 1), (9000, 100, 6), (3000, 700, 8)])
def test_counts_without_the_loss(rows, experts, k):
    x = torch.randn(rows, experts, device="cuda")
    valid = torch.rand(rows, device="cuda") < 0.8
    whole, r = A.route_topk(x, k, valid=valid, balance=True), A.route_topk(x, k, valid=valid, counts=True)
    assert r.balance is None and torch.equal(r.counts, whole.counts) and torch.equal(r.rows, whole.rows)
    assert torch.equal(r.rows, valid.sum()) and torch.equal(r.ids, whole.ids) and torch.equal(r.lse, whole.lse)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_views(dtype):
    """[batch, positions, experts] cut from wider rows, one row for all (a broadcast), a row alone, and a gradient written into a padded tensor."""
    wide = torch.randn(4, 9, 50, device="cuda").to(DT[dtype]).requires_grad_()
    x = wide[..., 3:43]
    r = A.route_topk(x, 5, balance=True)
    g = torch.randn(4, 9, 5, device="cuda")
    ((r.weights * g).sum() + r.lse.sum() * 0.1 + r.balance * 7).backward()
    flat = x.detach().reshape(36, 40)
    f = A.route_topk(flat, 5, balance=True)
    given = dict(grad_weights=g.view(36, 5), grad_lse=torch.full((36,), 0.1, device="cuda"), grad_balance=torch.tensor(7.0, device="cuda"))
    want = A.route_topk_backward(flat, *f[:5], **given)
    assert torch.equal(r.ids.view(36, 5), f.ids) and torch.equal(wide.grad[..., 3:43].reshape(36, 40), want)
    assert not wide.grad[..., :3].any() and not wide.grad[..., 43:].any()
    out = torch.full((36, 47), 3.0, device="cuda", dtype=DT[dtype])
    assert A.route_topk_backward(flat, *f[:5], grad=out[:, 2:42], **given).data_ptr() == out[:, 2:].data_ptr()
    assert torch.equal(out[:, 2:42], want) and (out[:, :2] == 3).all() and (out[:, 42:] == 3).all()
    row = torch.randn(40, device="cuda").to(DT[dtype]).requires_grad_()
    r = A.route_topk(row.expand(6, 40), 5)
    (r.weights * g[0, :6]).sum().backward()
    alone = row.detach().requires_grad_()
    r = A.route_topk(alone, 5)
    each = [torch.autograd.grad((r.weights * w).sum(), alone, retain_graph=True)[0].float() for w in g[0, :6]]
    # the sum over the rows is torch's, in the type: an addition of 6 numbers rounds 6 times at most
    size = torch.stack(each).abs().sum(0)
    assert ((row.grad.float() - torch.stack(each).sum(0)).abs() <= 6 * size * torch.finfo(DT[dtype]).eps / 2 + 6 * size * 2.0 ** -24).all()


def test_training_step():
    """A layer of experts: routed, balanced, trained; against the same in 64 bits, automatic differentiation of both."""
    torch.manual_seed(1)
    T, D, E, k = 64, 24, 6, 2
    x = torch.randn(T, D)
    gate, w = torch.randn(D, E) * 0.3, torch.randn(E, D, D) * 0.2
    valid = torch.rand(T) < 0.9

    def loss_of(weights, ids, lse, balance, y):
        out = torch.zeros_like(y[0])
        for j in range(k):
            out = out + weights[:, j:j + 1].to(out.dtype) * y.gather(0, ids[:, j].clamp(min=0)[None, :, None].expand(1, T, D))[0]
        return (out ** 2).sum() / T + 0.01 * balance + 1e-3 * torch.where(lse > -1e30, lse, 0.0).square().sum() / T

    gd, wd = gate.cuda().requires_grad_(), w.cuda().requires_grad_()
    xd, vd = x.cuda(), valid.cuda()
    r = A.route_topk(xd @ gd, k, valid=vd, counts=True, balance=True)
    a = loss_of(r.weights, r.ids, r.lse, r.balance, torch.einsum("td,edf->etf", xd, wd))
    a.backward()
    g64, w64 = gate.double().requires_grad_(), w.double().requires_grad_()
    logits = (xd @ gd.detach()).cpu().double() + (x.double() @ g64 - (x.double() @ g64).detach())
    p = torch.softmax(logits, -1)
    ids = r.ids.cpu()
    chosen = p.gather(1, ids.clamp(min=0))
    weights = torch.where(valid[:, None], chosen / chosen.sum(-1, keepdim=True), 0.0)
    n = valid.sum()
    counts = torch.bincount(ids[valid].flatten(), minlength=E)
    assert torch.equal(counts, r.counts.cpu())
    balance = E * (counts / (k * n) * p[valid].sum(0) / n).sum()
    lse = torch.where(valid, torch.logsumexp(logits, -1), -float("inf"))
    lse = torch.where(valid, lse, torch.full_like(lse, -float("inf")))
    b = loss_of(weights, ids, lse, balance, torch.einsum("td,edf->etf", x.double(), w64))
    b.backward()
    assert abs(a.item() - b.item()) < 1e-4 * abs(b.item())
    assert (gd.grad.cpu() - g64.grad).norm() < 1e-4 * g64.grad.norm()
    assert (wd.grad.cpu() - w64.grad).norm() < 1e-4 * w64.grad.norm()


def test_backward_in_a_graph():
    x = torch.randn(500, 32, device="cuda", requires_grad=True)
    def step(leaf):
        r = A.route_topk(leaf, 4, balance=True)
        return torch.autograd.grad(r.weights.square().sum() + r.balance, leaf)[0]
    want = step(x)
    leaf = x.detach().clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(leaf)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(leaf)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_backward_on_another_stream():
    side = torch.cuda.Stream()
    x = torch.randn(700, 48, device="cuda", requires_grad=True)
    want = torch.autograd.grad(A.route_topk(x, 4, balance=True).balance * 5, x)[0]
    side.wait_stream(torch.cuda.current_stream())
    r = A.route_topk(x, 4, balance=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(torch.autograd.grad(r.balance * 5, x)[0], want)
    d = x.detach()
    side.wait_stream(torch.cuda.current_stream())
    got = A.route_topk_backward(d, None, r.ids, r.lse.detach(), r.counts, r.rows, grad_balance=torch.tensor(5.0, device="cuda"),
                                stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_weights_changed_in_place_are_noticed():
    x = torch.randn(20, 16, device="cuda", requires_grad=True)
    r = A.route_topk(x, 3)
    loss = r.weights.sum()
    with torch.no_grad():
        r.weights.mul_(2.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_only_some_outputs_are_used():
    """Gradients of the outputs that a loss leaves out are not asked for; counts and ids have none."""
    x = torch.randn(50, 16, device="cuda", requires_grad=True)
    r = A.route_topk(x, 3, counts=True, balance=True)
    assert not r.ids.requires_grad and not r.counts.requires_grad and not r.rows.requires_grad
    one = torch.autograd.grad(r.lse.sum(), x, retain_graph=True)[0]
    assert torch.allclose(one, torch.softmax(x.detach(), -1), atol=1e-6)
    two = torch.autograd.grad(r.weights[:, 0].sum(), x)[0]  # gradients that are not contiguous
    w = r.weights.detach()
    want = torch.zeros_like(x).scatter_(1, r.ids, -w[:, :1] * w)
    want.scatter_add_(1, r.ids[:, :1], w[:, :1])
    assert torch.allclose(two, want, atol=1e-6)


def test_refuses():
    x = torch.zeros(4, 10, device="cuda")
    r = A.route_topk(x, 2, balance=True)
    g = torch.zeros(4, 2, device="cuda")
    for call in (lambda: A.route_topk(x, 0), lambda: A.route_topk(x, 11), lambda: A.route_topk(x.double(), 2),
                 lambda: A.route_topk(x.t(), 2), lambda: A.route_topk(x, 2, valid=g[:, 0]), lambda: A.route_topk(x.cpu(), 2),
                 lambda: A.route_topk(torch.zeros(2, 1025, device="cuda"), 2), lambda: A.route_topk(torch.zeros(2, 64, device="cuda"), 33),
                 lambda: A.route_topk_backward(x, r.weights, r.ids, r.lse, grad_balance=r.balance),
                 lambda: A.route_topk_backward(x, None, r.ids, r.lse, grad_weights=g),
                 lambda: A.route_topk_backward(x, r.weights, r.ids, r.lse, grad_weights=g[:2]),
                 lambda: A.route_topk_backward(x, r.weights, r.ids, None, grad_weights=g),
                 lambda: A.route_topk_backward(x, r.weights, r.ids, r.lse, grad_weights=g, grad=x[:2])):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call()
