"""Beam selection and reordering on the GPU against the definitions in 64 bits,
at the sizes, strides and masks where they can go wrong, and a search made of both."""
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


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_wise_arg_gb300.build import build
    build()


def on_gpu(x, dtype, pad=0, offset=0):
    """(logits on the GPU, rounded to the type, the rounded values in 64 bits); what lies around them is NaN."""
    items, beams, cols = x.shape
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype])
    buf = torch.full((offset + items * beams * (cols + pad) + 64,), float("nan"), dtype=DT[dtype], device="cuda")
    view = buf[offset:offset + items * beams * (cols + pad)].view(items, beams, cols + pad)[..., :cols]
    view.copy_(t.cuda())
    return view, t.double().numpy()


def same(got, want, bound, what):
    assert (np.isnan(got) == np.isnan(want)).all() and (np.isinf(got) == np.isinf(want)).all(), (what, got, want)
    ok = np.isfinite(want)
    assert (got[~ok & ~np.isnan(want)] == want[~ok & ~np.isnan(want)]).all(), what
    off = np.abs(got[ok] - want[ok]) / bound
    assert off.size == 0 or off.max() <= 1, f"{what}: {off.max():.2f} times the bound"


def check(x, dtype, scores, count, ended=None, end_token=0, scale=None, temp=1.0, pad=0, offset=0):
    xd, x64 = on_gpu(x, dtype, pad, offset)
    scores = scores.astype(np.float32)
    cuda = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    scale32 = None if scale is None else scale.astype(np.float32)
    r = A.beam_select(xd, cuda(scores), count, ended=cuda(ended), end_token=end_token, scale=cuda(scale32), temperature=temp)
    tokens, parents, totals = (t.cpu().numpy() for t in r)
    assert tokens.shape == parents.shape == totals.shape == (*x.shape[:1], count)
    cols = x.shape[2]
    # what the kernel's binary32 sum makes of a total, and its rounding at the end
    each = logits_ref.sum_error(cols)
    for i in range(x.shape[0]):
        e, w = None if ended is None else ended[i], None if scale is None else scale32[i]
        want = ref.beam_select(x64[i], scores[i], count, e, end_token, w, temp)
        magnitude = np.abs(want[2][np.isfinite(want[2])]).max(initial=0.0)
        same(totals[i].astype(np.float64), want[2], each + 2 * logits_ref.U32 * magnitude, f"item {i}, totals")
        if want[3] is None:
            assert (tokens[i] == -1).all() and (parents[i] == -1).all()
            continue
        # where no other rank lies within the error, the places are decided
        ranks = np.concatenate((want[3], [want[4]]))
        with np.errstate(invalid="ignore"):
            gap = np.abs(np.diff(ranks))
        gap[np.isnan(gap)] = 0.0  # -inf beside -inf: the same emptiness
        near = 2 * each * (1.0 if w is None else w.max())
        # exact ties within a beam are decided by the index
        tie = np.zeros(len(gap), bool)
        tie[:-1] = want[1][1:] == want[1][:-1]
        tie[-1] = True if want[4] == -np.inf or x.shape[1] == 1 else False
        sure = (gap > near) | tie
        fixed = np.concatenate(([True], sure[:-1])) & sure
        fixed |= want[1] == -1
        assert fixed.mean() >= 0.5 or count <= 4, "the case decides too little"
        assert (tokens[i][fixed] == want[0][fixed]).all(), (i, tokens[i], want[0])
        assert (parents[i][fixed] == want[1][fixed]).all(), (i, parents[i], want[1])
    return r


def data(items, beams, cols, seed, spread=3.0):
    rng = np.random.Generator(np.random.PCG64(seed))
    x = rng.normal(0, spread, (items, beams, cols))
    scores = np.sort(-20 - 3 * rng.random((items, beams)), -1)[:, ::-1]
    return rng, x, scores


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("items,beams,cols,count,pad,offset", [
    (1, 1, 1, 1, 0, 0), (1, 1, 7, 7, 0, 1), (2, 3, 5, 15, 0, 0), (3, 2, 1, 2, 3, 1), (2, 4, 33, 8, 0, 3),
    (1, 4, 32000, 8, 0, 0), (3, 5, 1003, 10, 0, 1), (2, 3, 4999, 6, 13, 5), (70, 2, 513, 4, 0, 0), (2, 64, 300, 128, 0, 0),
    (5, 16, 40000, 32, 0, 0), (3, 17, 2048, 20, 0, 0), (200, 8, 2000, 16, 0, 0), (400, 3, 100, 6, 1, 0),
    (1, 16, 150001, 33, 0, 0), (40, 4, 70000, 64, 0, 0)])
def test_sizes(dtype, items, beams, cols, count, pad, offset):
    _, x, scores = data(items, beams, cols, items * 1000 + beams)
    check(x, dtype, scores, count, pad=pad, offset=offset)


def test_long_rows():
    """Rows of several segments, several CTAs to each of a few beams."""
    _, x, scores = data(1, 2, 2300001, 5)
    check(x, "bf16", scores, 8)


@pytest.mark.parametrize("dtype,cols", [("f32", 45001), ("bf16", 90000), ("f16", 82001)])
@pytest.mark.parametrize("items,beams,count", [(15, 16, 20), (14, 17, 9), (20, 32, 128)])
def test_many_long_rows(dtype, cols, items, beams, count):
    """Rows that a persistent kernel reads, some of them not to be looked at (and full of NaN)."""
    rng, x, scores = data(items, beams, cols, items)
    ended = rng.random((items, beams)) < 0.2
    x[ended] = np.nan
    scores[3, 4:] = -np.inf
    x[3, 4:] = np.nan
    scores[5] = -np.inf
    x[6][rng.random((beams, cols)) < 0.9999] = -np.inf
    x[7] = np.round(x[7])  # ties
    check(x, dtype, scores, count, ended=ended, end_token=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_ties_than_are_ranked(dtype):
    """Beams that all go on alike: more entries tie for the last places than the merge ranks by counting."""
    items, beams, cols, count = 3, 64, 512, 100
    x = torch.zeros(items, beams, cols, device="cuda", dtype=DT[dtype])
    x[1, :, 100:] = -20.0
    r = A.beam_select(x, torch.full((items, beams), -2.0, device="cuda"), count)
    assert r.tokens[0].tolist() == list(range(100)) and r.parents[0].tolist() == [0] * 100
    assert r.tokens[1].tolist() == list(range(100)) and r.parents[1].tolist() == [0] * 100
    scores = torch.linspace(0, -1e-3, beams, device="cuda").expand(items, beams).contiguous()
    r = A.beam_select(x, scores, count)  # and where their totals lie between
    assert r.tokens[0].tolist() == list(range(100)) and r.parents[2].tolist() == [0] * 100


@pytest.mark.parametrize("dtype,cols", [("f32", 45003), ("bf16", 90007)])
def test_ties_in_masses(dtype, cols):
    """Long rows of one value, of few, and of few near the end: first alternatives, ties by the index."""
    items, beams, k = 19, 16, 40
    x = torch.zeros(items, beams, cols, device="cuda", dtype=DT[dtype])
    g = torch.Generator(device="cuda").manual_seed(1)
    x[1::3] = torch.randint(0, 3, x[1::3].shape, device="cuda", generator=g).to(x.dtype)
    x[2::3, :, cols - 5000:] = torch.randint(0, 2, (6, beams, 5000), device="cuda", generator=g).to(x.dtype)
    x[4, 3] = -float("inf")
    x[4, 3, ::700] = 1.0
    want = torch.stack([torch.sort(x[i], dim=-1, descending=True, stable=True).indices[:, :k] for i in range(items)])
    got = A.token_logprobs(x.view(-1, cols), None, top_k=k)
    assert torch.equal(got.top_ids.view(items, beams, k), want)
    # one beam of each item has begun
    scores = torch.full((items, beams), -float("inf"), device="cuda")
    begun = torch.arange(items, device="cuda") % beams
    scores[torch.arange(items, device="cuda"), begun] = -1.0
    r = A.beam_select(x, scores, k)
    assert torch.equal(r.tokens, want[torch.arange(items, device="cuda"), begun])
    assert torch.equal(r.parents, begun[:, None].expand(items, k))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("beams,cols,count", [(1, 200003, 5), (2, 131072, 8), (2, 131072, 32), (2, 131080, 64), (4, 80001, 128), (3, 40000, 20)])
def test_order_within_a_beam_read_by_several_ctas(dtype, beams, cols, count):
    """Different logits whose totals round to the same binary64 value: the larger logit is first, wherever it lies."""
    g = torch.Generator(device="cuda").manual_seed(count)
    x = torch.randn(2, beams, cols, device="cuda", generator=g).to(DT[dtype])
    x[1, 0, cols // 3] = 1e30  # beside it, the other logits vanish
    scores = -torch.arange(2.0 * beams, device="cuda").view(2, beams)
    best = torch.sort(x.float(), dim=-1, descending=True, stable=True).indices[..., :count]
    r = A.beam_select(x, scores, count, temperature=1e30)  # all totals of a beam are alike
    assert torch.equal(r.tokens[0], best[0, 0]) and (r.parents[0] == 0).all()
    first = torch.full_like(scores, -np.inf)
    first[:, 0] = -1.0
    r = A.beam_select(x, first, count)
    assert torch.equal(r.tokens, best[:, 0]) and (r.parents == 0).all()
    # where the lists of other beams lie between
    for temperature in (1.0, 1e30):
        r = A.beam_select(x, scores, count, temperature=temperature)
        for i in range(2):
            for b in range(beams):
                mine = r.tokens[i][r.parents[i] == b]
                assert torch.equal(mine, best[i, b, :len(mine)]), (temperature, i, b)


@pytest.mark.parametrize("beams", [6, 7, 9, 10, 11, 12, 13, 14, 15])
def test_clusters_of_every_size(beams):
    """A cluster of as many CTAs as beams, up to the last item count that gets clusters, and one more."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    most = (2 if beams <= 8 else 1) * sms // beams
    for items in (1, 3, most, most + 1):
        rng, x, scores = data(items, beams, 900 + beams, items)
        ended = np.zeros((items, beams), bool)
        ended[np.arange(items), rng.integers(0, beams - 1, items)] = True
        ended[::3] = False
        scores[:, -1] = -np.inf  # has not begun
        x[:, -1] = np.nan
        check(x, "bf16" if beams % 2 else "f32", scores, 2 * beams, ended=ended, end_token=1)


@pytest.mark.parametrize("items", [100, 2100])
def test_logarithm_of_the_sum(items):
    """n logits of 0 and a total that is ln n but for its rounding to binary32: what comes out lies near 0, so the output's rounding
    hides nothing of the merge's logarithm, which is off by less than 3e-9 (beam_select.cuh). n is an exact binary32 sum."""
    cols = 100000
    rng = np.random.Generator(np.random.PCG64(items))
    n = rng.integers(1, cols + 1, items)
    edges = [1, 2, 3, 5, 43690, 43691, 87381, 87382, 21845, 21846, 65535, 65536, 99999, 100000]  # 2/3 of powers of two, and around
    n[:len(edges)] = edges
    nd = torch.from_numpy(n).cuda()
    x = torch.where(torch.arange(cols, device="cuda") < nd[:, None], 0.0, -np.inf).bfloat16()[:, None]
    s = np.log(n.astype(np.float64)).astype(np.float32)
    r = A.beam_select(x, torch.from_numpy(s).cuda()[:, None], 1)
    assert (r.tokens == 0).all() and (r.parents == 0).all()
    off = np.abs(r.scores[:, 0].double().cpu().numpy() - (s.astype(np.float64) - np.log(n.astype(np.float64))))
    assert off.max() < 3e-9, off.max()


def test_totals_below_the_range():
    """A total that binary32 holds as -inf, though it is a number: a place by its rank, and over in the next step."""
    x = torch.full((1, 2, 10), LOWEST["f32"], device="cuda")
    x[..., 7] = 5.0
    r = A.beam_select(x, torch.tensor([[-1.0, -1.5]], device="cuda"), 6, temperature=0.5)
    assert r.tokens.tolist() == [[7, 7, 0, 1, 2, 3]] and r.parents.tolist() == [[0, 1, 0, 0, 0, 0]]
    assert torch.isfinite(r.scores[0, :2]).all() and (r.scores[0, 2:] == -np.inf).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_options(dtype):
    rng, x, scores = data(6, 5, 3001, 7)
    ended = rng.random((6, 5)) < 0.4
    ended[0] = True
    ended[1] = False
    scores[2, 1:] = -np.inf
    scores[3] = -np.inf
    scale = (6.0 / (5.0 + rng.integers(1, 40, (6, 5)))) ** 0.8
    check(x, dtype, scores, 10, ended=ended, end_token=3000)
    check(x, dtype, scores, 10, ended=ended, end_token=2, scale=scale)
    check(x, dtype, scores, 10, scale=scale, temp=0.7)
    check(x, dtype, scores, 10, temp=2.5, pad=1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masks(dtype):
    """Grammars that leave few tokens or none, the type's lowest value as a mask, and NaN where nothing looks."""
    rng, x, scores = data(5, 4, 9001, 11)
    x[0][rng.random((4, 9001)) < 0.999] = -np.inf
    x[1] = -np.inf
    x[1, 2, 17] = 1.0
    x[2, 0] = -np.inf  # a beam without a continuation beside others
    x[3][:, 4:] = LOWEST[dtype]
    x[4][:] = LOWEST[dtype]
    check(x, dtype, scores, 8)
    x[0, 1] = np.nan  # ended
    x[2, 3] = np.inf  # has not begun
    ended = np.zeros((5, 4), bool)
    ended[0, 1] = True
    scores[2, 3] = -np.inf
    check(x, dtype, scores, 8, ended=ended, end_token=5)


@pytest.mark.parametrize("what", ["nan logit", "inf logit", "nan total", "inf total", "zero scale", "nan scale", "negative scale"])
def test_items_with_a_mistake(what):
    """Such an item says so, the others are as ever."""
    _, x, scores = data(3, 4, 5000, 13)
    scale = np.ones((3, 4))
    if "logit" in what:
        x[1, 2, 4321] = np.nan if "nan" in what else np.inf
    elif "total" in what:
        scores[1, 2] = np.nan if "nan" in what else np.inf
    else:
        scale[1, 2] = {"zero": 0.0, "nan": np.nan, "negative": -1.0}[what.split()[0]]
    r = check(x, "f32", scores, 8, scale=scale)
    assert torch.isnan(r.scores[1]).all() and not torch.isnan(r.scores[0]).any() and not torch.isnan(r.scores[2]).any()


@pytest.mark.parametrize("cols", [64, 4096, 4100])
def test_ties_go_to_the_lowest_beam_and_token(cols):
    """Equal beams over equal logits: everything ties."""
    x = torch.zeros(2, 4, cols, device="cuda", dtype=torch.bfloat16)
    x[1, :, 5] = 1.0
    r = A.beam_select(x, torch.full((2, 4), -1.0, device="cuda"), 6)
    assert r.tokens[0].tolist() == list(range(6)) and r.parents[0].tolist() == [0] * 6
    # Rows of 4100 elements start at different places between two 32-byte boundaries, so their exponentials are
    # summed in different groups: the binary32 sums of the same 4100 terms may differ by sum_error, and beams
    # whose totals are that close may come in either order. Rows of the other sizes all start on a boundary.
    assert r.tokens[1].tolist()[:4] == [5, 5, 5, 5]
    order = r.parents[1].tolist()
    assert sorted(order[:4]) == [0, 1, 2, 3] if cols % 16 else (order == [0, 1, 2, 3, 0, 0] and r.tokens[1].tolist()[4:] == [0, 1])
    assert (r.scores[1, :4] - r.scores[1, 0]).abs().max() <= 2 * logits_ref.sum_error(cols)
    r = A.beam_select(x, torch.full((2, 4), -1.0, device="cuda"), 6, ended=torch.ones(2, 4, dtype=torch.bool, device="cuda"),
                      end_token=9)
    assert r.tokens.tolist() == [[9] * 4 + [-1] * 2] * 2 and r.parents.tolist() == [[0, 1, 2, 3, -1, -1]] * 2
    assert r.scores.tolist() == [[-1.0] * 4 + [-np.inf] * 2] * 2


def test_shapes():
    """[beams, vocab] alone, more leading dimensions, no items, the same row for every beam."""
    x = torch.randn(3, 2, 4, 100, device="cuda")
    s = -torch.rand(3, 2, 4, device="cuda")
    whole = A.beam_select(x, s, 5)
    assert whole.tokens.shape == (3, 2, 5)
    one = A.beam_select(x[1, 1], s[1, 1], 5)
    assert all(torch.equal(a[1, 1], b) for a, b in zip(whole, one))
    none = A.beam_select(x[:0], s[:0], 5)
    assert none.tokens.shape == (0, 2, 5)
    row = torch.randn(100, device="cuda")
    first = torch.tensor([0.0, -np.inf, -np.inf, -np.inf], device="cuda")
    r = A.beam_select(row.expand(4, 100), first, 8)
    assert r.tokens.tolist() == row.topk(8).indices.tolist() and r.parents.tolist() == [0] * 8


def test_other_stream_and_graph():
    _, x, scores = data(4, 4, 20011, 17)
    xd, s = torch.from_numpy(x).float().cuda(), torch.from_numpy(scores.copy()).float().cuda()
    want = A.beam_select(xd, s, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = A.beam_select(xd, s, 8, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    state = torch.randn(16, 3, 50, device="cuda")
    first = state.clone()
    with torch.cuda.stream(side):
        parents = want.parents[:, :4].contiguous()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = A.beam_select(xd, s, 8)
            A.beam_reorder(state, parents)
    state.copy_(first)
    xd += 1.0  # shifts nothing
    for _ in range(3):
        state.copy_(first)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.tokens, want.tokens) and torch.equal(got.parents, want.parents)
        assert torch.equal(state.cpu(), torch.from_numpy(ref.reorder(first.view(4, 4, 3, 50).cpu().numpy(), parents.cpu().numpy())).view(16, 3, 50))


def test_calls_at_once():
    """Two steps with scratch and two without, on two streams at a time, are each as they are alone."""
    work = [(20, 17, 30000, 24), (400, 3, 500, 6), (2, 4, 32000, 8), (15, 16, 90000, 20)]
    given = []
    for i, (items, beams, cols, count) in enumerate(work):
        g = torch.Generator(device="cuda").manual_seed(i)
        given.append((torch.randn(items, beams, cols, device="cuda", generator=g).bfloat16(),
                      torch.randn(items, beams, device="cuda", generator=g), count))
    want = [A.beam_select(*a) for a in given]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for turn in range(8):
        for i, a in enumerate(given):
            got.append((i, A.beam_select(*a, stream=streams[(i + turn) % 2])))
    torch.cuda.synchronize()
    for i, r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want[i])), i


def test_offsets_past_32_bits():
    """Rows and states whose parts begin beyond 2^31 elements."""
    stride = (1 << 30) + 64
    buf = torch.empty(3 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, 2, 2000), (2 * stride, stride, 1))
    near = torch.randn(2, 2, 2000, device="cuda").bfloat16()
    x.copy_(near)
    scores = torch.tensor([[-1.0, -1.5], [-2.0, -1.9]], device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(A.beam_select(x, scores, 9), A.beam_select(near, scores, 9)))
    parents = torch.tensor([[1, 0], [1, 1]], device="cuda")
    A.beam_reorder(x, parents)
    assert torch.equal(x, torch.stack([near[0].flip(0), near[1][[1, 1]]]))
    x.copy_(near)
    cut = x[:, :, 3:1996]  # unaligned
    A.beam_reorder(cut, parents, torch.tensor([1993, 1000], device="cuda"), dim=2)
    want = near.clone()
    want[0, :, 3:1996] = near[0].flip(0)[:, 3:1996]
    want[1, 0, 3:1003] = near[1, 1, 3:1003]
    assert torch.equal(x, want)


# -- reordering -------------------------------------------------------------------------------
PARENTS = {
    "stay": lambda rng, i, b: np.tile(np.arange(b), (i, 1)),
    "first": lambda rng, i, b: np.zeros((i, b), int),
    "round": lambda rng, i, b: np.tile(np.roll(np.arange(b), 1), (i, 1)),
    "random": lambda rng, i, b: rng.integers(0, b, (i, b)),
    "some": lambda rng, i, b: np.where(rng.random((i, b)) < 0.3, rng.choice([-1, -5, b, b + 7, 2**40]), rng.integers(0, b, (i, b))),
}


def filled(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    raw = torch.randint(0, 256, (max(n, 1),), dtype=torch.uint8, generator=g)[:n]
    return raw.view(dtype).view(shape) if n else torch.empty(shape, dtype=dtype)


def bits(t):
    return t.contiguous().cpu().view(torch.uint8).numpy()


def reference(t, parents, lengths, dim, items, beams):
    """The state after it, on the CPU, bytes of each element last."""
    c = t.contiguous().cpu()
    raw = c.view(torch.uint8).view(items, beams, *c.shape[1:], -1).numpy()
    return ref.reorder(raw, parents, lengths, None if dim is None else dim + 1)


@pytest.mark.parametrize("kind", PARENTS)
@pytest.mark.parametrize("items,beams,shape,dtype", [
    (1, 2, (1,), torch.int64), (3, 4, (2, 10, 16), torch.bfloat16), (2, 5, (3, 77, 33), torch.float32),
    (4, 3, (1, 513, 1), torch.int64), (2, 8, (2, 100, 64), torch.float16), (5, 11, (7, 3), torch.uint8),
    (1, 16, (4, 130, 128), torch.bfloat16), (2, 32, (1, 65, 24), torch.float32), (3, 33, (2, 9, 40), torch.float64),
    (2, 64, (3, 50, 17), torch.bfloat16), (300, 4, (5, 7), torch.int32), (1, 4, (2, 3000, 128), torch.bfloat16)])
def test_reorder(kind, items, beams, shape, dtype):
    rng = np.random.Generator(np.random.PCG64(beams))
    parents = PARENTS[kind](rng, items, beams).astype(np.int64)
    host = filled((items * beams, *shape), dtype, 3)
    p = torch.from_numpy(parents).cuda()
    for dim in (None, 2) if len(shape) == 3 else (None,):
        lengths = None if dim is None else rng.integers(-1, shape[1] + 3, items)
        t = host.cuda()
        n = None if lengths is None else torch.from_numpy(lengths).cuda()
        out = A.beam_reorder(t, p, n, dim=dim)
        assert out is t
        want = reference(host, parents, lengths, dim, items, beams)
        assert (bits(t).reshape(want.shape) == want).all()


def test_reorder_views():
    """Keys beside values in one buffer, unaligned and padded states, several kinds in one call, [batch, beams, ...]."""
    items, beams = 3, 4
    rng = np.random.Generator(np.random.PCG64(1))
    parents = rng.integers(-1, beams, (items, beams))
    lengths = rng.integers(0, 21, items)
    p, n = torch.from_numpy(parents).cuda(), torch.from_numpy(lengths).cuda()
    kv = filled((items * beams, 2, 5, 20, 9), torch.bfloat16, 5)
    odd = filled((1 + items * beams * 70,), torch.uint8, 6)
    wide = filled((items, beams, 6, 20, 12), torch.float32, 7)
    packed = filled((items * beams, 100), torch.float16, 8)
    tensors = [t.clone().cuda() for t in (kv, odd, wide, packed)]
    views = lambda ts: [ts[0][:, 0], ts[0][:, 1], ts[1][1:].view(items * beams, 70)[:, :60].view(items * beams, 3, 20),  # noqa: E731
                        ts[2][:, :, 1:4], ts[3][:, :20].unsqueeze(1), ts[3][:, 20:40].unsqueeze(1)]
    group = views(tensors)
    for i, dim in ((0, 2), (1, 2), (2, 2), (3, 3), (4, 2), (5, 2)):
        A.beam_reorder(group[i], p, n, dim=dim)
    host = [t.clone() for t in (kv, odd, wide, packed)]
    for view, dim in zip(views(host), (1, 1, 1, 2, 1, 1)):
        flat = view.reshape(items * beams, *view.shape[1 if view.shape[0] == items * beams else 2:])
        raw = torch.from_numpy(reference(flat, parents, lengths, 2, items, beams)).contiguous().view(view.dtype)
        view.copy_(raw.view(view.shape))
    for got, want in zip(tensors, host):
        assert (bits(got) == bits(want)).all()
    # the same in one call
    tensors = [t.clone().cuda() for t in (kv, odd, wide, packed)]
    group = views(tensors)
    group[3] = group[3].flatten(0, 1) if group[3].is_contiguous() else group[3]
    A.beam_reorder([group[0], group[1], group[2], group[4], group[5]], p, n, dim=2)
    A.beam_reorder([group[3]], p, n, dim=3)
    for got, want in zip(tensors, host):
        assert (bits(got) == bits(want)).all()


def test_reorder_nothing():
    """No items, no states, empty states, one beam; and what is refused is refused before anything has moved."""
    p = torch.tensor([[1, 0]], device="cuda")
    assert A.beam_reorder([], p) == []
    empty = torch.zeros(2, 0, 5, device="cuda")
    assert A.beam_reorder(empty, p, torch.tensor([3], device="cuda"), dim=1) is empty
    A.beam_reorder(torch.zeros(0, 3, device="cuda"), p[:0])
    one = torch.arange(6.0, device="cuda").view(3, 2)
    A.beam_reorder(one, torch.tensor([[0], [-1], [5]], device="cuda"))
    assert one.tolist() == [[0, 1], [2, 3], [4, 5]]
    a, b = torch.arange(4.0, device="cuda").view(2, 2), torch.arange(12.0, device="cuda").view(2, 6)
    with pytest.raises(RuntimeError):
        A.beam_reorder([a, b, b[:, :]], p)
    with pytest.raises(ValueError):
        A.beam_reorder([a, b, b[:, 2:5]], p)
    assert a.tolist() == [[0, 1], [2, 3]]
    A.beam_reorder([a, b[:, :2], b[:, 4:]], p)
    assert a.tolist() == [[2, 3], [0, 1]] and b.tolist() == [[6, 7, 2, 3, 10, 11], [0, 1, 8, 9, 4, 5]]


def test_reorder_many_items():
    """More items than a CTA plans at once, lengths of every size, short segments."""
    rng = np.random.Generator(np.random.PCG64(8))
    for items, beams in ((100, 3), (77, 20)):
        parents = rng.integers(-1, beams, (items, beams))
        lengths = rng.integers(0, 8, items)
        host = filled((items * beams, 9, 7, 3), torch.bfloat16, 2)
        t = host.cuda()
        A.beam_reorder(t, torch.from_numpy(parents).cuda(), torch.from_numpy(lengths).cuda(), dim=-2)
        want = reference(host, parents, lengths, 2, items, beams)
        assert (bits(t).reshape(want.shape) == want).all()


def test_reorder_many_states():
    """More states than a launch takes."""
    p = torch.tensor([[1, 0, 0]], device="cuda")
    states = [torch.arange(6.0, device="cuda").view(3, 2) + i for i in range(300)]
    A.beam_reorder(states, p)
    for i, s in enumerate(states):
        assert s.tolist() == [[2.0 + i, 3.0 + i], [i, 1.0 + i], [i, 1.0 + i]]


def test_reorder_on_another_stream():
    side = torch.cuda.Stream()
    host = filled((12, 3, 50, 8), torch.float32, 4)
    parents = np.array([[1, 0, 3, 3], [2, 2, 2, 2], [0, -1, 1, 9]])
    t, p = host.cuda(), torch.from_numpy(parents).cuda()
    side.wait_stream(torch.cuda.current_stream())
    assert A.beam_reorder([t], p, stream=side)[0] is t
    side.synchronize()
    want = reference(host, parents, None, None, 3, 4)
    assert (bits(t).reshape(want.shape) == want).all()


def test_reorder_counts_as_a_change():
    """What automatic differentiation saved of a state is not what it holds any more."""
    t = torch.randn(4, 6, device="cuda")
    leaf = torch.randn(4, 6, device="cuda", requires_grad=True)
    loss = (leaf * t).sum()
    A.beam_reorder(t, torch.tensor([[1, 0, 2, 3]], device="cuda"))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        u = torch.ones(2, 3, device="cuda")
        A.beam_reorder([u], torch.tensor([[1, 1]], device="cuda"))


def test_reorder_refuses():
    t = torch.zeros(6, 4, 8, device="cuda")
    p = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    n = torch.zeros(2, dtype=torch.int64, device="cuda")
    for call in (lambda: A.beam_reorder([t, t], p), lambda: A.beam_reorder([t, t[:, 1:3]], p), lambda: A.beam_reorder(t[:5], p),
                 lambda: A.beam_reorder(t, p, n), lambda: A.beam_reorder(t, p, n, dim=0), lambda: A.beam_reorder(t, p, n, dim=3),
                 lambda: A.beam_reorder(t.transpose(1, 2), p, n, dim=1), lambda: A.beam_reorder(t, p.int()),
                 lambda: A.beam_reorder(t, p[0]), lambda: A.beam_reorder(t.cpu(), p), lambda: A.beam_reorder(t, p, n[:1], dim=1),
                 lambda: A.beam_reorder(t[:1].expand(6, 4, 8), p), lambda: A.beam_reorder(t.requires_grad_(), p)):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call()


def test_select_refuses():
    x, s = torch.zeros(2, 3, 10, device="cuda"), torch.zeros(2, 3, device="cuda")
    for call in (lambda: A.beam_select(x, s, 0), lambda: A.beam_select(x, s, 31), lambda: A.beam_select(x, s[:1], 2),
                 lambda: A.beam_select(x, s.double(), 2), lambda: A.beam_select(x.double(), s, 2), lambda: A.beam_select(x, s.cpu(), 2),
                 lambda: A.beam_select(x.transpose(1, 2), s, 2), lambda: A.beam_select(x, None, 2),
                 lambda: A.beam_select(x, s, 2, ended=s), lambda: A.beam_select(x, s, 2, temperature=0.0),
                 lambda: A.beam_select(x[0, 0], s[0, 0], 2), lambda: A.beam_select(x.requires_grad_(), s, 2),
                 lambda: A.beam_select(torch.zeros(65, 9, device="cuda"), torch.zeros(65, device="cuda"), 2)):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            call()


def test_tangents_of_the_other_arguments_are_refused():
    import torch.autograd.forward_ad as fwd
    x, s = torch.randn(2, 3, 20, device="cuda"), torch.zeros(2, 3, device="cuda")
    ones = torch.ones(2, 3, device="cuda")
    y = torch.randn(6, 20, device="cuda")
    r = A.route_topk(y, 2, balance=True)
    t = A.token_logprobs(y, torch.zeros(6, dtype=torch.int64, device="cuda"), with_stats=True)
    one, two, loss = torch.ones(6, device="cuda"), torch.ones(6, 2, device="cuda"), torch.ones((), device="cuda")
    with fwd.dual_level():
        dual = lambda v: fwd.make_dual(v, torch.ones_like(v))  # noqa: E731
        back = lambda weights=r.weights, lse=r.lse, **g: A.route_topk_backward(y, weights, r.ids, lse, r.counts, r.rows, **g)  # noqa: E731
        for call in (lambda: A.beam_select(x, dual(s), 2), lambda: A.beam_select(x, s, 2, scale=dual(ones)),
                     lambda: back(weights=dual(r.weights), grad_weights=two), lambda: back(lse=dual(r.lse), grad_lse=one),
                     lambda: back(grad_weights=dual(two)), lambda: back(grad_lse=dual(one)), lambda: back(grad_balance=dual(loss)),
                     lambda: A.token_logprobs_backward(y, None, t.stats, grad_lse=dual(one)),
                     lambda: A.distill_topk(y, r.ids, dual(two))):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
        # and without a tangent all is as ever
        A.beam_select(x, s, 2, scale=ones)
        assert torch.equal(back(grad_lse=one), A.route_topk_backward(y, r.weights, r.ids, r.lse, grad_lse=one))


@pytest.mark.parametrize("items,beams", [(1, 2), (4, 4), (1, 16), (20, 17)])
def test_scratch_is_what_the_library_asks_for(monkeypatch, items, beams):
    """Also for few rows: which steps need scratch is the library's plan alone."""
    from row_wise_arg_gb300 import beam
    asked, given = [], []

    class Library:
        def __getattr__(self, name):
            return getattr(beam_lib, name)

        def argreduce_beam_scratch_bytes(self, *a):
            asked.append(a)
            return beam_lib.argreduce_beam_scratch_bytes(*a) + 4096

        def argreduce_beam_select(self, *a):
            given.append(a[-3:-1])
            return beam_lib.argreduce_beam_select(*a)

    beam_lib = beam._LIB
    x, s = torch.randn(items, beams, 700, device="cuda"), -torch.rand(items, beams, device="cuda")
    want = A.beam_select(x, s, 4)
    beam._scratch_bytes.cache_clear()
    monkeypatch.setattr(beam, "_LIB", Library())
    got = A.beam_select(x, s, 4)
    beam._scratch_bytes.cache_clear()
    need = beam_lib.argreduce_beam_scratch_bytes(items, beams, 700, 0, 4) + 4096
    assert asked and given[0][0] and given[0][1] == need
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("temp", [1e-3, 1e4, 1e-38, 1e38])
def test_temperatures(dtype, temp):
    """Far from 1, up to where log2(e) / T is still a number."""
    items, beams, cols = 2, 3, 40000
    _, x, scores = data(items, beams, cols, 23)
    x[:, :, 7] = 30.0  # one largest
    if 1e-5 < temp < 1e5:
        check(x, dtype, scores, 6, temp=temp)
        return
    xd, x64 = on_gpu(x, dtype)
    s = torch.from_numpy(scores.copy()).float().cuda()
    r = A.beam_select(xd, s, 6, temperature=temp)
    if temp < 1.0:  # all of a beam's probability is its largest's
        assert (r.tokens[:, :3] == 7).all() and (r.parents[:, :3] == torch.arange(3, device="cuda")).all()
        assert torch.equal(r.scores[:, :3], s)
    else:  # all tokens alike
        want = scores.astype(np.float32)[:, :1].astype(np.float64) - np.log(cols)
        assert (r.parents == 0).all() and (np.abs(r.scores.double().cpu().numpy() - want) <= logits_ref.sum_error(cols) + 4e-6).all()
        assert torch.equal(r.tokens, torch.sort(xd[:, 0].float(), dim=-1, descending=True, stable=True).indices[:, :6])


def test_many_items():
    """More items than a grid's second dimension would take, one beam and several."""
    for items, beams, cols in ((70001, 1, 9), (66000, 3, 5)):
        g = torch.Generator(device="cuda").manual_seed(items)
        x = torch.randn(items, beams, cols, device="cuda", generator=g)
        s = torch.zeros(items, beams, device="cuda") - torch.arange(beams, device="cuda") * 100.0
        r = A.beam_select(x, s, 4)
        want = torch.sort(x[:, 0], dim=-1, descending=True, stable=True).indices[:, :4]
        assert torch.equal(r.tokens, want) and (r.parents == 0).all()
        lp = torch.log_softmax(x[:, 0].double(), -1).gather(1, want)
        assert (r.scores.double() - lp).abs().max() <= logits_ref.sum_error(cols) + 8 * logits_ref.U32 * lp.abs().max().item()
        state, parents = torch.arange(items * beams, device="cuda").view(items, beams).clone(), (r.parents[:, :1] + beams - 1).expand(items, beams).contiguous()
        A.beam_reorder(state, parents)
        assert (state == state[:, -1:]).all() and torch.equal(state[:, 0] // beams, torch.arange(items, device="cuda"))


def test_graphs_beside_one_another():
    """Two captured steps with scratch, replayed at the same time on two streams."""
    given = []
    for i in range(2):
        g = torch.Generator(device="cuda").manual_seed(i)
        given.append((torch.randn(30, 17, 5000, device="cuda", generator=g), torch.randn(30, 17, device="cuda", generator=g), 12))
    want = [A.beam_select(*a) for a in given]
    side, sides, graphs, got = torch.cuda.Stream(), [torch.cuda.Stream(), torch.cuda.Stream()], [], []
    for a in given:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            got.append(A.beam_select(*a))
    for _ in range(20):
        for g, st in zip(graphs, sides):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.bool, torch.complex128, torch.complex64, torch.float8_e4m3fn, torch.int16])
def test_reorder_of_other_types(dtype):
    """What a state's elements are does not matter: their bytes move. Several types in one call."""
    p = torch.tensor([[1, 0, 3, 2], [2, 2, -1, 0]], device="cuda")
    n = torch.tensor([5, 3], device="cuda")
    raw = filled((8, 3, 6, 7, torch.empty(0, dtype=dtype).element_size()), torch.uint8, 9)
    if dtype is torch.bool:
        raw = raw & 1
    t, other = raw.cuda(), filled((8, 2, 6, 4), torch.bfloat16, 10).cuda()
    first = other.clone()
    A.beam_reorder([t.view(dtype).squeeze(-1), other], p, n, dim=2)
    want = ref.reorder(raw.view(2, 4, 3, 6, 7, -1).numpy(), p.cpu().numpy(), n.cpu().numpy(), 3)
    assert (t.cpu().numpy().reshape(want.shape) == want).all()
    want = reference(first, p.cpu().numpy(), n.cpu().numpy(), 2, 2, 4)
    assert (bits(other).reshape(want.shape) == want).all()


@pytest.mark.parametrize("graph", [False, True])
def test_search(graph):
    """A whole search: a model whose logits are a function of the last two tokens, its states reordered and
    written to each step. The best sequences are those of a search written plainly in 64 bits, and every
    beam's states are those of its own sequence."""
    vocab, items, beams, steps, end = 199, 3, 4, 12, 0
    g = torch.Generator("cuda").manual_seed(3)
    table = torch.randn(vocab, vocab, device="cuda", generator=g) * 2.0
    table[:, end] += 2.5
    first = torch.tensor([5, 9, 11], device="cuda")
    # the search by the operators
    history = torch.full((items, beams, steps + 1), -1, device="cuda")
    history[:, :, 0] = first[:, None]
    cache = torch.zeros(items * beams, 2, steps + 1, 3, device="cuda")
    cache[:, :, 0] = history[:, :, 0].flatten()[:, None, None]
    totals = torch.full((items, beams), -np.inf, device="cuda")
    totals[:, 0] = 0.0
    ended = torch.zeros(items, beams, dtype=torch.bool, device="cuda")
    length = torch.zeros(items, dtype=torch.int64, device="cuda")
    at = torch.ones((), dtype=torch.int64, device="cuda")

    def step():
        last = history.gather(2, (at - 1).expand(items, beams, 1))[..., 0].clamp(min=0)
        r = A.beam_select(table[last], totals, beams, ended=ended, end_token=end)
        length.copy_(at.expand(items))
        A.beam_reorder([history.unsqueeze(2)], r.parents, length, dim=3)
        A.beam_reorder(cache, r.parents, length, dim=2)
        history.scatter_(2, at.expand(items, beams, 1), r.tokens[..., None])
        cache.scatter_(2, at.expand(items * beams, 2, 1, 3), r.tokens.flatten()[:, None, None, None].expand(-1, 2, 1, 3).float())
        ended.copy_((ended.gather(1, r.parents.clamp(min=0)) | (r.tokens == end)) & (r.tokens >= 0))
        totals.copy_(r.scores)
        at.add_(1)

    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        recorded = torch.cuda.CUDAGraph()
        with torch.cuda.graph(recorded):
            step()
        for _ in range(steps - 1):
            recorded.replay()
    else:
        for _ in range(steps):
            step()
    # plainly
    lp = torch.log_softmax(table.double(), -1).cpu().numpy()
    for i in range(items):
        alive = [((int(first[i]),), 0.0, False)]
        for _ in range(steps):
            found = []
            for seq, total, over in alive:
                if over:
                    found.append((seq + (end,), total, True))
                else:
                    found += [(seq + (v,), total + lp[seq[-1], v], v == end) for v in range(vocab)]
            found.sort(key=lambda f: -f[1])
            alive = found[:beams]
        assert [tuple(h) for h in history[i].tolist()] == [a[0] for a in alive]
        assert np.allclose(totals[i].cpu().numpy(), [a[1] for a in alive], atol=1e-4)
        assert ended[i].tolist() == [a[2] for a in alive]
        kept = cache.view(items, beams, 2, steps + 1, 3)[i]
        assert torch.equal(kept, history[i][:, None, :, None].expand_as(kept).float())
