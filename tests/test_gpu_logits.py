"""Vocabulary-row operators on the GPU against the definitions in 64 bits:
log probabilities, entropy, top alternatives and the distillation loss, and
their gradients, at the sizes, strides and masks where they can go wrong. The
bounds come from logits_ref (derived there); indices are compared exactly."""
import numpy as np
import pytest

import logits_ref as ref

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

import row_wise_arg_gb300 as A  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}
CAPS = A.make_caps(152)


@pytest.fixture(scope="module", autouse=True)
def built():
    from row_wise_arg_gb300.build import build
    build()


def on_gpu(x, dtype, pad=0, offset=0):
    """(rows on the GPU, rounded to the type, the rounded values in 64 bits). The rows lie `pad` elements apart in a
    buffer that starts `offset` elements in; every other element is a NaN that a stray read would show."""
    rows, cols = x.shape
    t = torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype])
    buf = torch.full((offset + rows * (cols + pad) + 64,), float("nan"), dtype=DT[dtype], device="cuda")
    view = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(t.cuda())
    return view, t.double().numpy()


def close(got, want, bound, what):
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert (np.isnan(got) == np.isnan(want)).all(), f"{what}: NaNs at {np.argwhere(np.isnan(got) != np.isnan(want))[:4]}"
    bound = np.broadcast_to(bound, want.shape)
    inf = np.isinf(want)
    with np.errstate(invalid="ignore"):
        # a value that lies within the bound of binary32's largest may come out infinite
        over = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + bound > np.finfo(np.float32).max)
    assert (got[inf] == want[inf]).all() and not np.isinf(got[~inf & ~over]).any(), f"{what}: infinities"
    ok = np.isfinite(want) & ~over
    off = np.abs(got[ok] - want[ok]) / bound[ok]
    assert off.size == 0 or off.max() <= 1.0, f"{what}: {off.max():.2f} times the bound, at {np.argmax(off)}"


def check_logprobs(x, dtype, tokens=None, k=0, temp=1.0, plan=None, pad=0, offset=0):
    xd, x64 = on_gpu(x, dtype, pad, offset)
    rows, cols = x.shape
    tok = torch.from_numpy(tokens).cuda() if tokens is not None else None
    r = A.token_logprobs(xd, tok, k, temperature=temp, plan=plan)
    want = ref.logprobs(x64, tokens, k, temp)
    lnv = np.log(cols)
    close(r.lse, want["lse"], ref.logprob_bound(want["lse"], cols), "lse")
    close(r.entropy, want["entropy"], ref.entropy_bound(want["entropy"], lnv, cols), "entropy")
    if tokens is not None:
        close(r.logprob, want["logprob"], ref.logprob_bound(want["logprob"], cols), "logprob")
    else:
        assert r.logprob is None
    if k:
        np.testing.assert_array_equal(r.top_ids.cpu().numpy(), want["top_ids"])
        close(r.top_logprobs, want["top_logprobs"], ref.logprob_bound(want["top_logprobs"], cols), "top_logprobs")
    return r, x64


def check_logprobs_grad(x, dtype, tokens, temp=1.0, plan=None, pad=0, offset=0, in_place=False, out_pad=0, seed=0):
    rng = np.random.default_rng(seed)
    rows, cols = x.shape
    g, h, c = (rng.normal(size=rows).astype(np.float32) for _ in range(3))
    xd, x64 = on_gpu(x, dtype, pad, offset)
    tok = torch.from_numpy(tokens).cuda()
    r = A.token_logprobs(xd, tok, temperature=temp, with_stats=True)
    out = None
    if in_place:
        out = xd
    elif out_pad:
        out = torch.full((rows, cols + out_pad), 7.0, dtype=DT[dtype], device="cuda")[:, :cols]
    got = A.token_logprobs_backward(xd, tok, r.stats, *(torch.from_numpy(v).cuda() for v in (g, h, c)),
                                    temperature=temp, grad=out, plan=plan)
    want = ref.logprobs_grad(x64, tokens, g.astype(np.float64), h.astype(np.float64), c.astype(np.float64), temp)
    p = np.exp(ref.log_probs(x64, temp))
    with np.errstate(invalid="ignore"):
        lp = np.where(p > 0, np.abs(ref.log_probs(x64, temp)), 0.0)
    ent = ref.logprobs(x64, temp=temp)["entropy"][:, None]
    # the terms that a gradient element is the sum of; log p is off by logprob_bound, the entropy by entropy_bound
    terms = p * (np.abs(g)[:, None] + np.abs(c)[:, None] + np.abs(h)[:, None] * (lp + ent + 3 + 6 * np.log(cols + 1)))
    named = (np.arange(cols)[None] == tokens[:, None])
    terms = (terms * (1 + lp) + named * np.abs(g)[:, None]) / temp
    close(got, want, ref.grad_bound(want, np.nan_to_num(terms), cols, dtype), "grad")
    if out_pad:
        whole = got.as_strided((rows, cols + out_pad), (cols + out_pad, 1))
        assert (whole[:, cols:] == 7.0).all(), "the padding between the gradient's rows was written"
    if pad and in_place:
        assert torch.isnan(xd.as_strided((rows, cols + pad), (cols + pad, 1))[:, cols:]).all()


def slots_for(rng, rows, cols, slots, tail, absent=0.0):
    ids = np.stack([rng.permutation(cols)[:slots] if cols >= slots else
                    np.concatenate([rng.permutation(cols), np.full(slots - cols, -1)]) for _ in range(rows)])
    if absent:
        ids[rng.random(ids.shape) < absent] = -5
    if tail:
        val = np.log(rng.dirichlet(np.full(slots + 1, 0.5), rows)[:, :slots] + 1e-12)
    else:
        val = rng.normal(0, 3, (rows, slots))
    return ids.astype(np.int64).reshape(rows, slots), val.astype(np.float32).reshape(rows, slots)


def check_distill(x, dtype, ids, val, temp=1.0, tail=False, plan=None, grad_plan=None, step_plan=None, pad=0,
                  offset=0, in_place=False, out_pad=0, seed=0):
    """Forward, backward and both at once."""
    rng = np.random.default_rng(seed)
    rows, cols = x.shape
    g = rng.normal(size=rows).astype(np.float32)
    xd, x64 = on_gpu(x, dtype, pad, offset)
    i, v, gd = torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda(), torch.from_numpy(g).cuda()
    want, wgrad = ref.distill(x64, ids, val, temp, tail, g.astype(np.float64))
    kw = dict(temperature=temp, tail=tail)
    r = A.distill_topk(xd, i, v, plan=plan, with_stats=True, **kw)
    slots = max(1, ids.shape[1])
    # |loss| is at most what its terms add up to: q |ln q| <= ln slots + 1, q |ln p| <= the largest |ln p| of a slot
    lp = ref.log_probs(x64, temp)
    big = np.zeros(rows)
    dense = np.zeros(rows)
    for k in range(rows):
        here = (ids[k] >= 0) & (ids[k] < cols)
        s = lp[k][ids[k][here]]
        s = s[np.isfinite(s)]
        big[k] = 2 * (np.abs(s).max() if len(s) else 0.0) + np.log(slots) + 3
        t = ref.teacher(ids[k], val[k], cols, temp, tail)
        if t is not None and t[2] > 0:
            other = np.ones(cols, bool)
            other[ids[k][here]] = False
            mass = np.exp(lp[k])[other].sum()
            big[k] += t[2] * (abs(np.log(t[2])) + (abs(np.log(mass)) if mass > 0 else 0.0) + 8 + 8 / np.sqrt(t[2]))
            dense[k] = t[2] / mass if mass > 0 else 0.0
            if t[0].sum() >= 1 - 1e-4:  # what is left of 1 is all rounding
                big[k] += 100
                dense[k] += U_REST / max(mass, 1e-30)
    lbound = ref.logprob_bound(want, cols) + ref.sum_error(cols) * big
    close(r.loss, want, lbound, "loss")

    p = np.exp(lp)
    with np.errstate(invalid="ignore"):
        y = np.where(p > 0, np.abs(lp), 0.0)
    q = np.zeros_like(p)
    for k in range(rows):
        t = ref.teacher(ids[k], val[k], cols, temp, tail)
        if t is not None:
            here = ids[k] >= 0
            q[k][ids[k][here]] = np.where(t[0] > 0, t[0] * (2 + np.abs(np.where(t[0] > 0, t[1], 0.0))), 0.0)[here]
    terms = np.nan_to_num((p * (1 + y) * (1 + dense[:, None]) + q) * np.abs(g)[:, None] / temp)
    gbound = ref.grad_bound(wgrad, terms, cols, dtype)

    def out():
        if in_place:
            return on_gpu(x, dtype, pad, offset)[0]
        return torch.full((rows, cols + out_pad), 7.0, dtype=DT[dtype], device="cuda")[:, :cols] if out_pad else None
    for both in (False, True):
        o = out()
        src = o if in_place else xd
        if both:
            loss, got = A.distill_topk_step(src, i, v, gd, grad=o, plan=step_plan, **kw)
            close(loss, want, lbound, "step's loss")
        else:
            got = A.distill_topk_backward(src, i, v, r.stats, gd, grad=o, plan=grad_plan, **kw)
        close(got, wgrad, gbound, "step's grad" if both else "grad")
        if out_pad and not in_place:
            whole = got.as_strided((rows, cols + out_pad), (cols + out_pad, 1))
            assert (whole[:, cols:] == 7.0).all(), "the padding between the gradient's rows was written"


U_REST = 4 * 1024 * ref.U32  # a sum of up to 1024 slots near 1

SHAPES = [(1, 1), (3, 2), (5, 7), (2, 31), (4, 33), (7, 64), (70, 127), (2, 1000), (3, 4099), (2, 32000), (1, 65537),
          (160, 5001), (1, 202048), (2, 300007)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_logprobs_shapes(dtype, shape):
    rows, cols = shape
    rng = np.random.default_rng(rows * 1000 + cols)
    x = rng.normal(0, 3, shape).astype(np.float32)
    tokens = rng.integers(0, cols, rows)
    tokens[rng.random(rows) < 0.2] = -1
    for k, temp in ((0, 1.0), (1, 0.7), (5, 2.0), (20, 1.0), (128, 1.0)):
        check_logprobs(x, dtype, tokens, min(k, cols), temp)
    check_logprobs(x, dtype, None, min(3, cols))
    check_logprobs_grad(x, dtype, tokens)
    check_logprobs_grad(x, dtype, tokens, temp=0.7, in_place=True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (5, 3), (16, 8), (64, 16), (7, 32)])
def test_strides_and_addresses(dtype, pad, offset):
    rng = np.random.default_rng(pad * 100 + offset)
    for rows, cols in ((3, 1), (4, 50), (3, 3001), (2, 70001), (2, 32768)):
        x = rng.normal(0, 3, (rows, cols)).astype(np.float32)
        tokens = rng.integers(0, cols, rows)
        check_logprobs(x, dtype, tokens, min(9, cols), pad=pad, offset=offset)
        check_logprobs_grad(x, dtype, tokens, pad=pad, offset=offset)
        check_logprobs_grad(x, dtype, tokens, pad=pad, offset=offset, in_place=True)
        check_logprobs_grad(x, dtype, tokens, pad=pad, offset=offset, out_pad=3)
        ids, val = slots_for(rng, rows, cols, 6, True, 0.2)
        for kw in ({}, {"in_place": True}, {"out_pad": 5}, {"out_pad": 16}):
            check_distill(x, dtype, ids, val, 1.5, True, pad=pad, offset=offset, **kw)


def hard_rows(cols, low):
    """Rows whose masks, ties and special values can go wrong; `low`: the type's lowest finite value."""
    rng = np.random.default_rng(cols)
    base = rng.normal(0, 3, cols).astype(np.float32)
    rows = {"empty": np.full(cols, -np.inf), "lowest": np.full(cols, low), "zeros": np.zeros(cols),
            "rising": np.linspace(-5, 5, cols), "falling": np.linspace(5, -5, cols),
            "ties": rng.integers(0, 4, cols).astype(np.float32), "signed zeros": np.where(np.arange(cols) % 2, -0.0, 0.0),
            "large": base * 1000, "plain": base}
    one = np.full(cols, -np.inf)
    one[cols // 2] = 1.5
    rows["one allowed"] = one
    few = np.full(cols, -np.inf)
    few[rng.permutation(cols)[:max(1, cols // 300)]] = base[:max(1, cols // 300)]
    rows["few allowed"] = few
    lowmask = np.full(cols, low)
    lowmask[cols // 3] = 2.0
    rows["masked by the lowest"] = lowmask
    both = lowmask.copy()
    both[: cols // 4] = -np.inf
    rows["masked both ways"] = both
    peak = base.copy()
    peak[cols - 1] = 60.0
    rows["peaked"] = peak
    cluster = base.copy()
    cluster[cols // 2: cols // 2 + 200] += 20
    rows["clustered"] = cluster
    for name, at, value in (("nan first", 0, np.nan), ("nan last", cols - 1, np.nan), ("+inf", cols // 2, np.inf)):
        r = base.copy()
        r[at] = value
        rows[name] = r
    rows["all nan"] = np.full(cols, np.nan)
    nm = np.full(cols, -np.inf)
    nm[cols // 3] = np.nan
    rows["nan among -inf"] = nm
    return {n: r.astype(np.float32)[None] for n, r in rows.items()}


LOW = {"f32": -3.4028234663852886e38, "f16": -65504.0, "bf16": -3.3895313892515355e38}
HARD = list(hard_rows(8, -1.0))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("name", HARD)
def test_masks_ties_and_special_values(dtype, name):
    for cols in (5, 40, 1031, 40003):
        x = hard_rows(cols, LOW[dtype])[name]
        tokens = np.array([cols // 2])
        for k in (1, 5, 40, 128):
            check_logprobs(x, dtype, tokens, min(k, cols))
        check_logprobs_grad(x, dtype, tokens)
        rng = np.random.default_rng(cols)
        for tail in (False, True):
            ids, val = slots_for(rng, 1, cols, 4, tail)
            check_distill(x, dtype, ids, val, 1.0, tail)


@pytest.mark.parametrize("what", ["logprobs", "logprobs_backward", "distill", "distill_backward", "distill_step"])
def test_indices_outside_the_row(what):
    """Negative: nothing. Past the row: NaN in that row alone, and nothing outside it touched."""
    rng = np.random.default_rng(5)
    x = rng.normal(0, 2, (4, 1003)).astype(np.float32)
    tokens = np.array([-1, 1003, 1002, 2 ** 40])
    ids = np.array([[5, -1], [1003, 7], [0, 1002], [-100, -100]])
    val = np.log(np.full((4, 2), 0.3, np.float32))
    for dtype in DT:
        if what == "logprobs":
            check_logprobs(x, dtype, tokens, 3, pad=1, offset=1)
        elif what == "logprobs_backward":
            check_logprobs_grad(x, dtype, tokens, pad=1, out_pad=1)
        else:
            for tail in (False, True):
                check_distill(x, dtype, ids, val, 1.0, tail, pad=1, out_pad=1)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("rows,cols,slots", [(1, 1, 1), (2, 3, 3), (3, 40, 40), (2, 100, 0), (3, 1000, 1), (4, 5001, 33),
                                             (2, 1500, 1024), (3, 32001, 100), (1, 202048, 64), (200, 3001, 17),
                                             (2, 300007, 128), (2, 20, 50)])
def test_distill_shapes(dtype, tail, rows, cols, slots):
    rng = np.random.default_rng(rows + cols + slots)
    x = rng.normal(0, 3, (rows, cols)).astype(np.float32)
    for absent, temp in ((0.0, 1.0), (0.3, 2.0)):
        ids, val = slots_for(rng, rows, cols, slots, tail, absent)
        if absent:
            ids[0] = -1  # a row that nothing is taught
        check_distill(x, dtype, ids, val, temp, tail)


def test_distill_teacher_values():
    """Teacher values of -inf leave a slot without weight, not without a name; students that allow less than the
    teacher gives have an infinite loss and a finite gradient."""
    rng = np.random.default_rng(8)
    x = rng.normal(0, 2, (5, 600)).astype(np.float32)
    x[3, 10] = -np.inf
    ids = np.tile(np.array([10, 20, 30]), (5, 1))
    val = np.log(rng.dirichlet(np.ones(4), 5)[:, :3]).astype(np.float32)
    val[0, 1] = -np.inf
    val[1] = -np.inf
    for tail in (False, True):
        for dtype in DT:
            check_distill(x, dtype, ids, val, 1.0, tail)
    got = A.distill_topk(torch.from_numpy(x).cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda()).loss
    assert torch.isinf(got[3]) and got[1] == 0


def test_small_tail_keeps_its_digits():
    """A student whose tail is 1e-9 of the row: its log comes from the tail's own sum, not from 1 minus the rest."""
    x = np.full((1, 5000), -24.0, np.float32)
    x[0, 77] = 5.0
    x[0, 78] = 4.0
    ids = np.array([[77, 78]])
    val = np.log(np.array([[0.5, 0.25]], np.float32))
    got = A.distill_topk(torch.from_numpy(x).cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda(),
                         tail=True).loss
    want, _ = ref.distill(x.astype(np.float64), ids, val, 1.0, True)
    np.testing.assert_allclose(got.cpu().numpy(), want, rtol=2e-5)


def test_leading_dimensions_and_broadcast_rows():
    rng = np.random.default_rng(9)
    x = torch.from_numpy(rng.normal(0, 2, (2, 3, 517)).astype(np.float32)).cuda()
    tokens = torch.randint(0, 500, (2, 3), device="cuda")
    r = A.token_logprobs(x[..., :500], tokens, 4, with_stats=True)
    assert r.logprob.shape == (2, 3) and r.top_ids.shape == (2, 3, 4) and r.stats.shape == (2, 3, 4)
    flat = A.token_logprobs(x.reshape(6, 517)[:, :500].contiguous(), tokens.view(-1), 4)
    # the rows' addresses decide how their sums are grouped: equal to rounding, by the same bounds as everywhere
    want = ref.logprobs(x.reshape(6, 517)[:, :500].double().cpu().numpy(), tokens.view(-1).cpu().numpy(), 4)
    for got in (r, flat):
        close(got.logprob.view(-1), want["logprob"], ref.logprob_bound(want["logprob"], 500), "logprob")
        np.testing.assert_array_equal(got.top_ids.view(6, 4).cpu().numpy(), want["top_ids"])
    one = A.token_logprobs(x[0, 0], tokens[0, 0], 2)
    assert one.logprob.shape == () and one.top_ids.shape == (2,)
    same = A.token_logprobs(x[0, :1].expand(5, 517), torch.arange(5, device="cuda"), 1)
    want = torch.log_softmax(x[0, 0].double(), -1)[:5]
    assert (same.logprob - want).abs().max() < 2e-5
    none = A.token_logprobs(x[:0], tokens[:0], 3)
    assert none.logprob.shape == (0, 3) and none.top_ids.shape == (0, 3, 3)


def test_binding_refusals():
    x = torch.zeros(4, 100, device="cuda")
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    ids, val = torch.zeros(4, 2, dtype=torch.int64, device="cuda"), torch.zeros(4, 2, device="cuda")
    for bad in (lambda: A.token_logprobs(x.double(), tok), lambda: A.token_logprobs(x, tok.int()),
                lambda: A.distill_topk(x, ids.int(), val), lambda: A.distill_topk(x, ids, val.half())):
        with pytest.raises(TypeError):
            bad()
    big = torch.zeros(4, 1025, dtype=torch.int64, device="cuda")
    s = A.token_logprobs(x, tok, with_stats=True).stats
    for bad in (lambda: A.token_logprobs(x, tok[:3]), lambda: A.token_logprobs(x, tok, 101),
                lambda: A.token_logprobs(x, tok, -1), lambda: A.token_logprobs(x, tok, 129),
                lambda: A.token_logprobs(x.t(), tok), lambda: A.token_logprobs(x, tok.cpu()),
                lambda: A.token_logprobs(torch.zeros(2, 4, 3, device="cuda").transpose(0, 1), tok),
                lambda: A.token_logprobs(torch.zeros(4, 0, device="cuda"), tok),
                lambda: A.distill_topk(x, ids[:3], val), lambda: A.distill_topk(x, ids, val[:, :1]),
                lambda: A.distill_topk(x, big, big.float()),
                lambda: A.token_logprobs_backward(x, None, s, tok.float()),
                lambda: A.token_logprobs_backward(x, tok, s[:, :3], tok.float()),
                lambda: A.token_logprobs_backward(x, tok, s, tok.float(), grad=x.half()),
                lambda: A.token_logprobs_backward(x, tok, s, tok.float(), grad=x[:, :50])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: A.token_logprobs(x, tok, temperature=0.0),
                lambda: A.token_logprobs_backward(x[:, 1:], tok, s, tok.float(), grad=x[:, :-1])):
        with pytest.raises(A.ArgreduceError):
            bad()


def test_autograd_against_64_bits():
    g = torch.Generator("cuda").manual_seed(3)
    for dtype, tol in ((torch.float32, 2e-6), (torch.bfloat16, 5e-3)):
        x = (torch.randn(6, 1501, device="cuda", generator=g) * 2).to(dtype)
        tok = torch.randint(0, 1501, (6,), device="cuda", generator=g)
        a = x.clone().requires_grad_()
        r = A.token_logprobs(a, tok, 3, temperature=0.8)
        assert not r.top_logprobs.requires_grad and not r.stats.requires_grad
        (r.logprob.sum() + 0.1 * r.entropy.sum() + (0.01 * r.lse ** 2).sum()).backward()
        b = x.double().requires_grad_()
        lp = torch.log_softmax(b / 0.8, -1)
        lse = torch.logsumexp(b / 0.8, -1)
        (lp.gather(1, tok[:, None]).sum() - 0.1 * (lp.exp() * lp).sum() + (0.01 * lse ** 2).sum()).backward()
        assert a.grad.dtype is dtype
        assert (a.grad.double() - b.grad).abs().max() < tol * b.grad.abs().max() * 2
        only = x.clone().requires_grad_()
        A.token_logprobs(only).entropy.sum().backward()
        assert only.grad.abs().sum() > 0

        ids = torch.stack([torch.randperm(1501, device="cuda", generator=g)[:8] for _ in range(6)])
        val = torch.randn(6, 8, device="cuda", generator=g)
        a = x.clone().requires_grad_()
        A.distill_topk(a, ids, val, temperature=2.0).loss.mean().backward()
        b = x.double().requires_grad_()
        q = torch.softmax(val.double() / 2, -1)
        (q * (q.log() - torch.log_softmax(b / 2, -1).gather(1, ids))).sum(-1).mean().backward()
        assert (a.grad.double() - b.grad).abs().max() < tol * b.grad.abs().max() * 2


def test_gradients_against_differences():
    """Central differences of the kernels' own 32-bit losses, step 0.05: the truncation is at most step^2 / 6 times a
    third derivative of order 1, the rounding 1e-5 / step."""
    rng = np.random.default_rng(11)
    x = rng.normal(0, 1, (1, 37)).astype(np.float32)
    ids, val = slots_for(rng, 1, 37, 5, True)
    i, v = torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda()
    step = 0.05
    many = np.repeat(x, 74, 0)
    for j in range(37):
        many[2 * j, j] += step
        many[2 * j + 1, j] -= step
    m = torch.from_numpy(many).cuda()
    one = torch.from_numpy(x).cuda()
    loss = A.distill_topk(m, i.repeat(74, 1), v.repeat(74, 1), tail=True).loss.cpu().numpy().reshape(37, 2)
    _, grad = A.distill_topk_step(one, i, v, torch.ones(1, device="cuda"), tail=True)
    assert np.abs((loss[:, 0] - loss[:, 1]) / (2 * step) - grad.cpu().numpy()[0]).max() < 2e-3
    tok = torch.tensor([7], device="cuda")
    r = A.token_logprobs(m, tok.expand(74).contiguous())
    f = (r.logprob + 0.5 * r.entropy - 0.25 * r.lse).cpu().numpy().reshape(37, 2)
    s = A.token_logprobs(one, tok, with_stats=True).stats
    grad = A.token_logprobs_backward(one, tok, s, *(torch.full((1,), w, device="cuda") for w in (1.0, 0.5, -0.25)))
    assert np.abs((f[:, 0] - f[:, 1]) / (2 * step) - grad.cpu().numpy()[0]).max() < 2e-3


def test_streams_graphs_and_repeats():
    g = torch.Generator("cuda").manual_seed(4)
    x = (torch.randn(9, 40001, device="cuda", generator=g) * 3).bfloat16()
    tok = torch.randint(0, 40001, (9,), device="cuda", generator=g)
    first = A.token_logprobs(x, tok, 20, with_stats=True)
    ids, val = first.top_ids, first.top_logprobs
    w = torch.rand(9, device="cuda", generator=g)
    step = A.distill_topk_step(x, ids, val, w, tail=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = A.token_logprobs(x, tok, 20, with_stats=True)
        step2 = A.distill_topk_step(x, ids, val, w, tail=True)
    other = A.token_logprobs(x, tok, 20, stream=side, with_stats=True)
    side.synchronize()
    for a, b, c in zip(first, again, other):
        assert torch.equal(a, b) and torch.equal(a, c)
    for a, b in zip(step, step2):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = A.token_logprobs(x, tok, 20, with_stats=True)
        s = A.distill_topk_step(x, r.top_ids, r.top_logprobs, w, tail=True)
    for k in range(3):
        x.copy_((torch.randn(9, 40001, device="cuda", generator=g) * 3).bfloat16())
        graph.replay()
        eager = A.token_logprobs(x, tok, 20, with_stats=True)
        estep = A.distill_topk_step(x, eager.top_ids, eager.top_logprobs, w, tail=True)
        torch.cuda.synchronize()
        for a, b in zip(tuple(r) + tuple(s), tuple(eager) + tuple(estep)):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Rows that lie 2^31 elements apart, and a gradient whose rows do."""
    stride, cols = (1 << 31) + 24, 3001
    buf = torch.empty(stride * 2 + cols, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, cols), (stride, 1))
    small = (torch.randn(3, cols, device="cuda") * 3).bfloat16()
    x.copy_(small)
    tok = torch.tensor([0, 1500, 3000], device="cuda")
    a, b = A.token_logprobs(x, tok, 7), A.token_logprobs(small, tok, 7)
    x64 = small.double().cpu().numpy()
    want = ref.logprobs(x64, tok.cpu().numpy(), 7)
    for got in (a, b):  # the rows' addresses decide how their sums are grouped
        close(got.logprob, want["logprob"], ref.logprob_bound(want["logprob"], cols), "logprob")
        close(got.entropy, want["entropy"], ref.entropy_bound(want["entropy"], np.log(cols), cols), "entropy")
        np.testing.assert_array_equal(got.top_ids.cpu().numpy(), want["top_ids"])
    w = torch.rand(3, device="cuda")
    val = b.top_logprobs.cpu().numpy()
    loss, grad = ref.distill(x64, b.top_ids.cpu().numpy(), val, 1.0, True, w.double().cpu().numpy())
    wide = torch.empty_like(buf).as_strided((3, cols), (stride, 1))
    got = A.distill_topk_step(x, b.top_ids, b.top_logprobs, w, tail=True, grad=wide)
    near = A.distill_topk_step(small, b.top_ids, b.top_logprobs, w, tail=True)
    for g in (got, near):
        close(g[0], loss, ref.logprob_bound(loss, cols) + 40 * ref.sum_error(cols), "loss")
        close(g[1], grad, ref.grad_bound(grad, np.exp(ref.log_probs(x64, 1.0)) * 20 + 1e-3, cols, "bf16"), "grad")


def test_longest_row():
    """INT32_MAX columns: a row of zeros with a few planted values."""
    cols = 2 ** 31 - 1
    x = torch.zeros(1, cols, dtype=torch.float16, device="cuda")
    at = [cols - 1, 5, 2 ** 30 + 7, 2 ** 31 - 5]
    for n, j in enumerate(at):
        x[0, j] = 20.0 - n
    r = A.token_logprobs(x, torch.tensor([cols - 1], device="cuda"), 6, with_stats=True)
    s = float(np.exp([20.0, 19.0, 18.0, 17.0]).sum() + (cols - 4))
    assert r.top_ids[0].tolist() == at + [0, 1]
    assert abs(r.lse.item() - np.log(s)) < 1e-4
    assert abs(r.logprob.item() - (20 - np.log(s))) < 1e-4
    grad = A.token_logprobs_backward(x, torch.tensor([cols - 1], device="cuda"), r.stats,
                                     torch.ones(1, device="cuda"), grad=x)
    assert abs(grad[0, 5].item() + np.exp(19.0) / s) < 2e-3 and abs(grad[0, cols - 1].item() - 1 + np.exp(20.0) / s) < 2e-3


def test_teacher_to_student():
    """The two operators as they are used together: a teacher's alternatives, and a student taught from them."""
    g = torch.Generator("cuda").manual_seed(6)
    teacher = torch.randn(32, 2000, device="cuda", generator=g) * 3
    t = A.token_logprobs(teacher, top_k=50)
    student = torch.zeros(32, 2000, device="cuda", requires_grad=True)
    double = torch.zeros(32, 2000, device="cuda", dtype=torch.float64, requires_grad=True)
    opt = torch.optim.SGD([student, double], lr=40.0)
    q = t.top_logprobs.double().exp()
    rest = 1 - q.sum(-1)
    losses = []
    for _ in range(60):
        loss = A.distill_topk(student, t.top_ids, t.top_logprobs, tail=True).loss.mean()
        lp = torch.log_softmax(double, -1)
        mass = lp.exp().scatter(1, t.top_ids, 0.0).sum(-1)
        want = ((q * (q.log() - lp.gather(1, t.top_ids))).sum(-1) + rest * (rest.log() - mass.log())).mean()
        opt.zero_grad()
        (loss + want).backward()
        opt.step()
        losses.append(loss.item())
        assert abs(loss.item() - want.item()) < 1e-4
    assert losses[-1] < 0.5 * losses[0]
    assert torch.equal(A.argmax(student.detach()), t.top_ids[:, 0])


# ---------------------------------------------------------------------------
# Every kernel, whatever the planner would choose.
# ---------------------------------------------------------------------------
from row_wise_arg_gb300 import _lib  # noqa: E402


def forward_plan(cluster=1, block=256, grid=1 << 20, rows=1):
    p = _lib.argr_plan()
    p.path, p.block, p.cluster, p.blocks_per_row = _lib.ARGR_PATH_LOGITS, block, cluster, 1
    p.grid_rows, p.flags = min(grid, rows), _lib.ARGR_PLAN_PDL
    return p


def stream_plan(finishers=1, block=256, grid=4):
    p = _lib.argr_plan()
    p.path, p.block, p.cluster, p.blocks_per_row = _lib.ARGR_PATH_LOGITS_STREAM, block, 1, 1
    p.group, p.grid_rows, p.flags = finishers, grid, _lib.ARGR_PLAN_PDL
    return p


def step_plan(cluster=1, block=256, grid=4):
    p = forward_plan(cluster, block, grid, grid)
    p.path = _lib.ARGR_PATH_LOGITS_STEP
    return p


def grad_plan(chunks=1, block=256, grid=4):
    p = _lib.argr_plan()
    p.path, p.block, p.cluster, p.blocks_per_row = _lib.ARGR_PATH_LOGITS_GRAD, block, 1, chunks
    p.grid_rows = grid
    return p


FORWARD = [("cluster", dict(cluster=c, block=b, grid=g)) for c, b, g in
           ((1, 32, 1), (1, 512, 3), (2, 64, 2), (3, 96, 9), (5, 128, 1), (8, 256, 9), (16, 512, 2), (16, 32, 9))] + \
          [("stream", dict(finishers=f, block=b, grid=g)) for f, b, g in
           ((1, 64, 1), (1, 512, 2), (2, 96, 1), (2, 256, 3), (3, 128, 1), (3, 512, 9), (1, 96, 9))]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,how", FORWARD, ids=lambda v: v if isinstance(v, str) else "-".join(map(str, v.values())))
def test_forced_forward_plans(dtype, kind, how):
    rng = np.random.default_rng(17)
    for rows, cols, pad, offset in ((9, 1, 0, 0), (9, 70, 1, 1), (9, 5003, 0, 0), (3, 40001, 3, 5), (2, 65536, 0, 0)):
        plan = forward_plan(rows=rows, **how) if kind == "cluster" else stream_plan(**how)
        x = rng.normal(0, 3, (rows, cols)).astype(np.float32)
        tokens = rng.integers(-1, cols, rows)
        for k in (0, 1, 20, 128):
            check_logprobs(x, dtype, tokens, min(k, cols), 0.9, plan=plan, pad=pad, offset=offset)
        for slots, tail in ((7, False), (7, True), (130, True)):
            ids, val = slots_for(rng, rows, cols, slots, tail, 0.2)
            xd, x64 = on_gpu(x, dtype, pad, offset)
            r = A.distill_topk(xd, torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda(), tail=tail, plan=plan,
                               with_stats=True)
            same = A.distill_topk(xd, torch.from_numpy(ids).cuda(), torch.from_numpy(val).cuda(), tail=tail,
                                  plan=forward_plan(rows=rows), with_stats=True)
            # the two kernels against each other (the chosen one is checked against 64 bits everywhere else)
            want, _ = ref.distill(x64, ids, val, 1.0, tail)
            big = 40.0 + np.abs(want)
            close(r.loss, want, ref.sum_error(cols) * big * 3, "loss")
            close(r.stats[:, :2], same.stats[:, :2].double().cpu().numpy(), 2 * ref.sum_error(cols) * 30, "stats")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", HARD)
def test_forced_plans_on_hard_rows(dtype, name):
    for cols in (40, 1031, 40003):
        x = np.repeat(hard_rows(cols, LOW[dtype])[name], 3, 0)
        x[1] = np.random.default_rng(cols).normal(0, 3, cols)
        tokens = np.array([cols // 2, 0, -1])
        for plan in (forward_plan(4, 64, 3, 3), stream_plan(1, 128, 1), stream_plan(2, 512, 2)):
            for k in (1, 40, 128):
                check_logprobs(x, dtype, tokens, min(k, cols), plan=plan)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_forced_gradient_plans(dtype):
    rng = np.random.default_rng(19)
    for rows, cols, kw in ((5, 1, {}), (5, 70, {"pad": 1, "offset": 1}), (5, 5003, {"out_pad": 1}), (2, 40001, {}),
                           (3, 32768, {"out_pad": 8}), (3, 4096, {"in_place": True}), (3, 4099, {"in_place": True})):
        x = rng.normal(0, 3, (rows, cols)).astype(np.float32)
        tokens = rng.integers(-1, cols, rows)
        ids, val = slots_for(rng, rows, cols, 9, True, 0.1)
        for chunks, block, grid in ((1, 32, 1), (3, 256, 5), (40, 64, 2)):
            check_logprobs_grad(x, dtype, tokens, plan=grad_plan(chunks, block, grid), **kw)
            for cluster, sblock, sgrid in ((1, 256, 2), (3, 64, 5), (16, 32, 1)):
                if -(-(cols * ES[dtype] // 64) // cluster) * 64 > 108 * 1024:
                    continue
                check_distill(x, dtype, ids, val, 1.3, True, grad_plan=grad_plan(chunks, block, grid),
                              step_plan=step_plan(cluster, sblock, sgrid), **kw)
            check_distill(x, dtype, ids, val, 1.0, False, step_plan=forward_plan(2, 128, 3, rows), **kw)


def test_many_rows_through_the_persistent_kernel():
    """As many rows as two CTAs per SM, as the planner runs them."""
    rng = np.random.default_rng(23)
    for dtype, rows, cols in (("bf16", 300, 82003), ("f32", 304, 41000), ("f16", 290, 90001)):
        assert A.argreduce_logits_plan("logprobs", rows, cols, dtype, 20, CAPS).path == _lib.ARGR_PATH_LOGITS_STREAM
        x = rng.normal(0, 3, (rows, cols)).astype(np.float32)
        x[5] = -np.inf
        x[7, 100:] = -np.inf
        x[9] = 1.0
        tokens = rng.integers(0, cols, rows)
        for k in (0, 128):
            check_logprobs(x, dtype, tokens, k)
        for tail in (False, True):
            ids, val = slots_for(rng, rows, cols, 40, tail, 0.1)
            ids[11] = -1
            check_distill(x, dtype, ids, val, 1.0, tail)


def test_plan_refusals_on_the_device():
    x = torch.zeros(4, 100, device="cuda")
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    bad = [forward_plan(17), forward_plan(0), forward_plan(1, 48), forward_plan(1, 1024), stream_plan(0), stream_plan(4),
           stream_plan(3, 96), stream_plan(1, 32), stream_plan(1, 256, 0), grad_plan(), step_plan()]
    for p in bad:
        with pytest.raises(A.ArgreduceError):
            A.token_logprobs(x, tok, 3, plan=p)
    s = A.token_logprobs(x, tok, with_stats=True).stats
    for p in (grad_plan(0), grad_plan(1, 512), forward_plan(), stream_plan()):
        with pytest.raises(A.ArgreduceError):
            A.token_logprobs_backward(x, tok, s, torch.ones(4, device="cuda"), plan=p)
    wide = torch.zeros(1, 1 << 20, device="cuda")
    one = torch.zeros(1, 1, dtype=torch.int64, device="cuda")
    with pytest.raises(A.ArgreduceError):  # more than the shared memory of two CTAs per SM
        A.distill_topk(wide, one, one.float(), plan=stream_plan(3, 512))
    for p in (step_plan(17), step_plan(16, 512), step_plan(4), stream_plan(1, 512)):
        with pytest.raises(A.ArgreduceError):
            A.distill_topk_step(wide, one, one.float(), torch.ones(1, device="cuda"), plan=p)


def test_step_whose_copies_never_land():
    """A bounded wait that runs out is reported and leaves the library usable."""
    g = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(3, 30000, device="cuda", generator=g)
    ids, val = torch.arange(4, device="cuda").repeat(3, 1), torch.full((3, 4), -2.0, device="cuda")
    w = torch.ones(3, device="cuda")
    want = A.distill_topk_step(x, ids, val, w, tail=True)
    assert A.argreduce_read_error(0, 0) == _lib.ARGR_OK
    for cluster, grid in ((4, 3), (2, 1)):
        p = step_plan(cluster, 128, grid)
        p.flags |= _lib.ARGR_PLAN_TEST_EXPIRE
        A.distill_topk_step(x, ids, val, w, tail=True, plan=p)
        assert A.argreduce_read_error(0, 0) == _lib.ARGR_ETIMEOUT
        assert A.argreduce_read_error(0, 0) == _lib.ARGR_OK
    got = A.distill_topk_step(x, ids, val, w, tail=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill.py")
    spec = importlib.util.spec_from_file_location("example_distill", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, agree, rewards = example.main(rows=64, vocab=5003, steps=25, say=lambda s: None)
    assert losses[-1] < 0.5 * losses[0] and agree > 0.9
    assert sum(rewards[-5:]) > sum(rewards[:5]) + 0.5
