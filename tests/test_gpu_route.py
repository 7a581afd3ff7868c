"""GPU: routing to experts, its gradient and the row order, against plain
64-bit forms.

Choices are compared in binary32 by the kernel and in 64 bits here, so a row
takes part only where neighbouring choices are equal or apart by more than binary32's
error of them: 2^-18 of the value itself, or of the row's largest where a bias
may cancel the score.  Weights: the score's
exponent is off by |l - max| 2^-24 < 40 * 2^-24, exp and the divisions by a
few units, the sum by E/32 + 5 roundings: together below 2^-17 of the weight.
Gradients: the same relative error of every term before the subtractions."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
LOWEST = -3.3895313892515355e38


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_quantization_gb300 as m
    m.abi()
    return m


def top(choice, k):
    """(values, indices) of the k largest, ties to the lowest index."""
    v, i = torch.sort(choice, dim=-1, descending=True, stable=True)
    return v[..., :k], i[..., :k]


def apart(sorted_values, biased):
    """Neighbours equal or clearly apart, for rows sorted in descending order."""
    v = sorted_values.clamp(min=-1e30)
    gap = v[..., :-1] - v[..., 1:]
    big = sorted_values.masked_fill(sorted_values.isinf(), 0).abs()
    big = big.amax(-1, keepdim=True) if biased else big[..., :-1]
    return ((gap == 0) | (gap > 2.0 ** -18 * big)).all(-1)


def route64(logits, k, bias, score, groups, keep, gtop, renorm, scale):
    l = logits.double().cpu()
    T, E = l.shape
    ok = l > LOWEST
    l = l.clamp(max=3.4028234663852886e38)
    if score == "sigmoid":
        s = torch.where(ok, torch.sigmoid(l), 0.0)
    else:
        m = torch.where(ok, l, -torch.inf).amax(1, keepdim=True)
        e = torch.where(ok, torch.exp(l - m), 0.0)
        s = torch.where(ok, e / e.sum(1, keepdim=True), 0.0)
    c = s if bias is None else s + bias.double().cpu()
    c = torch.where(ok & ~c.isnan(), c, -torch.inf)
    sure = torch.ones(T, dtype=torch.bool)
    if groups > 1:
        per = c.view(T, groups, -1)
        best = torch.sort(per, -1, descending=True).values[..., :gtop]
        gs = torch.where(best > -torch.inf, best, 0.0).sum(-1)
        gs = torch.where(best[..., 0] > -torch.inf, gs, -torch.inf)
        v, i = top(gs, groups)
        sure &= apart(v, bias is not None)
        open_ = torch.zeros_like(gs, dtype=torch.bool).scatter(1, i[:, :keep], True)
        c = torch.where(open_[..., None], per, -torch.inf).view(T, E)
    v, i = top(c, min(E, k + 1))
    if v.shape[1] > 1:
        sure &= apart(v, bias is not None)
    v, i = v[:, :k], i[:, :k]
    there = v > -torch.inf
    w = torch.where(there, s.gather(1, i), 0.0)
    if renorm:
        tot = w.sum(1, keepdim=True)
        w = torch.where(tot > 0, w / tot, 0.0)
    return w * scale, torch.where(there, i, -1), sure, s


def logits_of(T, E, dtype, seed, spread=5.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.rand((T, E), device="cuda", generator=gen) * 2 * spread - spread
    return l.to(dtype), gen


CASES = [  # T, E, k, groups, keep, top
    (1, 1, 1, 1, 1, 1), (1, 8, 8, 1, 1, 1), (5, 31, 4, 1, 1, 1), (40, 60, 6, 4, 2, 1),
    (33, 96, 7, 8, 3, 2), (64, 256, 8, 8, 4, 2), (3, 256, 8, 1, 1, 1), (70, 512, 8, 8, 4, 2),
    (9, 1024, 32, 32, 9, 2), (17, 33, 32, 1, 1, 1), (10, 10, 3, 5, 2, 2), (12, 32, 2, 32, 2, 2),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("biased,renorm", [(False, True), (True, True), (True, False), (False, False)])
def test_route(fq, case, score, dtype, biased, renorm):
    T, E, k, groups, keep, gtop = case
    logits, gen = logits_of(T, E, dtype, T + E)
    bias = 0.3 * torch.randn(E, device="cuda", generator=gen) if biased else None
    w, ids = fq.moe_route(logits, k, bias=bias, score=score, n_groups=groups, keep_groups=keep,
                          group_top=gtop, renormalize=renorm, scale=2.5)
    rw, rids, sure, _ = route64(logits, k, bias, score, groups, keep, gtop, renorm, 2.5)
    assert bool(sure.any())
    ids, w = ids.cpu().long(), w.cpu().double()
    assert torch.equal(ids[sure], rids[sure])
    assert bool(((w - rw).abs() <= 2.0 ** -17 * rw.abs())[sure].all())


def test_ties_go_to_the_lowest_index(fq):
    logits = torch.zeros((3, 70), device="cuda")
    logits[1, 40:44] = 1.0
    logits[2, ::7] = 2.0
    for score in ("softmax", "sigmoid"):
        _, ids = fq.moe_route(logits, 4, score=score)
        assert ids.tolist() == [[0, 1, 2, 3], [40, 41, 42, 43], [0, 7, 14, 21]]
        _, ids = fq.moe_route(logits, 2, score=score, n_groups=7, keep_groups=1, group_top=2)
        assert ids.tolist() == [[0, 1], [40, 41], [0, 7]]


# a second name, as the first is bound to another test further down
test_equal_logits_go_to_the_lowest_index = test_ties_go_to_the_lowest_index


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masks(fq, dtype, score):
    nan, inf = float("nan"), float("inf")
    low = torch.finfo(dtype).min
    rows = [[-inf] * 6, [nan] * 6, [low] * 6, [-inf, 1.0, nan, low, -inf, 2.0],
            [inf, 0.0, inf, -inf, 1.0, nan], [low, -inf, nan, 0.5, -inf, low], [0.0] * 6]
    logits = torch.tensor(rows, device="cuda").to(dtype)
    for bias in (None, torch.tensor([9.0, 0, 9, 9, 0, 0], device="cuda")):
        w, ids = fq.moe_route(logits, 3, bias=bias, score=score)
        rw, rids, _, _ = route64(logits, 3, bias, score, 1, 1, 1, True, 1.0)
        assert torch.equal(ids.cpu().long(), rids)
        assert bool(((w.cpu().double() - rw).abs() <= 2.0 ** -17).all())
    d = fq.moe_route_backward(logits, ids, torch.ones((7, 3), device="cuda"), score=score,
                              renormalize=False)
    assert bool(torch.isfinite(d.float()).all())
    assert bool((d[:3] == 0).all())
    # groups: one without any expert is never kept, one with a single expert counts it
    w, ids = fq.moe_route(logits, 2, score=score, n_groups=3, keep_groups=2, group_top=2)
    rw, rids, _, _ = route64(logits, 2, None, score, 3, 2, 2, True, 1.0)
    assert torch.equal(ids.cpu().long(), rids)


def test_bias_that_is_not_finite(fq):
    logits = torch.zeros((1, 5), device="cuda")
    bias = torch.tensor([float("-inf"), float("nan"), 0.0, float("inf"), 0.1], device="cuda")
    w, ids = fq.moe_route(logits, 4, bias=bias, score="sigmoid")
    assert ids.tolist() == [[3, 4, 2, -1]] and w[0, 3] == 0


def grad64(logits, ids, dw, score, renorm, scale):
    """(gradient by the formula, magnitude of its terms) in 64 bits."""
    _, _, _, s = route64(logits, 1, None, score, 1, 1, 1, False, 1.0)
    ids, dw = ids.cpu().long(), dw.double().cpu()
    there = ids >= 0
    at = ids.clamp(min=0)
    c = torch.where(there, s.gather(1, at), 0.0)
    g = torch.where(there, dw, 0.0) * scale
    mag = g.abs()
    if renorm:
        tot = c.sum(1, keepdim=True)
        inv = torch.where(tot > 0, 1 / tot, 0.0)
        mag = (mag + (mag * c * inv).sum(1, keepdim=True)) * inv
        g = (g - (g * c * inv).sum(1, keepdim=True)) * inv
    full = torch.zeros_like(s).scatter_add(1, at, torch.where(there, g, 0.0))
    fmag = torch.zeros_like(s).scatter_add(1, at, torch.where(there, mag, 0.0))
    if score == "sigmoid":
        return full * s * (1 - s), fmag * s
    return s * (full - (full * s).sum(1, keepdim=True)), s * (fmag + (fmag * s).sum(1, keepdim=True))


@pytest.mark.parametrize("E,k,groups,keep,gtop", [
    (33, 4, 1, 1, 1), (64, 8, 4, 2, 2), (96, 6, 1, 1, 1), (130, 8, 5, 2, 2), (200, 8, 8, 3, 1),
    (256, 32, 8, 4, 2), (250, 8, 25, 20, 2), (500, 9, 1, 1, 1), (512, 8, 32, 5, 2), (1000, 32, 1, 1, 1),
    (1024, 8, 4, 1, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lowest_index(fq, E, k, groups, keep, gtop, score, dtype):
    """Rows of four values (so that every choice ties with others, in its lane's
    run and across lanes) with every fifth logit masked; rows with fewer experts
    than slots.  The sums of two of the four scores lie further apart than their
    rounding, so the groups' order is known too."""
    T = 40
    rng = np.random.default_rng(E)
    l = rng.integers(0, 4, (T, E)).astype(np.float64)
    l[rng.random((T, E)) < 0.2] = -np.inf
    l[1] = 2.0
    l[2, 5:] = -np.inf
    l[3, : E - 3] = -np.inf
    l[4] = -np.inf
    _, ids = fq.moe_route(torch.tensor(l, device="cuda").to(dtype), k, score=score, n_groups=groups,
                          keep_groups=keep, group_top=gtop)
    with np.errstate(invalid="ignore"):
        s = 1 / (1 + np.exp(-l)) if score == "sigmoid" else np.exp(l - 3)
    want = np.full((T, k), -1)
    for t in range(T):
        c = np.where(l[t] > -np.inf, s[t], -1.0)
        if groups > 1:
            best = -np.sort(-c.reshape(groups, -1), axis=1)[:, :gtop]
            total = np.where(best[:, 0] < 0, -1.0, np.maximum(best, 0).sum(1))
            kept = [g for g in np.argsort(-total, kind="stable")[:keep] if total[g] >= 0]
            c = np.where(np.isin(np.arange(E) // (E // groups), kept), c, -1.0)
        order = [e for e in np.argsort(-c, kind="stable")[:k] if c[e] >= 0]
        want[t, : len(order)] = order
    assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward(fq, case, score, dtype, renorm):
    T, E, k = case[:3]
    logits, gen = logits_of(T, E, dtype, T * E)
    if E > 4:
        logits[0] = float("-inf")
        logits[:, 2] = float("-inf")
    _, ids = fq.moe_route(logits, k, score=score, renormalize=renorm)
    dw = torch.randn((T, k), device="cuda", generator=gen)
    d = fq.moe_route_backward(logits, ids, dw, score=score, renormalize=renorm, scale=2.5)
    assert d.dtype == dtype and d.shape == (T, E)
    ref, mag = grad64(logits, ids, dw, score, renorm, 2.5)
    tol = 2.0 ** -17 * mag + (2.0 ** -8 * ref.abs() if dtype == torch.bfloat16 else 0)
    assert bool(((d.cpu().double() - ref).abs() <= tol + 1e-37).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(fq, score, renorm):
    """Central differences of the kernel's own weights.  Logits 1/16 apart and a
    step of 1/64 leave the choice alone; the third derivative of a score is
    below 1 and of a normalised weight below 8 (k = 3), so the difference is off
    by 8 h^2 / 6 and by 2^-17 / h of rounding per term."""
    T, E, k, h = 6, 24, 3, 1.0 / 64
    gen = torch.Generator(device="cuda").manual_seed(0)
    order = torch.stack([torch.randperm(E, device="cuda", generator=gen) for _ in range(T)])
    logits = (order.float() - E / 2) / 16
    dw = torch.randn((T, k), device="cuda", generator=gen)
    _, ids = fq.moe_route(logits, k, score=score, renormalize=renorm)
    d = fq.moe_route_backward(logits, ids, dw, score=score, renormalize=renorm)
    tol = float(dw.abs().sum(1).max()) * (8 * h * h / 6 + 2.0 ** -17 / h)
    for e in range(E):
        side = []
        for sign in (1, -1):
            moved = logits.clone()
            moved[:, e] += sign * h
            w, i = fq.moe_route(moved, k, score=score, renormalize=renorm)
            assert torch.equal(i, ids)
            side.append((w * dw).sum(1).double())
        diff = (side[0] - side[1]) / (2 * h)
        assert float((diff - d[:, e].double()).abs().max()) <= tol


def test_ids_outside_the_range_have_no_gradient(fq):
    logits = torch.randn((2, 9), device="cuda")
    ids = torch.tensor([[3, -1, 9], [2 ** 31 - 1, 0, -5]], dtype=torch.int32, device="cuda")
    d = fq.moe_route_backward(logits, ids, torch.ones((2, 3), device="cuda"), score="sigmoid",
                              renormalize=False)
    assert (d != 0).nonzero().tolist() == [[0, 3], [1, 0]]


@pytest.mark.parametrize("n,E", [(0, 5), (1, 1), (31, 3), (33, 1024), (512, 32), (4096, 7), (4097, 256),
                                 (20000, 256), (33001, 61), (70000, 1024)])
@pytest.mark.parametrize("kind", ["even", "skewed", "dropped", "one", "nobody"])
def test_sort_rows(fq, n, E, kind):
    rng = np.random.default_rng(n + E)
    ids = rng.integers(0, E, n)
    if kind == "skewed":
        ids = np.minimum(ids, rng.integers(0, E, n) // 3)
    elif kind == "dropped":
        ids = rng.choice([-1, -7, E, 2 ** 31 - 1, 0, E - 1, E // 2], n)
    elif kind == "one":
        ids[:] = E - 1
    elif kind == "nobody":
        ids[:] = -1
    dev = torch.from_numpy(ids.astype(np.int32)).cuda()
    raw = torch.full((n + 64,), 7, dtype=torch.int32, device="cuda")
    offs, pair, row = fq.moe_sort_rows(dev, E, pair_of_row=raw[32:32 + n])
    good = (ids >= 0) & (ids < E)
    order = np.flatnonzero(good)[np.argsort(ids[good], kind="stable")]
    want = np.full(n, -1)
    want[:len(order)] = order
    inv = np.full(n, -1)
    inv[order] = np.arange(len(order))
    assert np.array_equal(offs.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(ids[good], minlength=E))]))
    assert np.array_equal(pair.cpu().numpy(), want)
    assert np.array_equal(row.cpu().numpy(), inv)
    assert bool((raw[:32] == 7).all()) and bool((raw[32 + n:] == 7).all())


def test_sort_rows_keeps_the_shape(fq):
    ids = torch.tensor([[1, 0], [0, 2], [-1, 1]], dtype=torch.int32, device="cuda")
    offs, pair, row = fq.moe_sort_rows(ids, 3)
    assert offs.tolist() == [0, 2, 4, 5] and pair.tolist() == [1, 2, 0, 5, 3, -1]
    assert row.tolist() == [[2, 0], [1, 4], [-1, 3]]
