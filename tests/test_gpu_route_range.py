"""GPU: the router's weights and their gradient where the scores leave binary32's
comfortable range: experts chosen far below the row's largest logit, sigmoid
scores next to 0 and 1; and ids that stand twice in a row.

References are 64-bit forms.  Tolerances: a weight is a quotient of terms
exp(l - max) of the chosen logits, at most 45 apart here, so an exponent is off by 45 *
2^-24, exp and the divisions by a few units, the sum of at most 32 terms by
their 5 + 1 roundings: below 2^-17 of the weight.  A gradient is a sum of
such terms; each is off by 2^-17 of itself, the factor 1 - s of the sigmoid included.
BF16 gradients are rounded once (2^-8 of their value); 1e-37 covers results below
the normal numbers."""
import pytest
import torch

pytestmark = pytest.mark.gpu
REL = 2.0 ** -17


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import fp8_quantization_gb300 as m
    m.abi()
    return m


def log_score(l, score):
    """log of the score, up to a constant of the row (64 bits)."""
    l = l.double()
    return torch.nn.functional.logsigmoid(l) if score == "sigmoid" else l


def weights64(logits, ids, score, scale):
    """Renormalised weights of the chosen: a softmax over their log scores."""
    return scale * torch.softmax(log_score(logits.gather(1, ids.long()), score), 1)


def gradient64(logits, ids, dw, score, renorm, scale):
    """(gradient, magnitude of its terms); ids may repeat and may be -1."""
    T, E = logits.shape
    there = ids >= 0
    at = ids.long().clamp(min=0)
    g = torch.where(there, dw.double(), 0.0) * scale
    chosen = logits.double().gather(1, at)
    full, mag = torch.zeros((2, T, E), dtype=torch.float64, device=logits.device)
    if renorm:
        q = torch.softmax(log_score(chosen, score).masked_fill(~there, -torch.inf), 1)
        q = torch.where(there, q, 0.0)
        d = q * (g - (g * q).sum(1, keepdim=True))
        m = q * (g.abs() + (g * q).abs().sum(1, keepdim=True))
        if score == "sigmoid":
            slope = torch.sigmoid(-chosen)  # 1 - s without cancellation
            d, m = d * slope, m * slope
        return full.scatter_add(1, at, d), mag.scatter_add(1, at, m)
    if score == "sigmoid":
        d = torch.where(there, g * torch.sigmoid(chosen) * torch.sigmoid(-chosen), 0.0)
        return full.scatter_add(1, at, d), mag.scatter_add(1, at, d.abs())
    p = torch.softmax(logits.double(), 1)
    full, mag = full.scatter_add(1, at, g), mag.scatter_add(1, at, g.abs())
    return p * (full - (full * p).sum(1, keepdim=True)), p * (mag + (mag * p).sum(1, keepdim=True))


def close(d, ref, mag):
    tol = REL * mag + (2.0 ** -8 * ref.abs() if d.dtype == torch.bfloat16 else 0) + 1e-37
    err = (d.double() - ref).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol).max())} of the bound"


def far_below(T, E, low, high, dtype, seed):
    """Rows whose first expert leads by far and is taken out of the choice by its
    bias; the others' biases are distinct, so that they decide the choice."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.rand((T, E), device="cuda", generator=gen) * (high - low) + low
    logits[:, 0] = 3.0
    bias = 1.0 + torch.randperm(E, device="cuda", generator=gen).float() / E
    bias[0] = -torch.inf
    return logits.to(dtype), bias, gen


RANGES = [(-90.0, -80.0), (-120.0, -85.0), (-145.0, -105.0), (-2000.0, -1960.0)]


@pytest.mark.parametrize("low,high", RANGES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(9, 1), (33, 4), (256, 8), (1000, 32)])
def test_softmax_weights_far_below_the_largest_logit(fq, low, high, dtype, E, k):
    logits, bias, gen = far_below(40, E, low, high, dtype, E)
    w, ids = fq.moe_route(logits, k, bias=bias, scale=2.5)
    order = torch.argsort(bias, descending=True)[:k].int()
    assert torch.equal(ids, order.expand(40, k))
    ref = weights64(logits, ids, "softmax", 2.5)
    assert bool(((w.double() - ref).abs() <= REL * ref).all())
    dw = torch.randn((40, k), device="cuda", generator=gen)
    d = fq.moe_route_backward(logits, ids, dw, scale=2.5)
    close(d, *gradient64(logits, ids, dw, "softmax", True, 2.5))


def test_softmax_weights_below_the_largest_logit_of_a_closed_group(fq):
    """The same without a bias of -inf: a group of one leading and very poor experts
    loses to the others by the sum of its best two choices."""
    logits = torch.full((3, 8), -100.0, device="cuda")
    logits[:, 0] = 0.0
    logits[:, 4:] = torch.tensor([-95.0, -96.0, -97.5, -99.0], device="cuda")
    bias = torch.tensor([0.0, -5, -5, -5, 1, 1, 1, 1], device="cuda")
    w, ids = fq.moe_route(logits, 4, bias=bias, n_groups=2, keep_groups=1, group_top=2)
    assert ids.tolist() == [[4, 5, 6, 7]] * 3
    ref = weights64(logits, ids, "softmax", 1.0)
    assert bool(((w.double() - ref).abs() <= REL * ref).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_weights_against_differences(fq, score):
    """Central differences of the kernel's own weights, 95 to 100 below the leading
    logit (softmax) or at -100 to -95 (sigmoid): the backward pass is the derivative
    of the forward.  The bias decides the choice.  The third derivative of a
    normalised weight is below 8 (k = 3): off by 8 h^2 / 6, and by 2^-17 / h of
    rounding per term."""
    T, E, k, h = 6, 12, 3, 1.0 / 64
    logits, bias, gen = far_below(T, E, -100.0, -95.0, torch.float32, 5)
    logits = (logits * 1024).round() / 1024  # a step of 1/64 is exact
    if score == "sigmoid":
        logits[:, 0] = -100.0
    dw = torch.randn((T, k), device="cuda", generator=gen)
    _, ids = fq.moe_route(logits, k, bias=bias, score=score)
    d = fq.moe_route_backward(logits, ids, dw, score=score)
    assert bool((d.gather(1, ids.long()) != 0).any())
    tol = float(dw.abs().sum(1).max()) * (8 * h * h / 6 + REL / h)
    for e in range(E):
        side = []
        for sign in (1, -1):
            moved = logits.clone()
            moved[:, e] += sign * h
            w, i = fq.moe_route(moved, k, bias=bias, score=score)
            assert torch.equal(i, ids)
            side.append((w * dw).sum(1).double())
        diff = (side[0] - side[1]) / (2 * h)
        assert float((diff - d[:, e].double()).abs().max()) <= tol


@pytest.mark.parametrize("spread", [15.0, 30.0, 80.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(5, 2), (64, 8), (200, 32)])
def test_sigmoid_gradient_of_scores_next_to_one(fq, spread, dtype, renorm, E, k):
    """s (1 - s) has to keep its relative accuracy where s rounds to 1."""
    gen = torch.Generator(device="cuda").manual_seed(E)
    logits = ((torch.rand((50, E), device="cuda", generator=gen) * 2 - 1) * spread).to(dtype)
    ids = torch.stack([torch.randperm(E, device="cuda", generator=gen)[:k] for _ in range(50)]).int()
    # the chosen within 45 of each other (a renormalised weight's range)
    logits.scatter_(1, ids.long(), logits.gather(1, ids.long()).clamp(min=spread - 45))
    dw = torch.randn((50, k), device="cuda", generator=gen)
    d = fq.moe_route_backward(logits, ids, dw, score="sigmoid", renormalize=renorm, scale=2.5)
    close(d, *gradient64(logits, ids, dw, "sigmoid", renorm, 2.5))


@pytest.mark.parametrize("low,high", [(-100.0, -60.0), (-90.0, -80.0), (-145.0, -105.0), (-30.0, 15.0)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(9, 1), (33, 4), (256, 8)])
def test_sigmoid_weights_of_tiny_scores(fq, low, high, dtype, E, k):
    """Renormalised weights are quotients of scores that may lie below binary32's
    numbers; the gradient is of the size of dweights, which is large here."""
    logits, bias, gen = far_below(40, E, low, high, dtype, E)
    w, ids = fq.moe_route(logits, k, bias=bias, score="sigmoid", scale=2.5)
    if high < -20:  # the scores do not move the choice
        assert torch.equal(ids, torch.argsort(bias, descending=True)[:k].int().expand(40, k))
    ref = weights64(logits, ids, "sigmoid", 2.5)
    assert bool(((w.double() - ref).abs() <= REL * ref).all())
    dw = 3000.0 * torch.randn((40, k), device="cuda", generator=gen)
    d = fq.moe_route_backward(logits, ids, dw, score="sigmoid", scale=2.5)
    close(d, *gradient64(logits, ids, dw, "sigmoid", True, 2.5))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(3, 3), (40, 6), (40, 32), (300, 8)])
def test_gradients_of_an_id_that_stands_twice_are_added(fq, score, renorm, dtype, E, k):
    """Ids drawn with repetition, some without an expert: every slot's gradient
    counts, and the bits are the same each time."""
    gen = torch.Generator(device="cuda").manual_seed(E + k)
    logits = (torch.rand((60, E), device="cuda", generator=gen) * 10 - 5).to(dtype)
    ids = torch.randint(-1, min(E, 7), (60, k), device="cuda", generator=gen, dtype=torch.int32)
    ids[0] = 2
    dw = torch.randn((60, k), device="cuda", generator=gen)
    d = fq.moe_route_backward(logits, ids, dw, score=score, renormalize=renorm, scale=2.5)
    close(d, *gradient64(logits, ids, dw, score, renorm, 2.5))
    again = fq.moe_route_backward(logits, ids, dw, score=score, renormalize=renorm, scale=2.5)
    assert torch.equal(d, again)
