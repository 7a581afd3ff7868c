"""The operators of a mixture-of-experts FP8 layer, each in its plain form and through the library.

Five operators that run one after the other in such a layer, forward and backward:

* ``route``   ``moe_route`` (and ``moe_route_backward``): softmax or sigmoid scores, a selection
              bias, expert groups, top-k, renormalised weights.
* ``sort``    ``moe_sort_rows``: (token, choice) pairs ordered by expert; the group offsets that
              every ragged call of the library takes.
* ``matmul``  ``fp8_matmul``: E4M3 rows with 1x128 scales times E4M3 weights with 128x128 (or
              1x128) scales, for one weight or for the experts of ragged groups of rows.
* ``cols``    ``fp8_quantize_cols``: BF16 to transposed E4M3 with 128-token blocks per group, the
              weight gradient's operand layout.
* ``wgrad``   ``fp8_matmul_wgrad``: the product over the tokens of each group.

With ``own`` false, ``run`` computes an operator with elementary torch operations in 32 bits; with
``own`` true it makes the library's calls on the same state.
"""
import math

import numpy as np
import torch

own = False

FLT_MAX = 3.4028234663852886e38
MASKED = -3.3895313892515355e38  # BF16's lowest finite value: a logit at or below it masks its expert
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- the cases

def _route(name, T, E, k, score="softmax", bias=False, groups=1, keep=1, top=1, renorm=True,
           scale=1.0, dtype="f32", masked=False, grad=False):
    c = dict(op="route", T=T, E=E, k=k, score=score, bias=bias, groups=groups, keep=keep, top=top,
             renorm=renorm, scale=scale, dtype=dtype, masked=masked, grad=grad)
    return dict(c, name=name) if name else c


def _sort(name, T, k, E, dropped=False):
    c = dict(op="sort", T=T, k=k, E=E, dropped=dropped)
    return dict(c, name=name) if name else c


def _matmul(name, M, N, K, G=0, split="zipf", w_block=128, out="bf16"):
    c = dict(op="matmul", M=M, N=N, K=K, G=G, split=split, w_block=w_block, out=out)
    return dict(c, name=name) if name else c


def _cols(name, M, K, G, split="zipf"):
    c = dict(op="cols", M=M, K=K, G=G, split=split)
    return dict(c, name=name) if name else c


def _wgrad(name, M, N, K, G, split="zipf", out="f32"):
    c = dict(op="wgrad", M=M, N=N, K=K, G=G, split=split, out=out)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decode step of eight sequences: sigmoid scores, balance bias, 4 of 8 expert groups
        _route("route_decode", 8, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
        # a training batch's router, forward and backward, BF16 logits with some masked experts
        _route("route_train", 16384, 256, 8, "softmax", dtype="bf16", masked=True, grad=True),
        # the pairs of a decode step of 64 sequences
        _sort("sort_decode", 64, 8, 32),
        # the pairs of a training batch over many experts, with padded tokens
        _sort("sort_train", 65536, 8, 256, True),
        # one token through one weight: the latency and bandwidth of a dense decode step
        _matmul("matmul_one_token", 1, 14336, 4096),
        # a whole batch through one dense weight
        _matmul("matmul_dense", 16384, 4096, 7168),
        # a decode step's 64 x 8 rows through 32 experts (gate and up projection together)
        _matmul("experts_decode", 512, 4096, 7168, 32, "even"),
        # a training batch's ragged rows through 32 experts (down projection)
        _matmul("experts_train", 65536, 7168, 2048, 32),
        # few ragged tokens, odd count: rows of the transposed codes are not aligned
        _cols("cols_odd", 1003, 1408, 8, "holes"),
        # the gradient columns of a training batch
        _cols("cols_train", 65536, 2048, 32),
        # few ragged tokens, odd count, empty groups
        _wgrad("wgrad_odd", 1003, 1408, 2048, 8, "holes"),
        # the weight gradients of 32 experts over a training batch
        _wgrad("wgrad_train", 65536, 2048, 7168, 32),
    ]


def _log_int(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    v = min(max(v, -(-lo // step) * step), hi // step * step)
    return v + step if v == 24 * 128 else v


def draw(rng):
    op = rng.choice(["route", "sort", "matmul", "matmul", "matmul", "cols", "wgrad"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log_int(rng, max(2, 8 // groups), 512 // groups)
        keep = rng.randint(max(1, groups // 4), groups)
        score = rng.choice(["softmax", "sigmoid"])
        return _route("", _log_int(rng, 1, 16384), E, rng.randint(1, min(8, keep * (E // groups))),
                      score, score == "sigmoid" and rng.random() < 0.7, groups, keep,
                      rng.choice([1, 2]) if groups > 1 and E // groups > 1 else 1,
                      rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.choice(["f32", "bf16"]),
                      rng.random() < 0.5, rng.random() < 0.5)
    if op == "sort":
        E = _log_int(rng, 8, 512)
        return _sort("", _log_int(rng, 1, 65536), rng.randint(1, 8), E, rng.random() < 0.5)
    split = rng.choice(["zipf", "even", "holes"])
    if op == "matmul":
        G = 0 if rng.random() < 0.4 else _log_int(rng, 1, 32)
        M, N = _log_int(rng, 1, 65536 if G else 16384), _log_int(rng, 64, 8192, 8)
        K = _log_int(rng, 128, 7168, 128)
        while 2 * M * N * K > 0.96e12:
            M = M * 3 // 4
        return _matmul("", M, N, K, G, split, rng.choice([128, 128, 1]), rng.choice(["bf16", "bf16", "f32"]))
    if op == "cols":
        return _cols("", _log_int(rng, 1, 65536), _log_int(rng, 128, 2048, 128), _log_int(rng, 1, 32), split)
    M, N = _log_int(rng, 1, 65536), _log_int(rng, 128, 4096, 128)
    return _wgrad("", M, N, _log_int(rng, 128, 7168, 128), _log_int(rng, 1, 16), split,
                  rng.choice(["f32", "f32", "bf16"]))


# ---------------------------------------------------------------- inputs

def _offsets(M, G, split, seed):
    """Group offsets, as a list: Zipf(1.1) counts, equal odds, or equal odds with empty groups."""
    rng = np.random.default_rng(seed)
    p = np.arange(1, G + 1, dtype=np.float64) ** -1.1 if split == "zipf" else np.ones(G)
    if split == "holes":
        p[rng.permutation(G)[:G // 3]] = 0
    counts = np.bincount(rng.choice(G, size=M, p=p / p.sum()), minlength=G)
    return [0] + [int(v) for v in np.cumsum(counts)]


def _e4m3_blocks(x):
    """E4M3 codes and scales of blocks along the last axis ([..., block] float32): 448 / amax
    scaling, a block with NaN or Inf gets scale NaN and NaN codes."""
    amax = x.abs().amax(-1, keepdim=True)
    bad = ~torch.isfinite(amax)
    y = (x * (448.0 / amax).clamp(max=FLT_MAX)).clamp(-448.0, 448.0)
    nan = torch.full_like(amax, float("nan"))
    codes = torch.where(bad, nan, y).to(torch.float8_e4m3fn)
    return codes, torch.where(bad, nan, amax / 448.0).squeeze(-1)


def _slots(offsets, M):
    """For each token the row of the block-padded layout that holds it: 128-token blocks from each
    group's first token on."""
    counts = offsets[1:] - offsets[:-1]
    blocks = (counts + 127) // 128
    base = torch.cumsum(blocks, 0) - blocks
    t = torch.arange(M, device=offsets.device)
    g = torch.searchsorted(offsets[1:].contiguous(), t, right=True)
    return base[g] * 128 + t - offsets[g]


def _plain_cols(x, offsets):
    M, K = x.shape
    cap = -(-M // 128) + offsets.numel() - 1
    slots = _slots(offsets, M)
    padded = torch.zeros((cap * 128, K), dtype=torch.float32, device=x.device)
    padded[slots] = x.float()
    codes, scales = _e4m3_blocks(padded.view(cap, 128, K).transpose(1, 2))
    codes = codes.transpose(1, 2).reshape(cap * 128, K).view(torch.uint8)
    return codes[slots].t().contiguous(), scales.contiguous()


def _rows_fp8(x):
    M, K = x.shape
    codes, scales = _e4m3_blocks(x.float().view(M, K // 128, 128))
    return codes.view(torch.uint8).view(M, K), scales


def _tiles_fp8(w):
    N, K = w.shape
    n = -(-N // 128)
    p = torch.zeros((n * 128, K), dtype=torch.float32, device=w.device)
    p[:N] = w.float()
    t = p.view(n, 128, K // 128, 128).permute(0, 2, 1, 3).reshape(n, K // 128, 128 * 128)
    codes, scales = _e4m3_blocks(t)
    codes = codes.view(torch.uint8).view(n, K // 128, 128, 128).permute(0, 2, 1, 3)
    return codes.reshape(n * 128, K)[:N].contiguous(), scales


def _activations(M, K, gen):
    x = torch.randn((M, K), device="cuda", generator=gen)
    x *= torch.exp(torch.randn((M, 1), device="cuda", generator=gen))
    return x.bfloat16()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": dict(case)}
    op = case["op"]
    if op == "route":
        T, E = case["T"], case["E"]
        logits = 1.5 * torch.randn((T, E), device="cuda", generator=gen)
        logits += 0.5 * torch.randn((1, E), device="cuda", generator=gen)  # popular experts
        if case["masked"]:  # an expert out of service, and padded tokens with no expert at all
            logits[:, torch.randint(0, E, (1,), device="cuda", generator=gen)] = float("-inf")
            logits[torch.rand((T,), device="cuda", generator=gen) < 0.03] = float("-inf")
        st["logits"] = logits.to(DTYPES[case["dtype"]])
        st["bias"] = 0.1 * torch.randn((E,), device="cuda", generator=gen) if case["bias"] else None
        st["dweights"] = torch.randn((T, case["k"]), device="cuda", generator=gen)
    elif op == "sort":
        T, k, E = case["T"], case["k"], case["E"]
        odds = 1.1 * torch.log(torch.arange(1, E + 1, device="cuda").float())  # Zipf popularity
        noise = torch.rand((T, E), device="cuda", generator=gen).clamp_(1e-7, 1 - 1e-7)
        ids = torch.topk(-torch.log(-torch.log(noise)) - odds, k, dim=1).indices.int()
        if case["dropped"]:
            ids[torch.rand((T,), device="cuda", generator=gen) < 0.03] = -1
        st["ids"] = ids.contiguous()
    elif op == "matmul":
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        st["y"], st["ys"] = _rows_fp8(_activations(M, K, gen))
        rows, sets = (1 if case["w_block"] == 1 else 128), max(G, 1)
        w = torch.empty((sets, N, K), dtype=torch.uint8, device="cuda")
        ws = torch.empty((sets, -(-N // rows), K // 128), dtype=torch.float32, device="cuda")
        for g in range(sets):
            wg = (0.02 * torch.randn((N, K), device="cuda", generator=gen)).bfloat16()
            w[g], ws[g] = _rows_fp8(wg) if rows == 1 else _tiles_fp8(wg)
        st["w"], st["ws"], st["offsets"] = (w, ws, None) if G else (w[0], ws[0], None)
        st["bounds"] = _offsets(M, G, case["split"], seed) if G else [0, M]
        if G:
            st["offsets"] = torch.tensor(st["bounds"], dtype=torch.int64, device="cuda")
    elif op == "cols":
        st["x"] = _activations(case["M"], case["K"], gen)
        st["offsets"] = torch.tensor(_offsets(case["M"], case["G"], case["split"], seed),
                                     dtype=torch.int64, device="cuda")
    else:
        M = case["M"]
        st["bounds"] = _offsets(M, case["G"], case["split"], seed)
        st["offsets"] = torch.tensor(st["bounds"], dtype=torch.int64, device="cuda")
        st["a"], st["as"] = _plain_cols(_activations(M, case["N"], gen), st["offsets"])
        st["b"], st["bs"] = _plain_cols(_activations(M, case["K"], gen), st["offsets"])
    return st


# ---------------------------------------------------------------- plain forms

def _plain_scores(case, logits):
    """(availability, scores that the choice compares, scores that weigh)."""
    l = logits.float()
    ok = l > MASKED
    l = torch.where(ok, l.clamp(max=FLT_MAX), torch.full_like(l, -FLT_MAX))
    if case["score"] == "sigmoid":
        s = torch.where(ok, 1 / (1 + torch.exp(-l)), torch.zeros_like(l))
        return ok, s, s
    e = torch.where(ok, torch.exp(l - l.amax(-1, keepdim=True)), torch.zeros_like(l))
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    return ok, e, p  # e and p are in the same order


def _plain_route(st):
    c, logits = st["case"], st["logits"]
    T, E, k = c["T"], c["E"], c["k"]
    none = float("-inf")
    ok, choice, score = _plain_scores(c, logits)
    if st["bias"] is not None:
        choice = (score if c["score"] == "softmax" else choice) + st["bias"]
    choice = torch.where(ok, choice, torch.full_like(choice, none))
    if c["groups"] > 1:
        per = choice.view(T, c["groups"], -1)
        best = torch.sort(per, dim=-1, descending=True).values[..., :c["top"]]
        total = torch.where(best > none, best, torch.zeros_like(best)).sum(-1)
        total = torch.where(best[..., 0] > none, total, torch.full_like(total, none))
        first = torch.sort(total, dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros_like(total, dtype=torch.bool).scatter(1, first, True)
        choice = torch.where(kept.unsqueeze(-1), per, torch.full_like(per, none)).view(T, E)
    value, ids = torch.sort(choice, dim=-1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    there = value > none
    w = torch.where(there, score.gather(1, ids), torch.zeros_like(value))
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return w * c["scale"], torch.where(there, ids, torch.full_like(ids, -1)).int()


def _plain_route_backward(st, ids):
    """Chain rule from the weights back to the logits; an id of -1 has none."""
    c, logits = st["case"], st["logits"]
    _, _, score = _plain_scores(c, logits)
    there = ids >= 0
    at = ids.long().clamp(min=0)
    s = torch.where(there, score.gather(1, at), torch.zeros_like(st["dweights"]))
    ds = torch.where(there, st["dweights"], torch.zeros_like(s)) * c["scale"]
    if c["renorm"]:
        total = s.sum(-1, keepdim=True)
        ds = torch.where(total > 0, (ds - (ds * s).sum(-1, keepdim=True) / total) / total,
                         torch.zeros_like(ds))
    full = torch.zeros_like(score).scatter_add(1, at, torch.where(there, ds, torch.zeros_like(ds)))
    if c["score"] == "sigmoid":
        d = full * score * (1 - score)
    else:
        d = score * (full - (full * score).sum(-1, keepdim=True))
    return d.to(logits.dtype)


def _plain_sort(ids, E):
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    ordered, pair = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(E + 1, device=ids.device))
    row = torch.empty_like(flat)
    row[pair] = torch.arange(n, device=ids.device)
    none = torch.full_like(flat, -1)
    pair = torch.where(ordered < E, pair, none)
    row = torch.where(key < E, row, none)
    return offsets, pair.int(), row.int().view(ids.shape)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def _plain_weight(case, w, ws):
    if case["w_block"] == 1:
        return _values(w) * ws.repeat_interleave(128, 1)
    return _values(w) * ws.repeat_interleave(128, 0)[:case["N"]].repeat_interleave(128, 1)


def _plain_matmul(st):
    c = st["case"]
    a = _values(st["y"]) * st["ys"].repeat_interleave(128, 1)
    if not c["G"]:
        return (a @ _plain_weight(c, st["w"], st["ws"]).t()).to(DTYPES[c["out"]])
    out = torch.empty((c["M"], c["N"]), dtype=DTYPES[c["out"]], device="cuda")
    for g, (lo, hi) in enumerate(zip(st["bounds"], st["bounds"][1:])):  # ragged: a product a group
        if hi > lo:
            out[lo:hi] = a[lo:hi] @ _plain_weight(c, st["w"][g], st["ws"][g]).t()
    return out


def _plain_wgrad(st):
    c = st["case"]
    block = _slots(st["offsets"], c["M"]) // 128
    a = _values(st["a"]) * st["as"][block].t()
    b = _values(st["b"]) * st["bs"][block].t()
    out = torch.empty((c["G"], c["N"], c["K"]), dtype=DTYPES[c["out"]], device="cuda")
    for g, (lo, hi) in enumerate(zip(st["bounds"], st["bounds"][1:])):  # ragged: a product a group
        out[g] = a[:, lo:hi] @ b[:, lo:hi].t()
    return out


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        import fp8_quantization_gb300 as fq
    if op == "route":
        if own:
            w, ids = fq.moe_route(state["logits"], c["k"], bias=state["bias"], score=c["score"],
                                  n_groups=c["groups"], keep_groups=c["keep"], group_top=c["top"],
                                  renormalize=c["renorm"], scale=c["scale"])
            d = fq.moe_route_backward(state["logits"], ids, state["dweights"], score=c["score"],
                                      renormalize=c["renorm"], scale=c["scale"]) if c["grad"] else None
        else:
            w, ids = _plain_route(state)
            d = _plain_route_backward(state, ids) if c["grad"] else None
        return {"weights": w, "ids": ids, "dlogits": d}
    if op == "sort":
        offsets, pair, row = (fq.moe_sort_rows if own else _plain_sort)(state["ids"], c["E"])
        return {"offsets": offsets, "pair_of_row": pair, "row_of_pair": row}
    if op == "matmul":
        if own:
            return {"out": fq.fp8_matmul(state["y"], state["ys"], state["w"], state["ws"],
                                         state["offsets"], out_dtype=DTYPES[c["out"]])}
        return {"out": _plain_matmul(state)}
    if op == "cols":
        yT, scales = (fq.fp8_quantize_cols if own else _plain_cols)(state["x"], state["offsets"])
        return {"codes": yT.view(torch.float8_e4m3fn), "scales": scales}
    if own:
        return {"out": fq.fp8_matmul_wgrad(state["a"], state["as"], state["b"], state["bs"],
                                           state["offsets"], out_dtype=DTYPES[c["out"]])}
    return {"out": _plain_wgrad(state)}


# ---------------------------------------------------------------- what a pass needs

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "f32" else 2
        once = T * E * size + 8 * T * k + (4 * E if case["bias"] else 0)
        return {"bytes": once + (T * E * size + 4 * T * k if case["grad"] else 0),
                "flops": T * E * (10 if case["grad"] else 5)}
    if op == "sort":
        n = case["T"] * case["k"]
        return {"bytes": 12 * n + 8 * (case["E"] + 1), "flops": n}
    M, K = case["M"], case["K"]
    size = {"bf16": 2, "f32": 4}
    if op == "matmul":
        N, sets = case["N"], min(max(case["G"], 1), max(M, 1))
        scales = 4 * (M * (K // 128) + sets * -(-N // case["w_block"]) * (K // 128))
        return {"bytes": M * K + sets * N * K + scales + M * N * size[case["out"]],
                "flops": 2 * M * N * K}
    blocks = -(-M // 128)
    if op == "cols":
        return {"bytes": 3 * M * K + 4 * blocks * K, "flops": 2 * M * K}
    N, G = case["N"], case["G"]
    return {"bytes": M * (N + K) + 4 * blocks * (N + K) + G * N * K * size[case["out"]],
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_route(case, st):
    T, E, k = case["T"], case["E"], case["k"]
    logits = st["logits"].double()
    gone = logits <= MASKED
    if case["score"] == "sigmoid":
        score = torch.sigmoid(logits)
    else:
        score = torch.nan_to_num(torch.softmax(logits.masked_fill(gone, -math.inf), 1), 0.0)
    score = score.masked_fill(gone, 0.0)
    pick = score + (0.0 if st["bias"] is None else st["bias"].double())
    pick = pick.masked_fill(gone, -math.inf)
    if case["groups"] > 1:
        by = pick.reshape(T, case["groups"], E // case["groups"])
        v = by.topk(case["top"], -1).values
        mark = v.masked_fill(v == -math.inf, 0.0).sum(-1).masked_fill(v[..., 0] == -math.inf, -math.inf)
        lose = torch.ones_like(mark, dtype=torch.bool)
        lose.scatter_(1, mark.sort(dim=1, descending=True, stable=True).indices[:, :case["keep"]], False)
        pick = by.masked_fill(lose[..., None], -math.inf).reshape(T, E)
    order = pick.sort(dim=1, descending=True, stable=True)
    ids, missing = order.indices[:, :k], order.values[:, :k] == -math.inf
    mask = torch.zeros_like(score).scatter(1, ids, (~missing).double())
    s = score
    dw = torch.zeros_like(score).scatter(1, ids, st["dweights"].double().masked_fill(missing, 0.0))
    scale = float(case["scale"])
    chosen = s * mask
    if case["renorm"]:
        norm = chosen.sum(1, keepdim=True)
        inv = torch.where(norm > 0, 1 / norm.clamp(min=1e-300), torch.zeros_like(norm))
        weights = chosen * inv * scale
        back = mask * scale * inv * (dw - (dw * chosen).sum(1, keepdim=True) * inv)
    else:
        weights, back = chosen * scale, mask * scale * dw
    slope = back * s * (1 - s) if case["score"] == "sigmoid" else s * (back - (back * s).sum(1, keepdim=True))
    return {"weights": weights.gather(1, ids).masked_fill(missing, 0.0), "ids": None,
            "dlogits": slope if case["grad"] else None}


def _f64(codes):
    return codes.view(torch.float8_e4m3fn).double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(case, st)
    if op == "sort":
        return None
    if op == "cols":
        M, K = case["M"], case["K"]
        lo = st["offsets"].tolist()
        rows = [(st["x"][t:min(t + 128, b)].abs().amax(0).double() / 448)
                for a, b in zip(lo, lo[1:]) for t in range(a, b, 128)]
        scales = torch.zeros((-(-M // 128) + case["G"], K), dtype=torch.float64, device="cuda")
        scales[:len(rows)] = torch.stack(rows)
        return {"codes": None, "scales": scales}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        out = torch.empty((M, N), dtype=torch.float64, device="cuda")
        a = (_f64(st["y"]).view(M, K // 128, 128) * st["ys"].double()[..., None]).view(M, K)
        w, ws = (st["w"], st["ws"]) if case["G"] else (st["w"][None], st["ws"][None])
        for g, (lo, hi) in enumerate(zip(st["bounds"], st["bounds"][1:])):
            n = torch.arange(N, device="cuda") // case["w_block"]
            b = (_f64(w[g]).view(N, K // 128, 128) * ws[g].double()[n][..., None]).view(N, K)
            out[lo:hi] = a[lo:hi] @ b.t()
        return {"out": out}
    out = torch.zeros((case["G"], case["N"], case["K"]), dtype=torch.float64, device="cuda")
    block = 0
    for g, (lo, hi) in enumerate(zip(st["bounds"], st["bounds"][1:])):
        n = -(-(hi - lo) // 128)
        which = block + torch.arange(hi - lo, device="cuda") // 128
        a = _f64(st["a"][:, lo:hi].contiguous()) * st["as"].double()[which].t()
        b = _f64(st["b"][:, lo:hi].contiguous()) * st["bs"].double()[which].t()
        out[g] = a @ b.t()
        block += n
    return {"out": out}
