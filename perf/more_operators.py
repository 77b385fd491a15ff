"""Routing with scores, bias and groups, and the shared projection with low-rank adapters, as
measured work: cases, inputs, plain forms and 64-bit forms.

Operators (`case["op"]`):
  route  scores of a router's logits -> expert ids and weights: softmax or sigmoid, a bias that only
         the choice sees, groups of experts, top-k, renormalised weights
  lora   rows times a shared projection plus each row's own low-rank adapter, as a shared expert's
         gate/up product (with SiLU) or its down product

`own` false: elementary torch operations in 32 bits (the choice of experts in 64, since a score next
to a border decides whole numbers), rounded once at the end.  `own` true: the calls a user makes of
the framework.
"""
import math
import random

import torch

own = False

DEV = "cuda"
WEIGHT_STD = 0.02


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding sequence: all latency
        {"name": "route one token", "op": "route", "T": 1, "E": 256, "k": 8, "scoring": "sigmoid",
         "bias": True, "groups": 8, "topk_group": 4, "best": 2, "renormalize": True, "scale": 2.5,
         "dtype": "f32", "masked": 0.0, "pad": 0},
        # a decode batch of the plain softmax router
        {"name": "route decode softmax", "op": "route", "T": 64, "E": 256, "k": 6,
         "scoring": "softmax", "bias": False, "groups": 1, "topk_group": 1, "best": 1,
         "renormalize": True, "scale": 1.0, "dtype": "f32", "masked": 0.0, "pad": 0},
        # odd sizes, bf16 logits (ties), masked experts and tokens, rows of a wider matrix
        {"name": "route ragged masked", "op": "route", "T": 777, "E": 150, "k": 5,
         "scoring": "softmax", "bias": False, "groups": 5, "topk_group": 3, "best": 1,
         "renormalize": False, "scale": 1.0, "dtype": "bf16", "masked": 0.2, "pad": 10},
        # a prefill chunk, sigmoid scores with a balance bias, no groups
        {"name": "route prefill sigmoid", "op": "route", "T": 2048, "E": 384, "k": 6,
         "scoring": "sigmoid", "bias": True, "groups": 1, "topk_group": 1, "best": 1,
         "renormalize": True, "scale": 1.0, "dtype": "f32", "masked": 0.0, "pad": 0},
        # the most experts of the layer, softmax with a bias
        {"name": "route most experts", "op": "route", "T": 4096, "E": 1024, "k": 8,
         "scoring": "softmax", "bias": True, "groups": 1, "topk_group": 1, "best": 1,
         "renormalize": False, "scale": 1.5, "dtype": "bf16", "masked": 0.0, "pad": 0},
        # a long prefill with groups
        {"name": "route long prefill groups", "op": "route", "T": 16384, "E": 256, "k": 8,
         "scoring": "sigmoid", "bias": True, "groups": 8, "topk_group": 4, "best": 2,
         "renormalize": True, "scale": 2.5, "dtype": "f32", "masked": 0.0, "pad": 0},
        # the smallest projection: latency of the launches
        {"name": "lora tiny", "op": "lora", "M": 3, "N": 192, "K": 256, "r": 8, "L": 2, "slices": 1,
         "epilogue": "none", "order": "mixed", "without": 0.3, "pad": 0},
        # one decoding sequence on its adapter, gate/up of two shared experts of width 2048
        {"name": "lora one token gate/up", "op": "lora", "M": 1, "N": 8192, "K": 4096, "r": 16,
         "L": 8, "slices": 2, "epilogue": "silu", "order": "mixed", "without": 0.0, "pad": 0},
        # a decode batch, every sequence on an adapter of its own choice
        {"name": "lora decode gate/up", "op": "lora", "M": 16, "N": 8192, "K": 4096, "r": 16,
         "L": 32, "slices": 2, "epilogue": "silu", "order": "mixed", "without": 0.1, "pad": 0},
        # a larger decode batch through the down projection, rank 64
        {"name": "lora decode down", "op": "lora", "M": 64, "N": 4096, "K": 4096, "r": 64, "L": 40,
         "slices": 1, "epilogue": "none", "order": "mixed", "without": 0.1, "pad": 0},
        # sizes off every tile, a prefill and decoding sequences together, rows of a wider matrix
        {"name": "lora ragged", "op": "lora", "M": 777, "N": 1504, "K": 1448, "r": 24, "L": 9,
         "slices": 1, "epilogue": "none", "order": "mixed", "without": 0.3, "pad": 24},
        # a prefill chunk of a few requests
        {"name": "lora prefill gate/up", "op": "lora", "M": 2048, "N": 8192, "K": 4096, "r": 16,
         "L": 6, "slices": 2, "epilogue": "silu", "order": "runs", "without": 0.1, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    if rng.random() < 0.5:
        while True:
            T, E = _log_int(rng, 1, 16384), _log_int(rng, 2, 1024)
            if T * E <= 16384 * 256:
                break
        groups = rng.choice([1, 1] + [g for g in range(2, 33) if E % g == 0])
        topk_group = rng.randint(1, groups)
        k = rng.randint(1, min(8, topk_group * (E // groups)))
        return {"op": "route", "T": T, "E": E, "k": k, "scoring": rng.choice(("sigmoid", "softmax")),
                "bias": rng.random() < 0.6, "groups": groups, "topk_group": topk_group,
                "best": rng.choice((1, 2)), "renormalize": rng.random() < 0.7,
                "scale": rng.choice((1.0, 1.5, 2.5)), "dtype": rng.choice(("f32", "f32", "bf16")),
                "masked": rng.choice((0.0, 0.0, 0.1, 0.6)), "pad": rng.choice((0, 0, 2, 24))}
    while True:
        M = _log_int(rng, 1, 2048)
        slices, silu = rng.choice((1, 2)), rng.random() < 0.5
        N, K = 32 * _log_int(rng, 1, 256), 8 * _log_int(rng, 2, 768)
        r, L = 8 * rng.choice((1, 1, 2, 2, 3, 4, 8)), _log_int(rng, 1, 64)
        if M * N * K <= 2048 * 8192 * 4096 and N * K <= 8192 * 4096 and \
                L * r * (slices * K + N) <= 1 << 25:
            return {"op": "lora", "M": M, "N": N, "K": K, "r": r, "L": L, "slices": slices,
                    "epilogue": "silu" if silu else "none", "order": rng.choice(("runs", "mixed")),
                    "without": rng.choice((0.0, 0.1, 0.5)), "pad": rng.choice((0, 0, 8, 56))}


# ------------------------------------------------------------------ inputs
def _gen(seed, tag):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + tag * 7919) % (1 << 62))
    return g


def _router_logits(case, seed):
    """A router's logits: unit variance, some experts liked better than others, a share of the
    (token, expert) pairs masked and, with masks, one token without any expert."""
    T, E = case["T"], case["E"]
    g = _gen(seed, 1)
    liked = torch.randn(E, generator=g, device=DEV) * 0.5
    wide = torch.randn(T, E + case["pad"], generator=g, device=DEV)
    wide[:, :E] += liked
    if case["masked"] > 0:
        drop = torch.rand(T, E, generator=g, device=DEV) < case["masked"]
        drop[T // 2] = True
        wide[:, :E] = wide[:, :E].masked_fill(drop, float("-inf"))
    wide = wide.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    # a bias that has learned to push the liked experts back
    spread = 0.2 if case["scoring"] == "sigmoid" else 1.0 / E
    bias = (torch.randn(E, generator=g, device=DEV) * 0.3 - liked) * spread if case["bias"] else None
    return wide[:, :E], bias


def _adapter_ids(case, seed):
    """The adapter of every row (-1: none): decoding sequences in any order, or the rows of a few
    prefilled requests one after another."""
    M, L = case["M"], case["L"]
    g = _gen(seed, 2)
    if case["order"] == "mixed":
        ids = torch.randint(0, L, (M,), generator=g, device=DEV)
        ids[torch.rand(M, generator=g, device=DEV) < case["without"]] = -1
        return ids.to(torch.int32)
    n = max(1, min(M, L + 1))                          # requests
    cut = torch.sort(torch.randint(0, M + 1, (n - 1,), generator=g, device=DEV)).values
    request = torch.bucketize(torch.arange(M, device=DEV), cut, right=True)
    of = torch.randint(0, L, (n,), generator=g, device=DEV)
    of[torch.rand(n, generator=g, device=DEV) < case["without"]] = -1
    return of[request].to(torch.int32)


def prepare(case, seed):
    st = {"case": dict(case)}
    if case["op"] == "route":
        st["logits"], st["bias"] = _router_logits(case, seed)
        if own:
            st["ids"] = torch.empty(case["T"], case["k"], dtype=torch.int32, device=DEV)
            st["w"] = torch.empty(case["T"], case["k"], device=DEV)
        return st
    M, N, K, r, L, S = (case[n] for n in ("M", "N", "K", "r", "L", "slices"))
    g = _gen(seed, 3)
    x = torch.randn(M, K + case["pad"], generator=g, device=DEV)
    # activations as a layer meets them: a few channels much larger
    x[:, torch.randint(0, K, (max(1, K // 128),), generator=g, device=DEV)] *= 12.0
    st["x"] = x.to(torch.bfloat16)[:, :K]
    st["w"] = (torch.randn(N, K, generator=g, device=DEV) * WEIGHT_STD).to(torch.bfloat16)
    st["a"] = (torch.randn(L, S, r, K, generator=g, device=DEV) / math.sqrt(K)).to(torch.bfloat16)
    st["b"] = (torch.randn(L, N, r, generator=g, device=DEV) * 2 * WEIGHT_STD).to(torch.bfloat16)
    st["scale"] = torch.rand(L, generator=g, device=DEV) * 1.5 + 0.5
    ids = st["ids"] = _adapter_ids(case, seed)
    if own:
        import bit_quantized_moe_top_amd as mq
        # the batch's plan, which every projection of every layer reads, and the buffers
        st["plan"] = mq.moe_adapter_plan(ids, L)
        st["out"] = torch.empty(M, N // 2 if case["epilogue"] == "silu" else N, dtype=torch.bfloat16,
                                device=DEV)
        st["ws"] = torch.empty(mq.moe_shared_gemm_lora_ws_size(M, N, K, L, S, r), dtype=torch.uint8,
                               device=DEV)
    else:
        st["rows"] = [(l, torch.nonzero(ids == l).squeeze(1)) for l in sorted(set(ids.tolist()))
                      if l >= 0]
    return st


# -------------------------------------------------------------------- pass
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import bit_quantized_moe_top_amd as mq
    case = st["case"]
    if case["op"] == "route":
        scoring = mq.SCORE_SIGMOID if case["scoring"] == "sigmoid" else mq.SCORE_SOFTMAX
        ids, w = mq.moe_route_experts(
            st["logits"], case["k"], scoring=scoring, bias=st["bias"], n_group=case["groups"],
            topk_group=case["topk_group"], group_best=case["best"],
            renormalize=case["renormalize"], scale=case["scale"], ids=st["ids"], weights=st["w"])
        return {"ids": ids, "w": w}
    epilogue = mq.EPI_SILU_MUL if case["epilogue"] == "silu" else mq.EPI_NONE
    return mq.moe_shared_gemm_lora_bf16(st["x"], st["w"], st["a"], st["b"], st["scale"], st["plan"],
                                        epilogue=epilogue, out=st["out"], ws=st["ws"])


def _run_plain(st):
    return _plain_route(st) if st["case"]["op"] == "route" else _plain_lora(st)


def _plain_route(st):
    case, bias = st["case"], st["bias"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    low = float("-inf")
    logits = st["logits"].float()
    masked = logits == low
    wide = logits.double()
    top = wide.amax(1, keepdim=True)
    top = torch.where(top == low, torch.zeros_like(top), top)
    if case["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-wide))
    else:
        e = torch.exp(wide - top)
        score = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    choice = score if bias is None else score + bias.double()
    choice = choice.masked_fill(masked, low)
    if case["topk_group"] < G:
        best = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values[:, :, :case["best"]]
        group = torch.where(best == low, torch.zeros_like(best), best).sum(2)
        group = group.masked_fill(best[:, :, 0] == low, low)
        kept = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :case["topk_group"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        choice = choice.masked_fill(~keep.repeat_interleave(E // G, dim=1), low)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    live = torch.gather(choice, 1, ids) > low
    if case["scoring"] == "sigmoid":
        w = 1.0 / (1.0 + torch.exp(-torch.gather(logits, 1, ids)))
    else:
        e = torch.exp(logits - top.float())
        w = torch.gather(e, 1, ids) / e.sum(1, keepdim=True).clamp_min(1e-30)
    w = torch.where(live, w, torch.zeros_like(w))
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-30)
    return {"ids": ids.to(torch.int32), "w": w * case["scale"]}


def _plain_lora(st):
    case = st["case"]
    N, S = case["N"], case["slices"]
    x = st["x"].float()
    v = x @ st["w"].float().T
    for l, rows in st["rows"]:
        xl, part = x[rows], N // S
        b = st["b"][l].float() * st["scale"][l]
        for s in range(S):
            u = xl @ st["a"][l, s].float().T
            v[rows, s * part:(s + 1) * part] += u @ b[s * part:(s + 1) * part].T
    if case["epilogue"] == "silu":
        gate, up = v[:, :N // 2], v[:, N // 2:]
        v = gate / (1.0 + torch.exp(-gate)) * up
    return v.to(torch.bfloat16)


# ---------------------------------------------------------- the exact values
def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    return _exact_route(st) if case["op"] == "route" else _exact_lora(st)


def _picks(values, n):
    """The indices of every row's n largest entries, best first, the lowest index among equals."""
    at = torch.arange(values.shape[1], device=values.device).expand_as(values)
    taken = torch.zeros_like(values, dtype=torch.bool)
    picks = []
    for _ in range(n):
        top = values.masked_fill(taken, -math.inf).max(dim=1, keepdim=True).values
        first = torch.where((values == top) & ~taken, at, values.shape[1]).min(dim=1, keepdim=True)
        picks.append(first.values)
        taken.scatter_(1, first.values, True)
    return torch.cat(picks, dim=1)


def _exact_route(st):
    case = st["case"]
    E, k, G = case["E"], case["k"], case["groups"]
    size, none = E // G, -math.inf
    z = st["logits"].to(torch.float64)
    score = torch.sigmoid(z) if case["scoring"] == "sigmoid" else \
        torch.nan_to_num(torch.softmax(z, dim=1), nan=0.0)
    c = score.clone() if st["bias"] is None else score + st["bias"].to(torch.float64)
    c[torch.isneginf(z)] = none
    if case["topk_group"] < G:
        total = []
        for g in range(G):
            part = c[:, g * size:(g + 1) * size].clone()
            at = _picks(part, 1)
            first = part.gather(1, at).squeeze(1)
            part.scatter_(1, at, none)
            second = part.max(dim=1).values if case["best"] == 2 else torch.full_like(first, none)
            total.append(torch.where(torch.isneginf(second), first, first + second))
        kept = _picks(torch.stack(total, dim=1), case["topk_group"])
        gone = torch.ones(z.shape[0], G, dtype=torch.bool, device=z.device).scatter_(1, kept, False)
        c[gone.repeat_interleave(size, dim=1)] = none
    ids = _picks(c, k)
    w = torch.where(torch.isneginf(c.gather(1, ids)), 0.0, score.gather(1, ids))
    if case["renormalize"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1.0), 0.0)
    return {"ids": ids.to(torch.int32), "w": w * case["scale"]}


def _exact_lora(st):
    case = st["case"]
    M, N, S = case["M"], case["N"], case["slices"]
    x = st["x"].to(torch.float64)
    w = st["w"].to(torch.float64)
    parts = []
    ids = st["ids"].long()
    for s in range(S):
        cols = slice(s * (N // S), (s + 1) * (N // S))
        v = torch.mm(x, w[cols].t().contiguous())
        for l in range(case["L"]):
            mine = torch.nonzero(ids == l)[:, 0]
            if mine.numel() == 0:
                continue
            low = torch.mm(x.index_select(0, mine), st["a"][l, s].to(torch.float64).t().contiguous())
            full = torch.mm(low, st["b"][l, cols].to(torch.float64).t().contiguous())
            v.index_add_(0, mine, full * st["scale"][l].to(torch.float64))
        parts.append(v)
    v = torch.cat(parts, dim=1)
    if case["epilogue"] == "silu":
        v = v[:, :N // 2] * torch.sigmoid(v[:, :N // 2]) * v[:, N // 2:]
    return v


# -------------------------------------------------------------------- work
def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        # the logits and the bias in, ids and weights out; a score and k comparisons an expert
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 8 * T * k,
                "flops": T * E * 10}
    M, N, K, r, L, S = (case[n] for n in ("M", "N", "K", "r", "L", "slices"))
    rows = M * (1.0 - case["without"])
    # adapters that `rows` uniform choices reach, on average
    reached = min(rows, L) if L == 1 else L * (1.0 - (1.0 - 1.0 / L) ** rows)
    cols = N // 2 if case["epilogue"] == "silu" else N
    return {"bytes": 2 * (M * K + N * K + reached * r * (S * K + N) + M * cols),
            "flops": 2 * M * N * K + 2 * rows * r * (S * K + N)}
