"""The MXFP4 operators as measured work: cases, inputs, plain forms and 64-bit forms.

MXFP4: E2M1 codes (two per byte, the low nibble first) with one E8M0 scale byte per 32
consecutive elements of a row.

Operators (`case["op"]`):
  quant  rows -> MXFP4 and the values it stands for (quantisation, then the read-back)
  gemm   grouped product over the routed experts, activations and weights in MXFP4
  layer  a whole expert layer for a few tokens: routing, gate/up, SiLU, down, weighted sum

`own` false: elementary torch operations in 32 bits, rounded once at the end.  `own` true: the
calls a user makes of the framework.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BLOCK = 32                                   # elements per E8M0 scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
WEIGHT_STD = 0.02


# ------------------------------------------------------------------- cases
def listed():
    return [
        # a decode batch's activations: the smallest call, all latency
        {"name": "quant decode x", "op": "quant", "M": 4, "K": 4096, "dtype": "bf16", "pad": 0},
        # the routed rows' h between the two products of a prefill layer
        {"name": "quant prefill h", "op": "quant", "M": 12288, "K": 2048, "dtype": "bf16", "pad": 0},
        # fp32 columns of a wider matrix (rows strided), neither side a multiple of a tile
        {"name": "quant fp32 strided", "op": "quant", "M": 3001, "K": 1440, "dtype": "f32", "pad": 96},
        # the smallest layer's gate/up product: latency of one launch
        {"name": "gemm tiny gate/up", "op": "gemm", "T": 16, "k": 2, "E": 8, "N": 256, "K": 256,
         "epilogue": "silu", "routing": "uniform", "out": "bf16"},
        # decode: about one row per expert, a stream of weights
        {"name": "gemm decode gate/up", "op": "gemm", "T": 4, "k": 6, "E": 256, "N": 4096,
         "K": 4096, "epilogue": "silu", "routing": "uniform", "out": "bf16"},
        # prefill chunk of 2048 tokens, near-uniform routing: 48 rows per expert
        {"name": "gemm prefill gate/up", "op": "gemm", "T": 2048, "k": 6, "E": 256, "N": 4096,
         "K": 4096, "epilogue": "silu", "routing": "uniform", "out": "bf16"},
        # the down product of a prefill chunk whose experts are Zipf-popular
        {"name": "gemm skewed down", "op": "gemm", "T": 2048, "k": 6, "E": 256, "N": 4096,
         "K": 2048, "epilogue": "none", "routing": "zipf", "out": "bf16"},
        # sizes off every tile, fp32 out, a few experts with many rows each
        {"name": "gemm ragged fp32", "op": "gemm", "T": 777, "k": 3, "E": 12, "N": 1504, "K": 1440,
         "epilogue": "none", "routing": "zipf", "out": "f32"},
        # the smallest layer: nothing but latency
        {"name": "layer tiny", "op": "layer", "T": 5, "k": 3, "E": 10, "H": 288, "I": 96,
         "bias": True, "shared": True, "renormalize": True},
        # one decoding sequence
        {"name": "layer T=1", "op": "layer", "T": 1, "k": 6, "E": 256, "H": 4096, "I": 2048,
         "bias": False, "shared": False, "renormalize": True},
        # four decoding sequences
        {"name": "layer T=4", "op": "layer", "T": 4, "k": 6, "E": 256, "H": 4096, "I": 2048,
         "bias": False, "shared": False, "renormalize": True},
        # the most tokens of the call, with a router bias and a shared expert's output
        {"name": "layer T=16", "op": "layer", "T": 16, "k": 6, "E": 256, "H": 4096, "I": 2048,
         "bias": True, "shared": True, "renormalize": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _blocks(rng, lo, hi):
    """A size in whole blocks of 32, from lo to hi blocks."""
    return BLOCK * _log_int(rng, lo, hi)


def draw(rng: random.Random):
    op = rng.choice(("quant", "gemm", "gemm", "layer"))
    if op == "quant":
        while True:
            M, K = _log_int(rng, 1, 16384), _blocks(rng, 1, 256)
            if M * K <= 12288 * 2048:
                return {"op": op, "M": M, "K": K, "dtype": rng.choice(("bf16", "f32")),
                        "pad": rng.choice((0, 0, 8, 64, 104))}
    if op == "gemm":
        while True:
            E = _log_int(rng, 1, 256)
            k = rng.randint(1, min(8, E))
            T, N, K = _log_int(rng, 1, 2048), _blocks(rng, 1, 128), _blocks(rng, 1, 128)
            if E * N * K <= 2 ** 31 and T * k * N * K <= 2 ** 37:
                break
        epi = rng.choice(("silu", "none"))
        return {"op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "epilogue": epi,
                "routing": rng.choice(("uniform", "zipf")),
                "out": "bf16" if epi == "silu" else rng.choice(("bf16", "f32"))}
    while True:
        E = _log_int(rng, 2, 256)
        k = rng.randint(1, min(8, E))
        T, H, I = rng.randint(1, 16), _blocks(rng, 1, 160), _blocks(rng, 1, 96)
        if E * H * I <= 2 ** 31 and T * k * H * I <= 96 * 4096 * 2048:
            return {"op": op, "T": T, "k": k, "E": E, "H": H, "I": I,
                    "bias": rng.random() < 0.5, "shared": rng.random() < 0.5,
                    "renormalize": rng.random() < 0.7}


# ---------------------------------------------------------- plain MXFP4 format
def _plain_quant(x):
    """x [..., K] fp32 -> (packed codes [..., K/2], scale bytes [..., K/32]), uint8."""
    b = x.float().reshape(*x.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    # floor(log2 a) from the exponent field in 64 bits, where every fp32 value is normal; E2M1's
    # largest exponent is 2
    log2 = (amax.double().view(torch.int64) >> 52) - 1023
    e = torch.where(amax > 0, log2 - 2, torch.full_like(log2, -127)).clamp_(-127, 127)
    y = (b.double() * torch.exp2(-e.double())).abs().float()
    # nearest E2M1 value, ties to the even code
    c = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) +
         (y >= 3.5) + (y > 5.0)).to(torch.uint8)
    c = c | (torch.signbit(b).to(torch.uint8) << 3)
    c = c.reshape(*x.shape[:-1], -1, 2)
    return c[..., 0] | (c[..., 1] << 4), (e + 127).to(torch.uint8).squeeze(-1)


def _plain_values(q, s, dtype=torch.float32):
    """Packed codes [..., K/2] and scale bytes [..., K/32] -> values [..., K]."""
    lut = torch.tensor([v * sg for sg in (1.0, -1.0) for v in E2M1], device=q.device)
    pairs = lut.to(dtype)[torch.stack((q & 15, q >> 4), -1).int()]
    v = pairs.reshape(*q.shape[:-1], -1, BLOCK)
    return (v * torch.exp2(s.to(dtype) - 127.0).unsqueeze(-1)).reshape(*q.shape[:-1], -1)


# ------------------------------------------------------------------ inputs
def _gen(seed, tag):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + tag * 7919) % (1 << 62))
    return g


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _weights(E, N, K, seed, tag):
    """Expert weights N(0, WEIGHT_STD), quantised: codes [E, N, K/2], scales [E, N, K/32]."""
    g = _gen(seed, tag)
    q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(E, N, K // BLOCK, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        q[e:e + n], s[e:e + n] = _plain_quant(
            torch.randn(n, N, K, generator=g, device=DEV) * WEIGHT_STD)
    return q, s


def _route_logits(T, E, routing, seed, tag):
    g = _gen(seed, tag)
    logits = torch.randn(T, E, generator=g, device=DEV)
    if routing == "zipf":                  # Gumbel noise over a log-Zipf popularity
        u = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-9, 1 - 1e-7)
        rank = torch.randperm(E, generator=g, device=DEV).float() + 1
        logits = -torch.log(-torch.log(u)) - 1.1 * torch.log(rank)
    return logits


def _hidden(rows, K, seed, tag):
    """Activations as a layer meets them: unit variance, a few channels much larger."""
    g = _gen(seed, tag)
    x = torch.randn(rows, K, generator=g, device=DEV)
    gain = torch.ones(K, device=DEV)
    gain[torch.randint(0, K, (max(1, K // 128),), generator=g, device=DEV)] = 12.0
    return x * gain


def prepare(case, seed):
    op = case["op"]
    st = {"case": dict(case)}
    if op == "quant":
        wide = _hidden(case["M"], case["K"] + case["pad"], seed, 1).to(_dtype(case["dtype"]))
        st["x"] = wide[:, :case["K"]]
    elif op == "gemm":
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        logits = _route_logits(T, E, case["routing"], seed, 2)
        ids = logits.topk(k, dim=1).indices.to(torch.int32)
        rows = T if case["epilogue"] == "silu" else T * k
        # gate/up reads each token's x; the down product reads h, one row per routed row
        a = _hidden(rows, K, seed, 3) if case["epilogue"] == "silu" else \
            torch.randn(rows, K, generator=_gen(seed, 3), device=DEV) ** 2 * 0.5
        st["a_q"], st["a_s"] = _plain_quant(a)
        st["w_q"], st["w_s"] = _weights(E, N, K, seed, 4)
        order = torch.argsort(ids.reshape(-1).long(), stable=True)
        st["order"] = order                               # plan position -> routed row
        st["counts"] = torch.bincount(ids.reshape(-1).long(), minlength=E).tolist()
        st["ids"] = ids
    else:
        T, E, H, I = (case[n] for n in ("T", "E", "H", "I"))
        st["x"] = _hidden(T, H, seed, 5).to(torch.bfloat16)
        st["logits"] = _route_logits(T, E, "uniform", seed, 6)
        st["bias"] = torch.randn(E, generator=_gen(seed, 7), device=DEV) * 0.5 if case["bias"] \
            else None
        st["shared"] = torch.randn(T, H, generator=_gen(seed, 8), device=DEV).to(torch.bfloat16) \
            if case["shared"] else None
        st["w13_q"], st["w13_s"] = _weights(E, 2 * I, H, seed, 9)
        st["w2_q"], st["w2_s"] = _weights(E, H, I, seed, 10)
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """What a user's program keeps next to its inputs: the plan, weights in the kernels' order,
    output buffers."""
    import bit_quantized_moe_top_amd as mq
    case = st["case"]
    if case["op"] == "quant":
        M, K = case["M"], case["K"]
        st["q"] = torch.empty(M, K // 2, dtype=torch.uint8, device=DEV)
        st["s"] = torch.empty(M, K // BLOCK, dtype=torch.uint8, device=DEV)
        st["v"] = torch.empty(M, K, dtype=_dtype(case["dtype"]), device=DEV)
    elif case["op"] == "gemm":
        st["plan"], _, _ = mq.moe_permute(st["ids"], case["E"])
        st["w"], st["ws"] = mq.tile_mxfp4_weights(st.pop("w_q"), st.pop("w_s"))
        cols = case["N"] // 2 if case["epilogue"] == "silu" else case["N"]
        st["out"] = torch.empty(case["T"] * case["k"], cols, dtype=_dtype(case["out"]), device=DEV)
    else:
        st["w13"], st["ws13"] = mq.tile_mxfp4_weights(st.pop("w13_q"), st.pop("w13_s"))
        st["w2"], st["ws2"] = mq.tile_mxfp4_weights(st.pop("w2_q"), st.pop("w2_s"))
        st["out"] = {}


# -------------------------------------------------------------------- pass
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import bit_quantized_moe_top_amd as mq
    case = st["case"]
    if case["op"] == "quant":
        q, s = mq.quant_mxfp4(st["x"], q=st["q"], scale=st["s"])
        v = mq.dequant_mxfp4(q, s, out=st["v"])
        return {"values": v, "scale": s.view(torch.float8_e8m0fnu)}
    if case["op"] == "gemm":
        silu = case["epilogue"] == "silu"
        return mq.moe_grouped_gemm_mxfp4(
            st["a_q"], st["a_s"], st["plan"], st["w"], st["ws"],
            epilogue=mq.EPI_SILU_MUL if silu else mq.EPI_NONE, topk=case["k"] if silu else 0,
            out=st["out"])
    st["out"] = mq.moe_layer_mxfp4_few(
        st["logits"], st["x"], st["w13"], st["ws13"], st["w2"], st["ws2"], case["k"],
        bias=st["bias"], renormalize=case["renormalize"], shared=st["shared"], out=st["out"])
    return {"ids": st["out"]["ids"], "w": st["out"]["w"], "y": st["out"]["y"]}


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _run_plain(st):
    case = st["case"]
    if case["op"] == "quant":
        q, s = _plain_quant(st["x"])
        return {"values": _plain_values(q, s).to(st["x"].dtype),
                "scale": s.view(torch.float8_e8m0fnu)}
    if case["op"] == "gemm":
        return _gemm(st, torch.float32, _plain_values).to(_dtype(case["out"]))
    k, T = case["k"], case["T"]
    score = st["logits"] if st["bias"] is None else st["logits"] + st["bias"]
    ids = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :k]
    top = torch.gather(score, 1, ids)
    p = torch.exp(top - top[:, :1])
    den = p if case["renormalize"] else torch.exp(score - top[:, :1])
    w = p / den.sum(1, keepdim=True)
    y = torch.empty(T, case["H"], device=DEV)
    for t in range(T):
        e = ids[t]
        gu = torch.matmul(_plain_values(st["w13_q"][e], st["w13_s"][e]), st["x"][t].float())
        h = _silu(gu[:, :case["I"]]) * gu[:, case["I"]:]
        o = torch.matmul(_plain_values(st["w2_q"][e], st["w2_s"][e]), h.unsqueeze(-1)).squeeze(-1)
        y[t] = (w[t].unsqueeze(-1) * o).sum(0)
    if st["shared"] is not None:
        y = y + st["shared"].float()
    return {"ids": ids.to(torch.int32), "w": w, "y": y.to(torch.bfloat16)}


def _gemm(st, dtype, values):
    """The grouped product in plan order, expert by expert."""
    case = st["case"]
    silu, k = case["epilogue"] == "silu", case["k"]
    half = case["N"] // 2
    out = torch.empty(case["T"] * k, half if silu else case["N"], dtype=dtype, device=DEV)
    a = values(st["a_q"], st["a_s"], dtype)
    p0 = 0
    for e, n in enumerate(st["counts"]):
        if n == 0:
            continue
        rows = a[st["order"][p0:p0 + n] // k] if silu else a[p0:p0 + n]
        v = rows @ values(st["w_q"][e], st["w_s"][e], dtype).T
        out[p0:p0 + n] = _silu(v[:, :half]) * v[:, half:] if silu else v
        p0 += n
    return out


# ---------------------------------------------------------- the exact values
def _exact_quant(x):
    """From the definition, in 64 bits: (values, scales) of x [M, K]."""
    b = x.double().reshape(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    mant, ex = torch.frexp(amax)                        # amax = mant * 2^ex, mant in [1/2, 1)
    e = torch.where(amax > 0, ex.double() - 3.0, torch.full_like(amax, -127.0)).clamp(-127, 127)
    scale = torch.pow(torch.full_like(amax, 2.0), e)
    y = (b / scale).abs().contiguous()
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    below = torch.bucketize(y, mid)                     # a tie goes to the lower code
    above = torch.bucketize(y, mid, right=True)         # ... to the upper one
    code = torch.where(below % 2 == 0, below, above)    # ties: the even code
    v = torch.copysign(grid[code], b) * scale
    return v.reshape(x.shape), scale.squeeze(-1)


def _exact_values(q, s, dtype=torch.float64):
    c = torch.stack((q % 16, q // 16), dim=-1).reshape(*s.shape, BLOCK).long()
    mag = torch.tensor(E2M1, dtype=torch.float64, device=q.device)[c % 8]
    v = torch.where(c >= 8, -mag, mag) * torch.pow(2.0, s.double() - 127.0)[..., None]
    return v.reshape(*s.shape[:-1], -1)


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "quant":
        v, s = _exact_quant(st["x"])
        return {"values": v, "scale": s}
    if case["op"] == "gemm":
        k, silu, half = case["k"], case["epilogue"] == "silu", case["N"] // 2
        a = _exact_values(st["a_q"], st["a_s"])
        parts, p0 = [], 0
        for e, n in enumerate(st["counts"]):
            if n:
                pos = torch.arange(p0, p0 + n, device=DEV)
                rows = a.index_select(0, st["order"][pos] // k if silu else pos)
                v = torch.mm(rows, _exact_values(st["w_q"][e], st["w_s"][e]).t().contiguous())
                parts.append(torch.sigmoid(v[:, :half]) * v[:, :half] * v[:, half:] if silu else v)
            p0 += n
        return torch.cat(parts)
    # scores are one fp32 addition by definition; everything after it in 64 bits
    score = (st["logits"] if st["bias"] is None else st["logits"] + st["bias"]).double()
    x, k, I = st["x"].double(), case["k"], case["I"]
    ids, ws, ys = [], [], []
    for t in range(case["T"]):
        row = score[t].tolist()
        best = sorted(range(len(row)), key=lambda i: (-row[i], i))[:k]
        p = torch.softmax(score[t], 0)[best]
        p = p / p.sum() if case["renormalize"] else p
        y = torch.zeros(case["H"], dtype=torch.float64, device=DEV)
        for j, e in enumerate(best):
            gu = torch.mv(_exact_values(st["w13_q"][e], st["w13_s"][e]), x[t])
            h = torch.sigmoid(gu[:I]) * gu[:I] * gu[I:]
            y += p[j] * torch.mv(_exact_values(st["w2_q"][e], st["w2_s"][e]), h)
        if st["shared"] is not None:
            y += st["shared"][t].double()
        ids.append(best)
        ws.append(p)
        ys.append(y)
    return {"ids": torch.tensor(ids, dtype=torch.int32, device=DEV), "w": torch.stack(ws),
            "y": torch.stack(ys)}


# -------------------------------------------------------------------- work
def _distinct(E, rows):
    """Experts that `rows` uniform choices reach, on average."""
    return min(E, rows) if E == 1 else E * (1.0 - (1.0 - 1.0 / E) ** rows)


def work(case):
    per = 0.5 + 1.0 / BLOCK                              # bytes per MXFP4 element
    if case["op"] == "quant":
        n = case["M"] * case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        # x in, codes and scales out; codes and scales in, values out
        return {"bytes": n * (2 * size + 2 * per), "flops": 2 * n}
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    if case["op"] == "gemm":
        N, K = case["N"], case["K"]
        silu = case["epilogue"] == "silu"
        out = R * (N // 2 if silu else N) * (4 if case["out"] == "f32" else 2)
        return {"bytes": _distinct(E, R) * N * K * per + (T if silu else R) * K * per + out,
                "flops": 2 * R * N * K}
    H, I = case["H"], case["I"]
    # a token's k experts differ: _distinct over R choices is a slight underestimate
    return {"bytes": _distinct(E, R) * 3 * H * I * per + T * (E * 4 + H * 2 * (3 if case["shared"]
                                                                               else 2)),
            "flops": 2 * R * 3 * H * I}
