"""The layers with set_routing and set_shared_adapters: the calls composed, against the separate
calls (the same bits) and against float64."""
import numpy as np
import pytest
import torch

import bit_quantized_moe_top_amd as mq
import workloads as W
from oracle import lora as O
from oracle import route as R
from parity import rel_l2, to_np

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
H, I, E, K_TOP, S, L, RANK = 256, 128, 24, 4, 192, 5, 16
ROUTING = dict(scoring=mq.SCORE_SIGMOID, n_group=6, topk_group=3, group_best=2, scale=2.5)


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Set:
    """A layer with shared experts and their adapters, and a batch."""
    def __init__(self, T, kind="mxfp4", seed=0):
        g = gen(seed + T)
        if kind == "mxfp4":
            self.layer = mq.MxMoELayer(H, I, E, K_TOP, device=DEV)
        else:
            self.layer = mq.MoELayer(H, I, E, K_TOP, kind, device=DEV)
        self.layer.quantize_weights((torch.randn(E, 2 * I, H, generator=g) * .1).to(DEV),
                                    (torch.randn(E, H, I, generator=g) * .1).to(DEV))
        rnd = lambda *s, f=.1: (torch.randn(*s, generator=g) * f).to(BF)  # noqa: E731
        self.shared = [rnd(2 * S, H), rnd(H, S)]
        self.adapters = [rnd(L, 2, RANK, H), rnd(L, 2 * S, RANK, f=.2), rnd(L, 1, RANK, S),
                         rnd(L, H, RANK, f=.2), torch.rand(L, generator=g) + 0.5]
        self.x, self.logits = rnd(T, H, f=1.0), torch.randn(T, E, generator=g)
        self.bias = torch.randn(E, generator=g) * 0.1
        self.ids = torch.randint(-1, L, (T,), generator=g).to(torch.int32)
        self.layer.set_shared(*[t.to(DEV) for t in self.shared])
        self.layer.set_routing(**ROUTING)
        self.layer.set_shared_adapters(*[t.to(DEV) for t in self.adapters])

    def batch(self):
        return [t.to(DEV) for t in (self.x, self.logits, self.bias)]

    def plan(self):
        return mq.moe_adapter_plan(self.ids.to(DEV), L)


@pytest.mark.parametrize("kind", ["w4a8", "fp8row", "mxfp4"])
@pytest.mark.parametrize("T", [1, 9, 70])
def test_layer_equals_its_calls_and_float64(kind, T):
    s = Set(T, kind)
    x, logits, bias = s.batch()
    plan = s.plan()
    events = []
    b = s.layer.forward(x, logits, bias, return_all=True, adapter_plan=plan, events=events)
    assert [e[0] for e in events if e[0] in ("route", "shared_gate_up", "shared_down", "combine")] == (
        ["shared_gate_up", "shared_down", "route", "combine"] if kind == "mxfp4" else
        ["route", "shared_gate_up", "shared_down", "combine"])
    ids, w = mq.moe_route_experts(logits, K_TOP, bias=bias, **ROUTING)
    assert torch.equal(b["ids"], ids) and torch.equal(b["w"], w)
    a13, b13, a2, b2, scale = [t.to(DEV) for t in s.adapters]
    h = mq.moe_shared_gemm_lora_bf16(x, s.layer.ws13, a13, b13, scale, plan, mq.EPI_SILU_MUL)
    sh = mq.moe_shared_gemm_lora_bf16(h, s.layer.ws2, a2, b2, scale, plan)
    assert torch.equal(b["sh_h"], h) and torch.equal(b["shared"], sh)
    assert torch.equal(b["y"], mq.moe_combine(b["o"], b["plan"], w, sh, E=E))
    if kind != "mxfp4":
        xq, xs = mq.quant_fp8_per_token(x)
        p, xp_q, xp_s = mq.moe_permute(ids, E, xq, xs)
        mlp = mq.moe_expert_mlp_w4a8 if kind == "w4a8" else mq.moe_expert_mlp_fp8row
        o = mlp(xp_q, xp_s, p, s.layer.w13, s.layer.s13, s.layer.w2, s.layer.s2)["o"]
        assert torch.equal(b["o"], o)
    # float64: routing and the shared experts; the routed experts' rows as the layer computed them
    rid, rw = R.route_experts(s.logits.numpy(), K_TOP, bias=s.bias.numpy(), **ROUTING)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    f = [to_np(t) for t in s.adapters]
    v, _ = O.project(to_np(s.x), to_np(s.shared[0]), f[0], f[1], f[4], s.ids.numpy())
    v, _ = O.project(O.silu_mul(v), to_np(s.shared[1]), f[2], f[3], f[4], s.ids.numpy())
    pos = mq.plan_fields(b["plan"], E, T * K_TOP)["row_pos"].cpu().numpy().reshape(T, K_TOP)
    ref = v + np.einsum("tk,tkh->th", rw, to_np(b["o"]).astype(np.float64)[pos])
    # bf16 roundings of h, of the shared experts' output and of y, 1.65e-3 rms each: 2.9e-3
    assert rel_l2(to_np(b["y"]), ref) <= 4e-3


def test_hybrid_layer_with_routing():
    cfg = W.get_config("hybrid_tiny")
    inp = W.make_layer_inputs(cfg, device="cpu")
    hot_ids, cold_ids = W.hybrid_partition(cfg)
    layer = mq.HybridMoELayer(cfg.H, cfg.I, cfg.E, cfg.k, device=DEV)
    to = lambda d: {k: [t.to(DEV) for t in v] if isinstance(v, list) else v.to(DEV)  # noqa: E731
                    for k, v in d.items()}
    layer.set_hybrid_weights(hot_ids, cold_ids, to(W.make_nvfp4_slabs(cfg, len(hot_ids), device="cpu")),
                             to(W.make_aqlm_slabs(cfg, len(cold_ids), device="cpu")))
    x, logits = inp["x"].to(DEV), inp["logits"].to(DEV)
    plain = layer.forward(x, logits).clone()
    layer.set_routing(mq.SCORE_SOFTMAX)                 # the same routing by the other call
    b = layer.forward(x, logits, return_all=True)
    assert torch.equal(b["ids"], mq.moe_route_topk(logits, cfg.k)[0])
    # weights within 32 ulp (2^-18) of the plain routing's: that much of the sum of magnitudes, and
    # two roundings
    mag = mq.moe_combine(b["o"].abs(), b["plan"], b["w"], E=cfg.E).double()
    err = (b["y"].double() - plain.double()).abs()
    assert (err <= 2.0 ** -7 * plain.double().abs() + 2.0 ** -17 * mag).all()
    layer.set_routing(mq.SCORE_SIGMOID, n_group=2, topk_group=1)
    b = layer.forward(x, logits, return_all=True)
    ids, w = mq.moe_route_experts(logits, cfg.k, mq.SCORE_SIGMOID, n_group=2, topk_group=1)
    assert torch.equal(b["ids"], ids) and torch.equal(b["w"], w)
    layer.set_routing(None)
    assert torch.equal(layer.forward(x, logits), plain)


def test_few_token_layer_with_adapters():
    s = Set(7)
    x, logits, bias = s.batch()
    plan = s.plan()
    with pytest.raises(ValueError, match="set_routing"):
        s.layer.forward_few(x, logits, bias, adapter_plan=plan)
    s.layer.set_routing(None)
    y = s.layer.forward_few(x, logits, bias, adapter_plan=plan).clone()
    shared = s.layer.forward(x, logits, bias, return_all=True, adapter_plan=plan)["shared"]
    direct = mq.moe_layer_mxfp4_few(logits, x, s.layer.w13, s.layer.s13, s.layer.w2, s.layer.s2,
                                    K_TOP, bias=bias, shared=shared)
    assert torch.equal(y, direct["y"])
    assert not torch.equal(y, s.layer.forward_few(x, logits, bias))


@pytest.mark.parametrize("kind", ["w4a8", "mxfp4"])
def test_without_a_plan_and_without_adapters_as_before(kind):
    s = Set(11, kind)
    x, logits, bias = s.batch()
    plan = s.plan()
    other = Set(11, kind)
    other.layer.set_routing(None)
    other.layer.set_shared_adapters(None)
    s.layer.set_routing(None)
    assert torch.equal(s.layer.forward(x, logits, bias), other.layer.forward(x, logits, bias))
    with pytest.raises(ValueError, match="set_shared_adapters"):
        other.layer.forward(x, logits, bias, adapter_plan=plan)
    bare = mq.MoELayer(H, I, E, K_TOP, "w4a8", device=DEV)
    bare.set_weights(s.layer.w13, s.layer.s13, s.layer.w2, s.layer.s2)
    bare.set_shared_adapters(*[t.to(DEV) for t in s.adapters])
    if kind == "w4a8":
        with pytest.raises(ValueError, match="set_shared"):
            bare.forward(x, logits, bias, adapter_plan=plan)
        with pytest.raises(TypeError, match="bfloat16 x"):
            s.layer.forward(x.float(), logits, bias, adapter_plan=plan)
    for bad in (dict(n_group=5), dict(topk_group=2), dict(n_group=24, topk_group=3), dict(group_best=0),
                dict(scoring=9), dict(scale=float("nan"))):
        with pytest.raises(ValueError):
            s.layer.set_routing(**bad)


def test_masked_tokens_keep_the_shared_part():
    s = Set(8, "w4a8")
    s.logits[2] = float("-inf")
    x, logits, bias = s.batch()
    b = s.layer.forward(x, logits, bias, return_all=True, adapter_plan=s.plan())
    assert (b["w"][2] == 0).all() and torch.equal(b["y"][2], b["shared"][2])


@pytest.mark.parametrize("kind", ["w4a8", "mxfp4"])
@pytest.mark.parametrize("T", [3, 70])
def test_captured_and_replayed(kind, T):
    """Plan, routing, shared experts with adapters and routed experts in one graph."""
    s = Set(T, kind)
    g = gen(T)
    x, logits, bias = s.batch()
    ids = s.ids.to(DEV)
    plan = s.plan()

    def step():
        mq.moe_adapter_plan(ids, L, plan=plan)
        return s.layer.forward(x, logits, bias, return_all=True, adapter_plan=plan)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = step()

    def new():
        x.copy_(torch.randn(T, H, generator=g).to(BF))
        logits.copy_(torch.randn(T, E, generator=g))
        ids.copy_(torch.randint(-1, L, (T,), generator=g).to(torch.int32))
    for rep in range(4):
        new()
        kept = [t.clone() for t in (x, logits, ids)]
        expect = {n: t.clone() for n, t in step().items()}
        new()
        step()                                          # other values in every buffer
        for t, v in zip((x, logits, ids), kept):
            t.copy_(v)
        b["y"].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n in ("ids", "w", "sh_h", "shared", "y"):
            assert torch.equal(b[n], expect[n]), (rep, n)


def test_batches_of_two_sizes_and_two_streams_have_their_own_workspaces():
    a, b = Set(5, "w4a8", seed=1), Set(5, "w4a8", seed=2)
    args = [(s, *s.batch(), s.plan()) for s in (a, b)]
    refs = [s.layer.forward(x, z, c, adapter_plan=p).clone() for s, x, z, c, p in args]
    assert a.layer._lora_ws(5).data_ptr() != b.layer._lora_ws(5).data_ptr()
    assert a.layer._lora_ws(5).data_ptr() != a.layer._lora_ws(6).data_ptr()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        for (s, x, z, c, p), st in zip(args, streams):
            with torch.cuda.stream(st):
                s.layer.forward(x, z, c, adapter_plan=p)
    torch.cuda.synchronize()
    for (s, *_), ref in zip(args, refs):
        assert torch.equal(s.layer.buffers(5)["y"], ref)


@pytest.mark.parametrize("routed", [False, True])
def test_hybrid_layer_with_shared_experts_and_adapters(routed):
    cfg = W.get_config("hybrid_tiny")
    inp = W.make_layer_inputs(cfg, device="cpu")
    hot_ids, cold_ids = W.hybrid_partition(cfg)
    layer = mq.HybridMoELayer(cfg.H, cfg.I, cfg.E, cfg.k, device=DEV)
    to = lambda d: {k: [t.to(DEV) for t in v] if isinstance(v, list) else v.to(DEV)  # noqa: E731
                    for k, v in d.items()}
    layer.set_hybrid_weights(hot_ids, cold_ids, to(W.make_nvfp4_slabs(cfg, len(hot_ids), device="cpu")),
                             to(W.make_aqlm_slabs(cfg, len(cold_ids), device="cpu")))
    if routed:
        layer.set_routing(mq.SCORE_SIGMOID, n_group=2, topk_group=1)
    x, logits = inp["x"].to(BF).to(DEV), inp["logits"].to(DEV)
    bare = {n: t.clone() for n, t in layer.forward(x, logits, return_all=True).items()}
    s = Set(cfg.T)                                      # shared experts, adapters and ids of H = 256
    assert cfg.H == H
    a13, b13, a2, b2, scale = [t.to(DEV) for t in s.adapters]
    layer.set_shared(*[t.to(DEV) for t in s.shared])
    layer.set_shared_adapters(a13, b13, a2, b2, scale)
    plan = s.plan()
    for p in (None, plan):
        b = layer.forward(x, logits, return_all=True, adapter_plan=p)
        if p is None:
            h = mq.moe_shared_gemm_bf16(x, layer.ws13, mq.EPI_SILU_MUL)
            sh = mq.moe_shared_gemm_bf16(h, layer.ws2)
        else:
            h = mq.moe_shared_gemm_lora_bf16(x, layer.ws13, a13, b13, scale, plan, mq.EPI_SILU_MUL)
            sh = mq.moe_shared_gemm_lora_bf16(h, layer.ws2, a2, b2, scale, plan)
        assert torch.equal(b["shared"], sh) and sh.abs().max() > 0
        for n in ("ids", "w", "o"):
            assert torch.equal(b[n], bare[n]), n
        assert torch.equal(b["y"], mq.moe_combine(b["o"], b["plan"], b["w"], sh, E=cfg.E))
        assert not torch.equal(b["y"], bare["y"])
    layer.set_shared(None, None)
    assert torch.equal(layer.forward(x, logits), bare["y"])


@pytest.mark.parametrize("kind", ["w4a8", "fp8row", "mxfp4"])
def test_shared_experts_set_after_a_call(kind):
    s = Set(9, kind)
    x, logits, bias = s.batch()
    expect = s.layer.forward(x, logits, bias, adapter_plan=s.plan()).clone()
    late = Set(9, kind)
    late.layer.set_shared(None, None)
    late.layer.set_shared_adapters(None)
    plain = late.layer.forward(x, logits, bias).clone()
    late.layer.set_shared(*[t.to(DEV) for t in late.shared])
    late.layer.set_shared_adapters(*[t.to(DEV) for t in late.adapters])
    assert torch.equal(late.layer.forward(x, logits, bias, adapter_plan=late.plan()), expect)
    late.layer.set_shared(None, None)
    assert torch.equal(late.layer.forward(x, logits, bias), plain)


@pytest.mark.parametrize("kind", ["w4a8", "fp8row", "mxfp4"])
def test_no_tokens(kind):
    s = Set(3, kind)
    x, logits, bias = s.batch()
    plan = mq.moe_adapter_plan(s.ids[:0].to(DEV), L)
    assert s.layer.forward(x[:0], logits[:0], bias, adapter_plan=plan).shape == (0, H)
