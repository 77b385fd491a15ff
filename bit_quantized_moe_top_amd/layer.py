"""One quantized MoE expert layer as a fixed sequence of libmoeq calls.

    [router logits, when the layer holds the router weights]
      -> route + quantize x + permute (one call; one launch for T <= 16)
      -> expert MLP: gate/up GEMM (+SiLU) -> quantize h -> down GEMM (one call;
         two launches for decode-sized batches)
      -> combine (+ shared experts)

Only orchestration lives here: buffers are torch allocations, reused across
calls with the same token count, and every step is a C-ABI call into libmoeq.
"""
from __future__ import annotations

import functools
from typing import Optional

import torch

from . import (EPI_NONE, EPI_SILU_MUL, SCORE_SIGMOID, moe_combine, moe_expert_mlp_fp8row, moe_expert_mlp_w4a8,
               moe_grouped_gemm_aqlm, moe_grouped_gemm_fp8row, moe_grouped_gemm_nvfp4,
               moe_grouped_gemm_mxfp4, moe_grouped_gemm_w4a8, moe_layer_mxfp4_few, moe_permute,
               moe_plan_size,
               moe_requant_fp8_fnuz, moe_route_experts, moe_route_quant_permute, moe_route_topk,
               moe_router_logits, moe_shared_gemm_bf16, moe_shared_gemm_lora_bf16,
               moe_shared_gemm_lora_ws_size, pack_int4_g128,
               quant_fp8_per_token, quant_mxfp4, tile_mxfp4_weights)
from .route import _check_options


def _on_x_device(forward):
    """Runs forward(self, x, ...) with x's device current: kernels are launched on the current
    stream of the tensors' device, which has to be the current device for that."""
    @functools.wraps(forward)
    def call(self, x, *args, **kw):
        i = x.get_device()
        if i < 0 or i == torch.cuda.current_device():
            return forward(self, x, *args, **kw)
        with torch.cuda.device(i):
            return forward(self, x, *args, **kw)
    return call


class MoELayer:
    """Routed experts (W4A8 INT4-g128 or row-scaled FP8) plus optional bf16 shared experts.

    weight_format: "w4a8" (INT4 g128, fp32 group scales), "w4a8_bf16s" (INT4
    g128, bfloat16 group scales) or "fp8row" (E4M3, one fp32 scale per row).
    Weights: w13 [E, 2I, H] (gate rows then up rows), w2 [E, H, I].
    """

    def __init__(self, H: int, I: int, E: int, k: int, weight_format: str = "w4a8",
                 renormalize: bool = True, device="cuda"):
        if weight_format not in ("w4a8", "w4a8_bf16s", "fp8row"):
            raise ValueError(weight_format)
        self.H, self.I, self.E, self.k = H, I, E, k
        self.weight_format = weight_format
        self.renormalize = renormalize
        self.device = torch.device(device)
        self.w13 = self.s13 = self.w2 = self.s2 = None
        self.ws13 = self.ws2 = None
        self.w_router = None
        self.routing = None
        self.adapters = None
        self._bufs = {}
        self._adapter_ws = {}

    # --------------------------------------------------------------- weights
    def set_weights(self, w13, s13, w2, s2):
        """Already-quantized weights: INT4 in the GEMMs' tiled order (tile_int4_weights)
        with group scales, or E4M3 with row scales."""
        self.w13, self.s13, self.w2, self.s2 = w13, s13, w2, s2

    def quantize_weights(self, w13_f32: torch.Tensor, w2_f32: torch.Tensor):
        """Quantize fp32 weights on the device with the library's own kernels."""
        if self.weight_format in ("w4a8", "w4a8_bf16s"):
            sdt = torch.bfloat16 if self.weight_format == "w4a8_bf16s" else torch.float32
            self.w13, self.s13 = pack_int4_g128(w13_f32, scale_dtype=sdt, tiled=True)
            self.w2, self.s2 = pack_int4_g128(w2_f32, scale_dtype=sdt, tiled=True)
        else:
            self.w13, self.s13 = quant_fp8_per_token(w13_f32)
            self.w2, self.s2 = quant_fp8_per_token(w2_f32)

    def set_weights_fnuz(self, w13_fnuz, s13_fnuz, w2_fnuz, s2_fnuz):
        """Row-scaled E4M3FNUZ expert weights (the MI300X checkpoint layout: scales
        [E, out_channels], max|row| / 240), converted on the device to the
        row-scaled OCP E4M3 weights this layer runs on."""
        if self.weight_format != "fp8row":
            raise ValueError("E4M3FNUZ weights are row-scaled FP8 experts (weight_format='fp8row')")
        self.w13, self.s13 = moe_requant_fp8_fnuz(w13_fnuz, s13_fnuz)
        self.w2, self.s2 = moe_requant_fp8_fnuz(w2_fnuz, s2_fnuz)

    def set_router(self, w_router: Optional[torch.Tensor]):
        """fp32 router weights [E, H]; forward() then takes logits=None and computes
        them with moe_router_logits."""
        self.w_router = w_router

    def set_routing(self, scoring: Optional[int] = SCORE_SIGMOID, n_group: int = 1,
                    topk_group: int = 1, group_best: int = 1, scale: float = 1.0):
        """Routing by moe_route_experts: scores, groups, weights times scale, and forward()'s bias
        moves the choice of experts only.  scoring=None: back to moe_route_topk, where the bias is
        part of the softmax."""
        if scoring is None:
            self.routing = None
            return
        _check_options(self.E, self.k, scoring, n_group, topk_group, group_best, scale)
        self.routing = dict(scoring=scoring, n_group=n_group, topk_group=topk_group,
                            group_best=group_best, scale=scale)

    def set_shared(self, ws13: Optional[torch.Tensor], ws2: Optional[torch.Tensor]):
        self.ws13, self.ws2 = ws13, ws2

    def set_shared_adapters(self, a13: Optional[torch.Tensor], b13: Optional[torch.Tensor] = None,
                            a2: Optional[torch.Tensor] = None, b2: Optional[torch.Tensor] = None,
                            scale: Optional[torch.Tensor] = None):
        """Low-rank adapters of the shared experts, used where forward() is given an adapter_plan
        (moe_adapter_plan of the batch): a13 [L, 1 or 2, r, H], b13 [L, 2S, r] beside gate/up, a2
        [L, 1, r, S], b2 [L, H, r] beside down, scale [L] fp32.  a13=None: no adapters."""
        self.adapters = None if a13 is None else (a13, b13, a2, b2, scale)

    # ---------------------------------------------------------------- buffers
    def buffers(self, T: int) -> dict:
        # the shared experts' width is part of the key: set_shared may come after a call, and the
        # earlier buffers stay, since a captured graph may hold them
        S = 0 if self.ws13 is None else self.ws2.shape[1]
        b = self._bufs.get((T, S))
        if b is None:
            H, I, E, k, d = self.H, self.I, self.E, self.k, self.device
            R = T * k
            b = {
                "logits": torch.empty(T, E, dtype=torch.float32, device=d),
                "ids": torch.empty(T, k, dtype=torch.int32, device=d),
                "w": torch.empty(T, k, dtype=torch.float32, device=d),
                "x_q": torch.empty(T, H, dtype=torch.uint8, device=d),
                "x_s": torch.empty(T, dtype=torch.float32, device=d),
                "plan": torch.empty((moe_plan_size(E, R) + 3) // 4, dtype=torch.int32, device=d),
                "xp_q": torch.empty(R, H, dtype=torch.uint8, device=d),
                "xp_s": torch.empty(R, dtype=torch.float32, device=d),
                "h": torch.empty(R, I, dtype=torch.bfloat16, device=d),
                "h_q": torch.empty(R, I, dtype=torch.uint8, device=d),
                "h_s": torch.empty(R, dtype=torch.float32, device=d),
                "o": torch.empty(R, H, dtype=torch.bfloat16, device=d),
                "y": torch.empty(T, H, dtype=torch.bfloat16, device=d),
            }
            if self.ws13 is not None:
                b["sh_h"] = torch.empty(T, S, dtype=torch.bfloat16, device=d)
                b["shared"] = torch.empty(T, H, dtype=torch.bfloat16, device=d)
            self._bufs[T, S] = b
        return b

    def _lora_ws(self, T: int) -> torch.Tensor:
        """The workspace of the shared experts' two products with adapters, one per batch size and
        set of shapes, whatever the number of adapters, which its size does not depend on (earlier
        ones stay, since a captured graph may hold them)."""
        a13, _, a2, _, _ = self.adapters
        key = (T, self.ws13.shape, self.ws2.shape, a13.shape[1:], a2.shape[1:])
        ws = self._adapter_ws.get(key)
        if ws is None:
            n = max(moe_shared_gemm_lora_ws_size(T, *w.shape, *a.shape[:3])
                    for w, a in ((self.ws13, a13), (self.ws2, a2)))
            ws = self._adapter_ws[key] = torch.empty(n, dtype=torch.uint8, device=self.device)
        return ws

    def _shared(self, x, b, step, adapter_plan):
        """The shared experts' output, with the batch's adapters if there is a plan, or None."""
        if adapter_plan is not None and (self.adapters is None or self.ws13 is None):
            raise ValueError("adapter_plan needs shared experts (set_shared) with adapters "
                             "(set_shared_adapters)")
        if self.ws13 is None:
            return None
        # the shared experts are bf16 MLPs of the bf16 model: their input is x itself
        if x.dtype != torch.bfloat16:
            raise TypeError("shared experts take bfloat16 x")
        if adapter_plan is None:
            step("shared_gate_up", moe_shared_gemm_bf16, x, self.ws13, EPI_SILU_MUL, out=b["sh_h"])
            return step("shared_down", moe_shared_gemm_bf16, b["sh_h"], self.ws2, EPI_NONE,
                        out=b["shared"])
        a13, b13, a2, b2, scale = self.adapters
        ws = self._lora_ws(x.shape[0])
        step("shared_gate_up", moe_shared_gemm_lora_bf16, x, self.ws13, a13, b13, scale,
             adapter_plan, EPI_SILU_MUL, out=b["sh_h"], ws=ws)
        return step("shared_down", moe_shared_gemm_lora_bf16, b["sh_h"], self.ws2, a2, b2, scale,
                    adapter_plan, EPI_NONE, out=b["shared"], ws=ws)

    def _route(self, logits, bias, b, step):
        """ids and weights of set_routing, or of the plain softmax routing"""
        if self.routing is None:
            step("route", moe_route_topk, logits, self.k, bias, self.renormalize, ids=b["ids"],
                 weights=b["w"])
        else:
            step("route", moe_route_experts, logits, self.k, bias=bias,
                 renormalize=self.renormalize, ids=b["ids"], weights=b["w"], **self.routing)

    def _route_quant_permute(self, logits, x, bias, b, step):
        if self.routing is None:
            step("route_quant_permute", moe_route_quant_permute, logits, x, self.k, bias,
                 self.renormalize, out=b)
            return
        self._route(logits, bias, b, step)
        step("quant_x", quant_fp8_per_token, x, q=b["x_q"], scale=b["x_s"])
        step("permute", moe_permute, b["ids"], self.E, b["x_q"], b["x_s"], plan=b["plan"],
             xp_q=b["xp_q"], xp_s=b["xp_s"])

    # ---------------------------------------------------------------- forward
    @_on_x_device
    def forward(self, x: torch.Tensor, logits: Optional[torch.Tensor] = None,
                bias: Optional[torch.Tensor] = None,
                return_all: bool = False, events: Optional[list] = None,
                split_mlp: bool = False, adapter_plan: Optional[torch.Tensor] = None):
        """y = layer(x).  logits=None: the router's logits are computed from x and the
        weights given to set_router.  With `events` (a list), each call is bracketed by a pair of
        timing events on the current stream, appended as (name, start, end).
        split_mlp runs the expert MLP as its three separate calls (same results).
        adapter_plan: the batch's moe_adapter_plan, for the shared experts' adapters."""
        T = x.shape[0]
        b = self.buffers(T)
        w4 = self.weight_format != "fp8row"      # INT4 (scale dtype picks the entry point)
        gemm = moe_grouped_gemm_w4a8 if w4 else moe_grouped_gemm_fp8row
        mlp = moe_expert_mlp_w4a8 if w4 else moe_expert_mlp_fp8row

        def step(name, fn, *args, **kw):
            if events is None:
                return fn(*args, **kw)
            s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            s.record()
            r = fn(*args, **kw)
            e.record()
            events.append((name, s, e))
            return r

        if logits is None:
            if self.w_router is None:
                raise ValueError("logits=None needs router weights (set_router)")
            logits = step("router", moe_router_logits, x, self.w_router, out=b["logits"])
        self._route_quant_permute(logits, x, bias, b, step)
        if split_mlp:
            step("gemm_gate_up", gemm, b["xp_q"], b["xp_s"], b["plan"], self.w13, self.s13,
                 epilogue=EPI_SILU_MUL, out=b["h"])
            step("quant_h", quant_fp8_per_token, b["h"], q=b["h_q"], scale=b["h_s"])
            step("gemm_down", gemm, b["h_q"], b["h_s"], b["plan"], self.w2, self.s2,
                 epilogue=EPI_NONE, out=b["o"])
        else:
            step("expert_mlp", mlp, b["xp_q"], b["xp_s"], b["plan"], self.w13, self.s13, self.w2,
                 self.s2, out=b)
        shared = self._shared(x, b, step, adapter_plan)
        step("combine", moe_combine, b["o"], b["plan"], b["w"], shared, y=b["y"], E=self.E)
        return b if return_all else b["y"]

    __call__ = forward


class HybridMoELayer(MoELayer):
    """The NVFP4 + AQLM hybrid expert layer: each routed expert is either hot
    (an NVFP4 slab) or cold (an AQLM slab).  hot_ids / cold_ids list the routed
    expert of each slab and together partition 0 .. E-1.

    Hot slabs:  w13 [n_hot, 2I, H/2] E2M1 pairs, w13_bs [n_hot, 2I, H/16] E4M3,
                w13_s2 [n_hot] fp32; w2 [n_hot, H, I/2], w2_bs [n_hot, H, I/16], w2_s2.
    Cold slabs: per projection a list of code tensors ([n_cold, out, in/8], one
                per book), the list of fp16 codebooks [entries, 8], and the fp16
                row scales [n_cold, out].
    Each GEMM step runs both formats' kernels; each fills only its experts' rows.  Shared experts
    and their adapters as in MoELayer.
    """

    def __init__(self, H: int, I: int, E: int, k: int, renormalize: bool = True, device="cuda"):
        super().__init__(H, I, E, k, "w4a8", renormalize, device)
        self.weight_format = "hybrid"
        self.hot = self.cold = None

    def set_hybrid_weights(self, hot_ids, cold_ids, hot: dict, cold: dict):
        """hot: w13, w13_bs, w13_s2, w2, w2_bs, w2_s2; cold: w13_codes (list), w13_books
        (list), w13_scale, w2_codes, w2_books, w2_scale."""
        d = self.device
        hot_ids = torch.as_tensor(hot_ids, dtype=torch.int64)
        cold_ids = torch.as_tensor(cold_ids, dtype=torch.int64)
        if torch.cat([hot_ids, cold_ids]).sort().values.tolist() != list(range(self.E)):
            raise ValueError("hot_ids and cold_ids must partition the experts")
        hot_of = torch.full((self.E,), -1, dtype=torch.int32)
        cold_of = torch.full((self.E,), -1, dtype=torch.int32)
        hot_of[hot_ids] = torch.arange(len(hot_ids), dtype=torch.int32)
        cold_of[cold_ids] = torch.arange(len(cold_ids), dtype=torch.int32)
        self.hot_of, self.cold_of = hot_of.to(d), cold_of.to(d)
        self.hot, self.cold = hot, cold

    def _gemm_both(self, a_q, a_s, plan, proj: str, epilogue, out):
        h, c = self.hot, self.cold
        if h is not None and h[proj].shape[0] > 0:
            moe_grouped_gemm_nvfp4(a_q, a_s, plan, h[proj], h[proj + "_bs"], h[proj + "_s2"],
                                   epilogue=epilogue, out=out, slab_of=self.hot_of)
        if c is not None and c[proj + "_scale"].shape[0] > 0:
            moe_grouped_gemm_aqlm(a_q, a_s, plan, c[proj + "_codes"], c[proj + "_books"],
                                  c[proj + "_scale"], epilogue=epilogue, out=out,
                                  slab_of=self.cold_of)
        return out

    @_on_x_device
    def forward(self, x: torch.Tensor, logits: Optional[torch.Tensor] = None,
                bias: Optional[torch.Tensor] = None, return_all: bool = False,
                events: Optional[list] = None, split_mlp: bool = True,
                adapter_plan: Optional[torch.Tensor] = None):
        T = x.shape[0]
        b = self.buffers(T)

        def step(name, fn, *args, **kw):
            if events is None:
                return fn(*args, **kw)
            s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            s.record()
            r = fn(*args, **kw)
            e.record()
            events.append((name, s, e))
            return r

        if logits is None:
            if self.w_router is None:
                raise ValueError("logits=None needs router weights (set_router)")
            logits = step("router", moe_router_logits, x, self.w_router, out=b["logits"])
        self._route_quant_permute(logits, x, bias, b, step)
        step("gemm_gate_up", self._gemm_both, b["xp_q"], b["xp_s"], b["plan"], "w13",
             EPI_SILU_MUL, b["h"])
        step("quant_h", quant_fp8_per_token, b["h"], q=b["h_q"], scale=b["h_s"])
        step("gemm_down", self._gemm_both, b["h_q"], b["h_s"], b["plan"], "w2", EPI_NONE, b["o"])
        shared = self._shared(x, b, step, adapter_plan)
        step("combine", moe_combine, b["o"], b["plan"], b["w"], shared, y=b["y"], E=self.E)
        return b if return_all else b["y"]

    __call__ = forward


class MxMoELayer(MoELayer):
    """Routed experts with MXFP4 weights (E2M1 codes, an E8M0 scale per 32 K).

    forward(): any number of tokens, activations in MXFP4 too (route, quantize x, plan, gate/up
    product with SiLU, quantize h, down product, combine); the gate/up product reads each token's
    one quantized row, so no gathered copy is made.
    forward_few(): up to 16 tokens in two kernels, activations in bf16.  Its results are closer to
    the unquantized layer's than forward()'s, which rounds x and h to 4 bits.
    In both, scores of -inf mask experts: weight 0 and nothing added, whatever the expert's weights
    hold; a token with every expert masked gets the shared experts' output, or 0.
    """

    def __init__(self, H: int, I: int, E: int, k: int, renormalize: bool = True, device="cuda"):
        super().__init__(H, I, E, k, "w4a8", renormalize, device)
        self.weight_format = "mxfp4"
        self._few = {}

    # set_weights takes tiled weights and scales (tile_mxfp4_weights)

    def set_weights_fnuz(self, *args):
        raise ValueError("E4M3FNUZ weights are row-scaled FP8 experts (weight_format='fp8row')")

    def quantize_weights(self, w13: torch.Tensor, w2: torch.Tensor):
        """fp32 or bf16 weights [E, 2I, H] and [E, H, I], quantized and tiled on the device."""
        self.w13, self.s13 = tile_mxfp4_weights(*quant_mxfp4(w13))
        self.w2, self.s2 = tile_mxfp4_weights(*quant_mxfp4(w2))

    def buffers(self, T: int) -> dict:
        # the shared experts' width is part of the key: set_shared may come after a call, and the
        # earlier buffers stay, since a captured graph may hold them
        S = 0 if self.ws13 is None else self.ws2.shape[1]
        b = self._bufs.get((T, S))
        if b is None:
            H, I, E, k, d = self.H, self.I, self.E, self.k, self.device
            R = T * k

            def u8(*shape):
                return torch.empty(*shape, dtype=torch.uint8, device=d)

            def bf16(*shape):
                return torch.empty(*shape, dtype=torch.bfloat16, device=d)

            b = {
                "logits": torch.empty(T, E, dtype=torch.float32, device=d),
                "ids": torch.empty(T, k, dtype=torch.int32, device=d),
                "w": torch.empty(T, k, dtype=torch.float32, device=d),
                "plan": torch.empty((moe_plan_size(E, R) + 3) // 4, dtype=torch.int32, device=d),
                "x_q": u8(T, H // 2), "x_s": u8(T, H // 32), "h": bf16(R, I),
                "h_q": u8(R, I // 2), "h_s": u8(R, I // 32), "o": bf16(R, H), "y": bf16(T, H),
            }
            if self.ws13 is not None:
                b["sh_h"], b["shared"] = bf16(T, S), bf16(T, H)
            self._bufs[T, S] = b
        return b

    def _front(self, x, logits, b, step, adapter_plan=None):
        """(logits, the shared experts' output or None)"""
        if logits is None:
            if self.w_router is None:
                raise ValueError("logits=None needs router weights (set_router)")
            logits = step("router", moe_router_logits, x, self.w_router, out=b["logits"])
        return logits, self._shared(x, b, step, adapter_plan)

    @staticmethod
    def _steps(events):
        def step(name, fn, *args, **kw):
            if events is None:
                return fn(*args, **kw)
            s, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            s.record()
            r = fn(*args, **kw)
            e.record()
            events.append((name, s, e))
            return r
        return step

    @_on_x_device
    def forward(self, x: torch.Tensor, logits: Optional[torch.Tensor] = None,
                bias: Optional[torch.Tensor] = None, return_all: bool = False,
                events: Optional[list] = None, adapter_plan: Optional[torch.Tensor] = None):
        b, step = self.buffers(x.shape[0]), self._steps(events)
        logits, shared = self._front(x, logits, b, step, adapter_plan)
        self._route(logits, bias, b, step)
        step("quant_x", quant_mxfp4, x, q=b["x_q"], scale=b["x_s"])
        step("plan", moe_permute, b["ids"], self.E, plan=b["plan"])
        step("gemm_gate_up", moe_grouped_gemm_mxfp4, b["x_q"], b["x_s"], b["plan"], self.w13,
             self.s13, epilogue=EPI_SILU_MUL, topk=self.k, out=b["h"])
        step("quant_h", quant_mxfp4, b["h"], q=b["h_q"], scale=b["h_s"])
        step("gemm_down", moe_grouped_gemm_mxfp4, b["h_q"], b["h_s"], b["plan"], self.w2, self.s2,
             out=b["o"])
        step("combine", moe_combine, b["o"], b["plan"], b["w"], shared, y=b["y"], E=self.E)
        return b if return_all else b["y"]

    @_on_x_device
    def forward_few(self, x: torch.Tensor, logits: Optional[torch.Tensor] = None,
                    bias: Optional[torch.Tensor] = None, return_all: bool = False,
                    events: Optional[list] = None, adapter_plan: Optional[torch.Tensor] = None):
        """forward() for at most 16 tokens of bf16 x in two kernels, activations in bf16."""
        if self.routing is not None:
            raise ValueError("forward_few finds the experts itself, by the plain softmax routing: a "
                             "layer with set_routing takes forward()")
        T = x.shape[0]
        step = self._steps(events)
        needs = logits is None or self.ws13 is not None
        logits, shared = self._front(x, logits, self.buffers(T) if needs else None, step,
                                     adapter_plan)
        # (buffers of its own: the workspace belongs to this layer's calls)
        self._few[T] = o = step("few", moe_layer_mxfp4_few, logits, x, self.w13, self.s13, self.w2,
                                self.s2, self.k, bias=bias, renormalize=self.renormalize,
                                shared=shared, out=self._few.get(T))
        return o if return_all else o["y"]

    __call__ = forward
