"""The layer-level call a user makes: prepacked weights resident on the GPU,
then gate_up -> silu_and_mul -> down per batch of routed tokens.

Every step is a call into the C-ABI library (``ops``); this module only
allocates buffers (torch device memory) and sequences the calls on one
stream.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from . import ops


@dataclass
class PackedExperts:
    """Prepacked expert weights of one projection: [num_experts, n, k]."""
    packed: torch.Tensor
    num_experts: int
    n: int
    k: int

    layout: int = ops.W4A16_LAYOUT_KTILE64

    @classmethod
    def from_checkpoint(cls, q: torch.Tensor, scales: torch.Tensor, group: int = 32,
                        layout: int = ops.W4A16_LAYOUT_KTILE64):
        """layout W4A16_LAYOUT_KTILE64_GLU16 (gate_up weights only) enables the
        fused gate_up + activation call."""
        e, n, kh = q.shape
        return cls(ops.w4a16_prepack(q, scales, group, layout), e, n, kh * 2, layout)


def single_launch_default(gate_up_layout: int, deterministic: bool, inter: int,
                          block_m: int = 32) -> bool:
    """Whether a layer runs gate_up, the activation and down as one launch
    (w4a16_moe_layer) by default: GLU16 gate_up weights, no deterministic
    pass, a long down reduction (inter >= 1024) and routing blocks of at most
    32 rows. Measured: 303.8 vs 314.6 us at the EP8 decode shard (I = 2048,
    block_m 32); slower at the TP8 shard, I = 256, whose down items are two
    pipeline stages long (516.4 vs 418.5 us at T = 256), and at the EP8
    prefill shard, whose 64-row blocks need the early-release epilogue the
    single launch does not have (703.8 vs 634.3 us)."""
    return (gate_up_layout == ops.W4A16_LAYOUT_KTILE64_GLU16 and not deterministic
            and inter >= 1024 and block_m <= 32)


class W4A16MoE:
    """One MoE layer's expert pair on one GPU (gate_up [E, 2I, H], down [E, H, I])."""

    def __init__(self, gate_up: PackedExperts, down: PackedExperts, topk: int,
                 max_tokens: int, tok_e_hint: float = 0.0, device=None,
                 deterministic: bool = False, single_launch: Optional[bool] = None):
        """With gate_up packed as W4A16_LAYOUT_KTILE64_GLU16 the activation is
        fused into the gate_up call (forward skips the separate pass). With
        deterministic=True the down pass adds each token's top-k rows in a
        fixed order (W4A16_FLAG_DETERMINISTIC): the output bits do not depend
        on the schedule. single_launch=True (GLU16 gate_up weights) runs
        gate_up, the activation and down in one launch (w4a16_moe_layer);
        None applies single_launch_default."""
        assert gate_up.num_experts == down.num_experts
        assert gate_up.n == 2 * down.k and gate_up.k == down.n
        self.gate_up, self.down = gate_up, down
        self.num_experts = gate_up.num_experts
        self.hidden, self.inter = gate_up.k, down.k
        self.topk = topk
        self.device = device or gate_up.packed.device
        self.max_tokens = max_tokens
        self.tok_e_hint = tok_e_hint
        self.deterministic = deterministic
        glu = gate_up.layout == ops.W4A16_LAYOUT_KTILE64_GLU16
        if single_launch is None:
            block_m = ops.w4a16_plan(max_tokens, topk, gate_up.num_experts, gate_up.n, gate_up.k,
                                     tok_e_hint).block_m
            single_launch = single_launch_default(gate_up.layout, deterministic, down.k, block_m)
        self.single_launch = single_launch
        if single_launch and (not glu or deterministic):
            raise ValueError("single_launch needs GLU16 gate_up weights and no deterministic pass")
        self._plan_for(max_tokens)

    def _plan_for(self, tokens: int):
        hint = self.tok_e_hint
        self.plan_gu = ops.w4a16_plan(tokens, self.topk, self.num_experts, self.gate_up.n,
                                      self.gate_up.k, hint)
        self.plan_dn = ops.w4a16_plan(tokens, self.topk, self.num_experts, self.down.n,
                                      self.down.k, hint)
        self.fused_act = self.gate_up.layout == ops.W4A16_LAYOUT_KTILE64_GLU16
        self.plan_gu.layout = self.gate_up.layout
        if self.single_launch:
            # one launch over one set of routing blocks
            if self.plan_gu.block_m > 128:
                raise ValueError("single_launch needs routing blocks of at most 128 rows")
            self.plan_dn.block_m = self.plan_gu.block_m
        self.block_m = self.plan_gu.block_m
        numel = self.max_tokens * self.topk
        self.capacity = ops.w4a16_align_capacity(numel, self.num_experts, self.block_m)
        dev = self.device
        self.sorted_ids = torch.empty(self.capacity, dtype=torch.int32, device=dev)
        self.expert_ids = torch.empty(self.capacity // self.block_m, dtype=torch.int32, device=dev)
        self.ntp = torch.empty(1, dtype=torch.int32, device=dev)
        # The down GEMM may take other blocks than gate_up (when the plans
        # differ, e.g. a 256-row gate_up plan): gate_up writes its rows in
        # token order, so each GEMM reads its own routing.
        self.block_m_dn = self.plan_dn.block_m
        if self.block_m_dn != self.block_m:
            self.capacity_dn = ops.w4a16_align_capacity(numel, self.num_experts, self.block_m_dn)
            self.sorted_ids_dn = torch.empty(self.capacity_dn, dtype=torch.int32, device=dev)
            self.expert_ids_dn = torch.empty(self.capacity_dn // self.block_m_dn,
                                             dtype=torch.int32, device=dev)
            self.ntp_dn = torch.empty(1, dtype=torch.int32, device=dev)
        else:
            self.capacity_dn = self.capacity
            self.sorted_ids_dn, self.expert_ids_dn, self.ntp_dn = (
                self.sorted_ids, self.expert_ids, self.ntp)
        self.inter_buf = torch.empty((numel, 2 * self.inter), dtype=torch.bfloat16, device=dev)
        self.act_buf = torch.empty((numel, self.inter), dtype=torch.bfloat16, device=dev)
        # one workspace for both GEMMs (ordered on one stream): status words
        # and the routed rows of the wider activation (x, k = hidden)
        self.workspace = ops.new_workspace(
            self.plan_gu, dev, max(self.capacity, self.capacity_dn), max(self.hidden, self.inter),
            det_n=self.hidden if self.deterministic else 0, det_numel=numel)
        if self.single_launch:
            self.layer_workspace = torch.zeros(
                ops.w4a16_layer_workspace_size(self.plan_gu, self.capacity, self.hidden,
                                               self.inter), dtype=torch.uint8, device=dev)
        if self.fused_act:
            self.few_workspace = torch.zeros(
                ops.w4a16_moe_few_tokens_workspace_size(
                    min(self.max_tokens, ops.W4A16_FEW_TOKENS_MAX), self.topk, self.hidden,
                    self.inter), dtype=torch.uint8, device=dev)

    def align(self, topk_ids: torch.Tensor, stream=None):
        """Routing blocks of both GEMMs (one align, two when their block sizes
        differ)."""
        self._align_down(topk_ids, stream)
        return ops.w4a16_moe_align_block_size(
            topk_ids, self.num_experts, self.block_m, self.capacity,
            out=(self.sorted_ids, self.expert_ids, self.ntp), stream=stream)

    def _align_down(self, topk_ids: torch.Tensor, stream=None):
        if self.block_m_dn != self.block_m:
            ops.w4a16_moe_align_block_size(
                topk_ids, self.num_experts, self.block_m_dn, self.capacity_dn,
                out=(self.sorted_ids_dn, self.expert_ids_dn, self.ntp_dn), stream=stream)

    def gate_up_gemm(self, x: torch.Tensor, tokens: int, stream=None):
        numel = tokens * self.topk
        return ops.w4a16_moe_indexed_gemm(
            ops.W4A16_GATE_UP, self.gate_up.packed, self.num_experts, self.gate_up.n,
            self.gate_up.k, x, tokens, self.topk, self.sorted_ids, self.expert_ids, self.ntp,
            self.plan_gu, self.workspace, out=self.inter_buf[:numel], stream=stream)

    def gate_up_act(self, x: torch.Tensor, tokens: int, stream=None):
        """gate_up with the activation fused: writes act_buf directly."""
        numel = tokens * self.topk
        return ops.w4a16_moe_indexed_gemm(
            ops.W4A16_GATE_UP_SILU, self.gate_up.packed, self.num_experts, self.gate_up.n,
            self.gate_up.k, x, tokens, self.topk, self.sorted_ids, self.expert_ids, self.ntp,
            self.plan_gu, self.workspace, out=self.act_buf[:numel], stream=stream)

    def layer_single_launch(self, x: torch.Tensor, tokens: int, topk_weights: torch.Tensor,
                            out: torch.Tensor, stream=None):
        """gate_up, activation and down in one launch (w4a16_moe_layer)."""
        return ops.w4a16_moe_layer(
            self.gate_up.packed, self.down.packed, self.num_experts, self.hidden, self.inter, x,
            tokens, self.topk, self.sorted_ids, self.expert_ids, self.ntp, self.plan_gu,
            self.layer_workspace, topk_weights, out=out, stream=stream)

    def activation(self, tokens: int, stream=None):
        numel = tokens * self.topk
        return ops.w4a16_silu_and_mul(self.inter_buf[:numel], out=self.act_buf[:numel],
                                      stream=stream)

    def down_gemm(self, tokens: int, topk_weights: torch.Tensor, out: torch.Tensor, stream=None):
        numel = tokens * self.topk
        return ops.w4a16_moe_indexed_gemm(
            ops.W4A16_DOWN, self.down.packed, self.num_experts, self.down.n, self.down.k,
            self.act_buf[:numel], tokens, self.topk, self.sorted_ids_dn, self.expert_ids_dn,
            self.ntp_dn, self.plan_dn, self.workspace, topk_weights=topk_weights, out=out,
            flags=ops.W4A16_FLAG_DETERMINISTIC if self.deterministic else 0, stream=stream)

    def route(self, router_logits: torch.Tensor, expert_offset: int = 0,
              renormalize: bool = True, stream=None):
        """Router logits [T, E_global] (fp32 or BF16) -> (topk_ids, topk_weights)
        for this GPU's experts [expert_offset, expert_offset + num_experts),
        on the device (w4a16_topk_softmax)."""
        return ops.w4a16_topk_softmax(router_logits, self.topk, renormalize, expert_offset,
                                      self.num_experts,
                                      out=self._routing(router_logits.shape[0], stream),
                                      stream=stream)

    def _routing(self, tokens: int, stream):
        """The layer's own (topk_ids, topk_weights), made by the first call."""
        if tokens > self.max_tokens:
            raise ValueError("more tokens than the layer was planned for")
        if not hasattr(self, "_route_ids"):
            with ops.on_stream(stream):
                self._route_ids = torch.empty((self.max_tokens, self.topk), dtype=torch.int32,
                                              device=self.device)
                self._route_w = torch.empty((self.max_tokens, self.topk), dtype=torch.float32,
                                            device=self.device)
        return self._route_ids[:tokens], self._route_w[:tokens]

    def route_align(self, router_logits: torch.Tensor, expert_offset: int = 0,
                    renormalize: bool = True, stream=None):
        """route() and align() in one launch (w4a16_moe_route_align): returns
        (topk_ids, topk_weights) and fills the layer's routing tensors."""
        ids, w = self._routing(router_logits.shape[0], stream)
        if not hasattr(self, "_arrivals"):
            with ops.on_stream(stream):
                self._arrivals = torch.zeros(1, dtype=torch.int32, device=self.device)
        ops.w4a16_moe_route_align(
            router_logits, self.topk, self.block_m, self._arrivals, renormalize, expert_offset,
            self.num_experts, self.capacity,
            out=(ids, w, self.sorted_ids, self.expert_ids, self.ntp), stream=stream)
        # the down GEMM's own blocks over the same local ids
        self._align_down(ids, stream)
        return ids, w

    def forward_from_logits(self, x: torch.Tensor, router_logits: torch.Tensor,
                            expert_offset: int = 0, renormalize: bool = True,
                            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The whole layer from router logits: route + align (one launch),
        gate_up(+act), down."""
        _, w = self.route_align(router_logits, expert_offset, renormalize, stream)
        return self.experts(x, w, out=out, stream=stream)

    def forward(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """x BF16 [T, H], topk_ids int32 [T, topk], topk_weights fp32 [T, topk]
        -> fp32 [T, H] (this GPU's experts' share of the top-k weighted sum)."""
        tokens = x.shape[0]
        if tokens > self.max_tokens:
            raise ValueError("more tokens than the layer was planned for")
        if out is None:
            with ops.on_stream(stream):
                out = torch.empty((tokens, self.hidden), dtype=torch.float32, device=x.device)
        self.align(topk_ids, stream)
        return self.experts(x, topk_weights, out=out, stream=stream)

    def _few(self, x, ids, weights, x_scales, out, stream, **routing) -> torch.Tensor:
        if x.shape[0] > self.max_tokens:
            raise ValueError("more tokens than the layer was planned for")
        if not self.fused_act:
            raise ValueError("few_tokens needs GLU16 gate_up weights")
        return ops.w4a16_moe_few_tokens(
            self.gate_up.packed, self.down.packed, self.num_experts, self.hidden, self.inter, x,
            ids, weights, self.few_workspace, x_scales=x_scales, out=out, stream=stream,
            **routing)

    def few_tokens(self, x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                   x_scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
        """forward() for up to W4A16_FEW_TOKENS_MAX tokens in one launch
        (w4a16_moe_few_tokens): the arguments and the result of forward, with
        the activation kept to 22 bits and a fixed order of additions. x may also
        be e4m3 [T, H] with x_scales FP32 [T, ceil(H/128)]. Needs
        W4A16_LAYOUT_KTILE64_GLU16 gate_up weights."""
        return self._few(x, topk_ids, topk_weights, x_scales, out, stream)

    def few_tokens_from_logits(self, x: torch.Tensor, router_logits: torch.Tensor,
                               expert_offset: int = 0, renormalize: bool = True,
                               x_scales: Optional[torch.Tensor] = None,
                               out: Optional[torch.Tensor] = None, routing=None,
                               stream=None) -> torch.Tensor:
        """few_tokens from router logits [T, E_global], the routing in the same
        launch. routing: (topk_ids int32, topk_weights fp32) [T, topk] tensors
        that receive it (the layer's own buffers when None)."""
        if routing is None:
            routing = self._routing(x.shape[0], stream)
        return self._few(x, routing[0], routing[1], x_scales, out, stream, logits=router_logits,
                         renormalize=renormalize, expert_offset=expert_offset)

    def experts(self, x: torch.Tensor, topk_weights: torch.Tensor,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """gate_up(+act) and down over the routing tensors already aligned."""
        tokens = x.shape[0]
        if out is None:
            with ops.on_stream(stream):
                out = torch.empty((tokens, self.hidden), dtype=torch.float32, device=x.device)
        if self.single_launch:
            return self.layer_single_launch(x, tokens, topk_weights, out, stream)
        if self.fused_act:
            self.gate_up_act(x, tokens, stream)
        else:
            self.gate_up_gemm(x, tokens, stream)
            self.activation(tokens, stream)
        self.down_gemm(tokens, topk_weights, out, stream)
        return out


class SharedExpert:
    """An expert that every token passes, weights in BF16: gate_up [2I, H] (gate
    rows, then up rows) and down [H, I]. Two launches for any number of tokens
    (w4a16_dense); the activation between them is BF16."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor):
        if (gate_up.dim() != 2 or down.dim() != 2 or gate_up.shape[0] != 2 * down.shape[1]
                or gate_up.shape[1] != down.shape[0]):
            raise ValueError("gate_up is [2I, H], down [H, I]")
        self.gate_up, self.down = gate_up, down
        self.hidden, self.inter = down.shape

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, add: bool = False,
                stream=None) -> torch.Tensor:
        """x BF16 [T, H] -> fp32 [T, H]; add: onto what out holds."""
        if add and out is None:
            raise ValueError("add needs what it adds to")
        act = ops.w4a16_dense(x, self.gate_up, gated=True, stream=stream)
        return ops.w4a16_dense(act, self.down, addend=out if add else None,
                               out_dtype=torch.float32, out=out, stream=stream)


class PackedSharedExpert:
    """SharedExpert with INT4 weights in the routed experts' own format: gate_up
    packed with W4A16_LAYOUT_KTILE64_GLU16, both of one expert. Up to
    W4A16_FEW_TOKENS_MAX tokens take two launches (w4a16_linear_few_tokens), more
    the GEMM path, planned for max_tokens, with every token routed to the one
    expert. The few-token products round no weight and keep gate and up in FP32;
    the GEMM path rounds the scaled weights to BF16, and gate and up before silu,
    as it does for routed experts. Its calls share the expert's buffers: one
    stream at a time, while few-token calls share nothing."""

    def __init__(self, gate_up: PackedExperts, down: PackedExperts, max_tokens: int):
        if gate_up.num_experts != 1 or gate_up.layout != ops.W4A16_LAYOUT_KTILE64_GLU16:
            raise ValueError("a shared expert is one expert with GLU16 gate_up weights")
        if down.num_experts != 1 or gate_up.n != 2 * down.k or gate_up.k != down.n:
            raise ValueError("gate_up is [1, 2I, H], down [1, H, I]")
        self.gate_up, self.down = gate_up, down
        self.hidden, self.inter = down.n, down.k
        self.max_tokens = max_tokens
        self.layer = None
        if max_tokens > ops.W4A16_FEW_TOKENS_MAX:
            self.layer = W4A16MoE(gate_up, down, 1, max_tokens, single_launch=False)
            dev = self.layer.device
            self.ids = torch.zeros((max_tokens, 1), dtype=torch.int32, device=dev)
            self.weights = torch.ones((max_tokens, 1), dtype=torch.float32, device=dev)

    def forward(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, add: bool = False,
                stream=None) -> torch.Tensor:
        """x BF16 [T, H] (rows that are strided are copied where the GEMM path runs)
        -> fp32 [T, H]; add: onto what out holds."""
        if add and out is None:
            raise ValueError("add needs what it adds to")
        tokens = x.shape[0]
        if x.dtype is not torch.bfloat16 or x.shape != (tokens, self.hidden):
            raise ValueError(f"x: {x.dtype} {tuple(x.shape)}, not BF16 rows of {self.hidden}")
        if tokens > self.max_tokens:
            raise ValueError("more tokens than the expert was planned for")
        if tokens <= ops.W4A16_FEW_TOKENS_MAX:
            act = ops.w4a16_linear_few_tokens(x, self.gate_up.packed, self.gate_up.n,
                                              self.gate_up.layout, stream=stream)
            return ops.w4a16_linear_few_tokens(act, self.down.packed, self.down.n,
                                               addend=out if add else None,
                                               out_dtype=torch.float32, out=out, stream=stream)
        if out is not None and (out.dtype is not torch.float32 or out.shape != x.shape
                                or out.device != x.device or not out.is_contiguous()):
            raise ValueError(f"out: {out.dtype} {tuple(out.shape)} on {out.device}, "
                             f"not contiguous FP32 {tuple(x.shape)}")
        if x.device != self.gate_up.packed.device:
            raise ValueError(f"x on {x.device}, weights on {self.gate_up.packed.device}")
        if x.is_cuda and x.get_device() != ops._current_device():
            with torch.cuda.device(x.get_device()):   # (where the GEMM path launches)
                return self.forward(x, out, add, stream)
        if not x.is_contiguous():   # (the GEMM path reads rows in line)
            with ops.on_stream(stream):
                x = x.contiguous()
        layer = self.layer
        layer.align(self.ids[:tokens], stream)
        layer.gate_up_act(x, tokens, stream)
        return ops.w4a16_moe_indexed_gemm(
            ops.W4A16_DOWN, self.down.packed, 1, self.down.n, self.down.k, layer.act_buf[:tokens],
            tokens, 1, layer.sorted_ids_dn, layer.expert_ids_dn, layer.ntp_dn, layer.plan_dn,
            layer.workspace, topk_weights=self.weights[:tokens], out=out,
            flags=ops.W4A16_FLAG_ACCUMULATE if add else 0, stream=stream)


@dataclass
class BlockNorm:
    """The norms around the border between a block and the next one
    (w4a16_block_norm): the norm of the block's output (post_weight, None: none),
    its gate (BF16 [H] or [T, H]) and scales, the residual, and the norm in front
    of the next block (pre_weight). weight_offset is added to both weights."""
    pre_weight: torch.Tensor
    post_weight: Optional[torch.Tensor] = None
    gate: Optional[torch.Tensor] = None
    branch_scale: float = 1.0
    residual_scale: float = 1.0
    weight_offset: float = 0.0
    eps: float = 1e-6

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                fp8_group: int = ops.W4A16_FP8_NONE, stream=None):
        """x fp32 or BF16 [T, H], residual BF16 [T, H] -> (the next block's rows
        BF16, the new residual BF16, e4m3 rows and their scales or None)."""
        return ops.w4a16_block_norm(
            x, self.pre_weight, self.eps, post_weight=self.post_weight, gate=self.gate,
            residual=residual, branch_scale=self.branch_scale,
            residual_scale=self.residual_scale, weight_offset=self.weight_offset,
            fp8_group=fp8_group, stream=stream)


class MoEBlock:
    """The MoE half of a decoder layer on one GPU: the residual's addition and
    the RMS norm, the router's product, and the layer's experts.

    Up to W4A16_FEW_TOKENS_MAX tokens (with GLU16 gate_up weights) take three
    launches: norm, router, experts; more tokens take the layer's GEMM path
    (W4A16MoE.forward_from_logits). (The limit is the few-token call's own: with
    many rows an expert the GEMM path may be faster before it.) fp8_rows=True
    hands the few-token experts the norm's 8-bit rows (the form that tokens have
    after an exchange in 8 bits) and has no effect on the GEMM path; the router
    always reads the BF16 rows. shared (SharedExpert or PackedSharedExpert): the
    expert that every token passes, added to the routed experts' sum (where the
    routed experts are spread over GPUs, give it to one of them). after: the norms
    that forward_layer runs behind the block."""

    def __init__(self, norm_weight: torch.Tensor, router_weight: torch.Tensor, experts: W4A16MoE,
                 eps: float = 1e-6, expert_offset: int = 0, renormalize: bool = True,
                 fp8_rows: bool = False, shared=None, after: Optional[BlockNorm] = None):
        if shared is not None and shared.hidden != experts.hidden:
            raise ValueError("the shared expert does not match the layer's hidden size")
        if norm_weight.shape != (experts.hidden,) or router_weight.shape[1] != experts.hidden:
            raise ValueError("norm and router weights do not match the layer's hidden size")
        self.norm_weight, self.router_weight, self.layer = norm_weight, router_weight, experts
        self.eps, self.expert_offset, self.renormalize = eps, expert_offset, renormalize
        self.fp8_rows = fp8_rows
        self.shared, self.after = shared, after

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None):
        """x, residual BF16 [T, H] -> (fp32 [T, H] of this GPU's experts, the
        new residual BF16 [T, H], x itself when none was given)."""
        few = (x.shape[0] <= ops.W4A16_FEW_TOKENS_MAX
               and self.layer.gate_up.layout == ops.W4A16_LAYOUT_KTILE64_GLU16)
        fp8 = few and self.fp8_rows
        y, new_residual, y8, scales = ops.w4a16_add_rms_norm(
            x, self.norm_weight, self.eps, residual=residual,
            fp8_group=ops.W4A16_FP8_GROUP if fp8 else ops.W4A16_FP8_NONE, stream=stream)
        logits = ops.w4a16_router_logits(y, self.router_weight, stream=stream)
        if few:
            result = self.layer.few_tokens_from_logits(
                y8 if fp8 else y, logits, self.expert_offset, self.renormalize, x_scales=scales,
                out=out, stream=stream)
        else:
            result = self.layer.forward_from_logits(y, logits, self.expert_offset,
                                                    self.renormalize, out=out, stream=stream)
        if self.shared is not None:
            self.shared.forward(y, out=result, add=True, stream=stream)
        return result, x if residual is None else new_residual

    def forward_layer(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None,
                      fp8_group: int = ops.W4A16_FP8_NONE, stream=None):
        """forward() and the norms behind it (`after`), on a GPU that holds all of
        the layer's experts: (the next block's rows BF16 [T, H], the new residual
        BF16, e4m3 rows and their scales or None)."""
        if self.after is None:
            raise ValueError("forward_layer needs the norms behind the block")
        y, residual = self.forward(x, residual, stream=stream)
        return self.after.forward(y, residual, fp8_group, stream)
