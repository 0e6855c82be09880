"""A routed expert layer in training, and the block around it, on the library's kernels.

``ExpertLayer`` holds the layer's buffers and strings the operators of
include/moe_train.h together as a training step uses them:

  route     moe_route_topk or moe_route_scores -> moe_plan -> moe_plan_groups
  forward   moe_gather_rows -> moe_grouped_gemm (gate/up, SwiGLU epilogue)
            -> moe_grouped_gemm (down) -> moe_sum_routes
  backward  moe_gather_rows (of the output's gradient: the sum's gradient)
            -> moe_grouped_gemm (input gradient) -> moe_swiglu_backward
            -> moe_grouped_wgrad twice -> moe_grouped_gemm (input gradient)
            -> moe_sum_routes (the gather's gradient)
  step      moe_adamw_step over both weights

The route weight multiplies the SwiGLU output, so the combine is a plain sum
and the weights' gradient falls out of the SwiGLU gradient.  The trained
weights go on to moe_quantize_weight_128x128 and the FP8 forward
(``quantized``).

With ``scores`` the layer routes by scores (include/moe_block.h): ``route``
calls moe_route_scores, ``route_backward`` gives the logits' gradient and
``balance`` moves the balance bias.

``ExpertBlock`` is the layer with what stands around it: norm, router product,
experts, norm, gate and residual, forward, backward and served in FP8.
"""

import math

import torch

from . import _lib as L


class ExpertLayer:
    """A routed expert layer of E experts, hidden size H, intermediate size I.

    tokens: the batch's token count (the buffers' size).  Weights are kept in
    FP32 with a copy in `dtype` that the products read; states in 32 or 8 bits.
    scores: None for the plain router (the top_k logits, softmax over them), or the
    keywords of make_route_scores_args that say how to route by scores (score,
    groups, topk_groups, group_score, renormalize, routed_scale); with
    ``"balance": True`` among them the layer has a balance bias.
    """

    scores = bias = None                                  # the plain router

    def __init__(self, tokens, H, I, E, top_k, block_m=16, dtype=torch.bfloat16, state_bits=32, weight_decay=0.0,
                 device="cuda", generator=None, scores=None):
        self.M, self.H, self.I, self.E, self.top_k, self.block_m, self.dtype = tokens, H, I, E, top_k, block_m, dtype
        dev = torch.device(device)
        R = tokens * top_k
        cap, blocks = L.moe_plan_capacity(tokens, top_k, E, block_m)

        def empty(*shape, dt=dtype):
            return torch.empty(*shape, dtype=dt, device=dev)

        self.topk_ids, self.topk_weights = empty(tokens, top_k, dt=torch.int32), empty(tokens, top_k, dt=torch.float32)
        self.sorted_ids, self.expert_ids = empty(cap, dt=torch.int32), empty(blocks, dt=torch.int32)
        self.num_padded = empty(1, dt=torch.int32)
        self.plan_workspace = empty(max(L.moe_plan_workspace_size(tokens, top_k, E), 256), dt=torch.uint8)
        self.group_start, self.group_rows = empty(E, dt=torch.int32), empty(E, dt=torch.int32)
        self.route_slot = empty(R, dt=torch.int32)
        if scores is not None:
            self.scores = {k: v for k, v in scores.items() if k != "balance"}
            self.bias = torch.zeros(E, device=dev) if scores.get("balance") else None
        self._routed = None                               # the last route's logits and token count
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

        # rows in plan order
        self.xs, self.pre, self.h, self.ys = empty(cap, H), empty(cap, 2 * I), empty(cap, I), empty(cap, H)
        self.out, self.dx = empty(tokens, H), empty(tokens, H)
        self.dys, self.dh = empty(cap, H), empty(cap, I)
        self.dxs = self.ys                                # the forward's rows are no longer needed then
        self.dweights = torch.zeros(tokens, top_k, device=dev)

        self.params, self.models, self.grads = [], [], []
        for shape, fan_in in (((E, 2 * I, H), H), ((E, H, I), I)):
            p = torch.randn(*shape, device=dev, generator=generator) * fan_in ** -0.5
            self.params.append(p)
            self.models.append(p.to(dtype))
            self.grads.append(torch.zeros(*shape, dtype=dtype, device=dev))
        self.w13, self.w2 = self.models
        self.states = []
        for p in self.params:
            n = p.numel()
            if state_bits == 32:
                self.states.append({k: torch.zeros(n, device=dev) for k in ("exp_avg", "exp_avg_sq")})
            else:
                s = {k: torch.zeros(n, dtype=torch.uint8, device=dev) for k in ("exp_avg", "exp_avg_sq")}
                s |= {k + "_scale": torch.zeros(-(-n // 128), device=dev) for k in ("exp_avg", "exp_avg_sq")}
                self.states.append(s)
        self.table = L.AdamWTable(
            [{"param": p.view(-1), "model": m.view(-1), "grad": g.view(-1), **s}
             for p, m, g, s in zip(self.params, self.models, self.grads, self.states)], weight_decay=weight_decay)
        self._forward_done = False                        # pre, h and xs are those of a forward pass
        self.steps = 0                                    # steps that changed the weights
        self._calls = 0
        self._skipped = None                              # the last step's skip flag on its way to the host

        groups = (self.group_start, self.group_rows)
        self._up = L.make_grouped_args(self.xs, self.w13, self.h, *groups, epilogue=L.GROUPED_SWIGLU, pre=self.pre,
                                       route_ids=self.sorted_ids, route_weights=self.topk_weights,
                                       device_status=self.status)
        self._down = L.make_grouped_args(self.h, self.w2, self.ys, *groups, device_status=self.status)
        self._dh = L.make_grouped_args(self.dys, self.w2, self.dh, *groups, input_gradient=True,
                                       device_status=self.status)
        # dpre takes the place of pre, the recomputed h that of dh
        self._swiglu = L.make_swiglu_backward_args(self.dh, self.pre, self.pre, h=self.dh, route_ids=self.sorted_ids,
                                                   num_rows=self.num_padded, route_weights=self.topk_weights,
                                                   dweights=self.dweights)
        self._dw2 = L.make_grouped_wgrad_args(self.dys, self.dh, self.grads[1], *groups, device_status=self.status)
        self._dw13 = L.make_grouped_wgrad_args(self.pre, self.xs, self.grads[0], *groups, device_status=self.status)
        self._dxs = L.make_grouped_args(self.pre, self.w13, self.dxs, *groups, input_gradient=True,
                                        device_status=self.status)

    def _batch(self, name, t, width, dtypes):
        """ValueError unless t is a [tokens, width] tensor of one of the types (the layer's buffers hold as many rows)."""
        if tuple(t.shape) != (self.M, width):
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(self.M, width)}")
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")

    def route(self, logits, num_tokens=None):
        """Router, plan and groups from logits [tokens, E] (contiguous, float32 or bfloat16; by scores
        any row stride and float16 too).  num_tokens [1] int32 on the device, by scores only: the
        tokens from there on are padding and get no expert."""
        plain = self.scores is None
        self._batch("logits", logits, self.E, (torch.float32, torch.bfloat16) + (() if plain else (torch.float16,)))
        if plain and not logits.is_contiguous():
            raise ValueError("logits: a contiguous tensor is expected")
        if plain and num_tokens is not None:
            raise ValueError("num_tokens: the plain router takes whole batches")
        self._forward_done = False
        self._routed = None
        if plain:
            L.moe_route_topk(logits, self.top_k, self.topk_ids, self.topk_weights)
        else:
            L.moe_route_scores(L.make_route_scores_args(logits, self.topk_ids, self.topk_weights, bias=self.bias,
                                                        num_tokens=num_tokens, **self.scores))
        L.moe_plan(self.topk_ids, self.E, self.block_m, self.sorted_ids, self.expert_ids, self.num_padded,
                   self.plan_workspace)
        L.moe_plan_groups(self.sorted_ids, self.expert_ids, self.num_padded, self.block_m, self.M * self.top_k,
                          self.group_start, self.group_rows, self.route_slot)
        self._routed = logits, num_tokens

    def forward(self, x):
        """x [tokens, H] -> out [tokens, H] (the layer's own buffer)."""
        self._batch("x", x, self.H, (self.dtype,))
        L.moe_gather_rows(x, self.xs, self.sorted_ids, self.top_k, self.num_padded)
        L.moe_grouped_gemm(self._up)
        L.moe_grouped_gemm(self._down)
        L.moe_sum_routes(self.ys, self.out, self.route_slot, self.top_k)
        self._forward_done = True
        return self.out

    def backward(self, dout):
        """dout [tokens, H] -> (dx [tokens, H], the route weights' gradient
        [tokens, top_k]); fills grads.  Uses the last forward's buffers up:
        RuntimeError without a forward pass since the last route or backward."""
        self._batch("dout", dout, self.H, (self.dtype,))
        if not self._forward_done:
            raise RuntimeError("backward without a forward pass since the last route or backward")
        self._forward_done = False
        L.moe_gather_rows(dout, self.dys, self.sorted_ids, self.top_k, self.num_padded)
        L.moe_grouped_gemm(self._dh)
        self.dweights.zero_()                             # (the kernel leaves routes that the plan does not hold)
        L.moe_swiglu_backward(self._swiglu)
        L.moe_grouped_wgrad(self._dw2)
        L.moe_grouped_wgrad(self._dw13)
        L.moe_grouped_gemm(self._dxs)
        L.moe_sum_routes(self.dxs, self.dx, self.route_slot, self.top_k)
        return self.dx, self.dweights

    def route_backward(self, dweights, dlogits=None):
        """The gradient of the last route's logits from the route weights' (as ``backward`` returns
        it), in the logits' type.  The logits must still hold what was routed."""
        if self._routed is None:
            raise RuntimeError("route_backward without a route")
        logits, num_tokens = self._routed
        how = {"score": L.SCORE_SOFTMAX} if self.scores is None else {
            k: v for k, v in self.scores.items() if k in ("score", "renormalize", "routed_scale")}
        dlogits = torch.empty_like(logits) if dlogits is None else dlogits
        L.moe_route_scores_backward(L.make_route_scores_backward_args(logits, self.topk_ids, dweights, dlogits,
                                                                      num_tokens=num_tokens, **how))
        return dlogits

    def balance(self, rate):
        """One step of the balance bias towards an even load, from the last route's."""
        if self.bias is None:
            raise RuntimeError("the layer has no balance bias")
        if self._routed is None:
            raise RuntimeError("balance without a route")
        L.moe_route_balance(self.group_rows, self.bias, rate)

    def step(self, lr, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=None, skip=None):
        """One AdamW step of both weights from grads.

        skip [1] int32: where it is not 0 the step changes nothing and does not
        count (the bias corrections follow ``steps``).  The flag reaches the host
        behind the step; the next call waits for it, so that the host is at most
        a step ahead.  In a captured graph lr, the step's number and the seed
        would stay those of the capture: call it outside."""
        if self._skipped is not None:
            flag, copied = self._skipped
            copied.synchronize()
            self.steps -= 1 if int(flag) else 0
            self._skipped = None
        self.steps += 1
        self._calls += 1                                  # (each call's rounding has its own seed, skipped ones too)
        L.moe_adamw_step(L.make_adamw_args(self.table, lr=lr, step=self.steps, beta1=beta1, beta2=beta2, eps=eps,
                                           seed=self._calls, grad_scale=grad_scale, skip=skip))
        if skip is not None:
            flag, copied = torch.empty(1, dtype=torch.int32, pin_memory=True), torch.cuda.Event()
            flag.copy_(skip.view(-1)[:1], non_blocking=True)
            copied.record()
            self._skipped = flag, copied

    def quantized(self, out=None):
        """The trained weights as the FP8 forward takes them: (w13 interleaved,
        w13_scale, w2, w2_scale).  H, I multiples of 128; BF16 weights, ValueError for others.
        out: what an earlier call returned, written again instead of new tensors."""
        kinds = [k for w in self.models for k in (
            (tuple(w.shape), torch.uint8), ((w.shape[0], w.shape[1] // 128, w.shape[2] // 128), torch.float32))]
        if out is None:
            out = tuple(torch.empty(shape, dtype=dtype, device=self.models[0].device) for shape, dtype in kinds)
        elif [(tuple(t.shape), t.dtype) for t in out] != kinds or not all(t.is_contiguous() for t in out):
            raise ValueError("out: what an earlier call returned is expected")
        w13, w13_scale, w2, w2_scale = out
        rows = torch.empty_like(w13)                      # (before they are interleaved)
        L.moe_quantize_weight_128x128(self.models[0], rows, w13_scale)
        L.moe_quantize_weight_128x128(self.models[1], w2, w2_scale)
        L.moe_prep_weights(rows, w13)
        return out

    def weights_version(self):
        """Another value after each step of the layer and each write of torch's to the weights (tensors
        made in inference mode keep no count of those)."""
        return self._calls, tuple(0 if w.is_inference() else w._version for w in self.models)


class ExpertBlock:
    """norm -> router -> experts -> norm, gate, residual, on a stream x [tokens, H] of the layer's type:

      z   = N(x; w_pre)
      y   = experts(z), routed by scores of z w_router^T
      out = residual_scale x + gate * N(y; w_post)

    All parameters are FP32; the experts are an ``ExpertLayer`` (``layer``), whose keywords
    are passed on.  z and out come from a pass each over the stream (blocks in a row could share one:
    moe_norm_residual forms both).  The router's product is a library product of FP32 values, by torch's setting for those
    (torch.backends.cuda.matmul: TF32 where that allows it).  gate: a learned
    factor for each channel, starting at gate_init; None for none.
    """

    def __init__(self, tokens, H, I, E, top_k, scores=None, gate_init=1.0, residual_scale=1.0, eps=1e-6, dtype=torch.bfloat16,
                 device="cuda", generator=None, state_bits=32, weight_decay=0.0, **layer):
        scores = {"score": L.SCORE_SIGMOID, "balance": True} if scores is None else scores
        self.layer = ExpertLayer(tokens, H, I, E, top_k, dtype=dtype, device=device, generator=generator, scores=scores,
                                 state_bits=state_bits, weight_decay=weight_decay, **layer)
        dev = torch.device(device)
        self.M, self.H, self.E, self.dtype, self.residual_scale, self.eps = tokens, H, E, dtype, residual_scale, eps
        self.w_router = torch.randn(E, H, device=dev, generator=generator) * H ** -0.5
        self.w_pre, self.w_post = torch.ones(H, device=dev), torch.ones(H, device=dev)
        self.gate = None if gate_init is None else torch.full((H,), float(gate_init), device=dev)
        self.params = {"w_router": self.w_router, "w_pre": self.w_pre, "w_post": self.w_post}
        if self.gate is not None:
            self.params["gate"] = self.gate
        self.grads = {k: torch.zeros_like(p) for k, p in self.params.items()}
        rows = lambda: torch.empty(tokens, H, dtype=dtype, device=dev)                # noqa: E731
        self.z, self.out, self.dy, self.dr, self.dx = rows(), rows(), rows(), rows(), rows()
        self.logits = torch.empty(tokens, E, device=dev)
        self._workspace = torch.empty(L.moe_norm_residual_workspace_size(tokens, H), dtype=torch.uint8, device=dev)
        states = [{k: torch.zeros(p.numel(), device=dev) for k in ("exp_avg", "exp_avg_sq")} for p in self.params.values()]
        self._table = L.AdamWTable([{"param": p.view(-1), "grad": g.view(-1), **s}
                                    for p, g, s in zip(self.params.values(), self.grads.values(), states)])
        self._serving = None                              # what serve keeps, and the weights whose codes it holds
        self._served_version = None
        self._x = None                                    # the last forward's stream
        self._load, self._loaded = torch.zeros(E, dtype=torch.int32, device=dev), False        # its experts' loads

    @property
    def steps(self):
        return self.layer.steps

    @staticmethod
    def _product(a, b, out=None):
        """The router's product and its gradients: FP32 whatever torch.autocast says."""
        with torch.autocast("cuda", enabled=False):
            return torch.mm(a, b, out=out)

    @staticmethod
    def _apart(name, t, own):
        if t.numel() and any(t.untyped_storage().data_ptr() == o.untyped_storage().data_ptr() for o in own):
            raise ValueError(f"{name}: a buffer of the block itself")

    def _take(self, x, *own):
        """ValueError unless x is a batch and lies apart from what the pass writes."""
        self.layer._batch("x", x, self.H, (self.dtype,))
        self._apart("x", x, (self.z, self.out, *own))

    def _enter(self, x, num_tokens, **out):
        self._x = None                                    # (the buffers are no longer the last forward's)
        if num_tokens is not None:
            self.z.zero_()                                # (what padding rows hold goes through the router's product)
        L.moe_norm_residual(L.make_norm_residual_args(x, z=self.z, w_pre=self.w_pre, eps=self.eps, num_rows=num_tokens, **out))
        self._product(self.z.float(), self.w_router.t(), out=self.logits)
        self.layer.route(self.logits, num_tokens)

    def _leave(self, x, y, num_tokens):
        L.moe_norm_residual(L.make_norm_residual_args(y, h=self.out, r=x, gate=self.gate, w_post=self.w_post, eps=self.eps,
                                                      residual_scale=self.residual_scale, num_rows=num_tokens))
        return self.out

    def forward(self, x, num_tokens=None):
        """x [tokens, H] -> out [tokens, H] (the block's own buffer).  num_tokens [1] int32 on the
        device: rows from there on are padding; their out is not written.

        x is read again by ``backward``: it may be no buffer of the block or its layer."""
        layer = self.layer
        self._take(x, self.dy, self.dr, self.dx, layer.out, layer.dx, layer.xs, layer.pre, layer.h, layer.ys, layer.dys, layer.dh)
        self._enter(x, num_tokens)
        if layer.bias is not None:
            self._load.copy_(layer.group_rows)            # (a served batch has its own)
            self._loaded = True
        y = layer.forward(self.z)
        self._x = x, y, num_tokens
        return self._leave(x, y, num_tokens)

    def backward(self, dout):
        """dout [tokens, H] -> dx [tokens, H]; fills grads and the experts' grads.  x and num_tokens must
        still hold what the last forward pass was given."""
        if self._x is None:
            raise RuntimeError("backward without a forward pass")
        self.layer._batch("dout", dout, self.H, (self.dtype,))
        self._apart("dout", dout, (self.dy, self.dr, self.dx, self.layer.dx))
        x, y, num_tokens = self._x
        self._x = None
        if num_tokens is not None:
            for t in (self.dy, self.dr, self.dx):
                t.zero_()
        how = {"eps": self.eps, "workspace": self._workspace, "num_rows": num_tokens}
        L.moe_norm_residual_backward(L.make_norm_residual_backward_args(
            y, dh=dout, gate=self.gate, w_post=self.w_post, residual_scale=self.residual_scale, dy=self.dy, dr=self.dr,
            dgate=self.grads.get("gate"), dw_post=self.grads["w_post"], **how))
        dz, dweights = self.layer.backward(self.dy)
        dlogits = self.layer.route_backward(dweights)
        self._product(dlogits.t(), self.z.float(), out=self.grads["w_router"])
        dz.add_(self._product(dlogits, self.w_router))    # (rounded once more: the experts' part lies in 16 bits)
        L.moe_norm_residual_backward(L.make_norm_residual_backward_args(
            x, dh=self.dr, dz=dz, w_pre=self.w_pre, dy=self.dx, dw_pre=self.grads["w_pre"], **how))
        return self.dx

    def step(self, lr, balance_rate=0.0, **adam):
        """One AdamW step of all parameters from their grads (the experts' keywords: ``ExpertLayer.step``),
        and one of the balance bias towards an even load, from the last forward pass's.  A step that skip leaves
        out does not count for any of them."""
        layer = self.layer
        if balance_rate and layer.bias is None:
            raise RuntimeError("the layer has no balance bias")
        if balance_rate and not self._loaded:
            raise RuntimeError("balance without a forward pass")
        if balance_rate and not math.isfinite(balance_rate):
            raise ValueError(f"balance_rate: {balance_rate}")
        layer.step(lr, **adam)                            # (it settles the steps' number)
        L.moe_adamw_step(L.make_adamw_args(self._table, lr=lr, step=layer.steps, **adam))
        if balance_rate:
            skip = adam.get("skip")
            if skip is None:
                L.moe_route_balance(self._load, layer.bias, balance_rate)
            else:
                moved = torch.empty_like(layer.bias)
                L.moe_route_balance(self._load, layer.bias, balance_rate, out=moved)
                torch.where(skip.view(-1)[:1] == 0, moved, layer.bias, out=layer.bias)

    def _serving_buffers(self):
        layer, dev, I = self.layer, self.z.device, self.layer.I
        ws = torch.empty(L.moe_forward_workspace_size(self.M, self.H, I, self.E, layer.top_k, layer.block_m, layer.sorted_ids.numel()),
                         dtype=torch.uint8, device=dev)
        L.moe_workspace_init(ws)
        q, q_scale = torch.zeros(self.M, self.H, dtype=torch.uint8, device=dev), torch.zeros(self.M, self.H // 128, device=dev)
        y = torch.empty(self.M, self.H, dtype=torch.bfloat16, device=dev)
        codes = layer.quantized()
        return q, q_scale, y, codes, ws, L.make_fwd_args(
            q, q_scale, *codes, layer.topk_weights, layer.sorted_ids, layer.expert_ids, layer.num_padded, y, ws,
            layer.top_k, layer.block_m, device_status=layer.status)

    def refresh(self):
        """Forms the FP8 weights that ``serve`` reads anew, where they lie.  Needed after writes to the
        experts' weights that neither ``step`` (the block's or the layer's) nor torch has made, and
        after torch's where the block was made in inference mode."""
        self._quantise()

    def _quantise(self):
        """What serve keeps, with the codes of the present weights."""
        version = self.layer.weights_version()
        capturing = torch.cuda.is_current_stream_capturing()     # (nothing has run yet then)
        if self._serving is None:
            serving = self._serving_buffers()
            if capturing:
                return serving                            # the graph's own
            self._serving = serving
        else:
            self.layer.quantized(out=self._serving[3])
        self._served_version = None if capturing else version
        return self._serving

    def serve(self, x, num_tokens=None):
        """forward in FP8: the entry's norm writes the experts' input as E4M3 codes with 1x128 scales
        beside the router's, the experts run in moe_fp8_block_scale_forward.  H, I multiples of
        128, BF16.

        The weights are quantised when they have changed since the last call: by a step of the block or of
        its layer, or by torch's writes to ``layer.models`` (other writes: ``refresh``).  A captured call
        reads the codes where they lie, so that its replays follow the next call outside the graph; if the
        weights have changed before it, or nothing was served yet, the graph forms the codes itself, at each replay."""
        self._take(x)
        layer = self.layer
        fresh = self._serving is not None and self._served_version == layer.weights_version()
        serving = self._serving if fresh else self._quantise()
        q, q_scale, y, _, _, args = serving
        self._enter(x, num_tokens, q=q, q_scale=q_scale)
        y.zero_()
        L.moe_fp8_block_scale_forward(args)
        return self._leave(x, y, num_tokens)
