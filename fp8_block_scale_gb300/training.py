"""One routed expert layer in training, on the library's kernels.

``ExpertLayer`` holds the layer's buffers and strings the operators of
include/moe_train.h together as a training step uses them:

  route     moe_route_topk -> moe_plan -> moe_plan_groups
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
"""

import torch

from . import _lib as L


class ExpertLayer:
    """A routed expert layer of E experts, hidden size H, intermediate size I.

    tokens: the batch's token count (the buffers' size).  Weights are kept in
    FP32 with a copy in `dtype` that the products read; states in 32 or 8 bits.
    """

    def __init__(self, tokens, H, I, E, top_k, block_m=16, dtype=torch.bfloat16, state_bits=32, weight_decay=0.0,
                 device="cuda", generator=None):
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

    def route(self, logits):
        """Router, plan and groups from logits [tokens, E] (contiguous, float32 or bfloat16)."""
        self._batch("logits", logits, self.E, (torch.float32, torch.bfloat16))
        if not logits.is_contiguous():
            raise ValueError("logits: a contiguous tensor is expected")
        self._forward_done = False
        L.moe_route_topk(logits, self.top_k, self.topk_ids, self.topk_weights)
        L.moe_plan(self.topk_ids, self.E, self.block_m, self.sorted_ids, self.expert_ids, self.num_padded,
                   self.plan_workspace)
        L.moe_plan_groups(self.sorted_ids, self.expert_ids, self.num_padded, self.block_m, self.M * self.top_k,
                          self.group_start, self.group_rows, self.route_slot)

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

    def quantized(self):
        """The trained weights as the FP8 forward takes them: (w13 interleaved,
        w13_scale, w2, w2_scale).  H, I multiples of 128; BF16 weights, ValueError for others."""
        out = []
        for w in self.models:
            E, rows, cols = w.shape
            q = torch.empty(E, rows, cols, dtype=torch.uint8, device=w.device)
            s = torch.empty(E, rows // 128, cols // 128, dtype=torch.float32, device=w.device)
            L.moe_quantize_weight_128x128(w, q, s)
            out.append((q, s))
        w13 = torch.empty_like(out[0][0])
        L.moe_prep_weights(out[0][0], w13)
        return w13, out[0][1], out[1][0], out[1][1]
