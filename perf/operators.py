"""The operators of a training step of routed experts, measured: their cases,
their inputs, their plain form and their definition in 64 bits.

Rows are held in plan order: every expert's routes are contiguous slots, padded
to a multiple of BLOCK_M slots, as the routing plan lays them out.  Slots that
hold no route stay zero in every output.

Operators ("op" of a case):
  forward   y = x w^T per expert, optionally with the SwiGLU epilogue
  dgrad     the product's gradient by its input, dx = dy w per expert
  wgrad     its gradient by the weights, dw = dy^T x per expert
  swiglu    the gradient of h = silu(gate) * up * route weight
  gather    token rows into plan order
  sum       route rows summed per token
  adamw     one AdamW step over many tensors, states in 32 or in 8 bits
"""

import math

import numpy as np
import torch

own = False

BLOCK_M = 16      # the plan's row padding
ADAM = {"lr": 1e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1, "step": 100, "seed": 20240}
GROUP = 128       # elements that share a scale of the 8-bit states
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decoding model through its experts' gate/up product: latency and the weights' bytes
        {"name": "forward decode", "op": "forward", "tokens": 1, "experts": 257, "top_k": 9, "inner": 7168, "outer": 512,
         "swiglu": True, "skew": 0.0, "dtype": "bf16"},
        # a training batch of 8192 tokens: the gate/up product with its activation, the pre-activations kept
        {"name": "forward 8192", "op": "forward", "tokens": 8192, "experts": 288, "top_k": 8, "inner": 4096, "outer": 2048,
         "swiglu": True, "skew": 0.0, "dtype": "bf16"},
        # a small model with sizes that fill no tile, in the other 16-bit type, as in a unit of an ablation
        {"name": "forward odd", "op": "forward", "tokens": 517, "experts": 24, "top_k": 3, "inner": 1160, "outer": 712,
         "swiglu": False, "skew": 0.5, "dtype": "fp16"},
        # the down projection's input gradient under uneven routing
        {"name": "dgrad skewed", "op": "dgrad", "tokens": 4096, "experts": 512, "top_k": 10, "inner": 512, "outer": 4096,
         "skew": 1.0, "dtype": "bf16"},
        # the gate/up weights' gradient of a training batch: the largest output
        {"name": "wgrad 8192", "op": "wgrad", "tokens": 8192, "experts": 288, "top_k": 8, "inner": 4096, "outer": 2048,
         "skew": 0.0, "dtype": "bf16"},
        # the activation's gradient for a few rows (a late pipeline micro-batch) and for a whole batch
        {"name": "swiglu 64", "op": "swiglu", "tokens": 64, "experts": 257, "top_k": 9, "width": 256, "dtype": "bf16"},
        {"name": "swiglu 8192", "op": "swiglu", "tokens": 8192, "experts": 288, "top_k": 8, "width": 1024, "dtype": "bf16"},
        # tokens on their way to the experts, and the experts' rows on their way back
        {"name": "gather 8192", "op": "gather", "tokens": 8192, "experts": 288, "top_k": 8, "width": 4096, "dtype": "bf16"},
        {"name": "sum 1000", "op": "sum", "tokens": 1000, "experts": 257, "top_k": 9, "width": 7168, "dtype": "bf16"},
        # a router and its norms: many small tensors, where launches count
        {"name": "adamw many small", "op": "adamw", "tensors": 60, "elements": 1000001, "bits": 32, "grad": "fp32"},
        # 32 experts' gate/up weights with FP32 states, then with 8-bit states
        {"name": "adamw 32 bit", "op": "adamw", "tensors": 4, "elements": 268435456, "bits": 32, "grad": "bf16"},
        {"name": "adamw 8 bit", "op": "adamw", "tensors": 4, "elements": 268435456, "bits": 8, "grad": "bf16"},
    ]


def _log(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(mult, int(round(v / mult)) * mult)


def draw(rng):
    op = rng.choice(["forward", "forward", "dgrad", "wgrad", "swiglu", "gather", "sum", "adamw", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "adamw":
        return {"op": op, "tensors": _log(rng, 1, 60), "elements": _log(rng, 20000, 200000000), "bits": rng.choice([32, 8]),
                "grad": rng.choice(["bf16", "fp32", "fp16"])}
    experts, tokens = _log(rng, 8, 512), _log(rng, 1, 8192)
    case = {"op": op, "tokens": tokens, "experts": experts, "top_k": rng.randint(1, min(10, experts)), "dtype": dtype}
    if op in ("swiglu", "gather", "sum"):
        case["width"] = _log(rng, 128, 1024 if op == "swiglu" else 7168, 8)
        return case
    # one product's size: at most that of the largest listed one
    case["inner"], case["outer"] = _log(rng, 256, 7168, 8), _log(rng, 256, 7168, 16)
    while case["inner"] * case["outer"] > 4096 * 2048:
        side = "inner" if case["inner"] > case["outer"] else "outer"
        case[side] = max(256, case[side] // 32 * 16)
    case["experts"] = experts = min(experts, 288)
    case["top_k"] = min(case["top_k"], 8)
    case["skew"] = round(rng.uniform(0.0, 1.0), 2)
    if op == "forward":
        case["swiglu"] = rng.random() < 0.5
    return case


def _active(c):
    """Experts that some token picks, expected for even routing."""
    return c["experts"] * (1.0 - (1.0 - c["top_k"] / c["experts"]) ** c["tokens"])


def work(c):
    if c["op"] == "adamw":
        n, g = c["elements"], 4 if c["grad"] == "fp32" else 2
        # gradient read; parameter, both states read and written; 16-bit copy written
        state = 16 if c["bits"] == 32 else 4 + 16 / GROUP
        return {"bytes": n * (g + 8 + state + 2), "flops": 15 * n}
    rows = c["tokens"] * c["top_k"]
    if c["op"] == "swiglu":
        return {"bytes": rows * (6 * c["width"] * 2 + 12), "flops": 15 * rows * c["width"]}
    if c["op"] in ("gather", "sum"):
        return {"bytes": (rows + c["tokens"]) * c["width"] * 2 + 4 * rows, "flops": rows * c["width"]}
    k, n = c["inner"], c["outer"]
    if c["op"] == "wgrad":
        return {"bytes": 2 * (rows * (k + n) + c["experts"] * n * k), "flops": 2 * rows * n * k}
    out = n + n // 2 if c.get("swiglu") else n
    return {"bytes": 2 * (rows * (k + out) + _active(c) * n * k), "flops": 2 * rows * n * k}


# ------------------------------------------------------------------ inputs

def _routing(c, g):
    """top_k distinct experts a token; `skew` spreads the experts' popularity (standard deviation of its logarithm)."""
    M, E, k = c["tokens"], c["experts"], c["top_k"]
    popular = torch.randn(E, device="cuda", generator=g) * float(c.get("skew", 0.0))
    u = torch.rand(M, E, device="cuda", generator=g).clamp_(1e-7, 1 - 1e-7)
    return (popular - torch.log(-torch.log(u))).topk(k, dim=1).indices      # [M, k]


def _plan(c, g):
    """The routes in plan order, and the indexes that the plain form needs."""
    M, E, k = c["tokens"], c["experts"], c["top_k"]
    ids = _routing(c, g)
    flat = ids.reshape(-1)
    R = M * k
    order = torch.sort(flat, stable=True).indices                            # routes, expert by expert
    rows = torch.bincount(flat, minlength=E)
    padded = (rows + BLOCK_M - 1) // BLOCK_M * BLOCK_M
    start = torch.cumsum(padded, 0) - padded
    first = torch.cumsum(rows, 0) - rows
    e_of = flat[order]
    j_of = torch.arange(R, device="cuda") - first[e_of]
    slot = start[e_of] + j_of                                                # slot of each sorted route
    slots = -(-(R + min(E, R) * (BLOCK_M - 1)) // BLOCK_M) * BLOCK_M
    route = torch.full((slots,), R, dtype=torch.int32, device="cuda")
    route[slot] = order.to(torch.int32)
    route_slot = torch.empty(R, dtype=torch.int32, device="cuda")
    route_slot[order] = slot.to(torch.int32)
    active = torch.nonzero(rows).reshape(-1)
    rank = torch.cumsum((rows > 0).to(torch.int64), 0) - 1
    return {"R": R, "slots": slots, "start": start.to(torch.int32), "rows": rows.to(torch.int32), "route": route,
            "route_slot": route_slot, "padded": padded.sum().to(torch.int32).reshape(1), "active": active,
            "slot": slot, "pos": (rank[e_of], j_of), "most": int(rows.max())}


def _adam_sizes(c):
    """Sizes that fall off as 1 / (i + 1), none of them round; the last takes what is left."""
    n, T = c["elements"], c["tensors"]
    total = sum(1.0 / (i + 1) for i in range(T))
    sizes = [int(n / total / (i + 1)) | 1 for i in range(T - 1)]
    return sizes + [max(1, n - sum(sizes))]


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(*shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)

    st = {"c": c}
    if c["op"] == "adamw":
        st["tensors"] = []
        for n in _adam_sizes(c):
            t = {"param": normal(n, std=0.02), "model": torch.zeros(n, dtype=torch.bfloat16, device="cuda"),
                 "grad": normal(n, std=1e-3, dtype=DTYPES[c["grad"]])}
            # states as earlier steps left them: m well below the root of v
            m, r = normal(n, std=3e-4), normal(n, std=3e-4).abs_() + 8e-4
            if c["bits"] == 32:
                t["exp_avg"], t["exp_avg_sq"] = m, r * r
            else:
                t["exp_avg"], t["exp_avg_scale"] = _encode(m)
                t["exp_avg_sq"], t["exp_avg_sq_scale"] = _encode(r)
            st["tensors"].append(t)
        return st
    p = st["plan"] = _plan(c, g)
    dt = DTYPES[c["dtype"]]

    def rows_of(width, std=1.0):
        """Rows in plan order; what stands in slots without a route must not matter: here NaN."""
        x = normal(p["slots"], width, std=std, dtype=dt)
        x[p["route"] == p["R"]] = float("nan")
        return x

    def out(*shape):
        return torch.zeros(*shape, dtype=dt, device="cuda")

    if c["op"] in ("forward", "swiglu"):
        st["weights"] = torch.softmax(normal(c["tokens"], c["top_k"]), dim=1).reshape(-1)
    if c["op"] == "swiglu":
        st["dh"], st["pre"] = rows_of(c["width"], 0.01), rows_of(2 * c["width"])
        st["dpre"], st["h"] = out(p["slots"], 2 * c["width"]), out(p["slots"], c["width"])
        st["dweights"] = torch.zeros(p["R"], device="cuda")
    elif c["op"] == "gather":
        st["x"], st["xs"] = normal(c["tokens"], c["width"], dtype=dt), out(p["slots"], c["width"])
    elif c["op"] == "sum":
        st["y"], st["out"] = rows_of(c["width"]), out(c["tokens"], c["width"])
    else:
        k, n, E = c["inner"], c["outer"], c["experts"]
        if c["op"] == "wgrad":
            st["dy"], st["x"] = rows_of(n, 0.01), rows_of(k)
            st["dw"] = out(E, n, k)
        else:
            st["w"] = normal(E, n, k, std=0.02, dtype=dt)
            if c["op"] == "dgrad":
                st["dy"], st["dx"] = rows_of(n, 0.01), out(p["slots"], k)
            else:
                st["x"], st["y"] = rows_of(k), out(p["slots"], n)
                if c["swiglu"]:
                    st["h"] = out(p["slots"], n // 2)
    return st


# ------------------------------------------------------------------ plain form

def _blocks(x):
    """[n] -> [ceil(n / GROUP), GROUP], zero-padded."""
    return torch.nn.functional.pad(x, (0, -x.numel() % GROUP)).reshape(-1, GROUP)


def _encode(x):
    """E4M3 codes to nearest with one scale, the largest magnitude / 448, per GROUP elements."""
    b = _blocks(x)
    scale = b.abs().amax(1) / 448.0
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    q = (b / safe[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.reshape(-1)[:x.numel()].clone(), scale


def _decode(q, scale):
    return q.float() * scale.repeat_interleave(GROUP)[:q.numel()]


def _random20(n, tensor):
    """Twenty bits per element: an integer mix of seed, tensor and element (products below 2^63 by halves)."""
    def mul(a, b):
        return ((a & 0xFFFF) * b + (((a >> 16) * b & 0xFFFF) << 16)) & 0xFFFFFFFF

    i = torch.arange(n, device="cuda", dtype=torch.int64)
    key = (ADAM["seed"] + 0x9E3779B9 * (tensor + 1)) & 0xFFFFFFFF
    x = (mul(i & 0xFFFFFFFF, 0x9E3779B1) + mul(i >> 32, 0x85EBCA77) + key) & 0xFFFFFFFF
    x = mul(x ^ (x >> 16), 0x7FEB352D)
    x = mul(x ^ (x >> 15), 0x846CA68B)
    return (x ^ (x >> 16)) >> 12


def _encode_random(r, tensor):
    """Nonnegative values to E4M3 codes, rounded up with the probability of the part cut off; none above zero becomes zero."""
    b = _blocks(r)
    scale = b.amax(1) / 448.0
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    y = (b / safe[:, None]).reshape(-1)[:r.numel()]
    y = torch.where(r > 0, y.clamp(2.0 ** -9, 448.0), torch.zeros_like(y))
    u = _random20(r.numel(), tensor)
    normal = ((y.view(torch.int32) + u.to(torch.int32)) & ~0xFFFFF).view(torch.float32)
    small = torch.floor(y * 512.0 + u.float() * 2.0 ** -20) / 512.0
    y = torch.where(y >= 2.0 ** -6, normal, small).clamp(max=448.0)
    y = torch.where(scale.repeat_interleave(GROUP)[:r.numel()] > 0, y, torch.zeros_like(y))
    return y.to(torch.float8_e4m3fn), scale


def _adam(t, index, c):
    b1, b2 = ADAM["beta1"], ADAM["beta2"]
    c1, c2 = 1.0 - b1 ** ADAM["step"], 1.0 - b2 ** ADAM["step"]
    g = t["grad"].float()
    if c["bits"] == 32:
        m, v = t["exp_avg"], t["exp_avg_sq"]
    else:
        m, r = _decode(t["exp_avg"], t["exp_avg_scale"]), _decode(t["exp_avg_sq"], t["exp_avg_sq_scale"])
        v = r * r
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    r = torch.sqrt(v)
    p = t["param"] * (1.0 - ADAM["lr"] * ADAM["weight_decay"])
    p = p - (m * (ADAM["lr"] / c1)) / (r * (1.0 / math.sqrt(c2)) + ADAM["eps"])
    t["param"].copy_(p)
    t["model"].copy_(p)
    if c["bits"] == 32:
        t["exp_avg"].copy_(m)
        t["exp_avg_sq"].copy_(v)
    else:
        for name, (q, s) in (("exp_avg", _encode(m)), ("exp_avg_sq", _encode_random(r, index))):
            t[name].copy_(q)
            t[name + "_scale"].copy_(s)


def _padded(x, p):
    """Rows in plan order -> [active experts, most rows, width] in 32 bits, zero where an expert has fewer."""
    out = torch.zeros(p["active"].numel(), p["most"], x.shape[1], device="cuda")
    out[p["pos"]] = x[p["slot"]].float()
    return out


def _plain(st):
    c, p = st["c"], st.get("plan")
    op = c["op"]
    if op == "adamw":
        for i, t in enumerate(st["tensors"]):
            _adam(t, i, c)
        return _adam_out(st)
    if op in ("forward", "dgrad"):
        w = st["w"][p["active"]].float()
        x = _padded(st["x" if op == "forward" else "dy"], p)
        y = torch.bmm(x, w.transpose(1, 2) if op == "forward" else w)[p["pos"]]
        if op == "dgrad":
            st["dx"][p["slot"]] = y.to(st["dx"].dtype)
            return st["dx"]
        st["y"][p["slot"]] = y.to(st["y"].dtype)
        if not c["swiglu"]:
            return st["y"]
        gate, up = y.chunk(2, dim=1)
        wt = st["weights"][p["route"][p["slot"]].long()]
        st["h"][p["slot"]] = (gate * torch.sigmoid(gate) * up * wt[:, None]).to(st["h"].dtype)
        return {"pre": st["y"], "h": st["h"]}
    if op == "wgrad":
        dw = torch.bmm(_padded(st["dy"], p).transpose(1, 2), _padded(st["x"], p))
        st["dw"].zero_()
        st["dw"][p["active"]] = dw.to(st["dw"].dtype)
        return st["dw"]
    if op == "swiglu":
        gate, up = st["pre"][p["slot"]].float().chunk(2, dim=1)
        dh = st["dh"][p["slot"]].float()
        routes = p["route"][p["slot"]].long()
        wt = st["weights"][routes][:, None]
        sig = torch.sigmoid(gate)
        h = gate * sig * up
        st["dweights"][routes] = (dh * h).sum(1)
        dgate = dh * wt * up * sig * (1.0 + gate * (1.0 - sig))
        st["dpre"][p["slot"]] = torch.cat([dgate, dh * wt * gate * sig], 1).to(st["dpre"].dtype)
        st["h"][p["slot"]] = (h * wt).to(st["h"].dtype)
        return {"dpre": st["dpre"], "h": st["h"], "dweights": st["dweights"]}
    if op == "gather":
        st["xs"][p["slot"]] = st["x"][p["route"][p["slot"]].long() // c["top_k"]]
        return st["xs"]
    y = st["y"][p["route_slot"].long()].float().reshape(c["tokens"], c["top_k"], -1)
    st["out"].copy_(y.sum(1))
    return st["out"]


def _adam_out(st):
    # the largest, a middle and the last tensor whole: parameter, 16-bit copy, states
    T = st["tensors"]
    names = [n for n in T[0] if n != "grad"]
    return {"%d.%s" % (i, n): T[i][n] for i in sorted({0, len(T) // 2, len(T) - 1}) for n in names}


# ------------------------------------------------------------------ the framework's operators

def _handle(st):
    """The argument records that a user's program fills once and keeps beside its buffers."""
    import fp8_block_scale_gb300 as moe
    c, p = st["c"], st.get("plan")
    op = c["op"]
    if op == "adamw":
        table = moe.AdamWTable(st["tensors"], weight_decay=ADAM["weight_decay"])
        hyper = {k: ADAM[k] for k in ("lr", "beta1", "beta2", "eps", "step", "seed")}
        args = moe.make_adamw_args(table, **hyper)
        return lambda: moe.moe_adamw_step(args)
    if op == "forward":
        if c["swiglu"]:
            args = moe.make_grouped_args(st["x"], st["w"], st["h"], p["start"], p["rows"], epilogue=moe.GROUPED_SWIGLU, pre=st["y"],
                                         route_ids=p["route"], route_weights=st["weights"])
        else:
            args = moe.make_grouped_args(st["x"], st["w"], st["y"], p["start"], p["rows"])
        return lambda: moe.moe_grouped_gemm(args)
    if op == "dgrad":
        args = moe.make_grouped_args(st["dy"], st["w"], st["dx"], p["start"], p["rows"], input_gradient=True)
        return lambda: moe.moe_grouped_gemm(args)
    if op == "wgrad":
        args = moe.make_grouped_wgrad_args(st["dy"], st["x"], st["dw"], p["start"], p["rows"])
        return lambda: moe.moe_grouped_wgrad(args)
    if op == "swiglu":
        args = moe.make_swiglu_backward_args(st["dh"], st["pre"], st["dpre"], h=st["h"], route_ids=p["route"], num_rows=p["padded"],
                                             route_weights=st["weights"], dweights=st["dweights"])
        return lambda: moe.moe_swiglu_backward(args)
    if op == "gather":
        return lambda: moe.moe_gather_rows(st["x"], st["xs"], p["route"], c["top_k"], p["padded"])
    return lambda: moe.moe_sum_routes(st["y"], st["out"], p["route_slot"], c["top_k"])


def run(st):
    if not own:
        return _plain(st)
    if "call" not in st:
        st["call"] = _handle(st)
    st["call"]()
    c = st["c"]
    if c["op"] == "adamw":
        return _adam_out(st)
    if c["op"] == "forward":
        return {"pre": st["y"], "h": st["h"]} if c["swiglu"] else st["y"]
    if c["op"] == "swiglu":
        return {"dpre": st["dpre"], "h": st["h"], "dweights": st["dweights"]}
    return st[{"dgrad": "dx", "wgrad": "dw", "gather": "xs", "sum": "out"}[c["op"]]]


# ------------------------------------------------------------------ in 64 bits

def _exact_codes(x, r20):
    """x [n] float64 >= 0 or signed -> values of E4M3 codes and the scales; r20 None: to nearest, ties to even."""
    n = x.numel()
    b = torch.zeros(-(-n // GROUP) * GROUP, dtype=torch.float64, device=x.device)
    b[:n] = x.abs()
    scale = (b.view(-1, GROUP).max(1).values / 448).float()      # the scale is held in 32 bits
    s = scale.double().view(-1, 1).expand(-1, GROUP).reshape(-1)[:n]
    y = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0)
    if r20 is not None:
        y = torch.where(x > 0, y.clamp(min=2.0 ** -9), 0.0)
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    q = torch.round(y / step) if r20 is None else torch.floor(y / step + r20.double() / 2 ** 20)
    q = (q * step).clamp(max=448.0) * torch.sign(x)
    return torch.where(s > 0, q, 0.0), scale.double()


def exact(c, seed):
    st = prepare(c, seed)
    op = c["op"]
    if op == "adamw":
        b1, b2, n = ADAM["beta1"], ADAM["beta2"], ADAM["step"]
        got = {}
        T = st["tensors"]
        for i in sorted({0, len(T) // 2, len(T) - 1}):
            t = T[i]
            g = t["grad"].double()
            if c["bits"] == 32:
                m, v = t["exp_avg"].double(), t["exp_avg_sq"].double()
            else:
                wide = torch.arange(g.numel(), device="cuda") // GROUP
                m = t["exp_avg"].double() * t["exp_avg_scale"].double()[wide]
                v = (t["exp_avg_sq"].double() * t["exp_avg_sq_scale"].double()[wide]) ** 2
            m = b1 * m + (1 - b1) * g
            v = b2 * v + (1 - b2) * g ** 2
            w = t["param"].double() * (1 - ADAM["lr"] * ADAM["weight_decay"])
            w = w - ADAM["lr"] * (m / (1 - b1 ** n)) / ((v / (1 - b2 ** n)).sqrt() + ADAM["eps"])
            got["%d.param" % i] = got["%d.model" % i] = w
            if c["bits"] == 32:
                got["%d.exp_avg" % i], got["%d.exp_avg_sq" % i] = m, v
            else:
                got["%d.exp_avg" % i], got["%d.exp_avg_scale" % i] = _exact_codes(m, None)
                got["%d.exp_avg_sq" % i], got["%d.exp_avg_sq_scale" % i] = _exact_codes(v.sqrt(), _random20(v.numel(), i))
        return got
    p = st["plan"]
    start, rows = p["start"].tolist(), p["rows"].tolist()
    route, R = p["route"].tolist(), p["R"]
    if op in ("forward", "dgrad", "wgrad"):
        if work(c)["flops"] > 6e12:      # the card's 64-bit rate is about a hundredth of its 32-bit one
            return None
        k, n = c["inner"], c["outer"]
        spans = [(e, slice(a, a + r)) for e, (a, r) in enumerate(zip(start, rows)) if r]
        if op == "wgrad":
            dw = torch.zeros(c["experts"], n, k, dtype=torch.float64, device="cuda")
            for e, s in spans:
                dw[e] = st["dy"][s].double().t() @ st["x"][s].double()
            return dw
        y = torch.zeros(p["slots"], n if op == "forward" else k, dtype=torch.float64, device="cuda")
        for e, s in spans:
            w = st["w"][e].double()
            y[s] = st["x"][s].double() @ w.t() if op == "forward" else st["dy"][s].double() @ w
        if op == "dgrad" or not c["swiglu"]:
            return y
        wt = torch.zeros(p["slots"], 1, dtype=torch.float64, device="cuda")
        for e, s in spans:
            wt[s, 0] = st["weights"][p["route"][s].long()].double()
        a, b = y[:, : n // 2], y[:, n // 2:]
        return {"pre": y, "h": a / (1 + torch.exp(-a)) * b * wt}
    live = np.array([s for s, r in enumerate(route) if r < R])
    ids = np.array(route)[live]
    live_t, ids_t = torch.from_numpy(live).cuda(), torch.from_numpy(ids).cuda()
    if op == "swiglu":
        I = c["width"]
        dpre = torch.zeros(p["slots"], 2 * I, dtype=torch.float64, device="cuda")
        h = torch.zeros(p["slots"], I, dtype=torch.float64, device="cuda")
        dwt = torch.zeros(R, dtype=torch.float64, device="cuda")
        a, b = st["pre"][live_t, :I].double(), st["pre"][live_t, I:].double()
        d, wt = st["dh"][live_t].double(), st["weights"][ids_t].double().unsqueeze(1)
        s = 1 / (1 + torch.exp(-a))
        dpre[live_t, :I] = d * wt * b * (s + a * s * (1 - s))
        dpre[live_t, I:] = d * wt * a * s
        h[live_t] = a * s * b * wt
        dwt[ids_t] = torch.einsum("ri,ri->r", d, a * s * b)
        return {"dpre": dpre, "h": h, "dweights": dwt}
    if op == "gather":
        xs = torch.zeros(p["slots"], c["width"], dtype=torch.float64, device="cuda")
        xs[live_t] = st["x"].double()[torch.div(ids_t, c["top_k"], rounding_mode="floor")]
        return xs
    out = torch.zeros(c["tokens"], c["width"], dtype=torch.float64, device="cuda")
    out.index_add_(0, torch.div(ids_t, c["top_k"], rounding_mode="floor"), st["y"][live_t].double())
    return out
