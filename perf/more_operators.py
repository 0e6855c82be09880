"""What stands between the residual stream and the routed experts, measured:
the cases, their inputs, their plain form and their definition in 64 bits.

Operators ("op" of a case):
  route       logits to expert ids and route weights: softmax or sigmoid
              scores, a bias that only the choice sees, groups of experts,
              top-k, renormalised weights
  route_grad  the logits' gradient from the route weights', and the bias's
              step towards an even load
  norm        a block's exit and the next one's entry in one pass: norm of the
              branch, gate, residual scale, norm of the stream, optionally
              quantised to E4M3 with one scale per token and 128 columns
  norm_grad   its gradient: branch, stream, gate and both norms' weights

A batch may be padded: only the first "live" rows count.  Padding tokens get
no expert (id -1, weight 0) and no gradient; padding rows of the norms stay as
they are (zero here).
"""

import math

import torch

own = False

EPS = 1e-6
RATE = 1e-3       # the balance bias's step
SCALE = 2.5       # the routed experts' scale
GROUP = 128       # columns that share an E4M3 scale
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decoding step of eight sequences: sigmoid scores, balanced by a bias, half of the groups
        {"name": "route decode", "op": "route", "tokens": 8, "live": 8, "experts": 288, "groups": 8, "keep": 4, "pair": True,
         "top_k": 8, "score": "sigmoid", "bias": True, "renorm": True, "dtype": "fp32"},
        # a prompt of 8192 tokens, the last ones padding
        {"name": "route prefill", "op": "route", "tokens": 8192, "live": 8000, "experts": 512, "groups": 8, "keep": 4, "pair": True,
         "top_k": 10, "score": "sigmoid", "bias": True, "renorm": True, "dtype": "fp32"},
        # a training batch's router in 16 bits without groups: softmax probabilities as weights
        {"name": "route batch", "op": "route", "tokens": 65536, "live": 65536, "experts": 257, "groups": 1, "keep": 1, "pair": False,
         "top_k": 9, "score": "softmax", "bias": False, "renorm": False, "dtype": "bf16"},
        # the gradients of such routers: a few chosen logits a token, or a dense row
        {"name": "route_grad chosen", "op": "route_grad", "tokens": 8192, "live": 8000, "experts": 512, "top_k": 10, "score": "sigmoid",
         "renorm": True, "dtype": "fp32"},
        {"name": "route_grad dense", "op": "route_grad", "tokens": 65536, "live": 65536, "experts": 257, "top_k": 9, "score": "softmax",
         "renorm": False, "dtype": "bf16"},
        # one decoded token between two blocks: both norms, residual, the experts' FP8 input beside the router's 16-bit one
        {"name": "norm decode", "op": "norm", "rows": 1, "live": 1, "width": 7168, "dtype": "bf16", "stream": "same", "weights": "same",
         "post": True, "residual": 1.0, "gate": "none", "pre": True, "fp8": "fp32"},
        # a small model with sizes that fill no tile: a gate for each token, a residual scale, no norm of the branch
        {"name": "norm odd", "op": "norm", "rows": 517, "live": 500, "width": 1160, "dtype": "fp16", "stream": "same", "weights": "fp32",
         "post": False, "residual": 0.5, "gate": "token", "pre": True, "fp8": "none"},
        # a training batch: the stream in 32 bits, a learned scale for each channel
        {"name": "norm batch", "op": "norm", "rows": 8192, "live": 8192, "width": 4096, "dtype": "bf16", "stream": "fp32", "weights": "fp32",
         "post": True, "residual": 1.0, "gate": "channel", "pre": True, "fp8": "none"},
        # a large prompt: the experts' input with power-of-two scales
        {"name": "norm prompt", "op": "norm", "rows": 16384, "live": 16384, "width": 7168, "dtype": "bf16", "stream": "same", "weights": "same",
         "post": False, "residual": 1.0, "gate": "none", "pre": True, "fp8": "ue8m0"},
        # a late pipeline micro-batch of a few rows
        {"name": "norm_grad few", "op": "norm_grad", "rows": 64, "live": 64, "width": 4096, "dtype": "bf16", "stream": "same", "weights": "fp32",
         "post": True, "residual": 1.0, "gate": "none", "pre": True},
        # the training batch's gradients, with the channel scales', and with a gate for every element
        {"name": "norm_grad batch", "op": "norm_grad", "rows": 8192, "live": 8192, "width": 4096, "dtype": "bf16", "stream": "fp32",
         "weights": "fp32", "post": True, "residual": 1.0, "gate": "channel", "pre": True},
        {"name": "norm_grad wide", "op": "norm_grad", "rows": 16384, "live": 16384, "width": 7168, "dtype": "bf16", "stream": "same",
         "weights": "same", "post": True, "residual": 1.0, "gate": "full", "pre": True},
    ]


def _log(rng, lo, hi, mult=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(mult, int(round(v / mult)) * mult)


def _live(rng, n):
    return n if rng.random() < 0.6 else rng.randint(1, n)


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "norm", "norm", "norm_grad", "norm_grad"])
    if op in ("route", "route_grad"):
        M = _log(rng, 1, 65536)
        groups = rng.choice([1, 1, 2, 3, 4, 8, 12]) if op == "route" else 1
        size = max(2, _log(rng, 8, 768) // groups)
        E = groups * size
        while M * E > 65536 * 257:
            M = max(1, M // 2)
        keep = rng.randint(1, groups)
        c = {"op": op, "tokens": M, "live": _live(rng, M), "experts": E, "top_k": rng.randint(1, min(12, keep * size)),
             "score": rng.choice(["sigmoid", "softmax"]), "renorm": rng.random() < 0.6, "dtype": rng.choice(["fp32", "fp32", "bf16", "fp16"])}
        if op == "route":
            c.update(groups=groups, keep=keep, pair=groups > 1 and rng.random() < 0.6, bias=rng.random() < 0.6)
        return c
    fp8 = rng.choice(["none", "none", "fp32", "ue8m0"]) if op == "norm" else "none"
    H = _log(rng, 128, 8192, 128 if fp8 != "none" else 8)
    M = _log(rng, 1, 65536)
    while M * H > 8192 * 4096:
        M = max(1, M // 2)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    c = {"op": op, "rows": M, "live": _live(rng, M), "width": H, "dtype": dtype, "stream": rng.choice(["same", "fp32"]),
         "weights": rng.choice(["same", "fp32"]), "post": rng.random() < 0.5, "residual": rng.choice([0.0, 1.0, 1.0, 0.5]),
         "gate": rng.choice(["none", "none", "channel", "token", "full"]), "pre": True}
    if op == "norm":
        c["fp8"] = fp8
        c["pre"] = fp8 != "none" or not c["post"] or rng.random() < 0.8
    elif c["post"]:
        c["pre"] = rng.random() < 0.8
    return c


def _gate_count(c):
    return {"none": 0, "channel": c["width"], "token": c["live"], "full": c["live"] * c["width"]}[c["gate"]]


def work(c):
    if c["op"] == "route":
        n, e = c["live"], 4 if c["dtype"] == "fp32" else 2
        return {"bytes": n * c["experts"] * e + c["tokens"] * c["top_k"] * 8 + (4 * c["experts"] if c["bias"] else 0),
                "flops": 5 * n * c["experts"]}
    if c["op"] == "route_grad":
        n, k, E, e = c["live"], c["top_k"], c["experts"], 4 if c["dtype"] == "fp32" else 2
        read = E if c["score"] == "softmax" and not c["renorm"] else k
        return {"bytes": n * read * e + c["tokens"] * E * e + n * k * 8 + 12 * E, "flops": 5 * n * read}
    n = c["live"] * c["width"]
    b = 4 if c["dtype"] == "fp32" else 2
    s = 4 if c["stream"] == "fp32" else b
    w = (4 if c["weights"] == "fp32" else b) * c["width"]
    gate = _gate_count(c) * {"none": 0, "channel": w // c["width"], "token": 4, "full": b}[c["gate"]]
    norms = w * (int(c["post"]) + int(c["pre"]))
    if c["op"] == "norm":
        codes = n + n // GROUP * 4 if c["fp8"] != "none" else 0
        return {"bytes": n * (b + s * (2 if c["residual"] else 1) + (b if c["pre"] else 0)) + gate + norms + codes, "flops": 12 * n}
    reads = b + (s + b if c["pre"] else 0) + s
    gates = gate + _gate_count(c) * (b if c["gate"] == "full" else 4)
    return {"bytes": n * (reads + b + (s if c["residual"] else 0)) + gates + norms + 4 * c["width"] * (int(c["post"]) + int(c["pre"])),
            "flops": 24 * n}


# ------------------------------------------------------------------ inputs

def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(*shape, device="cuda", dtype=dtype).normal_(mean, std, generator=g)

    def zeros(*shape, dtype=torch.float32):
        return torch.zeros(*shape, device="cuda", dtype=dtype)

    st = {"c": c}
    if c["op"] in ("route", "route_grad"):
        M, E, k = c["tokens"], c["experts"], c["top_k"]
        # experts differ in popularity; a bias has begun to even it out
        popular = normal(E, std=0.5)
        logits = normal(M, E) + popular
        logits += -2.0 if c["score"] == "sigmoid" else 0.0
        st["logits"] = logits.to(DTYPES[c["dtype"]])
        st["live"] = torch.full((1,), c["live"], dtype=torch.int32, device="cuda")
        if c["op"] == "route":
            size = 0.1 if c["score"] == "sigmoid" else 1.0 / E
            st["bias"] = -size * popular + normal(E, std=0.2 * size) if c["bias"] else None
            st["ids"], st["weights"] = zeros(M, k, dtype=torch.int32), zeros(M, k)
            return st
        st["ids"] = st["logits"].float().topk(k, dim=1).indices.to(torch.int32)
        st["ids"][c["live"]:] = -1
        st["dweights"], st["dlogits"] = normal(M, k, std=0.1), torch.empty_like(st["logits"])
        flat = st["ids"].reshape(-1).long()
        st["load"] = torch.bincount(flat[flat >= 0], minlength=E).to(torch.int32)
        st["bias"], st["new_bias"] = normal(E, std=0.05), zeros(E)
        return st
    M, H, n = c["rows"], c["width"], c["live"]
    branch = DTYPES[c["dtype"]]
    stream = torch.float32 if c["stream"] == "fp32" else branch
    weights = torch.float32 if c["weights"] == "fp32" else branch
    st["live"] = torch.full((1,), n, dtype=torch.int32, device="cuda")
    st["y"] = normal(M, H, std=0.3, dtype=branch)
    st["w_post"] = normal(H, std=0.1, mean=0.5, dtype=weights) if c["post"] else None
    st["w_pre"] = normal(H, std=0.2, mean=1.0, dtype=weights) if c["pre"] else None
    st["gate"] = {"none": lambda: None, "channel": lambda: normal(H, std=0.1, mean=0.3, dtype=weights),
                  "token": lambda: torch.sigmoid(normal(M, 1)), "full": lambda: normal(M, H, std=0.5, dtype=branch)}[c["gate"]]()
    if c["op"] == "norm":
        st["r"] = normal(M, H, std=2.0, dtype=stream) if c["residual"] else None
        st["h"] = zeros(M, H, dtype=stream)
        st["z"] = zeros(M, H, dtype=branch) if c["pre"] else None
        if c["fp8"] != "none":
            st["q"], st["q_scale"] = zeros(M, H, dtype=torch.float8_e4m3fn), zeros(M, H // GROUP)
        return st
    # the stream as the forward pass left it (its gradient takes it as given)
    st["h"] = normal(M, H, std=2.0, dtype=stream) if c["pre"] else None
    st["dz"] = normal(M, H, std=0.01, dtype=branch) if c["pre"] else None
    st["dh"] = normal(M, H, std=0.01, dtype=stream)
    st["dy"] = zeros(M, H, dtype=branch)
    st["dr"] = zeros(M, H, dtype=stream) if c["residual"] else None
    st["dw_pre"] = zeros(H) if c["pre"] else None
    st["dw_post"] = zeros(H) if c["post"] else None
    st["dgate"] = {"none": lambda: None, "channel": lambda: zeros(H), "token": lambda: zeros(M, 1),
                   "full": lambda: zeros(M, H, dtype=branch)}[c["gate"]]()
    return st


# ------------------------------------------------------------------ plain form

def _probabilities(c, l):
    return torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)


def _plain_route(c, st):
    M, E, n, k = c["tokens"], c["experts"], c["live"], c["top_k"]
    logits = st["logits"][:n]
    if not c["bias"] and not c["pair"]:
        choice = logits                                        # the scores rise with the logits
    else:
        choice = _probabilities(c, logits.double())            # neighbours are told apart in 64 bits
        choice = choice + st["bias"].double() if c["bias"] else choice
    if c["groups"] > 1:
        by_group = choice.reshape(n, c["groups"], -1)
        best = by_group.sort(dim=2, descending=True).values[:, :, :2].sum(2) if c["pair"] else by_group.amax(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        out = torch.ones(n, c["groups"], dtype=torch.bool, device="cuda").scatter_(1, kept, False)
        choice = choice.masked_fill(out.repeat_interleave(E // c["groups"], 1), -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = _probabilities(c, logits.float()).gather(1, ids)
    w = w / w.sum(1, keepdim=True) if c["renorm"] else w
    st["ids"].fill_(-1)
    st["weights"].zero_()
    st["ids"][:n] = ids.to(torch.int32)
    st["weights"][:n] = w * SCALE
    return {"ids": st["ids"], "weights": st["weights"]}


def _plain_route_grad(c, st):
    n = c["live"]
    logits, ids, dw = st["logits"][:n].float(), st["ids"][:n].long(), st["dweights"][:n] * SCALE
    s = _probabilities(c, logits)
    p = s.gather(1, ids)
    if c["renorm"]:
        total = p.sum(1, keepdim=True)
        dw = (dw - (dw * p).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, ids, dw)
    if c["score"] == "sigmoid":
        dl = ds * s * (1.0 - s)
    else:
        dl = s * (ds - (dw * p).sum(1, keepdim=True))
    st["dlogits"][n:] = 0
    st["dlogits"][:n] = dl.to(st["dlogits"].dtype)
    load = st["load"].float()
    st["new_bias"].copy_(st["bias"] + RATE * torch.sign(load.sum() - load * c["experts"]))
    return {"dlogits": st["dlogits"], "bias": st["new_bias"]}


def _gate(c, st, n):
    if c["gate"] == "none":
        return 1.0
    return st["gate"].float() if c["gate"] == "channel" else st["gate"][:n].float()


def _inverse_rms(x):
    return torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)


def _power_of_two(s):
    """The smallest power of two that is not below s."""
    m, e = torch.frexp(s)
    return torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))


def _plain_norm(c, st):
    n = c["live"]
    u = st["y"][:n].float()
    if c["post"]:
        u = u * _inverse_rms(u) * st["w_post"].float()
    h = u * _gate(c, st, n)
    if c["residual"]:
        h = h + c["residual"] * st["r"][:n].float()
    st["h"][:n] = h.to(st["h"].dtype)
    got = {"h": st["h"]}
    if c["pre"]:
        z = h * _inverse_rms(h) * st["w_pre"].float()
        st["z"][:n] = z.to(st["z"].dtype)
        got["z"] = st["z"]
    if c["fp8"] != "none":
        blocks = z.reshape(n, -1, GROUP)
        scale = blocks.abs().amax(2) / 448.0
        scale = _power_of_two(scale) if c["fp8"] == "ue8m0" else scale
        safe = torch.where(scale > 0, scale, torch.ones_like(scale))
        st["q"][:n] = (blocks / safe[:, :, None]).clamp(-448.0, 448.0).reshape(n, -1).to(torch.float8_e4m3fn)
        st["q_scale"][:n] = scale
        got["q"], got["q_scale"] = st["q"], st["q_scale"]
    return got


def _plain_norm_grad(c, st):
    n, H = c["live"], c["width"]
    dh = st["dh"][:n].float()
    got = {}
    if c["pre"]:
        h, dz = st["h"][:n].float(), st["dz"][:n].float()
        inv = _inverse_rms(h)
        st["dw_pre"].copy_((dz * h * inv).sum(0))
        got["dw_pre"] = st["dw_pre"]
        dz = dz * st["w_pre"].float()
        dh = dh + inv * dz - h * (inv.pow(3) * (dz * h).mean(1, keepdim=True))
    y = st["y"][:n].float()
    u = y
    if c["post"]:
        inv = _inverse_rms(y)
        u = y * inv * st["w_post"].float()
    du = dh * _gate(c, st, n)
    if c["gate"] != "none":
        dg = dh * u
        if c["gate"] == "channel":
            st["dgate"].copy_(dg.sum(0))
        elif c["gate"] == "token":
            st["dgate"][:n] = dg.sum(1, keepdim=True)
        else:
            st["dgate"][:n] = dg.to(st["dgate"].dtype)
        got["dgate"] = st["dgate"]
    if c["post"]:
        st["dw_post"].copy_((du * y * inv).sum(0))
        got["dw_post"] = st["dw_post"]
        du = du * st["w_post"].float()
        du = inv * du - y * (inv.pow(3) * (du * y).mean(1, keepdim=True))
    st["dy"][:n] = du.to(st["dy"].dtype)
    got["dy"] = st["dy"]
    if c["residual"]:
        st["dr"][:n] = (c["residual"] * dh).to(st["dr"].dtype)
        got["dr"] = st["dr"]
    return got


# ------------------------------------------------------------------ the framework's operators

def _handle(st):
    """The argument records that a user's program fills once and keeps beside its buffers."""
    import fp8_block_scale_gb300 as moe
    c = st["c"]
    if c["op"] in ("route", "route_grad"):
        score = moe.SCORE_SIGMOID if c["score"] == "sigmoid" else moe.SCORE_SOFTMAX
        how = {"score": score, "renormalize": c["renorm"], "routed_scale": SCALE, "num_tokens": st["live"]}
        if c["op"] == "route":
            args = moe.make_route_scores_args(st["logits"], st["ids"], st["weights"], bias=st["bias"], groups=c["groups"],
                                              topk_groups=c["keep"], group_score=moe.GROUP_TOP2 if c["pair"] else moe.GROUP_MAX, **how)
            return lambda: moe.moe_route_scores(args)
        args = moe.make_route_scores_backward_args(st["logits"], st["ids"], st["dweights"], st["dlogits"], **how)

        def both():
            moe.moe_route_scores_backward(args)
            moe.moe_route_balance(st["load"], st["bias"], RATE, out=st["new_bias"])
        return both
    how = {"w_post": st["w_post"], "w_pre": st["w_pre"], "gate": st["gate"], "post_norm": c["post"],
           "residual_scale": c["residual"] if c["residual"] else 1.0, "eps": EPS, "num_rows": st["live"]}
    if c["op"] == "norm":
        codes = {} if c["fp8"] == "none" else {
            "q": st["q"], "q_scale": st["q_scale"], "scale_mode": moe.SCALES_UE8M0 if c["fp8"] == "ue8m0" else moe.SCALES_FP32}
        args = moe.make_norm_residual_args(st["y"], r=st["r"], h=st["h"], z=st["z"], **how, **codes)
        return lambda: moe.moe_norm_residual(args)
    workspace = torch.empty(moe.moe_norm_residual_workspace_size(c["rows"], c["width"]), dtype=torch.uint8, device="cuda")
    args = moe.make_norm_residual_backward_args(st["y"], dh=st["dh"], h=st["h"], dz=st["dz"], dy=st["dy"], dr=st["dr"], dw_pre=st["dw_pre"],
                                                dw_post=st["dw_post"], dgate=st["dgate"], workspace=workspace, **how)
    return lambda: moe.moe_norm_residual_backward(args)


def run(st):
    c = st["c"]
    if not own:
        return {"route": _plain_route, "route_grad": _plain_route_grad, "norm": _plain_norm, "norm_grad": _plain_norm_grad}[c["op"]](c, st)
    if "call" not in st:
        st["call"] = _handle(st)
    st["call"]()
    if c["op"] == "route":
        return {"ids": st["ids"], "weights": st["weights"]}
    if c["op"] == "route_grad":
        return {"dlogits": st["dlogits"], "bias": st["new_bias"]}
    names = ("h", "z", "q", "q_scale") if c["op"] == "norm" else ("dw_pre", "dgate", "dw_post", "dy", "dr")
    return {k: st[k] for k in names if st.get(k) is not None}


# ------------------------------------------------------------------ in 64 bits

def _exact_scores(c, l):
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _exact_route(c, st):
    M, E, n, k = c["tokens"], c["experts"], c["live"], c["top_k"]
    w = torch.zeros(M, k, dtype=torch.float64, device="cuda")
    l = st["logits"][:n].double()
    s = _exact_scores(c, l)
    # without a bias the order is the logits' own
    v = s + st["bias"].double() if c["bias"] else l
    if c["groups"] > 1:
        per = E // c["groups"]
        of = (s if c["pair"] and not c["bias"] else v).view(n, c["groups"], per)
        first = of.max(2)
        mark = first.values
        if c["pair"]:
            rest = of.clone().scatter_(2, first.indices.unsqueeze(2), -math.inf)
            mark = mark + rest.max(2).values
        left = mark.clone()
        for _ in range(c["groups"] - c["keep"]):               # the weakest group goes, of equals the last
            low = c["groups"] - 1 - left.flip(1).min(1).indices
            left.scatter_(1, low.unsqueeze(1), math.inf)
            v = v.masked_fill((torch.arange(E, device="cuda") // per) == low.unsqueeze(1), -math.inf)
    for j in range(k):
        best = v.max(1, keepdim=True)
        at = (v == best.values).int().argmax(1, keepdim=True)  # of equals the first
        w[:n, j] = s.gather(1, at)[:, 0]
        v = v.scatter(1, at, -math.inf)
    if c["renorm"]:
        w[:n] /= w[:n].sum(1, keepdim=True)
    return {"ids": None, "weights": w * SCALE}


def _exact_route_grad(c, st):
    M, E, n = c["tokens"], c["experts"], c["live"]
    l, ids = st["logits"][:n].double(), st["ids"][:n].long()
    s = _exact_scores(c, l)
    dw = SCALE * st["dweights"][:n].double()
    chosen = s.gather(1, ids)
    dl = torch.zeros(M, E, dtype=torch.float64, device="cuda")
    if c["renorm"]:
        share = chosen / chosen.sum(1, keepdim=True)
        part = share * (dw - torch.einsum("mk,mk->m", dw, share).unsqueeze(1))
        if c["score"] == "sigmoid":
            part = part / (1 + torch.exp(l.gather(1, ids)))
        dl[:n].scatter_(1, ids, part)
    elif c["score"] == "sigmoid":
        dl[:n].scatter_(1, ids, dw * chosen / (1 + torch.exp(l.gather(1, ids))))
    else:
        dl[:n] = -s * torch.einsum("mk,mk->m", dw, chosen).unsqueeze(1)
        dl[:n].scatter_add_(1, ids, dw * chosen)
    load = st["load"].to(torch.int64)
    return {"dlogits": dl, "bias": st["bias"].double() + RATE * torch.sign(load.sum() - load * E).double()}


def _rows64(M, n, v):
    out = torch.zeros(M, *v.shape[1:], dtype=torch.float64, device="cuda")
    out[:n] = v
    return out


def _exact_gate(c, st, n):
    if c["gate"] == "none":
        return None
    return st["gate"].double() if c["gate"] == "channel" else st["gate"][:n].double()


def _exact_codes(v, powers):
    """Values of the E4M3 codes and the scales of rows in blocks of GROUP columns, to nearest, ties to even."""
    b = v.reshape(v.shape[0], -1, GROUP)
    scale = b.abs().max(2).values / 448
    if powers:
        scale = torch.where(scale > 0, torch.exp2(torch.ceil(torch.log2(scale.clamp(min=1e-300)))), scale)
    scale = scale.float().double()                             # the scale is held in 32 bits
    y = torch.where(scale > 0, 1 / torch.where(scale > 0, scale, 1.0), 0.0).unsqueeze(2) * b
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return ((y / step).round() * step).clamp(-448, 448).reshape(v.shape), scale


def _exact_norm(c, st):
    M, H, n = c["rows"], c["width"], c["live"]
    h = st["y"][:n].double()
    if c["post"]:
        h = h / torch.sqrt((h * h).sum(1, keepdim=True) / H + EPS) * st["w_post"].double()
    g = _exact_gate(c, st, n)
    h = h if g is None else h * g
    if c["residual"]:
        h = h + c["residual"] * st["r"][:n].double()
    got = {"h": _rows64(M, n, h)}
    if c["pre"]:
        z = h / torch.sqrt((h * h).sum(1, keepdim=True) / H + EPS) * st["w_pre"].double()
        got["z"] = _rows64(M, n, z)
        if c["fp8"] != "none":
            q, scale = _exact_codes(z, c["fp8"] == "ue8m0")
            got["q"], got["q_scale"] = _rows64(M, n, q), _rows64(M, n, scale)
    return got


def _exact_norm_grad(c, st):
    M, H, n = c["rows"], c["width"], c["live"]

    def through(x, w, d):
        """Gradients of x / rms(x) * w by x and w."""
        rms = torch.sqrt((x * x).sum(1, keepdim=True) / H + EPS)
        unit = x / rms
        dw = torch.einsum("mh,mh->h", d, unit)
        d = d * w
        return (d - unit * (d * unit).sum(1, keepdim=True) / H) / rms, dw

    total = st["dh"][:n].double()
    got = {}
    if c["pre"]:
        d, got["dw_pre"] = through(st["h"][:n].double(), st["w_pre"].double(), st["dz"][:n].double())
        total = total + d
    y = st["y"][:n].double()
    g = _exact_gate(c, st, n)
    d = total if g is None else total * g
    if g is not None:
        u = y / torch.sqrt((y * y).sum(1, keepdim=True) / H + EPS) * st["w_post"].double() if c["post"] else y
        dg = total * u
        got["dgate"] = {"channel": lambda: dg.sum(0), "token": lambda: _rows64(M, n, dg.sum(1, keepdim=True)),
                        "full": lambda: _rows64(M, n, dg)}[c["gate"]]()
    if c["post"]:
        d, got["dw_post"] = through(y, st["w_post"].double(), d)
    got["dy"] = _rows64(M, n, d)
    if c["residual"]:
        got["dr"] = _rows64(M, n, c["residual"] * total)
    return got


def exact(c, seed):
    st = prepare(c, seed)
    return {"route": _exact_route, "route_grad": _exact_route_grad, "norm": _exact_norm, "norm_grad": _exact_norm_grad}[c["op"]](c, st)
