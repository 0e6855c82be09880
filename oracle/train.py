"""Float64 reference of the training side of the routed experts: the grouped
products and their gradients, the SwiGLU gradient, dispatch and combine, and
the AdamW step with FP32 or 8-bit states.

Written from the formulas, in numpy, one group or token at a time.  Beside
each product stands the sum of its terms' magnitudes, from which the tests
derive how far a 32-bit sum may be off.
"""

import numpy as np

GROUP = 128        # elements per scale of the 8-bit states
E4M3_MAX = 448.0


def spans(start, rows):
    """(expert, slots) of every non-empty group."""
    return [(e, np.arange(int(a), int(a) + int(n))) for e, (a, n) in enumerate(zip(start, rows)) if n > 0]


def grouped_forward(x, w, start, rows):
    """y[s] = w[e] x[s] and the sums of |terms|; NaN outside the groups."""
    y = np.full((x.shape[0], w.shape[1]), np.nan)
    mag = np.full_like(y, np.nan)
    for e, s in spans(start, rows):
        y[s] = x[s] @ w[e].T
        mag[s] = np.abs(x[s]) @ np.abs(w[e]).T
    return y, mag


def grouped_input_gradient(dy, w, start, rows):
    dx = np.full((dy.shape[0], w.shape[2]), np.nan)
    mag = np.full_like(dx, np.nan)
    for e, s in spans(start, rows):
        dx[s] = dy[s] @ w[e]
        mag[s] = np.abs(dy[s]) @ np.abs(w[e])
    return dx, mag


def grouped_wgrad(dy, x, start, rows):
    E = len(start)
    dw = np.zeros((E, dy.shape[1], x.shape[1]))
    mag = np.zeros_like(dw)
    for e, s in spans(start, rows):
        dw[e] = dy[s].T @ x[s]
        mag[e] = np.abs(dy[s]).T @ np.abs(x[s])
    return dw, mag


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def swiglu(pre, weight):
    """silu(gate) * up * weight, pre = [rows, gate | up]."""
    I = pre.shape[1] // 2
    g, u = pre[:, :I], pre[:, I:]
    return g * sigmoid(g) * u * weight[:, None]


def swiglu_backward(dh, pre, weight):
    """(dpre, h, dweight) by rows."""
    I = dh.shape[1]
    g, u = pre[:, :I], pre[:, I:]
    s = sigmoid(g)
    wt = weight[:, None]
    dg = dh * wt * u * s * (1.0 + g * (1.0 - s))
    du = dh * wt * g * s
    return np.concatenate([dg, du], axis=1), g * s * u * wt, (dh * g * s * u).sum(1)


def plan_groups(topk_ids, E, sorted_ids, block_m, P):
    """Starts, counts and route slots of a plan, by counting."""
    R = topk_ids.size
    slot = np.full(R, -1, np.int64)
    for s in range(P):
        if sorted_ids[s] < R:
            slot[sorted_ids[s]] = s
    flat = topk_ids.reshape(-1)
    rows = np.array([int((flat == e).sum()) for e in range(E)])
    start = np.array([int(slot[flat == e].min()) if rows[e] else 0 for e in range(E)])
    return start, rows, slot


# ------------------------------------------------------------------ AdamW

def adamw(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step):
    """(p, m, v, root of v, size of the update) after one step, float64."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    root = np.sqrt(v)
    upd = lr * (m / (1 - beta1 ** step)) / (root / np.sqrt(1 - beta2 ** step) + eps)
    return p * (1 - lr * weight_decay) - upd, m, v, root, np.abs(upd)


def group_max(x):
    b = np.zeros(-(-x.size // GROUP) * GROUP)
    b[: x.size] = np.abs(x)
    return b.reshape(-1, GROUP).max(1)


def per_element(scale, n):
    return np.repeat(scale, GROUP)[:n]


def e4m3_spacing(y):
    """Distance between neighbouring E4M3 values around y >= 0."""
    return np.exp2(np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)


def e4m3_nearest(y):
    """E4M3 value nearest to y (ties to even, saturated)."""
    a = np.abs(y)
    st = e4m3_spacing(a)
    return np.sign(y) * np.minimum(np.round(a / st) * st, E4M3_MAX)


def e4m3_random(y, u20):
    """Nonnegative y rounded up with probability (part cut off) / spacing, by
    u20 in [0, 2^20); no positive y below the smallest code."""
    a = np.where(y > 0, np.maximum(y, 2.0 ** -9), 0.0)
    st = e4m3_spacing(a)
    return np.minimum(np.floor(a / st + u20 / 2.0 ** 20) * st, E4M3_MAX)


def hash20(seed, tensor, n, first=0):
    """The twenty random bits of elements first .. first + n - 1 of a tensor.  The
    mixer is C. Wellons' published one ("Prospecting for Hash Functions", 2018)."""
    M = (1 << 32) - 1
    key = (seed + 0x9E3779B9 * (tensor + 1)) & M
    out = np.empty(n, np.int64)
    for k in range(n):
        i = first + k
        x = ((i & M) * 0x9E3779B1 + (i >> 32) * 0x85EBCA77 + key) & M
        x = ((x ^ (x >> 16)) * 0x7FEB352D) & M
        x = ((x ^ (x >> 15)) * 0x846CA68B) & M
        out[k] = (x ^ (x >> 16)) >> 12
    return out
