"""Float64 reference of what stands between the residual stream and the routed
experts: routing by scores with its gradient and the balance bias's step, and
the norms before and after a block with their gradient.

Written from the formulas, in numpy, a token at a time where choices are made.
Beside the norms' values stand sums of the magnitudes of their terms, from
which the tests derive how far 32-bit arithmetic may be off.
"""

import numpy as np

SOFTMAX, SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1


def sigmoid(l):
    e = np.exp(-np.abs(l))
    return np.where(l >= 0, 1.0, e) / (1.0 + e)


def scores(l, score):
    """Scores of one token's logits."""
    with np.errstate(invalid="ignore", over="ignore"):
        if score == SIGMOID:
            return np.where(np.isnan(l), np.nan, sigmoid(l))
        e = np.exp(l - np.max(l, initial=-np.inf, where=~np.isnan(l)))
        return e / e.sum()


def _order(values, index):
    """`index` sorted by falling value (NaN above everything), equal ones by rising index."""
    key = [(0, 0.0) if np.isnan(values[i]) else (1, -values[i]) for i in index]
    return [i for _, i in sorted(zip(key, index))]


def route_scores(logits, top_k, score=SIGMOID, bias=None, groups=1, topk_groups=1, group_score=GROUP_MAX, renormalize=True,
                 routed_scale=1.0, live=None):
    """(ids, weights) of all tokens; id -1 and weight 0 where there is no choice."""
    M, E = logits.shape
    ids, weights = np.full((M, top_k), -1, np.int64), np.zeros((M, top_k))
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    per = E // groups
    for t in range(M if live is None else min(max(live, 0), M)):
        l = logits[t]
        s = scores(l, score)
        c = s + b
        free = [e for e in range(E) if l[e] != -np.inf and b[e] != -np.inf]
        if groups > 1 and topk_groups < groups:
            by = l if bias is None and group_score == GROUP_MAX else c
            value = {}
            for g in range(groups):
                members = _order(by, [e for e in free if e // per == g])
                if members:
                    best = [by[e] for e in members[:2 if group_score == GROUP_TOP2 else 1]]
                    value[g] = np.nan if np.isnan(best).any() else sum(best)
            stay = _order(value, sorted(value))[:topk_groups]
            free = [e for e in free if e // per in stay]
        chosen = _order(l if bias is None else c, free)[:top_k]
        ids[t, :len(chosen)] = chosen
        if not chosen:
            continue
        if renormalize:
            if score == SIGMOID:      # over the largest one's exponential, so that nothing vanishes
                top = min(np.nanmax(l[chosen], initial=-np.inf), 0.0)
                w = np.exp(np.minimum(l[chosen], 0.0) - top) / (1.0 + np.exp(-np.abs(l[chosen])))
            else:
                with np.errstate(invalid="ignore"):
                    w = np.exp(l[chosen] - np.nanmax(l[chosen], initial=-np.inf))
            w = np.where(np.isnan(l[chosen]), np.nan, w)
            w = w / w.sum()
        else:
            w = s[chosen]
        weights[t, :len(chosen)] = w * routed_scale
    return ids, weights


def route_scores_backward(logits, ids, dweights, score=SIGMOID, renormalize=True, routed_scale=1.0, live=None):
    """(dlogits, sums of the magnitudes of each one's terms)."""
    M, E = logits.shape
    out, mag = np.zeros((M, E)), np.zeros((M, E))
    for t in range(M if live is None else min(max(live, 0), M)):
        l = logits[t]
        listed = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E and l[ids[t, j]] != -np.inf]
        if not listed:
            continue
        at, dw = ids[t, listed], dweights[t, listed] * routed_scale
        if renormalize:
            top = min(l[at].max(), 0.0) if score == SIGMOID else l[at].max()
            p = np.exp(np.minimum(l[at], 0.0) - top) / (1.0 + np.exp(-np.abs(l[at]))) if score == SIGMOID else np.exp(l[at] - top)
            p = p / p.sum()
            f = p * sigmoid(-l[at]) if score == SIGMOID else p
            np.add.at(out[t], at, f * (dw - (dw * p).sum()))
            np.add.at(mag[t], at, f * (np.abs(dw) + (np.abs(dw) * p).sum()))
        elif score == SIGMOID:
            f = sigmoid(l[at]) * sigmoid(-l[at])
            np.add.at(out[t], at, dw * f)
            np.add.at(mag[t], at, np.abs(dw) * f)
        else:
            s = scores(l, SOFTMAX)
            out[t] = -s * (dw * s[at]).sum()
            mag[t] = s * (np.abs(dw) * s[at]).sum()
            np.add.at(out[t], at, dw * s[at])
            np.add.at(mag[t], at, np.abs(dw) * s[at])
    return out, mag


def route_balance(load, bias, rate):
    load = load.astype(np.int64)
    return bias + rate * np.sign(load.sum() - load * load.size)


# ------------------------------------------------------------------ norms

def root(x, eps):
    return 1.0 / np.sqrt((x * x).mean(1, keepdims=True) + eps)


def norm_residual(y, r=None, gate=None, w_post=None, w_pre=None, post_norm=False, residual_scale=1.0, weight_offset=0.0, eps=1e-6):
    """{h, z and the magnitudes h_mag and z_mag}.  gate broadcasts against [M, H]; weights None: 1."""
    u = y
    if post_norm:
        u = y * root(y, eps) * (1.0 if w_post is None else w_post + weight_offset)
    h = u if gate is None else gate * u
    mag = np.abs(h)
    if r is not None:
        h = h + residual_scale * r
        mag = mag + np.abs(residual_scale * r)
    R = root(h, eps)
    w = 1.0 if w_pre is None else w_pre + weight_offset
    # a relative error of the terms of h moves z by its own element and by the root
    with np.errstate(invalid="ignore", divide="ignore"):
        moved = (mag * np.abs(h)).sum(1, keepdims=True) / np.maximum((h * h).sum(1, keepdims=True), 1e-300)
    return {"h": h, "z": h * R * w, "h_mag": mag, "z_mag": (mag + np.abs(h) * (1.0 + np.minimum(moved, 1e6))) * R * np.abs(w)}


def quantised(z, pow2):
    """The scales of each row's groups of 128 columns, before they are rounded to 32 bits."""
    scale = np.abs(z).reshape(z.shape[0], -1, 128).max(2) / 448.0
    if pow2:
        with np.errstate(divide="ignore"):
            scale = np.where(scale > 0, np.exp2(np.ceil(np.log2(scale))), 0.0)
    return scale


def _through(x, w, d, eps):
    """Gradient of N(x; w) by x with the magnitude of its terms, and that by w's rows with theirs."""
    R = root(x, eps)
    dw = d * w
    a, b = R * dw, x * R ** 3 * (dw * x).mean(1, keepdims=True)
    b_mag = np.abs(x) * R ** 3 * np.abs(dw * x).mean(1, keepdims=True)
    return a - b, np.abs(a) + b_mag, d * x * R


def norm_residual_backward(y, dh=None, dz=None, h=None, gate=None, w_post=None, w_pre=None, post_norm=False, residual_scale=1.0,
                           weight_offset=0.0, eps=1e-6):
    """{dy, dr, dw_pre, dw_post, dgate_full (before any sum)}, each with its magnitude under "..._mag"."""
    H = y.shape[1]
    ones = np.ones(H)
    total = np.zeros_like(y) if dh is None else dh.copy()
    mag = np.abs(total)
    out = {}
    if dz is not None:
        w = ones if w_pre is None else w_pre + weight_offset
        d, m, rows = _through(y if h is None else h, w, dz, eps)
        total, mag = total + d, mag + m
        out["dw_pre"], out["dw_pre_mag"] = rows.sum(0), np.abs(rows).sum(0)
    out["dr"], out["dr_mag"] = residual_scale * total, abs(residual_scale) * mag
    w = (ones if w_post is None else w_post + weight_offset) if post_norm else ones
    u = y * root(y, eps) * w if post_norm else y
    out["dgate_full"], out["dgate_full_mag"] = total * u, mag * np.abs(u)
    g = 1.0 if gate is None else gate
    d, m = total * g, mag * np.abs(g)
    if post_norm:
        R = root(y, eps)
        rows = d * y * R
        out["dw_post"], out["dw_post_mag"] = rows.sum(0), (m * np.abs(y) * R).sum(0)
        d, _, _ = _through(y, w, d, eps)
        m = R * m * np.abs(w) + np.abs(y) * R ** 3 * (m * np.abs(w * y)).mean(1, keepdims=True)
    out["dy"], out["dy_mag"] = d, m
    return out
