"""A mixture-of-experts router, its gradient and the routed experts, one
token at a time in float64 from their definitions.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Selection compares
32-bit values by definition: `selection` computes them in float32, each
operation rounded, where scores that round to the same value tie.  The weights
are then those of the float64 scores.
"""
import numpy as np

MOST = float(np.finfo(np.float32).max)
TINY = float(np.finfo(np.float32).tiny)


def scores(row, bias, score):
    """(p float64 [E], available bool [E])."""
    l = np.asarray(row, np.float64)
    there = ~(np.isnan(l) | (l == -np.inf))
    if bias is not None:
        there &= ~(np.isnan(bias) | (bias == -np.inf))
    p = np.zeros(l.shape)
    if there.any():
        v = np.minimum(l[there], MOST)
        if score == "softmax":
            e = np.exp(v - v.max())
            p[there] = e / e.sum()
        else:
            with np.errstate(over="ignore"):
                p[there] = 1.0 / (1.0 + np.exp(-v))
    return p, there


def selection(row, bias, score):
    """The float32 values that the selection compares."""
    l = np.minimum(np.asarray(row, np.float64), MOST).astype(np.float32)
    p, there = scores(row, bias, score)
    s = np.zeros(l.shape, np.float32)
    if there.any() and score == "softmax":
        e = np.zeros(1 << (len(l) - 1).bit_length(), np.float32)
        e[:len(l)][there] = np.exp(l[there] - l[there].max())
        tree = e
        while len(tree) > 1:
            tree = tree[0::2] + tree[1::2]
        s[there] = (e[:len(l)] / tree[0])[there]
    elif there.any():
        with np.errstate(over="ignore"):
            s[there] = np.float32(1) / (np.float32(1) + np.exp(-l[there]))
    return s if bias is None else s + np.asarray(bias, np.float32)


def route_row(row, k, bias=None, score="softmax", groups=1, top_groups=1, renorm=True, scale=1.0):
    """(ids, weights) of one token: plain loops over the definition."""
    E = len(row)
    p, there = scores(row, bias, score)
    s = selection(row, bias, score)
    live = [e for e in range(E) if there[e]]
    if top_groups < groups:
        size = E // groups
        value = []
        for q in range(groups):
            mine = sorted((s[e] for e in live if e // size == q), reverse=True)[:2]
            value.append(-np.inf if not mine else mine[0] if len(mine) == 1 else np.float32(mine[0] + mine[1]))
        best = sorted(range(groups), key=lambda q: (-value[q], q))[:top_groups]
        live = [e for e in live if e // size in best]
    ids = sorted(live, key=lambda e: (-s[e], e))[:k]
    w = np.array([p[e] for e in ids])
    if renorm and len(w):
        w = w / max(w.sum(), TINY)
    ids = np.array(ids + [-1] * (k - len(ids)), np.int64)
    return ids, np.concatenate([w * scale, np.zeros(k - len(w))])


def route(logits, k, **kw):
    rows = [route_row(r, k, **kw) for r in logits]
    return np.array([r[0] for r in rows]).reshape(-1, k), np.array([r[1] for r in rows]).reshape(-1, k)


def plan(ids, E):
    """(offsets [E+1], slots [T*k]): slots by expert, then by index; -1 past the routed ones."""
    flat = ids.reshape(-1)
    slots = [s for e in range(E) for s in range(len(flat)) if flat[s] == e]
    counts = [int((flat == e).sum()) for e in range(E)]
    return np.concatenate([[0], np.cumsum(counts)]), np.array(slots + [-1] * (len(flat) - len(slots)))


def weights_of(row, ids, bias=None, score="softmax", renorm=True, scale=1.0):
    """Weights of given experts (what the gradient differentiates)."""
    p, _ = scores(row, bias, score)
    w = np.array([p[e] if e >= 0 else 0.0 for e in ids])
    if renorm:
        w = w / max(w.sum(), TINY)
    return w * scale


def route_backward(logits, ids, dw, bias=None, score="softmax", renorm=True, scale=1.0):
    out = np.zeros(np.shape(logits))
    for t, row in enumerate(logits):
        p, _ = scores(row, bias, score)
        on = [(e, g * scale) for e, g in zip(ids[t], np.asarray(dw[t], np.float64)) if e >= 0]
        q = np.zeros(len(row))
        S = sum(p[e] for e, _ in on)
        clamped = renorm and S < TINY                     # w = scale p / TINY: nothing is shared out
        for e, g in on:
            q[e] = g if not renorm else g / TINY if clamped else (g - sum(h * p[i] for i, h in on) / S) / S
        if score == "softmax":
            out[t] = p * (q - (0.0 if renorm and not clamped else sum(q[e] * p[e] for e, _ in on)))
        else:
            out[t] = p * (1 - p) * q
    return out


def experts(x, ids, weights, gate, up, down):
    """out[t] = sum_j w * Down_e(silu(Gate_e x) * Up_e x); matrices float64 [E, ., .]."""
    x = np.asarray(x, np.float64)
    out = np.zeros((x.shape[0], down.shape[1]))
    for t in range(x.shape[0]):
        for e, w in zip(ids[t], weights[t]):
            if e >= 0:
                a, u = gate[e] @ x[t], up[e] @ x[t]
                out[t] += float(w) * (down[e] @ (a / (1.0 + np.exp(-a)) * u))
    return out


def experts_bound(x, ids, weights, gate, up, down, eps_gate, eps_down, eps_hidden):
    """A first-order bound of the error of `experts` where each product over k has an error of at most
    eps * sum|.| and the hidden value a relative one of eps_hidden (|silu'| <= 1.1)."""
    x = np.asarray(x, np.float64)
    out = np.zeros((x.shape[0], down.shape[1]))
    for t in range(x.shape[0]):
        for e, w in zip(ids[t], weights[t]):
            if e >= 0:
                a, u = gate[e] @ x[t], up[e] @ x[t]
                da, du = eps_gate * (np.abs(gate[e]) @ np.abs(x[t])), eps_gate * (np.abs(up[e]) @ np.abs(x[t]))
                s = a / (1.0 + np.exp(-a))
                dh = 1.1 * da * (np.abs(u) + du) + np.abs(s) * du + eps_hidden * (np.abs(s * u) + np.abs(s * u).max())
                out[t] += abs(float(w)) * (np.abs(down[e]) @ (dh + eps_down * np.abs(s * u)))
    return out
