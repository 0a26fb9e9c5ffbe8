"""The 8-bit cache of keys and values and the attention over it, from the definition.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Codes uint8 [blocks, 2, H, B, D] and float32 scales [blocks, 2, H]; a code c stands
for (c - 128) * scale.  Sequence s has rows offsets[s]..offsets[s+1]-1 of new
tokens or queries, the last of its lens[s] tokens; token t lies in block
table[s, t // B] at t % B.
"""
import numpy as np

F = np.float32


def tokens_of(table, offsets, lens, blocks, B, s):
    """(row, position, block or -1, place in the block) of each of a sequence's rows with a position."""
    n = offsets[s + 1] - offsets[s]
    for j in range(n):
        t = lens[s] - n + j
        if t >= 0:
            b = table[s, t // B]
            yield offsets[s] + j, t, (b if 0 <= b < blocks else -1), t % B


def write(codes, scales, table, offsets, lens, x):
    """x float32 [2, T, H, D] (keys, values) into copies of codes and scales, in 32-bit steps."""
    codes, scales = codes.copy(), scales.copy()
    P, _, H, B, D = codes.shape
    for s in range(len(lens)):
        into = {}
        for row, t, b, at in tokens_of(table, offsets, lens, P, B, s):
            if b >= 0:
                into.setdefault((t // B, b), []).append((row, at))
        for (_, b), where in into.items():
            rows, at = [w[0] for w in where], [w[1] for w in where]
            for kv in range(2):
                for h in range(H):
                    new = x[kv, rows, h].astype(F)
                    most = F(np.abs(new).max())
                    d0 = scales[b, kv, h] if at[0] > 0 else F(0)
                    if not np.isfinite(new).all() or np.isnan(d0):
                        scales[b, kv, h] = np.nan
                        continue
                    d = max(d0, F(most / F(127)) if most >= F(2.0 ** -96) else F(0))
                    if at[0] > 0 and d > d0:
                        old = codes[b, kv, h, :at[0]].astype(F) - F(128)
                        codes[b, kv, h, :at[0]] = np.rint(old * F(d0 / d)) + F(128)
                    with np.errstate(over="ignore"):
                        inv = min(F(F(1) / d), np.finfo(F).max) if d > 0 else F(0)
                    codes[b, kv, h, at] = np.clip(np.rint(new * inv), -127, 127) + F(128)
                    scales[b, kv, h] = d
    return codes, scales


def values(codes, scales):
    """[blocks, 2, H, B, D] float64."""
    return (codes.astype(np.float64) - 128.0) * scales.astype(np.float64)[..., None, None]


def context(codes, scales, table, lens, s, kv):
    """(values [L, H, D], there [L]) of a sequence's tokens; tokens without a block are not there."""
    P, _, H, B, D = codes.shape
    L = lens[s]
    x, there = np.zeros((L, H, D)), np.zeros(L, bool)
    for t0 in range(0, L, B):
        b, n = table[s, t0 // B], min(B, L - t0)
        if 0 <= b < P:
            c = codes[b, kv, :, :n].astype(np.float64) - 128.0
            x[t0:t0 + n] = (c * scales[b, kv].astype(np.float64)[:, None, None]).transpose(1, 0, 2)
            there[t0:t0 + n] = True
    return x, there


def seen(n, L, causal, window):
    """[n, L]: which tokens the last n of L see."""
    t, i = np.arange(L)[None, :], L - n + np.arange(n)[:, None]
    if not causal:
        return np.ones((n, L), bool)
    return (t <= i) & ((t > i - window) if window else True)


def attention(q, codes, scales, table, offsets, lens, scale, causal=True, window=0):
    """q float64 [T, Hq, D] -> dict of out, lse, and of what bounds a computed result's error, by row and head:
    spread = sum_t p_t |v_t| [.., D], score = the largest scale * sum_d |q_d k_d|, and
    top = the largest p_t times its block's value scale."""
    T, Hq, D = q.shape
    H, B = codes.shape[2], codes.shape[3]
    G = Hq // H
    r = {"out": np.zeros((T, Hq, D)), "lse": np.full((T, Hq), np.nan), "spread": np.zeros((T, Hq, D)),
         "score": np.zeros((T, Hq)), "top": np.zeros((T, Hq)), "rows": np.zeros(T, bool)}
    for s in range(len(lens)):
        a, b = offsets[s], offsets[s + 1]
        if a == b:
            continue
        k, there = context(codes, scales, table, lens, s, 0)
        v, _ = context(codes, scales, table, lens, s, 1)
        see = seen(b - a, lens[s], causal, window) & there[None, :]
        vs = np.zeros((lens[s], H))
        for t in np.nonzero(there)[0]:
            vs[t] = scales[table[s, t // B], 1]
        r["rows"][a:b] = True
        for h in range(Hq):
            z = scale * q[a:b, h] @ k[:, h // G].T if lens[s] else np.zeros((b - a, 0))
            z = np.where(see, z, -np.inf)
            top = z.max(1, initial=-np.inf)
            e = np.where(see, np.exp(z - np.where(np.isfinite(top), top, 0)[:, None]), 0)
            l = e.sum(1)
            p = e / np.where(l > 0, l, 1)[:, None]
            vh = np.where(see.any(0)[:, None], v[:, h // G], 0)
            r["out"][a:b, h], r["spread"][a:b, h] = p @ vh, p @ np.abs(vh)
            with np.errstate(divide="ignore"):
                r["lse"][a:b, h] = top + np.log(l)
            A = abs(scale) * np.abs(q[a:b, h]) @ np.abs(k[:, h // G]).T if lens[s] else np.zeros((b - a, 0))
            r["score"][a:b, h] = np.where(see, A, 0).max(1, initial=0)
            r["top"][a:b, h] = (p * vs[:, h // G]).max(1, initial=0)
    return r
