"""Cases of the 4-bit weight products and the mixture-of-experts operators.

Each case names one operator and its sizes.  ``prepare`` makes what a program
has in hand before the call, ``run`` is one pass through the operator: the
plain form in elementary torch operations, or, where ``own`` is true, the
library's call.  ``work`` counts what a pass cannot do without and ``exact``
gives the same results from the definition in 64 bits.

Operators
  gemv            out = x W^T, W 4-bit codes with a scale (and a zero point)
                  per group of consecutive k; the decode-shape product
  route           scores, balance bias, groups, top-k and renormalised weights
                  of a router, and the order of its slots by expert
  route_backward  the gradient of the routing weights to the router's logits
  experts         the routed experts' gated products (gate, up, SiLU, down)
                  with 4-bit weights, combined with the routing weights
"""
import numpy as np
import torch

own = False

DEV = torch.device("cuda" if torch.cuda.is_available() else "cpu")
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
MOST = torch.finfo(torch.float32).max
LEAST = torch.finfo(torch.float32).tiny


def listed():
    return [
        # one token of a decode step through a square projection, full precision
        dict(name="gemv 1x4096x4096 f32", op="gemv", M=1, N=4096, K=4096, group=128, zeros=False, type="f32"),
        # a small decode batch through a feed-forward projection
        dict(name="gemv 8x11008x4096 bf16", op="gemv", M=8, N=11008, K=4096, group=128, zeros=True, type="bf16"),
        # sizes that no tile divides, the finest groups
        dict(name="gemv 3x1000x1056 f16", op="gemv", M=3, N=1000, K=1056, group=32, zeros=True, type="f16"),
        # the widest projection and the largest decode batch
        dict(name="gemv 16x14336x4096 bf16", op="gemv", M=16, N=14336, K=4096, group=64, zeros=False, type="bf16"),
        # routing of one decoded token: latency
        dict(name="route 1x64 top6", op="route", T=1, E=64, k=6, score="softmax", bias=False, groups=1, top_groups=1,
             renorm=True, masked=False, type="f32"),
        # a decode batch, grouped experts, some experts unavailable and some rows padding
        dict(name="route 300x160 top6 groups", op="route", T=300, E=160, k=6, score="softmax", bias=False, groups=8,
             top_groups=3, renorm=False, masked=True, type="bf16"),
        # a prefill chunk through the widest router, balanced by a bias
        dict(name="route 16384x256 top8 bias", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, renorm=True, masked=False, type="f32"),
        # the router's gradient: a small batch, then a training batch
        dict(name="route_backward 100x60", op="route_backward", T=100, E=60, k=4, score="sigmoid", bias=True,
             groups=1, top_groups=1, renorm=True, masked=True, type="f32"),
        dict(name="route_backward 16384x128", op="route_backward", T=16384, E=128, k=8, score="softmax", bias=False,
             groups=1, top_groups=1, renorm=False, masked=False, type="f32"),
        # experts of one decoded token: the weights of the chosen experts are read once
        dict(name="experts 1 of 64 f32", op="experts", T=1, E=64, k=8, D=2048, F=1024, group=128, zeros=False,
             padded=False, type="f32"),
        # a decode batch with padding rows: nearly every expert is hit by a few tokens
        dict(name="experts 64 of 64 bf16", op="experts", T=64, E=64, k=8, D=2048, F=1024, group=128, zeros=True,
             padded=True, type="bf16"),
        # a prefill chunk: tensor-core work, ragged token counts per expert
        dict(name="experts 2048 of 64 bf16", op="experts", T=2048, E=64, k=8, D=2048, F=1024, group=128, zeros=True,
             padded=False, type="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, uniform in its logarithm."""
    return max(lo, min(hi, int(round(float(np.exp(rng.uniform(np.log(lo), np.log(hi))))))))


def draw(rng):
    op = rng.choice(["gemv", "route", "route_backward", "experts"])
    if op == "gemv":
        group = rng.choice([32, 64, 128])
        K = group * _spread(rng, max(1, 256 // group), 14336 // group)
        N = _spread(rng, 64, min(14336, 14336 * 4096 // K))
        return dict(op=op, M=rng.randint(1, 16), N=N, K=K, group=group, zeros=rng.random() < 0.5,
                    type=rng.choice(["f32", "f16", "bf16"]))
    if op == "experts":
        T = _spread(rng, 1, 2048)
        return dict(op=op, T=T, E=rng.randint(8, 64), k=rng.randint(1, 8), D=128 * _spread(rng, 2, 16),
                    F=64 * _spread(rng, 2, 16), group=rng.choice([32, 64, 128]) if T <= 64 else 128,
                    zeros=rng.random() < 0.5, padded=rng.random() < 0.5,
                    type=rng.choice(["f32", "f16", "bf16"]) if T <= 64 else "bf16")
    groups = rng.choice([1, 1, 4, 8])
    E = groups * _spread(rng, 8 if groups == 1 else 4, 256 // groups)
    top = 1 if groups == 1 else rng.randint(2, groups)
    # one renormalised weight is 1 whatever the logits are: nothing to differentiate
    renorm = rng.random() < 0.5
    k = rng.randint(2 if renorm and op == "route_backward" else 1, min(8, top * (E // groups)))
    return dict(op=op, T=_spread(rng, 1, 16384), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                bias=rng.random() < 0.5, groups=groups, top_groups=top, renorm=renorm, masked=rng.random() < 0.5,
                type=rng.choice(["f32", "f16", "bf16"]))


# ------------------------------------------------------------------ inputs ----
def _q4(g, E, N, K, group, zeros):
    """Codes [E, N, K/2] (even k in the low half byte), scales f16 [E, N, K/group],
    zero points u8 of the same shape or None (then 8)."""
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = (torch.rand((E, N, K // group), generator=g, device=DEV) * 0.015 + 0.002).to(torch.float16)
    z = torch.randint(5, 11, (E, N, K // group), generator=g, device=DEV, dtype=torch.uint8) if zeros else None
    return {"codes": codes, "scales": scales, "zeros": z, "group": group}


def _activations(g, T, K, dtype):
    """Unit-scale activations with a few outlier channels, as hidden states have."""
    x = torch.randn((T, K), generator=g, device=DEV)
    x[:, torch.randint(0, K, (max(1, K // 256),), generator=g, device=DEV)] *= 12.0
    return x.to(dtype)


def _logits(g, c):
    """Router logits; masked: experts that are unavailable for a token, and padding rows with none left."""
    l = torch.randn((c["T"], c["E"]), generator=g, device=DEV) * 1.5
    if c["masked"]:
        l = l.masked_fill(torch.rand((c["T"], c["E"]), generator=g, device=DEV) < 1 / 16, float("-inf"))
        l = l.masked_fill(torch.rand((c["T"], 1), generator=g, device=DEV) < 1 / 32, float("-inf"))
    return l.to(TYPES[c["type"]])


def _balance(g, c):
    """Balance biases move in fixed steps between batches."""
    if not c["bias"]:
        return None
    return torch.randint(-60, 61, (c["E"],), generator=g, device=DEV).float() * 0.001


def _plan(ids, E):
    """Slots t*k+j ordered by expert (then by slot) and each expert's range; -1 past the routed ones."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=key.device))
    return offsets.int(), torch.where(key == E, -1, order).int()


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    op, s = c["op"], {"case": case}
    if op == "gemv":
        s["x"] = _activations(g, c["M"], c["K"], TYPES[c["type"]])
        s["w"] = _q4(g, 1, c["N"], c["K"], c["group"], c["zeros"])
        s["out"] = torch.empty((c["M"], c["N"]), dtype=s["x"].dtype, device=DEV)
        if own:
            s["handle"] = _handle(s["w"])
    elif op == "experts":
        T, E, k, D, F = c["T"], c["E"], c["k"], c["D"], c["F"]
        s["x"] = _activations(g, T, D, TYPES[c["type"]])
        s["gate"], s["up"] = (_q4(g, E, F, D, c["group"], c["zeros"]) for _ in range(2))
        # the down projection's inner size need not be a multiple of the wide groups
        s["down"] = _q4(g, E, D, F, c["group"] if F % c["group"] == 0 else 32, c["zeros"])
        s["weights"], ids = torch.randn((T, E), generator=g, device=DEV).softmax(-1).topk(k)
        if c["padded"] and T > 1:
            pad = torch.rand((T, 1), generator=g, device=DEV) < 1 / 16
            ids, s["weights"] = ids.masked_fill(pad, -1), s["weights"].masked_fill(pad, 0.0)
        s["ids"] = ids.int()
        s["offsets"], s["slots"] = _plan(ids, E)
        s["out"] = torch.empty((T, D), dtype=s["x"].dtype, device=DEV)
        if own:
            s["handles"] = [_handle(s[n]) for n in ("gate", "up", "down")]
    else:
        s["logits"], s["bias"] = _logits(g, c), _balance(g, c)
        T, k = c["T"], c["k"]
        if op == "route":
            s["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
            s["weights"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
            s["offsets"] = torch.empty((c["E"] + 1,), dtype=torch.int32, device=DEV)
            s["slots"] = torch.empty((T * k,), dtype=torch.int32, device=DEV)
        else:
            s["ids"] = _choose(*_scores(s["logits"], s["bias"], c["score"]), c)[0].int()
            s["dweights"] = torch.randn((T, k), generator=g, device=DEV)
            s["dlogits"] = torch.empty_like(s["logits"])
    return s


def _handle(w):
    import binary_packed_weight_gb300 as bpw
    return bpw.q4_upload(w["codes"], w["scales"], w["zeros"], group=w["group"])


# ------------------------------------------------------------- plain forms ----
def _dequant(w, pick=None):
    """W f32 [E, N, K] = (code - zero) * scale, of the picked matrices only where given."""
    codes, scales, zeros = (None if t is None else t if pick is None else t[pick]
                            for t in (w["codes"], w["scales"], w["zeros"]))
    E, N, half = codes.shape
    q = torch.stack((codes & 15, codes >> 4), -1).view(E, N, -1, w["group"]).float()
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((q - z) * scales.float().unsqueeze(-1)).view(E, N, 2 * half)


def _pair_sums(e):
    """Row sums as a tree over neighbouring pairs, so that the order of the additions is part of the definition."""
    width = 1 << (e.shape[-1] - 1).bit_length()
    e = torch.nn.functional.pad(e, (0, width - e.shape[-1]))
    while e.shape[-1] > 1:
        e = e[..., 0::2] + e[..., 1::2]
    return e


def _scores(logits, bias, score):
    """Scores and what the selection goes by.  An expert is available where its logit and its bias are neither
    -inf nor NaN; one that is not has score 0 and is never selected."""
    l = logits.float()
    there = l > float("-inf")
    if bias is not None:
        there = there & (bias > float("-inf"))
    l = l.clamp(max=MOST)
    if score == "softmax":
        top = torch.where(there, l, float("-inf")).amax(-1, keepdim=True)
        e = torch.where(there, torch.exp(l - top), 0.0)
        p = torch.where(there, e / _pair_sums(e), 0.0)
    else:
        p = torch.where(there, 1.0 / (1.0 + torch.exp(-l)), 0.0)
    return p, torch.where(there, p if bias is None else p + bias, float("-inf"))


def _choose(p, sel, c):
    """The k best by selection value among the best groups (a group counts its two best); ties to the lowest index."""
    T, E, G = c["T"], c["E"], c["groups"]
    if c["top_groups"] < G:
        two = sel.view(T, G, E // G).sort(dim=-1, descending=True)[0][..., :2]
        value = two[..., 0] + torch.where(two[..., 1:] > float("-inf"), two[..., 1:], 0.0).sum(-1)
        best = value.sort(dim=-1, descending=True, stable=True)[1][:, : c["top_groups"]]
        inside = torch.zeros((T, G), dtype=torch.bool, device=sel.device).scatter_(1, best, True)
        sel = torch.where(inside.repeat_interleave(E // G, 1), sel, float("-inf"))
    v, ids = sel.sort(dim=-1, descending=True, stable=True)
    v, ids = v[:, : c["k"]], ids[:, : c["k"]]
    chosen = v > float("-inf")
    return torch.where(chosen, ids, -1), torch.where(chosen, p.gather(1, ids), 0.0)


SCALE = 2.5                                                   # the factor some routers put on renormalised weights


def _route(s):
    c = s["case"]
    ids, w = _choose(*_scores(s["logits"], s["bias"], c["score"]), c)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=LEAST)
    offsets, slots = _plan(ids, c["E"])
    return {"ids": ids.int(), "weights": w * SCALE, "offsets": offsets, "slots": slots}


def _route_backward(s):
    c = s["case"]
    p, _ = _scores(s["logits"], s["bias"], c["score"])
    ids, dw = s["ids"].long(), s["dweights"] * SCALE
    chosen = ids >= 0
    at = ids.clamp(min=0)
    dw, w = torch.where(chosen, dw, 0.0), torch.where(chosen, p.gather(1, at), 0.0)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True).clamp(min=LEAST)
        dw = torch.where(chosen, (dw - (dw * w).sum(-1, keepdim=True) / total) / total, 0.0)
    dp = torch.zeros_like(p).scatter_add_(1, at, dw)
    dl = p * (dp - (dp * p).sum(-1, keepdim=True)) if c["score"] == "softmax" else p * (1.0 - p) * dp
    return dl.to(s["logits"].dtype)


def _experts(s):
    """Rows sorted by expert in blocks of equal height, one batched product per matrix."""
    c, x = s["case"], s["x"]
    T, E, k = c["T"], c["E"], c["k"]
    S = T * k
    rows = max(1, min(64, S // E))
    nb = S // rows + min(E, S)
    offsets, slots = s["offsets"].long(), s["slots"].long()
    count = offsets[1:] - offsets[:-1]
    blocks = (count + rows - 1) // rows
    end = blocks.cumsum(0)
    b = torch.arange(nb, device=x.device)
    e = torch.searchsorted(end, b, right=True).clamp(max=E - 1)
    at = (b - (end - blocks)[e]).unsqueeze(1) * rows + torch.arange(rows, device=x.device)
    valid = (at < count[e].unsqueeze(1)) & (b < end[-1]).unsqueeze(1)
    slot = torch.where(valid, slots[(offsets[e].unsqueeze(1) + at).clamp(max=S - 1)], S)
    few = nb < E
    gate, up, down = (_dequant(s[n], e) if few else _dequant(s[n])[e] for n in ("gate", "up", "down"))
    xb = x.float()[(slot // k).clamp(max=T - 1)]
    a, u = xb @ gate.transpose(1, 2), xb @ up.transpose(1, 2)
    y = (a / (1.0 + torch.exp(-a)) * u) @ down.transpose(1, 2)
    by_slot = torch.zeros((S + 1, c["D"]), device=x.device)
    by_slot[slot.view(-1)] = y.view(-1, c["D"])
    by_slot = by_slot[:S].view(T, k, -1)
    return (torch.where(s["ids"].unsqueeze(-1) >= 0, by_slot * s["weights"].unsqueeze(-1), 0.0)).sum(1).to(x.dtype)


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "gemv":
            return (s["x"].float() @ _dequant(s["w"])[0].T).to(s["x"].dtype)
        return {"route": _route, "route_backward": _route_backward, "experts": _experts}[op](s)
    import binary_packed_weight_gb300 as bpw
    if op == "gemv":
        return bpw.q4_gemm(s["handle"], s["x"], s["out"])
    if op == "experts":
        return bpw.moe_experts(*s["handles"], s["x"], s["ids"], s["weights"], s["offsets"], s["slots"], s["out"])
    if op == "route":
        bpw.moe_route(s["logits"], s["ids"], s["weights"], s["offsets"], s["slots"], bias=s["bias"],
                      score=c["score"], groups=c["groups"], top_groups=c["top_groups"], renorm=c["renorm"],
                      scale=SCALE)
        return {n: s[n] for n in ("ids", "weights", "offsets", "slots")}
    return bpw.moe_route_backward(s["logits"], s["ids"], s["dweights"], s["dlogits"], bias=s["bias"],
                                  score=c["score"], renorm=c["renorm"], scale=SCALE)


# -------------------------------------------------------------------- work ----
def _q4_bytes(N, K, group, zeros):
    return N * K / 2 + N * (K // group) * (3 if zeros else 2)


def work(case):
    c = case
    size = BYTES[c["type"]]
    if c["op"] == "gemv":
        return {"bytes": _q4_bytes(c["N"], c["K"], c["group"], c["zeros"]) + size * c["M"] * (c["N"] + c["K"]),
                "flops": 2.0 * c["M"] * c["N"] * c["K"]}
    if c["op"] == "experts":
        T, E, k, D, F = c["T"], c["E"], c["k"], c["D"], c["F"]
        hit = E * (1.0 - (1.0 - k / E) ** T)                  # experts that some token chose, on average
        down = c["group"] if F % c["group"] == 0 else 32
        return {"bytes": hit * (2 * _q4_bytes(F, D, c["group"], c["zeros"]) + _q4_bytes(D, F, down, c["zeros"]))
                + 2 * size * T * D + 8 * T * k + 4 * (E + 1), "flops": 6.0 * T * k * D * F}
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "route":
        return {"bytes": size * T * E + 12 * T * k + 4 * (E + 1), "flops": 8.0 * T * E}
    dense = c["score"] == "softmax" and not c["renorm"]       # else only the chosen logits matter
    return {"bytes": size * T * E + size * T * (E if dense else k) + 8 * T * k, "flops": 6.0 * T * (E if dense else k)}


# ----------------------------------------------------------- from the definition ----
def _exact_weight(w, e):
    codes, scales, zeros = (None if t is None else t[e] for t in (w["codes"], w["scales"], w["zeros"]))
    W = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.float64, device=DEV)
    W[:, 0::2] = (codes % 16).double()
    W[:, 1::2] = (codes // 16).double()
    z = torch.full_like(scales, 8.0).double() if zeros is None else zeros.double()
    return (W - z.repeat_interleave(w["group"], 1)) * scales.double().repeat_interleave(w["group"], 1)


def _exact_scores(s):
    l = s["logits"].double().cpu().numpy()
    bias = None if s["bias"] is None else s["bias"].double().cpu().numpy()
    shut = np.isnan(l) | (l == -np.inf)
    l = np.minimum(l, MOST)
    p = np.zeros_like(l)
    if s["case"]["score"] == "softmax":
        live = ~shut.all(1)
        m = np.where(shut, -np.inf, l)[live]
        m = np.exp(m - m.max(1, keepdims=True))
        p[live] = m / m.sum(1, keepdims=True)
    else:
        p = np.where(shut, 0.0, 1.0 / (1.0 + np.exp(-np.where(shut, 0.0, l))))
    return p, shut, bias


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "gemv":
        return s["x"].double() @ _exact_weight(s["w"], 0).T
    if c["op"] == "experts":
        T, k = c["T"], c["k"]
        out = torch.zeros((T, c["D"]), dtype=torch.float64, device=DEV)
        ids = s["ids"].long()
        for e in range(c["E"]):
            t, j = (ids == e).nonzero(as_tuple=True)
            if t.numel():
                x = s["x"][t].double()
                a, u = x @ _exact_weight(s["gate"], e).T, x @ _exact_weight(s["up"], e).T
                y = (a * torch.sigmoid(a) * u) @ _exact_weight(s["down"], e).T
                out.index_add_(0, t, y * s["weights"][t, j].double().unsqueeze(1))
        return out
    p, shut, bias = _exact_scores(s)
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    if c["op"] == "route":
        # selection goes by 32-bit values, by definition
        sel = p.astype(np.float32) + (0 if bias is None else bias.astype(np.float32))
        sel = np.where(shut, -np.inf, sel).astype(np.float32)
        if c["top_groups"] < G:
            two = -np.sort(-sel.reshape(T, G, E // G), -1)[..., :2]
            value = two[..., 0] + np.where(np.isinf(two[..., 1]), np.float32(0), two[..., 1])
            rank = np.argsort(np.argsort(-value, -1, kind="stable"), -1)
            sel = np.where(np.repeat(rank < c["top_groups"], E // G, 1), sel, -np.inf)
        ids = np.argsort(-sel, -1, kind="stable")[:, :k]
        w = np.where(np.isinf(np.take_along_axis(sel, ids, 1)), 0.0, np.take_along_axis(p, ids, 1))
        if c["renorm"]:
            w = w / np.maximum(w.sum(1, keepdims=True), LEAST)
        return {"ids": None, "weights": torch.from_numpy(w * SCALE), "offsets": None, "slots": None}
    ids, dw = s["ids"].cpu().numpy().astype(np.int64), s["dweights"].double().cpu().numpy() * SCALE
    at, chosen = np.maximum(ids, 0), ids >= 0
    w = np.where(chosen, np.take_along_axis(p, at, 1), 0.0)
    dw = np.where(chosen, dw, 0.0)
    if c["renorm"]:
        total = np.maximum(w.sum(1, keepdims=True), LEAST)
        dw = np.where(chosen, dw / total - (dw * w).sum(1, keepdims=True) / total ** 2, 0.0)
    dl = np.zeros_like(p)
    rows = np.arange(T)[:, None] + np.zeros_like(at)
    ps = np.take_along_axis(p, at, 1)
    if c["score"] == "softmax":
        dl = -p * (dw * ps).sum(1, keepdims=True)
        np.add.at(dl, (rows, at), dw * ps)
        if c["renorm"]:                                       # the sum vanishes: nothing flows to the others
            dl[:] = 0.0
            np.add.at(dl, (rows, at), dw * ps)
    else:
        np.add.at(dl, (rows, at), dw * ps * (1.0 - ps))
    return torch.from_numpy(dl)
