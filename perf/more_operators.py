"""Cases of the 8-bit cache of keys and values, and of the attention that reads it.

A cache is a pool of blocks of ``B`` tokens: codes uint8 [blocks, 2, H, B, D]
(keys, then values) and one float32 scale [blocks, 2, H] for a block's tokens in a
head.  A code c stands for (c - 128) * scale.  Each sequence has a row of a table
of block numbers.

Each case names one operator and its sizes.  ``prepare`` makes what a program has in
hand before the call, ``run`` is one pass: the plain form in elementary torch
operations, or, where ``own`` is true, the library's calls.  ``work`` counts what a
pass cannot do without and ``exact`` gives the same results from the definition in
64 bits.

Operators
  write    new tokens' keys and values are quantised as they enter the blocks (a block
           that is part full keeps its tokens, on a coarser scale where the new ones
           need it), and the blocks that were touched are read back
  read     the tokens of some sequences as values again
  attend   softmax(scale q k^T) v of each sequence's last tokens over its cache, query
           heads in groups that share a head of the cache; causal, inside a window, or
           over all of it; and the logarithm of the softmax's sum
"""
import math
import random

import numpy as np
import torch

own = False

DEV = torch.device("cuda" if torch.cuda.is_available() else "cpu")
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
SMALLEST = 2.0 ** -96                                         # a block whose largest value is below counts as zeros


def listed():
    return [
        # a decode step of 48 sequences: each block gains one token
        dict(name="write 48 tokens bf16", op="write", S=48, new=1, most=4096, H=8, D=128, B=64, type="bf16"),
        # prompts of three sequences that start afresh and continue
        dict(name="write 16384 tokens bf16", op="write", S=3, new=8000, most=9000, H=8, D=128, B=64, type="bf16"),
        # chunks that begin and end inside small blocks, full precision
        dict(name="write chunks f32", op="write", S=10, new=300, most=1500, H=5, D=64, B=16, type="f32"),
        # one short sequence taken out of the cache: latency
        dict(name="read 1 of 333 f32", op="read", S=1, new=333, most=333, H=3, D=64, B=32, type="f32"),
        # sequences handed on as plain values
        dict(name="read 8 of 8192 bf16", op="read", S=8, new=8192, most=8192, H=8, D=128, B=128, type="bf16"),
        # one decoded token after a short prompt: latency
        dict(name="attend 1 of 700 bf16", op="attend", S=1, new=1, most=700, H=8, G=4, D=128, B=64, causal=True,
             window=0, pad=0, type="bf16"),
        # a decode step of a ragged batch
        dict(name="attend 64 of 8192 bf16", op="attend", S=64, new=1, most=8192, H=8, G=4, D=128, B=64, causal=True,
             window=0, pad=0, type="bf16"),
        # one token of a very long context: all of the card for one sequence
        dict(name="attend 1 of 131072 f16", op="attend", S=1, new=1, most=131072, H=4, G=8, D=128, B=128, causal=True,
             window=0, pad=0, type="f16"),
        # a few drafted tokens a sequence, odd sizes, sequences without tokens, rows of padding, full precision
        dict(name="attend drafts f32", op="attend", S=7, new=4, most=1000, H=3, G=5, D=64, B=16, causal=True,
             window=300, pad=3, type="f32"),
        # a prompt in one piece: tensor-core work
        dict(name="attend prompt 8192 bf16", op="attend", S=1, new=8192, most=8192, H=8, G=4, D=128, B=64, causal=True,
             window=0, pad=0, type="bf16"),
        # chunks of prompts beside decoded tokens, a sliding window
        dict(name="attend chunks f16", op="attend", S=6, new=700, most=6000, H=4, G=6, D=64, B=32, causal=True,
             window=2048, pad=5, type="f16"),
        # tokens of a decoder over an encoder's states of another length
        dict(name="attend states bf16", op="attend", S=4, new=200, most=1500, H=16, G=1, D=64, B=64, causal=False,
             window=0, pad=0, type="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    c = dict(op=op, D=rng.choice([64, 128]), B=rng.choice([16, 32, 64, 128]), type=rng.choice(["f32", "f16", "bf16"]))
    if op != "attend":
        S, H = _spread(rng, 1, 64), rng.randint(1, 8)
        new = _spread(rng, 1, 8192 // S) if rng.random() < 0.7 else 1
        most = new + (_spread(rng, 1, 4096) if op == "write" else 0)
        return dict(c, S=S, new=new, most=most, H=H)
    kind = rng.choice(["decode", "drafts", "chunks", "states"])
    S, H, G = _spread(rng, 1, 64), rng.randint(1, 8), rng.randint(1, 8)
    new = {"decode": 1, "drafts": rng.randint(2, 8)}.get(kind) or _spread(rng, 16, 2048)
    # no more tokens than the largest ragged batch, no more scores than the longest prompt
    most = _spread(rng, max(16, new), max(16, new, min(65536, (1 << 19) // S, (1 << 29) // (S * H * G * new))))
    S = max(1, min(S, (1 << 30) // (H * G * new * most), (1 << 19) // (H * G * new)))
    causal = kind != "states"
    return dict(c, S=S, new=new, most=most, H=H, G=G, causal=causal,
                window=_spread(rng, 1, most) if causal and rng.random() < 0.3 else 0, pad=rng.choice([0, 0, 1, 9]))


# ------------------------------------------------------------------ inputs ----
def _lengths(c):
    """New tokens and length after them of each sequence: a case's sizes alone decide them."""
    rng = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    S, new, most = c["S"], c["new"], c["most"]
    n = [new if new == 1 or c["op"] == "read" or S == 1 else rng.randint(max(1, new // 8), new) for _ in range(S)]
    if S == 1 or c["op"] == "read":
        total = [most] * S
    else:
        total = [rng.randint(min(most, max(k, most // 16)), most) for k in n]
    if c["op"] == "write" and S > 1 and new > 1:              # some start afresh
        total = [n[i] if i % 3 == 0 else total[i] for i in range(S)]
    if c["op"] == "attend" and S > 3:
        n[S // 2] = 0                                         # a sequence that waits
        if new > 1:
            n[S - 1] = 1                                      # one that decodes beside the others
        total[1] = 0 if c["new"] <= 8 else total[1]           # and one that has no tokens yet
    return n, total


def _pool(g, c, total):
    """A cache whose blocks are handed out in no order, with stale contents where no token is; and its table."""
    B, H, D = c["B"], c["H"], c["D"]
    need = [-(-t // B) for t in total]
    width = max(1, max(need)) + 1
    P = sum(need) + 5
    codes = torch.randn((P, 2, H, B, D), generator=g, device=DEV).mul_(36.0).round_().clamp_(-127, 127).add_(128)
    codes = codes.to(torch.uint8)
    scales = torch.rand((P, 2, H), generator=g, device=DEV) * 0.04 + 0.01
    order = torch.randperm(P, generator=g, device=DEV).int()
    need_t = torch.tensor(need, device=DEV)
    first = need_t.cumsum(0) - need_t
    col = torch.arange(width, device=DEV)
    at = (first.unsqueeze(1) + col).clamp(max=P - 1)
    table = torch.where(col < need_t.unsqueeze(1), order[at], -1).int()
    return codes, scales, table


def _tokens(g, T, H, D, dtype):
    """Keys or values of new tokens, cut out of a wider projection's rows; a few channels stand out."""
    x = torch.randn((T, H + 2, D), generator=g, device=DEV)
    x[:, :, torch.randint(0, D, (2,), generator=g, device=DEV)] *= 6.0
    return x.to(dtype)[:, 1:H + 1]


def _batch(n, total):
    """Offsets of the sequences' new tokens, lengths, and for each token its sequence and position."""
    n_t, l_t = torch.tensor(n, device=DEV), torch.tensor(total, device=DEV)
    offsets = torch.cat((n_t.new_zeros(1), n_t.cumsum(0)))
    seq = torch.repeat_interleave(torch.arange(len(n), device=DEV), n_t)
    at = torch.arange(int(offsets[-1]), device=DEV) - offsets[seq]
    return offsets.int(), l_t.int(), seq, at, l_t[seq] - n_t[seq] + at


def prepare(case, seed):
    c, g = case, torch.Generator(device=DEV).manual_seed(seed)
    n, total = _lengths(c)
    s = {"case": c, "n": n, "total": total}
    s["codes"], s["scales"], s["table"] = _pool(g, c, total)
    s["offsets"], s["lens"], s["seq"], s["at"], s["pos"] = _batch(n, total)
    T, H, D, dtype = sum(n), c["H"], c["D"], TYPES[c["type"]]
    if c["op"] == "attend":
        Hq = H * c["G"]
        rows = T + c["pad"]
        q = torch.randn((rows, Hq + 2, D), generator=g, device=DEV) * 1.5
        s["q"] = q.to(dtype)[:, :Hq]
        s["out"] = torch.zeros((rows, Hq, D), dtype=dtype, device=DEV)
        s["lse"] = torch.zeros((rows, Hq), device=DEV)
    else:
        back = n
        if c["op"] == "write":
            s["k"], s["v"] = _tokens(g, T, H, D, dtype), _tokens(g, T, H, D, dtype)
            # read back from the first token of the first block that was touched
            back = [k + (t - k) % c["B"] for k, t in zip(n, total)]
            # the blocks that the new tokens enter, and for each token which of them
            s["touched"], s["into"] = s["table"][s["seq"], s["pos"] // c["B"]].long().unique(return_inverse=True)
        s["back"], _, s["back_seq"], _, s["back_pos"] = _batch(back, total)
        s["k_out"] = torch.empty((sum(back), H, D), dtype=dtype, device=DEV)
        s["v_out"] = torch.empty_like(s["k_out"])
    if own:
        import binary_packed_weight_gb300 as bpw
        s["cache"] = bpw.KV8Cache(s["codes"], s["scales"])
        s["batch"] = bpw.KV8Batch(s["table"], s["offsets"], s["lens"])
        if c["op"] != "attend":
            s["back_batch"] = bpw.KV8Batch(s["table"], s["back"], s["lens"])
    return s


# ------------------------------------------------------------- plain forms ----
def _values(s, block):
    """Keys and values float32 of whole blocks [.., H, B, D]."""
    return ((s["codes"][block].float() - 128.0) * s["scales"][block][..., None, None]).unbind(-4)


def _write(s):
    c = s["case"]
    B, H, block = c["B"], c["H"], s["touched"]
    N = len(block)
    x = torch.stack((s["k"], s["v"]), 1).float()                                       # [T, 2, H, D]
    into, slot = s["into"], s["pos"] % B
    # the largest new magnitude of each touched block, and how many of its tokens were there before
    most = torch.zeros((N, 2, H), device=DEV)
    most.scatter_reduce_(0, into.view(-1, 1, 1).expand(-1, 2, H), x.abs().amax(-1), "amax")
    kept = torch.full((N,), B, device=DEV).scatter_reduce_(0, into, slot, "amin")
    fresh = torch.where(most >= SMALLEST, most / 127.0, 0.0)
    before = torch.where((kept > 0).view(-1, 1, 1), s["scales"][block], 0.0)
    scales = torch.maximum(before, fresh)
    codes = s["codes"][block].float() - 128.0
    shrunk = torch.round(codes * (before / scales)[..., None, None])
    there = torch.arange(B, device=DEV) < kept.view(-1, 1)
    coarser = (scales > before)[..., None, None] & there.view(N, 1, 1, B, 1)
    codes = torch.where(coarser, shrunk, codes)
    inverse = torch.where(scales > 0, 1.0 / scales, 0.0)[into].unsqueeze(-1)
    codes[into, :, :, slot] = torch.round(x * inverse).clamp(-127, 127)
    s["codes"][block] = (codes + 128.0).to(torch.uint8)
    s["scales"][block] = scales


def _read(s):
    B = s["case"]["B"]
    block, slot = s["table"][s["back_seq"], s["back_pos"] // B].long(), s["back_pos"] % B
    x = (s["codes"][block, :, :, slot].float() - 128.0) * s["scales"][block].unsqueeze(-1)
    return {"k": x[:, 0].to(s["k_out"].dtype), "v": x[:, 1].to(s["k_out"].dtype)}


def _attend(s):
    """All sequences at once, queries and contexts padded to the longest."""
    c, q = s["case"], s["q"]
    S, H, G, D, B = c["S"], c["H"], c["G"], c["D"], c["B"]
    seq, at = s["seq"], s["at"]
    n, L = max(s["n"]), s["table"].shape[1] * B
    k, v = (x.transpose(1, 2).reshape(S, H, L, D) for x in _values(s, s["table"].clamp(min=0).long()))
    qp = torch.zeros((S, n, H * G, D), device=DEV)
    qp[seq, at] = q[: len(seq)].float()
    qp = qp.view(S, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * n, D)
    score = (qp @ k.transpose(2, 3)).view(S, H, G, n, L) * D ** -0.5
    length = s["lens"].view(S, 1, 1).long()
    t = torch.arange(L, device=DEV)
    seen = (t < length).expand(S, n, L)
    if c["causal"]:
        p = (length - (s["offsets"][1:] - s["offsets"][:-1]).view(S, 1, 1) + torch.arange(n, device=DEV).view(1, n, 1))
        seen = seen & (t <= p)
        if c["window"]:
            seen = seen & (t > p - c["window"])
    score = score.masked_fill_(~seen.view(S, 1, 1, n, L), float("-inf"))
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top > float("-inf"), top, 0.0))
    total = e.sum(-1, keepdim=True)
    e = (e / torch.where(total > 0, total, 1.0)).view(S, H, G * n, L)
    o = (e @ v).view(S, H, G, n, D).permute(0, 3, 1, 2, 4).reshape(S, n, H * G, D)
    lse = (torch.log(total) + top).view(S, H, G, n).permute(0, 3, 1, 2).reshape(S, n, H * G)
    s["out"][: len(seq)] = o[seq, at].to(q.dtype)
    s["lse"][: len(seq)] = lse[seq, at]
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "attend":
            return _attend(s)
        if c["op"] == "write":
            _write(s)
        return _read(s)
    import binary_packed_weight_gb300 as bpw
    if c["op"] == "attend":
        bpw.kv8_attention(s["cache"], s["batch"], s["q"], s["out"], s["lse"], causal=c["causal"], window=c["window"],
                          max_q=max(s["n"]))
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "write":
        bpw.kv8_write(s["cache"], s["batch"], s["k"], s["v"])
    bpw.kv8_read(s["cache"], s["back_batch"], s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


# -------------------------------------------------------------------- work ----
def work(case):
    c = case
    n, total = _lengths(c)
    H, D, B, size = c["H"], c["D"], c["B"], BYTES[c["type"]]
    if c["op"] == "read":
        tokens = sum(n)
        return {"bytes": 2 * H * tokens * D * (1 + size) + 8 * H * sum(-(-t // B) for t in total), "flops": 2.0 * H * tokens * D}
    if c["op"] == "write":
        tokens, kept = sum(n), sum((t - k) % B for k, t in zip(n, total))
        return {"bytes": 2 * H * D * (tokens * (size + 1 + size) + kept * (2 + size)), "flops": 8.0 * H * D * tokens}
    window, pairs, tokens = c["window"], 0, 0
    for k, t in zip(n, total):
        if not c["causal"]:
            pairs, tokens = pairs + k * t, tokens + (t if k else 0)
            continue
        p = np.arange(max(t - k, 0), t)                       # the queries' positions
        seen = np.minimum(p + 1, window) if window else p + 1
        pairs += int(seen.sum())
        tokens += int(t - max(0, t - k - window + 1 if window else 0)) if k and t else 0
    rows = sum(n) * H * c["G"]
    return {"bytes": 2 * H * tokens * D + 8 * H * tokens / B + rows * (2 * size * D + 4), "flops": 4.0 * pairs * H * c["G"] * D}


# ----------------------------------------------------------- from the definition ----
def _exact_written(s):
    """Codes and scales after a write, block by block; scales and products are 32-bit by definition."""
    c, B = s["case"], s["case"]["B"]
    codes, scales = s["codes"].clone(), s["scales"].clone()
    table = s["table"].tolist()
    offsets = s["offsets"].tolist()
    for i, (n, total) in enumerate(zip(s["n"], s["total"])):
        start = total - n
        for b in range(start // B, -(-total // B)) if n else ():
            lo, hi = max(start, b * B), min(total, (b + 1) * B)
            p, rows = table[i][b], slice(offsets[i] + lo - start, offsets[i] + hi - start)
            for j, x in enumerate((s["k"][rows], s["v"][rows])):
                x = x.double()
                peak = x.abs().amax((0, 2))
                want = torch.where(peak >= SMALLEST, peak / 127.0, 0.0).float()
                had = scales[p, j] if lo > b * B else torch.zeros_like(want)
                now = torch.maximum(had, want)
                if lo > b * B:
                    ratio = (had.double() / now.double()).float().double()
                    kept = codes[p, j, :, : lo - b * B].double() - 128
                    kept = torch.where((now > had)[:, None, None], (kept * ratio[:, None, None]).round(), kept)
                    codes[p, j, :, : lo - b * B] = (kept + 128).to(torch.uint8)
                inv = torch.where(now > 0, (1.0 / now.double()).float().double(), 0.0)
                y = (x * inv[None, :, None]).float().double().round().clamp(-127, 127)
                codes[p, j, :, lo - b * B: hi - b * B] = (y + 128).to(torch.uint8).transpose(0, 1)
                scales[p, j] = now
    return codes, scales


def exact(case, seed):
    c, s = case, prepare(case, seed)
    B, H, D = c["B"], c["H"], c["D"]
    codes, scales = _exact_written(s) if c["op"] == "write" else (s["codes"], s["scales"])
    table, n, total = s["table"].long(), s["n"], s["total"]

    def context(i, head, j, lo, hi):
        p = table[i, lo // B: -(-hi // B)]
        x = (codes[p, j, head].double() - 128.0) * scales[p, j, head].double()[:, None, None]
        return x.reshape(-1, D)[lo - lo // B * B:][: hi - lo]

    if c["op"] != "attend":
        back = s["back"].tolist()
        out = torch.empty((2, back[-1], H, D), dtype=torch.float64, device=DEV)
        for i in range(c["S"]):
            count = back[i + 1] - back[i]
            for head in range(H if count else 0):
                for j in (0, 1):
                    out[j, back[i]: back[i + 1], head] = context(i, head, j, total[i] - count, total[i])
        return {"k": out[0], "v": out[1]}
    rows, G = s["q"].shape[0], c["G"]
    out = torch.zeros((rows, H * G, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((rows, H * G), dtype=torch.float64, device=DEV)
    offsets = s["offsets"].tolist()
    for i in range(c["S"]):
        r = slice(offsets[i], offsets[i + 1])
        if n[i] == 0:
            continue
        if total[i] == 0:
            lse[r] = float("-inf")
            continue
        t = torch.arange(total[i], device=DEV)
        p = torch.arange(total[i] - n[i], total[i], device=DEV).unsqueeze(1)
        dead = torch.zeros((n[i], total[i]), dtype=torch.bool, device=DEV)
        if c["causal"]:
            dead = t > p
            if c["window"]:
                dead |= t <= p - c["window"]
        empty = dead.all(1, keepdim=True)
        for head in range(H):
            k, v = context(i, head, 0, 0, total[i]), context(i, head, 1, 0, total[i])
            for h in range(head * G, (head + 1) * G):
                z = s["q"][r, h].double() @ k.T / math.sqrt(D)
                z = z.masked_fill(dead, float("-inf"))
                l = torch.logsumexp(z, 1, keepdim=True)
                out[r, h] = torch.where(empty, 0.0, torch.exp(z - l)) @ v
                lse[r, h] = l[:, 0]
    return {"out": out, "lse": lse}
