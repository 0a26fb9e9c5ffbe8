"""Cases and bounds of the tests of the 8-bit cache."""
import numpy as np

from oracle import kv8

HALF_ULP = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


class Cache:
    """A random pool with stale contents everywhere, a table that hands its blocks out in no order, and both on the GPU."""

    def __init__(self, lib, rng, lens, n, H=2, D=64, B=16, spare=3, width=None, first=0, spread=1.0):
        import torch
        self.lens, self.offsets = np.array(lens, np.int32), np.concatenate(([0], np.cumsum(n))).astype(np.int32)
        need = [-(-t // B) for t in lens]
        P = first + sum(need) + spare
        order = first + rng.permutation(P - first)
        self.table = np.full((len(lens), width or max(max(need), 1)), -1, np.int32)
        at = 0
        for s, k in enumerate(need):
            self.table[s, :k] = order[at:at + k]
            at += k
        self.codes = rng.integers(1, 256, (P, 2, H, B, D), dtype=np.uint8)
        self.scales = (rng.uniform(0.5, 1.5, (P, 2, H)) * 2.0 ** rng.uniform(-spread, spread, (P, 2, H)) / 64).astype(np.float32)
        self.lib, self.H, self.D, self.B, self.T = lib, H, D, B, int(self.offsets[-1])
        if lib is not None:
            self.d = {k: torch.from_numpy(getattr(self, k)).cuda() for k in ("codes", "scales", "table", "offsets", "lens")}
            self.cache = lib.KV8Cache(self.d["codes"], self.d["scales"])
            self.batch = lib.KV8Batch(self.d["table"], self.d["offsets"], self.d["lens"])

    def on_gpu(self):
        """Codes and scales as the GPU holds them."""
        return self.d["codes"].cpu().numpy(), self.d["scales"].cpu().numpy()

    def upload(self):
        import torch
        for k in self.d:
            self.d[k].copy_(torch.from_numpy(getattr(self, k)))

    def attend(self, q, dtype, pad=0, beside=(0, 0), lse=True, **options):
        """q float64 numpy [T, Hq, D] rounded to dtype -> (q as the call saw it, out, lse), float64; pad: rows of no
        sequence behind the last, beside: heads more than there are and elements a row starts off."""
        import torch
        dt = getattr(torch, dtype)
        T, Hq, D = q.shape
        more, shift = beside
        qb = torch.full((T + pad, (Hq + more) * D + shift), 3.0, dtype=dt, device="cuda")
        ob = torch.full_like(qb, 7.0)
        view = [b[:, shift:].view(T + pad, Hq + more, D)[:, :Hq] if not shift else
                b.as_strided((T + pad, Hq, D), (b.stride(0), D, 1), shift) for b in (qb, ob)]
        view[0][:T].copy_(torch.from_numpy(q).to(dt))
        l = torch.full((T + pad, Hq), 5.0, device="cuda") if lse else None
        self.lib.kv8_attention(self.cache, self.batch, view[0], view[1], l, **options)
        self.lib.device_status()
        rest = ob.clone()
        rest.as_strided((T, Hq, D), (ob.stride(0), D, 1), shift).fill_(7.0)
        assert bool((rest == 7.0).all())                       # nothing beside the rows
        assert l is None or bool((l[T:] == 5.0).all())
        return (view[0][:T].cpu().double().numpy(), view[1][:T].cpu().double().numpy(),
                None if l is None else l[:T].cpu().double().numpy())


def check_attention(got, lse, want, dtype, D, L, where=""):
    """Bound, with A the largest scale * sum |q k| of a row and L its tokens.
    A score is off by (D/16 + 6) steps of 2^-22 A (sums of 16 products that may truncate; f32 queries and the factors
    2^-22 more each) and by 2^-23 of the exponent's range it is added to, at most 2 A + 8 + log2 L wide;
    a weight by twice that, the exponential's 2^-21 and its rounding (f16 2^-11 for bf16 results, two parts 2^-21; at least 2^-30 of the
    largest weight times its block's scale, of a code of 127).  The sums add L/16 + 64 steps of 2^-22.  Then
    half a step of the output's type."""
    A, top, spread = want["score"], want["top"], want["spread"]
    score = (D / 16 + 6) * 2.0 ** -22 * A + 2.0 ** -23 * (2 * A + 8 + np.log2(max(L, 2)))
    sums = (L / 16 + 64) * 2.0 ** -22
    weight = 2 * score + 2.0 ** -21 + (2.0 ** -11 if dtype == "bfloat16" else 2.0 ** -21)
    bound = (weight + sums)[..., None] * spread + (2.0 ** -30 * 127 * L * top)[..., None]
    bound = bound + HALF_ULP[dtype] * np.abs(want["out"]) + (2.0 ** -24 if dtype == "float16" else 1e-37)
    rows = want["rows"]
    bad = ~(np.abs(got - want["out"]) <= bound)[rows]
    assert not bad.any(), f"{where}: {bad.sum()} of {bad.size} off, {np.nanmax((np.abs(got - want['out']) / bound)[rows]):.3g} of the bound"
    if lse is not None:
        w = want["lse"]
        none = np.isneginf(w)
        assert np.array_equal(np.isneginf(lse[rows]), none[rows]), where
        off = np.abs(np.where(none, 0, lse) - np.where(none, 0, w))
        bad = ~(off <= score + sums + 2.0 ** -21 + 2.0 ** -22 * np.abs(np.where(none, 0, w)))[rows]
        assert not bad.any(), f"{where}: lse of {bad.sum()} rows off, worst {np.nanmax(off[rows]):.3g}"


def queries(rng, T, Hq, D):
    q = rng.normal(size=(T, Hq, D)) * 1.5
    q[:, :, rng.integers(0, D)] *= 4
    return q


def attention_of(c, q, scale=None, **options):
    return kv8.attention(q, c.codes, c.scales, c.table, c.offsets, c.lens, c.D ** -0.5 if scale is None else scale, **options)
