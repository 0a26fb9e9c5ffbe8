"""GPU parity of the router, its gradient and the routed experts against the f64 oracle.

Ids and the plan are equal, whatever is masked.  Bounds (derived before the
first run): a score is a handful of f32 operations (exp within 2 ulp, a sum of
at most 1024 positives as a tree of depth 10, a division), so weights are
within 2^-19 of their size; their gradient adds sums over at most 32 terms
whose absolute sum scales it.  Products are bounded as in test_gpu_q4.py; with
many tokens an expert (f16, bf16) the weights are rounded to f16 as well, up to
2^-11 of each, and one accumulator runs over all of k, K/16 steps of 2^-22.
"""
import numpy as np
import pytest

from oracle import moe as omoe
from oracle import q4 as oq4
from test_gpu_q4 import HALF_ULP, planes, upload

pytestmark = pytest.mark.gpu


def grid_logits(rng, T, E, dtype, masked):
    """Logits a step apart within a row (exact in every type), some equal, some masked in every way."""
    l = np.array([rng.permutation(E) for _ in range(T)]) * 0.0625 - 0.03125 * E
    if E > 8:
        l[:, 5] = l[:, 2]                                             # exact ties
    if masked:
        l[rng.random((T, E)) < 0.2] = -np.inf
        l[rng.random((T, E)) < 0.05] = np.nan
        l[rng.random(T) < 0.1] = -np.inf                              # rows that nothing is left of
    return l


def run_route(lib, l, k, dtype="float32", bias=None, plan=True, pad=0, **kw):
    import torch
    T, E = l.shape
    buf = torch.full((T, E + pad), float("nan"), dtype=getattr(torch, dtype), device="cuda")
    buf[:, :E] = torch.from_numpy(l).to(buf.dtype)
    ids = torch.full((T, k), 99, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    off = torch.full((E + 1,), 99, dtype=torch.int32, device="cuda") if plan else None
    slots = torch.full((T * k,), 99, dtype=torch.int32, device="cuda") if plan else None
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    lib.moe_route(buf[:, :E], ids, w, off, slots, bias=b, **kw)
    torch.cuda.synchronize()
    return ids, w, off, slots


def check_route(lib, l, k, dtype="float32", **kw):
    ids, w, off, slots = run_route(lib, l, k, dtype, **kw)
    kw.pop("pad", None)
    want_ids, want_w = omoe.route(l, k, **kw)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert np.all(np.abs(w.cpu().double().numpy() - want_w) <= 2.0 ** -19 * np.abs(want_w))
    want_off, want_slots = omoe.plan(want_ids, l.shape[1])
    assert np.array_equal(off.cpu().numpy(), want_off)
    assert np.array_equal(slots.cpu().numpy(), want_slots)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 6), (3, 5, 5), (31, 60, 4), (32, 33, 2), (33, 160, 6),
                                   (200, 17, 8), (70, 600, 3), (40, 1024, 32)])
def test_route(lib, score, renorm, T, E, k):
    rng = np.random.default_rng(T * 1000 + E)
    for masked in (False, True):
        check_route(lib, grid_logits(rng, T, E, "float32", masked), k, score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_route_types_and_strides(lib, dtype, pad):
    rng = np.random.default_rng(3)
    for T, E in ((5, 64), (50, 56)):
        check_route(lib, grid_logits(rng, T, E, dtype, True), 6, dtype, pad=pad, score="softmax")


@pytest.mark.parametrize("E,groups,top", [(32, 4, 2), (256, 8, 4), (160, 8, 3), (60, 4, 1), (64, 32, 5), (64, 1, 1),
                                          (24, 24, 7), (64, 4, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_with_bias(lib, E, groups, top, score):
    rng = np.random.default_rng(E + groups)
    bias = rng.permutation(E) * 0.0013 - 0.02
    bias[1] = -np.inf
    k = min(6, top * (E // groups))
    for T, masked in ((7, True), (90, False), (90, True)):
        check_route(lib, grid_logits(rng, T, E, "float32", masked), k, score=score, bias=bias, groups=groups,
                    top_groups=top)


def test_route_ties_and_extremes(lib):
    most = float(np.finfo(np.float32).max)
    rows = np.zeros((6, 16))                                          # row 0: all equal
    rows[1] = -most                                                   # masks of the type's lowest value: still there
    rows[2] = -most
    rows[2, 9] = 0.0
    rows[3] = -np.inf
    rows[3, 4] = np.inf                                               # an infinite logit takes everything
    rows[4] = np.nan
    rows[5] = np.linspace(-200.0, 200.0, 16)                          # scores that underflow
    for score in ("softmax", "sigmoid"):
        check_route(lib, rows[:2], 5, score=score, groups=4, top_groups=2)
        ids, w, _, _ = run_route(lib, rows, 4, score=score)
        ids, w = ids.cpu().numpy(), w.cpu().numpy()
        assert ids[0].tolist() == [0, 1, 2, 3] and np.allclose(w[0], 0.25)
        assert ids[2, 0] == 9 and w[2, 0] == 1.0 and not w[2, 1:].any()
        assert ids[3].tolist() == [4, -1, -1, -1] and w[3].tolist() == [1.0, 0.0, 0.0, 0.0]
        assert ids[4].tolist() == [-1] * 4 and not w[4].any()
        assert np.all(np.isfinite(w))
    assert run_route(lib, rows, 4)[0][5].tolist()[0] == 15


def test_route_many_tokens(lib):
    """Many chunks: the plan against a stable sort of the ids."""
    import torch
    rng = np.random.default_rng(8)
    for T, E, k in ((5000, 64, 8), (20011, 96, 3), (3000, 1000, 12)):
        l = rng.normal(size=(T, E))
        l[rng.random(T) < 0.05] = -np.inf
        ids, w, off, slots = run_route(lib, l, k)
        flat = ids.reshape(-1).long()
        key = torch.where(flat < 0, E, flat)
        want = torch.sort(key, stable=True)
        n = int((flat >= 0).sum())
        assert torch.equal(slots[:n].long(), want[1][:n]) and bool((slots[n:] == -1).all())
        assert torch.equal(off.long(), torch.searchsorted(want[0], torch.arange(E + 1, device="cuda")))
        p = torch.from_numpy(l).float().cuda()
        v, i = p.sort(dim=-1, descending=True, stable=True)
        rows = v[:, 0] > -np.inf
        assert torch.equal(ids[rows].long(), i[rows, :k])


@pytest.mark.parametrize("E", [1, 3])
def test_route_most_tokens(lib, E):
    """2^24 slots; of one expert, every count of a plan's chunk is as large as it gets."""
    import torch
    T = 1 << 24
    gen = torch.Generator(device="cuda").manual_seed(17)
    logits = torch.randn((T, E), device="cuda", generator=gen).half()
    logits[T // 4:T // 2, 1:] = -float("inf")
    ids, w = torch.empty((T, 1), dtype=torch.int32, device="cuda"), torch.empty((T, 1), device="cuda")
    off, slots = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(T, dtype=torch.int32, device="cuda")
    lib.moe_route(logits, ids, w, off, slots)
    lib.device_status()
    top = logits.float().max(1, keepdim=True).values
    want = (logits.float() == top).to(torch.uint8).argmax(1)              # the first of equals
    assert torch.equal(ids[:, 0].long(), want)
    counts = torch.bincount(want, minlength=E)
    assert off.tolist() == [0] + torch.cumsum(counts, 0).tolist()
    assert torch.equal(slots.long(), torch.sort(want, stable=True).indices)


def test_route_empty_and_without_plan(lib):
    import torch
    off = torch.full((9,), 5, dtype=torch.int32, device="cuda")
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    w = torch.empty((0, 2), device="cuda")
    lib.moe_route(torch.empty((0, 8), device="cuda"), ids, w, off, torch.empty((0,), dtype=torch.int32, device="cuda"))
    assert not off.any()
    rng = np.random.default_rng(9)
    l = grid_logits(rng, 40, 8, "float32", True)
    ids, w, _, _ = run_route(lib, l, 2, plan=False)
    assert np.array_equal(ids.cpu().numpy(), omoe.route(l, 2)[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_route_backward(lib, score, renorm, dtype):
    import torch
    rng = np.random.default_rng(12)
    for T, E, k, pad in ((1, 1, 1, 0), (5, 60, 4, 0), (37, 64, 8, 3), (9, 1000, 32, 0), (300, 128, 2, 8)):
        for biased in (False, True):
            l = grid_logits(rng, T, E, dtype, E > 1) * (0.1 if E > 100 else 1.0)
            bias = rng.normal(size=E) * 0.01 if biased else None
            dt = getattr(torch, dtype)
            buf = torch.zeros((T, E + pad), dtype=dt, device="cuda")
            buf[:, :E] = torch.from_numpy(l).to(dt)
            seen = buf[:, :E].cpu().double().numpy()
            ids, _ = omoe.route(seen, k, score=score, bias=bias)
            dw = rng.normal(size=(T, k)).astype(np.float32)
            out = torch.full((T, E + pad), 7.0, dtype=dt, device="cuda")
            lib.moe_route_backward(buf[:, :E], torch.from_numpy(ids).int().cuda(), torch.from_numpy(dw).cuda(),
                                   out[:, :E], score=score, renorm=renorm, scale=2.5,
                                   bias=None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda())
            got = out.cpu().double().numpy()
            assert np.all(got[:, E:] == 7.0)
            want = omoe.route_backward(seen, ids, dw, score=score, renorm=renorm, scale=2.5, bias=bias)
            # what cancels in the formula: |p_e| (|q_e| + sum |g p|/S) with |q| <= (|g| + sum|g p|/S)/S
            p = np.array([omoe.scores(r, bias, score)[0] for r in seen])
            on = ids >= 0
            ps = np.where(on, np.take_along_axis(p, np.maximum(ids, 0), 1), 0.0)
            g = np.abs(np.where(on, dw, 0.0)) * 2.5
            S = np.maximum(ps.sum(1, keepdims=True), omoe.TINY) if renorm else 1.0
            tot = (g * ps).sum(1, keepdims=True) / S
            size = np.zeros_like(p)
            np.add.at(size, (np.arange(T)[:, None] + np.zeros_like(ids), np.maximum(ids, 0)), np.where(on, g / S, 0.0))
            size = p * (size + tot / S if renorm else size + tot)
            bound = 2.0 ** -18 * size + HALF_ULP[dtype] * np.abs(want) + (2.0 ** -25 if dtype == "float16" else 0.0)
            assert np.all(np.abs(got[:, :E] - want) <= bound), (T, E, k, biased)


def run_experts(lib, x, ids, weights, w3, dtype, E, pad=0):
    import torch
    dt = getattr(torch, dtype)
    T, D = x.shape
    xb = torch.full((T, D + pad), float("nan"), dtype=dt, device="cuda")
    xb[:, :D] = torch.from_numpy(x).to(dt)
    off, slots = omoe.plan(ids, E)
    ob = torch.full((T, D + pad), 7.0, dtype=dt, device="cuda")
    lib.moe_experts(*w3, xb[:, :D], torch.from_numpy(ids).int().cuda(), torch.from_numpy(weights).float().cuda(),
                    torch.from_numpy(off).int().cuda(), torch.from_numpy(slots).int().cuda(), ob[:, :D])
    lib.device_status()
    got = ob.cpu().double().numpy()
    assert np.all(got[:, D:] == 7.0)
    return xb[:, :D].cpu().double().numpy(), got[:, :D]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("T,E,k,D,F,group,zeros", [(1, 4, 2, 256, 128, 128, False), (1, 1, 1, 128, 32, 32, True),
                                                   (6, 8, 3, 384, 96, 32, True), (40, 5, 2, 256, 320, 64, False),
                                                   (90, 3, 3, 128, 64, 32, False), (17, 16, 4, 288, 1056, 32, True),
                                                   (600, 2, 1, 384, 96, 32, True), (300, 4, 2, 544, 352, 32, False),
                                                   (130, 1, 1, 256, 1024, 128, True), (700, 3, 2, 64, 192, 64, True)])
def test_experts(lib, dtype, T, E, k, D, F, group, zeros):
    rng = np.random.default_rng(T + E)
    mats, handles = [], []
    for N, K in ((F, D), (F, D), (D, F)):
        c, d, z = planes(rng, E, N, K, group, zeros)
        mats.append(oq4.dequant(c, d.view(np.uint16), z, group))
        handles.append(upload(lib, c, d, z, group))
    # uneven loads: some experts get nearly all, one none, one token none
    pref = rng.random(E) ** 3
    ids = np.array([rng.permutation(E)[:k] if i % 3 else np.argsort(-pref - 0.05 * rng.random(E))[:k]
                    for i in range(T)])
    if T > 1:
        ids[T // 2] = -1
        ids[0, k - 1] = -1
    weights = rng.random((T, k)).astype(np.float32)
    x, got = run_experts(lib, rng.normal(size=(T, D)) * 0.2, ids, weights, handles, dtype, E, pad=5 if T == 6 else 0)
    want = omoe.experts(x, ids, weights, *mats)
    eps = (8 + max(D, F) / group + 16) * 2.0 ** -22 + 2.0 ** -22
    if dtype != "float32" and T * k >= 32 * E:                        # the path of many tokens an expert
        eps = 2.0 ** -11 + (max(D, F) / 16 + 16) * 2.0 ** -22
    bound = omoe.experts_bound(x, ids, weights, *mats, eps, eps, 2.0 ** -20 if dtype == "float32" else 2.0 ** -11)
    bound = 1.01 * bound + (k * 2.0 ** -23) * np.abs(bound) + (HALF_ULP[dtype] + k * 2.0 ** -22) * np.abs(want) + 1e-7
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} off, worst {np.max(np.abs(got - want) / bound):.3g} of the bound"


@pytest.mark.parametrize("magnitude", [1e-12, 1e-4, 1e4])
def test_experts_many_tokens_of_any_magnitude(lib, magnitude):
    """The f16 operands of the path of many tokens are scaled by row: rows of any size come out alike."""
    rng = np.random.default_rng(21)
    E, T, D, F = 2, 100, 256, 128
    mats, handles = [], []
    for N, K in ((F, D), (F, D), (D, F)):
        c, d, z = planes(rng, E, N, K, 128, True)
        mats.append(oq4.dequant(c, d.view(np.uint16), z, 128))
        handles.append(upload(lib, c, d, z, 128))
    ids = np.arange(T)[:, None] % E
    x0 = rng.normal(size=(T, D))
    x0[: T // 2] *= magnitude                                         # beside rows of ordinary size
    x, got = run_experts(lib, x0, ids, np.ones((T, 1)), handles, "bfloat16", E)
    want = omoe.experts(x, ids, np.ones((T, 1)), *mats)
    eps = 2.0 ** -11 + (D / 16 + 16) * 2.0 ** -22
    bound = omoe.experts_bound(x, ids, np.ones((T, 1)), *mats, eps, eps, 2.0 ** -11)
    bound = 1.02 * bound + 2.0 ** -8 * np.abs(want) + 1e-36
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("seed", [0, 1])
def test_experts_tiles_of_every_width(lib, seed):
    """Several tiles of very different widths one after the other in each CTA; positions beside the widths' limits
    are compared (one expert a token, so that a token is a position)."""
    rng = np.random.default_rng(30 + seed)
    E, D, F, group = 40, 576, 832, 64
    counts = [384, 385, 320, 321, 256, 257, 1, 0, 2, 31, 33, 64, 97, 128, 160, 255, 300, 352, 383, 511, 512, 513, 768, 769]
    counts = rng.permutation(counts + list(rng.integers(200, 400, E - len(counts))))
    mats, handles = [], []
    for N, K in ((F, D), (F, D), (D, F)):
        c, d, z = planes(rng, E, N, K, group, True)
        mats.append(oq4.dequant(c, d.view(np.uint16), z, group))
        handles.append(upload(lib, c, d, z, group))
    ids = rng.permutation(np.repeat(np.arange(E), counts))[:, None]
    T = len(ids)
    weights = rng.random((T, 1)).astype(np.float32)
    x, got = run_experts(lib, rng.normal(size=(T, D)) * 0.2, ids, weights, handles, "bfloat16", E)
    pick = []
    for e in range(E):
        of = np.flatnonzero(ids[:, 0] == e)
        pick += [of[p] for p in {0, len(of) // 2, len(of) - 1, 127, 255, 256, 319, 320, 383} if 0 <= p < len(of)]
    x, got, ids, weights = x[pick], got[pick], ids[pick], weights[pick]
    want = omoe.experts(x, ids, weights, *mats)
    eps = 2.0 ** -11 + (F / 16 + 16) * 2.0 ** -22
    bound = omoe.experts_bound(x, ids, weights, *mats, eps, eps, 2.0 ** -11)
    bound = 1.02 * bound + (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 1e-7
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} off, worst {np.max(np.abs(got - want) / bound):.3g} of the bound"


@pytest.mark.parametrize("E,T,F", [(4, 40000, 8192), (64, 1600, 12288)])
def test_experts_many_tiles(lib, E, T, F):
    """More tiles than a CTA looks up ahead, wide and narrow ones; sampled tokens of three experts."""
    rng = np.random.default_rng(40 + E)
    D, group = 128, 128
    some = [0, E // 2, E - 1]
    mats, handles = [], []
    for N, K in ((F, D), (F, D), (D, F)):
        c, d, z = planes(rng, E, N, K, group, False)
        mats.append(oq4.dequant(c[some], d[some].view(np.uint16), z, group))
        handles.append(upload(lib, c, d, z, group))
    ids = rng.integers(0, E, (T, 1))
    weights = rng.random((T, 1)).astype(np.float32)
    x, got = run_experts(lib, rng.normal(size=(T, D)) * 0.2, ids, weights, handles, "bfloat16", E)
    of = [np.flatnonzero(ids[:, 0] == e) for e in some]
    pick = np.concatenate([p[[0, 1, len(p) // 2, -2, -1]] for p in of])
    local = np.repeat(np.arange(3), 5)[:, None]
    x, got, weights = x[pick], got[pick], weights[pick]
    want = omoe.experts(x, local, weights, *mats)
    eps = 2.0 ** -11 + (F / 16 + 16) * 2.0 ** -22
    bound = omoe.experts_bound(x, local, weights, *mats, eps, eps, 2.0 ** -11)
    bound = 1.02 * bound + (2.0 ** -8 + 2.0 ** -22) * np.abs(want) + 1e-7
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("T,E,k,D,F,group,zeros", [(9, 2, 1, 32, 32, 32, True), (5, 3, 3, 64, 160, 32, False),
                                                   (31, 7, 1, 416, 96, 32, True), (21, 4, 1, 320, 448, 64, False),
                                                   (26, 5, 2, 640, 128, 128, True), (43, 1, 3, 192, 64, 64, True)])
def test_experts_of_few_rows(lib, dtype, T, E, k, D, F, group, zeros):
    """Between 4 and 130 rows an expert; some slots are not routed, and with one expert the rest of a token's."""
    rng = np.random.default_rng(50 + T)
    mats, handles = [], []
    for N, K in ((F, D), (F, D), (D, F)):
        c, d, z = planes(rng, E, N, K, group, zeros)
        mats.append(oq4.dequant(c, d.view(np.uint16), z, group))
        handles.append(upload(lib, c, d, z, group))
    ids = rng.integers(0, E, (T, k))
    ids[T // 3, 0] = -1
    weights = rng.random((T, k)).astype(np.float32)
    x, got = run_experts(lib, rng.normal(size=(T, D)) * 0.2, ids, weights, handles, dtype, E, pad=3)
    want = omoe.experts(x, ids, weights, *mats)
    eps = 2.0 ** -11 + (max(D, F) / 16 + 16) * 2.0 ** -22
    bound = omoe.experts_bound(x, ids, weights, *mats, eps, eps, 2.0 ** -11)
    bound = 1.02 * bound + (HALF_ULP[dtype] + k * 2.0 ** -22) * np.abs(want) + 1e-7
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} off, worst {np.max(np.abs(got - want) / bound):.3g} of the bound"


def test_experts_no_tokens_and_no_slots(lib):
    import torch
    rng = np.random.default_rng(4)
    h = [upload(lib, *planes(rng, 2, N, K, 32, False), 32) for N, K in ((64, 128), (64, 128), (128, 64))]
    ids = np.full((3, 2), -1)
    _, got = run_experts(lib, rng.normal(size=(3, 128)), ids, np.ones((3, 2)), h, "bfloat16", 2)
    assert not got.any()
    e = torch.empty((0, 128), device="cuda")
    i = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    lib.moe_experts(*h, e, i, i.float(), torch.zeros(3, dtype=torch.int32, device="cuda"), i.reshape(-1), e.clone())


def test_experts_refusals(lib):
    import torch
    rng = np.random.default_rng(5)
    g, u, d = [upload(lib, *planes(rng, 2, N, K, 32, False), 32) for N, K in ((64, 128), (64, 128), (128, 64))]
    other = upload(lib, *planes(rng, 2, 96, 128, 32, False), 32)
    x, out = torch.zeros((3, 128), device="cuda"), torch.zeros((3, 128), device="cuda")
    ids, w = torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.zeros((3, 2), device="cuda")
    off, slots = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.full((6,), -1, dtype=torch.int32, device="cuda")
    for bad in ((g, other, d), (g, u, g)):
        with pytest.raises(lib.TQ2Error) as info:
            lib.moe_experts(*bad, x, ids, w, off, slots, out)
        assert info.value.status == 2
    with pytest.raises(ValueError):
        lib.moe_experts(g, u, d, x, ids, w, off[:2], slots, out)
    with pytest.raises(ValueError):
        lib.moe_experts(g, u, d, x, ids.long(), w, off, slots, out)
    with pytest.raises(ValueError):
        lib.moe_route(torch.zeros((3, 8), device="cuda"), ids, w, score="tanh")
    with pytest.raises(lib.TQ2Error):
        lib.moe_route(torch.zeros((3, 8), device="cuda"), ids, w, groups=3)


def test_experts_too_many_for_one_call(lib):
    """Refused before anything is allocated or read (the tensors are views of one row)."""
    import torch
    rng = np.random.default_rng(15)
    g, u, d = [upload(lib, *planes(rng, 1, N, K, 128, False), 128) for N, K in ((128, 4096), (128, 4096), (4096, 128))]
    T, k = 1 << 19, 16
    x = torch.zeros((1, 4096), dtype=torch.bfloat16, device="cuda").expand(T, 4096)
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    off, slots = torch.zeros(2, dtype=torch.int32, device="cuda"), ids.reshape(-1)
    rc = lib.load().moe_experts(g.handle, u.handle, d.handle, x.data_ptr(), 4096, 2, ids.data_ptr(), ids.data_ptr(),
                                off.data_ptr(), slots.data_ptr(), x.data_ptr(), 4096, T, k, None)
    assert rc == 2


@pytest.mark.parametrize("T", [6, 120])
@pytest.mark.parametrize("kind", ["back and forth", "out of range"])
def test_experts_of_no_plan_stay_inside(lib, T, kind):
    """offsets and slots that are no plan: the result is unspecified, but nothing beside out is written."""
    import torch
    rng = np.random.default_rng(16)
    E, k, D, F = 8, 2, 128, 64
    h = [upload(lib, *planes(rng, E, N, K, 32, False), 32) for N, K in ((F, D), (F, D), (D, F))]
    S = T * k
    off = [0, S] * 4 + [0] if kind == "back and forth" else [-9] * 4 + [3 * S] * 5
    slots = rng.integers(0, S, S) if kind == "back and forth" else rng.choice([-5, S, 10 ** 9], S)
    x = torch.randn((T, D), device="cuda").to(torch.bfloat16)
    buf = torch.full((T + 2, D + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    ids = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32)).cuda()
    lib.moe_experts(*h, x, ids, torch.ones((T, k), device="cuda"), torch.tensor(off, dtype=torch.int32, device="cuda"),
                    torch.from_numpy(slots.astype(np.int32)).cuda(), buf[1:T + 1, 8:D + 8])
    lib.device_status()
    assert bool((buf[0] == 7).all() and (buf[-1] == 7).all() and (buf[:, :8] == 7).all() and (buf[:, -8:] == 7).all())


def test_route_feeds_experts(lib):
    """The two together, as a layer: logits -> plan -> experts, twice with the same bits."""
    import torch
    rng = np.random.default_rng(6)
    E, k, D, F, T = 8, 2, 256, 128, 50
    mats, handles = [], []
    for N, K in ((F, D), (F, D), (D, F)):
        c, d, z = planes(rng, E, N, K, 128, True)
        mats.append(oq4.dequant(c, d.view(np.uint16), z, 128))
        handles.append(upload(lib, c, d, z, 128))
    l = grid_logits(rng, T, E, "float32", True)
    x = torch.from_numpy(rng.normal(size=(T, D)) * 0.2).to(torch.bfloat16).cuda()
    outs = []
    for _ in range(2):
        ids, w, off, slots = run_route(lib, l, k)
        out = torch.empty_like(x)
        lib.moe_experts(*handles, x, ids, w, off, slots, out)
        outs.append(out.cpu())
    assert torch.equal(outs[0], outs[1])
    want = omoe.experts(x.cpu().double().numpy(), ids.cpu().numpy(), w.cpu().numpy(), *mats)
    err = np.linalg.norm(outs[0].double().numpy() - want) / np.linalg.norm(want)
    assert err < 2.0 ** -8
