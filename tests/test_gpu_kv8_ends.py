"""The 8-bit cache at the ends of what its arguments may be, against the f64 oracle.

The bound of the attention is derived in kv8_util.check_attention.
"""
import numpy as np
import pytest

from kv8_util import Cache, attention_of, check_attention, queries
from oracle import kv8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,n", [("float32", 1), ("float16", 1), ("float16", 3), ("bfloat16", 1), ("bfloat16", 3)])
@pytest.mark.parametrize("D,B", [(64, 16), (128, 128)])
def test_rings_that_go_round_many_times(lib, dtype, n, D, B):
    """Some 70 chunks a CTA through a ring of four: every repeat has the same bits, and they are right."""
    rng = np.random.default_rng(70)
    lens = rng.integers(3000, 4000, 340)
    c = Cache(lib, rng, [4000] * 2, [n] * 2, H=2, D=D, B=B)
    c.table = c.table[np.arange(340) % 2]                     # many sequences share two sequences' blocks
    c.lens, c.offsets, c.T = lens.astype(np.int32), (np.arange(341) * n).astype(np.int32), 340 * n
    import torch
    c.d = {k: torch.from_numpy(getattr(c, k)).cuda() for k in ("codes", "scales", "table", "offsets", "lens")}
    c.cache, c.batch = lib.KV8Cache(c.d["codes"], c.d["scales"]), lib.KV8Batch(c.d["table"], c.d["offsets"], c.d["lens"])
    q, out, lse = c.attend(queries(rng, c.T, 8, D), dtype, max_q=n)
    some = [0, 1, 170, 339]
    rows = np.concatenate([np.arange(s * n, s * n + n) for s in some])
    c.table, c.lens, c.offsets = c.table[some], c.lens[some], (np.arange(5) * n).astype(np.int32)
    check_attention(out[rows], lse[rows], attention_of(c, q[rows]), dtype, D, 4000)
    c.T = 340 * n
    for _ in range(8):
        again = c.attend(q, dtype, max_q=n)
        assert np.array_equal(again[1], out) and np.array_equal(again[2], lse)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [1, 90])
def test_blocks_that_come_and_go(lib, dtype, n):
    """Slots of the rings hold a block, then none, then one again: what is not there is never taken for what was."""
    rng = np.random.default_rng(71)
    c = Cache(lib, rng, [3000, 2000, 2500], [n] * 3, H=2, D=64, B=16)
    c.table[rng.random(c.table.shape) < 0.4] = -1
    c.upload()
    q, out, lse = c.attend(queries(rng, c.T, 4, 64), dtype)
    check_attention(out, lse, attention_of(c, q), dtype, 64, 3000)
    for _ in range(8):
        again = c.attend(q, dtype)
        assert np.array_equal(again[1], out) and np.array_equal(again[2], lse)


# -------------------------------------------------- scales of values at the ends ----
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -103, 2.0 ** -60])
def test_values_of_zeros_at_length(lib, dtype, n, scale):
    """A million tokens whose values are (about) zeros: their weights add up like any others'.  The longest chain of
    additions is that of test_tens_of_millions_of_tokens, 16 times shorter."""
    import torch
    rng = np.random.default_rng(72)
    c = Cache(lib, rng, [128], [n], H=1, D=64, B=128)
    c.scales[:, 1] = scale
    c.upload()
    blocks = 1 << 13                                          # all of them the same 128 tokens
    c.batch = lib.KV8Batch(c.d["table"].repeat(1, blocks), c.d["offsets"], c.d["lens"] * blocks)
    q, out, lse = c.attend(queries(rng, n, 4, 64) * 0.01, dtype, causal=False)    # of about the same weight
    check_attention(out, lse - np.log(blocks), attention_of(c, q, causal=False), dtype, 64, 16 * 5600)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("G", [1, 40])
@pytest.mark.parametrize("scale", [0.0, 2.0 ** -103, 2.0 ** -20])
def test_weights_that_rise_within_one_piece(lib, dtype, G, scale):
    """Sequences of 12800 tokens, one for every place that works at once; the first 128 tokens weigh 2^7.8 times less."""
    import torch
    rng = np.random.default_rng(73)
    S, blocks, D = 304, 100, 64
    c = Cache(lib, rng, [256], [1], H=1, D=D, B=128)
    first, rest = c.table[0]
    c.codes[:] = 128
    c.codes[rest, 0, 0, :, 0] = 228
    c.codes[:, 1] = rng.integers(1, 256, c.codes[:, 1].shape)
    c.scales[:, 0], c.scales[:, 1] = 0.054, scale
    c.upload()
    table = torch.full((S, blocks), int(rest), dtype=torch.int32, device="cuda")
    table[:, 0] = int(first)
    c.batch = lib.KV8Batch(table, torch.arange(S + 1, dtype=torch.int32, device="cuda"),
                           torch.full((S,), 128 * blocks, dtype=torch.int32, device="cuda"))
    q = np.zeros((S, G, D))
    q[:, :, 0] = 1.0
    q, out, lse = c.attend(q, dtype, scale=1.0)
    c.table, c.lens = table[:1].cpu().numpy(), np.array([128 * blocks], np.int32)
    c.offsets = np.array([0, 1], np.int32)
    want = attention_of(c, q[:1], scale=1.0)
    for s in (0, 150, 303):
        check_attention(out[s:s + 1], lse[s:s + 1], want, dtype, D, 128 * blocks)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("small,large", [(0.0, 28), (0.0, 31), (0.0, 60), (0.0, 100), (-60, 60), (-100, 100), (-103, 120)])
def test_value_scales_at_both_ends(lib, dtype, n, small, large):
    """Blocks of the smallest and of the largest values in one row, in every order: a weight counts in the sum whatever
    its value's scale is."""
    rng = np.random.default_rng(74)
    lens = [96 + n] * 4
    c = Cache(lib, rng, lens, [n] * 4, H=1, D=64, B=16)
    c.scales[:, 0] = 0.01
    for s, blocks in enumerate(([0, 1, 4], [3, 5], [5], [1, 2, 3, 4, 5])):   # those of large values
        c.scales[c.table[s], 1] = small and 2.0 ** small
        c.scales[c.table[s, blocks], 1] = 2.0 ** large
    c.upload()
    q, out, lse = c.attend(queries(rng, c.T, 2, 64), dtype)
    check_attention(out, lse, attention_of(c, q), dtype, 64, max(lens))
    for options in ({"window": 40}, {"causal": False}):
        q, out, lse = c.attend(queries(rng, c.T, 2, 64), dtype, **options)
        check_attention(out, lse, attention_of(c, q, **options), dtype, 64, max(lens))


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("exponents", [(None, 0), (None, 0, 45), (None, 0, -60, -90)])
def test_blocks_of_zeros_among_others_at_length(lib, dtype, n, exponents):
    """Long sequences over many pieces in which blocks of zeros, small and large values follow in no order."""
    rng = np.random.default_rng(80)
    c = Cache(lib, rng, [3000, 2500, 129], [n] * 3, H=2, D=64, B=16)
    kind = rng.integers(0, len(exponents), c.scales[:, 1].shape)
    c.scales[:, 1] *= np.array([0.0 if e is None else 2.0 ** e for e in exponents], np.float32)[kind]
    if dtype == "float16":
        c.scales[:, 1] = np.minimum(c.scales[:, 1], 400.0)    # (results within the type)
    c.upload()
    for options in ({}, {"window": 700}):
        q, out, lse = c.attend(queries(rng, c.T, 4, 64), dtype, **options)
        check_attention(out, lse, attention_of(c, q, **options), dtype, 64, 3000)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("G", [1, 40])
@pytest.mark.parametrize("gap", [10, 30])
def test_zeros_that_outweigh_all_others(lib, dtype, G, gap):
    """A block of zeros whose tokens weigh 2^gap times the others (a first token that draws all attention): what is
    left of the others is as precise as ever."""
    rng = np.random.default_rng(84)
    c = Cache(lib, rng, [512], [1], H=1, D=64, B=128)
    c.codes[:] = 128
    c.codes[c.table[0, 0], 0, 0, :, 0] = 228
    c.codes[:, 1] = rng.integers(1, 256, c.codes[:, 1].shape)
    c.scales[:, 0], c.scales[:, 1] = gap / 100 / np.log2(np.e), 0.02
    c.scales[c.table[0, 0], 1] = 0.0
    c.upload()
    q = np.zeros((1, G, 64))
    q[:, :, 0] = 1.0
    q, out, lse = c.attend(q, dtype, scale=1.0)
    check_attention(out, lse, attention_of(c, q, scale=1.0), dtype, 64, 512)


@pytest.mark.parametrize("G", [1, 40])
def test_value_scales_up_to_the_largest_number(lib, G):
    """Values of 0 and the largest f32, with weights that come close to where the running reference moves."""
    rng = np.random.default_rng(81)
    c = Cache(lib, rng, [512], [1], H=1, D=64, B=128)
    c.codes[:] = 128
    c.codes[c.table[0, 1:], 0, 0, :, 0] = 228
    c.codes[:, 1] = rng.integers(128, 130, c.codes[:, 1].shape)
    c.scales[:, 0], c.scales[:, 1] = 7.9999 / 100 / np.log2(np.e), np.finfo(np.float32).max
    c.upload()
    q = np.zeros((1, G, 64))
    q[:, :, 0] = 1.0
    q, out, lse = c.attend(q, "float32", scale=1.0)
    check_attention(out, lse, attention_of(c, q, scale=1.0), "float32", 64, 512)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("n", [1, 3, 150])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_values_that_are_no_numbers_leave_the_sum(lib, dtype, n, bad):
    """A scale of the values alone that is no number (Inf counts as none): rows that see a token of its block have NaN
    in out; lse does not depend on values."""
    rng = np.random.default_rng(75)
    c = Cache(lib, rng, [400, 390], [n, n], H=2, D=64, B=16)
    clean = c.scales.copy()
    for at in ([399 // 16], [2, 7], list(range(25))):
        c.scales = clean.copy()
        c.scales[c.table[0, at], 1] = bad
        c.upload()
        for options in ({}, {"window": 150}, {"causal": False}):
            q, out, lse = c.attend(queries(rng, c.T, 4, 64), dtype, **options)
            keep, c.scales = c.scales, clean
            want = attention_of(c, q, **options)
            c.scales = keep
            i = 400 - n + np.arange(n)[:, None]
            first = np.array(at)[None, :] * 16
            sees = np.zeros(c.T, bool)
            window = options.get("window", 1 << 20)
            sees[:n] = ((first <= i) & (first + 15 > i - window)).any(1) if options.get("causal", True) else True
            assert np.isnan(out[sees]).all(), (at, options)
            check_attention(np.where(sees[:, None, None], want["out"], out), lse, want, dtype, 64, 400, f"{at} {options}")


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("G", [1, 5, 40])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_keys_that_are_no_numbers(lib, dtype, G, bad):
    """A scale of the keys that is no number (Inf counts as none), whatever signs the scores would have."""
    rng = np.random.default_rng(85)
    c = Cache(lib, rng, [1, 1, 30, 40], [1] * 4, H=1, D=64, B=16)
    for s, code in enumerate((1, 255, 90)):                   # scores of one sign alone
        own = c.table[s][c.table[s] >= 0]
        c.codes[own, 0], c.scales[own, 0] = code, bad
    c.upload()
    q = np.abs(queries(rng, 4, G, 64))
    q, out, lse = c.attend(q, dtype)
    assert np.isnan(out[:3]).all() and np.isnan(lse[:3]).all()
    c.scales[:, 0] = np.where(np.isfinite(c.scales[:, 0]), c.scales[:, 0], 0)
    want = {k: v[3:] for k, v in attention_of(c, q).items()}
    check_attention(out[3:], lse[3:], want, dtype, 64, 40)


# ----------------------------------------------------------- queries at the ends ----
@pytest.mark.parametrize("n", [1, 40])
def test_queries_up_to_the_largest_number(lib, n):
    """Rows whose largest element is the largest f32; the keys' scales and the factor keep the scores small."""
    rng = np.random.default_rng(76)
    c = Cache(lib, rng, [100], [n], H=1, D=64, B=16)
    c.scales[:, 0] *= np.float32(2.0 ** -60)
    c.upload()
    q = np.clip(queries(rng, n, 2, 64), -6, 6)
    q[:, :, 7], q[:, 1, 9] = 6.0, -6.0
    q = q / 6.0 * float(np.finfo(np.float32).max)
    scale = float(np.float32(0.75 * 2.0 ** -67))
    q, out, lse = c.attend(q, "float32", scale=scale)
    check_attention(out, lse, attention_of(c, q, scale=scale), "float32", 64, 100)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("G", [1, 5, 40])
def test_queries_that_are_no_numbers_and_see_no_token(lib, dtype, G):
    """A row that sees no token (of a table without blocks, of a length of zero) has 0 and -Inf whatever it holds."""
    rng = np.random.default_rng(82)
    c = Cache(lib, rng, [300, 0, 300], [1] * 3, H=1, D=64, B=16)
    c.table[0] = -1
    c.table[2, 3:7] = len(c.codes)
    c.upload()
    q = queries(rng, 3, G, 64)
    q[:2, -1] = np.nan
    got, out, lse = c.attend(q, dtype)
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all()
    check_attention(out, lse, attention_of(c, np.nan_to_num(got)), dtype, 64, 300)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("G", [1, 5, 40])
@pytest.mark.parametrize("scale", [0.1, -0.1, 0.0])
def test_infinite_queries_are_no_numbers(lib, dtype, G, scale):
    """An Inf in q leaves NaN in its row whatever signs the codes have, and 0 where the row sees no token."""
    rng = np.random.default_rng(77)
    lens = [1, 1, 1, 40, 0, 33]
    c = Cache(lib, rng, lens, [1] * 6, H=1, D=64, B=16)
    c.codes[c.table[0, 0], 0, 0, 0, 5] = 1                    # of a sign each, and none
    c.codes[c.table[1, 0], 0, 0, 0, 5] = 255
    c.codes[c.table[2, 0], 0, 0, 0, 5] = 128
    c.codes[c.table[3], 0, 0, :, 5] = 90                      # one sign in all tokens
    c.table[5] = -1
    c.upload()
    for bad in (np.inf, -np.inf):
        q = queries(rng, 6, G, 64)
        q[:, -1, 5] = bad
        got, out, lse = c.attend(q, dtype, scale=scale)
        assert np.isnan(out[:4, -1]).all() and np.isnan(lse[:4, -1]).all()
        assert (out[4:, -1] == 0).all() and np.isneginf(lse[4:, -1]).all()
        if G > 1:
            want = attention_of(c, got[:, :-1], scale=scale)
            check_attention(out[:, :-1], lse[:, :-1], want, dtype, 64, 40)


# ----------------------------------------------------------------- small scales ----
def test_tokens_behind_others_of_the_smallest_scales(lib):
    """A block whose scale is a subnormal number (no write makes one): zeros stay zeros beside its tokens."""
    from test_gpu_kv8 import tokens, write_and_check
    rng = np.random.default_rng(83)
    c = Cache(lib, rng, [20, 20, 20], [3, 3, 3], H=2, D=64, B=32)
    c.scales[c.table[:, 0]] = np.array([1e-40, 1e-45, 2.0 ** -126], np.float32)[:, None, None]
    c.upload()
    k, v = tokens(rng, 9, 2, 64, "float32"), tokens(rng, 9, 2, 64, "float32")
    k.zero_()
    v *= 2.0 ** -110
    v[:, :, ::3] = 0.0
    write_and_check(lib, c, k, v)
    assert (c.codes[c.table[:, 0], 0][:, :, 17:20] == 128).all()


# ------------------------------------------------------- offsets that move or lie ----
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_captured_writes_follow_the_offsets(lib, dtype):
    """Captured once; offsets and lengths move on the GPU between replays."""
    import torch
    from test_gpu_kv8 import host, tokens
    rng = np.random.default_rng(78)
    c = Cache(lib, rng, [80, 80, 80], [30, 20, 10], H=2, D=64, B=16)
    k, v = tokens(rng, 60, 2, 64, dtype), tokens(rng, 60, 2, 64, dtype)
    x = np.stack((host(k), host(v)))
    ko, vo = torch.empty_like(k), torch.empty_like(v)

    def step():
        lib.kv8_write(c.cache, c.batch, k, v)
        lib.kv8_read(c.cache, c.batch, ko, vo)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for offsets, lens in (([0, 30, 50, 60], [80, 80, 80]), ([0, 1, 2, 3], [33, 80, 1]), ([5, 5, 40, 57], [10, 70, 17]),
                          ([0, 60, 60, 60], [64, 3, 0])):
        c.upload()
        c.d["offsets"].copy_(torch.tensor(offsets, dtype=torch.int32))
        c.d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        ko.fill_(9.0), vo.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        want = kv8.write(c.codes, c.scales, c.table, np.array(offsets), np.array(lens), x)
        codes, scales = c.on_gpu()
        assert np.array_equal(codes, want[0]) and np.array_equal(scales, want[1])
        values = kv8.values(codes, scales)
        back = np.full((2, 60, 2, 64), 9.0)
        for s in range(3):
            for row, _, b, at in kv8.tokens_of(c.table, offsets, lens, len(codes), 16, s):
                back[:, row] = values[b, :, :, at]
        for got, w in zip((ko, vo), back):
            assert torch.equal(got.cpu(), torch.from_numpy(w).float().to(got.dtype))
    lib.device_status()


def test_offsets_and_lengths_out_of_range_touch_their_own_blocks_alone(lib):
    """Clamped to the rows and the table; what that leaves is written and read, and nothing else."""
    import torch
    from test_gpu_kv8 import host, tokens
    rng = np.random.default_rng(79)
    c = Cache(lib, rng, [48] * 5, [8] * 5, H=2, D=64, B=16, spare=4)
    T = c.T
    k, v = tokens(rng, T, 2, 64, "float32"), tokens(rng, T, 2, 64, "float32")
    x = np.stack((host(k), host(v)))
    offsets, lens = [-7, 9, 4, 12, 1 << 30, -(1 << 31)], [1 << 30, 48, 5, (1 << 31) - 1, 48]
    c.d["offsets"].copy_(torch.tensor(offsets, dtype=torch.int32))
    c.d["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
    codes, scales = c.codes, c.scales
    back = np.full((2, T, 2, 64), 9.0)
    some = []
    for s in range(5):
        a = min(max(offsets[s], 0), T)
        o, l = np.array([a, min(max(offsets[s + 1], a), T)]), np.array([min(max(lens[s], 0), 48)])
        some.append((s, o, l))
        codes, scales = kv8.write(codes, scales, c.table[s:s + 1], o, l, x)
    assert sum(o[1] - o[0] for _, o, _ in some) == 9 + 8 + T - 12
    lib.kv8_write(c.cache, c.batch, k, v)
    got = c.on_gpu()
    assert np.array_equal(got[0], codes) and np.array_equal(got[1], scales)
    values = kv8.values(codes, scales)
    taken = {}
    for s, o, l in some:
        for row, t, b, at in kv8.tokens_of(c.table[s:s + 1], o, l, len(codes), 16, 0):
            taken.setdefault(row, []).append(values[b, :, :, at])
    ko, vo = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
    lib.kv8_read(c.cache, c.batch, ko, vo)
    lib.device_status()
    for kv, got in enumerate((host(ko), host(vo))):
        for row in range(T):                                  # (an element of two ranges' row is either's)
            allowed = [w[kv].astype(np.float32) for w in taken.get(row, [np.full((2, 2, 64), 9.0)])]
            assert np.any([got[row] == w for w in allowed], 0).all(), (kv, row)
