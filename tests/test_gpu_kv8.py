"""The 8-bit cache and the attention over it against the f64 oracle.

Codes and scales are compared bit by bit (the definition is in 32-bit steps); the bound of
the attention is derived in kv8_util.check_attention.
"""
import numpy as np
import pytest

from kv8_util import Cache, attention_of, check_attention, queries
from oracle import kv8

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ write and read ----
def tokens(rng, T, H, D, dtype, more=1, shift=0):
    """(x float32 [T, H, D] as dtype holds it, the strided tensor)."""
    import torch
    b = torch.full((T, (H + more) * D + shift), float("nan"), dtype=getattr(torch, dtype), device="cuda")
    v = b.as_strided((T, H, D), (b.stride(0), D, 1), shift)
    v.copy_(torch.from_numpy(rng.normal(size=(T, H, D)) * 2.0 ** rng.uniform(-6, 6, (T, H, 1))))
    return v


def host(v):
    return v.float().cpu().numpy()


def write_and_check(lib, c, k, v):
    want = kv8.write(c.codes, c.scales, c.table, c.offsets, c.lens, np.stack((host(k), host(v))))
    lib.kv8_write(c.cache, c.batch, k, v)
    lib.device_status()
    codes, scales = c.on_gpu()
    assert np.array_equal(scales.view(np.uint32) & 0x7fffffff, want[1].view(np.uint32) & 0x7fffffff) or \
        np.array_equal(scales, want[1], equal_nan=True)
    bad = np.isnan(want[1])[..., None, None] | np.zeros(codes.shape, bool)
    assert np.array_equal(np.where(bad, 0, codes), np.where(bad, 0, want[0]))
    c.codes, c.scales = codes, scales


SEQUENCES = {
    "one token each": ([1, 17, 64, 129, 31], [1, 1, 1, 1, 1]),
    "fresh prompts": ([5, 40, 128, 1, 200], [5, 40, 128, 1, 200]),
    "appended chunks": ([37, 300, 33, 16, 0], [20, 150, 1, 16, 0]),
    "one of many": ([700], [333]),
}


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("D,B", [(64, 16), (128, 64), (128, 128), (64, 32), (128, 16), (64, 128)])
@pytest.mark.parametrize("lens,n", SEQUENCES.values(), ids=SEQUENCES.keys())
def test_write_and_read_are_exact(lib, dtype, D, B, lens, n):
    import torch
    rng = np.random.default_rng(11)
    c = Cache(lib, rng, lens, n, H=3, D=D, B=B)
    for shift in (0, 1):                                     # aligned rows, and rows that are not
        k, v = (tokens(rng, c.T, 3, D, dtype, shift=shift) for _ in range(2))
        write_and_check(lib, c, k, v)
        ko, vo = (torch.full_like(x, 9.0) for x in (k, v))
        ko, vo = (tokens(rng, c.T, 3, D, dtype, shift=shift).fill_(9.0) for _ in range(2))
        lib.kv8_read(c.cache, c.batch, ko, vo)
        lib.device_status()
        x = kv8.values(c.codes, c.scales)
        for kv, got in enumerate((ko, vo)):
            want = np.zeros((c.T, 3, D))
            for s in range(len(lens)):
                for row, t, b, at in kv8.tokens_of(c.table, c.offsets, c.lens, len(c.codes), B, s):
                    want[row] = x[b, kv, :, at]
            want = torch.from_numpy(want).float().to(got.dtype)              # a code times a scale is rounded once to f32
            assert torch.equal(got.cpu(), want)


def test_blocks_grow_coarser_and_begin_anew(lib):
    """A token larger than all before makes its block's scale coarser; a smaller one leaves it; a token at a block's
    first place takes no notice of what the block held."""
    rng = np.random.default_rng(12)
    c = Cache(lib, rng, [15, 16, 17], [15, 1, 1], H=2, D=64, B=16)
    c.scales[c.table[2, 1]] = 1e30                            # of an earlier owner
    c.upload()
    for size in (1.0, 0.25, 64.0):
        k, v = tokens(rng, 17, 2, 64, "float32") , tokens(rng, 17, 2, 64, "float32")
        k[15:] *= size
        write_and_check(lib, c, k, v)


@pytest.mark.parametrize("what", ["zeros", "tiny", "huge", "nan", "inf"])
def test_values_at_the_ends(lib, what):
    import torch
    rng = np.random.default_rng(13)
    c = Cache(lib, rng, [3, 20, 36], [3, 4, 36], H=2, D=64, B=16)
    k, v = tokens(rng, 43, 2, 64, "float32"), tokens(rng, 43, 2, 64, "float32")
    if what == "zeros":
        k.zero_()
        v[3:7] = -0.0
    elif what == "tiny":                                      # below, at and above 2^-96
        k[:3] = 2.0 ** -97
        k[3:7] = 2.0 ** -96
        v *= 2.0 ** -100
    elif what == "huge":
        k *= 2.0 ** 110
        v[5, 1, 7] = torch.finfo(torch.float32).max
    else:
        k[4, 0, 9] = float(what)
        v[30, 1, 63] = -float(what)
    write_and_check(lib, c, k, v)
    if what in ("nan", "inf"):
        assert np.isnan(c.scales).sum() == 2
    write_and_check(lib, c, tokens(rng, 43, 2, 64, "float32"), tokens(rng, 43, 2, 64, "float32"))


def test_tokens_without_place(lib):
    """More new tokens than the length has places, numbers that name no block, ranges that go back."""
    import torch
    rng = np.random.default_rng(14)
    c = Cache(lib, rng, [4, 40, 40, 10], [9, 40, 20, 0], H=1, D=64, B=16)
    c.table[1, 1], c.table[2, 2] = len(c.codes), -7
    c.upload()
    k, v = tokens(rng, c.T, 1, 64, "float32"), tokens(rng, c.T, 1, 64, "float32")
    write_and_check(lib, c, k, v)
    ko = torch.full_like(k, 9.0)
    lib.kv8_read(c.cache, c.batch, ko, torch.empty_like(v))
    got = host(ko)
    placed = np.zeros(c.T, bool)
    for s in range(4):
        for row, t, b, at in kv8.tokens_of(c.table, c.offsets, c.lens, len(c.codes), 16, s):
            placed[row] = b >= 0
    assert (got[~placed] == 9.0).all() and placed.sum() == 4 + 24 + 12
    # offsets that go back and out of the rows, lengths out of the table: nothing but its own blocks is touched
    c.d["offsets"].copy_(torch.tensor([5, 3, 60, 1 << 30, -4], dtype=torch.int32))
    c.d["lens"].copy_(torch.tensor([1 << 30, -5, 48, 7], dtype=torch.int32))
    lib.kv8_write(c.cache, c.batch, k, v)
    lib.kv8_read(c.cache, c.batch, ko, torch.empty_like(v))
    lib.device_status()


# ----------------------------------------------------------------- attention ----
ATTEND = [
    # lens, n, heads, G, options
    ([1], [1], 1, 1, {}),
    ([700], [1], 2, 4, {}),
    ([1, 64, 65, 1000, 0, 130], [1, 1, 1, 1, 1, 0], 2, 8, {}),
    ([300, 17, 5], [4, 3, 5], 1, 5, {}),
    ([300, 17, 5], [4, 3, 5], 1, 5, {"window": 9}),
    ([300, 90, 3], [2, 70, 7], 2, 3, {"window": 64}),
    ([33, 400], [33, 130], 1, 4, {}),
    ([250, 130, 0], [3, 129, 2], 2, 1, {"causal": False}),
    ([40], [1], 1, 33, {}),
    ([129], [129], 1, 16, {"scale": -0.3}),
]


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("D,B", [(64, 16), (128, 64), (128, 128), (64, 128), (128, 32)])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention(lib, dtype, D, B, case):
    lens, n, H, G, options = ATTEND[case]
    rng = np.random.default_rng(20 + case)
    c = Cache(lib, rng, lens, n, H=H, D=D, B=B)
    for beside, pad in (((2, 0), 0), ((0, 1), 3)):
        q, out, lse = c.attend(queries(rng, c.T, H * G, D), dtype, pad=pad, beside=beside, **options)
        check_attention(out, lse, attention_of(c, q, **options), dtype, D, max(lens), f"{case} {beside}")
    assert np.array_equal(c.attend(q, dtype, pad=pad, beside=beside, lse=False, **options)[1], out)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [1, 200])
def test_scales_far_apart(lib, dtype, n):
    """Blocks whose scales differ by many powers of two, zero scales, and scores that leave one block alone."""
    rng = np.random.default_rng(40)
    c = Cache(lib, rng, [640, 320], [n, n], H=2, D=64, B=16, spread=12.0)
    c.scales[c.table[0, 3]] = 0.0
    c.scales[c.table[0, 5], 1] = 0.0
    c.scales[:, 0] = np.minimum(c.scales[:, 0], 0.1)
    c.upload()
    q, out, lse = c.attend(queries(rng, c.T, 4, 64), dtype)
    check_attention(out, lse, attention_of(c, q), dtype, 64, 640)
    c.scales[:, 1] = 0.0                                      # values that are all zeros
    c.upload()
    q, out, lse = c.attend(queries(rng, c.T, 4, 64), dtype)
    assert (out == 0).all()
    check_attention(out, lse, attention_of(c, q), dtype, 64, 640)


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("n", [1, 3, 150])
def test_what_no_row_sees_reaches_none(lib, dtype, n):
    """NaN scales in blocks of others, past the end, before the window and behind a causal row; stale blocks of 255s."""
    rng = np.random.default_rng(41)
    c = Cache(lib, rng, [400, 390], [n, n], H=2, D=64, B=16, width=30)
    clean = c.scales.copy()
    for options in ({}, {"window": 20}):
        c.scales = clean.copy()
        used = set(c.table[c.table >= 0].tolist())
        for b in set(range(len(c.codes))) - used:
            c.scales[b] = np.nan
        want = attention_of(c, np.zeros((c.T, 4, 64)), **options)
        if options:
            c.scales[c.table[1, :(390 - n - 20 + 1) // 16 - 1 if n < 150 else 10]] = np.nan     # before every window
        c.upload()
        q, out, lse = c.attend(queries(rng, c.T, 4, 64), dtype, **options)
        keep = c.scales.copy()
        c.scales = np.nan_to_num(keep, nan=0.0)
        want = attention_of(c, q, **options)
        check_attention(out, lse, want, dtype, 64, 400)
    # the last block of sequence 0 is NaN: rows that see it are, the others are not
    c.scales = clean.copy()
    c.scales[c.table[0, 399 // 16]] = np.nan
    c.upload()
    q, out, lse = c.attend(queries(rng, c.T, 4, 64), dtype)
    sees = 400 - n + np.arange(n) >= 399 // 16 * 16
    assert np.isnan(out[:n][sees]).all() and np.isnan(lse[:n][sees]).all()
    assert np.isfinite(out[:n][~sees]).all() and np.isfinite(out[n:]).all()


@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("n", [2, 140])
def test_rows_that_are_no_numbers_stay_alone(lib, dtype, n):
    rng = np.random.default_rng(42)
    c = Cache(lib, rng, [200], [n], H=1, D=128, B=32)
    q = queries(rng, n, 4, 128)
    q[0, 1, 5], q[1, 2, 127], q[1, 3] = np.nan, np.inf, 0.0
    got, out, lse = c.attend(q, dtype)
    assert np.isnan(out[0, 1]).all() and not np.isfinite(out[1, 2]).any()
    fine = np.ones((n, 4), bool)
    fine[0, 1] = fine[1, 2] = False
    assert np.isfinite(out[fine]).all()
    want = attention_of(c, np.where(np.isfinite(got), got, 0.0))
    check_attention(np.where(fine[..., None], out, want["out"]), np.where(fine, lse, want["lse"]), want, dtype, 128, 200)


@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -40, 2.0 ** 40, 2.0 ** 100])
def test_queries_of_any_size(lib, size):
    """The row's power of two keeps small and large queries; scale undoes it."""
    rng = np.random.default_rng(43)
    c = Cache(lib, rng, [100], [3], H=1, D=64, B=16)
    q, out, lse = c.attend(queries(rng, 3, 2, 64) * size, "float32", scale=0.125 / size)
    check_attention(out, lse, attention_of(c, q, scale=float(np.float32(0.125 / size))), "float32", 64, 100)


def test_tables_without_blocks_and_out_of_range(lib):
    """Tokens without a block are seen by nobody; offsets and lengths of any contents stay inside."""
    import torch
    rng = np.random.default_rng(44)
    for n in (1, 2, 100):
        c = Cache(lib, rng, [200, 120, 300], [n, n, n], H=2, D=64, B=32)
        c.table[0, [1, 3]], c.table[1, :], c.table[2, 9] = -1, 1 << 30, len(c.codes)
        c.upload()
        q, out, lse = c.attend(queries(rng, c.T, 6, 64), "bfloat16")
        check_attention(out, lse, attention_of(c, q), "bfloat16", 64, 300)
        assert (out[n:2 * n] == 0).all() and np.isneginf(lse[n:2 * n]).all()
        c.d["offsets"].copy_(torch.tensor([n, -3, 2 * n, 1 << 30], dtype=torch.int32))
        c.d["lens"].copy_(torch.tensor([-4, 1 << 30, 70], dtype=torch.int32))
        c.attend(queries(rng, c.T, 6, 64), "bfloat16")


def test_offsets_beyond_32_bits(lib):
    """Blocks past 4 GB of codes."""
    import torch
    rng = np.random.default_rng(45)
    B, H, D, P = 128, 8, 128, 17000
    small = Cache(lib, rng, [300, 129], [2, 129], H=H, D=D, B=B)
    shift = P - len(small.codes)
    codes = torch.zeros((P, 2, H, B, D), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((P, 2, H), device="cuda")
    codes[shift:], scales[shift:] = small.d["codes"], small.d["scales"]
    assert codes.numel() > 1 << 32
    table = torch.where(small.d["table"] >= 0, small.d["table"] + shift, -1)
    small.cache, small.batch = lib.KV8Cache(codes, scales), lib.KV8Batch(table, small.d["offsets"], small.d["lens"])
    q, out, lse = small.attend(queries(rng, small.T, 16, D), "bfloat16")
    check_attention(out, lse, attention_of(small, q), "bfloat16", D, 300)
    k, v = tokens(rng, small.T, H, D, "bfloat16"), tokens(rng, small.T, H, D, "bfloat16")
    want = kv8.write(small.codes, small.scales, small.table, small.offsets, small.lens, np.stack((host(k), host(v))))
    lib.kv8_write(small.cache, small.batch, k, v)
    lib.device_status()
    assert np.array_equal(codes[shift:].cpu().numpy(), want[0])
    assert not bool(codes[:shift].any())


@pytest.mark.parametrize("S,n", [(300, 1), (1000, 1), (70, 3)])
def test_many_sequences(lib, S, n):
    rng = np.random.default_rng(46)
    lens = rng.integers(0, 90, S)
    c = Cache(lib, rng, lens.tolist(), np.minimum(lens, n).tolist(), H=1, D=64, B=16)
    q, out, lse = c.attend(queries(rng, c.T, 2, 64), "float16")
    check_attention(out, lse, attention_of(c, q), "float16", 64, 90)


@pytest.mark.parametrize("dtype,D,G,L", [("bfloat16", 128, 8, 40000), ("float32", 64, 1, 70001)])
def test_one_long_sequence(lib, dtype, D, G, L):
    """One sequence over the whole GPU: many pieces joined."""
    rng = np.random.default_rng(47)
    c = Cache(lib, rng, [L], [1], H=1, D=D, B=128)
    q, out, lse = c.attend(queries(rng, 1, G, D), dtype)
    check_attention(out, lse, attention_of(c, q), dtype, D, L)
    again = c.attend(q, dtype)
    assert np.array_equal(again[1], out) and np.array_equal(again[2], lse)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("repeats", [1 << 17, (1 << 17) + 1])
def test_tens_of_millions_of_tokens(lib, dtype, repeats):
    """Tables of 2^24 tokens and one block more, all of them the same 128: their mean is the block's, the sum
    `repeats` times it.  The longest chain of f32 additions is a CTA's: 3 tiles of rows (f32: 6) of 2^18 chunks over
    300 CTAs, 5300, and the pieces, 300."""
    import torch
    rng = np.random.default_rng(50)
    c = Cache(lib, rng, [128], [3], H=1, D=64, B=128)
    table = torch.full((1, repeats), int(c.table[0, 0]), dtype=torch.int32, device="cuda")
    c.batch = lib.KV8Batch(table, c.d["offsets"], torch.tensor([repeats * 128], dtype=torch.int32, device="cuda"))
    q, out, lse = c.attend(queries(rng, 3, 16, 64), dtype, causal=False)
    check_attention(out, lse - np.log(repeats), attention_of(c, q, causal=False), dtype, 64, 16 * 5600)


def test_rows_far_apart_in_a_long_list(lib):
    """Two prompts with 2^18 sequences without rows between them."""
    import torch
    rng = np.random.default_rng(51)
    S = (1 << 18) + 2
    c = Cache(lib, rng, [90, 70], [40, 50], H=1, D=64, B=16)
    table = torch.full((S, c.table.shape[1]), -1, dtype=torch.int32, device="cuda")
    table[0], table[-1] = c.d["table"][0], c.d["table"][1]
    offsets = torch.full((S + 1,), 40, dtype=torch.int32, device="cuda")
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    offsets[0], offsets[-1], lens[0], lens[-1] = 0, 90, 90, 70
    c.batch = lib.KV8Batch(table, offsets, lens)
    q, out, lse = c.attend(queries(rng, c.T, 2, 64), "bfloat16")
    check_attention(out, lse, attention_of(c, q), "bfloat16", 64, 90)


@pytest.mark.parametrize("n", [100, 257, 1000])
def test_prompt_rows_match_decoded_ones(lib, n):
    """Row i of a prompt is what a lone token at its position gets, within both results' bounds."""
    rng = np.random.default_rng(48)
    c = Cache(lib, rng, [n], [n], H=1, D=64, B=32)
    q, out, lse = c.attend(queries(rng, n, 3, 64), "bfloat16")
    want = attention_of(c, q)
    check_attention(out, lse, want, "bfloat16", 64, n)
    one = Cache(lib, rng, [n] * 4, [1] * 4, H=1, D=64, B=32)
    at = [0, 31, 32, n - 1]
    one.codes, one.scales, one.table = c.codes, c.scales, np.repeat(c.table, 4, 0)
    one.lens = np.array([p + 1 for p in at], np.int32)
    import torch
    one.cache, one.batch = c.cache, lib.KV8Batch(torch.from_numpy(one.table).cuda(), one.d["offsets"],
                                                 torch.from_numpy(one.lens).cuda())
    _, lone, _ = one.attend(q[at], "bfloat16")
    check_attention(lone, None, {k: v[at] for k, v in want.items()}, "bfloat16", 64, n)
