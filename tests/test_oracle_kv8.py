"""The oracle of the 8-bit cache against values that the definition fixes and against brute force (CPU)."""
import numpy as np
import pytest

from kv8_util import Cache
from oracle import kv8


def pool(rng, lens, n, **k):
    return Cache(None, rng, lens, n, **k)


def test_codes_of_known_values():
    c = pool(np.random.default_rng(0), [2], [2], H=1, D=64, B=16)
    x = np.zeros((2, 2, 1, 64), np.float32)
    x[0, 0, 0, :4] = [127.0, -127.0, 0.5, 1.5]                # scale 1: halves to even
    x[1, 1, 0, :2] = [254.0, 3.0]                             # scale 2
    codes, scales = kv8.write(c.codes, c.scales, c.table, c.offsets, c.lens, x)
    b = c.table[0, 0]
    assert scales[b, 0, 0] == 1.0 and scales[b, 1, 0] == 2.0
    assert codes[b, 0, 0, 0, :5].tolist() == [255, 1, 128, 130, 128]
    assert codes[b, 1, 0, 1, :3].tolist() == [255, 130, 128]
    assert np.array_equal(codes[b, :, :, 2:], c.codes[b, :, :, 2:])
    assert np.array_equal(kv8.values(codes, scales)[b, 0, 0, 0, :2], [127.0, -127.0])


def test_a_larger_token_makes_the_block_coarser():
    rng = np.random.default_rng(1)
    c = pool(rng, [3], [1], H=1, D=64, B=16)
    b = c.table[0, 0]
    c.scales[b] = 1.0
    before = c.codes.copy()
    x = np.zeros((2, 1, 1, 64), np.float32)
    x[0, 0, 0, 0], x[1, 0, 0, 0] = 254.0, 100.0
    codes, scales = kv8.write(c.codes, c.scales, c.table, c.offsets, c.lens, x)
    assert scales[b, 0, 0] == 2.0 and scales[b, 1, 0] == 1.0
    assert np.array_equal(codes[b, 0, 0, :2].astype(int) - 128, np.rint((before[b, 0, 0, :2].astype(int) - 128) / 2))
    assert np.array_equal(codes[b, 1, 0, :2], before[b, 1, 0, :2])
    assert codes[b, 0, 0, 2, 0] == 255 and codes[b, 1, 0, 2, 0] == 228


@pytest.mark.parametrize("B", [16, 64])
def test_quantised_values_are_within_half_a_step(B):
    rng = np.random.default_rng(2)
    lens = [B, 2 * B + 3, 5]
    c = pool(rng, lens, lens, H=2, D=64, B=B)
    x = rng.normal(size=(2, c.T, 2, 64)).astype(np.float32)
    codes, scales = kv8.write(c.codes, c.scales, c.table, c.offsets, c.lens, x)
    v = kv8.values(codes, scales)
    for s in range(3):
        for row, t, b, at in kv8.tokens_of(c.table, c.offsets, c.lens, len(codes), B, s):
            step = scales[b].astype(np.float64)[..., None]
            # the reciprocal and the product are each rounded: 2^-23 of up to 127 steps
            assert (np.abs(v[b, :, :, at] - x[:, row]) <= (0.5 + 127 * 2.0 ** -22) * step).all()
            assert codes[b, :, :, at].min() >= 1


def test_attention_by_brute_force():
    rng = np.random.default_rng(3)
    lens, n = [37, 5, 0, 20], [3, 7, 2, 0]
    c = pool(rng, lens, n, H=2, D=64, B=16)
    q = rng.normal(size=(c.T, 4, 64))
    v = kv8.values(c.codes, c.scales)
    for causal, window in ((True, 0), (True, 4), (False, 0)):
        got = kv8.attention(q, c.codes, c.scales, c.table, c.offsets, c.lens, 0.2, causal, window)
        for s in range(4):
            for j in range(n[s]):
                i = lens[s] - n[s] + j
                for h in range(4):
                    num, den = np.zeros(64), 0.0
                    for t in range(lens[s]):
                        if causal and (t > i or (window and t <= i - window)):
                            continue
                        b, at = c.table[s, t // 16], t % 16
                        e = np.exp(0.2 * q[c.offsets[s] + j, h] @ v[b, 0, h // 2, at])
                        num, den = num + e * v[b, 1, h // 2, at], den + e
                    row = c.offsets[s] + j
                    if den == 0:
                        assert (got["out"][row, h] == 0).all() and np.isneginf(got["lse"][row, h])
                    else:
                        assert np.allclose(got["out"][row, h], num / den, rtol=1e-12)
                        assert np.isclose(got["lse"][row, h], np.log(den), rtol=1e-12)


def test_a_block_that_is_not_there_is_not_seen():
    rng = np.random.default_rng(4)
    c = pool(rng, [48], [1], H=1, D=64, B=16)
    q = rng.normal(size=(1, 1, 64))
    c.table[0, 1] = -1
    got = kv8.attention(q, c.codes, c.scales, c.table, c.offsets, c.lens, 0.1)
    short = c.table[:, [0, 2]]
    want = kv8.attention(q, c.codes, c.scales, short, c.offsets, np.array([32]), 0.1)
    assert np.allclose(got["out"], want["out"], rtol=1e-13) and np.allclose(got["lse"], want["lse"], rtol=1e-13)
