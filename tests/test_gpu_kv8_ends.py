"""The 8-bit cache at the ends of what its arguments may be, against the f64 oracle.

The bound of the attention is derived in kv8_util.check_attention.
"""
import numpy as np
import pytest

from kv8_util import Cache, attention_of, check_attention, queries

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
