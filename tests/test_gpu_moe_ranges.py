"""The routed experts on both sides of the tensor cores and at the ends of their weights' range.

Bounds (derived before the first run).  Rounding to f16 is off by 2^-11 of a
value at most and by 2.1e-4 of it in the root mean square (bf16: 1.7e-3), and
independent roundings add in squares: an expert's output in f16 carries those of the
gated product and of itself (streaming products: 3.0e-4), and of the three weights
besides, where silu passes Gate's on with a factor of about 1.2 (tensor cores:
4.9e-4).  The norm of the error over all outputs may be 1.4 times that.
"""
import numpy as np
import pytest

from oracle import moe as omoe
from oracle import q4 as oq4
from test_gpu_moe import run_experts
from test_gpu_q4 import upload

pytestmark = pytest.mark.gpu

# relative error of a call's outputs in the norm: (streaming, tensor cores)
NORM = {"float16": (4.2e-4, 7e-4), "bfloat16": (1.9e-3, 1.9e-3)}


def layer(lib, rng, E, D, F, group=32, gate=None, up=None, down=None):
    """Random matrices whose scales are multiplied by the given factors (of the scales' shape); (float64, handles)."""
    mats, handles = [], []
    for (N, K), f in zip(((F, D), (F, D), (D, F)), (gate, up, down)):
        c = rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
        d = rng.uniform(0.005, 0.01, (E, N, K // group)) * rng.choice([-1, 1], (E, N, K // group))
        d = (d if f is None else d * f).astype(np.float16)
        z = rng.integers(5, 11, (E, N, K // group), dtype=np.uint8)
        mats.append(oq4.dequant(c, d.view(np.uint16), z, group))
        handles.append(upload(lib, c, d, z, group))
    return mats, handles


def norm_error(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("T", [32, 33, 1000])
def test_experts_on_both_sides_of_the_tensor_cores(lib, dtype, T):
    """4 slots a matrix, one slot more, and wide tiles, against the norm that each path's roundings allow."""
    rng = np.random.default_rng(70)
    E, D, F = 8, 512, 256
    mats, handles = layer(lib, rng, E, D, F)
    ids = rng.permutation(np.arange(T) % E)[:, None]
    w = rng.uniform(0.5, 1.0, (T, 1)).astype(np.float32)
    x, got = run_experts(lib, rng.normal(size=(T, D)), ids, w, handles, dtype, E)
    assert norm_error(got, omoe.experts(x, ids, w, *mats)) < NORM[dtype][T > 4 * E]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("large", ["gate", "up", "down"])
@pytest.mark.parametrize("T", [8, 9, 12, 300])
def test_experts_of_large_weights(lib, dtype, large, T):
    """Scales up to the largest of f16: a weight is up to 15 times as much, beyond f16 itself."""
    rng = np.random.default_rng(71)
    E, D, F = 2, 256, 128
    most = {large: 65504.0 / 0.01}
    mats, handles = layer(lib, rng, E, D, F, **most)
    ids = (np.arange(T) % E)[:, None]
    w = np.ones((T, 1), np.float32)
    # outputs within the range of f16
    x0 = rng.normal(size=(T, D)) * (2.0 ** -12 if large == "down" else 2.0 ** -9)
    x0[:, ::7] = 0.0
    x, got = run_experts(lib, x0, ids, w, handles, dtype, E)
    want = omoe.experts(x, ids, w, *mats)
    assert np.abs(mats[("gate", "up", "down").index(large)]).max() > 65504.0 and np.abs(want).max() < 6e4
    assert np.all(np.isfinite(got))
    # (f16 outputs in its subnormal range are off by 2^-25 at most)
    assert np.linalg.norm(got - want) < NORM[dtype][1] * np.linalg.norm(want) + 2.0 ** -25 * np.sqrt(want.size)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("T", [8, 40, 300])
@pytest.mark.parametrize("factor", [30.0, 1000.0])
def test_experts_with_a_few_large_rows(lib, dtype, T, factor):
    """32 of Gate's and Up's rows are `factor` times the others and Down's columns that meet them as much smaller, so
    that all gated values count alike, large and ordinary ones."""
    rng = np.random.default_rng(72)
    E, D, F = 2, 1024, 512
    rows = np.ones((E, F, 1))
    rows[:, 64:96] = factor
    columns = np.full((E, 1, F // 32), 200.0)
    columns[:, :, 2] /= factor ** 2
    mats, handles = layer(lib, rng, E, D, F, gate=rows, up=rows, down=columns)
    ids = (np.arange(T) % E)[:, None]
    w = np.ones((T, 1), np.float32)
    x, got = run_experts(lib, rng.normal(size=(T, D)) * 0.2, ids, w, handles, dtype, E)
    assert norm_error(got, omoe.experts(x, ids, w, *mats)) < NORM[dtype][T > 4 * E]


@pytest.mark.parametrize("tiny", [0.0, 2.0 ** -24])
def test_experts_with_dead_rows(lib, tiny):
    """Rows of Gate and Up whose scales are nothing, or next to it, and one expert all of them."""
    rng = np.random.default_rng(73)
    E, D, F, T = 3, 512, 256, 60
    dead = np.where(rng.random((E, F, 1)) < 0.1, tiny / 0.01, 1.0)
    dead[2] = tiny / 0.01
    mats, handles = layer(lib, rng, E, D, F, gate=dead, up=dead)
    ids = (np.arange(T) % E)[:, None]
    w = np.ones((T, 1), np.float32)
    x, got = run_experts(lib, rng.normal(size=(T, D)), ids, w, handles, "float16", E)
    want = omoe.experts(x, ids, w, *mats)
    assert norm_error(got[ids[:, 0] < 2], want[ids[:, 0] < 2]) < NORM["float16"][1]
    assert np.abs(got[ids[:, 0] == 2] - want[ids[:, 0] == 2]).max() <= 2.0 ** -25       # outputs next to nothing


@pytest.mark.parametrize("bad", [np.inf, np.nan])
@pytest.mark.parametrize("T", [6, 60])
def test_experts_beside_a_broken_one(lib, bad, T):
    """A scale that is no number spoils its expert's tokens and no others."""
    rng = np.random.default_rng(74)
    E, D, F = 3, 256, 128
    planted = np.ones((E, F, 1))
    planted[1, 5] = bad
    mats, handles = layer(lib, rng, E, D, F, gate=planted)
    ids = (np.arange(T) % E)[:, None]
    w = np.ones((T, 1), np.float32)
    x, got = run_experts(lib, rng.normal(size=(T, D)), ids, w, handles, "float16", E)
    sound = ids[:, 0] != 1
    assert norm_error(got[sound], omoe.experts(x[sound], ids[sound], w[sound], *mats)) < NORM["float16"][T > 4 * E]
    assert not np.isfinite(got[~sound]).any()
