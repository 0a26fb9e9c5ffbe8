"""The router's gradient at the ends of its range, against the float64 oracle."""
import numpy as np
import pytest

from oracle import moe as omoe

pytestmark = pytest.mark.gpu

LOWEST = -float(np.finfo(np.float32).max)


def backward(lib, l, ids, dw, **kw):
    import torch
    bias = kw.pop("bias", None)
    dev = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (l.astype(np.float32), ids.astype(np.int32),
                                                                      dw.astype(np.float32))]
    out = torch.full(l.shape, 7.0, device="cuda")
    lib.moe_route_backward(*dev, out, bias=None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda(),
                           **kw)
    lib.device_status()
    return out.cpu().double().numpy()


def check_backward(got, l, ids, dw, scale, bias, score, renorm):
    """A score is within 2^-19 of its size and 2^-148; so is its share r = p / max(sum, 2^-126), within 2^-19 r and
    2^-22; a gradient is a sum of products of shares and upstream gradients."""
    want = omoe.route_backward(l, ids, dw, bias=bias, score=score, renorm=renorm, scale=scale)
    p = np.array([omoe.scores(r, bias, score)[0] for r in l])
    on = ids >= 0
    at = np.maximum(ids, 0)
    ps = np.where(on, np.take_along_axis(p, at, 1), 0.0)
    S = np.maximum(ps.sum(1, keepdims=True), omoe.TINY) if renorm else 1.0
    g = np.abs(np.where(on, dw, 0.0)) * scale
    r = ps / S
    tot = (g * r).sum(1, keepdims=True)
    size = p * tot
    np.add.at(size, (np.arange(len(l))[:, None] + np.zeros_like(ids), at), r * (g + tot))
    bound = 2.0 ** -17 * size + 2.0 ** -21 * g.sum(1, keepdims=True)
    assert np.all(np.isfinite(got))
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


SATURATED = [-1e4, LOWEST, -150.0, -3e30, -86.0, -86.5, -85.0, -87.0]


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("size", [1.0, 100.0])
def test_backward_of_saturated_sigmoids(lib, renorm, size):
    """Every selected score next to nothing or nothing; upstream gradients that exceed 2^128 / 2^126."""
    rng = np.random.default_rng(60)
    E, k = 16, 4
    l = np.array([np.full(E, v) for v in SATURATED] + [rng.choice([-86.0, -86.5, -85.5, -1e4], E) for _ in range(9)])
    l[-1, :8] = 0.0                                                    # some ordinary scores among them
    ids = np.array([omoe.route_row(r, k, score="sigmoid")[0] for r in l])
    ids[2, 1] = -1
    dw = rng.normal(size=(len(l), k)).astype(np.float32) * size
    dw[0] = [2 * size, -size, 0, 1]
    got = backward(lib, l, ids, dw, score="sigmoid", renorm=renorm, scale=2.5)
    check_backward(got, l, ids, dw, 2.5, None, "sigmoid", renorm)


@pytest.mark.parametrize("renorm", [False, True])
def test_backward_of_softmax_scores_that_underflow(lib, renorm):
    """A bias selects experts whose softmax is next to nothing (or nothing) beside another's."""
    rng = np.random.default_rng(61)
    E, k = 40, 3
    l = np.zeros((12, E))
    l[:, 1:] = rng.choice([-84.0, -85.0, -84.5, -86.0], (12, E - 1))
    l[3:6, 1:] = -1e4
    l[6, 1:] = LOWEST
    l[7, 5:] = -np.inf
    bias = np.where(np.arange(E) % 3 == 2, 5.0, 0.0)
    ids = np.array([omoe.route_row(r, k, bias=bias)[0] for r in l])
    assert not (ids == 0).any(axis=1)[:7].any()
    dw = (rng.normal(size=(12, k)) * 50).astype(np.float32)
    got = backward(lib, l, ids, dw, renorm=renorm, scale=2.5, bias=bias)
    check_backward(got, l, ids, dw, 2.5, bias, "softmax", renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_backward_where_the_sum_is_clamped(lib, score):
    """Below 2^-126 the divisor of the weights is a constant."""
    rng = np.random.default_rng(62)
    E, k = 12, 2
    l = rng.uniform(-88.6, -87.4, (20, E)).astype(np.float32).astype(np.float64)
    l[10:] -= 0.0 if score == "sigmoid" else 1.0
    l[:, 0] = -1e4 if score == "sigmoid" else 0.0                      # (a softmax with a score of one)
    ids = np.array([1 + rng.permutation(E - 1)[:k] for _ in range(20)])
    ids[4:8, 1] = -1
    p = np.array([omoe.scores(r, None, score)[0] for r in l])
    assert np.sum(np.where(ids >= 0, np.take_along_axis(p, np.maximum(ids, 0), 1), 0).sum(1) < omoe.TINY) >= 4
    bias = np.where(np.arange(E) > 0, 2.0, 0.0)                        # why they were selected
    dw = rng.normal(size=(20, k)).astype(np.float32)
    got = backward(lib, l, ids, dw, score=score, scale=2.5, bias=bias)
    check_backward(got, l, ids, dw, 2.5, bias, score, True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E", [60, 1000])
def test_backward_in_place(lib, score, renorm, E):
    """dlogits may be the logits' own memory."""
    import torch
    rng = np.random.default_rng(63)
    l = torch.from_numpy(rng.normal(size=(700, E)).astype(np.float32)).cuda()
    ids = torch.topk(l, 8).indices.int()
    dw = torch.from_numpy(rng.normal(size=(700, 8)).astype(np.float32)).cuda()
    want = lib.moe_route_backward(l, ids, dw, torch.empty_like(l), score=score, renorm=renorm)
    got = l.clone()
    lib.moe_route_backward(got, ids, dw, got, score=score, renorm=renorm)
    assert torch.equal(got, want)
