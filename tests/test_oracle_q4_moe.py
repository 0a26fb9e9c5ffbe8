"""Pins of the oracle of the 4-bit weights and the mixture-of-experts operators (CPU only)."""
import numpy as np
import pytest

from oracle import moe, q4


def test_codes_even_k_in_the_low_half():
    codes = np.array([[0x21, 0xF0]], dtype=np.uint8)
    assert q4.unpack(codes).tolist() == [[1, 2, 0, 15]]
    assert np.array_equal(q4.pack(q4.unpack(codes)), codes)


def test_dequant_of_hand_written_groups():
    codes = q4.pack(np.tile(np.arange(16, dtype=np.uint8), (1, 4)))          # K = 64, two groups of 32
    d = np.array([[0.5, -2.0]], np.float16).view(np.uint16)
    want = (np.arange(16) - 8.0)
    W = q4.dequant(codes, d, None, 32)
    assert np.array_equal(W[0, :16], want * 0.5) and np.array_equal(W[0, 48:], want * -2.0)
    W = q4.dequant(codes, d, np.array([[0, 15]], np.uint8), 32)
    assert np.array_equal(W[0, :16], np.arange(16) * 0.5) and np.array_equal(W[0, 32:48], (np.arange(16) - 15.0) * -2.0)


@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_error_is_half_a_step_and_grid_weights_return(zeros):
    rng = np.random.default_rng(3)
    w = rng.normal(size=(5, 128)).astype(np.float32) + np.float32(0.3)
    codes, d, z = q4.quantize(w, 32, zeros)
    step = np.repeat(d.view(np.float16).astype(np.float64), 32, -1)
    err = np.abs(q4.dequant(codes, d, z, 32) - w)
    # half a step, and at the ends what rounding the scale to f16 moves 15 steps, and the zero point's half step
    assert np.all(err <= step * (0.5 + 15 * 2.0 ** -11 + (0.5 if zeros else 0.0)) + 1e-9)
    again = q4.quantize(q4.dequant(codes, d, z, 32).astype(np.float32), 32, zeros)
    same = q4.dequant(*again, 32)
    assert np.all(np.abs(same - q4.dequant(codes, d, z, 32)) <= step * 1.01)


def test_route_hand_cases():
    row = np.array([1.0, 3.0, 3.0, -np.inf, np.nan, 2.0])
    ids, w = moe.route_row(row, 3)
    assert ids.tolist() == [1, 2, 5]                                        # ties to the lower index
    e = np.exp([3.0, 3.0, 2.0])
    assert np.allclose(w, e / e.sum(), rtol=1e-12)
    ids, w = moe.route_row(row, 6, renorm=False, score="sigmoid", scale=2.0)
    assert ids.tolist() == [1, 2, 5, 0, -1, -1] and w[4] == w[5] == 0.0
    assert np.isclose(w[0], 2.0 / (1.0 + np.exp(-3.0)))
    ids, w = moe.route_row(np.full(4, -np.inf), 2)
    assert ids.tolist() == [-1, -1] and not w.any()
    # the bias moves the selection and not the weights
    ids, w = moe.route_row(np.array([0.0, 1.0, 2.0]), 1, bias=np.array([0.9, 0.0, 0.0]), score="sigmoid", renorm=False)
    assert ids.tolist() == [0] and np.isclose(w[0], 0.5)


def test_route_groups_take_part_by_their_two_best():
    # group 0 holds the single best expert, group 1 the best pair
    row = np.log(np.array([0.40, 0.01, 0.28, 0.27, 0.02, 0.02]))
    ids, _ = moe.route_row(row, 2, groups=3, top_groups=1)
    assert ids.tolist() == [2, 3]
    ids, _ = moe.route_row(row, 2, groups=3, top_groups=2)
    assert ids.tolist() == [0, 2]


def test_plan_orders_by_expert_then_slot():
    off, slots = moe.plan(np.array([[2, 0], [0, -1], [2, 1]]), 4)
    assert off.tolist() == [0, 2, 3, 5, 5] and slots.tolist() == [1, 2, 5, 0, 4, -1]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(5)
    l = rng.normal(size=(3, 7))
    l[1, 2] = -np.inf
    ids = np.array([moe.route_row(r, 3)[0] for r in l])
    ids[2, 2] = -1
    dw = rng.normal(size=(3, 3))
    got = moe.route_backward(l, ids, dw, score=score, renorm=renorm, scale=1.5)
    h = 1e-6
    for t in range(3):
        for e in range(7):
            up, dn = l[t].copy(), l[t].copy()
            up[e] += h
            dn[e] -= h
            diff = (moe.weights_of(up, ids[t], score=score, renorm=renorm, scale=1.5)
                    - moe.weights_of(dn, ids[t], score=score, renorm=renorm, scale=1.5)) / (2 * h)
            # central differences of functions of size 1.5: rounding 1.5 * 2^-52 / h, curvature h^2
            assert abs(got[t, e] - diff @ np.where(ids[t] >= 0, dw[t], 0.0)) < 1e-8


def test_experts_closed_forms():
    rng = np.random.default_rng(6)
    E, D, F = 3, 4, 5
    gate, up, down = rng.normal(size=(E, F, D)), rng.normal(size=(E, F, D)), rng.normal(size=(E, D, F))
    x = rng.normal(size=(2, D))
    ids = np.array([[0, 2], [-1, -1]])
    w = np.array([[0.25, 0.5], [0.7, 0.3]])
    out = moe.experts(x, ids, w, gate, up, down)
    assert not out[1].any()
    # linear in up, in down and in the weights
    assert np.allclose(moe.experts(x, ids, w, gate, 2 * up, 3 * down), 6 * out)
    assert np.allclose(moe.experts(x, ids, 2 * w, gate, up, down), 2 * out)
    # a large gate passes its value through: silu(v) -> v
    one = moe.experts(x, np.array([[1], [1]]), np.ones((2, 1)), 1e4 * np.abs(gate) * np.sign(x[0]), up, down)
    v = 1e4 * (np.abs(gate[1]) @ np.abs(x[0]))
    assert np.allclose(one[0], down[1] @ (v * (up[1] @ x[0])))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("logits", [(-87.5, -89.0, -88.0), (-88.0, -1e4, -90.0), (-87.2, -86.5, -91.0)])
def test_route_gradient_where_the_sum_is_clamped(score, logits):
    """Selected scores that sum to less than 2^-126 (and, last, to a little more): the weights' divisor is a constant."""
    row = np.array(logits + (0.0, -0.5 if score == "softmax" else -1e4))
    ids, dw = np.array([0, 1, 2]), np.array([0.7, -1.3, 0.4])
    got = moe.route_backward(row[None], ids[None], dw[None], score=score, scale=1.5)[0]
    h = 1e-5
    for e in range(len(row)):
        up, dn = row.copy(), row.copy()
        up[e] += h
        dn[e] -= h
        diff = (moe.weights_of(up, ids, score=score, scale=1.5) - moe.weights_of(dn, ids, score=score, scale=1.5)) / (2 * h)
        # central differences of functions of size 1.5: curvature h^2, rounding 2^-50 / h
        assert abs(got[e] - diff @ dw) < 1e-9
