"""Pins of oracle/block.py: hand-worked routes, gradients against central
differences, and the residual norm against written-out sums."""
import numpy as np
import pytest

from oracle import block as ob


def test_hand_worked_sigmoid_route_with_bias_and_groups():
    # sigmoid(ln 3) = 3/4, sigmoid(0) = 1/2, sigmoid(-ln 3) = 1/4
    a = np.log(3.0)
    logits = np.array([[a, 0.0, 0.0, 0.0, -a, -a, a, a]])
    # groups of two: (0.75, 0.5) (0.5, 0.5) (0.25, 0.25) (0.75, 0.75)
    ids, w, counts = ob.route_scored(logits, None, 3, "sigmoid", 4, 2, 2)
    assert ids.tolist() == [[0, 6, 7]]           # groups 0 and 3 stay
    assert np.allclose(w, 1 / 3)
    assert counts.tolist() == [1, 0, 0, 0, 0, 0, 1, 1]
    # a bias of 1 on expert 4 wins group 2 a place (1.5) and expert 4 a slot,
    # and leaves its weight at its score
    bias = np.zeros(8)
    bias[4] = 1.0
    ids, w, _ = ob.route_scored(logits, bias, 3, "sigmoid", 4, 2, 2,
                                scale=2.0)
    assert ids.tolist() == [[4, 6, 7]]
    assert np.allclose(w, 2 * np.array([[0.25, 0.75, 0.75]]) / 1.75)


def test_softmax_scores_and_masks():
    inf = np.inf
    s = ob.scores(np.array([[0.0, np.log(3.0), -inf, np.nan],
                            [-inf] * 4, [inf, 1.0, inf, -inf]]), "softmax")
    assert np.allclose(s, [[0.25, 0.75, 0, 0], [0] * 4, [0.5, 0, 0.5, 0]])
    ids, w, _ = ob.route_scored(np.array([[-inf, 1.0, np.nan, -inf]]), None, 3)
    assert ids.tolist() == [[1, 0, 2]] and w.tolist() == [[1, 0, 0]]
    # a dead group loses to a live one, whatever its place
    ids, w, _ = ob.route_scored(np.array([[-inf, -inf, -9.0, -inf]]), None, 2,
                                "sigmoid", 2, 1, 2)
    assert ids.tolist() == [[2, 3]] and w.tolist() == [[1, 0]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((4, 12))
    logits[1, 5] = -np.inf
    ids, _, _ = ob.route_scored(logits, None, 4, score, renormalize=renorm)
    d_w = rng.standard_normal((4, 4))

    def loss(l):
        s = ob.scores(l, score)
        w = np.take_along_axis(s, ids, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return float((1.7 * w * d_w).sum())

    got = ob.route_scored_backward(logits, ids, d_w, score, renorm, 1.7)
    for t in range(4):
        for e in range(12):
            if np.isinf(logits[t, e]):
                assert got[t, e] == 0
                continue
            h, up, down = 1e-6, logits.copy(), logits.copy()
            up[t, e] += h
            down[t, e] -= h
            assert got[t, e] == pytest.approx(
                (loss(up) - loss(down)) / (2 * h), abs=1e-8)


@pytest.mark.parametrize("gate_shape", [None, (1, 1), (3, 1), (1, 5), (3, 5)])
@pytest.mark.parametrize("post", [True, False])
def test_norm_gradients_against_differences(gate_shape, post):
    rng = np.random.default_rng(8)
    kw = dict(eps=1e-3, gain_offset=1.0, residual_scale=0.7)
    v = dict(y=rng.standard_normal((3, 5)), r=rng.standard_normal((3, 5)),
             post=rng.standard_normal(5) if post else None,
             gate=None if gate_shape is None
             else rng.standard_normal(gate_shape),
             pre=rng.standard_normal(5))
    d_x, d_ro = rng.standard_normal((3, 5)), rng.standard_normal((3, 5))

    def loss(v):
        ro, x = ob.residual_norm(v["y"], v["r"], v["post"], v["gate"],
                                 v["pre"], **kw)
        return float((ro * d_ro).sum() + (x * d_x).sum())

    ro, _ = ob.residual_norm(v["y"], v["r"], v["post"], v["gate"], v["pre"],
                             **kw)
    got = ob.residual_norm_backward(v["y"], ro, v["post"], v["gate"],
                                    v["pre"], d_x, d_ro, **kw)
    for name, key in (("y", "d_y"), ("r", "d_resid"), ("post", "d_post"),
                      ("gate", "d_gate"), ("pre", "d_pre")):
        if v[name] is None:
            assert key not in got
            continue
        for at in np.ndindex(v[name].shape):
            h = 1e-6
            side = []
            for s in (h, -h):
                c = dict(v)
                c[name] = v[name].copy()
                c[name][at] += s
                side.append(loss(c))
            assert got[key][at] == pytest.approx(
                (side[0] - side[1]) / (2 * h), abs=2e-8), (name, at)


def test_unit_by_hand():
    assert np.allclose(ob.unit(np.array([[3.0, 4.0]]), 0.0),
                       [[3 / np.sqrt(12.5), 4 / np.sqrt(12.5)]])
    r, x = ob.residual_norm(np.array([[3.0, 4.0]]), np.array([[1.0, 1.0]]),
                            None, np.array([[2.0]]), np.array([1.0, 2.0]),
                            eps=0.0, residual_scale=0.5)
    assert np.allclose(r, [[4.0, 5.0]])
    assert np.allclose(x, [[4 / np.sqrt(20.5), 10 / np.sqrt(20.5)]])


def test_combine_gradients_against_differences():
    rng = np.random.default_rng(4)
    pair_row = np.array([[1, -1], [2, 0], [-1, -1]])
    y, w = rng.standard_normal((4, 3)), rng.random((3, 2))
    d_out = rng.standard_normal((3, 3))
    d_y, d_w = ob.combine_backward(d_out, y, pair_row, w)

    def loss(y, w):
        return float((ob.combine_rows(y, pair_row, w, None) * d_out).sum())

    for at in np.ndindex(w.shape):                  # the combine is linear
        up = w.copy()
        up[at] += 1
        assert d_w[at] == pytest.approx(loss(y, up) - loss(y, w))
    assert np.isnan(d_y[3]).all()                   # a row of no pair
    for at in np.ndindex(3, 3):
        up = y.copy()
        up[at] += 1
        assert d_y[at] == pytest.approx(loss(up, w) - loss(y, w))
