"""Pins of the training oracle: the checkpoint format by hand and against
torch's E4M3, the experts' gradients against central differences."""
import numpy as np
import pytest

from oracle import moe as omoe
from oracle import train as ot


def test_scales_by_hand():
    assert ot.checkpoint_scale([448.0]) == 1.0
    assert ot.checkpoint_scale([449.0, 3.0]) == 2.0
    assert ot.checkpoint_scale([224.0]) == 0.5
    assert ot.checkpoint_scale([225.0]) == 1.0
    assert ot.checkpoint_scale([0.0, -0.0]) == 1.0
    assert ot.checkpoint_scale([1e-40]) == 2.0 ** -100
    assert ot.checkpoint_scale([np.inf, np.nan, -1.75]) == 2.0 ** -8
    assert ot.checkpoint_scale([np.finfo(np.float32).max]) == 2.0 ** 120


def test_codes_by_hand():
    rows = np.zeros((1, 130))
    rows[0, :6] = [448.0, -1.0, 0.0625 + 0.00390625, np.nan, np.inf, -17.0]
    rows[0, 128:] = [3.0, -0.5]
    codes, scales = ot.checkpoint(rows)
    assert scales.tolist() == [[1.0, 2.0 ** -7]]
    # 448, -1, 0.0664 (a tie between 0.0625 and 0.0703: even), -17 -> -16 (tie)
    assert codes[0, :6].tolist() == [0x7E, 0xB8, 0x18, 0x7F, 0x7F, 0xD8]
    # the last group: 3 * 128 = 384 and -0.5 * 128 = -64
    v = ot.values(codes, scales)
    assert v[0, 128:].tolist() == [3.0, -0.5] and v[0, 0] == 448.0
    assert np.isnan(v[0, 3:5]).all()


def test_the_largest_values_stay_finite():
    top = float(np.finfo(np.float32).max)
    codes, scales = ot.checkpoint(np.array([[top, -top, 1.0]]))
    v = ot.values(codes, scales)
    assert v[0].tolist() == [240.0 * 2.0 ** 120, -240.0 * 2.0 ** 120, 0.0]


def test_codes_against_torch():
    import torch
    g = torch.Generator().manual_seed(3)
    rows = torch.randn(40, 300, generator=g) * torch.randn(300, generator=g).exp()
    codes, scales = ot.checkpoint(rows.numpy())
    s = torch.from_numpy(scales).repeat_interleave(128, 1)[:, :300]
    ref = (rows / s).to(torch.float8_e4m3fn)
    assert np.array_equal(codes, ref.view(torch.uint8).numpy())
    assert np.array_equal(ot.values(codes, scales), (ref.double() * s).numpy())


def test_values_are_exact_in_bf16():
    rng = np.random.default_rng(5)
    rows = rng.normal(size=(8, 256)) * np.exp(rng.normal(size=(8, 256)) * 8)
    v = ot.values(*ot.checkpoint(rows.astype(np.float32)))
    assert np.array_equal(omoe.round_to_bf16(v), v)


@pytest.mark.parametrize("which", ["x", "w", "wg", "wu", "wd"])
def test_gradients_against_differences(which):
    rng = np.random.default_rng(7)
    n, H, I = 3, 4, 5
    a = dict(x=rng.normal(size=(n, H)), w=rng.random(n),
             wg=rng.normal(size=(H, I)), wu=rng.normal(size=(H, I)),
             wd=rng.normal(size=(I, H)))
    d = rng.normal(size=(n, H))

    def loss(v):
        y = ot.expert_forward(v["x"], v["wg"], v["wu"], v["wd"],
                              round_h=False)[2]
        return float((v["w"][:, None] * y * d).sum())

    g, u, _ = ot.expert_forward(a["x"], a["wg"], a["wu"], a["wd"], False)
    got = dict(zip(("x", "w", "wg", "wu", "wd"), ot.expert_backward(
        a["x"], g, u, a["w"], d, a["wg"], a["wu"], a["wd"])))[which]
    step = 1e-5
    for i in np.ndindex(a[which].shape):
        up, down = ({k: v.copy() for k, v in a.items()} for _ in range(2))
        up[which][i] += step
        down[which][i] -= step
        diff = (loss(up) - loss(down)) / (2 * step)
        assert abs(diff - got[i]) <= 1e-7 * (1 + abs(diff))


def test_few_layer_equals_the_layer():
    rng = np.random.default_rng(9)
    T, H, I, E, k = 5, 8, 4, 6, 2
    x = omoe.round_to_bf16(rng.normal(size=(T, H)))
    experts = [tuple(omoe.round_to_bf16(rng.normal(size=s)) for s in
                     ((H, I), (H, I), (I, H))) for _ in range(3)]
    logits = rng.normal(size=(T, E)).astype(np.float32)
    ids, w, _ = omoe.route_topk(logits, k)
    got = ot.few_layer(x, ids, w, 2, experts)
    rows = omoe.dispatch(ids, 2, 3, *omoe.identity_map(3), 3)
    y = np.zeros((rows.N, H))
    for r in range(rows.N):
        y[r] = ot.expert_forward(x[rows.row_token[r]][None],
                                 *experts[rows.row_phys[r]])[2][0]
    ref = omoe.combine(y, rows.pair_row, w, None, T, H)
    assert np.allclose(got, ref, rtol=1e-12, atol=1e-12)
