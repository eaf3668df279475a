"""The experts' forward and backward pass with 8-bit checkpoints on the GPU
against the float64 oracle, element by element.

Bounds, with u = 2^-24 and b = 2^-8 (a rounding to bf16, relative): a float32
sum of n products is off by at most (n + 1) u of the products' magnitudes in
any order; magnitudes M(.) are the same formulas on absolute values.  silu and
its derivative are evaluated in float32 with an exponential and a division:
16 u of |g| + 1 covers them, and the derivative is at most 1.1."""
import numpy as np
import pytest

from oracle import moe as omoe
from oracle import train as ot
from synth import make_workload

from .helpers import check_output, device_layer, phys_to_logical_from_map

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8


def f64(t):
    return t.detach().double().cpu().numpy()


def weights_of(wl, d):
    return tuple(omoe.bf16_to_f64(d[n]) for n in ("wg", "wu", "wd"))


class Step:
    """A layer, its routes and buffers: forward, then backward."""

    def __init__(self, wl, grads="f32", l2p=None, rep=None, P=None,
                 phys=None, seed=7):
        import torch
        from expert_moe_fp32_amd.runner import to_dev
        self.wl = wl
        self.dl = device_layer(wl, l2p=l2p, rep=rep, P=P, phys_to_logical=phys)
        self.P = self.dl.p.num_physical
        self.phys = list(range(self.P)) if phys is None else phys
        self.l2p = omoe.identity_map(wl.num_local)[0] if l2p is None else l2p
        self.rep = np.ones(wl.num_local, int) if rep is None else rep
        self.b = self.dl.train_buffers(grads)
        self.ids, self.w, _ = omoe.route_topk(wl.logits, wl.k)
        self.w = self.w.astype(np.float32)
        self.x = to_dev(wl.x).view(torch.bfloat16)
        self.dev = (to_dev(self.ids.astype(np.int32)), to_dev(self.w))
        g = torch.Generator().manual_seed(seed)
        self.d_out = torch.randn(wl.T, wl.H, generator=g).bfloat16().cuda()
        self.cap = wl.T * min(wl.k, wl.num_local)
        self.disp = omoe.dispatch(self.ids, wl.expert_begin, wl.num_local,
                                  self.l2p, self.rep, self.P)

    def forward(self):
        self.dl.experts_forward(self.b, self.x, *self.dev)

    def backward(self):
        self.dl.experts_backward(self.b, self.d_out)

    def groups(self):
        """(name, weights, token of each row, rows in the intermediate
        arrays, route weights) of every physical expert and the shared one."""
        d, wl = self.disp, self.wl
        for p in range(self.P):
            r = np.arange(d.offsets[p], d.offsets[p + 1])
            yield (p, weights_of(wl, wl.expert(self.phys[p])), d.row_token[r],
                   r, self.w[d.row_token[r], d.row_slot[r]].astype(float))
        if wl.shared:
            t = np.arange(wl.T)
            yield ("sh", weights_of(wl, wl.shared_expert), t, self.cap + t,
                   np.ones(wl.T))

    def outputs(self):
        b = self.b
        n = self.disp.N
        s = {k: v.clone() for k, v in b.saved.items()}
        for k in ("row_token", "row_weight"):
            s[k] = s[k][:n]
        for k in ("gu_codes", "gu_scales"):      # rows of no pair: anything
            s[k][n:self.cap] = 0
        return {**s, "out": b.out.clone(), "d_x": b.d_x.clone(),
                "d_w": b.d_w.clone(), **{k: v.clone() for k, v in b.grads.items()}}


def check_step(s):
    import torch
    wl, b, d = s.wl, s.b, s.disp
    T, H, I, k, N = wl.T, wl.H, wl.I, wl.k, d.N
    for v in b.saved.values():
        v.view(torch.uint8).fill_(0x5A)
    s.forward()
    torch.cuda.synchronize()
    sv = {n: v.cpu().numpy() for n, v in b.saved.items()}
    # the permutation, bit for bit, and nothing behind it
    assert np.array_equal(sv["offsets"], d.offsets)
    assert np.array_equal(sv["row_token"][:N], d.row_token)
    assert np.array_equal(sv["pair_row"], d.pair_row)
    assert np.array_equal(sv["row_weight"][:N], s.w[d.row_token, d.row_slot])
    for n, end in (("row_token", s.cap), ("gu_codes", s.cap),
                   ("gu_scales", s.cap)):
        assert (np.ascontiguousarray(sv[n][N:end]).view(np.uint8) == 0x5A).all(), n
    # the input's checkpoint, bit for bit
    x = omoe.bf16_to_f64(wl.x)
    rc, rs = ot.checkpoint(x)
    assert np.array_equal(sv["x_codes"], rc)
    assert np.array_equal(sv["x_scales"], rs)
    # gate and up: half an E4M3 step of the value (2^-4 of it, or half of
    # s 2^-9 at the grid's low end), and the float32 product's error before
    # it; the scale that of the largest value within that error
    y = np.zeros((N, H))
    y_sh = None
    for name, (wg, wu, wd), tok, rows, w in s.groups():
        if not len(rows):
            continue
        for at, m in ((0, wg), (I, wu)):
            ref, err = x[tok] @ m, (H + 1) * U * (np.abs(x[tok]) @ np.abs(m))
            got = ot.values(sv["gu_codes"][rows, at:at + I],
                            sv["gu_scales"][rows, at // 128:(at + I) // 128])
            sc = np.repeat(sv["gu_scales"][rows, at // 128:(at + I) // 128], 128, 1)
            half = np.maximum(2.0 ** -4 * (np.abs(ref) + err), sc * 2.0 ** -10)
            assert (np.abs(got - ref) <= half + err).all(), (name, at)
            for n in range(I // 128):
                c = slice(128 * n, 128 * n + 128)
                for i in range(len(rows)):
                    lo = ot.checkpoint_scale(np.maximum(np.abs(ref[i, c]) - err[i, c], 0))
                    hi = ot.checkpoint_scale(np.abs(ref[i, c]) + err[i, c])
                    assert lo <= sc[i, 128 * n] <= hi
        yy = ot.expert_forward(x[tok], wg, wu, wd)[2]
        if name == "sh":
            y_sh = yy
        else:
            y[rows] = yy
    ref = omoe.combine(y, d.pair_row, s.w.astype(float), y_sh, T, H)
    if ref.any():
        check_output(f64(b.out)[:T], ref, wl.out, 1e-2)
    else:
        assert not b.out.any()
    # -------------------------------------------------------- backward
    for t in (b.d_x, b.d_w, *b.grads.values()):
        t.fill_(7.0)
    s.backward()
    torch.cuda.synchronize()
    for n, v in b.saved.items():                  # only read
        assert np.array_equal(v.cpu().numpy(), sv[n]), n
    xh = ot.values(sv["x_codes"], sv["x_scales"])
    dd = f64(s.d_out)
    d_x, e_x = np.zeros((T, H)), np.zeros((T, H))
    d_w, e_w = np.zeros((T, k)), np.zeros((T, k))
    out_b = {"f32": U, "bf16": B}[
        "f32" if b.grads["d_gate"].dtype == torch.float32 else "bf16"]

    def near(got, ref, err, what):
        bad = np.abs(got - ref) > out_b * np.abs(ref) + err * (1 + out_b)
        assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])

    stats = []
    for name, (wg, wu, wd), tok, rows, w in s.groups():
        names = (("sh_gate", "sh_up", "sh_down") if name == "sh" else
                 ("d_gate", "d_up", "d_down"))
        got = [f64(b.grads[n] if name == "sh" else b.grads[n][name]) for n in names]
        if not len(rows):
            assert not any(g.any() for g in got), name
            continue
        gu = ot.values(sv["gu_codes"][rows], sv["gu_scales"][rows])
        g, u = gu[:, :I], gu[:, I:]
        rx, rw, rg, ru, rd = ot.expert_backward(xh[tok], g, u, w, dd[tok], wg, wu, wd)
        q = ot.sigmoid(g)
        e = dd[tok] @ wd.T
        me = np.abs(dd[tok]) @ np.abs(wd.T)
        ee = (H + 1) * U * me                     # of e
        h, eh = g * q * u, 16 * U * (np.abs(g) + 1) * np.abs(u)
        e_wr = (I + 8) * U * (np.abs(e) * np.abs(h)).sum(1) + (
            ee * np.abs(h) + np.abs(e) * eh).sum(1)
        # dg, du, w h: the float32 error, then one rounding
        slope = q + g * q * (1 - q)
        dg, du = w[:, None] * e * u * slope, w[:, None] * e * g * q
        edg = w[:, None] * np.abs(u) * (ee * 1.1 + np.abs(e) * 16 * U * (np.abs(g) + 1))
        edu = w[:, None] * (ee * np.abs(g * q) + np.abs(e) * 16 * U * (np.abs(g) + 1))
        edg += B * (np.abs(dg) + edg)
        edu += B * (np.abs(du) + edu)
        ehw = w[:, None] * eh
        ehw += B * (np.abs(w[:, None] * h) + ehw)
        n = len(rows) + 1
        ax = np.abs(xh[tok])
        near(got[0], rg, ax.T @ edg + n * U * (ax.T @ (np.abs(dg) + edg)), (name, "gate"))
        near(got[1], ru, ax.T @ edu + n * U * (ax.T @ (np.abs(du) + edu)), (name, "up"))
        ad = np.abs(dd[tok])
        near(got[2], rd, ehw.T @ ad + n * U * ((np.abs(w[:, None] * h) + ehw).T @ ad),
             (name, "down"))
        ex = edg @ np.abs(wg.T) + edu @ np.abs(wu.T)
        ex += (2 * I + 1) * U * (np.abs(dg) @ np.abs(wg.T) + np.abs(du) @ np.abs(wu.T) + ex)
        np.add.at(d_x, tok, rx)
        np.add.at(e_x, tok, ex + (k + 2) * U * np.abs(rx))
        if name != "sh":
            slot = d.row_slot[rows]
            d_w[tok, slot], e_w[tok, slot] = rw, e_wr
        stats += [(g_, r_) for g_, r_ in zip(got, (rg, ru, rd))]
    gx = f64(b.d_x)[:T]
    bad = np.abs(gx - d_x) > B * np.abs(d_x) + e_x * (1 + B)
    assert not bad.any(), (np.argwhere(bad)[:4], gx[bad][:4], d_x[bad][:4])
    gw = f64(b.d_w)[:T]
    assert (np.abs(gw - d_w) <= e_w + U * np.abs(d_w)).all()
    assert not gw[d.pair_row < 0].any()
    # In the mean: every term carries one independent rounding of at most b
    # and the output one of at most out_b, so the root mean square of the
    # errors is below b + out_b of the result's.
    if len(stats) and N > 8:
        err = np.sqrt(sum(np.sum((g_ - r_) ** 2) for g_, r_ in stats))
        ref = np.sqrt(sum(np.sum(r_ ** 2) for _, r_ in stats))
        print("   grads: rms error / rms", err / ref, flush=True)
        assert err <= (B + out_b) * ref
        assert np.sqrt(np.sum((gx - d_x) ** 2)) <= 2 * B * np.sqrt(np.sum(d_x ** 2))


CASES = [
    (dict(T=1, H=128, I=128, E=4, num_local=4, k=1, shared=False), "f32"),
    (dict(T=1, H=256, I=128, E=64, num_local=8, k=2, shared=True), "bf16"),
    (dict(T=2, H=128, I=256, E=32, num_local=1, k=2, shared=False), "f32"),
    (dict(T=31, H=256, I=128, E=8, num_local=8, k=3, shared=True), "f32"),
    (dict(T=33, H=384, I=384, E=4, num_local=2, k=2, shared=False), "bf16"),
    (dict(T=200, H=128, I=128, E=4, num_local=4, k=4, shared=False), "f32"),
    (dict(T=130, H=640, I=256, E=16, num_local=4, k=4, shared=True), "bf16"),
    (dict(T=97, H=256, I=640, E=128, num_local=64, k=8, shared=False), "f32"),
    (dict(T=300, H=512, I=128, E=3, num_local=1, k=2, shared=True), "f32"),
    (dict(T=40, H=128, I=128, E=400, num_local=300, k=16, shared=False), "bf16"),
    (dict(T=1100, H=128, I=128, E=8, num_local=8, k=2, shared=False), "f32"),
    (dict(T=2500, H=128, I=128, E=2, num_local=2, k=1, shared=True), "f32"),
    (dict(T=2305, H=128, I=128, E=1, num_local=1, k=1, shared=False, out="f32"),
     "bf16"),
]


@pytest.mark.parametrize("kw,grads", CASES, ids=str)
def test_against_the_oracle(kw, grads):
    print(kw, grads, flush=True)
    check_step(Step(make_workload("prefill", seed=201, **kw), grads))


LARGE = [
    (dict(T=1500, H=768, I=640, E=8, num_local=8, k=2, shared=True), "f32"),
    (dict(T=2000, H=640, I=896, E=3, num_local=2, k=2, shared=False), "bf16"),
    (dict(T=2500, H=768, I=640, E=8, num_local=8, k=2, shared=True), "bf16"),
    (dict(T=4500, H=640, I=896, E=3, num_local=2, k=2, shared=False), "f32"),
]


@pytest.mark.parametrize("kw,grads", LARGE, ids=str)
def test_on_large_tiles(kw, grads):
    print(kw, grads, flush=True)
    check_step(Step(make_workload("prefill", seed=211, **kw), grads))


STRIPS = [
    # outputs of 6 x 9 and 5 x 6 tiles of 256 x 256 (the last ones half), in
    # strips of four tiles along M: 4 + 2 and 4 + 1
    (dict(T=40, H=1408, I=1152, E=3, num_local=3, k=2, shared=True), "f32"),
    # 9 x 11 and 6 x 9: strips of 4 + 4 + 1 and 4 + 2
    (dict(T=23, H=2176, I=1408, E=4, num_local=2, k=2, shared=False), "bf16"),
    # 7 x 12 and 6 x 7: strips of 4 + 3 and 4 + 2; groups of several quads
    (dict(T=300, H=1792, I=1536, E=1, num_local=1, k=1, shared=False), "f32"),
]


@pytest.mark.parametrize("kw,grads", STRIPS, ids=str)
def test_weight_gradients_of_several_strips(kw, grads):
    print(kw, grads, flush=True)
    assert kw["H"] > 1024 and kw["I"] > 1024
    check_step(Step(make_workload("prefill", seed=213, **kw), grads))


def test_a_share_in_the_middle_and_replicas():
    wl = make_workload("prefill", seed=202, T=70, H=256, I=128, E=16,
                       num_local=8, k=4, shared=True)
    wl.expert_begin = 4
    l2p = np.array([[0, 8], [1, -1], [2, -1], [3, -1], [4, 9], [5, -1],
                    [-1, 6], [7, -1]], dtype=np.int32)
    rep = np.array([2, 1, 1, 1, 2, 1, 2, 1], dtype=np.int32)
    phys = [e if e >= 0 else 0 for e in phys_to_logical_from_map(l2p, rep, 10)]
    check_step(Step(wl, "f32", l2p, rep, 10, phys))


def test_no_pair_is_local():
    """Zero output and gradients without a shared expert."""
    import torch
    wl = make_workload("prefill", seed=203, T=20, H=256, I=128, E=16,
                       num_local=4, k=2, shared=False)
    wl.logits[:, :4] = -50.0
    s = Step(wl)
    for t in (s.b.out, s.b.d_x, s.b.d_w, *s.b.grads.values()):
        t.fill_(3.0)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    assert not s.b.saved["offsets"].any()
    assert (s.b.saved["pair_row"] == -1).all()
    for t in (s.b.out, s.b.d_x, s.b.d_w, *s.b.grads.values()):
        assert not t.any()


def test_no_tokens_clear_the_weights_gradients():
    import torch
    import expert_moe_fp32_amd as m
    wl = make_workload("prefill", seed=204, T=4, H=256, I=128, E=4,
                       num_local=4, k=2, shared=True)
    for grads in ("f32", "bf16"):
        s = Step(wl, grads)
        s.dl.p = m.make_problem(0, 256, 128, 4, 2, has_shared=True)
        for t in s.b.grads.values():
            t.fill_(3.0)
        s.b.out.fill_(3.0)
        s.forward()
        s.backward()
        torch.cuda.synchronize()
        assert not any(t.any() for t in s.b.grads.values())
        assert (s.b.out == 3.0).all()


def test_each_output_alone():
    """Any of the three outputs may be left out; the others are the same."""
    import torch
    import expert_moe_fp32_amd as m
    s = Step(make_workload("prefill", seed=205, T=90, H=256, I=256, E=8,
                           num_local=8, k=2, shared=True))
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    ref = s.outputs()
    b = s.b
    for x, w, g in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 1, 1)):
        for t in (b.d_x, b.d_w, *b.grads.values()):
            t.fill_(3.0)
        m.moe_experts_backward(s.dl.p, b.handle, s.d_out, s.dl.weights,
                               b.d_x if x else None, b.d_w if w else None,
                               b.grads_handle if g else None, b.ws,
                               b.ws.numel())
        torch.cuda.synchronize()
        got = s.outputs()
        for n in ("d_x", "d_w", *b.grads):
            on = {"d_x": x, "d_w": w}.get(n, g)
            assert torch.equal(got[n], ref[n]) if on else (got[n] == 3.0).all()


def test_the_output_is_the_layers():
    """The forward pass gives what moe_layer_forward gives, to the bars of the
    recipe: it differs by the order of sums alone."""
    import torch
    from .helpers import out_to_f64
    wl = make_workload("prefill", seed=206, T=700, H=512, I=256, E=8,
                       num_local=8, k=4, shared=True)
    s = Step(wl)
    s.forward()
    from expert_moe_fp32_amd.runner import to_dev
    lb = s.dl.buffers()
    s.dl.forward(lb, to_dev(wl.logits), None, s.x)
    torch.cuda.synchronize()
    check_output(f64(s.b.out), out_to_f64(lb, wl), "bf16", 1e-2)


def test_one_bad_row_stays_its_own():
    """A token of NaN reaches its own d_x and its experts' gradients only."""
    import torch
    wl = make_workload("prefill", seed=207, T=60, H=256, I=128, E=32,
                       num_local=32, k=2, shared=False)
    s = Step(wl)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    ref = s.outputs()
    s.d_out[5] = float("nan")
    s.backward()
    torch.cuda.synchronize()
    got = s.outputs()
    others = [t for t in range(60) if t != 5]
    assert got["d_x"][5].isnan().all() and got["d_w"][5].isnan().all()
    assert torch.equal(got["d_x"][others], ref["d_x"][others])
    assert torch.equal(got["d_w"][others], ref["d_w"][others])
    mine = set(s.ids[5].tolist())
    for e in range(32):
        for n in ("d_gate", "d_up", "d_down"):
            if e in mine:
                assert got[n][e].isnan().all()
            else:
                assert torch.equal(got[n][e], ref[n][e]), (n, e)


def test_replays_from_a_graph():
    """Forward and backward captured; replays with eager work between them
    equal the eager run bit for bit, also after the inputs change."""
    import torch
    kw = dict(T=150, H=256, I=256, E=16, num_local=8, k=4, shared=True)
    s = Step(make_workload("prefill", seed=208, **kw))
    other = Step(make_workload("prefill", seed=209, **kw), "bf16")

    def step():
        s.forward()
        s.backward()

    step()
    torch.cuda.synchronize()
    eager = s.outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for r in range(4):
        for t in (s.b.out, s.b.d_x, s.b.d_w, *s.b.grads.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, v in s.outputs().items():
            assert torch.equal(v, eager[n]), (r, n)
        other.forward()
        other.backward()
        torch.cuda.synchronize()
    s.x.copy_(s.x.flip(0).clone())
    s.d_out.copy_(s.d_out.flip(0).clone())
    step()
    torch.cuda.synchronize()
    eager = s.outputs()
    graph.replay()
    torch.cuda.synchronize()
    for n, v in s.outputs().items():
        assert torch.equal(v, eager[n]), n


def test_intermediate_arrays_beyond_32_bits():
    """More than 2^32 elements of gate and up: 70 copies of 1000 tokens get
    what the first copy gets, bit for bit (a row's result does not depend on
    its place), and the first what a pass of 1000 gets, to two roundings.  The
    weights' gradients are 70 times the pass's: a sum of n products in float32
    is within n u of the sum of their magnitudes, about 20 times such a sum of
    random signs here (1000 independent terms, 70 times over: 0.8 sqrt(1000))."""
    import torch
    copies, kw = 70, dict(H=128, I=16384, E=2, num_local=2, k=2, shared=False)
    wl = make_workload("prefill", seed=212, T=1000, **kw)
    one = Step(wl)
    one.forward()
    one.backward()
    torch.cuda.synchronize()

    class Copies(type(wl)):
        logits = property(lambda self: np.tile(wl.logits, (copies, 1)))
        x = property(lambda self: np.tile(wl.x, (copies, 1)))

    big = make_workload("prefill", seed=212, T=1000 * copies, **kw)
    big.__class__ = Copies
    s = Step(big)
    s.d_out = one.d_out.repeat(copies, 1)
    assert s.cap * 2 * wl.I > 2 ** 32
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    for name in ("out", "d_x", "d_w"):
        v = getattr(s.b, name).view(copies, 1000, -1)
        assert torch.equal(v, v[:1].expand_as(v)), name
        a, b = v[0].double(), getattr(one.b, name).double().view(1000, -1)
        assert (a - b).norm() <= 2 * B * b.norm(), name
    n = big.T * 2
    for name, v in s.b.grads.items():
        if v.numel():
            ref = copies * one.b.grads[name].double()
            assert (v.double() - ref).norm() <= 20 * n * U * ref.norm(), name


def test_weight_gradients_of_rows_beyond_32_bits():
    """Gradients of only the last of 70 copies of 1000 tokens, whose rows of
    the second expert lie past 2^32 elements of gate and up: what a pass of
    these 1000 gives, in norm to two roundings of the products' factors (the
    order of the float32 sums may differ: each is within (n + 1) u, n = 1000, of
    terms whose magnitudes add up to some 25 times the result, 1.5e-3)."""
    import torch
    copies, kw = 70, dict(H=128, I=16384, E=2, num_local=2, k=2, shared=False)
    wl = make_workload("prefill", seed=212, T=1000, **kw)
    one = Step(wl)
    one.forward()
    one.backward()

    class Copies(type(wl)):
        logits = property(lambda self: np.tile(wl.logits, (copies, 1)))
        x = property(lambda self: np.tile(wl.x, (copies, 1)))

    big = make_workload("prefill", seed=212, T=1000 * copies, **kw)
    big.__class__ = Copies
    s = Step(big)
    s.d_out = torch.zeros(big.T, wl.H, dtype=torch.bfloat16, device="cuda")
    s.d_out[-1000:] = one.d_out
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    # every token chose both experts: 70000 rows each
    assert s.disp.offsets[1] == big.T and (2 * big.T - 1000) * 2 * wl.I > 2 ** 32
    for name, v in s.b.grads.items():
        for p in range(2):
            ref = one.b.grads[name][p].double()
            err = (v[p].double() - ref).norm() / ref.norm()
            print(name, p, float(err), flush=True)
            assert err <= 2 * B, (name, p, float(err))


def test_two_streams_at_once():
    import torch
    runs = [(Step(make_workload("prefill", seed=210 + i, T=T, H=256, I=256,
                                E=8, num_local=8, k=2, shared=bool(i))),
             torch.cuda.Stream()) for i, T in enumerate((300, 77))]
    ref = []
    for s, _ in runs:
        s.forward()
        s.backward()
        torch.cuda.synchronize()
        ref.append(s.outputs())
    for _ in range(3):
        for s, q in runs:
            with torch.cuda.stream(q):
                s.forward()
                s.backward()
    torch.cuda.synchronize()
    for (s, _), r in zip(runs, ref):
        for n, v in s.outputs().items():
            assert torch.equal(v, r[n]), n


def test_a_training_step():
    """Router, experts and the norm at the layer's end, forward and backward,
    as a block runs them, against automatic differentiation of the whole
    formula in float64 with the choice held.  What separates the two is the
    8-bit checkpoint, at most 2^-4 a value and its root mean square below
    2^-5, through three factors of a product (x, g, u), and the bf16
    roundings: the root mean square of every gradient's error stays below an
    eighth of the gradient's."""
    import torch
    import expert_moe_fp32_amd as m
    wl = make_workload("prefill", seed=212, T=64, H=256, I=128, E=8,
                       num_local=8, k=2, shared=True)
    s = Step(wl)
    T, H, E, k = wl.T, wl.H, wl.E, wl.k
    g = torch.Generator().manual_seed(3)
    r = lambda *z: torch.randn(*z, generator=g).cuda()
    router = m.make_router(T, E, k, "sigmoid", scale=2.0)
    # (weights of 0.02 make small outputs: a norm behind them, as in a model)
    n = m.make_norm(T, H, "bf16", "f32", "f32", eps=1e-12)
    logits, resid, post, pre = r(T, E), r(T, H), r(H), r(H)
    d_x_next, d_ro = r(T, H), r(T, H)
    e = lambda *z, dt=torch.float32: torch.empty(*z, dtype=dt, device="cuda")
    ids, w = e(T, k, dt=torch.int32), e(T, k)
    ro, xn, d_block, d_resid = e(T, H), e(T, H), e(T, H, dt=torch.bfloat16), e(T, H)
    d_post, d_pre, d_logits = e(H), e(H), e(T, E)
    nws = torch.empty(m.moe_residual_norm_workspace_size(n), dtype=torch.uint8,
                      device="cuda")
    m.moe_route_scored(router, logits, None, ids, w)
    s.dl.experts_forward(s.b, s.x, ids, w)
    m.moe_residual_norm(n, s.b.out, resid, post, None, pre, ro, xn)
    m.moe_residual_norm_backward(n, s.b.out, ro, post, None, pre, d_x_next,
                                 d_ro, d_block, d_resid, d_post, None, d_pre,
                                 nws, nws.numel())
    s.dl.experts_backward(s.b, d_block)
    m.moe_route_scored_backward(router, logits, ids, s.b.d_w, d_logits)
    torch.cuda.synchronize()
    leaf = lambda a: torch.as_tensor(a).double().cpu().requires_grad_()
    x, lg = leaf(s.x), leaf(logits)
    W = [[leaf(v) for v in weights_of(wl, wl.expert(p))] for p in range(E)]
    Ws = [leaf(v) for v in weights_of(wl, wl.shared_expert)]
    ff = lambda z, v: (torch.nn.functional.silu(z @ v[0]) * (z @ v[1])) @ v[2]
    sc = lg.sigmoid().gather(1, ids.long().cpu())
    sc = 2.0 * sc / sc.sum(-1, keepdim=True)
    y = ff(x, Ws)
    every = torch.stack([ff(x, v) for v in W], 1)
    y = y + (every.gather(1, ids.long().cpu()[..., None].expand(T, k, H)) *
             sc[..., None]).sum(1)
    unit = lambda z: z / (z.pow(2).mean(-1, keepdim=True) + 1e-12).sqrt()
    ro64 = resid.double().cpu() + unit(y) * post.double().cpu()
    x64 = unit(ro64) * pre.double().cpu()
    ((x64 * d_x_next.double().cpu()).sum() +
     (ro64 * d_ro.double().cpu()).sum()).backward()
    pairs = [("x", s.b.d_x, x.grad), ("logits", d_logits, lg.grad)]
    for i, name in enumerate(("gate", "up", "down")):
        pairs.append((name, s.b.grads["d_" + name],
                      torch.stack([v[i].grad for v in W])))
        pairs.append(("shared " + name, s.b.grads["sh_" + name], Ws[i].grad))
    for name, got, ref in pairs:
        err = (got.double().cpu() - ref).pow(2).mean().sqrt() / ref.pow(2).mean().sqrt()
        print(name, float(err), flush=True)
        assert err <= 0.125, (name, float(err))


def copies_of(v, n):
    """Whether v's rows are its first n over and over."""
    import torch
    whole = v.shape[0] // n
    a = v[:whole * n].view(whole, n, -1)
    return (torch.equal(a, a[:1].expand_as(a)) and
            torch.equal(v[whole * n:], v[:v.shape[0] - whole * n]))


@pytest.mark.parametrize("shared", [False, True])
def test_more_tokens_than_a_launch_has_workgroups_for(shared):
    """2^24 + 4099 tokens of one expert, 4096 of them over and over: every
    copy gets what the first gets, bit for bit, and the first what a pass of
    4096 gets, to two roundings."""
    import torch
    import expert_moe_fp32_amd as m
    from expert_moe_fp32_amd.runner import DeviceLayer
    n, H, I = 4096, 128, 128
    g = torch.Generator().manual_seed(17)
    bits = lambda t: t.bfloat16().view(torch.int16).numpy().view(np.uint16)
    expert = lambda: dict(wg=bits(torch.randn(H, I, generator=g) / 11),
                          wu=bits(torch.randn(H, I, generator=g) / 11),
                          wd=bits(torch.randn(I, H, generator=g) / 11))
    first, also = expert(), expert()
    x, d_out = (torch.randn(n, H, generator=g).bfloat16().cuda() for _ in range(2))
    w = torch.rand(n, 1, generator=g).cuda()

    def run(T):
        dl = DeviceLayer(m.make_problem(T, H, I, 1, 1, has_shared=shared),
                         [first], also if shared else None)
        many = lambda t: t.repeat(-(-T // n), 1)[:T].contiguous()
        ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
        b = dl.train_buffers()
        for t in (b.out, b.d_x, b.d_w):
            t.fill_(7.0)
        dl.experts_forward(b, many(x), ids, many(w))
        dl.experts_backward(b, many(d_out))
        torch.cuda.synchronize()
        return b
    small, big = run(n), run(2 ** 24 + 4099)
    for name in ("out", "d_x", "d_w"):
        v, ref = getattr(big, name), getattr(small, name).double()
        assert copies_of(v, n), name
        assert (v[:n].double() - ref).norm() <= 2 * B * ref.norm(), name
