"""The residual norm and its gradients on the GPU against the float64 oracle,
within bounds that count roundings (tests/norm_cases.py)."""
import numpy as np
import pytest

from .norm_cases import NormCase, check_backward, check_forward

pytestmark = pytest.mark.gpu

CASES = [
    dict(T=1, H=7168),
    dict(T=5, H=6144, gate="channel", rscale=0.22),
    dict(T=300, H=256, post=False),
    dict(T=3, H=16384, block="f32", resid="f32", out="f32", gate="full"),
    dict(T=70, H=8200, resid="f32", gain="bf16", offset=1.0),
    dict(T=9, H=1), dict(T=9, H=7, gate="full"),
    dict(T=33, H=65, block="f32", resid="f32", out="f32", gate="token"),
    dict(T=21, H=1003, gate="scalar", gain="bf16"),
    dict(T=21, H=1004, block="f32", out="f32", pads=(4, 0, 12, 8)),
    dict(T=17, H=2048, pads=(8, 16, 0, 24), gate="token"),
    dict(T=17, H=2048, pads=(1, 3, 5, 7), resid="f32"),
    dict(T=12, H=512, shift=1), dict(T=12, H=512, shift=3, resid="f32"),
    dict(T=12, H=16383, gate="channel", post=False, out="f32"),
    dict(T=1031, H=136, gate="channel"), dict(T=1031, H=24, gate="scalar"),
    dict(T=2, H=512, eps=0.0),
    dict(T=40, H=768, pre=False), dict(T=40, H=768, y=False, post=False),
    dict(T=1, H=2), dict(T=5, H=3, block="f32", resid="f32", out="f32"),
    dict(T=33, H=16384, gate="channel"), dict(T=300, H=12288, out="f32"),
    dict(T=270, H=4096, gate="token"), dict(T=20, H=7168, post=False),
    dict(T=600, H=2048, block="f32", resid="f32", out="f32", gate="channel"),
    dict(T=1031, H=512, gate="full"), dict(T=1031, H=512, gate="scalar"),
    dict(T=530, H=8192, resid="f32", gate="channel", rscale=-0.5),
]


@pytest.mark.parametrize("kw", CASES, ids=[str(c) for c in CASES])
def test_forward(kw):
    import torch
    c = NormCase(**kw, seed=1)
    before = c.edges(c.resid_out, c.x)
    print(kw, flush=True)
    c.forward()
    torch.cuda.synchronize()
    for (a, b), (d, e) in zip(before, c.edges(c.resid_out, c.x)):
        assert torch.equal(a, d) and torch.equal(b, e)
    check_forward(c, c.f64(c.resid_out), c.f64(c.x))


def run_backward(c, d_ro=True, in_place=False, poison=True):
    """Gradients of a case whose resid_out the forward made."""
    import torch
    import expert_moe_fp32_amd as m
    c.forward()
    d_x = c.rows(c.types["out"], c.pads[3]) if c.pre is not None else None
    d_r_out = c.rows(c.types["resid"], c.pads[2]) if d_ro else None
    dx64, dro64 = c.f64(d_x), c.f64(d_r_out)
    d_y = c.rows(c.types["block"], c.pads[0])
    d_r = d_r_out if in_place else c.rows(c.types["resid"], c.pads[1])
    new = lambda t: None if t is None else torch.full(t.shape, 7.0, device="cuda")
    d_post, d_gate, d_pre = new(c.post), new(c.gate), new(c.pre)
    size = m.moe_residual_norm_workspace_size(c.n)
    ws = torch.full((size,), 0xFF if poison else 0, dtype=torch.uint8,
                    device="cuda")                   # NaN throughout
    before = c.edges(d_y, d_r)
    m.moe_residual_norm_backward(c.n, c.y, c.resid_out, c.post, c.gate, c.pre,
                                 d_x, d_r_out, d_y, d_r, d_post, d_gate,
                                 d_pre, ws, size)
    torch.cuda.synchronize()
    for (a, b), (d, e) in zip(before, c.edges(d_y, d_r)):
        assert torch.equal(a, d) and torch.equal(b, e)
    got = dict(d_resid=c.f64(d_r), d_y=c.f64(d_y))
    for name, t in (("d_post", d_post), ("d_gate", d_gate), ("d_pre", d_pre)):
        if t is not None:
            got[name] = t.double().cpu().numpy()
    return got, c.f64(c.resid_out), dx64, dro64


@pytest.mark.parametrize("kw", CASES, ids=[str(c) for c in CASES])
def test_backward(kw):
    print(kw, flush=True)
    c = NormCase(**kw, seed=2)
    got, r, d_x, d_ro = run_backward(c)
    check_backward(c, got, r, d_x, d_ro)


@pytest.mark.parametrize("kw", [dict(T=64, H=1024),
                                dict(T=50, H=333, gate="full")])
def test_backward_without_and_over_the_residual_gradient(kw):
    c = NormCase(**kw, seed=3)
    got, r, d_x, d_ro = run_backward(c, d_ro=False)
    check_backward(c, got, r, d_x, None)
    got, r, d_x, d_ro = run_backward(c, in_place=True)
    check_backward(c, got, r, d_x, d_ro)


def test_each_gradient_alone():
    """Any one output without the others equals the same output of a call
    that asks for all."""
    import torch
    import expert_moe_fp32_amd as m
    c = NormCase(37, 776, gate="channel", seed=4)
    c.forward()
    d_x, d_ro = c.rows("bf16", 0), c.rows("bf16", 0)
    size = m.moe_residual_norm_workspace_size(c.n)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def call(which):
        outs = [c.rows("bf16", 0), c.rows("bf16", 0),
                torch.empty(776, device="cuda"),
                torch.empty(1, 776, device="cuda"),
                torch.empty(776, device="cuda")]
        args = [o if i in which else None for i, o in enumerate(outs)]
        m.moe_residual_norm_backward(c.n, c.y, c.resid_out, c.post, c.gate,
                                     c.pre, d_x, d_ro, *args, ws, size)
        torch.cuda.synchronize()
        return [o[:37] if o.dim() == 2 and o.shape[0] == 38 else o for o in outs]

    every = call(range(5))
    for i in range(5):
        assert torch.equal(call([i])[i], every[i]), i


def test_in_place_residual():
    import torch
    import expert_moe_fp32_amd as m
    for H in (1024, 1001):
        c = NormCase(31, H, seed=5)
        c.forward()
        r, x = c.resid.clone(), torch.empty_like(c.x)
        m.moe_residual_norm(c.n, c.y, r, c.post, c.gate, c.pre, r, x)
        torch.cuda.synchronize()
        assert torch.equal(r[:31], c.resid_out[:31])
        assert torch.equal(x[:31], c.x[:31])


def test_one_output_at_a_time():
    import torch
    import expert_moe_fp32_amd as m
    c = NormCase(31, 512, seed=6)
    c.forward()
    x = torch.empty_like(c.x)
    m.moe_residual_norm(c.n, c.y, c.resid, c.post, None, c.pre, None, x)
    r = torch.empty_like(c.resid_out)
    m.moe_residual_norm(c.n, c.y, c.resid, c.post, None, None, r, None)
    torch.cuda.synchronize()
    assert torch.equal(x[:31], c.x[:31]) and torch.equal(r[:31], c.resid_out[:31])


def test_bad_rows_stay_alone():
    """NaN and infinities in one row leave the others' results and come out
    in their own; a row of zeros gives zeros."""
    import torch
    c = NormCase(9, 640, seed=7)
    c.forward()
    torch.cuda.synchronize()
    r0, x0 = c.resid_out.clone(), c.x.clone()
    c.y[2, 5] = float("nan")
    c.resid[4, 6] = float("inf")
    c.y[6] = 0
    c.resid[6] = 0
    c.forward()
    torch.cuda.synchronize()
    for t in (0, 1, 3, 5, 7, 8):
        assert torch.equal(c.resid_out[t], r0[t]) and torch.equal(c.x[t], x0[t])
    assert torch.isnan(c.x[2]).all() and torch.isinf(c.resid_out[4, 6])
    assert (c.resid_out[6] == 0).all() and (c.x[6] == 0).all()


def test_zero_rows_clear_the_sums():
    import torch
    import expert_moe_fp32_amd as m
    n = m.make_norm(0, 520, gate_shape=(1, 520))
    v = torch.ones(520, device="cuda")
    outs = [torch.ones(520, device="cuda") for _ in range(3)]
    m.moe_residual_norm_backward(n, None, None, v, v, v, None, None, None,
                                 None, *outs, None, 0, stream=torch.cuda
                                 .current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert all((o == 0).all() for o in outs)


def test_repeatable():
    import torch
    c = NormCase(1500, 1000, gate="scalar", seed=8)
    a = run_backward(c)[0]
    c = NormCase(1500, 1000, gate="scalar", seed=8)
    b = run_backward(c, poison=False)[0]
    for name in a:
        assert np.array_equal(a[name], b[name]), name


def test_offsets_past_32_bits():
    """T * H beyond 2^31: the last rows equal the same rows on their own."""
    import torch
    import expert_moe_fp32_amd as m
    H = 8192
    T = 2 ** 31 // H + 300
    bf = torch.bfloat16
    y = torch.ones(T, H, dtype=bf, device="cuda")
    r = torch.ones(T, H, dtype=bf, device="cuda")
    y[-16:] = torch.randn(16, H, device="cuda").to(bf)
    gain = torch.randn(H, device="cuda")
    ro, x = torch.empty_like(r), torch.empty_like(r)
    n = m.make_norm(T, H)
    m.moe_residual_norm(n, y, r, gain, None, gain, ro, x)
    n2 = m.make_norm(16, H)
    ro2, x2 = torch.empty(16, H, dtype=bf, device="cuda"), torch.empty(
        16, H, dtype=bf, device="cuda")
    m.moe_residual_norm(n2, y[-16:], r[-16:], gain, None, gain, ro2, x2)
    torch.cuda.synchronize()
    assert torch.equal(ro[-16:], ro2) and torch.equal(x[-16:], x2)
    d_y, d_r = torch.empty_like(y), torch.empty_like(y)
    ws = torch.empty(m.moe_residual_norm_workspace_size(n), dtype=torch.uint8,
                     device="cuda")
    m.moe_residual_norm_backward(n, y, ro, gain, None, gain, x, None, d_y, d_r,
                                 None, None, None, ws, ws.numel())
    d_y2, d_r2 = torch.empty_like(x2), torch.empty_like(x2)
    m.moe_residual_norm_backward(n2, y[-16:], ro2, gain, None, gain, x2, None,
                                 d_y2, d_r2, None, None, None, ws, ws.numel())
    torch.cuda.synchronize()
    assert torch.equal(d_y[-16:], d_y2) and torch.equal(d_r[-16:], d_r2)


def test_one_workspace_for_every_batch():
    """A buffer of the largest batch's size serves the smaller ones."""
    import torch
    import expert_moe_fp32_amd as m
    size = m.moe_residual_norm_workspace_size(m.make_norm(1000, 512))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    for T in (1000, 257, 256, 3):
        c = NormCase(T, 512, seed=10)
        c.forward()
        d_x, outs = c.rows("bf16", 0), []
        for w in (ws, torch.empty(m.moe_residual_norm_workspace_size(c.n),
                                  dtype=torch.uint8, device="cuda")):
            d_r, d_pre = c.rows("bf16", 0), torch.empty(512, device="cuda")
            m.moe_residual_norm_backward(c.n, c.y, c.resid_out, c.post, None,
                                         c.pre, d_x, None, None, d_r, None,
                                         None, d_pre, w, w.numel())
            outs.append((d_r[:T], d_pre))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("T,H,post,gate", [
    (1031, 512, True, "scalar"), (258, 256, False, None),
    (261, 72, True, "channel")])
def test_infinite_gradient_in_the_last_row(T, H, post, gate):
    """An infinity in the last row's d_x reaches its own column's d_pre as an
    infinity, whatever the number of rows that share a workgroup; the other
    columns stay as they are."""
    import torch
    import expert_moe_fp32_amd as m
    c = NormCase(T, H, post=post, gate=gate, seed=9)
    c.forward()
    d_x = c.rows("bf16", 0)
    size = m.moe_residual_norm_workspace_size(c.n)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def d_pre():
        out = torch.empty(H, device="cuda")
        m.moe_residual_norm_backward(
            c.n, c.y, c.resid_out, c.post, c.gate, c.pre, d_x, None,
            c.rows("bf16", 0), c.rows("bf16", 0), None, None, out, ws, size)
        torch.cuda.synchronize()
        return out

    at = H // 2 + 1
    assert c.resid_out[T - 1, at] != 0
    ref = d_pre()
    d_x[T - 1, at] = float("inf")
    got = d_pre()
    sign = float(torch.sign(c.resid_out[T - 1, at].float()))
    assert float(got[at]) == sign * float("inf")
    keep = torch.arange(H, device="cuda") != at
    assert torch.equal(got[keep], ref[keep])
