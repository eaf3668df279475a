"""Scored routing, residual norm and combine gradients without a GPU: every
bad argument is refused with the documented status before a device is
touched, and empty batches succeed."""
import pytest

import expert_moe_fp32_amd as m
from expert_moe_fp32_amd import _lib as L

BAD, UNSUP, WS = (L.MOE_ERR_INVALID_ARGUMENT, L.MOE_ERR_UNSUPPORTED,
                  L.MOE_ERR_WORKSPACE)
P = 4096                      # an address that is never read


def router(**kw):
    base = dict(T=64, E=256, k=8, score="sigmoid", groups=8, topk_groups=4,
                group_top=2)
    base.update(kw)
    field = {n: base.pop(n) for n in list(base) if n.startswith("_")}
    r = m.make_router(**base)
    for n, v in field.items():
        setattr(r, n[1:], v)
    return r


@pytest.mark.parametrize("kw,status", [
    (dict(), L.MOE_OK),
    (dict(T=0), L.MOE_OK),
    (dict(T=-1), BAD),
    (dict(k=0), BAD),
    (dict(k=17, groups=1, topk_groups=1), UNSUP),
    (dict(E=4, k=5, groups=1, topk_groups=1), BAD),
    (dict(E=2048), UNSUP),
    (dict(groups=0), BAD),
    (dict(groups=7), BAD),                       # does not divide E
    (dict(groups=128, topk_groups=64), UNSUP),
    (dict(topk_groups=0), BAD),
    (dict(topk_groups=9), BAD),
    (dict(E=16, groups=8, topk_groups=2), BAD),  # keeps 4 of 8 experts wanted
    (dict(group_top=0), BAD),
    (dict(group_top=3), BAD),
    (dict(_renormalize=2), BAD),
    (dict(_score=2), BAD),
    (dict(scale=float("nan")), BAD),
    (dict(scale=float("inf")), BAD),
    (dict(logits="bf16"), L.MOE_OK),
    (dict(logits="fp8"), UNSUP),
    (dict(_logits_dtype=9), BAD),
    (dict(logits_stride=255), BAD),
    (dict(logits_stride=257), L.MOE_OK),
    (dict(T=2 ** 28), UNSUP),                    # T * k past 32 bits
])
def test_router_validation(kw, status):
    r = router(**kw)
    assert m.moe_check_router(r) == status
    if status != L.MOE_OK:
        assert m.moe_route_scored(r, P, P, P, P, P, P, 1 << 30, stream=0,
                                  check=False) == status
        assert m.moe_route_scored_backward(r, P, P, P, 2 * P, stream=0,
                                           check=False) == status
        with pytest.raises(m.MoeError):
            m.moe_route_scored_workspace_size(r)


def test_router_arguments():
    r = router()
    for miss in range(4):
        args = [P, P, P, P]                # logits, bias, ids, weights
        args[miss] = None
        if miss == 1:
            continue                       # the bias is optional
        assert m.moe_route_scored(r, *args, stream=0, check=False) == BAD
    for miss in range(4):
        args = [P, P, P, 2 * P]
        args[miss] = None
        assert m.moe_route_scored_backward(r, *args, stream=0,
                                           check=False) == BAD
    assert m.moe_route_scored_backward(r, P, P, P, P, stream=0,
                                       check=False) == BAD    # in place
    big = router(T=100000)
    need = m.moe_route_scored_workspace_size(big)
    assert need > 0
    for ws, n in ((None, need), (P, need - 1)):
        assert m.moe_route_scored(big, P, P, P, P, P, ws, n, stream=0,
                                  check=False) == WS


def norm(**kw):
    base = dict(T=8, H=256)
    base.update(kw)
    return m.make_norm(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(), L.MOE_OK),
    (dict(T=0), L.MOE_OK),
    (dict(T=-1), BAD),
    (dict(H=0), BAD),
    (dict(H=1), L.MOE_OK),
    (dict(H=16384), L.MOE_OK),
    (dict(H=16385), UNSUP),
    (dict(eps=-1e-6), BAD),
    (dict(eps=float("nan")), BAD),
    (dict(eps=0.0), L.MOE_OK),
    (dict(residual_scale=float("inf")), BAD),
    (dict(gain_offset=float("nan")), BAD),
    (dict(block="fp8"), UNSUP),
    (dict(resid="fp8"), UNSUP),
    (dict(out="fp8"), UNSUP),
    (dict(gain="fp8"), UNSUP),
    (dict(block_stride=255), BAD),
    (dict(resid_stride=255), BAD),
    (dict(resid_out_stride=255), BAD),
    (dict(out_stride=255), BAD),
    (dict(out_stride=300), L.MOE_OK),
])
def test_norm_validation(kw, status):
    n = norm(**kw)
    assert m.moe_check_norm(n) == status
    if status != L.MOE_OK:
        assert m.moe_residual_norm(n, P, P, None, None, P, P, P, stream=0,
                                   check=False) == status
        with pytest.raises(m.MoeError):
            m.moe_residual_norm_workspace_size(n)


def forward(n, y=P, resid=P, post=None, gate=None, pre=P, ro=2 * P, x=3 * P):
    return m.moe_residual_norm(n, y, resid, post, gate, pre, ro, x, stream=0,
                               check=False)


def test_norm_arguments():
    n = norm()
    assert forward(n, resid=None) == BAD
    assert forward(n, pre=None) == BAD               # x_out without a gain
    assert forward(n, x=None) == BAD                 # a gain without x_out
    assert forward(n, pre=None, x=None, ro=None) == BAD
    assert forward(n, y=None, post=P) == BAD
    assert forward(n, y=None, gate=P) == BAD
    for shape in ((2, 1), (1, 2), (0, 1), (8, 255), (256, 8)):
        assert forward(norm(gate_shape=shape), gate=P) == BAD


def test_norm_in_place_needs_one_stride():
    n = norm(resid_stride=300)
    assert forward(n, ro=P) == BAD
    assert backward(n, d_ro=P, d_r=P) == BAD


def backward(n, y=P, ro=P, post=P, gate=None, pre=P, d_x=P, d_ro=P, d_y=P,
             d_r=P, d_post=P, d_gate=None, d_pre=P, ws=P, size=1 << 30):
    return m.moe_residual_norm_backward(
        n, y, ro, post, gate, pre, d_x, d_ro, d_y, d_r, d_post, d_gate, d_pre,
        ws, size, stream=0, check=False)


def test_norm_backward_arguments():
    n = norm()
    need = m.moe_residual_norm_workspace_size(n)
    assert backward(n, size=need - 1) == WS
    assert backward(n, ws=None) == WS
    assert backward(n, y=None) == BAD
    assert backward(n, ro=None) == BAD
    assert backward(n, d_x=None) == BAD
    assert backward(n, pre=None, d_pre=None) == BAD          # d_x without it
    assert backward(n, pre=None, d_x=None) == BAD            # d_pre without it
    assert backward(n, post=None) == BAD                     # d_post without it
    assert backward(n, d_gate=P) == BAD                      # no gate
    assert backward(n, pre=None, d_x=None, d_pre=None, d_ro=None) == BAD
    assert backward(n, d_y=None, d_r=None, d_post=None, d_pre=None) == BAD
    assert backward(norm(gate_shape=(3, 1)), gate=P) == BAD


def problem(**kw):
    base = dict(T=8, H=256, I=128, E=16, k=4, num_local=8)
    base.update(kw)
    return m.make_problem(**base)


def test_combine_norm_arguments():
    p, n = problem(), norm()

    def call(p=p, n=n, y=P, rows=P, w=P, sh=None, resid=P, pre=P, ro=P, x=P,
             gate=None):
        return m.moe_combine_norm(p, n, y, rows, w, sh, resid, None, gate,
                                  pre, None, ro, x, stream=0, check=False)

    assert call(y=None) == BAD
    assert call(rows=None) == BAD
    assert call(w=None) == BAD
    assert call(resid=None) == BAD
    assert call(x=None) == BAD
    assert call(ro=None, x=None, pre=None) == BAD
    assert call(y=P + 4) == BAD
    assert call(sh=P + 8) == BAD
    assert call(n=norm(T=9)) == BAD
    assert call(n=norm(H=384)) == BAD
    assert call(n=norm(gate_shape=(2, 2)), gate=P) == BAD
    assert call(n=norm(eps=-1.0)) == BAD
    assert call(p=problem(H=200)) == UNSUP
    assert call(p=problem(T=0), n=norm(T=0), y=None) == L.MOE_OK


def test_combine_backward_arguments():
    p = problem()

    def call(d=P, y=P, rows=P, w=P, dy=P, dw=P, ds=None, p=p):
        return m.moe_combine_backward(p, d, y, rows, w, dy, dw, ds, stream=0,
                                      check=False)

    assert call(d=None) == BAD
    assert call(rows=None) == BAD
    assert call(w=None) == BAD
    assert call(y=None) == BAD                   # d_topk_w needs the rows
    assert call(dy=None, dw=None) == BAD
    for name in ("d", "y", "dy", "ds"):
        assert call(**{name: P + 8}) == BAD
    assert call(p=problem(T=0), d=None) == L.MOE_OK


def test_scored_layer_arguments():
    p, n, r = problem(), norm(), m.make_router(8, 16, 4)
    w = L.Weights()
    w.w_gate = w.w_up = w.w_down = P

    def call(p=p, r=r, n=n, logits=P, x=P, weights=w, resid=P, pre=P, out=None,
             ro=P, xo=P, ws=P, size=1 << 40):
        return m.moe_layer_forward_scored(
            p, r, n, logits, None, x, weights, None, None, resid, None, None,
            pre, out, ro, xo, None, ws, size, stream=0, check=False)

    assert call(r=m.make_router(9, 16, 4)) == BAD
    assert call(r=m.make_router(8, 32, 4)) == BAD
    assert call(r=m.make_router(8, 16, 3)) == BAD
    assert call(r=m.make_router(8, 16, 4, groups=3)) == BAD
    assert call(n=norm(H=128)) == BAD
    assert call(logits=None) == BAD
    assert call(x=None) == BAD
    assert call(x=P + 2) == BAD
    assert call(resid=None) == BAD
    assert call(pre=None) == BAD
    assert call(weights=L.Weights()) == BAD
    assert call(n=None, out=P) == BAD            # the norm's arrays without it
    none = dict(n=None, resid=None, pre=None, ro=None, xo=None)
    assert call(**none) == BAD                   # no out either
    assert call(**none, out=P, ws=None) == WS
    assert call(size=m.moe_layer_workspace_size(p) - 1) == WS


def test_zero_tokens_enqueue_nothing():
    r, n = router(T=0), norm(T=0)
    assert m.moe_route_scored(r, None, None, None, None, stream=0,
                              check=False) == L.MOE_OK
    assert m.moe_route_scored_backward(r, None, None, None, None, stream=0,
                                       check=False) == L.MOE_OK
    assert m.moe_residual_norm(n, None, None, None, None, None, None, None,
                               stream=0, check=False) == L.MOE_OK
    assert m.moe_residual_norm_backward(
        n, *[None] * 12, None, 0, stream=0, check=False) == L.MOE_OK


def test_calls_go_to_the_device_of_their_arrays(monkeypatch):
    """Without a stream argument a call runs on the current stream of the
    device that holds its arrays, with that device current."""
    import contextlib

    import torch

    class OnDevice1:
        is_cuda = True
        device = torch.device("cuda", 1)

        def data_ptr(self):
            return P

    seen = []

    @contextlib.contextmanager
    def device(d):
        seen.append(("enter", d))
        yield
        seen.append(("leave", d))

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(L, "_raw_stream", lambda d: seen.append(("stream", d)) or 0)
    a = OnDevice1()
    m.moe_residual_norm(norm(T=0), a, a, None, None, a, a, a)
    assert seen == [("enter", 1), ("stream", 1), ("leave", 1)]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    del seen[:]
    m.moe_route_scored_backward(router(T=0), a, a, a, a)
    assert seen == [("stream", 1)]


def bare_layer(p):
    """A DeviceLayer's calls without its weights or a device."""
    from expert_moe_fp32_amd.runner import DeviceLayer
    dl = object.__new__(DeviceLayer)
    dl.p, dl.weights, dl.l2p, dl.rep = p, L.Weights(), None, None
    return dl


class Anything:
    """Buffers that stand for addresses."""

    def __getattr__(self, name):
        return type("Buffer", (), {"numel": lambda s: 1 << 40,
                                   "data_ptr": lambda s: P})()


@pytest.mark.parametrize("kw", [
    dict(block="f32"),                           # rows twice as long
    dict(block_stride=264),
    dict(block="f32", block_stride=512),
], ids=str)
def test_layer_buffers_take_no_other_block_rows(monkeypatch, kw):
    """A layer's `out` buffer holds T x H elements of the problem's out_dtype:
    combined rows of another type or stride never go there."""
    for name in ("moe_layer_forward_scored", "moe_combine_norm"):
        monkeypatch.setattr(L, name, lambda *a, _n=name, **k: _n)
    p, b = problem(out="bf16"), Anything()
    dl, r = bare_layer(p), m.make_router(8, 16, 4)
    n = norm(**kw)

    def calls(n, **k):
        return [lambda: dl.forward_scored(b, r, P, None, P, n, P, None, None,
                                          P, P, P, **k),
                lambda: dl.combine_norm(b, n, P, None, None, P, P, P, **k)]

    for call in calls(n):
        with pytest.raises(m.MoeError) as e:
            call()
        assert e.value.status == BAD
    for call in calls(n, out=False) + calls(norm()):     # no rows, or fitting
        assert call().startswith("moe_")
    assert dl.forward_scored(b, r, P, None, P) == "moe_layer_forward_scored"
    one = bare_layer(problem(T=1))               # a single row has no stride
    assert one.combine_norm(b, norm(T=1, block_stride=264), P, None, None, P,
                            P, P) == "moe_combine_norm"
    f32 = bare_layer(problem(out="f32", act="f32", wdt="f32"))
    with pytest.raises(m.MoeError):
        f32.combine_norm(b, norm(), P, None, None, P, P, P)


@pytest.mark.parametrize("size", [(9, 16, 4), (8, 32, 4), (8, 16, 5)],
                         ids=str)
def test_layer_buffers_take_no_other_routing(monkeypatch, size):
    """A layer's ids, weights and counts hold its problem's T, k and E."""
    monkeypatch.setattr(L, "moe_route_scored", lambda *a, **k: "called")
    dl = bare_layer(problem())
    dl.device = "cpu"
    with pytest.raises(m.MoeError) as e:
        dl.route_scored(Anything(), m.make_router(*size), P, None)
    assert e.value.status == BAD
    for fits in ((8, 16, 4), (4, 16, 4), (8, 8, 4)):
        assert dl.route_scored(Anything(), m.make_router(*fits), P,
                               None) == "called"


def test_a_buffer_for_many_rows_serves_fewer():
    """Workspaces never shrink as T grows, and a call takes the buffer that
    the query gave for a larger batch."""
    edges = sorted({0, 1, 2, 8, 9, 64, 4097, 8192, 9001, 20000, 100000} | {
        t + d for t in (128, 256, 320, 512, 768, 1024, 1280, 1792, 2048, 4096)
        for d in (-1, 0, 1, 2, 3, 40)})
    for H in (1, 64, 72, 512, 520, 1000, 1024, 1032, 2501, 4096, 4104, 7168,
              8192, 8200, 16384):
        size = [m.moe_residual_norm_workspace_size(norm(T=t, H=H)) for t in edges]
        assert size == sorted(size), H
    for E, k in ((8, 2), (64, 6), (65, 8), (256, 16), (256, 8), (1000, 1)):
        size = [m.moe_route_scored_workspace_size(m.make_router(t, E, k))
                for t in edges]
        assert size == sorted(size), (E, k)


def test_any_array_names_the_device(monkeypatch):
    """A batch of no rows may come without the arrays that usually name the
    device; the sums that it clears name it as well."""
    import contextlib

    import torch

    class OnDevice1:
        is_cuda = True
        device = torch.device("cuda", 1)

        def data_ptr(self):
            return P

    seen = []

    @contextlib.contextmanager
    def device(d):
        seen.append(d)
        yield

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(L, "_raw_stream", lambda d: d)
    calls = {}

    class Library:                         # nothing is launched
        def __getattr__(self, name):
            def call(*args):
                calls[name] = args[-1]
                return L.MOE_OK
            call.__name__ = name
            return call

    monkeypatch.setattr(L, "_lib", Library())
    monkeypatch.setattr(L, "lib", lambda: L._lib)
    n, r, p, w = norm(T=0), router(T=0), problem(T=0), L.Weights()
    # (name, call on a list of arrays, how many)
    for name, count, call in (
            ("moe_route_scored", 6, lambda a: m.moe_route_scored(r, *a)),
            ("moe_route_scored_backward", 4,
             lambda a: m.moe_route_scored_backward(r, *a)),
            ("moe_residual_norm", 7, lambda a: m.moe_residual_norm(n, *a)),
            ("moe_residual_norm_backward", 13,
             lambda a: m.moe_residual_norm_backward(n, *a, 0)),
            ("moe_combine_norm", 11, lambda a: m.moe_combine_norm(p, n, *a)),
            ("moe_combine_backward", 7,
             lambda a: m.moe_combine_backward(p, *a)),
            ("moe_layer_forward_scored", 14, lambda a:
             m.moe_layer_forward_scored(p, r, n, *a[:3], w, *a[3:], 0))):
        for at in range(count):
            arrays = [None] * count
            arrays[at] = OnDevice1()
            del seen[:]
            call(arrays)
            assert seen == [1] and calls[name] == 1, (name, at)
