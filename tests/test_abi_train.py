"""The layer for a few tokens, 8-bit checkpoints and the experts' training
passes without a GPU: bad arguments are refused with the documented status
before a device is touched, and empty batches succeed."""
import pytest

import expert_moe_fp32_amd as m
from expert_moe_fp32_amd import _lib as L

BAD, UNSUP, WS = (L.MOE_ERR_INVALID_ARGUMENT, L.MOE_ERR_UNSUPPORTED,
                  L.MOE_ERR_WORKSPACE)
P = 4096                      # an address that is never read
BIG = 1 << 40


def problem(**kw):
    base = dict(T=8, H=256, I=128, E=16, k=2, num_local=4)
    base.update(kw)
    return m.make_problem(**base)


def weights(p=None, **without):
    w = L.Weights(*[P] * 12)
    for n in without:
        setattr(w, n, None)
    return w


# -------------------------------------------------------------- few tokens
def few(p, r=None, logits=P, bias=None, x=P, w=None, l2p=None, rep=None,
        out=P, counts=None, ws=P, n=BIG):
    return m.moe_layer_forward_few(p, r, logits, bias, x,
                                   weights() if w is None else w, l2p, rep,
                                   out, counts, ws, n, stream=0, check=False)


@pytest.mark.parametrize("kw,status", [
    (dict(T=17), UNSUP), (dict(T=-1), BAD), (dict(k=0), BAD),
    (dict(k=17, E=32), UNSUP), (dict(E=2048), UNSUP), (dict(H=200), UNSUP),
    (dict(act="f32", wdt="f32", out="f32"), UNSUP), (dict(T=2 ** 30), UNSUP),
], ids=str)
def test_few_validation(kw, status):
    p = problem(**kw)
    assert few(p) == status
    with pytest.raises(m.MoeError) as e:
        m.moe_layer_few_workspace_size(p)
    assert e.value.status == status


@pytest.mark.parametrize("kw,status", [
    (dict(H=2 ** 27 - 128), WS), (dict(H=2 ** 27), UNSUP),
    # 4 experts here: I / 16 of each
    (dict(I=2 ** 31 - 128), WS),
    (dict(I=2 ** 31 - 128, num_local=16, T=1), UNSUP),
    (dict(I=2 ** 30, num_local=16, E=256, k=16), WS),
    (dict(I=2 ** 30, num_local=16, E=256, k=16, has_shared=True), WS),
    (dict(I=2 ** 30, num_local=31, E=256, k=16, has_shared=True), UNSUP),
    (dict(I=2 ** 27, num_local=256, E=256, k=16), UNSUP),
    (dict(I=2 ** 27 - 128, num_local=256, E=256, k=16), WS),
    (dict(I=2 ** 27 - 128, num_local=256, E=256, k=16, has_shared=True), UNSUP),
], ids=str)
def test_few_limits(kw, status):
    assert few(problem(**kw), n=4096) == status


def test_few_arguments():
    p = problem()
    need = m.moe_layer_few_workspace_size(p)
    assert few(p, ws=None) == WS and few(p, n=need - 1) == WS
    for kw in (dict(logits=None), dict(x=None), dict(out=None), dict(x=P + 8),
               dict(out=P + 2), dict(w=weights(w_up=0)), dict(rep=P),
               dict(l2p=P)):
        assert few(p, **kw) == BAD, kw
    assert few(problem(num_physical=5)) == BAD           # without a map
    assert few(problem(has_shared=True), w=weights(sh_down=0)) == BAD
    assert few(problem(wdt="fp8"), w=weights(s_gate=0)) == BAD
    for r in (m.make_router(7, 16, 2), m.make_router(8, 15, 2),
              m.make_router(8, 16, 3)):
        assert few(p, r=r) == BAD
    assert few(p, r=m.make_router(8, 16, 2, groups=3)) == BAD
    # the query is the same for every batch, so one buffer serves them
    assert m.moe_layer_few_workspace_size(problem(T=1)) == need
    assert few(problem(T=0), logits=None, x=None, out=None, ws=None) == L.MOE_OK


# -------------------------------------------------------------- checkpoints
@pytest.mark.parametrize("kw,status", [
    (dict(), L.MOE_OK), (dict(rows=0), L.MOE_OK), (dict(rows=-1), BAD),
    (dict(cols=0), BAD), (dict(stride=99), BAD), (dict(stride=101), L.MOE_OK),
    (dict(dtype="fp8"), UNSUP), (dict(rows=2 ** 31 - 1, cols=129), UNSUP),
], ids=str)
def test_rows_validation(kw, status):
    base = dict(rows=4, cols=100, dtype="f32")
    base.update(kw)
    r = m.make_rows(**base)
    assert m.moe_check_rows(r) == status
    if status != L.MOE_OK:
        assert m.moe_checkpoint_rows(r, P, P, P, stream=0, check=False) == status
        assert m.moe_restore_rows(r, P, P, P, stream=0, check=False) == status


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols,status", [
    (2 ** 31 - 129, L.MOE_OK), (2 ** 31 - 128, L.MOE_OK),
    (2 ** 31 - 127, UNSUP), (2 ** 31 - 1, UNSUP)])
def test_columns_whose_last_group_leaves_32_bits(cols, status, dtype):
    r = m.make_rows(1, cols, dtype=dtype)
    assert m.moe_check_rows(r) == status
    if status != L.MOE_OK:
        assert m.moe_checkpoint_rows(r, P, P, P, stream=0, check=False) == status
        assert m.moe_restore_rows(r, P, P, P, stream=0, check=False) == status


def test_rows_arguments():
    r = m.make_rows(4, 100)
    r.dtype = 7
    assert m.moe_check_rows(r) == BAD
    r = m.make_rows(4, 100)
    for miss in range(3):
        args = [P, P, P]
        args[miss] = None
        assert m.moe_checkpoint_rows(r, *args, stream=0, check=False) == BAD
        assert m.moe_restore_rows(r, *args, stream=0, check=False) == BAD
    none = m.make_rows(0, 100)
    assert m.moe_checkpoint_rows(none, None, None, None, stream=0) == L.MOE_OK
    assert m.moe_restore_rows(none, None, None, None, stream=0) == L.MOE_OK


# ----------------------------------------------------------------- training
SAVED = ("offsets", "row_token", "row_weight", "pair_row", "x_codes",
         "x_scales", "gu_codes", "gu_scales")


def saved(**kw):
    return m.make_saved(**{**{n: P for n in SAVED}, **kw})


def forward(p, x=P, ids=P, w=P, l2p=None, rep=None, mw=None, sv=None, out=P,
            ws=P, n=BIG):
    return m.moe_experts_forward(p, x, ids, w, l2p, rep,
                                 weights() if mw is None else mw,
                                 saved() if sv is None else sv, out, ws, n,
                                 stream=0, check=False)


def backward(p, sv=None, d_out=P, mw=None, d_x=P, d_w=P, grads=None, ws=P,
             n=BIG):
    return m.moe_experts_backward(p, saved() if sv is None else sv, d_out,
                                  weights() if mw is None else mw, d_x, d_w,
                                  grads, ws, n, stream=0, check=False)


@pytest.mark.parametrize("kw,status", [
    (dict(act="f32", wdt="f32", out="f32"), UNSUP), (dict(wdt="fp8"), UNSUP),
    (dict(T=-1), BAD), (dict(I=100), UNSUP), (dict(E=2048), UNSUP),
], ids=str)
def test_training_validation(kw, status):
    p = problem(**kw)
    assert forward(p) == status and backward(p) == status
    with pytest.raises(m.MoeError):
        m.moe_experts_workspace_size(p)


@pytest.mark.parametrize("kw,status", [
    (dict(H=65536), WS), (dict(H=65536 + 128), UNSUP),
    (dict(I=65536), WS), (dict(I=65536 + 128), UNSUP),
    (dict(T=2 ** 30 - 1, k=1), WS), (dict(T=2 ** 30, k=1), UNSUP),
], ids=str)
def test_training_limits(kw, status):
    p = problem(**kw)
    assert forward(p, n=4096) == status and backward(p, n=4096) == status


def test_d_x_is_not_d_out():
    assert backward(problem(), d_x=P, d_out=P) == BAD


def test_forward_arguments():
    p = problem()
    for kw in (dict(x=None), dict(ids=None), dict(w=None), dict(out=None),
               dict(x=P + 2), dict(out=P + 8), dict(mw=weights(w_gate=0)),
               dict(rep=P), dict(l2p=P), dict(sv=saved(x_codes=P + 4)),
               dict(sv=saved(gu_codes=P + 8))):
        assert forward(p, **kw) == BAD, kw
    for n in SAVED:
        assert forward(p, sv=saved(**{n: None})) == BAD, n
    assert forward(p, ws=None) == WS and forward(p, n=4096) == WS
    assert forward(problem(has_shared=True), mw=weights(sh_up=0)) == BAD
    assert forward(problem(T=0), x=None, ids=None, w=None, out=None,
                   ws=None) == L.MOE_OK


def test_backward_arguments():
    p = problem()
    g = lambda **kw: m.make_weight_grads(**{**dict(
        d_gate=P, d_up=P, d_down=P), **kw})
    for kw in (dict(d_out=None), dict(d_out=P + 2), dict(d_x=P + 4),
               dict(mw=weights(w_down=0)), dict(grads=g(d_up=None)),
               dict(grads=g(d_down=P + 8)), dict(d_x=None, d_w=None)):
        assert backward(p, **kw) == BAD, kw
    for n in SAVED:
        assert backward(p, sv=saved(**{n: None})) == BAD, n
    assert backward(p, ws=None) == WS and backward(p, n=4096) == WS
    assert backward(p, grads=g(dtype="fp8")) == UNSUP
    bad = g()
    bad.dtype = 5
    assert backward(p, grads=bad) == BAD
    shared = problem(has_shared=True)
    assert backward(shared, grads=g(), n=0) == BAD       # sh_* missing
    assert backward(shared, grads=g(sh_gate=P, sh_up=P, sh_down=P), n=0) == WS
    assert backward(problem(T=0), d_out=None, ws=None) == L.MOE_OK


@pytest.mark.parametrize("kw", [dict(), dict(has_shared=True),
                                dict(num_local=16, k=8)], ids=str)
def test_workspace_grows_with_the_batch(kw):
    sizes = [m.moe_experts_workspace_size(problem(T=T, **kw))
             for T in (0, 1, 7, 8, 255, 256, 257, 1024, 1025, 5000)]
    assert sizes == sorted(sizes)
