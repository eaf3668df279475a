"""Scored routing and its gradient on the GPU against the float64 oracle.

Ids and counts are equal.  The weights and gradients are evaluated in 64 bits
and rounded once, so they are off by half a step of their type (bf16 ones go
through float32: half a step of each) and the 64-bit terms' own rounding."""
import numpy as np
import pytest

from oracle import block as ob

pytestmark = pytest.mark.gpu


def make_logits(T, E, dtype, seed, masked=0.0, ties=False, pad=0):
    import torch
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E + pad, generator=g)
    if ties:
        l = torch.round(2 * l) / 2
    if masked:
        l[torch.rand(T, E + pad, generator=g) < masked] = float("-inf")
    return l.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def route(logits, bias, k, counts=True, **kw):
    """The call on a [T][E] view of `logits`; returns device results."""
    import torch
    import expert_moe_fp32_amd as m
    T, E = logits.shape
    r = m.make_router(T, E, k, logits="bf16" if logits.dtype ==
                      torch.bfloat16 else "f32",
                      logits_stride=logits.stride(0) if T > 1 else None, **kw)
    ids = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    c = torch.full((E,), 123, dtype=torch.int32, device="cuda")
    n = m.moe_route_scored_workspace_size(r)
    ws = torch.full((n,), 77, dtype=torch.uint8, device="cuda") if n else None
    m.moe_route_scored(r, logits, bias, ids, w, c if counts else None, ws, n)
    torch.cuda.synchronize()
    assert (ids[T] == -7).all() and (w[T] == -7.0).all()
    return r, ids[:T], w[:T], c


def to_f64(t):
    return t.double().cpu().numpy()


def check_route(logits, bias, k, **kw):
    _, ids, w, c = route(logits, bias, k, **kw)
    rid, rw, rc = ob.route_scored(to_f64(logits),
                                  None if bias is None else to_f64(bias), k,
                                  **kw)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.array_equal(c.cpu().numpy(), rc)
    tol = np.abs(rw) * 2.0 ** -24 * (1 + 1e-6) + 2.0 ** -149
    assert (np.abs(to_f64(w) - rw) <= tol).all()
    return rid


SHAPES = [  # T, E, k, groups, topk_groups, group_top
    (1, 256, 8, 8, 4, 2), (37, 256, 8, 8, 4, 2), (700, 256, 8, 1, 1, 1),
    (64, 160, 6, 8, 3, 1), (33, 8, 2, 1, 1, 1), (5, 1, 1, 1, 1, 1),
    (130, 16, 16, 1, 1, 1), (67, 64, 6, 64, 6, 1), (50, 60, 4, 5, 2, 2),
    (41, 100, 5, 4, 1, 2), (29, 128, 8, 4, 4, 2), (23, 384, 8, 6, 3, 2),
    (19, 1024, 16, 64, 5, 2), (11, 1000, 12, 8, 2, 2), (9, 30, 3, 3, 1, 2),
    (17, 192, 6, 3, 2, 1),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_shapes(shape, score, dtype):
    import torch
    T, E, k, G, keep, top = shape
    print(shape, score, dtype, flush=True)
    logits = make_logits(T, E, dtype, 11).cuda()
    bias = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(3))).cuda()
    kw = dict(score=score, groups=G, topk_groups=keep, group_top=top)
    check_route(logits, bias, k, scale=2.5, **kw)
    check_route(logits, None, k, renormalize=False, **kw)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep", [(256, 8, 4), (48, 4, 2), (512, 1, 1)])
def test_ties_take_the_lowest_id(score, E, G, keep):
    import torch
    logits = make_logits(200, E, "bf16", 5, ties=True).cuda()
    logits[3] = 1.0
    logits[4] = -0.0
    logits[4, ::2] = 0.0
    bias = torch.zeros(E).cuda()
    for b in (None, bias):
        ids = check_route(logits, b, 6, score=score, groups=G,
                          topk_groups=keep, group_top=2)
        assert ids[3].tolist() == ids[4].tolist() == list(range(6))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep,k", [(256, 8, 4, 8), (24, 4, 2, 9),
                                        (640, 10, 1, 16)])
def test_masked_experts_and_rows(score, E, G, keep, k):
    import torch
    inf, nan = float("inf"), float("nan")
    logits = make_logits(120, E, "f32", 9, masked=0.7)
    logits[0] = -inf                       # a row masked throughout
    logits[1] = nan
    logits[2, 1:] = -inf                   # one expert left
    logits[3] = -inf
    logits[3, E - 1] = -80.0
    logits[4, :E // 2] = nan
    logits[5, 5] = inf
    logits[6, 5:9] = inf
    logits[7] = torch.finfo(torch.float32).min
    logits[8] = -120.0                     # scores far below float32's range
    logits[8, 7] = -119.0
    bias = 0.3 * torch.randn(E, generator=torch.Generator().manual_seed(1))
    bias[2], bias[3], bias[4] = -inf, nan, 1e30
    logits, bias = logits.cuda(), bias.cuda()
    kw = dict(score=score, groups=G, topk_groups=keep, group_top=2)
    for b in (None, bias):
        check_route(logits, b, k, **kw)
        check_route(logits, b, k, renormalize=False, **kw)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep", [(256, 8, 4), (64, 1, 1), (120, 6, 3)])
def test_choices_closer_than_float32_resolves(score, E, G, keep):
    """Equal logits told apart by biases some 1e-9 apart, and distinct logits
    whose choices a bias brings together: the order is that of 64 bits."""
    import torch
    g = torch.Generator().manual_seed(8)
    logits = make_logits(300, E, "f32", 14, ties=True)
    bias = 1e-9 * torch.randn(E, generator=g)
    # rows of one value but for steps of an ulp or so
    logits[::3] = 1.0 + 2.0 ** -23 * torch.randint(0, 4, (100, E), generator=g)
    logits, bias = logits.cuda(), bias.cuda()
    for b in (bias, None):
        check_route(logits, b, 8, score=score, groups=G, topk_groups=keep,
                    group_top=2)
    # choices all within 1e-7: the bias undoes the scores of one row
    row = logits[1:2].expand(64, E).contiguous()
    s = ob.scores(to_f64(row), score)[0]
    undo = torch.from_numpy((0.5 - s).astype(np.float32)).cuda()
    check_route(row, undo, 8, score=score, groups=G, topk_groups=keep,
                group_top=2)


def test_sliced_logits():
    """Rows of a wider array, from a base that is not 16-byte aligned."""
    for dtype in ("f32", "bf16"):
        wide = make_logits(77, 256, dtype, 21, pad=5).cuda()
        for at in (0, 1, 5):
            check_route(wide[:, at:at + 256], None, 8, score="sigmoid",
                        groups=8, topk_groups=4, group_top=2)


def test_large_batch_counts():
    """More pairs than one workgroup counts; all of them on one expert too."""
    import torch
    logits = make_logits(9001, 64, "f32", 2).cuda()
    check_route(logits, None, 6, score="sigmoid")
    bias = torch.zeros(64)
    bias[63] = 50.0
    check_route(logits, bias.cuda(), 1, score="sigmoid")


def test_zero_tokens_clear_the_counts():
    import torch
    import expert_moe_fp32_amd as m
    c = torch.full((256,), 5, dtype=torch.int32, device="cuda")
    m.moe_route_scored(m.make_router(0, 256, 8), None, None, None, None, c)
    assert (c == 0).all()


def check_backward(logits, k, out_pad=0, **kw):
    import torch
    import expert_moe_fp32_amd as m
    T, E = logits.shape
    r, ids, _, _ = route(logits, None, k, **kw)
    d_w = torch.randn(T, k, device="cuda",
                      generator=torch.Generator("cuda").manual_seed(4))
    stride = logits.stride(0) if T > 1 else E
    d = torch.full((T + 1, stride), 9.0, device="cuda", dtype=logits.dtype)
    m.moe_route_scored_backward(r, logits, ids, d_w, d)
    torch.cuda.synchronize()
    if stride > E:
        assert (d[:, E:] == 9.0).all()
    assert (d[T] == 9.0).all()
    got = to_f64(d[:T, :E])
    sc, ren = kw.get("score", "softmax"), kw.get("renormalize", True)
    scale = kw.get("scale", 1.0)
    l64, id64 = to_f64(logits), ids.cpu().numpy()
    ref = ob.route_scored_backward(l64, id64, to_f64(d_w), sc, ren, scale)
    half = 2.0 ** -24
    if logits.dtype == torch.bfloat16:
        half += 2.0 ** -8
    # the 64-bit evaluation: a dozen roundings of terms no larger than
    # scale |d_w| s / S (S the chosen scores' sum), summed over the slots
    s = ob.scores(l64, sc)
    S = np.take_along_axis(s, id64, 1).sum(1, keepdims=True) if ren else 1.0
    big = scale * np.abs(to_f64(d_w)).sum(1, keepdims=True)
    live = np.broadcast_to(np.asarray(S) > 0, (T, 1))
    term = np.where(live, big * s / np.where(live, S, 1.0), 0.0)
    tol = np.abs(ref) * half * (1 + 1e-6) + 32 * 2.0 ** -53 * term + 2.0 ** -133
    assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_shapes(shape, score, renorm):
    T, E, k, G, keep, top = shape
    print(shape, score, renorm, flush=True)
    for dtype in ("f32", "bf16"):
        check_backward(make_logits(T, E, dtype, 31).cuda(), k, score=score,
                       groups=G, topk_groups=keep, group_top=top,
                       renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_masked_and_sliced(score, renorm):
    logits = make_logits(90, 40, "f32", 13, masked=0.8, pad=3)
    logits[0] = float("-inf")
    logits[1] = float("nan")
    logits[2, 4] = 60.0                    # a saturated sigmoid
    logits[3] = -90.0
    check_backward(logits.cuda()[:, :40], 5, score=score, renormalize=renorm)


def test_backward_ids_out_of_range_and_twice():
    """An id outside the experts gets no gradient; an id given twice gets
    both slots' parts."""
    import torch
    import expert_moe_fp32_amd as m
    logits = make_logits(2, 12, "f32", 3).cuda()
    ids = torch.tensor([[3, 12, -1, 11], [2, 2, 2, 0]], dtype=torch.int32,
                       device="cuda")
    d_w = torch.ones(2, 4, device="cuda")
    d = torch.empty(2, 12, device="cuda")
    r = m.make_router(2, 12, 4, score="sigmoid", renormalize=False)
    m.moe_route_scored_backward(r, logits, ids, d_w, d)
    s = ob.scores(to_f64(logits), "sigmoid")
    ref = np.zeros((2, 12))
    ref[0, [3, 11]] = (s * (1 - s))[0, [3, 11]]
    ref[1, 2], ref[1, 0] = 3 * (s * (1 - s))[1, 2], (s * (1 - s))[1, 0]
    assert np.allclose(to_f64(d), ref, rtol=1e-6, atol=0)


def test_offsets_past_32_bits():
    """T * E beyond 2^31: the last rows equal the same rows on their own."""
    import torch
    import expert_moe_fp32_amd as m
    E, k = 1024, 4
    T = 2 ** 31 // E + 1001
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    logits[-64:] = make_logits(64, E, "bf16", 6).cuda()
    kw = dict(score="sigmoid", groups=8, topk_groups=4, group_top=2,
              logits="bf16")
    r = m.make_router(T, E, k, **kw)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    m.moe_route_scored(r, logits, None, ids, w)
    d = torch.empty_like(logits)
    m.moe_route_scored_backward(r, logits, ids, w, d)
    tail = logits[-64:].contiguous()
    _, i2, w2, _ = route(tail, None, k, counts=False, **{
        n: v for n, v in kw.items() if n != "logits"})
    d2 = torch.empty_like(tail)
    m.moe_route_scored_backward(m.make_router(64, E, k, **kw), tail, i2, w2, d2)
    torch.cuda.synchronize()
    assert torch.equal(ids[-64:], i2) and torch.equal(w[-64:], w2)
    assert torch.equal(d[-64:], d2)
    assert (ids[:1000] == torch.arange(k, device="cuda")).all()


def vanishing_logits(E, chosen):
    """(logits, bias) of a softmax router whose bias lifts `chosen` experts
    far below the row's largest logit: by 500 (scores that 64 bits hold), 800
    and the type's lowest value (scores of 0), by an unchosen +inf, and with
    one chosen expert at the top."""
    import torch
    l = torch.randn(8, E, generator=torch.Generator().manual_seed(17))
    for row, drop in ((1, -500.0), (2, -800.0),
                      (3, torch.finfo(torch.float32).min), (4, 0.0)):
        l[row, chosen] += drop
    l[4, (chosen[0] + 1) % E] = float("inf")
    l[5, chosen] -= 900.0
    l[5, chosen[1]] = 4.0
    l[6] = torch.finfo(torch.float32).min      # equal shares
    l[7, chosen] = float("-inf")
    l[7, chosen[0]] = -2000.0
    bias = torch.zeros(E)
    bias[chosen] = 4.0
    return l, bias


@pytest.mark.parametrize("E,chosen", [(40, [39, 3, 17]), (12, [2, 3, 4]),
                                      (256, [7, 200, 64, 65]),
                                      (1000, [999, 0, 512])])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradient_of_vanishing_softmax_scores(E, chosen, dtype):
    """Renormalised weights are the softmax over the k chosen, w: their
    gradient is scale w_j (dw_j - sum_i dw_i w_i), and 0 in rows whose chosen
    scores are all 0 in the softmax over the row, where the weights are 0."""
    import torch
    import expert_moe_fp32_amd as m
    l, bias = vanishing_logits(E, chosen)
    logits = (l if dtype == "f32" else l.clamp(
        min=torch.finfo(torch.bfloat16).min).to(torch.bfloat16)).cuda()
    T, k = l.shape[0], len(chosen)
    r, ids, w, _ = route(logits, bias.cuda(), k, score="softmax", scale=2.5)
    d_w = torch.randn(T, k, device="cuda",
                      generator=torch.Generator("cuda").manual_seed(4))
    d = torch.full((T, E), 9.0, device="cuda", dtype=logits.dtype)
    m.moe_route_scored_backward(r, logits, ids, d_w, d)
    torch.cuda.synchronize()
    id64, dw = ids.cpu().numpy(), to_f64(d_w)
    lj = np.take_along_axis(to_f64(logits), id64.astype(np.int64), 1)
    rid, rw, _ = ob.route_scored(to_f64(logits), to_f64(bias), k,
                                 score="softmax")
    assert np.array_equal(id64, rid)
    dead = (rw == 0).all(1)
    assert dead[[2, 3]].all() and (to_f64(w)[dead] == 0).all()
    top = lj.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):          # inf - inf
        p = np.where(lj == top, 1.0, np.exp(lj - top))
    p[lj == -np.inf] = 0.0
    p[dead] = 0.0
    p /= np.where(dead, 1.0, p.sum(1))[:, None]
    part = 2.5 * p * (dw - (dw * p).sum(1, keepdims=True))
    ref = np.zeros((T, E))
    np.put_along_axis(ref, id64.astype(np.int64), part, 1)
    big = 2.5 * np.abs(dw).sum(1, keepdims=True)
    half = 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    tol = np.abs(ref) * half * (1 + 1e-6) + 32 * 2.0 ** -53 * big * (ref != 0) \
        + 2.0 ** -133
    err = np.abs(to_f64(d) - ref)
    assert (err <= tol).all(), np.argwhere(~(err <= tol))[:4].tolist()


@pytest.mark.parametrize("E", [16, 256])
@pytest.mark.parametrize("at,dw_scale", [(-715.0, 1.0), (-680.0, 1e20),
                                         (-300.0, 1e30)])
def test_gradient_of_tiny_sigmoid_scores(E, at, dw_scale):
    """Chosen scores near the end of 64 bits: 1 / S and dw / S pass its range,
    the gradient w_j (dw_j - sum_i dw_i w_i) (1 - s_j) does not."""
    import torch
    import expert_moe_fp32_amd as m
    k = 4
    l = torch.full((6, E), float("-inf"))
    g = torch.Generator().manual_seed(19)
    l[:, ::2] = at + torch.rand(6, E // 2, generator=g)
    logits = l.cuda()
    r, ids, w, _ = route(logits, None, k, score="sigmoid", scale=1.5)
    d_w = dw_scale * torch.randn(6, k, device="cuda", generator=torch.Generator(
        "cuda").manual_seed(5))
    d = torch.empty(6, E, device="cuda")
    m.moe_route_scored_backward(r, logits, ids, d_w, d)
    torch.cuda.synchronize()
    id64, dw = ids.cpu().numpy().astype(np.int64), to_f64(d_w)
    # sigmoid(l) = exp(l) and 1 - sigmoid(l) = 1 to 64 bits this far down
    p = np.exp(np.take_along_axis(l.double().numpy(), id64, 1) - at)
    p /= p.sum(1, keepdims=True)
    part = 1.5 * p * (dw - (dw * p).sum(1, keepdims=True))
    ref = np.zeros((6, E))
    np.put_along_axis(ref, id64, part, 1)
    # scores of exp(-715) are held in steps of 2^-1074: 2^-42 of them, which
    # the weights, their sum and the products count a few times
    big = 1.5 * np.abs(dw).sum(1, keepdims=True)
    tol = np.abs(ref) * 2.0 ** -24 * (1 + 1e-6) + big * 2.0 ** -38 * (ref != 0)
    assert (np.abs(to_f64(d) - ref) <= tol).all()


@pytest.mark.parametrize("shape", [  # T, E, k, groups, topk_groups, group_top
    (4100, 256, 8, 8, 4, 2), (8195, 256, 8, 8, 4, 2),
    (4500, 1000, 4, 8, 3, 2),      # groups of 125: eight wavefronts' scratch
    (4300, 100, 5, 4, 2, 2), (1500, 90, 6, 1, 1, 1),
    (16500, 60, 4, 5, 2, 2),       # four tokens a wavefront
], ids=str)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_more_tokens_than_wavefronts(shape, score):
    """Batches whose wavefronts walk on to a second token and whose counts
    are summed over the workgroups, of any number of experts."""
    import torch
    T, E, k, G, keep, top = shape
    print(shape, score, flush=True)
    logits = make_logits(T, E, "f32", 41, masked=0.02).cuda()
    bias = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(6))).cuda()
    check_route(logits, bias, k, score=score, groups=G, topk_groups=keep,
                group_top=top, scale=2.5)
