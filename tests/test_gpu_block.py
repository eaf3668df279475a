"""The combine's end and gradients, the scored layer, and a whole block's run
forward and backward, on the GPU."""
import numpy as np
import pytest

from oracle import block as ob
from synth import make_workload

from .helpers import device_layer
from .norm_cases import U, NormCase, check_forward

pytestmark = pytest.mark.gpu


def make_pairs(T, k, local, seed, empty=()):
    """(pair_row [T][k] int32, rows): a random share of local pairs, rows in a
    random order; tokens in `empty` have none."""
    rng = np.random.default_rng(seed)
    here = rng.random((T, k)) < local
    here[list(empty)] = False
    rows = np.full((T, k), -1, dtype=np.int32)
    rows[here] = rng.permutation(int(here.sum()))
    return rows, int(here.sum())


def problem(T, H, k, shared, out="bf16"):
    import expert_moe_fp32_amd as m
    act = "f32" if H % 128 else "bf16"
    return m.make_problem(T, H, 128, max(k, 8), k, has_shared=shared, act=act,
                          wdt=act, out=out)


def combine_inputs(T, H, k, shared, seed, local=0.4):
    import torch
    g = torch.Generator().manual_seed(seed)
    pair_row, N = make_pairs(T, k, local, seed, empty=[0] if T > 1 else [])
    y = torch.randn(N + 2, H, generator=g)
    y[N:] = float("nan")                  # rows of no pair are never read
    w = torch.rand(T, k, generator=g)
    sh = torch.randn(T, H, generator=g) if shared else None
    dev = lambda t: None if t is None else t.cuda()
    return dev(torch.from_numpy(pair_row)), dev(y), dev(w), dev(sh), N


@pytest.mark.parametrize("kw", [
    dict(T=1, H=7168, k=8, shared=True),
    dict(T=40, H=6144, k=8, shared=False),
    dict(T=130, H=256, k=2, shared=True, block="f32", gate="token", post=False),
    dict(T=21, H=1004, k=16, shared=False, gate="channel", pads=(4, 0, 8, 12)),
    dict(T=21, H=36, k=4, shared=True, block="f32", resid="f32", out="f32"),
    dict(T=11, H=16384, k=3, shared=True, resid="f32", gain="bf16", offset=1.0),
    dict(T=33, H=640, k=5, shared=False, pre=False, gate="full", rscale=0.5),
    dict(T=33, H=640, k=5, shared=True, pads=(1, 3, 5, 7)),
    dict(T=530, H=8192, k=8, shared=False, resid="f32"),
    dict(T=20, H=4, k=2, shared=True, block="f32"),
], ids=str)
def test_combine_norm(kw):
    import torch
    import expert_moe_fp32_amd as m
    kw = dict(kw)
    k, shared = kw.pop("k"), kw.pop("shared")
    print(kw, k, shared, flush=True)
    c = NormCase(**kw, seed=11)
    rows, y, w, sh, N = combine_inputs(c.T, c.H, k, shared, 12)
    p = problem(c.T, c.H, k, shared)
    block = c.rows(c.types["block"], c.pads[0])
    before = c.edges(block, c.resid_out, c.x)
    m.moe_combine_norm(p, c.n, y, rows, w, sh, c.resid, c.post, c.gate, c.pre,
                       block, c.resid_out, c.x)
    torch.cuda.synchronize()
    for (a, b), (d, e) in zip(before, c.edges(block, c.resid_out, c.x)):
        assert torch.equal(a, d) and torch.equal(b, e)
    f = lambda t: None if t is None else t.double().cpu().numpy()
    comb = ob.combine_rows(f(y), f(rows).astype(int), f(w), f(sh))
    mag = ob.combine_rows(np.abs(f(y)), f(rows).astype(int), f(w),
                          None if sh is None else np.abs(f(sh)))
    # one product and at most k + 1 additions a column: (k + 2) u of the
    # magnitudes, within the 60 u that the check counts on each
    check_forward(c, c.f64(c.resid_out), c.f64(c.x), comb, mag)
    half = {"f32": U, "bf16": 2.0 ** -8}[c.types["block"]]
    assert (np.abs(c.f64(block) - comb) <= half * np.abs(comb) +
            (k + 2) * U * mag).all()
    # without the combined rows the outputs are the same
    r, x = c.resid_out.clone(), None if c.x is None else c.x.clone()
    c.resid_out.fill_(3.0)
    m.moe_combine_norm(p, c.n, y, rows, w, sh, c.resid, c.post, c.gate, c.pre,
                       None, c.resid_out, c.x)
    torch.cuda.synchronize()
    assert torch.equal(c.resid_out[:c.T, :c.H], r[:c.T, :c.H])
    if x is not None:
        assert torch.equal(c.x, x)


@pytest.mark.parametrize("T,H,k,shared,out", [
    (1, 7168, 8, True, "bf16"), (50, 256, 2, False, "f32"),
    (133, 1024, 16, True, "f32"), (20, 36, 3, True, "bf16"),
    (9, 4, 2, False, "f32"), (7, 20480, 4, True, "bf16"),
    (300, 6144, 8, False, "bf16"), (1500, 7168, 2, True, "bf16"),
    (3, 8196, 5, True, "f32"),
])
def test_combine_backward(T, H, k, shared, out):
    import torch
    import expert_moe_fp32_amd as m
    rows, y, w, sh, N = combine_inputs(T, H, k, shared, 21)
    p = problem(T, H, k, shared, out)
    g = torch.Generator().manual_seed(22)
    d = torch.randn(T, H, generator=g).to(
        torch.bfloat16 if out == "bf16" else torch.float32).cuda()
    d_y = torch.full_like(y, 5.0)
    d_w = torch.full((T + 1, k), 5.0, device="cuda")
    d_s = None if sh is None else torch.full((T + 1, H), 5.0, device="cuda")
    m.moe_combine_backward(p, d, y, rows, w, d_y, d_w, d_s)
    torch.cuda.synchronize()
    f = lambda t: t.double().cpu().numpy()
    r = f(rows).astype(int)
    ry, rw = ob.combine_backward(f(d), f(y), r, f(w))
    assert (d_y[N:] == 5.0).all() and (d_w[T] == 5.0).all()
    assert (np.abs(f(d_y)[:N] - ry[:N]) <= U * np.abs(ry[:N])).all()
    # chains of at most 64 float32 additions over a row
    _, mag = ob.combine_backward(np.abs(f(d)), np.abs(f(y)), r, f(w))
    assert (np.abs(f(d_w)[:T] - rw) <= 64 * U * mag).all()
    assert (f(d_w)[:T][r < 0] == 0).all()
    if d_s is not None:
        assert torch.equal(d_s[:T], d.float()) and (d_s[T] == 5.0).all()
    # each output alone
    one, zero = torch.full_like(y, 5.0), torch.full((T, k), 5.0, device="cuda")
    m.moe_combine_backward(p, d, None, rows, w, one, None, None)
    m.moe_combine_backward(p, d, y, rows, w, None, zero, None)
    torch.cuda.synchronize()
    assert torch.equal(one, d_y) and torch.equal(zero, d_w[:T])


def test_rows_past_the_capacity_are_dropped():
    import torch
    import expert_moe_fp32_amd as m
    p = m.make_problem(2, 128, 128, 8, 2, num_local=1)      # capacity 2 rows
    rows = torch.tensor([[0, 2], [2 ** 30, 1]], dtype=torch.int32).cuda()
    y = torch.ones(2, 128).cuda()
    w = torch.full((2, 2), 0.5).cuda()
    d = torch.ones(2, 128, dtype=torch.bfloat16).cuda()
    d_y, d_w = torch.zeros(2, 128).cuda(), torch.ones(2, 2).cuda()
    m.moe_combine_backward(p, d, y, rows, w, d_y, d_w, None)
    n = m.make_norm(2, 128, resid="f32")
    ro = torch.empty(2, 128).cuda()
    m.moe_combine_norm(p, n, y, rows, w, None, torch.zeros(2, 128).cuda(),
                       None, None, None, None, ro, None)
    torch.cuda.synchronize()
    assert d_w.tolist() == [[128.0, 0.0], [0.0, 128.0]]
    assert (d_y == 0.5).all() and (ro == 0.5).all()


# -------------------------------------------------------- the scored layer
LAYERS = [
    ("decode", dict(T=50, H=384, I=256, E=32, num_local=8, k=4), False),
    ("prefill", dict(T=300, H=256, I=256, E=16, num_local=8, k=4), True),
    ("lowlat", dict(H=512, I=256, E=64, num_local=8, T=40), False),
    ("tiny", dict(), False),
]


def scored_setup(name, kw, seed=31):
    import torch
    import expert_moe_fp32_amd as m
    from expert_moe_fp32_amd.runner import to_dev
    wl = make_workload(name, seed=seed, **kw)
    dl = device_layer(wl)
    router = m.make_router(wl.T, wl.E, wl.k, "sigmoid", 4, 2, 2, scale=2.5)
    bias = (0.1 * torch.randn(wl.E, generator=torch.Generator()
                              .manual_seed(1))).cuda()
    act = "f32" if wl.act == "f32" else "bf16"
    c = NormCase(wl.T, wl.H, block=wl.out, resid=act, out=act, seed=32)
    c.x, c.resid_out = c.x[:wl.T], c.resid_out[:wl.T]
    return wl, dl, router, bias, c, to_dev(wl.logits), to_dev(wl.x)


@pytest.mark.parametrize("name,kw,shared", LAYERS)
def test_scored_layer_equals_its_steps(name, kw, shared):
    """The layer against the single calls (each checked against the oracle),
    bit for bit, with and without the norm."""
    import torch
    wl, dl, router, bias, c, logits, x = scored_setup(name, kw)
    assert wl.shared == shared
    b = dl.buffers()
    dl.forward_scored(b, router, logits, bias, x, c.n, c.resid, c.post, None,
                      c.pre, c.resid_out, c.x)
    torch.cuda.synchronize()
    s = dl.buffers()
    dl.route_scored(s, router, logits, bias)
    dl.dispatch(s, x)
    dl.ffn(s, x_shared=x if shared else None)
    ro, xo = torch.empty_like(c.resid_out), torch.empty_like(c.x)
    dl.combine_norm(s, c.n, c.resid, c.post, None, c.pre, ro, xo)
    torch.cuda.synchronize()
    assert torch.equal(s.counts, b.counts)
    assert torch.equal(ro, c.resid_out) and torch.equal(xo, c.x)
    assert torch.equal(s.out, b.out)
    dl.combine(s)                                  # the layer without a norm
    dl.forward_scored(b, router, logits, bias, x)
    torch.cuda.synchronize()
    assert torch.equal(s.out, b.out)


def test_scored_layer_with_softmax_equals_the_plain_layer():
    """A softmax router without groups, bias or scale chooses and weighs as
    moe_route_topk does (its weights to float32 rounding): ids and counts are
    equal and the outputs agree to the bf16 output's rounding."""
    import torch
    import expert_moe_fp32_amd as m
    wl, dl, _, _, _, logits, x = scored_setup(*LAYERS[1][:2])
    a, b = dl.buffers(), dl.buffers()
    dl.forward(a, logits, None, x)
    dl.forward_scored(b, m.make_router(wl.T, wl.E, wl.k), logits, None, x)
    torch.cuda.synchronize()
    assert torch.equal(a.counts, b.counts)
    fa, fb = (t.out.view(torch.bfloat16).double() for t in (a, b))
    assert ((fa - fb).abs() <= 2.0 ** -7 * fa.abs() + 1e-5).all()


def test_zero_token_layer():
    import torch
    import expert_moe_fp32_amd as m
    wl, dl, _, _, _, _, _ = scored_setup(*LAYERS[0][:2])
    dl.p.T = 0
    b = dl.buffers()
    b.counts.fill_(4)
    dl.forward_scored(b, m.make_router(0, wl.E, wl.k), None, None, None)
    torch.cuda.synchronize()
    assert (b.counts == 0).all()


# --------------------------------------------- a block forward and backward
class Block:
    """Every new operator in the order of a training step: route, (dispatch
    and experts stand as fixed rows,) combine with the norms, and back to the
    logits."""

    def __init__(self, T=24, H=256, E=32, k=4, seed=41, score="sigmoid"):
        import torch
        import expert_moe_fp32_amd as m
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).cuda()
        self.T, self.H, self.E, self.k = T, H, E, k
        self.router = m.make_router(T, E, k, score, 4, 2, 2, scale=1.5)
        self.p = m.make_problem(T, H, 128, E, k, has_shared=True, act="bf16",
                                wdt="bf16", out="f32")
        self.n = m.make_norm(T, H, "f32", "f32", "f32", gate_shape=(1, H),
                             residual_scale=0.5)
        self.logits, self.bias = r(T, E), 0.1 * r(E)
        self.y_perm, self.shared = r(T * k, H), r(T, H)
        self.resid, self.d_x, self.d_ro = r(T, H), r(T, H), r(T, H)
        self.post, self.pre, self.gate = r(H), r(H), r(1, H)
        self.rows = torch.arange(T * k, dtype=torch.int32).view(T, k).cuda()
        e = lambda *s: torch.empty(*s, device="cuda")
        self.ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
        self.counts = torch.empty(E, dtype=torch.int32, device="cuda")
        self.w, self.d_w = e(T, k), e(T, k)
        self.block, self.ro, self.x = e(T, H), e(T, H), e(T, H)
        self.d_block, self.d_resid = e(T, H), e(T, H)
        self.d_post, self.d_pre, self.d_gate = e(H), e(H), e(1, H)
        self.d_y_perm, self.d_shared = e(T * k, H), e(T, H)
        self.d_logits = e(T, E)
        self.ws = torch.empty(m.moe_residual_norm_workspace_size(self.n),
                              dtype=torch.uint8, device="cuda")

    def step(self):
        import expert_moe_fp32_amd as m
        m.moe_route_scored(self.router, self.logits, self.bias, self.ids,
                           self.w, self.counts)
        m.moe_combine_norm(self.p, self.n, self.y_perm, self.rows, self.w,
                           self.shared, self.resid, self.post, self.gate,
                           self.pre, self.block, self.ro, self.x)
        m.moe_residual_norm_backward(
            self.n, self.block, self.ro, self.post, self.gate, self.pre,
            self.d_x, self.d_ro, self.d_block, self.d_resid, self.d_post,
            self.d_gate, self.d_pre, self.ws, self.ws.numel())
        m.moe_combine_backward(self.p, self.d_block, self.y_perm, self.rows,
                               self.w, self.d_y_perm, self.d_w, self.d_shared)
        m.moe_route_scored_backward(self.router, self.logits, self.ids,
                                    self.d_w, self.d_logits)

    OUT = ("ids", "w", "counts", "block", "ro", "x", "d_block", "d_resid",
           "d_post", "d_pre", "d_gate", "d_y_perm", "d_w", "d_shared",
           "d_logits")

    def outputs(self):
        return {n: getattr(self, n).clone() for n in self.OUT}


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_block_gradients(score):
    """Every gradient of the run against automatic differentiation of the
    whole formula in float64, with the choice held."""
    import torch
    b = Block(score=score)
    b.step()
    torch.cuda.synchronize()
    d = {n: getattr(b, n).double().cpu().requires_grad_() for n in (
        "logits", "y_perm", "shared", "resid", "post", "pre", "gate")}
    ids = b.ids.long().cpu()
    s = d["logits"].sigmoid() if score == "sigmoid" else d["logits"].softmax(-1)
    w = s.gather(1, ids)
    w = 1.5 * w / w.sum(-1, keepdim=True)
    y = (d["y_perm"].view(b.T, b.k, b.H) * w[..., None]).sum(1) + d["shared"]
    unit = lambda z: z / (z.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    ro = d["resid"] + 0.5 * d["gate"] * (unit(y) * d["post"])
    x = unit(ro) * d["pre"]
    ((x * b.d_x.double().cpu()).sum() + (ro * b.d_ro.double().cpu()).sum()).backward()
    for name, got in (("logits", b.d_logits), ("y_perm", b.d_y_perm),
                      ("shared", b.d_shared), ("resid", b.d_resid),
                      ("post", b.d_post), ("pre", b.d_pre),
                      ("gate", b.d_gate)):
        ref = d[name].grad.numpy()
        err = np.abs(got.double().cpu().numpy() - ref)
        # some hundred float32 roundings along the chain of five calls, on
        # terms up to some tens of the result's RMS: 4096 u of the RMS
        assert err.max() <= 4096 * U * np.sqrt(np.mean(ref ** 2)), name


def test_block_replays_from_a_graph():
    """The run captured; replays with eager work and synchronisation between
    them equal the eager run bit for bit, also after the inputs change."""
    import torch
    b, other = Block(seed=51), Block(T=70, seed=52)
    b.step()
    torch.cuda.synchronize()
    eager = b.outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    logits = b.logits.clone()
    for r in range(4):
        for n in Block.OUT:
            getattr(b, n).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, v in b.outputs().items():
            assert torch.equal(v, eager[n]), (r, n)
        other.step()
        torch.cuda.synchronize()
    b.logits.copy_(logits.flip(0))
    b.step()
    torch.cuda.synchronize()
    eager = b.outputs()
    graph.replay()
    torch.cuda.synchronize()
    for n, v in b.outputs().items():
        assert torch.equal(v, eager[n]), n


def test_two_streams_at_once():
    """Two runs on two streams, each with its own buffers and workspace."""
    import torch
    pairs = [(Block(seed=61), torch.cuda.Stream()),
             (Block(T=90, seed=62), torch.cuda.Stream())]
    ref = []
    for b, _ in pairs:
        b.step()
        torch.cuda.synchronize()
        ref.append(b.outputs())
        for n in Block.OUT:
            getattr(b, n).zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for b, s in pairs:
            with torch.cuda.stream(s):
                b.step()
    torch.cuda.synchronize()
    for (b, _), r in zip(pairs, ref):
        for n, v in b.outputs().items():
            assert torch.equal(v, r[n]), n


def layer_arrays(wl, gate, seed=71):
    """(router, bias, logits, x, norm case, its outputs) of a scored layer
    that ends in a norm with a gate."""
    import torch
    import expert_moe_fp32_amd as m
    from expert_moe_fp32_amd.runner import to_dev
    router = m.make_router(wl.T, wl.E, wl.k, "sigmoid", 4, 2, 2, scale=2.5)
    bias = (0.1 * torch.randn(wl.E, generator=torch.Generator()
                              .manual_seed(seed))).cuda()
    c = NormCase(wl.T, wl.H, block=wl.out, gate=gate, rscale=0.5, seed=seed)
    outs = [torch.full((wl.T, wl.H), 3.0, dtype=torch.bfloat16, device="cuda")
            for _ in range(2)]
    return router, bias, to_dev(wl.logits), to_dev(wl.x), c, outs


@pytest.mark.parametrize("gate", ["token", "channel"])
def test_scored_layer_with_replicas_and_a_gate(gate):
    """As test_scored_layer_equals_its_steps, some experts held twice."""
    import torch
    from oracle import eplb
    from .helpers import phys_to_logical_from_map
    wl = make_workload("prefill", seed=33, T=200, H=256, I=256, E=16,
                       num_local=8, k=4)
    l2p, rep, P = eplb.hottest_replica_map(np.arange(8) ** 2, 3)
    dl = device_layer(wl, l2p=l2p, rep=rep, P=P,
                      phys_to_logical=phys_to_logical_from_map(l2p, rep, P))
    router, bias, logits, x, c, (ro, xo) = layer_arrays(wl, gate)
    b, s = dl.buffers(), dl.buffers()
    dl.forward_scored(b, router, logits, bias, x, c.n, c.resid, c.post, c.gate,
                      c.pre, ro, xo)
    dl.route_scored(s, router, logits, bias)
    dl.dispatch(s, x)
    dl.ffn(s, x_shared=x if wl.shared else None)
    ro2, xo2 = torch.empty_like(ro), torch.empty_like(xo)
    dl.combine_norm(s, c.n, c.resid, c.post, c.gate, c.pre, ro2, xo2)
    torch.cuda.synchronize()
    assert torch.equal(s.counts, b.counts) and torch.equal(s.out, b.out)
    assert torch.equal(ro, ro2) and torch.equal(xo, xo2)


@pytest.mark.parametrize("name,kw,shared", LAYERS[:3])
def test_scored_layer_replays_from_a_graph(name, kw, shared):
    """The layer captured; replays with eager work between them equal the
    eager call bit for bit, also after its inputs change."""
    import torch
    wl = make_workload(name, seed=34, **kw)
    dl = device_layer(wl)
    router, bias, logits, x, c, (ro, xo) = layer_arrays(wl, "token")
    b, other = dl.buffers(), dl.buffers()

    def call(buffers=b, l=logits, out=(ro, xo)):
        dl.forward_scored(buffers, router, l, bias, x, c.n, c.resid, c.post,
                          c.gate, c.pre, *out)

    def outputs():
        torch.cuda.synchronize()
        return [t.clone() for t in (ro, xo, b.out, b.counts)]

    call()
    eager = outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    flipped = logits.flip(0).contiguous()
    aside = [torch.empty_like(ro), torch.empty_like(xo)]
    for r in range(4):
        for t in (ro, xo, b.out, b.counts):
            t.zero_()
        graph.replay()
        for i, (got, ref) in enumerate(zip(outputs(), eager)):
            assert torch.equal(got, ref), (r, i)
        call(other, flipped, aside)
        torch.cuda.synchronize()
    logits.copy_(flipped)
    call()
    eager = outputs()
    graph.replay()
    assert all(torch.equal(g, e) for g, e in zip(outputs(), eager))
