"""The layer for a few tokens on the GPU against the float64 oracle."""
import numpy as np
import pytest

from oracle import block as ob
from oracle import fp8 as ofp8
from oracle import moe as omoe
from oracle import train as ot
from synth import make_workload

from .helpers import (check_output, device_layer, out_to_f64,
                      phys_to_logical_from_map)

pytestmark = pytest.mark.gpu
BAR = 1e-2       # of the output's RMS beyond its rounding: the bf16 recipe's


def logical_weights(wl, d):
    """An expert's matrices as the numbers that the recipe's weights hold."""
    if wl.wdt == "fp8":
        return tuple(ofp8.dequantize_blocks_2d(*ofp8.quantize_blocks_2d(d[n]))
                     for n in ("wg", "wu", "wd"))
    return tuple(omoe.bf16_to_f64(d[n]) for n in ("wg", "wu", "wd"))


def oracle_out(wl, ids, w, here=None):
    experts = [logical_weights(wl, wl.expert(e)) for e in range(wl.num_local)]
    shared = logical_weights(wl, wl.shared_expert) if wl.shared else None
    return ot.few_layer(omoe.bf16_to_f64(wl.x), ids, w, wl.expert_begin,
                        experts, here, shared)


def new_out(wl, fmt="bf16"):
    import torch
    dt = torch.bfloat16 if fmt == "bf16" else torch.float32
    return torch.full((wl.T + 1, wl.H), 5.0, dtype=dt, device="cuda")


SHAPES = [
    ("prefill", dict(T=1, H=128, I=128, E=2, num_local=1, k=1)),
    ("prefill", dict(T=1, H=256, I=128, E=8, num_local=8, k=2)),
    ("decode", dict(T=16, H=512, I=256, E=64, num_local=8, k=8)),
    ("decode", dict(T=7, H=1152, I=384, E=256, num_local=32, k=8)),
    ("prefill", dict(T=13, H=640, I=128, E=300, num_local=40, k=5)),
    ("prefill", dict(T=16, H=256, I=256, E=16, num_local=16, k=16)),
    ("fp8", dict(T=1, H=256, I=128, E=8, num_local=8, k=2)),
    ("fp8", dict(T=16, H=512, I=384, E=64, num_local=16, k=6)),
    ("fp8", dict(T=5, H=1280, I=256, E=256, num_local=32, k=8)),
    ("prefill", dict(T=2, H=128, I=256, E=1024, num_local=1024, k=3)),
]


@pytest.mark.parametrize("name,kw", SHAPES, ids=str)
@pytest.mark.parametrize("shared", [False, True])
def test_against_the_oracle(name, kw, shared):
    import torch
    from expert_moe_fp32_amd.runner import to_dev
    print(name, kw, shared, flush=True)
    wl = make_workload(name, seed=101, shared=shared, **kw)
    dl = device_layer(wl)
    out = new_out(wl, wl.out)
    counts = torch.full((wl.E + 1,), 9, dtype=torch.int32, device="cuda")
    dl.forward_few(to_dev(wl.logits), None, to_dev(wl.x), out, counts)
    torch.cuda.synchronize()
    ids, w, c = omoe.route_topk(wl.logits, wl.k)
    assert np.array_equal(counts[:wl.E].cpu().numpy(), c) and counts[wl.E] == 9
    assert (out[wl.T] == 5.0).all()
    ref = oracle_out(wl, ids, w)
    got = out[:wl.T].double().cpu().numpy()
    if not ref.any():
        assert not got.any()
    else:
        check_output(got, ref, wl.out, BAR, f"{name} {kw}")


@pytest.mark.parametrize("name", ["prefill", "fp8"])
@pytest.mark.parametrize("T,H,I", [(16, 512, 640), (16, 1152, 1152),
                                   (3, 1280, 1152), (16, 128, 1664)])
@pytest.mark.parametrize("shared", [False, True])
def test_more_items_than_workgroups(name, T, H, I, shared):
    """The first kernel's 512 workgroups take two, three or four of the items
    (16 channels of an expert in use), not all of them equally many; H of 128
    and 512 leave some wavefronts without a share of the reduction."""
    import torch
    from expert_moe_fp32_amd.runner import to_dev
    wl = make_workload(name, seed=114, T=T, H=H, I=I, E=16, num_local=16,
                       k=16, shared=shared)
    items = (16 + shared) * I // 16          # every expert is in use
    print(name, T, H, I, shared, items, flush=True)
    assert items > (512 if I == 640 else 1024) and items % 512
    dl, out = device_layer(wl), new_out(wl, wl.out)
    counts = torch.full((17,), 9, dtype=torch.int32, device="cuda")
    dl.forward_few(to_dev(wl.logits), None, to_dev(wl.x), out, counts)
    torch.cuda.synchronize()
    ids, w, c = omoe.route_topk(wl.logits, wl.k)
    assert (c == T).all() and np.array_equal(counts[:16].cpu().numpy(), c)
    assert counts[16] == 9 and (out[T] == 5.0).all()
    check_output(out[:T].double().cpu().numpy(), oracle_out(wl, ids, w),
                 wl.out, BAR, f"{name} {T} {H} {I}")


@pytest.mark.parametrize("T", list(range(1, 17)))
def test_every_count_of_tokens(T):
    """Against the general layer on the same weights (bf16 recipe: both round
    h, so they differ by the order of float32 sums and h values that these
    carry over a rounding border)."""
    import torch
    from expert_moe_fp32_amd.runner import to_dev
    wl = make_workload("prefill", seed=102 + T, T=T, H=512, I=256, E=16,
                       num_local=8, k=4)
    dl = device_layer(wl)
    b, out = dl.buffers(), new_out(wl)
    logits, x = to_dev(wl.logits), to_dev(wl.x)
    dl.forward(b, logits, None, x)
    dl.forward_few(logits, None, x, out)
    torch.cuda.synchronize()
    check_output(out[:T].double().cpu().numpy(), out_to_f64(b, wl), "bf16",
                 BAR, str(T))


def test_float32_output_and_bias():
    import torch
    from expert_moe_fp32_amd.runner import to_dev
    wl = make_workload("decode", seed=103, T=9, H=384, I=256, E=32,
                       num_local=8, k=4, out="f32")
    rng = np.random.default_rng(4)
    bias = rng.normal(size=wl.E).astype(np.float32)
    dl = device_layer(wl)
    out = new_out(wl, "f32")
    dl.forward_few(to_dev(wl.logits), to_dev(bias), to_dev(wl.x), out)
    torch.cuda.synchronize()
    ids, w, _ = omoe.route_topk(wl.logits, wl.k, bias)
    check_output(out[:wl.T].double().cpu().numpy(), oracle_out(wl, ids, w),
                 "f32", BAR, literal=True)


@pytest.mark.parametrize("score,dtype", [("sigmoid", "f32"),
                                         ("softmax", "bf16")])
def test_scored_routing(score, dtype):
    import torch
    import expert_moe_fp32_amd as m
    from expert_moe_fp32_amd.runner import to_dev
    wl = make_workload("decode", seed=104, T=11, H=256, I=128, E=64,
                       num_local=32, k=6)
    rng = np.random.default_rng(5)
    bias = (0.2 * rng.normal(size=wl.E)).astype(np.float32)
    logits = to_dev(wl.logits)
    if dtype == "bf16":
        logits = logits.bfloat16()
    wide = torch.zeros(wl.T, wl.E + 3, dtype=logits.dtype, device="cuda")
    wide[:, :wl.E] = logits
    r = m.make_router(wl.T, wl.E, wl.k, score, 8, 4, 2, scale=2.5,
                      logits=dtype, logits_stride=wl.E + 3)
    dl, out = device_layer(wl), new_out(wl)
    counts = torch.empty(wl.E, dtype=torch.int32, device="cuda")
    dl.forward_few(wide, to_dev(bias), to_dev(wl.x), out, counts, r)
    torch.cuda.synchronize()
    ids, w, c = ob.route_scored(logits.double().cpu().numpy(), bias, wl.k,
                                score, 8, 4, 2, scale=2.5)
    assert np.array_equal(counts.cpu().numpy(), c)
    check_output(out[:wl.T].double().cpu().numpy(), oracle_out(wl, ids, w),
                 "bf16", BAR)


def test_a_share_in_the_middle_and_replicas():
    """Experts [4, 12) of 16, the hottest held twice, one replica of another
    expert on another rank."""
    import torch
    from expert_moe_fp32_amd.runner import to_dev
    wl = make_workload("prefill", seed=105, T=16, H=256, I=128, E=16,
                       num_local=8, k=4)
    wl.expert_begin = 4
    l2p = np.array([[0, 8], [1, -1], [2, -1], [3, -1], [4, 9], [5, -1],
                    [-1, 6], [7, -1]], dtype=np.int32)
    rep = np.array([2, 1, 1, 1, 2, 1, 2, 1], dtype=np.int32)
    dl = device_layer(wl, l2p=l2p, rep=rep, P=10, phys_to_logical=[
        e if e >= 0 else 0 for e in phys_to_logical_from_map(l2p, rep, 10)])
    out = new_out(wl)
    dl.forward_few(to_dev(wl.logits), None, to_dev(wl.x), out)
    torch.cuda.synchronize()
    ids, w, _ = omoe.route_topk(wl.logits, wl.k)
    d = omoe.dispatch(ids, 4, 8, l2p, rep, 10)
    check_output(out[:wl.T].double().cpu().numpy(),
                 oracle_out(wl, ids, w, d.pair_row >= 0), "bf16", BAR)


def test_counts_of_replicas_out_of_range():
    """Taken as the nearest count that the map has room for, as dispatch
    takes them."""
    import torch
    from expert_moe_fp32_amd.runner import to_dev
    wl = make_workload("prefill", seed=113, T=16, H=256, I=128, E=8,
                       num_local=8, k=4)
    l2p = np.array([[0, 8]] + [[i, -1] for i in range(1, 7)] + [[7, 9]],
                   dtype=np.int32)
    rep = np.array([7, 0, 1, -3, 1, 1, 1, 2 ** 30], dtype=np.int32)
    real = np.array([2, 1, 1, 1, 1, 1, 1, 2], dtype=np.int32)
    dl = device_layer(wl, l2p=l2p, rep=rep, P=10,
                      phys_to_logical=phys_to_logical_from_map(l2p, real, 10))
    out = new_out(wl)
    dl.forward_few(to_dev(wl.logits), None, to_dev(wl.x), out)
    torch.cuda.synchronize()
    ids, w, _ = omoe.route_topk(wl.logits, wl.k)
    check_output(out[:wl.T].double().cpu().numpy(), oracle_out(wl, ids, w),
                 "bf16", BAR)


def test_tokens_without_a_local_expert_get_zeros():
    import torch
    from expert_moe_fp32_amd.runner import to_dev
    wl = make_workload("decode", seed=106, T=6, H=256, I=128, E=32,
                       num_local=4, k=2)
    wl.logits[:4, :4] = -50.0
    dl, out = device_layer(wl), new_out(wl)
    dl.forward_few(to_dev(wl.logits), None, to_dev(wl.x), out)
    torch.cuda.synchronize()
    assert not out[:4].any() and (out[6] == 5.0).all()
    wl.logits[:, :4] = -50.0                       # nobody has one
    dl.forward_few(to_dev(wl.logits), None, to_dev(wl.x), out)
    torch.cuda.synchronize()
    assert not out[:6].any()


def test_one_tokens_nan_stays_its_own():
    """Other tokens do not see a row of NaN, nor what the workspace held."""
    import torch
    from expert_moe_fp32_amd.runner import to_dev
    wl = make_workload("prefill", seed=107, T=8, H=256, I=128, E=8,
                       num_local=8, k=2)
    dl = device_layer(wl)
    import expert_moe_fp32_amd as m
    ws = torch.full((m.moe_layer_few_workspace_size(dl.p),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    out, ref = new_out(wl), new_out(wl)
    logits, x = to_dev(wl.logits), to_dev(wl.x)
    dl.forward_few(logits, None, x, ref, ws=ws)
    x.view(torch.bfloat16)[3] = float("nan")
    dl.forward_few(logits, None, x, out, ws=ws)
    torch.cuda.synchronize()
    assert out[3].isnan().all()
    keep = [t for t in range(8) if t != 3]
    assert torch.equal(out[keep], ref[keep]) and not ref.isnan().any()


def test_no_tokens():
    import torch
    import expert_moe_fp32_amd as m
    wl = make_workload("decode", seed=108, T=4, H=256, I=128, E=8,
                       num_local=8, k=2)
    dl = device_layer(wl)
    dl.p = m.make_problem(0, 256, 128, 8, 2)
    counts = torch.full((8,), 3, dtype=torch.int32, device="cuda")
    dl.forward_few(None, None, None, None, counts)
    torch.cuda.synchronize()
    assert not counts.any()


@pytest.mark.parametrize("name,scored", [("prefill", False), ("fp8", True)])
def test_replays_from_a_graph(name, scored):
    import torch
    import expert_moe_fp32_amd as m
    from expert_moe_fp32_amd.runner import to_dev
    wl = make_workload(name, seed=109, T=9, H=384, I=256, E=32, num_local=16,
                       k=4)
    dl = device_layer(wl)
    logits, x = to_dev(wl.logits), to_dev(wl.x)
    r = m.make_router(wl.T, wl.E, wl.k, "sigmoid") if scored else None
    n = m.moe_layer_few_workspace_size(dl.p)
    ws, ws2 = (torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    out, aside = new_out(wl, wl.out), new_out(wl, wl.out)
    counts = torch.empty(wl.E, dtype=torch.int32, device="cuda")
    flipped = logits.flip(0).contiguous()
    call = lambda: dl.forward_few(logits, None, x, out, counts, r, ws)
    call()
    torch.cuda.synchronize()
    eager, c = out.clone(), counts.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(4):
        out.zero_()
        counts.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[:wl.T], eager[:wl.T]) and torch.equal(counts, c)
        dl.forward_few(flipped, None, x, aside, None, r, ws2)
        torch.cuda.synchronize()
    logits.copy_(flipped)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[:wl.T], aside[:wl.T])


def test_two_streams_at_once():
    import torch
    from expert_moe_fp32_amd.runner import to_dev
    runs = []
    for seed, T in ((110, 16), (111, 3)):
        wl = make_workload("prefill", seed=seed, T=T, H=512, I=512, E=16,
                           num_local=16, k=4)
        dl = device_layer(wl)
        args = (to_dev(wl.logits), None, to_dev(wl.x))
        ref, out = new_out(wl), new_out(wl)
        dl.forward_few(*args, ref)
        import expert_moe_fp32_amd as m
        ws = torch.empty(m.moe_layer_few_workspace_size(dl.p),
                         dtype=torch.uint8, device="cuda")
        runs.append((dl, args, ref, out, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for dl, args, ref, out, ws, s in runs:
            with torch.cuda.stream(s):
                dl.forward_few(*args, out, ws=ws)
    torch.cuda.synchronize()
    for _, _, ref, out, _, _ in runs:
        assert torch.equal(out, ref)
