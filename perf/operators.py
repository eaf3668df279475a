"""Timing cases of the router, residual-norm and combine operators.

Six operators, each in its plain form (elementary torch operations) and as a
user of the library calls it:

  route             scored routing: sigmoid or softmax scores, balance bias,
                    expert groups, top-k, weights, expert counts
  route_backward    its gradient, d_logits from d_topk_w
  norm              post-norm of a block's output, gate, residual add and the
                    next block's pre-norm, in one pass
  norm_backward     its gradients
  combine_norm      the weighted combine of the expert rows, then `norm`
  combine_backward  the combine's gradients

``own`` selects the library's kernels; without it nothing but torch is used.
"""
import numpy as np
import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
DT = {"f32": F32, "bf16": BF16}
BYTES = {"f32": 4, "bf16": 2}
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _route(op, T, E, k, score, groups=1, keep=1, top=1, renorm=True,
           scale=1.0, bias=True, logits="f32", pad=0, masked=0.0):
    return dict(op=op, T=T, E=E, k=k, score=score, groups=groups, keep=keep,
                top=top, renorm=renorm, scale=scale, bias=bias, logits=logits,
                pad=pad, masked=masked)


def _norm(op, T, H, block="bf16", resid="bf16", out="bf16", gain="f32",
          post=True, gate="none", offset=0.0, rscale=1.0, pad=0):
    return dict(op=op, T=T, H=H, block=block, resid=resid, out=out, gain=gain,
                post=post, gate=gate, offset=offset, rscale=rscale, pad=pad)


def _combine(op, T, H, E, L, k, shared, block="bf16", resid="bf16",
             out="bf16", gain="f32", post=False, gate="none", offset=0.0,
             rscale=1.0):
    return dict(op=op, T=T, H=H, E=E, L=L, k=k, shared=shared, block=block,
                resid=resid, out=out, gain=gain, post=post, gate=gate,
                offset=offset, rscale=rscale, pad=0)


def listed():
    cases = {
        # one decoded token of a 256-expert model with 4 of 8 groups kept
        "route token": _route("route", 1, 256, 8, "sigmoid", 8, 4, 2,
                              scale=2.5),
        # a prefill chunk of the same router
        "route prefill": _route("route", 8192, 256, 8, "sigmoid", 8, 4, 2,
                                scale=2.5),
        # a training micro-batch of that router
        "route_backward train": _route("route_backward", 8192, 256, 8,
                                       "sigmoid", 8, 4, 2, scale=2.5),
        # a ragged batch of a softmax router with plain softmax weights, its
        # bf16 logits a slice of a wider projection, some experts disabled
        "route_backward ragged": _route("route_backward", 1021, 160, 6,
                                        "softmax", renorm=False, scale=16.0,
                                        logits="bf16", pad=3, masked=0.02),
        # one decoded token, norms on both sides of the block
        "norm token": _norm("norm", 1, 7168),
        # a prefill chunk, norms on both sides
        "norm prefill": _norm("norm", 8192, 7168),
        # a training micro-batch with a learned scale per channel
        "norm_backward train": _norm("norm_backward", 4096, 7168,
                                     gate="channel"),
        # an odd hidden size and batch, float32 stream, gate per token
        "norm_backward odd": _norm("norm_backward", 1021, 2501, "f32", "f32",
                                   "f32", gate="token", offset=1.0, pad=2),
        # a low-latency decode batch: 32 of 256 experts here, shared expert
        "combine_norm decode": _combine("combine_norm", 128, 7168, 256, 32, 8,
                                        True),
        # a prefill chunk of the same layer
        "combine_norm prefill": _combine("combine_norm", 8192, 7168, 256, 32,
                                         8, True),
        # a small layer with every expert here
        "combine_backward small": _combine("combine_backward", 128, 256, 8, 8,
                                           2, False, block="f32"),
        # a training micro-batch: 32 of 256 experts here, shared expert
        "combine_backward train": _combine("combine_backward", 4096, 7168,
                                           256, 32, 8, True),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "route_backward", "norm", "norm_backward",
                     "combine_norm", "combine_backward"])
    T = _log_int(rng, 1, 8192)
    if op.startswith("route"):
        groups = rng.choice([1, 1, 4, 8])
        per = _log_int(rng, 2 if groups > 1 else 8, 512 // groups)
        E = groups * per
        keep = rng.randint(1, groups)
        score = rng.choice(["sigmoid", "softmax"])
        return _route(op, T, E, rng.randint(1, min(16, keep * per)), score,
                      groups, keep, rng.choice([1, 2]),
                      renorm=rng.random() < 0.7,
                      scale=rng.choice([1.0, 2.5]),
                      bias=rng.random() < 0.7,
                      logits=rng.choice(["f32", "bf16"]),
                      pad=rng.choice([0, 0, 1, 8]),
                      masked=rng.choice([0.0, 0.0, 0.05]))
    types = dict(block=rng.choice(["bf16", "f32"]),
                 resid=rng.choice(["bf16", "f32"]),
                 out=rng.choice(["bf16", "f32"]),
                 gain=rng.choice(["bf16", "f32"]), post=rng.random() < 0.6,
                 gate=rng.choice(["none", "scalar", "token", "channel",
                                  "full"]),
                 offset=rng.choice([0.0, 1.0]),
                 rscale=rng.choice([1.0, 0.22]))
    if op.startswith("norm"):
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.5:
            H -= H % 8
        T = min(T, 2 ** 25 // H)
        return _norm(op, T, H, pad=rng.choice([0, 0, 8, 3]), **types)
    H = _log_int(rng, 64, 8192)
    H -= H % 4
    T = min(T, 2 ** 25 // H)
    E = 8 * _log_int(rng, 1, 32)
    L = E // rng.choice([1, 4, 8])
    k = rng.randint(1, min(8, E))
    if L == E:
        T = min(T, 2 ** 25 // (H * k) + 1)
    return _combine(op, T, H, E, L, k, rng.random() < 0.5, **types)


# ----------------------------------------------------------------- inputs
def _gate_shape(c):
    return {"none": None, "scalar": (1, 1), "token": (c["T"], 1),
            "channel": (1, c["H"]), "full": (c["T"], c["H"])}[c["gate"]]


def _uses_block(c):
    """Whether the norm's gradients need the block's output."""
    return c["post"] or c["gate"] != "none"


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, s = c["T"], {"case": c}

    def randn(*shape, scale=1.0, mean=0.0, dtype=F32):
        t = torch.randn(*shape, device="cuda", generator=g)
        return t.mul_(scale).add_(mean).to(dtype)

    def rows(n, width, dtype, scale=1.0):
        """[n][width] rows of a wider array where the case says so."""
        return randn(n, width + c["pad"], scale=scale, dtype=dtype)[:, :width]

    def empty(*shape, dtype=F32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    if c["op"].startswith("route"):
        E, k = c["E"], c["k"]
        logits = rows(T, E, DT[c["logits"]])
        if c["masked"]:
            off = torch.rand(E, device="cuda", generator=g) < c["masked"]
            logits[:, off] = float("-inf")
        s["logits"] = logits
        s["bias"] = randn(E, scale=0.05) if c["bias"] else None
        s["ids"] = empty(T, k, dtype=torch.int32)
        s["w"] = empty(T, k)
        s["counts"] = empty(E, dtype=torch.int32)
        if c["op"] == "route_backward":
            s["ids"] = _route_plain(s)[0]
            s["d_w"] = randn(T, k)
            s["d_logits"] = rows(T, E, DT[c["logits"]])
        if own:
            import expert_moe_fp32_amd as m
            s["router"] = m.make_router(
                T, E, k, score=c["score"], groups=c["groups"],
                topk_groups=c["keep"], group_top=c["top"],
                renormalize=c["renorm"], scale=c["scale"],
                logits=c["logits"], logits_stride=E + c["pad"])
            s["ws"] = empty(max(1, m.moe_route_scored_workspace_size(
                s["router"])), dtype=torch.uint8)
        return s

    H = c["H"]
    block, resid, out, gain = (DT[c[n]] for n in ("block", "resid", "out",
                                                   "gain"))
    shape = _gate_shape(c)
    if c["op"] != "combine_backward":
        mean = 1.0 - c["offset"]
        s["post"] = (randn(H, scale=0.1, mean=mean, dtype=gain) if c["post"]
                     else None)
        s["pre"] = randn(H, scale=0.1, mean=mean, dtype=gain)
        s["gate"] = (None if shape is None
                     else randn(*shape, scale=0.3, mean=0.5))
        s["resid"] = rows(T, H, resid, scale=2.0)
        if c["op"] == "norm_backward":
            s["y"] = rows(T, H, block)
            s["d_x"], s["d_resid_out"] = rows(T, H, out), rows(T, H, resid)
            s["d_y"], s["d_resid"] = rows(T, H, block), rows(T, H, resid)
            s["d_pre"] = empty(H)
            s["d_post"] = empty(H) if c["post"] else None
            s["d_gate"] = None if shape is None else empty(*shape)
        else:
            s["resid_out"], s["x"] = rows(T, H, resid), rows(T, H, out)
            if c["op"] == "norm":
                s["y"] = rows(T, H, block)
        if own:
            import expert_moe_fp32_amd as m
            s["norm"] = m.make_norm(
                T, H, block=c["block"], resid=c["resid"], out=c["out"],
                gain=c["gain"], gate_shape=shape, eps=EPS,
                gain_offset=c["offset"], residual_scale=c["rscale"],
                block_stride=H + c["pad"], resid_stride=H + c["pad"],
                resid_out_stride=H + c["pad"], out_stride=H + c["pad"])
            if c["op"] == "norm_backward":
                s["ws"] = empty(m.moe_residual_norm_workspace_size(s["norm"]),
                                dtype=torch.uint8)
    if c["op"].startswith("combine"):
        E, L, k = c["E"], c["L"], c["k"]
        ids = torch.rand(T, E, device="cuda", generator=g).topk(k).indices
        pairs = torch.nonzero((ids < L).reshape(-1)).reshape(-1)
        order = torch.argsort(ids.reshape(-1)[pairs], stable=True)
        pairs = pairs[order]                 # row -> pair, expert by expert
        N = pairs.numel()
        pair_row = torch.full((T * k,), -1, device="cuda", dtype=torch.int32)
        pair_row[pairs] = torch.arange(N, device="cuda", dtype=torch.int32)
        s["pairs"], s["pair_row"] = pairs, pair_row.reshape(T, k)
        s["w"] = randn(T, k).softmax(-1)
        # room for the local pairs: the expected ones and six deviations
        mean = T * k * L / E
        room = min(T * min(k, L), int(mean + 6 * mean ** 0.5) + 8)
        s["y_perm"] = randn(room, H)
        s["y_shared"] = randn(T, H) if c["shared"] else None
        if c["op"] == "combine_backward":
            s["d_out"] = randn(T, H, dtype=block)
            s["d_y_perm"] = torch.zeros(room, H, device="cuda")
            s["d_w"] = empty(T, k)
            s["d_y_shared"] = empty(T, H) if c["shared"] else None
        if own:
            import expert_moe_fp32_amd as m
            act = "f32" if H % 128 else "bf16"
            s["problem"] = m.make_problem(
                T, H, 128, E, k, num_local=L, has_shared=c["shared"],
                act=act, wdt=act, out=c["block"])
    return s


# ------------------------------------------------------- the plain forms
def _scores(c, logits):
    """Scores in 64 bits: neighbouring values decide the choice."""
    l = logits.double()
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def _route_plain(s):
    c, logits = s["case"], s["logits"]
    T, E, k = c["T"], c["E"], c["k"]
    low = float("-inf")
    score = _scores(c, logits)
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(logits.double() > low, choice, low)
    if c["groups"] > 1:
        per = choice.reshape(T, c["groups"], -1)
        best = per.sort(dim=-1, descending=True).values[..., :c["top"]]
        total = torch.where(best > low, best, 0.0).sum(-1)
        total = torch.where(best[..., 0] > low, total, low)
        kept = total.sort(dim=-1, descending=True, stable=True).indices
        drop = torch.ones_like(total, dtype=torch.bool)
        drop.scatter_(1, kept[:, :c["keep"]], False)
        drop = drop[..., None].expand_as(per).reshape(T, E)
        # live experts, then masked ones of the kept groups, then the rest
        order = choice.masked_fill(drop, low)
        first = order.sort(dim=-1, descending=True, stable=True).indices
        rest = drop.gather(1, first).sort(dim=-1, stable=True).indices
        ids = first.gather(1, rest)[:, :k]
    else:
        ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    counts = (ids.reshape(-1)[:, None] == torch.arange(
        E, device=ids.device)).sum(0) if T * k * E < 2 ** 24 else \
        torch.bincount(ids.reshape(-1), minlength=E)
    return ids.int(), (w * c["scale"]).float(), counts.int()


def _route_backward_plain(s):
    c, ids = s["case"], s["ids"].long()
    p = _scores(c, s["logits"])
    chosen, d_w = p.gather(1, ids), s["d_w"].double() * c["scale"]
    if c["renorm"]:
        total = chosen.sum(-1, keepdim=True)
        d_s = (d_w - (d_w * chosen).sum(-1, keepdim=True) / total) / total
    else:
        d_s = d_w
    if c["score"] == "sigmoid":
        d = torch.zeros_like(p).scatter_(1, ids, d_s * chosen * (1 - chosen))
    else:
        d = -p * (d_s * chosen).sum(-1, keepdim=True)
        d.scatter_add_(1, ids, d_s * chosen)
    return d.to(s["logits"].dtype)


def _gain(c, g):
    return g.float() + c["offset"]


def _rsqrt(t):
    return torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS)


def _norm_plain(s, y):
    c = s["case"]
    v = y if s["post"] is None else y * _rsqrt(y) * _gain(c, s["post"])
    if s["gate"] is not None:
        v = v * s["gate"]
    r = s["resid"].float() + c["rscale"] * v
    x = r * _rsqrt(r) * _gain(c, s["pre"])
    return r.to(DT[c["resid"]]), x.to(DT[c["out"]])


def _norm_backward_plain(s):
    c = s["case"]
    r, d_x, y = s["resid"].float(), s["d_x"].float(), s["y"].float()
    rs = _rsqrt(r)
    g = d_x * _gain(c, s["pre"])
    d_r = s["d_resid_out"].float() + rs * (
        g - r * rs * (g * r * rs).mean(-1, keepdim=True))
    d_pre = (d_x * r * rs).sum(0)
    ys = _rsqrt(y) if s["post"] is not None else 1.0
    v = y * ys
    if s["post"] is not None:
        v = v * _gain(c, s["post"])
    d_v, d_gate = c["rscale"] * d_r, None
    if s["gate"] is not None:
        d_gate = d_v * v
        if s["gate"].shape[0] == 1:
            d_gate = d_gate.sum(0, keepdim=True)
        if s["gate"].shape[1] == 1:
            d_gate = d_gate.sum(1, keepdim=True)
        d_v = d_v * s["gate"]
    d_post, d_y = None, d_v
    if s["post"] is not None:
        d_post = (d_v * y * ys).sum(0)
        g = d_v * _gain(c, s["post"])
        d_y = ys * (g - y * ys * (g * y * ys).mean(-1, keepdim=True))
    return (d_r.to(DT[c["resid"]]), d_y.to(DT[c["block"]]), d_pre, d_post,
            d_gate)


def _combine_plain(s):
    c, pairs = s["case"], s["pairs"]
    y = (s["y_shared"].clone() if s["y_shared"] is not None else
         torch.zeros(c["T"], c["H"], device=pairs.device))
    rows = s["y_perm"][:pairs.numel()] * s["w"].reshape(-1)[pairs][:, None]
    return y.index_add_(0, pairs // c["k"], rows)


def _combine_backward_plain(s):
    c, pairs = s["case"], s["pairs"]
    N = pairs.numel()
    d = s["d_out"].float()
    per_row = d[pairs // c["k"]]
    d_y = torch.zeros_like(s["d_y_perm"])
    d_y[:N] = per_row * s["w"].reshape(-1)[pairs][:, None]
    d_w = torch.zeros(c["T"] * c["k"], device=d.device)
    d_w[pairs] = (per_row * s["y_perm"][:N]).sum(-1)
    return (d_y, d_w.reshape(c["T"], c["k"]), d if c["shared"] else None)


# ------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "route":
            return _route_plain(s)
        if op == "route_backward":
            return _route_backward_plain(s)
        if op == "norm":
            return _norm_plain(s, s["y"].float())
        if op == "norm_backward":
            return _norm_backward_plain(s)
        if op == "combine_norm":
            return _norm_plain(s, _combine_plain(s))
        return _combine_backward_plain(s)
    import expert_moe_fp32_amd as m
    if op == "route":
        m.moe_route_scored(s["router"], s["logits"], s["bias"], s["ids"],
                           s["w"], s["counts"], s["ws"], s["ws"].numel())
        return s["ids"], s["w"], s["counts"]
    if op == "route_backward":
        m.moe_route_scored_backward(s["router"], s["logits"], s["ids"],
                                    s["d_w"], s["d_logits"])
        return s["d_logits"]
    if op == "norm":
        m.moe_residual_norm(s["norm"], s["y"], s["resid"], s["post"],
                            s["gate"], s["pre"], s["resid_out"], s["x"])
        return s["resid_out"], s["x"]
    if op == "norm_backward":
        m.moe_residual_norm_backward(
            s["norm"], s["y"] if _uses_block(c) else None, s["resid"],
            s["post"], s["gate"], s["pre"], s["d_x"], s["d_resid_out"],
            s["d_y"], s["d_resid"], s["d_post"], s["d_gate"], s["d_pre"],
            s["ws"], s["ws"].numel())
        return s["d_resid"], s["d_y"], s["d_pre"], s["d_post"], s["d_gate"]
    if op == "combine_norm":
        m.moe_combine_norm(s["problem"], s["norm"], s["y_perm"],
                           s["pair_row"], s["w"], s["y_shared"], s["resid"],
                           s["post"], s["gate"], s["pre"], None,
                           s["resid_out"], s["x"])
        return s["resid_out"], s["x"]
    m.moe_combine_backward(s["problem"], s["d_out"], s["y_perm"],
                           s["pair_row"], s["w"], s["d_y_perm"], s["d_w"],
                           s["d_y_shared"])
    return s["d_y_perm"], s["d_w"], s["d_y_shared"]


# --------------------------------------------------- what a pass must move
def work(case):
    c = case
    T = c["T"]
    if c["op"].startswith("route"):
        E, k, b = c["E"], c["k"], BYTES[c["logits"]]
        if c["op"] == "route":
            return {"bytes": T * E * b + T * k * 8 + E * 4 +
                    (E * 4 if c["bias"] else 0), "flops": 10 * T * E}
        full = c["score"] == "softmax" and not c["renorm"]
        return {"bytes": T * E * b + T * (E if full else k) * b + T * k * 8,
                "flops": 10 * T * (E if full else k)}
    H = c["H"]
    yb, rb, xb, gb = (BYTES[c[n]] for n in ("block", "resid", "out", "gain"))
    gate = {"none": 0, "scalar": 1, "token": T, "channel": H,
            "full": T * H}[c["gate"]] * 4
    gains = H * gb * (2 if c["post"] else 1)
    if c["op"] == "norm":
        return {"bytes": T * H * (yb + 2 * rb + xb) + gains + gate,
                "flops": 12 * T * H}
    if c["op"] == "norm_backward":
        y = yb if _uses_block(c) else 0
        return {"bytes": T * H * (y + yb + 3 * rb + xb) + gains + 2 * gate +
                H * 4 * (2 if c["post"] else 1), "flops": 30 * T * H}
    pairs = T * c["k"] * c["L"] / c["E"]
    if c["op"] == "combine_norm":
        return {"bytes": pairs * H * 4 + T * c["k"] * 8 +
                (T * H * 4 if c["shared"] else 0) + T * H * (2 * rb + xb) +
                gains + gate, "flops": 2 * pairs * H + 12 * T * H}
    return {"bytes": pairs * H * 8 + T * H * yb + T * c["k"] * 12 +
            (T * H * 4 if c["shared"] else 0), "flops": 3 * pairs * H}


# ----------------------------------------- the definitions, in 64 bits
def _exact_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].double().cpu().numpy()
    with np.errstate(all="ignore"):
        if c["score"] == "sigmoid":
            p = np.exp(-np.logaddexp(0.0, -l))
            p[np.isneginf(l)] = 0.0
        else:
            p = np.exp(l - np.logaddexp.reduce(l, axis=1, keepdims=True))
    q = p if s["bias"] is None else p + s["bias"].double().cpu().numpy()
    q = np.where(np.isneginf(l), -np.inf, q)
    ids = np.empty((T, k), np.int64)
    for t in range(T):
        best = []
        for g in range(G):
            live = [v for v in q[t, g * (E // G):(g + 1) * (E // G)]
                    if v > -np.inf]
            live.sort(reverse=True)
            best.append(sum(live[:c["top"]]) if live else -np.inf)
        kept = sorted(range(G), key=lambda g: (-best[g], g))[:c["keep"]]
        e = np.concatenate([np.arange(g * (E // G), (g + 1) * (E // G))
                            for g in sorted(kept)])
        ids[t] = e[np.lexsort((e, -q[t, e]))[:k]]
    w = np.take_along_axis(p, ids, 1)
    if c["renorm"]:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return (ids.astype(np.int32), w * c["scale"],
            np.bincount(ids.reshape(-1), minlength=E).astype(np.int32))


def _exact_route_backward(s):
    c = s["case"]
    l = s["logits"].double().requires_grad_()
    p = (torch.sigmoid(l) if c["score"] == "sigmoid"
         else torch.log_softmax(l, -1).exp())
    w = torch.gather(p, 1, s["ids"].long())
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    (w * c["scale"]).backward(s["d_w"].double())
    return torch.where(torch.isneginf(l), 0.0, l.grad).detach()


def _exact_norm(c, y, r, post, gate, pre):
    """The block's end as a formula on 64-bit values."""
    def unit(z):
        return z / (z.pow(2).sum(-1, keepdim=True) / c["H"] + EPS).sqrt()
    v = y if post is None else unit(y) * (post + c["offset"])
    out = r + (c["rscale"] * v if gate is None else c["rscale"] * gate * v)
    return out, (None if pre is None else unit(out) * (pre + c["offset"]))


def _exact_combine(s):
    c = s["case"]
    y = (s["y_shared"].double() if c["shared"] else
         torch.zeros(c["T"], c["H"], device="cuda", dtype=torch.float64))
    for j in range(c["k"]):
        row = s["pair_row"][:, j].long()
        here = torch.nonzero(row >= 0).reshape(-1)
        y[here] += (s["w"][here, j].double()[:, None] *
                    s["y_perm"][row[here]].double())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "route_backward":
        return _exact_route_backward(s)
    if op == "combine_backward":
        d, d_y = s["d_out"].double(), torch.zeros_like(
            s["d_y_perm"], dtype=torch.float64)
        d_w = torch.zeros(c["T"], c["k"], device="cuda", dtype=torch.float64)
        for j in range(c["k"]):
            row = s["pair_row"][:, j].long()
            here = torch.nonzero(row >= 0).reshape(-1)
            d_y[row[here]] = d[here] * s["w"][here, j].double()[:, None]
            d_w[here, j] = (d[here] * s["y_perm"][row[here]].double()).sum(-1)
        return d_y, d_w, d if c["shared"] else None

    def leaf(t):
        return None if t is None else t.double().requires_grad_()

    post, gate, pre = leaf(s["post"]), leaf(s["gate"]), leaf(s["pre"])
    if op != "norm_backward":
        with torch.no_grad():
            y = s["y"].double() if op == "norm" else _exact_combine(s)
            return _exact_norm(c, y, s["resid"].double(), post, gate, pre)
    # the gradient that reaches r' (given as `resid`): through the pre-norm
    # and directly; then back through the post-norm, gate and residual add
    r = leaf(s["resid"])
    with torch.enable_grad():
        x = _exact_norm(c, torch.zeros_like(r), r, None, None, pre)[1]
        d_r, d_pre = torch.autograd.grad(x, (r, pre), s["d_x"].double())
        d_r = d_r + s["d_resid_out"].double()
        y = leaf(s["y"])
        out = _exact_norm(c, y, r.detach(), post, gate, None)[0]
        wrt = [t for t in (y, post, gate) if t is not None]
        got = list(torch.autograd.grad(out, wrt, d_r))
    d_y = got.pop(0)
    d_post = got.pop(0) if post is not None else None
    return d_r, d_y, d_pre, d_post, got.pop(0) if gate is not None else None
