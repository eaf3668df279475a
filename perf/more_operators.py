"""Timing cases of the layer for a few tokens, of 8-bit activation
checkpoints, and of the experts' forward and backward pass that use them.

Five operators, each in its plain form (elementary torch operations) and as a
user of the library calls it:

  few         the whole layer, from the router's logits, for up to 16 tokens
  checkpoint  rows of activations to E4M3 codes, one power-of-two scale for
              each 128 columns
  restore     the codes back to rows
  forward     dispatch, experts and combine, leaving 8-bit checkpoints of the
              layer's input and of the experts' gate and up products
  backward    the gradients of `forward` from those checkpoints: of its input,
              of the route weights and of the experts' weights

``own`` selects the library's kernels; without it nothing but torch is used.
"""
import torch

own = False

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
FP8 = torch.float8_e4m3fn
DT = {"f32": F32, "bf16": BF16}
BYTES = {"f32": 4, "bf16": 2, "fp8": 1}


# ------------------------------------------------------------------ cases
def _few(T, H, I, E, L, k, wdt="bf16", shared=False, score="topk"):
    return dict(op="few", T=T, H=H, I=I, E=E, L=L, k=k, wdt=wdt,
                shared=shared, score=score)


def _rows(op, T, C, dtype="bf16", pad=0):
    return dict(op=op, T=T, C=C, dtype=dtype, pad=pad)


def _experts(op, T, H, I, E, L, k, shared=False, skew=0.0):
    return dict(op=op, T=T, H=H, I=I, E=E, L=L, k=k, shared=shared, skew=skew)


def listed():
    cases = {
        # one token of a small model, every expert here
        "few small": _few(1, 256, 128, 8, 8, 2),
        # sixteen decoding sequences of a 256-expert model, 32 experts here
        "few decode": _few(16, 6144, 2048, 256, 32, 8, score="sigmoid"),
        # a few sequences with FP8 weights and a shared expert
        "few lowlat": _few(4, 7168, 2048, 256, 32, 8, "fp8", True),
        # the layer's input in a prefill-sized micro-batch
        "checkpoint train": _rows("checkpoint", 8192, 7168),
        # float32 rows of odd sizes, a slice of a wider array
        "checkpoint odd": _rows("checkpoint", 1021, 2501, "f32", 3),
        # the same micro-batch back to bf16
        "restore train": _rows("restore", 8192, 7168),
        # a small batch back to float32 rows
        "restore small": _rows("restore", 128, 256, "f32"),
        # a ragged batch of a small model, every expert here
        "forward small": _experts("forward", 509, 1024, 512, 16, 16, 2),
        # a training micro-batch: 32 of 256 experts here, shared expert
        "forward train": _experts("forward", 4096, 7168, 2048, 256, 32, 8,
                                  True),
        # the backward of the ragged batch
        "backward small": _experts("backward", 509, 1024, 512, 16, 16, 2),
        # many small experts, all here, with an uneven load
        "backward uneven": _experts("backward", 2048, 2048, 768, 64, 64, 8,
                                    skew=0.5),
        # the backward of the training micro-batch
        "backward train": _experts("backward", 4096, 7168, 2048, 256, 32, 8,
                                   True),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["few", "few", "checkpoint", "restore", "forward",
                     "backward"])
    if op in ("checkpoint", "restore"):
        C = _log_int(rng, 1, 8192)
        if rng.random() < 0.6 and C >= 128:
            C -= C % 128
        T = min(_log_int(rng, 1, 8192), 2 ** 26 // C)
        return _rows(op, T, C, rng.choice(["bf16", "f32"]),
                     rng.choice([0, 0, 8, 3]))
    E = 8 * _log_int(rng, 1, 32)
    L = E // rng.choice([1, 4, 8])
    k = rng.randint(1, min(8, E))
    I = 128 * _log_int(rng, 1, 16)
    H = 128 * _log_int(rng, 1, 56)
    while L * H * I > 2 ** 29:
        L //= 2
    shared = rng.random() < 0.4
    if op == "few":
        return _few(rng.randint(1, 16), H, I, E, L, k,
                    rng.choice(["bf16", "fp8"]), shared,
                    rng.choice(["topk", "sigmoid"]))
    T = _log_int(rng, 1, 4096)
    rows = T * k * L / E + (T if shared else 0)
    T = max(1, min(T, int(T * 8192 * 7168 * 2048 / (rows * H * I + 1))))
    return _experts(op, T, H, I, E, L, k, shared,
                    rng.choice([0.0, 0.0, 0.5]))


# ----------------------------------------------------------------- inputs
def _code(v):
    """E4M3 codes and power-of-two scales of 32-bit rows: for each 128
    columns the smallest power of two s with |v| / s <= 448."""
    T, C = v.shape
    n = -(-C // 128)
    v = torch.nn.functional.pad(v, (0, n * 128 - C)).reshape(T, n, 128)
    amax = v.abs().amax(-1)
    m, e = torch.frexp(amax)                  # amax = m 2^e, m in [1/2, 1)
    e = (e - torch.where(m <= 0.875, 9, 8)).clamp(min=-100)
    s = ((e.int() + 127) << 23).view(F32)     # 2^e
    s = torch.where(amax > 0, s, 1.0)
    codes = (v / s[..., None]).to(FP8).reshape(T, n * 128)[:, :C]
    return codes.contiguous().view(torch.uint8), s


def _values(codes, scales, T, C):
    """What codes [T][C] and scales [T][ceil(C / 128)] stand for."""
    s = scales.repeat_interleave(128, 1)[:, :C]
    return codes.view(FP8).to(s.dtype) * s


def _route(c, g):
    """ids [T][k] and weights, with an expert's odds falling as skew says."""
    logits = torch.randn(c["T"], c["E"], device="cuda", generator=g)
    rank = torch.randperm(c["E"], device="cuda", generator=g) + 1
    top = (logits - c["skew"] * rank.log()).topk(c["k"])
    return top.indices.int(), top.values.softmax(-1)


def _index(c, ids, N):
    """Rows of the local pairs, expert by expert: (pair of each row, its
    expert, offsets [L + 1])."""
    flat = ids.reshape(-1).long()
    order = torch.where(flat < c["L"], flat, c["L"]).argsort(stable=True)
    pairs = order[:N]
    e = flat[pairs]
    counts = (e[:, None] == torch.arange(c["L"], device=e.device)).sum(0)
    offsets = torch.zeros(c["L"] + 1, device=e.device, dtype=torch.int64)
    offsets[1:] = counts.cumsum(0)
    return pairs, e, offsets


def _weights(c, g, s):
    """Expert weights [P][H][I], [P][H][I], [P][I][H], the shared expert last;
    FP8: codes and scales of 128 x 128 blocks."""
    P, H, I = c["L"] + int(c["shared"]), c["H"], c["I"]
    for name, K, N in (("wg", H, I), ("wu", H, I), ("wd", I, H)):
        w = torch.randn(P, K, N, device="cuda", generator=g).mul_(K ** -0.5)
        if c.get("wdt") == "fp8":
            b = w.reshape(P, K // 128, 128, N // 128, 128)
            sc = b.abs().amax((2, 4)) / 448.0
            q = (b / sc[:, :, None, :, None]).clamp(-448, 448)
            s[name] = q.to(FP8).reshape(P, K, N)
            s["s" + name[1]] = sc
        else:
            s[name] = w.to(BF16)
    if not own:
        return
    import expert_moe_fp32_amd as m
    fp8 = c.get("wdt") == "fp8"
    experts = []
    for p in range(P):
        d = {}
        for name in ("wg", "wu", "wd"):
            src = s[name][p]
            K, N = src.shape
            src = src.view(torch.uint8) if fp8 else src
            dst = torch.empty_like(src)
            m.moe_prepack_weights(src, K, N,
                                  m._lib.MOE_FP8_E4M3 if fp8
                                  else m._lib.MOE_BF16, m.MOE_LAYOUT_KN, dst)
            d[name] = dst
            if fp8:
                d["s" + name[1]] = s["s" + name[1]][p].t().contiguous()
        experts.append(d)
    shared = experts.pop() if c["shared"] else None
    s["weights"] = m.device_weights(experts, shared)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, s = c["T"], {"case": c}

    def randn(*shape, scale=1.0, dtype=F32):
        t = torch.randn(*shape, device="cuda", generator=g)
        return t.mul_(scale).to(dtype)

    def empty(*shape, dtype=F32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    if c["op"] in ("checkpoint", "restore"):
        C, n = c["C"], -(-c["C"] // 128)
        rows = randn(T, C + c["pad"], dtype=DT[c["dtype"]])[:, :C]
        # channels of different size, as activations have them
        s["rows"] = rows.mul_(randn(C).exp().to(rows.dtype))
        s["codes"] = empty(T, C, dtype=torch.uint8)
        s["scales"] = empty(T, n)
        if c["op"] == "restore":
            s["codes"], s["scales"] = _code(s["rows"].float())
        if own:
            import expert_moe_fp32_amd as m
            s["desc"] = m.make_rows(T, C, dtype=c["dtype"],
                                    stride=C + c["pad"])
        return s

    H, I, E, L, k = (c[n] for n in ("H", "I", "E", "L", "k"))
    s["x"] = randn(T, H, dtype=BF16)
    _weights(c, g, s)
    if own:
        import expert_moe_fp32_amd as m
        s["problem"] = m.make_problem(T, H, I, E, k, num_local=L,
                                      has_shared=c["shared"],
                                      wdt=c.get("wdt", "bf16"))
    if c["op"] == "few":
        s["logits"] = randn(T, E)
        sigmoid = c["score"] == "sigmoid"
        s["bias"] = randn(E, scale=0.05) if sigmoid else None
        s["out"] = empty(T, H, dtype=BF16)
        if own:
            s["router"] = (m.make_router(T, E, k, score="sigmoid", scale=2.5)
                           if sigmoid else None)
            s["ws"] = empty(m.moe_layer_few_workspace_size(s["problem"]),
                            dtype=torch.uint8)
        return s

    s["ids"], s["w"] = _route(c, g)
    # host sizes for slices of what a pass returns and for the plain form
    counts = torch.bincount(s["ids"].reshape(-1), minlength=E)[:L].tolist()
    s["N"], s["most"] = sum(counts), max(counts)
    cap = T * min(k, L)
    rows = cap + (T if c["shared"] else 0)
    # routed rows of what a pass returns: room for the local pairs (the
    # expected ones and six deviations), the rows behind the last one zero
    mean = T * k * L / E
    s["room"] = (cap if c["skew"] else
                 min(cap, int(mean + 6 * mean ** 0.5) + 8))
    saved = dict(
        offsets=empty(L + 1, dtype=torch.int32),
        row_token=empty(cap, dtype=torch.int32), row_weight=empty(cap),
        pair_row=empty(T, k, dtype=torch.int32),
        x_codes=empty(T, H, dtype=torch.uint8), x_scales=empty(T, H // 128),
        gu_codes=empty(rows, 2 * I, dtype=torch.uint8).zero_(),
        gu_scales=empty(rows, 2 * I // 128).zero_())
    s["saved"], s["cap"] = saved, cap
    if c["op"] == "forward":
        s["out"] = empty(T, H, dtype=BF16)
    else:
        # what the forward pass left
        pairs, _, offsets = _index(c, s["ids"], s["N"])
        N = s["N"]
        saved["offsets"].copy_(offsets)
        saved["row_token"][:N] = pairs // k
        saved["row_weight"][:N] = s["w"].reshape(-1)[pairs]
        saved["pair_row"].fill_(-1).reshape(-1)[pairs] = torch.arange(
            N, device="cuda", dtype=torch.int32)
        saved["x_codes"], saved["x_scales"] = _code(s["x"].float())
        for at, n in ((0, N), (cap, rows - cap)):
            codes, scales = _code(randn(n, 2 * I))
            saved["gu_codes"][at:at + n] = codes
            saved["gu_scales"][at:at + n] = scales
        s["d_out"] = randn(T, H, dtype=BF16)
        s["d_x"] = empty(T, H, dtype=BF16)
        s["d_w"] = empty(T, k)
        P = L + int(c["shared"])
        s["d_wg"], s["d_wu"] = (empty(P, H, I, dtype=BF16) for _ in range(2))
        s["d_wd"] = empty(P, I, H, dtype=BF16)
    if own:
        s["handle"] = m.make_saved(**saved)
        if c["op"] == "backward":
            end = dict(sh_gate=s["d_wg"][L], sh_up=s["d_wu"][L],
                       sh_down=s["d_wd"][L]) if c["shared"] else {}
            s["grads"] = m.make_weight_grads(s["d_wg"], s["d_wu"], s["d_wd"],
                                             dtype="bf16", **end)
        s["ws"] = empty(m.moe_experts_workspace_size(s["problem"]),
                        dtype=torch.uint8)
    return s


# ------------------------------------------------------- the plain forms
def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _matrix(s, name, which, dtype):
    """Weights of the experts `which` (indices) as plain numbers."""
    w = s[name][which]
    if w.dtype != FP8:
        return w.to(dtype)
    sc = s["s" + name[1]][which].to(dtype)
    return w.to(dtype) * sc.repeat_interleave(128, 1).repeat_interleave(128, 2)


def _few_route(s):
    """ids and weights [T][k] (choices of a sigmoid router in 64 bits)."""
    c = s["case"]
    if c["score"] == "topk":
        order = s["logits"].sort(dim=-1, descending=True, stable=True)
        ids = order.indices[:, :c["k"]]
        top = order.values[:, :c["k"]]
        e = torch.exp(top - top[:, :1])
        return ids, e / e.sum(-1, keepdim=True)
    score = 1.0 / (1.0 + torch.exp(-s["logits"].double()))
    order = (score + s["bias"].double()).sort(dim=-1, descending=True,
                                              stable=True)
    ids = order.indices[:, :c["k"]]
    w = score.gather(1, ids)
    return ids, (2.5 * w / w.sum(-1, keepdim=True)).float()


def _few_plain(s):
    c = s["case"]
    T, L = c["T"], c["L"]
    ids, w = _few_route(s)
    # weight of every expert here for every token, and the experts in use
    share = torch.zeros(T, c["E"], device=ids.device).scatter_(1, ids, w)
    share = share[:, :L]
    used = torch.zeros(T, c["E"], device=ids.device).scatter_(1, ids, 1.0)
    used = torch.nonzero(used[:, :L].amax(0)).reshape(-1)
    share = share[:, used]
    if c["shared"]:
        used = torch.nn.functional.pad(used, (0, 1), value=L)
        share = torch.nn.functional.pad(share, (0, 1), value=1.0)
    x = s["x"].float().expand(used.numel(), T, c["H"])
    h = _silu(torch.bmm(x, _matrix(s, "wg", used, F32))) * torch.bmm(
        x, _matrix(s, "wu", used, F32))
    y = torch.bmm(h, _matrix(s, "wd", used, F32))
    return (y * share.t()[..., None]).sum(0).to(BF16)


def _spread(rows, e, pos, P, most):
    """Rows of experts as [P][most][columns], zeros between."""
    out = torch.zeros(P, most, rows.shape[1], device=rows.device,
                      dtype=rows.dtype)
    out[e, pos] = rows
    return out


def _forward_plain(s):
    c, N = s["case"], s["N"]
    L, k, I = c["L"], c["k"], c["I"]
    pairs, e, offsets = _index(c, s["ids"], N)
    pos = torch.arange(N, device=e.device) - offsets[e]
    token = pairs // k
    x = s["x"].float()
    xp = _spread(x[token], e, pos, L, s["most"])
    g = torch.bmm(xp, s["wg"][:L].float())
    u = torch.bmm(xp, s["wu"][:L].float())
    y = torch.bmm(_silu(g) * u, s["wd"][:L].float())
    out = torch.zeros_like(x).index_add_(
        0, token, y[e, pos] * s["w"].reshape(-1)[pairs][:, None])
    gu, gu_shared = torch.cat([g[e, pos], u[e, pos]], 1), None
    if c["shared"]:
        g, u = x @ s["wg"][L].float(), x @ s["wu"][L].float()
        out += (_silu(g) * u) @ s["wd"][L].float()
        gu_shared = _values(*_code(torch.cat([g, u], 1)), c["T"],
                            2 * I).to(BF16)
    pair_row = torch.full((c["T"] * k,), -1, device=e.device,
                          dtype=torch.int32)
    pair_row[pairs] = torch.arange(N, device=e.device, dtype=torch.int32)
    return (out.to(BF16), offsets.int(), pair_row.reshape(c["T"], k),
            _values(*_code(x), c["T"], c["H"]).to(BF16),
            torch.nn.functional.pad(_values(*_code(gu), N, 2 * I).to(BF16),
                                    (0, 0, 0, s["room"] - N)), gu_shared)


def _backward_plain(s):
    c, N, sv = s["case"], s["N"], s["saved"]
    T, H, I, L, k, cap = c["T"], c["H"], c["I"], c["L"], c["k"], s["cap"]
    pairs, e, offsets = _index(c, s["ids"], N)
    pos = torch.arange(N, device=e.device) - offsets[e]
    token = pairs // k
    x = _values(sv["x_codes"], sv["x_scales"], T, H)
    d = s["d_out"].float()

    def through(g, u, dh):
        """silu(g) u and the gradients of g and u"""
        q = 1.0 / (1.0 + torch.exp(-g))
        return (g * q * u, dh * u * q * (1.0 + g * (1.0 - q)), dh * g * q)

    gu = _values(sv["gu_codes"][:N], sv["gu_scales"][:N], N, 2 * I)
    gu = _spread(gu, e, pos, L, s["most"])
    xp = _spread(x[token], e, pos, L, s["most"])
    dp = _spread(d[token], e, pos, L, s["most"])
    wp = _spread(s["w"].reshape(-1, 1)[pairs], e, pos, L, s["most"])
    wg, wu, wd = (s[n][:L].float() for n in ("wg", "wu", "wd"))
    dh = torch.bmm(dp, wd.transpose(1, 2).contiguous())
    h, dg, du = through(gu[..., :I], gu[..., I:], dh * wp)
    d_w = torch.zeros(T * k, device=d.device)
    d_w[pairs] = (h * dh).sum(-1)[e, pos]
    dx = torch.bmm(dg, wg.transpose(1, 2).contiguous())
    dx += torch.bmm(du, wu.transpose(1, 2).contiguous())
    d_x = torch.zeros_like(x).index_add_(0, token, dx[e, pos])
    xt = xp.transpose(1, 2).contiguous()
    d_wg, d_wu = torch.bmm(xt, dg), torch.bmm(xt, du)
    d_wd = torch.bmm((h * wp).transpose(1, 2).contiguous(), dp)
    ends = (None,) * 3
    if c["shared"]:
        gu = _values(sv["gu_codes"][cap:], sv["gu_scales"][cap:], T, 2 * I)
        wg, wu, wd = (s[n][L].float() for n in ("wg", "wu", "wd"))
        h, dg, du = through(gu[:, :I], gu[:, I:], d @ wd.t())
        d_x += dg @ wg.t() + du @ wu.t()
        ends = (x.t() @ dg).to(BF16), (x.t() @ du).to(BF16), (
            h.t() @ d).to(BF16)
    return (d_x.to(BF16), d_w.reshape(T, k), d_wg.to(BF16), d_wu.to(BF16),
            d_wd.to(BF16), *ends)


# ------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "few":
            return _few_plain(s)
        if op == "checkpoint":
            codes, scales = _code(s["rows"].float())
            return codes.view(FP8), scales
        if op == "restore":
            return _values(s["codes"], s["scales"], c["T"],
                           c["C"]).to(DT[c["dtype"]])
        return _forward_plain(s) if op == "forward" else _backward_plain(s)
    import expert_moe_fp32_amd as m
    if op == "few":
        m.moe_layer_forward_few(s["problem"], s["router"], s["logits"],
                                s["bias"], s["x"], s["weights"].struct, None,
                                None, s["out"], None, s["ws"],
                                s["ws"].numel())
        return s["out"]
    if op == "checkpoint":
        m.moe_checkpoint_rows(s["desc"], s["rows"], s["codes"], s["scales"])
        return s["codes"].view(FP8), s["scales"]
    if op == "restore":
        m.moe_restore_rows(s["desc"], s["codes"], s["scales"], s["rows"])
        return s["rows"]
    sv, room, L = s["saved"], s["room"], c["L"]
    if op == "forward":
        m.moe_experts_forward(s["problem"], s["x"], s["ids"], s["w"], None,
                              None, s["weights"].struct, s["handle"],
                              s["out"], s["ws"], s["ws"].numel())

        def values(codes, scales):
            rows = torch.empty(codes.shape, device=codes.device, dtype=BF16)
            m.moe_restore_rows(m.make_rows(*codes.shape), codes, scales, rows)
            return rows
        cap = s["cap"]
        return (s["out"], sv["offsets"], sv["pair_row"],
                values(sv["x_codes"], sv["x_scales"]),
                values(sv["gu_codes"][:room], sv["gu_scales"][:room]),
                values(sv["gu_codes"][cap:], sv["gu_scales"][cap:])
                if c["shared"] else None)
    m.moe_experts_backward(s["problem"], s["handle"], s["d_out"],
                           s["weights"].struct, s["d_x"], s["d_w"],
                           s["grads"], s["ws"], s["ws"].numel())
    ends = ((s["d_wg"][L], s["d_wu"][L], s["d_wd"][L]) if c["shared"]
            else (None,) * 3)
    return (s["d_x"], s["d_w"], s["d_wg"][:L], s["d_wu"][:L], s["d_wd"][:L],
            *ends)


# --------------------------------------------------- what a pass must move
def work(case):
    c = case
    T = c["T"]
    if c["op"] in ("checkpoint", "restore"):
        return {"bytes": T * c["C"] * (BYTES[c["dtype"]] + 1 + 4 / 128),
                "flops": 2 * T * c["C"]}
    H, I, L, E, k = (c[n] for n in ("H", "I", "L", "E", "k"))
    sh = int(c["shared"])
    pairs = T * k * L / E
    rows = pairs + sh * T
    active = L * (1 - (1 - k / E) ** T) + sh      # experts with a row
    weights = 3 * H * I * active
    if c["op"] == "few":
        return {"bytes": weights * BYTES[c["wdt"]] + T * E * 4 + T * H * 4,
                "flops": 6 * rows * H * I}
    kept = T * H * (1 + 4 / 128) + rows * 2 * I * (1 + 4 / 128)
    if c["op"] == "forward":
        return {"bytes": weights * 2 + T * H * 4 + kept + T * k * 12,
                "flops": 6 * rows * H * I}
    return {"bytes": weights * 2 + 3 * H * I * (L + sh) * 2 + T * H * 4 +
            kept + T * k * 8, "flops": 12 * rows * H * I}


# ----------------------------------------- the definitions, in 64 bits
def _exact_code(v):
    """The values that 8 bits hold of 64-bit rows, written by the grid: steps
    of 2^-3 of the value's power of two, of 2^-9 below 2^-6."""
    T, C = v.shape
    out = torch.empty_like(v)

    def power(e):
        return ((e.clamp(-1000, 1000).long() + 1023) << 52).view(F64)
    scales = torch.empty(T, -(-C // 128), device=v.device, dtype=F64)
    for n in range(scales.shape[1]):
        part = v[:, 128 * n:128 * n + 128]
        top = part.abs().max(dim=1).values
        s = power(torch.ceil(torch.log2(top / 448.0)))
        s = torch.where(top / s > 448.0, 2 * s, s)
        s = torch.where(top <= 224.0 * s, s / 2, s)
        s = torch.where(top > 0, s, 1.0)
        q = part / s[:, None]
        size = q.abs().clamp(min=2.0 ** -6)
        step = power(torch.floor(torch.log2(size)))
        step = torch.where(step > size, step / 2, step)
        step = torch.where(2 * step <= size, 2 * step, step) / 8
        out[:, 128 * n:128 * n + 128] = torch.round(q / step) * step
        scales[:, n] = s
    return out, scales


def _exact_values(v):
    codes, scales = _exact_code(v)
    return codes * scales.repeat_interleave(128, 1)[:, :v.shape[1]]


def exact(case, seed):
    s = prepare(case, seed)
    c, op, T = s["case"], case["op"], case["T"]
    if op == "checkpoint":
        return _exact_code(s["rows"].double())
    if op == "restore":
        out = torch.empty(T, c["C"], device="cuda", dtype=F64)
        for n in range(s["scales"].shape[1]):
            at = slice(128 * n, 128 * n + 128)
            b = s["codes"][:, at].int()           # sign, exponent, fraction
            x, f = (b >> 3) & 15, (b & 7).double()
            two = ((x.long() + 1016) << 52).view(F64)          # 2^(x - 7)
            v = torch.where(x > 0, (1 + f / 8) * two, f / 512)
            v = torch.where(b > 127, -v, v)
            out[:, at] = v * s["scales"][:, n:n + 1].double()
        return out
    L, k, I = c["L"], c["k"], c["I"]
    x, sh = s["x"].double(), c["shared"]

    def matrix(name, p):
        return _matrix(s, name, slice(p, p + 1), F64)[0]

    def expert(p, rows):
        g = rows @ matrix("wg", p)
        u = rows @ matrix("wu", p)
        return g, u, (g * torch.sigmoid(g) * u) @ matrix("wd", p)

    if op == "few":
        out = torch.zeros_like(x)
        choice = s["logits"].double()
        if c["score"] == "sigmoid":
            choice = torch.sigmoid(choice)
            score = choice
            choice = choice + s["bias"].double()
        else:
            score = torch.softmax(choice, -1)
        for t in range(T):
            row = choice[t].tolist()
            ids = sorted(range(c["E"]), key=lambda e: (-row[e], e))[:k]
            total = sum(score[t, e] for e in ids)
            for e in ids:
                if e < L:
                    w = score[t, e] / total
                    w = 2.5 * w if c["score"] == "sigmoid" else w
                    out[t] += w * expert(e, x[t:t + 1])[2][0]
        if sh:
            out += expert(L, x)[2]
        return out

    ids, w = s["ids"].long(), s["w"].double()
    where = [torch.nonzero(ids == p) for p in range(L)]   # token, slot
    starts = [0]
    for q in where:
        starts.append(starts[-1] + len(q))
    if op == "forward":
        out = torch.zeros_like(x)
        gu = torch.zeros(s["room"], 2 * I, device="cuda", dtype=F64)
        for p, q in enumerate(where):
            g, u, y = expert(p, x[q[:, 0]])
            gu[starts[p]:starts[p + 1]] = torch.cat([g, u], 1)
            out.index_add_(0, q[:, 0], y * w[q[:, 0], q[:, 1]][:, None])
        end = None
        if sh:
            g, u, y = expert(L, x)
            out += y
            end = _exact_values(torch.cat([g, u], 1))
        return out, None, None, _exact_values(x), _exact_values(gu), end

    sv, cap = s["saved"], s["cap"]
    x = _values(sv["x_codes"], sv["x_scales"].double(), T, c["H"])
    d = s["d_out"].double()
    d_x, d_w = torch.zeros_like(x), torch.zeros_like(w)
    d_wg, d_wu, d_wd = [], [], []
    for p in range(L + int(sh)):
        at = (slice(starts[p], starts[p + 1]) if p < L
              else slice(cap, cap + T))
        n = at.stop - at.start
        t = where[p][:, 0] if p < L else torch.arange(T, device="cuda")
        g, u = _values(sv["gu_codes"][at], sv["gu_scales"][at].double(), n,
                       2 * I).split(I, 1)
        g.requires_grad_()
        with torch.enable_grad():
            a = g * torch.sigmoid(g)
            da = torch.autograd.grad(a.sum(), g)[0]
        a, g = a.detach(), g.detach()
        dy = d[t]
        dh = dy @ matrix("wd", p).t()
        if p < L:
            d_w[t, where[p][:, 1]] = (dh * a * u).sum(-1)
            scale = w[t, where[p][:, 1]][:, None]
            dh, dy = dh * scale, dy * scale
        dg, du = dh * u * da, dh * a
        d_x.index_add_(0, t, dg @ matrix("wg", p).t() +
                       du @ matrix("wu", p).t())
        d_wg.append((x[t].t() @ dg).to(F32))
        d_wu.append((x[t].t() @ du).to(F32))
        d_wd.append(((a * u).t() @ dy).to(F32))
    ends = (d_wg.pop(), d_wu.pop(), d_wd.pop()) if sh else (None,) * 3
    return (d_x, d_w, torch.stack(d_wg), torch.stack(d_wu),
            torch.stack(d_wd), *ends)
