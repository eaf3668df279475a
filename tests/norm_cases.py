"""Inputs, calls and error bounds of the residual-norm tests.

Bounds count float32 roundings (u = 2^-24) on the magnitudes that enter each
sum, and half a step of the type an output is rounded to.  A sum of squares
passes at most 16 terms in a thread, 6 exchanges in a wavefront and 16
partial sums: below 40 u, half of it in the root; the products and the root
add fewer than 10 u."""
import numpy as np

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def torch_dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


class NormCase:
    def __init__(self, T, H, block="bf16", resid="bf16", out="bf16",
                 gain="f32", post=True, pre=True, gate=None, offset=0.0,
                 rscale=1.0, eps=1e-5, pads=(0, 0, 0, 0), shift=0, seed=0,
                 y=True):
        import torch
        import expert_moe_fp32_amd as m
        self.T, self.H = T, H
        self.types = dict(block=block, resid=resid, out=out, gain=gain)
        g = torch.Generator().manual_seed(seed)
        shape = {None: None, "scalar": (1, 1), "token": (T, 1),
                 "channel": (1, H), "full": (T, H)}[gate]

        def vec(*s, scale=1.0, mean=0.0, dt="f32"):
            t = mean + scale * torch.randn(*s, generator=g)
            return t.to(torch_dtype(dt)).cuda()

        # rows [T+1][H+pad], `shift` elements off the allocation's start; the
        # last row and the pads are never to be touched
        def rows(dt, pad, scale=1.0):
            flat = vec(shift + (T + 1) * (H + pad), scale=scale, dt=dt)
            return flat[shift:].view(T + 1, H + pad)

        self.rows = rows
        self.pads = pads
        self.n = m.make_norm(T, H, **self.types, eps=eps, gain_offset=offset,
                             residual_scale=rscale, gate_shape=shape,
                             block_stride=H + pads[0],
                             resid_stride=H + pads[1],
                             resid_out_stride=H + pads[2],
                             out_stride=H + pads[3])
        self.kw = dict(eps=float(np.float32(eps)), gain_offset=offset,
                       residual_scale=float(np.float32(rscale)))
        self.y = rows(block, pads[0]) if y else None
        self.resid = rows(resid, pads[1], 2.0)
        self.post = vec(H, scale=0.2, mean=1 - offset, dt=gain) if post else None
        self.pre = vec(H, scale=0.2, mean=1 - offset, dt=gain) if pre else None
        self.gate = None if shape is None else vec(*shape, scale=0.5, mean=0.3)
        self.resid_out = rows(resid, pads[2])
        self.x = rows(out, pads[3]) if pre else None

    def f64(self, t):
        if t is None:
            return None
        if t.dim() == 2 and t.shape[0] == self.T + 1:
            t = t[:self.T, :self.H]
        return t.double().cpu().numpy()

    def forward(self):
        import expert_moe_fp32_amd as m
        m.moe_residual_norm(self.n, self.y, self.resid, self.post, self.gate,
                            self.pre, self.resid_out, self.x)

    def edges(self, *tensors):
        """What lies around each array's rows."""
        return [(t[self.T].clone(), t[:, self.H:].clone()) for t in tensors
                if t is not None]


def rms_inv(z, eps):
    return 1.0 / np.sqrt(np.mean(z * z, -1, keepdims=True) + eps)


def norm2(z):
    return np.sqrt(np.mean(z * z, -1, keepdims=True))


def ratio(a, b):
    """|a| / |b| row by row, at least 1 (0 / 0 = 1)."""
    a, b = norm2(a), norm2(b)
    return np.maximum(1.0, np.divide(a, b, out=np.ones_like(a), where=b > 0))


def check_forward(c, got_r, got_x, y=None, y_mag=None):
    """`y`, `y_mag`: the block rows in float64 and the magnitude of the terms
    that a float32 sum made them from (default: exact rows)."""
    from oracle import block as ob
    y = c.f64(c.y) if y is None else y
    y_mag = np.zeros(1) if y_mag is None else y_mag
    r, post, gate, pre = (c.f64(t) for t in (c.resid, c.post, c.gate, c.pre))
    ref_r, ref_x = ob.residual_norm(y, r, post, gate, pre, **c.kw)
    mag = np.abs(r)                         # magnitude of resid_out's terms
    if y is not None:
        v, e = np.abs(y), np.abs(y_mag)
        if post is not None:
            s = rms_inv(y, c.kw["eps"]) * np.abs(c.kw["gain_offset"] + post)
            spread = ratio(y_mag, y) if y_mag.size > 1 else 1.0
            v, e = v * s * spread, e * s
        f = abs(c.kw["residual_scale"]) * (1.0 if gate is None else np.abs(gate))
        mag = mag + f * (v + e)
    tol = HALF[c.types["resid"]] * np.abs(ref_r) + 60 * U * mag
    err = np.abs(got_r - ref_r)
    assert (err <= tol).all(), f"resid_out {np.max(err / tol)} of its bound"
    if pre is not None:
        s = rms_inv(ref_r, c.kw["eps"]) * np.abs(c.kw["gain_offset"] + pre)
        tol = HALF[c.types["out"]] * np.abs(ref_x) + 60 * U * (
            mag * s + np.abs(ref_x) * (1 + ratio(mag, ref_r)))
        err = np.abs(got_x - ref_x)
        assert (err <= tol).all(), f"x_out {np.max(err / tol)} of its bound"


def check_backward(c, got, resid_out, d_x, d_ro):
    """got: dict of float64 results; the bounds follow the terms through the
    two norms' backward (a mean of products each, so magnitudes replace the
    products)."""
    from oracle import block as ob
    y, post, gate, pre = (c.f64(t) for t in (c.y, c.post, c.gate, c.pre))
    ref = ob.residual_norm_backward(y, resid_out, post, gate, pre, d_x, d_ro,
                                    **c.kw)
    eps, off, sc = c.kw["eps"], c.kw["gain_offset"], abs(c.kw["residual_scale"])
    mg = np.zeros((c.T, c.H)) if d_ro is None else np.abs(d_ro)
    if pre is not None:
        a = np.abs(resid_out)
        rs = rms_inv(resid_out, eps)
        gp = np.abs(d_x * (off + pre))
        mg = mg + rs * (gp + a * rs * rs * np.mean(gp * a, -1, keepdims=True))

    def check(name, tol_abs, out_type):
        if name not in got:
            return
        tol = HALF[out_type] * np.abs(ref[name]) + tol_abs + 1e-42
        err = np.abs(got[name] - ref[name])
        assert (err <= tol).all(), f"{name} {np.max(err / tol)} of its bound"

    many = 160 + c.T / 64                   # chains of a sum over the rows
    check("d_resid", 80 * U * mg, c.types["resid"])
    if pre is not None:
        check("d_pre", many * U * np.sum(np.abs(d_x * resid_out) * rs, 0), "f32")
    f = sc * (1.0 if gate is None else np.abs(gate))
    mv = f * mg
    if y is not None:
        ya = np.abs(y)
        ys = rms_inv(y, eps) if post is not None else 1.0
        pg = np.abs(off + post) if post is not None else 1.0
        if gate is not None:
            check("d_gate", many * U * ob.reduce_to(sc * mg * ya * ys * pg,
                                                    gate.shape), "f32")
        if post is not None:
            check("d_post", many * U * np.sum(mv * ya * ys, 0), "f32")
            q = mv * pg
            mv = ys * (q + ya * ys * ys * np.mean(q * ya, -1, keepdims=True))
    check("d_y", 160 * U * mv, c.types["block"])
