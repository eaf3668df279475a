"""8-bit checkpoints of rows on the GPU: codes and scales bit for bit, and
back."""
import numpy as np
import pytest

from oracle import train as ot

pytestmark = pytest.mark.gpu


def rows_of(T, C, dtype, pad, seed, shift=0):
    """Rows [T][C] of a wider array, `shift` elements into its memory."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, C + pad, generator=g) * torch.randn(
        C + pad, generator=g).mul(2).exp()
    x[T // 2] = 0.0
    if C > 200:
        x[0, 128:256] = 0.0
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    flat = torch.empty(T * (C + pad) + shift, dtype=dt, device="cuda")
    v = flat[shift:].view(T, C + pad)
    v.copy_(x.to(dt))
    return v


@pytest.mark.parametrize("T,C,dtype,pad,shift", [
    (1, 1, "f32", 0, 0), (1, 1, "bf16", 0, 0), (3, 7, "bf16", 2, 1),
    (5, 128, "bf16", 0, 0), (4, 127, "f32", 5, 0), (9, 129, "bf16", 0, 0),
    (17, 256, "f32", 0, 1), (33, 1004, "bf16", 4, 0), (33, 1004, "f32", 4, 0),
    (6, 2501, "f32", 3, 0), (6, 2501, "bf16", 0, 0), (40, 7168, "bf16", 8, 0),
    (300, 7168, "bf16", 0, 0), (2200, 640, "f32", 0, 0),
    (3000, 1001, "bf16", 0, 0), (1500, 1536, "bf16", 0, 3),
])
def test_codes_and_back(T, C, dtype, pad, shift):
    import torch
    import expert_moe_fp32_amd as m
    print(T, C, dtype, pad, shift, flush=True)
    x = rows_of(T, C, dtype, pad, T + C, shift)
    n = -(-C // 128)
    codes = torch.full((T + 1, C), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((T + 1, n), 7.0, device="cuda")
    d = m.make_rows(T, C, dtype=dtype, stride=C + pad)
    m.moe_checkpoint_rows(d, x, codes, scales)
    torch.cuda.synchronize()
    assert (codes[T] == 77).all() and (scales[T] == 7.0).all()
    some = np.unique(np.r_[0, T // 2, T - 1, np.arange(0, T, max(1, T // 20))])
    rc, rs = ot.checkpoint(x[some, :C].double().cpu().numpy())
    assert np.array_equal(scales[:T].cpu().numpy()[some], rs)
    assert np.array_equal(codes[:T].cpu().numpy()[some], rc)
    # back: exactly code * scale, which both types hold
    for to in ("f32", "bf16"):
        dt = {"f32": torch.float32, "bf16": torch.bfloat16}[to]
        y = torch.full((T + 1, C + pad), 9.0, dtype=dt, device="cuda")
        m.moe_restore_rows(m.make_rows(T, C, dtype=to, stride=C + pad), codes,
                           scales, y)
        torch.cuda.synchronize()
        v = codes[:T].view(torch.float8_e4m3fn).double()
        v = v * scales[:T].double().repeat_interleave(128, 1)[:, :C]
        assert torch.equal(y[:T, :C].double(), v)
        assert (y[:T, C:] == 9.0).all() and (y[T] == 9.0).all()


def test_what_is_not_finite_becomes_nan():
    import torch
    import expert_moe_fp32_amd as m
    x = torch.randn(3, 256, device="cuda")
    x[0, 3], x[0, 200], x[1, 5] = float("inf"), float("nan"), -float("inf")
    x[2, :128] = float("nan")
    codes = torch.empty(3, 256, dtype=torch.uint8, device="cuda")
    scales = torch.empty(3, 2, device="cuda")
    m.moe_checkpoint_rows(m.make_rows(3, 256, dtype="f32"), x, codes, scales)
    y = torch.empty_like(x)
    m.moe_restore_rows(m.make_rows(3, 256, dtype="f32"), codes, scales, y)
    torch.cuda.synchronize()
    rc, rs = ot.checkpoint(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    want = ot.values(rc, rs)
    assert np.array_equal(y.double().cpu().numpy(), want, equal_nan=True)
    assert np.isnan(want).sum() == 131


def test_the_ends_of_the_range():
    """Magnitudes from the smallest to the largest of float32, powers of two
    and the scales' borders among them."""
    import torch
    import expert_moe_fp32_amd as m
    top = torch.finfo(torch.float32).max
    sizes = [top, 2.0 ** 127, 448.0, np.nextafter(np.float32(448.0), np.float32(500.0)),
             449.0, 256.0, 224.0, 1.75, 1.0, 1e-3, 2.0 ** -90, 2.0 ** -100,
             2.0 ** -115, 1e-38, 1e-45]
    x = torch.zeros(len(sizes), 128)
    g = torch.Generator().manual_seed(1)
    for i, s in enumerate(sizes):
        x[i] = torch.rand(128, generator=g) * 2 - 1
        x[i] *= s
        x[i, 7], x[i, 11] = float(s), -float(s)
    x = x.cuda()
    codes = torch.empty(len(sizes), 128, dtype=torch.uint8, device="cuda")
    scales = torch.empty(len(sizes), 1, device="cuda")
    m.moe_checkpoint_rows(m.make_rows(len(sizes), 128, dtype="f32"), x, codes,
                          scales)
    torch.cuda.synchronize()
    rc, rs = ot.checkpoint(x.double().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), rs)
    assert np.array_equal(codes.cpu().numpy(), rc)


def test_scales_of_any_value_are_rounded_once():
    import torch
    import expert_moe_fp32_amd as m
    g = torch.Generator().manual_seed(2)
    codes = torch.randint(0, 127, (20, 300), generator=g, dtype=torch.uint8).cuda()
    scales = torch.rand(20, 3, generator=g).cuda()
    for to, half in (("f32", 2.0 ** -24), ("bf16", 2.0 ** -8)):
        dt = {"f32": torch.float32, "bf16": torch.bfloat16}[to]
        y = torch.empty(20, 300, dtype=dt, device="cuda")
        m.moe_restore_rows(m.make_rows(20, 300, dtype=to), codes, scales, y)
        torch.cuda.synchronize()
        v = codes.view(torch.float8_e4m3fn).double() * \
            scales.double().repeat_interleave(128, 1)[:, :300]
        # one product in float32, then the rounding to the type
        assert ((y.double() - v).abs() <= (half + 2.0 ** -24) * v.abs()).all()


@pytest.mark.parametrize("C", [65664, 65601])
def test_rows_beyond_32_bits(C):
    """2^32 elements and more: the rows at the end as in a small call."""
    import torch
    import expert_moe_fp32_amd as m
    T, n = 65536, -(-C // 128)
    assert T * C > 2 ** 32
    x = torch.zeros(T, C, dtype=torch.bfloat16, device="cuda")
    last = rows_of(5, C, "bf16", 0, 11)
    x[-5:] = last
    codes = torch.full((T, C), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((T, n), 7.0, device="cuda")
    small = torch.empty(5, C, dtype=torch.uint8, device="cuda"), torch.empty(5, n, device="cuda")
    m.moe_checkpoint_rows(m.make_rows(T, C, dtype="bf16"), x, codes, scales)
    m.moe_checkpoint_rows(m.make_rows(5, C, dtype="bf16"), last, *small)
    torch.cuda.synchronize()
    assert torch.equal(codes[-5:], small[0]) and torch.equal(scales[-5:], small[1])
    assert not codes[:-5:64].any() and (scales[:-5] == 1.0).all()
    x.fill_(9.0)
    m.moe_restore_rows(m.make_rows(T, C, dtype="bf16"), codes, scales, x)
    m.moe_restore_rows(m.make_rows(5, C, dtype="bf16"), *small, last)
    torch.cuda.synchronize()
    assert torch.equal(x[-5:], last) and not x[:-5:64].any()


@pytest.mark.parametrize("cut", [0, 61])
def test_the_longest_row(cut):
    """One row of almost 2^31 columns is what its groups are as rows of their
    own (and the cut group at its end)."""
    import torch
    import expert_moe_fp32_amd as m
    C = 2 ** 31 - 128 - cut
    n, whole = -(-C // 128), C // 128
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(C, device="cuda", dtype=torch.bfloat16, generator=g)
    codes, parts = (torch.full((C,), 77, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales, own = (torch.full((n,), 7.0, device="cuda") for _ in range(2))
    m.moe_checkpoint_rows(m.make_rows(1, C), x, codes, scales)
    m.moe_checkpoint_rows(m.make_rows(whole, 128), x, parts, own)
    if cut:
        m.moe_checkpoint_rows(m.make_rows(1, C % 128), x[whole * 128:],
                              parts[whole * 128:], own[whole:])
    torch.cuda.synchronize()
    assert torch.equal(codes, parts) and torch.equal(scales, own)
    y = torch.full((C,), 9.0, dtype=torch.bfloat16, device="cuda")
    m.moe_restore_rows(m.make_rows(1, C), codes, scales, y)
    m.moe_restore_rows(m.make_rows(whole, 128), codes, scales, x)
    if cut:
        m.moe_restore_rows(m.make_rows(1, C % 128), codes[whole * 128:],
                           scales[whole:], x[whole * 128:])
    torch.cuda.synchronize()
    assert torch.equal(y, x)


@pytest.mark.parametrize("T,dtype", [(2 ** 29 + 4099, "f32"),
                                     (2 ** 30 + 4099, "bf16")])
def test_more_groups_than_a_launch_has_threads_for(T, dtype):
    """Rows of one column, more than 2^29 (float32) or 2^30:
    every one as the same value in a small call."""
    import torch
    import expert_moe_fp32_amd as m
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    n = 4096
    g = torch.Generator(device="cuda").manual_seed(6)
    part = torch.randn(n, device="cuda", generator=g).mul_(3).exp().to(dt)
    codes, scales = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty(n, device="cuda")
    back = torch.empty(n, dtype=dt, device="cuda")
    few = m.make_rows(n, 1, dtype=dtype)
    m.moe_checkpoint_rows(few, part, codes, scales)
    m.moe_restore_rows(few, codes, scales, back)
    x = torch.empty(T, dtype=dt, device="cuda")
    all_codes = torch.full((T + 1,), 77, dtype=torch.uint8, device="cuda")
    all_scales = torch.full((T + 1,), 7.0, device="cuda")
    whole = T // n * n

    def copies(a, of):
        return (torch.equal(a[:whole].view(-1, n), of.expand(whole // n, n)) and
                torch.equal(a[whole:T], of[:T - whole]))
    x[:whole].view(-1, n).copy_(part.expand(whole // n, n))
    x[whole:] = part[:T - whole]
    many = m.make_rows(T, 1, dtype=dtype)
    m.moe_checkpoint_rows(many, x, all_codes, all_scales)
    torch.cuda.synchronize()
    assert copies(all_codes, codes) and copies(all_scales, scales)
    assert all_codes[T] == 77 and all_scales[T] == 7.0
    y = torch.full((T + 1,), 9.0, dtype=dt, device="cuda")
    m.moe_restore_rows(many, all_codes, all_scales, y)
    torch.cuda.synchronize()
    assert copies(y, back) and y[T] == 9.0


@pytest.mark.parametrize("C,pad", [(2048, 0), (2001, 2), (1, 0), (130, 6)])
def test_large_float32_calls(C, pad):
    """From 65536 groups on a workgroup takes four runs of them: every row as
    in calls of 64 rows."""
    import torch
    import expert_moe_fp32_amd as m
    n = -(-C // 128)
    T = 65536 // n + 77
    assert T * n >= 65536 and 64 * n < 65536
    x = rows_of(T, C, "f32", pad, C)
    codes, part = (torch.full((T + 1, C), 77, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales, own = (torch.full((T + 1, n), 7.0, device="cuda") for _ in range(2))
    y, back = (torch.full((T + 1, C + pad), 9.0, device="cuda") for _ in range(2))
    d = m.make_rows(T, C, dtype="f32", stride=C + pad)
    m.moe_checkpoint_rows(d, x, codes, scales)
    m.moe_restore_rows(d, codes, scales, y)
    for at in range(0, T, 64):
        d = m.make_rows(min(64, T - at), C, dtype="f32", stride=C + pad)
        m.moe_checkpoint_rows(d, x[at:], part[at:], own[at:])
        m.moe_restore_rows(d, part[at:], own[at:], back[at:])
    torch.cuda.synchronize()
    assert torch.equal(codes, part) and torch.equal(scales, own)
    assert torch.equal(y, back)
    assert (y[:, C:] == 9.0).all() and (y[T] == 9.0).all()
    assert (codes[T] == 77).all() and (scales[T] == 7.0).all()
    some = np.r_[0, T // 3, T - 1]
    rc, rs = ot.checkpoint(x[some, :C].double().cpu().numpy())
    assert np.array_equal(codes[:T].cpu().numpy()[some], rc)
    assert np.array_equal(scales[:T].cpu().numpy()[some], rs)
