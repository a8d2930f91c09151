"""Activation checkpoints in 8 bits and the gated activation over them, against
the definition in 64 bits on the CPU."""
import numpy as np
import pytest
import torch

import layer_reference as ref
from gpu_util import dev, say

pytestmark = pytest.mark.gpu
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
SHAPES = [(1, 1), (1, 31), (2, 32), (3, 33), (1, 64), (5, 100), (7, 256), (9, 257), (64, 2048),
          (33, 2049), (4, 8191), (2, 70000), (1000, 40), (0, 64), (3, 0)]


@pytest.fixture(scope="module")
def tide():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixed_precision_rs_amd as t
    return t


def window(t, pad, fill=0.0):
    """t on the GPU, as a window of a buffer whose rows are `pad` wider."""
    b = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=torch.float32).to(t.dtype).to(dev())
    w = b[:, pad // 2: pad // 2 + t.shape[1]]
    w.copy_(t.to(dev()))
    return w


def empty_saved(n, D, pad=0, fill=0x5A):
    c = torch.full((n, D + pad), fill, dtype=torch.uint8, device=dev()).view(E4M3)
    s = torch.full((n, -(-D // 32) + pad), fill, dtype=torch.uint8, device=dev()).view(E8M0)
    return c[:, pad // 2: pad // 2 + D], s[:, pad // 2: pad // 2 + -(-D // 32)], c, s


def untouched(whole, lo, n, fill=0x5A):
    b = whole.view(torch.uint8).cpu()
    return bool((b[:, :lo] == fill).all() and (b[:, lo + n:] == fill).all())


def same_saved(got, x, what):
    q, e = ref.pack(x)
    assert np.array_equal(got[1].cpu().view(torch.uint8).numpy().astype(np.int64) - 127, e), what
    c = got[0].cpu().float().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(c), np.isnan(q)), what
    assert np.array_equal(c[~np.isnan(c)], q[~np.isnan(q)]), what


def wide_values(n, D, dtype, seed):
    """Magnitudes over many powers of two, ties of the rounding, zeros, borders of the scale."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, D, generator=g) * torch.exp2(torch.randint(-12, 12, (n, D), generator=g).float())
    x *= torch.exp2(torch.randint(-60, 60, (n, 1), generator=g).float())
    flat = x.view(-1)
    if flat.numel():
        flat[::7] = torch.sign(flat[::7]) * torch.exp2(torch.floor(torch.log2(flat[::7].abs() + 1e-30))) * 1.0625
        flat[::11] = 0.0
        flat[::13] = 448.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("n,D", SHAPES)
def test_pack_and_unpack(tide, n, D, pad, dtype):
    say("pack", n, D, pad, dtype)
    x = wide_values(n, D, dtype, seed=n + D)
    codes, scales, wc, ws = empty_saved(n, D, pad)
    tide.checkpoint_pack(window(x, pad), (codes, scales))
    same_saved((codes, scales), x, "pack")
    assert untouched(wc, pad // 2, D) and untouched(ws, pad // 2, -(-D // 32))
    for out_t in (torch.bfloat16, torch.float32):
        whole = torch.full((n, D + pad), -3.0, dtype=out_t, device=dev())
        out = whole[:, pad // 2: pad // 2 + D]
        tide.checkpoint_unpack((codes, scales), out)
        ref.close(out, ref.unpack(codes.cpu(), scales.cpu()), 0.0, "unpack")       # exact
        if pad:
            w = whole.cpu()
            assert (w[:, : pad // 2] == -3.0).all() and (w[:, pad // 2 + D:] == -3.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pack_every_bf16_value(tide, dtype):
    """Each of the 65536 bf16 values alone in its block (the other elements 0),
    and beside a block maximum of its own magnitude's neighbours."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = torch.zeros(65536, 32, dtype=dtype)
    x[:, 9] = bits.view(torch.bfloat16).to(dtype)
    codes, scales, _, _ = empty_saved(65536, 32)
    tide.checkpoint_pack(x.to(dev()), (codes, scales))
    same_saved((codes, scales), x, "alone")
    x = bits.view(torch.bfloat16).to(dtype).view(2048, 32).contiguous()
    codes, scales, _, _ = empty_saved(2048, 32)
    tide.checkpoint_pack(x.to(dev()), (codes, scales))
    same_saved((codes, scales), x, "in order")


def test_pack_fp32_near_the_codes_borders(tide):
    """fp32 values one step either side of every rounding border and of the scale's."""
    q = torch.arange(0, 0x7F, dtype=torch.uint8).view(E4M3).double()
    mid = ((q[1:] + q[:-1]) / 2).float()
    v = torch.cat([mid, torch.nextafter(mid, torch.tensor(1e9)), torch.nextafter(mid, torch.tensor(0.0)),
                   torch.tensor([447.99997, 448.0])])
    x = torch.zeros(v.numel(), 32)
    x[:, 0] = 448.0                                     # the scale is 1
    x[:, 17] = v
    x[:, 30] = -v
    y = torch.zeros(3, 32)
    y[:, 2] = torch.tensor([448.0, 448.00003, 447.99997])
    for t in (x, y):
        codes, scales, _, _ = empty_saved(t.shape[0], 32)
        tide.checkpoint_pack(t.to(dev()), (codes, scales))
        same_saved((codes, scales), t, "borders")


def test_not_finite_values(tide):
    x = ref.normal((6, 96), torch.float32, seed=1)
    x[0, 3] = float("nan")
    x[1, 40] = float("inf")
    x[2, 70] = -float("inf")
    x[3, :32] = float("nan")
    x[4, 5] = 3.4e38
    x[5, :] = 1e-45
    codes, scales, _, _ = empty_saved(6, 96)
    tide.checkpoint_pack(x.to(dev()), (codes, scales))
    same_saved((codes, scales), x, "not finite")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("n,D", SHAPES)
def test_gated_forward(tide, n, D, pad, dtype):
    say("gated", n, D, pad, dtype)
    g, u = ref.normal((n, D), dtype, seed=1, scale=4.0), ref.normal((n, D), dtype, seed=2)
    gd, ud = window(g, pad), window(u, pad)
    want = ref.gated(g, u)
    # exp within 2^-22, the sigmoid 2^-22 more, three products and quotients: under 2^-20 of the value
    bound = (ref.HALF[dtype] + 2.0 ** -20) * want.abs()
    for save in ("none", "gate", "both"):
        whole = torch.full((n, D + pad), -3.0, dtype=dtype, device=dev())
        out = whole[:, pad // 2: pad // 2 + D]
        a, b = empty_saved(n, D, pad), empty_saved(n, D, pad)
        tide.gated_silu(gd, ud, out, gate_saved=a[:2] if save != "none" else None,
                        up_saved=b[:2] if save == "both" else None)
        ref.close(out, want, bound, "gated")
        w = whole.cpu()
        assert (w[:, : pad // 2] == -3.0).all() and (w[:, pad // 2 + D:] == -3.0).all()
        if save != "none":
            same_saved(a, g, "gate_saved")
        if save == "both":
            same_saved(b, u, "up_saved")
        assert untouched(a[2], pad // 2, D) and untouched(b[2], pad // 2, D)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("n,D", SHAPES)
def test_gated_gradient(tide, n, D, pad, dtype):
    say("gated_grad", n, D, pad, dtype)
    d = ref.normal((n, D), dtype, seed=3)
    gs = ref.saved_of(ref.normal((n, D), torch.float32, seed=1, scale=4.0))
    us = ref.saved_of(ref.normal((n, D), torch.float32, seed=2))
    dg, du, h, mag = ref.gated_grad(d, ref.unpack(*gs), ref.unpack(*us))
    put = lambda s: tuple(t.to(dev()) for t in s)  # noqa: E731
    outs = [torch.full((n, D + pad), -3.0, dtype=dtype, device=dev()) for _ in range(3)]
    views = [t[:, pad // 2: pad // 2 + D] for t in outs]
    tide.gated_silu_grad(window(d, pad), put(gs), put(us), views[0], views[1], out=views[2])
    half = ref.HALF[dtype]
    ref.close(views[0], dg, half * dg.abs() + 2.0 ** -20 * mag, "dgate")   # the two terms may cancel
    ref.close(views[1], du, (half + 2.0 ** -20) * du.abs(), "dup")
    ref.close(views[2], h, (half + 2.0 ** -20) * h.abs(), "out")
    for t in outs:
        w = t.cpu()
        assert (w[:, : pad // 2] == -3.0).all() and (w[:, pad // 2 + D:] == -3.0).all()
    a, b = torch.empty_like(views[0]), torch.empty_like(views[1])
    tide.gated_silu_grad(window(d, pad), put(gs), put(us), a, b)
    assert torch.equal(a, views[0]) and torch.equal(b, views[1])


def test_gated_gradient_by_differences(tide):
    """Central differences of the forward call, at values that a checkpoint holds exactly."""
    g = torch.tensor([[-6.0, -2.0, -1.25, -0.5, 0.0, 0.5, 1.25, 2.0, 6.0, 16.0]], device=dev())
    u = torch.full_like(g, 1.5)
    gs, us = empty_saved(1, 10)[:2], empty_saved(1, 10)[:2]
    out = torch.empty_like(g)
    tide.gated_silu(g, u, out, gate_saved=gs, up_saved=us)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    tide.gated_silu_grad(torch.ones_like(g), gs, us, dg, du)
    h = 2.0 ** -5

    def f(g, u):
        o = torch.empty_like(g)
        tide.gated_silu(g, u, o)
        return o.double()

    # |third derivative of silu| < 1, so the difference is off by 1.5 h^2 / 6, and by the
    # forward's 2^-19 * |silu u| <= 24 * 2^-19 over 2 h
    tol = 1.5 * h * h / 6 + 24 * 2.0 ** -19 / h
    assert (((f(g + h, u) - f(g - h, u)) / (2 * h) - dg.double()).abs() < tol).all()
    assert (((f(g, u + h) - f(g, u - h)) / (2 * h) - du.double()).abs() < tol).all()


def test_gated_extremes(tide):
    """Large gates of both signs, infinities and NaN follow the formula."""
    inf = float("inf")
    g = torch.tensor([[-1e4, -88.0, -90.0, 88.0, 1e4, 0.0, float("nan"), 2.0, inf, -inf, inf, 3e38, -3e38]])
    u = torch.tensor([[1.0, 1.0, 2.0, 1.0, 3.0, 5.0, 1.0, inf, 2.0, 1.0, 0.0, 0.5, 1.0]])
    out = torch.empty_like(g, device=dev())
    tide.gated_silu(g.to(dev()), u.to(dev()), out)
    want = ref.gated(g, u)
    ref.close(out, want, 2.0 ** -20 * torch.nan_to_num(want, 0, 0, 0).abs() + 2.0 ** -126, "extremes")


def test_halves_of_one_tensor(tide):
    """gate and up, and their gradients, as the two halves of one wide tensor."""
    n, F = 37, 104
    gu = ref.normal((n, 2 * F), torch.bfloat16, seed=9)
    d = gu.to(dev())
    gs, us = empty_saved(n, F)[:2], empty_saved(n, F)[:2]
    out = torch.empty(n, F, dtype=torch.bfloat16, device=dev())
    tide.gated_silu(d[:, :F], d[:, F:], out, gate_saved=gs, up_saved=us)
    want = ref.gated(gu[:, :F], gu[:, F:])
    ref.close(out, want, (2.0 ** -8 + 2.0 ** -20) * want.abs())
    dgu = torch.empty(n, 2 * F, dtype=torch.bfloat16, device=dev())
    tide.gated_silu_grad(out, gs, us, dgu[:, :F], dgu[:, F:])
    dg, du, _, mag = ref.gated_grad(out.cpu(), ref.unpack(*(t.cpu() for t in gs)), ref.unpack(*(t.cpu() for t in us)))
    ref.close(dgu[:, :F], dg, 2.0 ** -8 * dg.abs() + 2.0 ** -20 * mag)
    ref.close(dgu[:, F:], du, (2.0 ** -8 + 2.0 ** -20) * du.abs())


def test_rows_past_32_bit_offsets(tide):
    n, D, stride = 2100, 96, 1 << 21
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GiB of GPU memory")
    x = ref.normal((n, D), torch.bfloat16, seed=4)
    wide = torch.empty(n, stride, dtype=torch.bfloat16, device=dev())
    v = wide[:, 7: 7 + D]
    v.copy_(x.to(dev()))
    codes = torch.empty(n, stride, dtype=torch.uint8, device=dev()).view(E4M3)[:, 3: 3 + D]
    scales = torch.empty(n, 3, dtype=torch.uint8, device=dev()).view(E8M0)
    tide.checkpoint_pack(v, (codes, scales))
    same_saved((codes, scales), x, "far rows")
    tide.checkpoint_unpack((codes, scales), v)
    ref.close(v, ref.unpack(codes.cpu(), scales.cpu()), 0.0)
