"""The gradient norm over many tensors and clipping against the definition in 64
bits on the CPU."""
import math

import pytest
import torch

import layer_reference as ref
import step_reference as step
from gpu_util import dev, say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tide():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixed_precision_rs_amd as t
    return t


def total_of(tide, tensors, **kw):
    total = torch.full((1,), 7.0, dtype=torch.float64, device=dev())
    tide.grad_squares(tensors, total, **kw)
    return total


def odd(t, offset):
    """t on the GPU, `offset` elements into a buffer."""
    b = torch.full((t.numel() + offset + 9,), 3.0, dtype=t.dtype, device=dev())
    v = b[offset: offset + t.numel()].view(t.shape)
    v.copy_(t.to(dev()))
    return v, b


SETS = [[], [(0,)], [(1,)], [(7,), (9,)], [(3, 5), (16384,), (16385,), (0, 4), (1,)], [(100000,)], [(i % 61 + 1,) for i in range(300)],
        [(40000,), (8,), (70001,)]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("which", range(len(SETS)))
def test_squares_and_clip(tide, which, dtype):
    say("clip", which, dtype)
    cpu = [ref.normal(s, dtype, i) for i, s in enumerate(SETS[which])]
    gpu = [odd(t, i % 5)[0] for i, t in enumerate(cpu)]
    want = step.squares(cpu)
    total = total_of(tide, gpu)
    n = sum(t.numel() for t in cpu)
    assert abs(float(total) - want) <= (n + 8) * 2.0 ** -53 * want
    assert abs(float(total_of(tide, gpu, accumulate=True)) - (want + 7.0)) <= (n + 9) * 2.0 ** -53 * (want + 7.0)
    table = tide.TensorTable(gpu)
    assert torch.equal(total_of(tide, table), total)
    for most in (0.0, 0.3 * math.sqrt(want), math.sqrt(float(total)), 10.0 + math.sqrt(want), math.inf):
        outs = [odd(torch.full_like(t, 5.0), (i + 2) % 7) for i, t in enumerate(cpu)]
        norm = torch.empty(1, device=dev())
        tide.clip_grads(table, total, most, out=[o for o, _ in outs], norm=norm)
        assert abs(float(norm) - math.sqrt(want)) <= 2 * step.U * math.sqrt(want)
        for i, (t, (o, whole)) in enumerate(zip(cpu, outs)):
            v, lim = step.clipped(t, float(total), most)
            ref.close(o, v, lim + (step.HALF[dtype] * v.abs() if dtype is BF16 else 0.0), "clipped")
            if most >= math.sqrt(float(total)):
                assert torch.equal(o.cpu(), t)
            off = (i + 2) % 7
            assert (whole[:off] == 3.0).all() and (whole[off + t.numel():] == 3.0).all()
        place = [odd(t, i % 5)[0] for i, t in enumerate(cpu)]
        tide.clip_grads(place, total, most)
        assert all(torch.equal(a, b) for a, (b, _) in zip(place, outs))
    assert all(torch.equal(a.cpu(), b) for a, b in zip(gpu, cpu))


def test_one_tensor_and_two_types(tide):
    a, b = ref.normal((33, 70), BF16, 1), ref.normal((500,), F32, 2)
    total = total_of(tide, a.to(dev()))
    tide.grad_squares([b.to(dev())], total, accumulate=True)
    want = step.squares([a, b])
    assert abs(float(total) - want) <= 3000 * 2.0 ** -53 * want


def test_squares_beyond_fp32(tide):
    """Squares that fp32 could not hold: 1e30 and 1e-30, subnormals; the norm is
    right and the clipped tensors are what a wider type would give."""
    for value in (1e30, 3e38, 1e-30, 1e-42):
        t = torch.full((1000,), value)
        total = total_of(tide, [t.to(dev())])
        want = step.squares([t])
        assert abs(float(total) - want) <= 1010 * 2.0 ** -53 * want and want > 0
        out, norm = torch.empty(1000, device=dev()), torch.empty(1, device=dev())
        most = 0.25 * math.sqrt(want)
        tide.clip_grads([t.to(dev())], total, most, out=[out], norm=norm)
        v, lim = step.clipped(t, float(total), most)
        ref.close(out, v, lim, "clipped %g" % value)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_norms_that_are_not_finite(tide, bad):
    t = ref.normal((20000,), F32, 1)
    t[15000] = bad
    g = t.to(dev())
    total = total_of(tide, [g])
    assert not math.isfinite(float(total))
    norm, out = torch.zeros(1, device=dev()), torch.zeros(20000, device=dev())
    tide.clip_grads([g], total, 1.0, norm=norm)
    tide.clip_grads([g], total, 1.0, out=[out])
    assert not math.isfinite(float(norm))
    for r in (g, out):
        assert torch.equal(r.cpu().nan_to_num(9.0, 8.0, 7.0), t.nan_to_num(9.0, 8.0, 7.0))   # left as they were
    zero = total_of(tide, [torch.zeros(10, device=dev())])
    assert float(zero) == 0.0
    z = torch.zeros(10, device=dev())
    tide.clip_grads([z], zero, 0.0)
    assert not z.any()


def test_many_tiles_and_the_same_bits(tide):
    """More tiles than workgroups, more tensors than one launch takes."""
    g = torch.Generator(device=dev()).manual_seed(1)
    big = torch.randn(50_000_001, generator=g, device=dev(), dtype=BF16)
    parts = list(big.split(123_457))
    a, b = total_of(tide, parts), total_of(tide, parts)
    need = tide.grad_squares_workspace_bytes(parts)
    c = total_of(tide, parts, workspace=torch.full((need,), 255, dtype=torch.uint8, device=dev()))
    assert torch.equal(a, b) and torch.equal(a, c)
    want = float((big.double() ** 2).sum())
    assert abs(float(a) - want) <= 1e-9 * want
    out = torch.empty_like(big)
    tide.clip_grads(parts, a, 100.0, out=list(out.split(123_457)))
    f = 100.0 / math.sqrt(float(a))
    # fp64 product to fp32 to bf16, as torch rounds it
    assert torch.equal(out, (big.double() * f).float().to(BF16))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_tensors_that_pass_the_caches(tide, dtype):
    """Over 192 MiB in all, into outputs and in place, tensors at odd elements."""
    g = torch.Generator(device=dev()).manual_seed(3)
    n = (200 << 20) // dtype.itemsize
    big = torch.randn(n + 9, generator=g, device=dev(), dtype=dtype)
    sizes = [n // 3 + 1, 5, n // 7, 16384, n - n // 3 - n // 7 - 16384 - 6]
    parts = list(big[3: n + 3].split(sizes))
    total = total_of(tide, parts)
    want = float((big[3: n + 3].double() ** 2).sum())
    assert abs(float(total) - want) <= 2 * (n + 8) * 2.0 ** -53 * want           # both sums
    out = torch.full((n + 9,), 3.0, dtype=dtype, device=dev())
    tide.clip_grads(parts, total, 100.0, out=list(out[1: n + 1].split(sizes)))
    clipped = (big.double() * (100.0 / math.sqrt(float(total)))).float().to(dtype)
    assert torch.equal(out[1: n + 1], clipped[3: n + 3]) and (out[:1] == 3.0).all() and (out[n + 1:] == 3.0).all()
    edges = big[:3].clone(), big[n + 3:].clone()
    tide.clip_grads(parts, total, 100.0)
    assert torch.equal(big[3: n + 3], clipped[3: n + 3]) and torch.equal(big[:3], edges[0]) and torch.equal(big[n + 3:], edges[1])


def test_tensor_past_two_gib(tide):
    n = (1 << 31) + 100
    t = torch.zeros(n, dtype=BF16, device=dev())
    t[0], t[1 << 31], t[n - 1] = 3.0, 4.0, 12.0
    total = total_of(tide, [t])
    assert float(total) == 169.0
    tide.clip_grads([t], total, 6.5)
    assert float(t[0]) == 1.5 and float(t[1 << 31]) == 2.0 and float(t[n - 1]) == 6.0
