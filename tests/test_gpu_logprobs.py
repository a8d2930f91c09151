"""Log probabilities, entropy and alternatives, and the gradient to the logits,
against the definition in 64 bits on the CPU."""
import math

import pytest
import torch

import layer_reference as ref
import step_reference as step
from gpu_util import dev, say

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module")
def tide():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixed_precision_rs_amd as t
    return t


def window(t, pad, fill=NAN):
    b = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=torch.float32).to(t.dtype).to(dev())
    w = b[:, pad // 2: pad // 2 + t.shape[1]]
    w.copy_(t.to(dev()))
    return w


def run(tide, x, targets, top=0, pad=0, **kw):
    T = x.shape[0]
    f = lambda *s: torch.full(s, 55.0, device=dev())  # noqa: E731
    got = {"logprob": f(T), "stats": f(T, 2), "entropy": f(T)}
    if top:
        got.update(top_ids=torch.full((T, top), 55, dtype=torch.int32, device=dev()), top_logprobs=f(T, top))
    tide.token_logprobs(window(x, pad), targets.to(dev()), **got, **kw)
    return got


def check(got, want, top, what):
    ref.close(got["logprob"], want["logprob"], want["d_logprob"], what + " logprob")
    bad = torch.isnan(want["log_s"])
    ref.close(got["stats"][:, 1], want["log_s"], want["d_log_s"], what + " log s")
    assert torch.equal(got["stats"][:, 0].cpu()[~bad].double(), want["m"][~bad]), what
    ref.close(got["entropy"], want["entropy"], want["d_entropy"], what + " entropy")
    if top:
        assert torch.equal(got["top_ids"].cpu(), want["top_ids"]), what
        ref.close(got["top_logprobs"], want["top_logprobs"], want["d_top"], what + " alternatives")


def some_targets(T, V, seed, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, max(V, 1), (T,), generator=g)
    t[::5] = -100
    if T > 3:
        t[3] = V
    if T > 8 and dtype == torch.int64:
        t[8] = 2 ** 33
    return t.to(dtype)


SHAPES = [(1, 1, 1), (2, 3, 5), (3, 7, 2), (4, 8, 0), (9, 64, 8), (5, 65, 32), (11, 1000, 20), (3, 2047, 7), (2, 2048, 1),
          (6, 8193, 3), (3, 50001, 20), (2, 131072, 8), (0, 10, 2), (3, 0, 2)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("T,V,top", SHAPES)
def test_forward(tide, T, V, top, pad, dtype):
    say("logprobs", T, V, top, pad, dtype)
    x = ref.normal((T, V), dtype, T + V, 3.0)
    targets = some_targets(T, V, V, torch.int32 if pad else torch.int64)
    if V == 0:
        targets = targets.clamp(max=-1)
    check(run(tide, x, targets, top, pad), step.logprobs(x, targets, top), top, "normal")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [5, 300, 9000])
def test_rows_of_masks_infinities_and_nan(tide, V, dtype):
    g = torch.Generator().manual_seed(V)
    low = torch.finfo(dtype).min
    x = torch.randn(14, V, generator=g)
    x[0] = -INF                                         # nothing is left
    x[1, : V - 2] = -INF
    x[2] = low
    x[3, 1:] = low
    x[4, V // 2] = NAN
    x[5, V - 1] = INF
    x[6] = INF
    x[7, 0] = torch.finfo(dtype).max
    x[8] = -INF
    x[8, V - 1] = -3.0
    x[9] = NAN
    x[10] = x[10] * 1e30
    x[11, ::2] = -INF
    x[12] = 4.0                                         # all equal
    x[13] = torch.randint(-2, 3, (V,), generator=g).float()   # many equal
    x = x.to(dtype)
    targets = torch.randint(0, V, (14,), generator=g)
    for t in (targets, torch.full((14,), V - 1), torch.full((14,), -1)):
        check(run(tide, x, t, 6), step.logprobs(x, t, 6), 6, "odd rows")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_alternatives_that_one_lane_or_one_stretch_holds(tide, dtype):
    """The largest logits side by side, at every multiple of a power of two, rising
    and falling through the row, or all equal: whatever share of a row a lane has,
    one of these puts more alternatives into it than others hold."""
    V, top = 40000, 32
    rows = []
    for stride in (1, 2, 4, 8, 16, 32, 64, 128, 256, 512, 1024, 2048, 4096, 8192):
        x = torch.zeros(V)
        at = torch.arange(0, V, stride)[:40]
        x[at] = 5.0 + torch.arange(len(at)).float() % 7
        rows.append(x)
    rows += [torch.linspace(-4, 4, V), torch.linspace(4, -4, V), torch.zeros(V), torch.full((V,), -INF)]
    rows[-1][V - 20:] = 1.0
    for lanes in (64, 256, 512, 1024):                   # one lane's vectors rise, all others are low
        x = torch.full((V,), -9.0)
        n = 16 // dtype.itemsize
        for i, u in enumerate(range(3, V // n, lanes)):
            x[u * n: u * n + n] = torch.arange(n).float() / 8 + i % 3
        rows.append(x)
    x = torch.stack(rows).to(dtype)
    t = torch.arange(len(rows))
    want = step.logprobs(x, t, top)
    for times in (1, 7, 13, 24, 48):                     # few rows are split, more have a workgroup each, of fewer threads
        got = run(tide, x.repeat(times, 1), t.repeat(times), top)
        first = {k: v[: len(rows)] for k, v in got.items()}
        check(first, want, top, "stretches")
        for k, v in got.items():
            assert torch.equal(v, first[k].repeat(times, *[1] * (v.dim() - 1))), k


@pytest.mark.parametrize("T", [3, 70, 300, 600])
def test_more_candidates_than_are_ranked_at_once(tide, T):
    """A lane whose whole share of a long row is ahead of all others', and 32 of them,
    for every number of lanes that a row may have."""
    V, top, n = 262144, 32, 8
    u = torch.arange(V) // n
    for lanes in (256, 512, 1024):
        one = torch.full((V,), -9.0)
        mine = u % lanes == 5
        one[mine] = (torch.arange(V)[mine] % 97).float() / 8
        many = torch.where((u % lanes % (lanes // 64) == 0) & (u % lanes < lanes // 2), 1.0 + (u % lanes) // (lanes // 64), -9.0)
        for row in (one, many):
            x = row.to(BF16)
            want = torch.sort(x.float(), descending=True, stable=True)
            got = run(tide, x.expand(T, V).contiguous(), torch.arange(T), top)
            assert (got["top_ids"].cpu() == want.indices[:top].int()).all()
            log_s = torch.logsumexp(x.double(), 0)
            room = (V / 16 + 30 + 5 * 42 + 8 * 50) * step.U          # the reference's: logits from -9 to 33, log s below 50
            ref.close(got["top_logprobs"], (want.values[:top].double() - log_s).expand(T, top), room, "many")


def test_outputs_left_out(tide):
    x, t = ref.normal((5, 777), BF16, 1), some_targets(5, 777, 1)
    full = run(tide, x, t, 4)
    lp = torch.empty(5, device=dev())
    tide.token_logprobs(x.to(dev()), t.to(dev()), lp)
    assert torch.equal(lp, full["logprob"])
    again = run(tide, x, t, 4)
    assert all(torch.equal(full[k], again[k]) for k in full)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("top", [0, 7])
@pytest.mark.parametrize("T,V", [(3, 50001), (3, 600), (1100, 2100), (600, 4200), (300, 8300), (70, 16500)])
def test_without_entropy(tide, T, V, top, dtype):
    """Rows in parts, and by workgroups of 64 to 1024 threads, whose entropy is not asked for."""
    say("without entropy", T, V, top, dtype)
    x = ref.normal((3, V), dtype, V, 3.0)
    x[1, : V - 5] = -INF                                # fewer than `top` are left
    x[2, V // 2] = INF if top else NAN
    t = torch.tensor([V - 1, V - 3, -100])
    rows = torch.arange(T) % 3
    f = lambda *s: torch.full(s, 55.0, device=dev())  # noqa: E731
    got = {"logprob": f(T), "stats": f(T, 2)}
    if top:
        got.update(top_ids=torch.full((T, top), 55, dtype=torch.int32, device=dev()), top_logprobs=f(T, top))
    tide.token_logprobs(x[rows].to(dev()), t[rows].to(dev()), **got)
    want = {k: v[rows] for k, v in step.logprobs(x, t, top).items()}
    check({**got, "entropy": want["entropy"]}, want, top, "without entropy")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("T,V", [(1, 1), (2, 3), (9, 64), (5, 65), (11, 1000), (3, 2047), (2, 50001), (0, 8), (3, 0)])
def test_gradient(tide, T, V, pad, dtype):
    say("logprobs gradient", T, V, pad, dtype)
    x = ref.normal((T, V), dtype, T + V, 3.0)
    targets = some_targets(T, V, V, torch.int32 if pad else torch.int64)
    if V == 0:
        targets = targets.clamp(max=-1)
    got = run(tide, x, targets)
    d, h = ref.normal((T,), F32, 3), ref.normal((T,), F32, 4)
    d[::5] = NAN                                        # those rows' targets do not count
    for with_h in (False, True):
        kw = {"entropy": got["entropy"], "dentropy": h.to(dev())} if with_h else {}
        want, lim = step.logprobs_grad(x, targets, got["stats"].cpu(), d, got["entropy"].cpu(), h if with_h else None)
        lim = lim + (step.HALF[dtype] + 2 * step.U) * want.abs()
        whole = torch.full((T, V + pad), 3.0, dtype=dtype, device=dev())
        dx = whole[:, pad // 2: pad // 2 + V]
        tide.token_logprobs_grad(window(x, pad), targets.to(dev()), got["stats"], d.to(dev()), dx, **kw)
        ref.close(dx, want, lim, "gradient")
        if pad:
            w = whole.cpu()
            assert (w[:, : pad // 2] == 3.0).all() and (w[:, pad // 2 + V:] == 3.0).all()
        place = window(x, pad)
        tide.token_logprobs_grad(place, targets.to(dev()), got["stats"], d.to(dev()), place, **kw)
        assert torch.equal(place, dx), "in place"


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient_of_masked_rows(tide, dtype):
    V = 300
    x = ref.normal((6, V), F32, 1)
    x[0] = -INF
    x[1, 7:] = -INF
    x[2] = torch.finfo(dtype).min
    x[3, ::2] = -INF
    x = x.to(dtype)
    t = torch.tensor([3, 2, 9, 1, 5, -1])
    got = run(tide, x, t)
    d, h = ref.normal((6,), F32, 3), ref.normal((6,), F32, 4)
    want, lim = step.logprobs_grad(x, t, got["stats"].cpu(), d, got["entropy"].cpu(), h)
    dx = torch.empty(6, V, dtype=dtype, device=dev())
    tide.token_logprobs_grad(x.to(dev()), t.to(dev()), got["stats"], d.to(dev()), dx, entropy=got["entropy"], dentropy=h.to(dev()))
    ref.close(dx, want, lim + (step.HALF[dtype] + 2 * step.U) * want.abs(), "masked")
    assert not dx[0].any()
    x = ref.normal((3, V), F32, 1)
    x[0, 5], x[1, 6] = NAN, INF
    got = run(tide, x, t[1:4])
    dx = torch.empty(3, V, device=dev())
    tide.token_logprobs_grad(x.to(dev()), t[1:4].to(dev()), got["stats"], d[:3].to(dev()), dx)
    assert torch.isnan(dx[:2]).all() and torch.isfinite(dx[2]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [300, 9001])
@pytest.mark.parametrize("shift", [40, -40, 300, -300, 5000, -5000, 60000, -60000, 70000])
def test_rows_far_from_zero(tide, shift, V, dtype):
    """A constant added to a row changes neither its probabilities nor what their
    error may be: each row moved by about `shift`, some of them confident, where the
    target's gradient is d (1 - p), a difference of nearly equal numbers."""
    say("far from zero", shift, V, dtype)
    T = 8
    x = ref.normal((T, V), F32, V, 3.0) + shift
    t = torch.tensor([3, V - 1, 0, 17, V // 2, -1, 5, 250])
    for r, above in ((0, 14.0), (1, 25.0), (4, 18.0), (6, 60.0)):
        x[r, t[r]] = x[r].max() + above
    x[7, ::3] = -INF
    x = x.to(dtype)
    got = run(tide, x, t, 4)
    check(got, step.logprobs(x, t, 4), 4, "far")
    d, h = 1 + ref.normal((T,), F32, 3).abs(), ref.normal((T,), F32, 4)
    for with_h in (False, True):
        kw = {"entropy": got["entropy"], "dentropy": h.to(dev())} if with_h else {}
        want, lim = step.logprobs_grad(x, t, got["stats"].cpu(), d, got["entropy"].cpu(), h if with_h else None)
        # p is the product of 2^q and a factor within 2^(2^-8) of 1; the instruction gives 0 for a 2^q below 2^-126.
        # So p is off by up to 2^-125 besides, and p (lp + H), where p is that small and lp from -88 on falling, by
        # 2^-125 (88 + |H|).
        tiny = d + (h.abs() * (88 + got["entropy"].cpu().abs()) if with_h else 0.0)
        lim = lim + (step.HALF[dtype] + 2 * step.U) * want.abs() + 2.0 ** -125 * tiny.double()[:, None]
        dx = torch.empty(T, V, dtype=dtype, device=dev())
        tide.token_logprobs_grad(x.to(dev()), t.to(dev()), got["stats"], d.to(dev()), dx, **kw)
        ref.close(dx, want, lim, "gradient")


def test_gradient_against_differences(tide):
    """sum_t d_t logprob_t + h_t entropy_t at logits a step apart, in 64 bits."""
    T, V, eps = 4, 60, 1e-5
    x, t = ref.normal((T, V), F32, 5, 2.0), torch.tensor([3, 59, -1, 0])
    d, h = ref.normal((T,), F32, 6), ref.normal((T,), F32, 7)

    def value(y):
        lp = torch.log_softmax(y, 1)
        at = torch.where(t >= 0, t, 0)
        return (torch.where(t >= 0, lp.gather(1, at[:, None])[:, 0], 0.0) * d.double()).sum() - (lp.exp() * lp).sum(1) @ h.double()

    got = run(tide, x, t)
    dx = torch.empty(T, V, device=dev())
    tide.token_logprobs_grad(x.to(dev()), t.to(dev()), got["stats"], d.to(dev()), dx, entropy=got["entropy"], dentropy=h.to(dev()))
    for r, c in ((0, 3), (0, 10), (1, 59), (2, 7), (3, 0), (3, 30)):
        up, down = x.double().clone(), x.double().clone()
        up[r, c] += eps
        down[r, c] -= eps
        diff = float(value(up) - value(down)) / (2 * eps)
        # the third derivative times eps^2 is below 1e-9, fp32 inputs of the gradient are off by 1e-6
        assert abs(float(dx[r, c]) - diff) < 2e-5 * (1 + float(d[r].abs() + h[r].abs())), (r, c)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V,times", [(700, 1), (700, 1000), (9000, 50), (40000, 1), (40000, 20), (40000, 100)])
def test_nan_of_every_kind_is_no_alternative(tide, V, times, dtype):
    """Quiet and signalling NaN of both signs beside the largest logits: the row's log
    probabilities are NaN, its alternatives all others."""
    bits, kind = ([0x7FC0, 0x7F81, 0xFFC0, 0xFF81, 0x7FFF], torch.int16) if dtype is BF16 else (
        [0x7FC00000, 0x7F800001, 0xFFC00000, 0xFF800001, 0x7FFFFFFF], torch.int32)
    wrap = 1 << (8 * dtype.itemsize)
    say("NaN of every kind", V, times, dtype)
    top = 32
    x = ref.normal((len(bits), V), dtype, 5, 3.0)
    for r, b in enumerate(bits):
        x[r, 16:48] = 30.0 + torch.arange(32).to(dtype)
        x.view(kind)[r, 16:48:3] = b if b < wrap // 2 else b - wrap
    assert torch.isnan(x[:, 16:48:3]).all()
    got = run(tide, x.repeat(times, 1), torch.full((len(bits) * times,), 17), top)
    want = torch.sort(torch.where(torch.isnan(x), -INF, x.float()), dim=1, descending=True, stable=True).indices[:, :top].int()
    assert torch.equal(got["top_ids"].cpu(), want.repeat(times, 1))
    assert all(torch.isnan(got[k]).all() for k in ("logprob", "entropy", "top_logprobs")) and torch.isnan(got["stats"][:, 1]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_rows_than_workgroups(tide, dtype):
    """Over 2^20 rows that repeat 1009: the bits of those alone."""
    T, V, top = (1 << 20) + 4099, 19, 3
    x, t = ref.normal((1009, V), dtype, 1, 3.0), some_targets(1009, V, 2)
    few = run(tide, x, t, top)
    check(few, step.logprobs(x, t, top), top, "few")
    at = torch.arange(T, device=dev()) % 1009
    x, t = x.to(dev()), t.to(dev())
    got = run(tide, x[at], t[at], top)
    for k, v in got.items():
        assert torch.equal(v, few[k][at]), k
    d = ref.normal((1009,), F32, 3).to(dev())
    one, dx = torch.empty_like(x), x[at]
    tide.token_logprobs_grad(x, t, few["stats"], d, one, entropy=few["entropy"], dentropy=d)
    tide.token_logprobs_grad(dx, t[at], got["stats"], d[at], dx, entropy=got["entropy"], dentropy=d[at])
    assert torch.equal(dx, one[at])


def test_rows_past_two_gib(tide):
    T, V = 9, 1 << 28
    x = torch.zeros(T, V, dtype=BF16, device=dev())
    x[8, V - 1], x[8, 3] = 21.0, 20.5
    t = torch.full((T,), V - 1, device=dev())
    lp, st, H = (torch.empty(s, device=dev()) for s in ((T,), (T, 2), (T,)))
    ids, tops = torch.empty(T, 2, dtype=torch.int32, device=dev()), torch.empty(T, 2, device=dev())
    tide.token_logprobs(x, t, lp, stats=st, entropy=H, top_ids=ids, top_logprobs=tops)
    s8 = 1 + math.exp(-0.5) + (V - 2) * math.exp(-21.0)
    room = (V / 16 + 30) * step.U                        # the reference's bound; here most of it is the sum of equal terms
    assert ids[8].tolist() == [V - 1, 3] and ids[7].tolist() == [0, 1]
    assert abs(float(lp[8]) + math.log(s8)) < 1e-3 and abs(float(lp[0]) + math.log(V)) < min(room, 1e-3)
    d = torch.ones(T, device=dev())
    tide.token_logprobs_grad(x, t, st, d, x)
    assert abs(float(x[8, V - 1]) - (1 - 1 / s8)) < 2 ** -8 and abs(float(x[8, 3]) + math.exp(-0.5) / s8) < 2 ** -8
