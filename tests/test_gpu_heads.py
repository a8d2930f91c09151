"""Norm and rotation of queries and keys and the gradient, against the definition
in 64 bits on the CPU."""
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


def tables(rows, pairs, pad=0):
    a = torch.arange(rows, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))
    return torch.cos(a).float(), torch.sin(a).float()


def in_rows(t, pad):
    """(rows, n) on the GPU as a window of wider rows."""
    b = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), device=dev())
    w = b[:, pad // 2: pad // 2 + t.shape[1]]
    w.copy_(t.to(dev()))
    return w


class Case:
    """q and k as windows of a fused projection's rows (layout "fused"), each
    contiguous ("apart"), or head by head ("heads first")."""

    def __init__(self, T, Hq, Hk, D, pairs, adjacent, dtype, layout="fused", seed=0, weights=True, rows=37, ids=torch.int64):
        self.dims, self.dtype, self.layout, self.adjacent = (T, Hq, Hk, D), dtype, layout, adjacent
        self.q, self.k = ref.normal((T, Hq, D), dtype, seed, 2.0), ref.normal((T, Hk, D), dtype, seed + 1, 0.5)
        self.dqo, self.dko = ref.normal((T, Hq, D), dtype, seed + 2), ref.normal((T, Hk, D), dtype, seed + 3)
        self.qw = self.kw = None
        if weights:
            self.qw, self.kw = 1 + ref.normal((D,), dtype, seed + 4, 0.2), 1 + ref.normal((D,), dtype, seed + 5, 0.2)
        self.cos = self.sin = self.positions = None
        if pairs:
            self.cos, self.sin = tables(rows, pairs)
            g = torch.Generator().manual_seed(seed)
            self.positions = torch.randint(0, rows, (T,), generator=g).to(ids)
            if T > 2:
                self.positions[1], self.positions[2] = -1, rows          # not rotated

    def place(self, t, like=None):
        """A tensor of t's shape in the layout, holding t (or, without t, 3s)."""
        T, H, D = t.shape
        if self.layout == "apart":
            return t.to(dev()).contiguous()
        if self.layout == "heads first":
            return t.to(dev()).transpose(0, 1).contiguous().transpose(0, 1)
        if self.layout == "odd":                                          # rows and heads apart, at odd elements
            b = torch.full((T, H * (D + 3) + 5), 3.0, dtype=t.dtype, device=dev())
            v = b[:, 1: 1 + H * (D + 3)].view(T, H, D + 3)[..., :D] if T * H else b[:, :0].view(T, H, D)
            v.copy_(t.to(dev()))
            return v
        raise AssertionError

    def pair(self, a, b):
        if self.layout != "fused":
            return self.place(a), self.place(b)
        T, Hq, Hk, D = self.dims
        f = torch.full((T, Hq + 2 * Hk, D), 3.0, dtype=a.dtype, device=dev())
        f[:, :Hq], f[:, Hq: Hq + Hk] = a.to(dev()), b.to(dev())
        return f[:, :Hq], f[:, Hq: Hq + Hk]

    def kw_args(self, pad=0):
        on = lambda t: None if t is None else t.to(dev())  # noqa: E731
        cos, sin = (None, None) if self.cos is None else (in_rows(self.cos, pad), in_rows(self.sin, pad))
        return dict(q_weight=on(self.qw), k_weight=on(self.kw), positions=on(self.positions), cos=cos, sin=sin,
                    adjacent=self.adjacent)

    def where(self, eps):
        return self.positions, self.cos, self.sin, eps, self.adjacent


CASES = [  # T, Hq, Hk, D, pairs, adjacent
    (1, 32, 4, 128, 64, False), (5, 3, 1, 64, 32, False), (37, 4, 2, 128, 64, True), (9, 2, 2, 128, 32, False),
    (9, 2, 2, 128, 32, True), (4, 5, 1, 80, 40, False), (4, 3, 3, 96, 20, False), (6, 2, 1, 2, 1, False), (6, 2, 1, 2, 1, True),
    (3, 2, 1, 20, 7, False), (3, 2, 1, 20, 7, True), (3, 1, 1, 512, 256, False), (3, 1, 1, 510, 255, True), (3, 2, 1, 500, 100, False),
    (5, 2, 1, 80, 20, False), (5, 2, 1, 80, 20, True), (3, 1, 1, 512, 100, False),
    (7, 3, 2, 256, 128, True), (8, 2, 1, 64, 0, False), (130, 9, 1, 128, 64, False), (0, 2, 1, 64, 32, False), (3, 0, 2, 64, 32, False),
    (3, 2, 0, 64, 32, False), (2, 2, 1, 0, 0, False)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["fused", "apart", "odd", "heads first"])
@pytest.mark.parametrize("T,Hq,Hk,D,pairs,adjacent", CASES)
def test_forward_and_gradient(tide, T, Hq, Hk, D, pairs, adjacent, layout, dtype):
    say("heads", T, Hq, Hk, D, pairs, adjacent, layout, dtype)
    c = Case(T, Hq, Hk, D, pairs, adjacent, dtype, layout, seed=T + D, weights=layout != "apart",
             ids=torch.int32 if layout == "odd" else torch.int64)
    eps, kw, pad = 1e-5, c.kw_args(5 if layout == "odd" else 0), layout == "odd"
    q, k = c.pair(c.q, c.k)
    qo, ko = c.pair(torch.full_like(c.q, 3.0), torch.full_like(c.k, 3.0))
    tide.norm_rotate(q, k, qo, ko, eps=eps, **kw)
    for got, x, w, what in ((qo, c.q, c.qw, "q"), (ko, c.k, c.kw, "k")):
        want, lim = step.norm_rotate(x, w, *c.where(eps))
        ref.close(got, want, lim + step.HALF[dtype] * want.abs(), what)
    dqo, dko = c.pair(c.dqo, c.dko)
    old = [1 + ref.normal((D,), dtype, 8), ref.normal((D,), dtype, 9)]
    for more in (False, True):
        dq, dk = c.pair(torch.full_like(c.q, 3.0), torch.full_like(c.k, 3.0))
        dw = [t.to(dev()).clone() for t in old]
        tide.norm_rotate_grad(dqo, dko, q, k, dq, dk, dq_weight=dw[0], dk_weight=dw[1], eps=eps, accumulate=more, **kw)
        for i, (got, x, d, w) in enumerate(((dq, c.q, c.dqo, c.qw), (dk, c.k, c.dko, c.kw))):
            dx, lim, want_w, lim_w = step.norm_rotate_grad(d, x, w, *c.where(eps))
            ref.close(got, dx, lim + step.HALF[dtype] * dx.abs(), "dx %d" % i)
            if more:
                want_w = want_w + old[i].double()
            ref.close(dw[i], want_w, lim_w + (step.HALF[dtype] + step.U) * want_w.abs(), "dw %d" % i)
    if pad and T and Hq and D:                                            # what lies between heads and rows
        for t in (qo, dq):
            b = torch.as_strided(t, (T, Hq, 3), t.stride(), t.storage_offset() + D).cpu()
            assert (b == 3.0).all()
    if layout == "fused" and T and Hk and D:                              # the values' window
        for t in (ko, dk):
            b = torch.as_strided(t, (T, Hk, D), t.stride(), t.storage_offset() + Hk * D).cpu()
            assert (b == 3.0).all()


def test_queries_alone_and_table_rows_by_token(tide):
    c = Case(20, 3, 1, 64, 32, False, BF16)
    q, _ = c.pair(c.q, c.k)
    cos, sin = c.cos.to(dev()), c.sin.to(dev())
    out = torch.empty(20, 3, 64, dtype=BF16, device=dev())
    tide.norm_rotate(q, None, out, None, q_weight=c.qw.to(dev()), cos=cos, sin=sin)
    want, lim = step.norm_rotate(c.q, c.qw, None, c.cos, c.sin, 1e-6, False)
    ref.close(out, want, lim + 2.0 ** -8 * want.abs(), "row t")
    dq, dw = torch.empty_like(out), torch.empty(64, dtype=BF16, device=dev())
    tide.norm_rotate_grad(c.dqo.to(dev()), None, q, None, dq, None, q_weight=c.qw.to(dev()), cos=cos, sin=sin, dq_weight=dw)
    dx, lim, ww, lw = step.norm_rotate_grad(c.dqo, c.q, c.qw, None, c.cos, c.sin, 1e-6, False)
    ref.close(dq, dx, lim + 2.0 ** -8 * dx.abs(), "dx")
    ref.close(dw, ww, lw + 2.0 ** -8 * ww.abs(), "dw")
    only = torch.empty_like(out)
    tide.norm_rotate_grad(c.dqo.to(dev()), None, q, None, only, None, q_weight=c.qw.to(dev()), cos=cos, sin=sin)
    assert torch.equal(only, dq)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_small_and_zero_heads(tide, dtype):
    """Heads whose squares are subnormal or vanish: eps 0 takes the norm of what is
    there, a head of zeros is 0 with eps above 0."""
    x = ref.normal((6, 2, 64), F32, 1)
    for t, e in enumerate((-10, -40, -55, -60, -62, 40)):
        x[t] *= 2.0 ** e
    x[3, 1] = 0.0
    x = x.to(dtype)
    out = torch.empty(6, 2, 64, dtype=dtype, device=dev())
    tide.norm_rotate(x.to(dev()), None, out, None, eps=1e-6)
    want, lim = step.norm_rotate(x, None, None, None, None, 1e-6, False)
    ref.close(out, want, lim + step.HALF[dtype] * want.abs() + 2.0 ** -133, "eps")
    x[3, 1] = 1.0
    tide.norm_rotate(x.to(dev()), None, out, None, eps=0.0)
    want, lim = step.norm_rotate(x, None, None, None, None, 0.0, False)
    # squares down to 2^-124 - 2^-20 of them lost below 2^-149: off by 2^-149 each
    sq = (x.double() ** 2).mean(-1, keepdim=True)
    ref.close(out, want, lim + (step.HALF[dtype] + 2.0 ** -149 / sq) * want.abs(), "no eps")
    x[0, 0, 5], x[1, 1, 7] = float("nan"), float("inf")
    tide.norm_rotate(x.to(dev()), None, out, None)
    assert torch.isnan(out[0, 0]).all() and torch.isfinite(out[0, 1]).all() and torch.isfinite(out[2:]).all()


def test_gradient_against_differences(tide):
    c = Case(3, 2, 1, 12, 4, False, F32, "apart", seed=3)
    c.qw = 1 + ref.normal((12,), F32, 1, 0.2)
    kw = c.kw_args()
    dq, dk = torch.empty(3, 2, 12, device=dev()), torch.empty(3, 1, 12, device=dev())
    dw = torch.empty(12, device=dev())
    tide.norm_rotate_grad(c.dqo.to(dev()), c.dko.to(dev()), c.q.to(dev()), c.k.to(dev()), dq, dk, dq_weight=dw, eps=0.1, **kw)

    def value(x, w):
        return float((step.norm_rotate(x, w, *c.where(0.1))[0] * c.dqo.double()).sum())

    e = 1e-5
    for at in ((0, 0, 0), (0, 1, 5), (1, 0, 11), (2, 1, 8)):
        up, down = c.q.double().clone(), c.q.double().clone()
        up[at] += e
        down[at] -= e
        assert abs(float(dq[at]) - (value(up, c.qw) - value(down, c.qw)) / (2 * e)) < 2e-5 * (1 + float(dq[at].abs()))
    for i in (0, 4, 11):
        up, down = c.qw.double().clone(), c.qw.double().clone()
        up[i] += e
        down[i] -= e
        assert abs(float(dw[i]) - (value(c.q, up) - value(c.q, down)) / (2 * e)) < 2e-5 * (1 + float(dw[i].abs()))


def test_many_tokens_and_the_same_bits(tide):
    """More rows than the gradient has workgroups' heads at once, twice."""
    c = Case(3001, 4, 1, 64, 32, False, BF16, seed=2)
    kw = c.kw_args()
    q, k = c.pair(c.q, c.k)
    found = []
    for _ in range(2):
        dq, dk = c.pair(c.q, c.k)
        dw = [torch.empty(64, dtype=BF16, device=dev()) for _ in range(2)]
        need = tide.norm_rotate_grad_workspace_bytes(3001, 5, 64)
        tide.norm_rotate_grad(c.dqo.to(dev()), c.dko.to(dev()), q, k, dq, dk, dq_weight=dw[0], dk_weight=dw[1],
                              workspace=torch.full((need,), 255, dtype=torch.uint8, device=dev()), **kw)
        found.append([dq.clone(), dk.clone(), *dw])
    assert all(torch.equal(a, b) for a, b in zip(*found))
    for i, (x, d, w) in enumerate(((c.q, c.dqo, c.qw), (c.k, c.dko, c.kw))):
        dx, lim, ww, lw = step.norm_rotate_grad(d, x, w, *c.where(1e-6))
        ref.close(found[0][i], dx, lim + 2.0 ** -8 * dx.abs(), "dx")
        ref.close(found[0][2 + i], ww, lw + 2.0 ** -8 * ww.abs(), "dw")


MANY = [  # T, Hq, Hk, D, pairs, adjacent: 16384 heads and more, of which a wave takes two sets
    (2100, 8, 1, 128, 64, False), (2053, 7, 1, 128, 64, True), (1700, 8, 2, 80, 20, False), (1700, 6, 4, 80, 40, True),
    (600, 20, 8, 64, 32, False), (1100, 12, 3, 256, 64, False), (16400, 1, 0, 64, 32, False), (550, 24, 6, 512, 256, True),
    (1100, 14, 1, 96, 0, False), (5, 3300, 7, 16, 8, False)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["fused", "odd"])
@pytest.mark.parametrize("T,Hq,Hk,D,pairs,adjacent", MANY)
def test_forward_of_many_heads(tide, T, Hq, Hk, D, pairs, adjacent, layout, dtype):
    """Sets of heads that end in a wave's first or second, odd numbers of sets, keys
    that begin inside a set."""
    say("many heads", T, Hq, Hk, D, pairs, adjacent, layout, dtype)
    c = Case(T, Hq, Hk, D, pairs, adjacent, dtype, layout, seed=T + D, ids=torch.int32 if layout == "odd" else torch.int64)
    q, k = c.pair(c.q, c.k)
    qo, ko = c.pair(torch.full_like(c.q, 3.0), torch.full_like(c.k, 3.0))
    tide.norm_rotate(q, k, qo, ko, eps=1e-5, **c.kw_args(5 if layout == "odd" else 0))
    for got, x, w, what in ((qo, c.q, c.qw, "q"), (ko, c.k, c.kw, "k")):
        want, lim = step.norm_rotate(x, w, *c.where(1e-5))
        ref.close(got, want, lim + step.HALF[dtype] * want.abs(), what)
    if layout == "odd":                                                   # what lies between heads and rows
        assert (torch.as_strided(qo, (T, Hq, 3), qo.stride(), qo.storage_offset() + D) == 3.0).all()
        assert not Hk or (torch.as_strided(ko, (T, Hk, 3), ko.stride(), ko.storage_offset() + D) == 3.0).all()
    elif Hk:                                                              # the values' window
        assert (torch.as_strided(ko, (T, Hk, D), ko.stride(), ko.storage_offset() + Hk * D) == 3.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_tokens_than_waves(tide, dtype):
    """Over 2^24 tokens of one short head: what they are in pieces."""
    T = (1 << 24) + 4099
    g = torch.Generator(device=dev()).manual_seed(1)
    x = torch.randn(T, 1, 8, generator=g, device=dev(), dtype=dtype)
    out, part = torch.empty_like(x), torch.empty_like(x)
    tide.norm_rotate(x, None, out, None, eps=1e-5)
    for a, b in zip(x.split(1 << 20), part.split(1 << 20)):
        tide.norm_rotate(a, None, b, None, eps=1e-5)
    assert torch.equal(out, part)
    for at in (slice(0, 50), slice(T - 50, T)):
        want, lim = step.norm_rotate(x[at].cpu(), None, None, None, None, 1e-5, False)
        ref.close(out[at], want, lim + step.HALF[dtype] * want.abs(), "ends")


def test_heads_past_two_gib(tide):
    T, H, D = 3, 4, 64
    big = torch.zeros(T, 1 << 30, dtype=BF16, device=dev())
    x = big[:, -H * D:].view(T, H, D)
    src = ref.normal((T, H, D), BF16, 1)
    x.copy_(src.to(dev()))
    out = big[:, :H * D].view(T, H, D)
    tide.norm_rotate(x, None, out, None)
    want, lim = step.norm_rotate(src, None, None, None, None, 1e-6, False)
    ref.close(out, want, lim + 2.0 ** -8 * want.abs(), "far")
