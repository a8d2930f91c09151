"""Tokens sorted by expert and back, and the gradients, against the definition
in 64 bits on the CPU, through the package's entry points."""
import numpy as np
import pytest
import torch

import layer_reference as ref
from gpu_util import dev, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tide():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixed_precision_rs_amd as t
    return t


def routed(tide, ids, E, **kw):
    T, k = ids.shape
    d = ids.to(dev())
    off = torch.full((E + 1,), -7, dtype=torch.int32, device=dev())
    tok = torch.full((T * k,), -7, dtype=torch.int32, device=dev())
    slots = torch.full((T, k), -7, dtype=torch.int32, device=dev())
    tide.route_tokens(d, E, off, tok, slots, **kw)
    return off, tok, slots


def check_route(tide, ids, E):
    off, tok, slots = (t.cpu().numpy() for t in routed(tide, ids, E))
    woff, wtok, wslots = ref.route(ids.numpy(), E)
    assert np.array_equal(off, woff)
    assert np.array_equal(tok[: woff[-1]], wtok)
    assert (tok[woff[-1]:] == -7).all()                 # rows behind the last: left as they were
    assert np.array_equal(slots, wslots)


@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,E,masked", [
    (1, 1, 1, 0), (1, 8, 128, 0), (1, 8, 8, 1.0), (3, 2, 5, 0), (64, 1, 64, 0.3), (63, 3, 7, 0.1),
    (511, 8, 128, 0.05), (512, 8, 128, 0), (513, 8, 128, 0), (600, 7, 512, 0.5), (4096, 2, 60, 0),
    (4097, 1, 511, 0.2), (2731, 3, 2, 0.9), (16384, 8, 128, 0.05), (40000, 7, 33, 0),
])
def test_route(tide, T, k, E, masked, idt):
    say("route", T, k, E, masked, idt)
    check_route(tide, ref.experts(T, k, E, seed=T + k, masked=masked, dtype=idt), E)


def test_route_ids_out_of_range_repeated_and_one_expert(tide):
    ids = torch.tensor([[0, 0, 9], [-1, 3, 3], [2 ** 31 + 1, 4, -2 ** 40], [1, 1, 1]])
    check_route(tide, ids, 4)
    check_route(tide, torch.full((3000, 4), 5, dtype=torch.int32), 17)     # all to one
    check_route(tide, torch.full((3000, 4), -1, dtype=torch.int32), 17)    # none anywhere


def test_route_no_tokens(tide):
    off, _, _ = routed(tide, torch.empty((0, 8), dtype=torch.int64), 16)
    assert (off.cpu() == 0).all()


def test_route_workspace_of_the_caller(tide):
    ids = ref.experts(9000, 4, 128, seed=3)
    need = tide.route_workspace_bytes(9000, 4, 128)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=dev())
    a = routed(tide, ids, 128, workspace=ws)
    b = routed(tide, ids, 128)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def sorted_case(tide, T, k, E, masked, seed):
    ids = ref.experts(T, k, E, seed=seed, masked=masked)
    off, tok, slots = routed(tide, ids, E)
    return off, tok, slots, slots.cpu()


SHAPES = [  # T, k, E, width
    (1, 8, 128, 2048), (1, 1, 1, 1), (2, 3, 4, 7), (17, 2, 8, 64), (33, 8, 16, 65), (5, 5, 5, 513),
    (129, 8, 128, 2047), (1000, 4, 60, 96), (257, 9, 32, 520), (70, 17, 64, 1030), (3, 2, 8, 20000),
]


def buffer(rows, width, dtype, pad, fill):
    """A rows x width window of a wider, filled buffer, and the buffer."""
    b = torch.full((rows, width + pad), fill, dtype=dtype, device=dev())
    return b[:, pad // 2: pad // 2 + width], b


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("T,k,E,D", SHAPES)
def test_dispatch_and_combine(tide, T, k, E, D, pad, dtype):
    say("dispatch/combine", T, k, E, D, pad, dtype)
    off, tok, slots, hslots = sorted_case(tide, T, k, E, 0.2, seed=D)
    x = ref.normal((T, D), dtype, seed=1)
    xd, _ = buffer(T, D, dtype, pad, 0)
    xd.copy_(x)
    rows, whole = buffer(T * k, D, dtype, pad, -77.0)
    tide.dispatch_tokens(xd, slots, rows)
    n = int(off[-1])
    got = rows.cpu()
    assert torch.equal(got[:n], x[tok[:n].cpu().long()])
    assert (got[n:] == -77.0).all()
    if pad:                                             # nothing beside the window either
        side = whole.cpu()
        assert (side[:, : pad // 2] == -77.0).all() and (side[:, pad // 2 + D:] == -77.0).all()
    # and back, on other rows, with and without weights
    ys, _ = buffer(T * k, D, dtype, pad, 0)
    y = ref.normal((T * k, D), dtype, seed=2)
    ys.copy_(y)
    w = ref.normal((T, k), torch.float32, seed=3)
    w[hslots < 0] = float("nan")                        # a weight without a row is not read
    for weights in (None, w):
        out, whole = buffer(T, D, dtype, pad, -77.0)
        tide.combine_tokens(ys, slots, out, weights=None if weights is None else weights.to(dev()))
        want, mag = ref.combine(y, hslots, weights)
        # k fused multiply-adds, each off by 2^-24 of at most the magnitudes' sum, then one rounding
        close = ref.HALF[dtype] * want.abs() + (k + 1) * 2.0 ** -24 * mag
        ref.close(out, want, close, "combine")
        if pad:
            side = whole.cpu()
            assert (side[:, : pad // 2] == -77.0).all() and (side[:, pad // 2 + D:] == -77.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("T,k,E,D", SHAPES)
def test_combine_grad(tide, T, k, E, D, pad, dtype):
    say("combine_grad", T, k, E, D, pad, dtype)
    off, _, slots, hslots = sorted_case(tide, T, k, E, 0.2, seed=D + 1)
    y, d = ref.normal((T * k, D), dtype, seed=4), ref.normal((T, D), dtype, seed=5)
    w = ref.normal((T, k), torch.float32, seed=6)
    ys, _ = buffer(T * k, D, dtype, pad, 0)
    ys.copy_(y)
    dd, _ = buffer(T, D, dtype, pad, 0)
    dd.copy_(d)
    some = hslots >= 0
    at = hslots[some].long()
    for weights in (w, None):
        dr, _ = buffer(T * k, D, dtype, pad, -77.0)
        dw = torch.full((T, k), -77.0, device=dev())
        wd = None if weights is None else w.to(dev())
        tide.combine_tokens_grad(dd, ys, slots, wd, dr, dw)
        want = torch.full((T * k, D), -77.0, dtype=torch.float64)
        scaled = (d.double()[:, None, :] * (1.0 if weights is None else w.double()[..., None])).expand(T, k, D)
        want[at] = scaled[some]
        # one fp32 product, then the rounding
        ref.close(dr, want, (ref.HALF[dtype] + 2.0 ** -24) * want.abs(), "drows")
        prod = torch.zeros(T, k, D, dtype=torch.float64)
        prod[some] = y[at].double() * d.double()[:, None, :].expand(T, k, D)[some]
        # at most D additions, each off by 2^-24 of the magnitudes' sum
        ref.close(dw, prod.sum(-1), D * 2.0 ** -24 * prod.abs().sum(-1), "dweights")
        only = torch.full((T * k, D), -77.0, dtype=dtype, device=dev())
        tide.combine_tokens_grad(dd, None, slots, wd, only, None)
        assert torch.equal(only, dr)


def test_gradients_by_differences(tide):
    """The loss L = sum(c * combine(rows, weights)), rows = dispatch(x): its
    gradients against central differences of the forward calls, in fp32."""
    T, k, E, D = 6, 3, 5, 24
    _, _, slots, hslots = sorted_case(tide, T, k, E, 0.2, seed=11)
    x, c = (ref.normal((T, D), torch.float32, seed=s).to(dev()) for s in (1, 2))
    w = ref.normal((T, k), torch.float32, seed=3).to(dev())

    def loss(x, w):
        rows = torch.zeros(T * k, D, device=dev())
        out = torch.empty(T, D, device=dev())
        tide.dispatch_tokens(x, slots, rows)
        tide.combine_tokens(rows, slots, out, weights=w)
        return float((c.double() * out.double()).sum()), rows

    _, rows = loss(x, w)
    drows, dw = torch.zeros_like(rows), torch.empty_like(w)
    tide.combine_tokens_grad(c, rows, slots, w, drows, dw)
    dx = torch.empty_like(x)
    tide.combine_tokens(drows, slots, dx)
    # The loss is linear in x and in w, so a difference with step h = 1 has no truncation error:
    # what is left is the outputs' fp32 rounding, (k + 2) 2^-24 of sum |c w x| <= 400 in all.
    tol = 2 * 400 * (k + 2) * 2.0 ** -24
    for t, i in [(0, 0), (1, 5), (2, 23), (5, 11)]:
        a, b = x.clone(), x.clone()
        a[t, i] += 0.5
        b[t, i] -= 0.5
        assert abs(loss(a, w)[0] - loss(b, w)[0] - float(dx[t, i])) < tol
    for t, j in [(0, 0), (1, 2), (3, 1), (5, 2)]:
        a, b = w.clone(), w.clone()
        a[t, j] += 0.5
        b[t, j] -= 0.5
        assert abs(loss(x, a)[0] - loss(x, b)[0] - float(dw[t, j])) < tol


def test_not_finite_rows_stay_where_they_are(tide):
    """A NaN or infinite row reaches its own token only; rows that no slot
    names are never read."""
    T, k, E, D = 40, 2, 8, 96
    off, tok, slots, hslots = sorted_case(tide, T, k, E, 0.3, seed=5)
    y = ref.normal((T * k, D), torch.bfloat16, seed=7)
    n = int(off[-1])
    y[n:] = float("nan")
    y[3, 5] = float("nan")
    y[4, 6] = float("inf")
    out = torch.empty(T, D, dtype=torch.bfloat16, device=dev())
    tide.combine_tokens(y.to(dev()), slots, out)
    want, mag = ref.combine(y, hslots, None)
    ref.close(out, want, 2.0 ** -8 * want.abs() + 3 * 2.0 ** -24 * torch.nan_to_num(mag, 0, 0), "combine")


def test_no_tokens_and_no_columns(tide):
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=dev())  # noqa: E731
    s0, s4 = e(0, 2, dt=torch.int32), torch.zeros(4, 2, dtype=torch.int32, device=dev())
    tide.dispatch_tokens(e(0, 8), s0, e(0, 8))
    tide.combine_tokens(e(0, 8), s0, e(0, 8))
    tide.dispatch_tokens(e(4, 0), s4, e(8, 0))
    tide.combine_tokens(e(8, 0), s4, e(4, 0))
    dw = torch.full((4, 2), -7.0, device=dev())
    tide.combine_tokens_grad(e(4, 0), e(8, 0), s4, None, e(8, 0), dw)
    assert (dw.cpu() == 0).all()                        # an empty dot product
    out = torch.full((4, 8), 3.0, dtype=torch.bfloat16, device=dev())
    tide.combine_tokens(e(0, 8), torch.full_like(s4, -1), out)
    assert (out.cpu() == 0).all()                       # tokens without any row


def test_slots_out_of_range_are_skipped(tide):
    slots = torch.tensor([[0, 7], [-5, 1]], dtype=torch.int32, device=dev())
    x = torch.ones(2, 16, dtype=torch.bfloat16, device=dev())
    rows = torch.zeros(2, 16, dtype=torch.bfloat16, device=dev())
    tide.dispatch_tokens(x, slots, rows)
    out = torch.empty_like(x)
    tide.combine_tokens(rows, slots, out)
    assert (rows.cpu() == 1).all() and (out.cpu() == 1).all()


def test_rows_past_32_bit_offsets(tide):
    """Rows 2^20 elements apart: the last ones lie past 2^32 bytes and 2^31 elements."""
    T, k, D, stride = 600, 4, 72, 1 << 20
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GiB of GPU memory")
    _, tok, slots, hslots = sorted_case(tide, T, k, 8, 0.0, seed=2)
    wide = torch.empty(T * k, stride, dtype=torch.bfloat16, device=dev())
    rows = wide[:, 5: 5 + D]
    x = ref.normal((T, D), torch.bfloat16, seed=1)
    tide.dispatch_tokens(x.to(dev()), slots, rows)
    assert torch.equal(rows.cpu(), x[tok.cpu().long()])
    out = torch.empty(T, D, dtype=torch.bfloat16, device=dev())
    tide.combine_tokens(rows, slots, out)
    ref.close(out, 4 * x.double(), 0.0)
    dw = torch.empty(T, k, device=dev())
    more = torch.zeros(T * k, D, dtype=torch.bfloat16, device=dev())
    tide.combine_tokens_grad(x.to(dev()), rows, slots, None, more, dw)
    want = (x.double() ** 2).sum(1, keepdim=True).expand(T, k)
    ref.close(dw, want, D * 2.0 ** -24 * want)
