"""The calls at the ends of a training step and in front of its attention on the
host (no GPU): workspace sizes, and that bad arguments are refused by the library
and by the binding before any launch."""
import ctypes
import math

import pytest
import torch

FAKE = 0x7F0000000000          # never dereferenced: every call here is refused first
OK, ARG, ALIGN, OVER, UNSUP, HIP = 0, 1, 2, 3, 4, 6
BIG = 1 << 40


@pytest.fixture(scope="module")
def tide():
    import mixed_precision_rs_amd as t
    return t


@pytest.fixture(scope="module")
def call(tide):
    from mixed_precision_rs_amd import _layer

    def go(name, *args):
        return _layer._fn("tide_" + name)(*args)
    return go


def table_of(call, name, ok):
    """refused(**changed): the status with some of the arguments changed."""
    names = list(ok)

    def refused(**kw):
        assert set(kw) <= set(names)
        return call(name, *[kw.get(n, v) for n, v in ok.items()])
    return refused


def at(i):
    return FAKE + i * BIG


def test_workspaces(tide):
    for T, V in ((0, 0), (1, 1), (4096, 262144), (4097, 10), (1 << 20, 1 << 30)):
        assert tide.sort_ids_workspace_bytes(T, V) >= 4 + 4 * T
    assert tide.sort_ids_workspace_bytes((1 << 31) - 1, 5) > 0
    assert tide.embed_tokens_grad_workspace_bytes(0, 64) >= 0
    assert tide.norm_rotate_grad_workspace_bytes(0, 4, 64) > 0
    most = tide.norm_rotate_grad_workspace_bytes(1 << 20, 72, 128)
    assert 0 < most <= 16 << 20
    for f, bad in ((tide.sort_ids_workspace_bytes, [(-1, 1), (1, -1)]), (tide.embed_tokens_grad_workspace_bytes, [(-1, 1), (1, -1)]),
                   (tide.norm_rotate_grad_workspace_bytes, [(-1, 1, 64), (1, -1, 64), (1, 1, -2)])):
        for b in bad:
            with pytest.raises(tide.TideError, match="INVALID_ARG"):
                f(*b)
    for f, bad in ((tide.sort_ids_workspace_bytes, [(1 << 31, 1), (1, 1 << 31)]), (tide.embed_tokens_grad_workspace_bytes, [(1 << 31, 1)]),
                   (tide.norm_rotate_grad_workspace_bytes, [(1, 1, 63), (1, 1, 514), (1 << 31, 1, 64)])):
        for b in bad:
            with pytest.raises(tide.TideError, match="UNSUPPORTED"):
                f(*b)


def test_sort_ids_refuses(call):
    r = table_of(call, "sort_ids", dict(ids=at(0), id_bytes=8, tokens=100, vocab=50, offsets=at(1), order=at(2), ws=at(3), wsn=1 << 20,
                                        stream=None))
    assert r(id_bytes=2) == ARG and r(tokens=-1) == ARG and r(vocab=-1) == ARG
    assert r(tokens=1 << 31) == UNSUP and r(vocab=1 << 31) == UNSUP
    for n in ("ids", "offsets", "order", "ws"):
        assert r(**{n: None}) == ARG and r(**{n: at(6) + 2}) == ALIGN, n
    assert r(wsn=100) == ARG and r(offsets=at(0) + 8) == ARG and r(order=at(1)) == ARG and r(ws=at(2)) == ARG


def test_embed_refuses(call):
    r = table_of(call, "embed_tokens", dict(dtype=0, ids=at(0), id_bytes=4, tokens=10, table=at(1), ts=64, vocab=50, width=64, scale=1.0,
                                            out=at(2), os=64, stream=None))
    assert r(dtype=2) == ARG and r(id_bytes=1) == ARG and r(tokens=-1) == ARG and r(vocab=-1) == ARG and r(width=-1) == ARG
    assert r(ids=None) == ARG and r(table=None) == ARG and r(out=None) == ARG and r(ts=63) == ARG and r(os=63) == ARG
    assert r(ids=at(0) + 2) == ALIGN and r(table=at(1) + 1) == ALIGN and r(out=at(2) + 1) == ALIGN
    assert r(out=at(1) + 64) == ARG and r(out=at(0)) == ARG and r(ts=1 << 62) == OVER


def test_embed_grad_refuses(call, tide):
    need = tide.embed_tokens_grad_workspace_bytes(10, 64)
    r = table_of(call, "embed_tokens_grad", dict(dtype=0, dout=at(0), ds=64, tokens=10, width=64, offsets=at(1), order=at(2), vocab=50,
                                                 scale=1.0, grad=at(3), gs=64, accumulate=0, ws=at(4), wsn=need, stream=None))
    assert r(dtype=7) == ARG and r(tokens=-1) == ARG and r(vocab=-1) == ARG and r(width=-1) == ARG
    assert r(tokens=1 << 31) == UNSUP and r(vocab=1 << 31) == UNSUP and r(ds=1) == ARG and r(gs=1) == ARG
    for n in ("dout", "offsets", "order", "grad"):
        assert r(**{n: None}) == ARG and r(**{n: at(6) + 1}) == ALIGN, n
    assert r(grad=at(0)) == ARG and r(grad=at(1)) == ARG and r(grad=at(2)) == ARG
    if need:
        assert r(ws=None) == ARG and r(wsn=need - 1) == ARG and r(ws=at(4) + 8) == ALIGN and r(ws=at(3)) == ARG


def test_logprobs_refuse(call):
    r = table_of(call, "token_logprobs", dict(dtype=0, x=at(0), xs=100, tokens=10, vocab=100, targets=at(1), id_bytes=8, lp=at(2), st=at(3),
                                              H=at(4), top=3, ids=at(5), tops=at(6), ws=None, wsn=0, stream=None))
    assert r(dtype=2) == ARG and r(id_bytes=3) == ARG and r(tokens=-1) == ARG and r(vocab=-1) == ARG and r(top=-1) == ARG
    assert r(top=33) == UNSUP and r(vocab=1 << 31) == UNSUP and r(xs=99) == ARG and r(xs=1 << 62) == OVER
    for n in ("x", "targets", "lp", "ids", "tops"):
        assert r(**{n: None}) == ARG and r(**{n: at(8) + 1}) == ALIGN, n
    assert r(st=at(8) + 2) == ALIGN and r(H=at(8) + 2) == ALIGN
    assert r(lp=at(0) + 4) == ARG and r(st=at(2)) == ARG and r(H=at(1)) == ARG and r(tops=at(5) + 4) == ARG
    need = ctypes.c_int64()
    assert call("token_logprobs_workspace", 0, 10, 131072, 3, need) == OK and need.value > 0
    large = dict(vocab=131072, xs=131072, ws=at(7), wsn=need.value)
    assert r(**{**large, "ws": None}) == ARG and r(**{**large, "wsn": need.value - 1}) == ARG and r(**{**large, "ws": at(7) + 4}) == ALIGN
    assert r(**{**large, "ws": at(2)}) == ARG and r(**{**large, "ws": at(0)}) == ARG
    assert call("token_logprobs_workspace", 0, 5000, 131072, 3, need) == OK and need.value == 0
    assert call("token_logprobs_workspace", 0, -1, 5, 3, need) == ARG and call("token_logprobs_workspace", 3, 1, 5, 3, need) == ARG
    assert call("token_logprobs_workspace", 0, 1, 5, 33, need) == UNSUP and call("token_logprobs_workspace", 0, 1, 5, 3, None) == ARG
    g = table_of(call, "token_logprobs_grad", dict(dtype=1, x=at(0), xs=100, tokens=10, vocab=100, targets=at(1), id_bytes=8, st=at(2),
                                                   d=at(3), H=at(4), h=at(5), dx=at(6), dxs=100, stream=None))
    assert g(dtype=2) == ARG and g(id_bytes=3) == ARG and g(tokens=-1) == ARG and g(H=None) == ARG and g(dxs=99) == ARG
    for n in ("x", "targets", "st", "d", "dx"):
        assert g(**{n: None}) == ARG and g(**{n: at(8) + 2}) == ALIGN, n
    assert g(dx=at(0) + 400) == ARG and g(dx=at(0), dxs=101) == ARG and g(dx=at(3)) == ARG and g(dx=at(2)) == ARG


def heads(i, token_stride=1024, head_stride=64, n=8, reserved=0):
    from mixed_precision_rs_amd._step import Heads
    return Heads(0 if i is None else at(i), token_stride, head_stride, n, reserved)


def rotation(**kw):
    from mixed_precision_rs_amd._step import Rotation
    ok = dict(positions=at(10), cos=at(11), sin=at(12), table_rows=100, table_stride=32, id_bytes=8, pairs=32, adjacent=0, reserved=0)
    ok.update(kw)
    return Rotation(*[v or 0 for v in ok.values()])


def test_norm_rotate_refuses(call):
    r = table_of(call, "norm_rotate", dict(dtype=0, tokens=5, dim=64, q=heads(0), k=heads(1, n=2), qw=at(2), kw=at(3), eps=1e-6, rot=rotation(),
                                           qo=heads(4), ko=heads(5, n=2), stream=None))
    assert r(dtype=2) == ARG and r(tokens=-1) == ARG and r(dim=-2) == ARG and r(dim=63) == UNSUP and r(dim=514) == UNSUP
    assert r(tokens=1 << 31) == UNSUP
    for e in (-1e-6, math.nan, math.inf):
        assert r(eps=e) == ARG
    assert r(q=None) == ARG and r(qo=None) == ARG and r(ko=None) == ARG and r(k=None) == ARG
    assert r(q=heads(None)) == ARG and r(q=heads(0, reserved=1)) == ARG and r(q=heads(0, n=-1)) == ARG and r(qo=heads(4, n=7)) == ARG
    assert r(q=heads(0, token_stride=63)) == ARG and r(q=heads(0, head_stride=63)) == ARG
    assert r(q=heads(0, token_stride=100, head_stride=64)) == ARG                 # tokens and heads interleave
    assert r(q=heads(0, token_stride=1 << 62)) == OVER
    from mixed_precision_rs_amd._step import Heads
    assert r(q=Heads(at(0) + 1, 1024, 64, 8, 0)) == ALIGN and r(qw=at(2) + 1) == ALIGN and r(kw=at(3) + 1) == ALIGN
    assert r(qo=heads(0)) == ARG and r(ko=heads(4, n=2)) == ARG and r(qo=heads(2)) == ARG and r(ko=heads(11, n=2)) == ARG
    for kw in (dict(pairs=33), dict(pairs=-1), dict(reserved=1), dict(id_bytes=2), dict(cos=None), dict(sin=None), dict(table_stride=31),
               dict(positions=None, table_rows=4), dict(table_rows=-1)):
        assert r(rot=rotation(**kw)) == ARG, kw
    assert r(rot=rotation(cos=at(11) + 2)) == ALIGN and r(rot=rotation(positions=at(10) + 4)) == ALIGN


def test_norm_rotate_grad_refuses(call, tide):
    need = tide.norm_rotate_grad_workspace_bytes(5, 10, 64)
    r = table_of(call, "norm_rotate_grad", dict(dtype=0, tokens=5, dim=64, gq=heads(0), gk=heads(1, n=2), q=heads(2), k=heads(3, n=2), qw=at(4),
                                                kw=at(5), eps=1e-6, rot=rotation(), dq=heads(6), dk=heads(7, n=2), dqw=at(8), dkw=at(9),
                                                accumulate=0, ws=at(13), wsn=need, stream=None))
    assert r(dtype=2) == ARG and r(dim=3) == UNSUP and r(eps=-1.0) == ARG and r(q=None) == ARG and r(gq=None) == ARG and r(dq=None) == ARG
    assert r(gk=None) == ARG and r(dk=None) == ARG and r(k=None) == ARG and r(dk=heads(7, n=3)) == ARG
    assert r(ws=None) == ARG and r(wsn=need - 4) == ARG and r(ws=at(13) + 8) == ALIGN and r(ws=at(8)) == ARG
    assert r(dq=heads(0)) == ARG and r(dk=heads(6, n=2)) == ARG and r(dqw=at(4)) == ARG and r(dkw=at(8)) == ARG
    assert r(dqw=at(8) + 1) == ALIGN and r(rot=rotation(pairs=33)) == ARG


def lists(*pointers, n=100000):
    return (ctypes.c_void_p * len(pointers))(*pointers), (ctypes.c_int64 * len(pointers))(*[n] * len(pointers))


def test_grad_squares_refuses(call):
    p, n = lists(at(0), at(1))
    r = table_of(call, "grad_squares", dict(dtype=0, grads=p, elems=n, tensors=2, total=at(2), accumulate=0, ws=at(3), wsn=1 << 20, stream=None))
    assert r(dtype=2) == ARG and r(tensors=-1) == ARG and r(grads=None) == ARG and r(elems=None) == ARG
    assert r(total=None) == ARG and r(total=at(2) + 4) == ALIGN and r(ws=None) == ARG and r(wsn=8) == ARG and r(ws=at(3) + 4) == ALIGN
    assert r(grads=lists(at(0), None)[0]) == ARG and r(grads=lists(at(0), at(1) + 1)[0]) == ALIGN
    assert r(total=at(0) + 8) == ARG and r(ws=at(1)) == ARG and r(total=at(3)) == ARG
    assert r(elems=(ctypes.c_int64 * 2)(5, -1)) == ARG and r(elems=(ctypes.c_int64 * 2)(1 << 62, 1 << 62)) == OVER
    need = ctypes.c_int64()
    assert call("grad_squares_workspace", 0, n, 2, None) == ARG and call("grad_squares_workspace", 0, n, 2, need) == OK and need.value == 26 * 8
    few = (ctypes.c_int64 * 2)(100, 7)
    assert call("grad_squares_workspace", 0, few, 2, need) == OK and need.value == 0
    assert call("grad_squares_workspace", 1, None, 0, need) == OK and need.value == 0


def test_clip_refuses(call):
    p, n = lists(at(0), at(1))
    o, _ = lists(at(4), at(5))
    r = table_of(call, "clip_grads", dict(dtype=1, grads=p, elems=n, tensors=2, total=at(2), most=1.0, out=o, norm=at(3), stream=None))
    assert r(dtype=2) == ARG and r(tensors=-1) == ARG and r(grads=None) == ARG and r(total=None) == ARG and r(total=at(2) + 4) == ALIGN
    assert r(most=-1.0) == ARG and r(most=math.nan) == ARG and r(norm=at(3) + 2) == ALIGN
    assert r(grads=lists(at(0), None)[0]) == ARG and r(out=lists(at(4), None)[0]) == ARG and r(out=lists(at(4), at(5) + 2)[0]) == ALIGN
    assert r(out=lists(at(4), at(4) + 399996)[0]) == ARG                          # two outputs share four bytes
    assert r(out=lists(at(1), at(5))[0]) == ARG                                # an output is another gradient
    assert r(out=lists(at(0) + 4, at(5))[0]) == ARG                            # not quite in place
    assert r(out=lists(at(2), at(5))[0]) == ARG and r(norm=at(4)) == ARG and r(norm=at(2)) == ARG and r(norm=at(0) + 8) == ARG
    same = lists(at(0), at(0))[0]
    assert r(grads=same, out=None) == ARG and r(grads=same, out=same) == ARG   # twice in place
    if not torch.cuda.is_available():                                          # accepted: the call then finds no GPU
        assert r(grads=same) == HIP and r(out=None) == HIP and r(out=lists(at(0), at(1) + 400000)[0]) == HIP


def test_clip_refuses_every_shared_byte_and_nothing_else(call):
    """Random small ranges, in place and not, against a comparison of every pair."""
    if torch.cuda.is_available():
        pytest.skip("the accepted calls would run on the fake addresses")
    import random
    rng = random.Random(1)
    seen = {ARG: 0, HIP: 0}
    for _ in range(3000):
        n = rng.randint(1, 6)
        size = [rng.randint(0, 3) for _ in range(n)]
        spread = rng.choice([20, 60, 200])
        src = [rng.randrange(spread) for _ in range(n)]
        dst = [s if rng.random() < 0.4 else rng.randrange(spread) for s in src]
        total, norm = 2 * rng.randrange(spread // 2), rng.randrange(spread)
        reads = [(total, total + 2)] + [(a, a + k) for a, b, k in zip(src, dst, size) if a != b]
        writes = [(norm, norm + 1)] + [(b, b + k) for b, k in zip(dst, size)]
        meet = lambda x, y: x[0] < y[1] and y[0] < x[1] and x[0] < x[1] and y[0] < y[1]  # noqa: E731
        bad = any(meet(w, r) for w in writes for r in reads) or any(
            meet(writes[i], writes[j]) for i in range(len(writes)) for j in range(i))
        place = lambda v: FAKE + 4 * v  # noqa: E731
        got = call("clip_grads", 1, (ctypes.c_void_p * n)(*map(place, src)), (ctypes.c_int64 * n)(*size), n, place(total), 1.0,
                   (ctypes.c_void_p * n)(*map(place, dst)), place(norm), None)
        assert got == (ARG if bad else HIP), (src, dst, size, total, norm)
        seen[got] += 1
    assert min(seen.values()) > 300, seen


def test_windows_of_fused_rows_do_not_overlap(call):
    """dq, dk as windows of one gradient of the fused projection pass the check."""
    if torch.cuda.is_available():
        pytest.skip("the accepted call would run on the fake addresses")
    from mixed_precision_rs_amd._step import Heads
    win = lambda base, first, n: Heads(at(base) + 2 * 64 * first, 12 * 64, 64, n, 0)  # noqa: E731
    go = lambda ko: call("norm_rotate", 0, 5, 64, win(0, 0, 8), win(0, 8, 2), None, None, 1e-6, None, win(1, 0, 8), ko, None)  # noqa: E731
    assert go(win(1, 8, 2)) == HIP and go(win(1, 7, 2)) == ARG
    one = lambda base, first, n: Heads(at(base) + 2 * 64 * first, 64, 64, n, 0)  # noqa: E731
    assert call("norm_rotate", 0, 1, 64, one(0, 0, 8), one(0, 8, 2), None, None, 1e-6, None, one(1, 0, 8), one(1, 8, 2), None) == HIP


def test_binding_refuses(tide):
    """The binding's own checks, on CPU tensors: each is refused before the library sees an address."""
    from mixed_precision_rs_amd import _step as st
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(TypeError, match="int32 or torch.int64"):
        st._ids(z(4, dt=torch.int16), "ids", None, None)
    with pytest.raises(ValueError, match="shape"):
        st._ids(z(2, 2, dt=torch.int32), "ids", None, None)
    with pytest.raises(ValueError, match="not a GPU tensor"):
        st._ids(z(4, dt=torch.int32), "ids", None, None)
    for bad, what in ((z(4, 4), "dimensions"), (z(3, 2, 8), "tokens"), (z(4, 3, 8), "heads"), (z(4, 2, 6), "elements a head"),
                      (z(8, 2, 4).transpose(0, 2), "not adjacent"), (z(4, 2, 8), "not a GPU tensor")):
        with pytest.raises(ValueError, match=what):
            st._heads(bad, "q", torch.bfloat16, 4, 2, 8, None)
    with pytest.raises(TypeError):
        st._heads(z(4, 2, 8), "q", torch.float32, 4, 2, 8, None)
    with pytest.raises(ValueError, match="together"):
        st._rotation(None, z(4, 4, dt=torch.float32), None, False, 4, None)
    with pytest.raises(ValueError, match="positions without"):
        st._rotation(z(4, dt=torch.int32), None, None, False, 4, None)
    with pytest.raises(TypeError, match="expected torch.bfloat16 or"):
        tide.TensorTable([z(4, dt=torch.float16)])
    with pytest.raises(ValueError, match="not a GPU tensor"):
        tide.TensorTable([z(4)])
    with pytest.raises(ValueError, match="not contiguous"):
        tide.TensorTable([z(4, 4).t()])
    with pytest.raises(TypeError, match="no sizes"):
        tide.grad_squares(tide._lib.PointerTable([]), z(1, dt=torch.float64))
    empty = tide.TensorTable([])
    assert empty.n == 0 and empty.workspace_bytes == 0
    with pytest.raises(ValueError, match="not a GPU tensor"):
        tide.grad_squares(empty, z(1, dt=torch.float64))
    with pytest.raises(ValueError, match="go together"):
        tide.norm_rotate(FakeGpu(z(1, 1, 2)), FakeGpu(z(1, 1, 2)), FakeGpu(z(1, 1, 2)), None)


class FakeGpu:
    """A CPU tensor that says it is on a GPU; only its shape is looked at."""

    def __init__(self, t):
        self.t, self.is_cuda, self.dtype, self.shape = t, True, t.dtype, t.shape
        for name in ("dim", "stride", "numel", "data_ptr"):
            setattr(self, name, getattr(t, name))

    def get_device(self):
        return -1


def test_exact_sums_notice():
    """The whole numbers that the table's gradient is compared on bit for bit: a
    token left out gives another result."""
    import layer_reference as ref
    for T, V in ((300, 7), (5000, 40), (9001, 3), (40000, 2)):
        d = ref.whole((T, 72), 9, T).double()
        total = 2.0 * d.sum(0)
        for t in range(0, T, max(T // 20, 1)):
            assert not torch.equal(total.float(), (total - 2.0 * d[t]).float()), t
