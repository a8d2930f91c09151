"""The training-layer calls on the host (no GPU): workspace sizes, and that bad
arguments are refused by the library and by the binding before any launch."""
import ctypes

import pytest
import torch

FAKE = 0x7F0000000000          # never dereferenced: every call here is refused first
OK, ARG, ALIGN, OVER, UNSUP = 0, 1, 2, 3, 4
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


def saved(codes=FAKE + 4 * BIG, scales=FAKE + 5 * BIG, cs=64, ss=2):
    from mixed_precision_rs_amd._layer import Saved
    return Saved(codes, scales, cs, ss)


def test_workspaces(tide):
    assert tide.route_workspace_bytes(0, 1, 1) == 0
    assert tide.route_workspace_bytes(1, 8, 128) == 0
    many = tide.route_workspace_bytes(1 << 20, 8, 512)
    assert 0 < many <= 1 << 20
    assert tide.weight_grads_workspace_bytes(0, 64, 64) == 0
    assert tide.weight_grads_workspace_bytes(4096, 28672, 8192) == 0
    split = tide.weight_grads_workspace_bytes(8192, 128, 2048)         # few tiles, a long sum
    assert split >= 2 * 128 * 2048 * 4 and split % (128 * 2048 * 4) == 0
    for bad in [(-1, 1, 1), (1, 0, 1), (1, 1, 0)]:
        with pytest.raises(tide.TideError, match="INVALID_ARG"):
            tide.route_workspace_bytes(*bad)
    for bad in [(1, 1, 513), (1 << 30, 4, 8)]:
        with pytest.raises(tide.TideError, match="UNSUPPORTED"):
            tide.route_workspace_bytes(*bad)
    for bad in [(-1, 1, 1, 1), (1, -1, 1, 1), (1, 1, -1, 1), (1, 1, 1, 0)]:
        with pytest.raises(tide.TideError, match="INVALID_ARG"):
            tide.weight_grads_workspace_bytes(*bad)
    with pytest.raises(tide.TideError, match="UNSUPPORTED"):
        tide.weight_grads_workspace_bytes(1 << 31, 8, 8)


def test_route_refuses(call):
    ok = [FAKE, 8, 100, 2, 8, FAKE + BIG, FAKE + 2 * BIG, FAKE + 3 * BIG, None, 0, None]

    def with_(i, v):
        a = list(ok)
        a[i] = v
        return call("route_tokens", *a)
    assert with_(1, 2) == ARG and with_(2, -1) == ARG and with_(3, 0) == ARG and with_(4, 0) == ARG
    assert with_(4, 513) == UNSUP and with_(2, 1 << 31) == UNSUP
    for i in (0, 5, 6, 7):
        assert with_(i, None) == ARG and with_(i, FAKE + 6 * BIG + 2) == ALIGN
    assert with_(5, FAKE + 8) == ARG and with_(7, FAKE + 2 * BIG) == ARG        # overlaps
    big = list(ok)
    big[2] = 100000
    assert call("route_tokens", *big) == ARG                                   # no workspace
    big[8], big[9] = FAKE + 7 * BIG, 16
    assert call("route_tokens", *big) == ARG                                   # too small


def test_dispatch_and_combine_refuse(call):
    ok = [0, FAKE, 64, 10, 64, FAKE + BIG, 2, FAKE + 2 * BIG, 64, 20, None]

    def d(i, v):
        a = list(ok)
        a[i] = v
        return call("dispatch_tokens", *a)
    assert d(0, 2) == ARG and d(0, -1) == ARG
    assert d(2, 63) == ARG and d(8, 63) == ARG and d(3, -1) == ARG and d(4, -1) == ARG
    assert d(6, 0) == ARG and d(9, -1) == ARG and d(9, 1 << 31) == UNSUP and d(3, 1 << 30) == UNSUP
    assert d(1, None) == ARG and d(5, None) == ARG and d(7, None) == ARG
    assert d(1, FAKE + 1) == ALIGN and d(5, FAKE + BIG + 2) == ALIGN
    assert d(7, FAKE + 2) == ARG and d(7, FAKE + BIG) == ARG
    assert d(2, 1 << 62) == OVER
    ok2 = [1, FAKE, 64, 20, 64, FAKE + BIG, FAKE + 3 * BIG, 10, 2, FAKE + 2 * BIG, 64, None]

    def c(i, v):
        a = list(ok2)
        a[i] = v
        return call("combine_tokens", *a)
    assert c(0, 7) == ARG and c(1, None) == ARG and c(5, None) == ARG and c(9, None) == ARG
    assert c(1, FAKE + 2) == ALIGN and c(6, FAKE + 3 * BIG + 2) == ALIGN and c(10, 5) == ARG
    assert c(9, FAKE + 256) == ARG and c(9, FAKE + 3 * BIG) == ARG
    ok3 = [0, FAKE, 64, FAKE + BIG, 64, 20, 64, FAKE + 2 * BIG, FAKE + 3 * BIG, 10, 2, FAKE + 4 * BIG, 64,
           FAKE + 5 * BIG, None]

    def g(i, v):
        a = list(ok3)
        a[i] = v
        return call("combine_tokens_grad", *a)
    assert g(0, 3) == ARG and g(1, None) == ARG and g(3, None) == ARG and g(7, None) == ARG
    assert g(11, None) == ARG and g(11, FAKE + BIG) == ARG and g(13, FAKE + 4 * BIG) == ARG
    assert g(13, FAKE + 5 * BIG + 1) == ALIGN and g(12, 1) == ARG


def test_checkpoint_calls_refuse(call):
    s = saved()
    assert call("checkpoint_pack", 5, FAKE, 64, 4, 64, s, None) == ARG
    assert call("checkpoint_pack", 0, FAKE, 64, -4, 64, s, None) == ARG
    assert call("checkpoint_pack", 0, FAKE, 64, 4, 64, None, None) == ARG
    assert call("checkpoint_pack", 0, None, 64, 4, 64, s, None) == ARG
    assert call("checkpoint_pack", 1, FAKE + 2, 64, 4, 64, s, None) == ALIGN
    assert call("checkpoint_pack", 0, FAKE, 63, 4, 64, s, None) == ARG
    assert call("checkpoint_pack", 0, FAKE, 64, 4, 64, saved(cs=63), None) == ARG
    assert call("checkpoint_pack", 0, FAKE, 64, 4, 64, saved(ss=1), None) == ARG
    assert call("checkpoint_pack", 0, FAKE, 64, 4, 64, saved(codes=FAKE + 100), None) == ARG
    assert call("checkpoint_pack", 0, FAKE, 64, 4, 64, saved(codes=None), None) == ARG
    assert call("checkpoint_unpack", 0, s, 4, 64, None, 64, None) == ARG
    assert call("checkpoint_unpack", 0, s, 4, 64, s.scales, 64, None) == ARG
    assert call("checkpoint_unpack", 0, s, 1 << 40, 64, FAKE, 1 << 30, None) == OVER
    a, b = saved(), saved(FAKE + 6 * BIG, FAKE + 7 * BIG)
    ok = [0, FAKE, 64, FAKE + BIG, 64, 4, 64, FAKE + 2 * BIG, 64, a, b, None]
    for i, v, want in [(0, 2, ARG), (1, None, ARG), (3, None, ARG), (7, None, ARG), (7, FAKE, ARG), (2, 1, ARG),
                       (9, b, ARG), (3, FAKE + BIG + 1, ALIGN)]:
        t = list(ok)
        t[i] = v
        assert call("gated_silu", *t) == want, (i, v)
    ok = [0, FAKE, 64, a, b, 4, 64, FAKE + BIG, 64, FAKE + 2 * BIG, 64, FAKE + 3 * BIG, 64, None]
    for i, v, want in [(0, 9, ARG), (1, None, ARG), (3, None, ARG), (4, None, ARG), (7, None, ARG), (9, None, ARG),
                       (9, FAKE + BIG, ARG), (11, FAKE, ARG), (11, FAKE + 3 * BIG + 1, ALIGN), (8, 63, ARG)]:
        t = list(ok)
        t[i] = v
        assert call("gated_silu_grad", *t) == want, (i, v)


def test_weight_grads_refuses(call):
    arr = (ctypes.c_void_p * 2)(FAKE + 8 * BIG, FAKE + 9 * BIG)
    ok = [FAKE, 64, 50, 64, FAKE + BIG, 64, None, 50, 64, FAKE + 2 * BIG, FAKE + 3 * BIG, 2, arr, 0, None, 0, None]

    def w(**kw):
        names = ["dy", "dy_stride", "rows", "out", "x", "x_stride", "saved", "x_rows", "in_", "offsets", "tokens",
                 "experts", "grads", "accumulate", "ws", "ws_bytes", "stream"]
        a = list(ok)
        for n, v in kw.items():
            a[names.index(n)] = v
        return call("weight_grads_bf16", *a)
    assert w(dy=None) == ARG and w(dy=FAKE + 1) == ALIGN and w(dy_stride=63) == ARG and w(rows=-1) == ARG
    assert w(x=None) == ARG and w(saved=saved()) == ARG                # neither and both
    assert w(x_stride=10) == ARG and w(x_rows=-1) == ARG and w(x_rows=1 << 31) == UNSUP
    assert w(offsets=None) == ARG and w(offsets=FAKE + 2 * BIG + 2) == ALIGN
    assert w(tokens=None, x_rows=49) == ARG and w(tokens=FAKE + 3 * BIG + 1) == ALIGN
    assert w(experts=0) == ARG and w(grads=None) == ARG
    assert w(grads=(ctypes.c_void_p * 2)(FAKE + 8 * BIG, None)) == ARG
    assert w(grads=(ctypes.c_void_p * 2)(FAKE + 8 * BIG, FAKE + 8 * BIG + 64)) == ARG
    assert w(grads=(ctypes.c_void_p * 2)(FAKE + 8 * BIG, FAKE + 128)) == ARG
    assert w(grads=(ctypes.c_void_p * 2)(FAKE + 8 * BIG + 1, FAKE + 9 * BIG)) == ALIGN
    assert w(out=1 << 31) == UNSUP and w(out=1 << 30, in_=1 << 30, experts=1 << 30) == OVER
    assert w(x=None, saved=saved(ss=1)) == ARG and w(x=None, saved=saved(cs=1)) == ARG


def test_column_windows_of_one_tensor_do_not_overlap(call):
    """Halves of one 128-wide matrix pass the overlap check (and the call then
    finds no GPU, or would run); windows that share a column do not."""
    if torch.cuda.is_available():
        pytest.skip("the accepted call would run on the fake addresses")
    a = saved()
    ok = [0, FAKE, 64, a, saved(FAKE + 6 * BIG, FAKE + 7 * BIG), 4, 64, FAKE + BIG, 128, FAKE + BIG + 128, 128, None, 0,
          None]
    assert call("gated_silu_grad", *ok) == 6                           # TIDE_ERR_HIP: no GPU here
    ok[9] = FAKE + BIG + 126
    assert call("gated_silu_grad", *ok) == ARG


def test_binding_refuses(tide):
    """The binding's own checks, on CPU tensors: each is refused before the library sees an address."""
    from mixed_precision_rs_amd import _layer as lay
    b = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(TypeError, match="bfloat16 or torch.float32"):
        lay._dtype_code(b(2, 2, dt=torch.float16), "x")
    with pytest.raises(TypeError):
        lay._mat(b(2, 2), "x", torch.float32, None, None, None)
    with pytest.raises(ValueError, match="dimensions"):
        lay._mat(b(2), "x", torch.bfloat16, None, None, None)
    with pytest.raises(ValueError, match="2 x 3"):
        lay._mat(b(2, 3), "x", torch.bfloat16, None, 4, None)
    with pytest.raises(ValueError, match="not adjacent"):
        lay._mat(b(4, 4).t(), "x", torch.bfloat16, None, None, None)
    with pytest.raises(ValueError, match="rows overlap"):
        lay._mat(b(1, 4).expand(3, 4), "x", torch.bfloat16, None, None, None)
    with pytest.raises(ValueError, match="not a GPU tensor"):
        lay._mat(b(4, 4), "x", torch.bfloat16, None, None, None)
    with pytest.raises(ValueError, match="not contiguous"):
        lay._flat(b(4, 4)[:, :2], "slots", torch.bfloat16, (4, 2), None)
    with pytest.raises(ValueError, match="shape"):
        lay._flat(b(4), "slots", torch.bfloat16, (5,), None)
    codes, scales = b(2, 64, dt=torch.float8_e4m3fn), b(2, 2, dt=torch.uint8).view(torch.float8_e8m0fnu)
    with pytest.raises(ValueError, match="not a GPU tensor"):
        lay._saved((codes, scales), "saved", 2, 64, None)
    with pytest.raises(TypeError):
        lay._saved((codes.view(torch.uint8), scales), "saved", 2, 64, None)


def test_list_of_gradients_refuses_other_shapes(tide):
    """A list's tensors have to be (out, in) each: the transposed shape and a flat
    tensor hold as many elements."""
    from mixed_precision_rs_amd import _layer as lay
    g = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    for bad in (g(24, 16), g(16 * 24), g(1, 16, 24), g(16, 23)):
        with pytest.raises(ValueError, match=r"grads\[1\] has shape .* expected \(16, 24\)"):
            lay._grads_list([FAKE, bad], 16, 24, None)
    with pytest.raises(ValueError, match="not contiguous"):
        lay._grads_list([g(24, 16).t()], 16, 24, None)
    with pytest.raises(ValueError, match="not a GPU tensor"):
        lay._grads_list([g(16, 24)], 16, 24, None)
    assert list(lay._grads_list([FAKE, None], 16, 24, 0)) == [FAKE, None]


class OnGpu:
    """What the binding asks of a tensor about its place."""
    is_cuda = True

    def __init__(self, dev):
        self.dev = dev

    def get_device(self):
        return self.dev


def test_raw_handles_take_the_tensors_device(tide, monkeypatch):
    """With a raw stream handle, also the null one, the workspace is allocated and
    the other tensors are expected on the first tensor's GPU, which need not be the
    current one."""
    import contextlib
    from mixed_precision_rs_amd import _layer as lay
    for handle in (77, 0):
        assert lay._on(handle, OnGpu(3)) == (handle, None, 3)
        assert lay._on(handle, OnGpu(-1)) == (handle, None, None)      # a CPU tensor: refused as such later
    lay._place(OnGpu(3), "x", 3)
    with pytest.raises(ValueError, match="x is on GPU 1, the call on GPU 3"):
        lay._place(OnGpu(1), "x", 3)

    class Stream:
        def __init__(self, handle, device):
            self.device = device

    made, buf = [], torch.zeros(100, dtype=torch.uint8)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device="current": Stream(handle, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device="current": Stream(0, device))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: (made.append((n, device)), buf)[1])
    for handle in (77, 0):
        lay._workspace(100, None, handle, 3)
    assert made == [(100, 3), (100, 3)]


@pytest.mark.parametrize("n,O,I", [(9001, 64, 40), (6000, 128, 512), (5000, 96, 97), (2100, 128, 512), (129, 64, 64)])
def test_exact_sums_notice(n, O, I):
    """The whole numbers that the weight gradients are compared on bit for bit: a
    row left out, and sums joined from four partials in bf16, give other results."""
    import layer_reference as ref
    dy, x, all_ = ref.whole((n, O), 3, n), ref.whole((n, I), 3, I), torch.tensor([0, n])
    want = ref.rounded_sum(dy, x, all_, None)
    for r in list(range(0, n, n // 20)) + [n - 1]:
        less = (dy.double().t() @ x.double() - dy[r].double()[:, None] * x[r].double())[None]
        assert not torch.equal(less.float().to(torch.bfloat16), want), r
    parts = [ref.rounded_sum(dy[i::4], x[i::4], torch.tensor([0, len(dy[i::4])]), None).float() for i in range(4)]
    # whole numbers up to 256 are exact in bf16: partials that stay there (33 rows' do) lose nothing
    if max(float(p.abs().max()) for p in parts) > 256:
        assert not torch.equal(sum(parts).to(torch.bfloat16), want)
    else:
        assert n < 200
