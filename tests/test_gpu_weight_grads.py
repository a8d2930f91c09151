"""Weight gradients, from bf16 activations and from checkpoints, for one expert
and for many, against the definition in 64 bits on the CPU."""
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


def window(t, pad):
    b = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=torch.float32).to(t.dtype).to(dev())
    w = b[:, pad // 2: pad // 2 + t.shape[1]]
    w.copy_(t.to(dev()))
    return w


def window_bytes(t, pad):
    """The same of an 8-bit type, with 0xFF (NaN) around it."""
    b = torch.full((t.shape[0], t.shape[1] + pad), 0xFF, dtype=torch.uint8, device=dev())
    b[:, pad // 2: pad // 2 + t.shape[1]] = t.view(torch.uint8).to(dev())
    return b.view(t.dtype)[:, pad // 2: pad // 2 + t.shape[1]]


def bound(want, mag, rows):
    """One bf16 rounding of the result, and `rows` additions in the matrix unit
    (and one for the old value), each off by at most a step, 2^-23, of the
    magnitudes' sum."""
    return 2.0 ** -8 * want.abs() + (rows + 2) * 2.0 ** -23 * mag


def check(tide, dy, x, saved, offsets, tokens, pad=0, old=None):
    n, O = dy.shape
    I = x.shape[1]
    xin = x
    if saved:
        s = ref.saved_of(x)
        xv = ref.unpack(*s)
        xin = (window_bytes(s[0], pad), window_bytes(s[1], pad))
    else:
        xv = x
        xin = window(x, pad)
    E = 1 if offsets is None else len(offsets) - 1
    off = torch.tensor([0, n]) if offsets is None else offsets
    want, mag, cnt = ref.weight_grads(dy, xv, off, tokens)
    grads = torch.full((E + 2, O, I), 5.0, dtype=torch.bfloat16, device=dev())     # a guard on each side
    if old is not None:
        grads[1:-1] = old.to(dev())
        want = want + old.double()
        mag = mag + old.double().abs()
    tide.weight_grads_bf16(window(dy, pad), xin, grads[1:-1],
                           offsets=None if offsets is None else offsets.int().to(dev()),
                           token_of_row=None if tokens is None else tokens.int().to(dev()),
                           accumulate=old is not None)
    for e in range(E):
        ref.close(grads[1 + e], want[e], bound(want[e], mag[e], cnt[e]), "expert %d" % e)
    assert (grads[0].cpu() == 5.0).all() and (grads[-1].cpu() == 5.0).all()
    return grads[1:-1]


DENSE = [(1, 1, 1), (1, 64, 64), (2, 7, 130), (15, 64, 32), (16, 65, 96), (17, 128, 128), (31, 256, 256),
         (32, 257, 40), (33, 40, 513), (64, 300, 300), (100, 512, 2048), (129, 130, 1), (127, 1, 260),
         (1000, 512, 160), (4097, 128, 136), (0, 16, 48), (300, 768, 264)]


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("n,O,I", DENSE)
def test_one_parameter(tide, n, O, I, pad, saved):
    say("weight_grads", n, O, I, pad, saved)
    check(tide, ref.normal((n, O), torch.bfloat16, seed=n), ref.normal((n, I), torch.bfloat16, seed=I),
          saved, None, None, pad)


GROUPED = [  # tokens, k, experts, out, in, masked
    (1, 1, 2, 64, 64, 0), (1, 8, 128, 40, 48, 0), (50, 2, 8, 96, 128, 0.2), (200, 3, 5, 257, 130, 0),
    (300, 8, 16, 128, 256, 0.1), (97, 4, 60, 72, 33, 0.5), (30, 2, 300, 33, 64, 0), (1500, 2, 3, 264, 520, 0),
]


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("T,k,E,O,I,masked", GROUPED)
def test_many_experts(tide, T, k, E, O, I, masked, pad, saved):
    say("weight_grads", T, k, E, O, I, masked, pad, saved)
    off, tok, _ = ref.route(ref.experts(T, k, E, seed=T, masked=masked).numpy(), E)
    tokens = torch.full((T * k,), -1, dtype=torch.int64)
    tokens[: len(tok)] = torch.from_numpy(tok)
    dy = ref.normal((T * k, O), torch.bfloat16, seed=1)
    dy[len(tok):] = float("nan")                        # rows behind the last: in no sum
    check(tide, dy, ref.normal((T, I), torch.bfloat16, seed=2), saved, torch.from_numpy(off), tokens, pad)


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("n,O,I", [(1, 4096, 2816), (64, 4104, 2600), (100, 2570, 4611), (333, 4160, 2592),
                                   (700, 4100, 2570), (1000, 3856, 2832)])
def test_one_large_parameter(tide, n, O, I, pad, saved):
    """Enough tiles for the large ones, ragged at both edges."""
    say("weight_grads", n, O, I, pad, saved)
    check(tide, ref.normal((n, O), torch.bfloat16, seed=n), ref.normal((n, I), torch.bfloat16, seed=I),
          saved, None, None, pad)


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("T,k,E,O,I", [(700, 4, 48, 512, 520), (333, 8, 64, 257, 513), (2000, 1, 170, 136, 48)])
def test_many_experts_in_large_tiles(tide, T, k, E, O, I, pad, saved):
    say("weight_grads", T, k, E, O, I, pad, saved)
    off, tok, _ = ref.route(ref.experts(T, k, E, seed=T, masked=0.05).numpy(), E)
    tokens = torch.full((T * k,), -1, dtype=torch.int64)
    tokens[: len(tok)] = torch.from_numpy(tok)
    check(tide, ref.normal((T * k, O), torch.bfloat16, seed=1), ref.normal((T, I), torch.bfloat16, seed=2), saved,
          torch.from_numpy(off), tokens, pad)


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("n,O,I", [(2100, 128, 512), (5000, 96, 97), (1500, 61, 64), (9001, 64, 40), (700, 8, 16),
                                   (6000, 128, 512)])
def test_few_tiles_and_many_rows(tide, n, O, I, pad, saved):
    """Rows divided among waves and, the longest, among workgroups."""
    say("weight_grads", n, O, I, pad, saved)
    dy, x = ref.normal((n, O), torch.bfloat16, seed=n), ref.normal((n, I), torch.bfloat16, seed=I)
    check(tide, dy, x, saved, None, None, pad)
    check(tide, dy, x, saved, None, None, pad, old=ref.normal((1, O, I), torch.bfloat16, seed=3, scale=10.0))
    half = n // 3
    check(tide, dy, x, saved, torch.tensor([5, 5, half, n - 1]), None, pad)


def test_workspace_of_the_caller(tide):
    n, O, I = 3000, 128, 256
    dy, x = ref.normal((n, O), torch.bfloat16, seed=1).to(dev()), ref.normal((n, I), torch.bfloat16, seed=2).to(dev())
    need = tide.weight_grads_workspace_bytes(n, O, I)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=dev())       # whatever it holds
    a, b = (torch.empty(1, O, I, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    tide.weight_grads_bf16(dy, x, a, workspace=ws)
    tide.weight_grads_bf16(dy, x, b)
    assert torch.equal(a, b)
    with pytest.raises(tide.TideError, match="INVALID_ARG"):
        tide.weight_grads_bf16(dy, x, a, workspace=ws[: need - 1])


@pytest.mark.parametrize("saved", [False, True])
def test_segments_without_a_sort(tide, saved):
    """Offsets with empty experts, rows in no expert at both ends, x by row."""
    off = torch.tensor([3, 3, 20, 20, 53, 54, 54, 90])
    dy, x = ref.normal((100, 72), torch.bfloat16, seed=3), ref.normal((100, 80), torch.bfloat16, seed=4)
    dy[:3] = dy[90:] = float("nan")
    x[:3] = x[90:] = float("nan")
    check(tide, dy, x, saved, off, None)


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("E", [1, 4])
def test_accumulate(tide, E, saved):
    n, O, I = 200, 136, 96
    off = None if E == 1 else torch.tensor([0, 60, 60, 130, 200])
    check(tide, ref.normal((n, O), torch.bfloat16, seed=1), ref.normal((n, I), torch.bfloat16, seed=2), saved,
          off, None, old=ref.normal((E, O, I), torch.bfloat16, seed=3, scale=10.0))


@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("n,O,I", [(100, 2570, 4611), (700, 4100, 2570), (300, 1030, 2050), (600, 520, 515)])
def test_accumulate_in_large_tiles(tide, n, O, I, pad):
    check(tide, ref.normal((n, O), torch.bfloat16, seed=1), ref.normal((n, I), torch.bfloat16, seed=2), True,
          None, None, pad, old=ref.normal((1, O, I), torch.bfloat16, seed=3, scale=10.0))


def test_lists_and_tables_of_gradients(tide):
    n, O, I, E = 150, 64, 72, 3
    off = torch.tensor([0, 40, 90, 150], dtype=torch.int32, device=dev())
    dy = ref.normal((n, O), torch.bfloat16, seed=1).to(dev())
    x = ref.normal((n, I), torch.bfloat16, seed=2).to(dev())
    whole = torch.empty(E, O, I, dtype=torch.bfloat16, device=dev())
    tide.weight_grads_bf16(dy, x, whole, offsets=off)
    parts = [torch.empty(O, I, dtype=torch.bfloat16, device=dev()) for _ in range(E)]
    tide.weight_grads_bf16(dy, x, parts[::-1], offsets=off)
    assert all(torch.equal(p, w) for p, w in zip(parts[::-1], whole))
    again = [torch.empty_like(p) for p in parts]
    tide.weight_grads_bf16(dy, x, tide.PointerTable(again), offsets=off)
    assert all(torch.equal(p, w) for p, w in zip(again, whole))


def test_not_finite_values_stay_in_their_rows_and_columns(tide):
    n, O, I = 100, 72, 96
    dy, x = ref.normal((n, O), torch.bfloat16, seed=5), ref.normal((n, I), torch.bfloat16, seed=6)
    dy[4, 11] = float("nan")
    x[50, 70] = float("inf")
    for saved in (False, True):
        g = torch.empty(1, O, I, dtype=torch.bfloat16, device=dev())
        xin = x.to(dev())
        if saved:
            s = tuple(t.to(dev()) for t in ref.saved_of(x))
            xin = s
        tide.weight_grads_bf16(dy.to(dev()), xin, g)
        bad = ~torch.isfinite(g[0].cpu().float())
        want = torch.zeros(O, I, dtype=torch.bool)
        want[11] = True
        want[:, 70] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("big", [-100, 100])
def test_checkpoints_of_extreme_scales(tide, big):
    """Values near both ends of the scales' range decode as unpacking does."""
    n, O, I = 70, 24, 64
    x = ref.normal((n, I), torch.float32, seed=8) * 2.0 ** big
    x[:, ::5] *= 2.0 ** (-14 if big < 0 else 14)
    dy = (ref.normal((n, O), torch.float32, seed=9) * 2.0 ** (60 if big < 0 else -60)).to(torch.bfloat16)
    s = ref.saved_of(x)
    g = torch.empty(1, O, I, dtype=torch.bfloat16, device=dev())
    tide.weight_grads_bf16(dy.to(dev()), tuple(t.to(dev()) for t in s), g)
    want, mag, cnt = ref.weight_grads(dy, ref.unpack(*s), torch.tensor([0, n]), None)
    ref.close(g[0], want[0], bound(want[0], mag[0], cnt[0]))


def test_tokens_out_of_range_add_nothing(tide):
    n, O, I = 90, 40, 64
    tokens = torch.arange(n) % 50
    tokens[[3, 40, 77]] = torch.tensor([-1, 50, 2 ** 31 - 1])
    for saved in (False, True):
        check(tide, ref.normal((n, O), torch.bfloat16, seed=1), ref.normal((50, I), torch.bfloat16, seed=2), saved,
              torch.tensor([0, 44, 90]), tokens)


def test_offsets_past_the_rows_are_clamped(tide):
    n, O, I = 70, 40, 64
    dy, x = ref.normal((n, O), torch.bfloat16, seed=1).to(dev()), ref.normal((n, I), torch.bfloat16, seed=2).to(dev())
    a, b = (torch.empty(2, O, I, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    tide.weight_grads_bf16(dy, x, a, offsets=torch.tensor([-5, 30, 900], dtype=torch.int32, device=dev()))
    tide.weight_grads_bf16(dy, x, b, offsets=torch.tensor([0, 30, 70], dtype=torch.int32, device=dev()))
    assert torch.equal(a, b)


@pytest.mark.parametrize("saved", [False, True])
def test_same_bits_every_time(tide, saved):
    n, O, I = 3001, 264, 520
    dy, x = ref.normal((n, O), torch.bfloat16, seed=1).to(dev()), ref.normal((n, I), torch.bfloat16, seed=2)
    xin = tuple(t.to(dev()) for t in ref.saved_of(x)) if saved else x.to(dev())
    first = torch.empty(1, O, I, dtype=torch.bfloat16, device=dev())
    tide.weight_grads_bf16(dy, xin, first)
    for _ in range(5):
        g = torch.full_like(first, 9.0)
        tide.weight_grads_bf16(dy, xin, g)
        assert torch.equal(g, first)


@pytest.mark.parametrize("saved", [False, True])
def test_rows_past_32_bit_offsets(tide, saved):
    n, O, I, stride = 2200, 40, 48, 1 << 21
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GiB of GPU memory")
    dy, x = ref.normal((n, O), torch.bfloat16, seed=1), ref.normal((n, I), torch.bfloat16, seed=2)
    far = torch.empty(n, stride, dtype=torch.bfloat16, device=dev())
    d = far[:, 16: 16 + O]
    d.copy_(dy.to(dev()))
    if saved:
        s = ref.saved_of(x)
        c = torch.empty(n, stride, dtype=torch.uint8, device=dev())
        c[:, 32: 32 + I] = s[0].view(torch.uint8).to(dev())
        xin = (c.view(torch.float8_e4m3fn)[:, 32: 32 + I], s[1].to(dev()))
        xv = ref.unpack(*s)
    else:
        xin = torch.empty(n, stride, dtype=torch.bfloat16, device=dev())[:, 16: 16 + I]
        xin.copy_(x.to(dev()))
        xv = x
    g = torch.empty(1, O, I, dtype=torch.bfloat16, device=dev())
    tide.weight_grads_bf16(d, xin, g)
    want, mag, cnt = ref.weight_grads(dy, xv, torch.tensor([0, n]), None)
    ref.close(g[0], want[0], bound(want[0], mag[0], cnt[0]))


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("n,O,I", [(700, 45, 70), (1500, 520, 515), (300, 4103, 2601)])
def test_tokens_of_rows_past_32_bit_offsets(tide, n, O, I, saved):
    T, stride = 1100, 1 << 21
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GiB of GPU memory")
    dy, x = ref.normal((n, O), torch.bfloat16, seed=3), ref.normal((T, I), torch.bfloat16, seed=4)
    tokens = torch.randint(0, T, (n,), generator=torch.Generator().manual_seed(5))
    tokens[[0, 1, 5, n - 1]] = torch.tensor([T - 1, 0, -1, T])        # rows of no token add nothing
    tokens = tokens.to(torch.int32)
    if saved:
        s = ref.saved_of(x)
        c = torch.empty(T, stride, dtype=torch.uint8, device=dev())[:, 3: 3 + I]
        c.copy_(s[0].view(torch.uint8).to(dev()))
        xin, xv = (c.view(torch.float8_e4m3fn), s[1].to(dev())), ref.unpack(*s)
    else:
        xin, xv = torch.empty(T, stride, dtype=torch.bfloat16, device=dev())[:, 3: 3 + I], x
        xin.copy_(x.to(dev()))
    g = torch.empty(1, O, I, dtype=torch.bfloat16, device=dev())
    tide.weight_grads_bf16(dy.to(dev()), xin, g, token_of_row=tokens.to(dev()))
    want, mag, cnt = ref.weight_grads(dy, xv, torch.tensor([0, n]), tokens)
    ref.close(g[0], want[0], bound(want[0], mag[0], cnt[0]))


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("far", ["dy", "x"])
@pytest.mark.parametrize("n,O,I", [(100, 45, 70), (130, 520, 515), (70, 4103, 2601)])
def test_strides_past_32_mib(tide, n, O, I, far, saved):
    stride = (1 << 25) + 3 if saved and far == "x" else (1 << 24) + 3
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GiB of GPU memory")
    dy, x = ref.normal((n, O), torch.bfloat16, seed=6), ref.normal((n, I), torch.bfloat16, seed=7)

    def spread(t):
        s = torch.empty(n, stride, dtype=t.dtype, device=dev())[:, 5: 5 + t.shape[1]]
        s.copy_(t.to(dev()))
        return s

    d = spread(dy) if far == "dy" else dy.to(dev())
    if saved:
        s = ref.saved_of(x)
        c = s[0].view(torch.uint8)
        c = spread(c) if far == "x" else c.to(dev())
        xin, xv = (c.view(torch.float8_e4m3fn), s[1].to(dev())), ref.unpack(*s)
    else:
        xin, xv = spread(x) if far == "x" else x.to(dev()), x
    g = torch.empty(1, O, I, dtype=torch.bfloat16, device=dev())
    tide.weight_grads_bf16(d, xin, g)
    want, mag, cnt = ref.weight_grads(dy, xv, torch.tensor([0, n]), None)
    ref.close(g[0], want[0], bound(want[0], mag[0], cnt[0]))


def rows_without_a_token(tokens, dy, x_rows, seed):
    """A tenth of the rows, the first and the last among them, get tokens out of
    range, and values that no sum may meet."""
    n = tokens.numel()
    bad = torch.rand(n, generator=torch.Generator().manual_seed(seed)) < 0.1
    bad[[0, n - 1]] = True
    m = int(bad.sum())
    tokens[bad] = torch.tensor([-1, x_rows, 2 ** 31 - 1, -2 ** 31]).repeat(m // 4 + 1)[:m]
    held = torch.tensor([float("nan"), float("inf"), -float("inf")]).repeat(m // 3 + 1)[:m]
    dy[bad] = held.to(dy.dtype)[:, None]


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("n,O,I", [  # each tile, the split sums, rows shorter than a load
    (90, 40, 64), (6000, 128, 512), (70, 1990, 2039), (64, 4104, 2600), (700, 4100, 2570), (100, 7, 130)])
def test_rows_without_a_token_add_nothing_whatever_they_hold(tide, n, O, I, pad, saved):
    say("weight_grads, rows without a token", n, O, I, pad, saved)
    T = n // 2 + 1
    dy, x = ref.normal((n, O), torch.bfloat16, seed=n), ref.normal((T, I), torch.bfloat16, seed=I)
    tokens = torch.randint(0, T, (n,), generator=torch.Generator().manual_seed(8))
    rows_without_a_token(tokens, dy, T, seed=9)
    check(tide, dy, x, saved, None, tokens, pad)
    check(tide, dy, x, saved, torch.tensor([0, n // 3, n // 3, n]), tokens, pad,
          old=ref.normal((3, O, I), torch.bfloat16, seed=3))


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("n,O,I", [(700, 45, 70), (500, 1500, 2000), (300, 4103, 2601), (700, 4100, 2570)])
def test_rows_without_a_token_and_far_rows(tide, n, O, I, saved):
    """The same where x passes 32-bit offsets, in each tile."""
    T, stride = 1100, 1 << 21
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GiB of GPU memory")
    say("weight_grads, rows without a token, far rows", n, O, I, saved)
    dy, x = ref.normal((n, O), torch.bfloat16, seed=3), ref.normal((T, I), torch.bfloat16, seed=4)
    tokens = torch.randint(0, T, (n,), generator=torch.Generator().manual_seed(5))
    rows_without_a_token(tokens, dy, T, seed=6)
    if saved:
        s = ref.saved_of(x)
        c = torch.empty(T, stride, dtype=torch.uint8, device=dev())[:, 3: 3 + I]
        c.copy_(s[0].view(torch.uint8).to(dev()))
        xin, xv = (c.view(torch.float8_e4m3fn), s[1].to(dev())), ref.unpack(*s)
    else:
        xin, xv = torch.empty(T, stride, dtype=torch.bfloat16, device=dev())[:, 3: 3 + I], x
        xin.copy_(x.to(dev()))
    g = torch.empty(1, O, I, dtype=torch.bfloat16, device=dev())
    tide.weight_grads_bf16(dy.to(dev()), xin, g, token_of_row=tokens.int().to(dev()))
    want, mag, cnt = ref.weight_grads(dy, xv, torch.tensor([0, n]), tokens)
    ref.close(g[0], want[0], bound(want[0], mag[0], cnt[0]))


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("far", ["dy", "x"])
@pytest.mark.parametrize("n,O,I", [(70, 1990, 2039), (700, 4100, 2570)])
def test_strides_past_32_mib_in_the_other_tiles(tide, n, O, I, far, saved):
    """As test_strides_past_32_mib, at sizes that take the 128 x 128 and the 256 x 256 tile."""
    test_strides_past_32_mib(tide, n, O, I, far, saved)


EXACT = [  # split sums, teams of waves with ragged shares, each tile, rows shorter than a load
    (9001, 64, 40), (6000, 128, 512), (5000, 96, 97), (4097, 128, 136), (2100, 128, 512), (3001, 264, 520), (700, 8, 16),
    (33, 70, 70), (129, 64, 64), (2001, 1500, 2000), (1000, 1024, 1500), (300, 4103, 2601), (700, 4100, 2570), (1000, 7, 130)]


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("n,O,I", EXACT)
def test_sums_of_whole_numbers_bit_for_bit(tide, n, O, I, saved):
    """Small whole numbers, whose sums fp32 holds exactly in any order: one lost
    row, or partial sums in fewer bits, would show (test_exact_sums_notice)."""
    say("weight_grads, whole numbers", n, O, I, saved)
    T = n // 2 + 1
    dy, x, xt = ref.whole((n, O), 3, n), ref.whole((n, I), 3, I), ref.whole((T, I), 3, I + 1)
    old = ref.whole((3, O, I), 256, 7)
    tokens = torch.randint(-1, T + 1, (n,), generator=torch.Generator().manual_seed(8))
    put = lambda t: tuple(v.to(dev()) for v in ref.saved_of(t)) if saved else t.to(dev())  # noqa: E731
    if saved:
        assert torch.equal(ref.unpack(*ref.saved_of(x)), x.double())
    for off, xx, tok in ((torch.tensor([0, n]), x, None), (torch.tensor([3, n // 3, n // 3 + 1, n - 1]), x, None),
                         (torch.tensor([0, n // 3, n // 2, n]), xt, tokens)):
        E = len(off) - 1
        for start in (None, old[:E]):
            g = torch.full((E, O, I), 5.0, dtype=torch.bfloat16, device=dev()) if start is None else start.to(dev())
            tide.weight_grads_bf16(dy.to(dev()), put(xx), g, offsets=off.int().to(dev()),
                                   token_of_row=None if tok is None else tok.int().to(dev()),
                                   accumulate=start is not None)
            assert torch.equal(g.cpu(), ref.rounded_sum(dy, xx, off, tok, start)), (off, start is not None)
