"""Tokens sorted by id, embedding lookup and the table's gradient against the
definition on the CPU."""
import numpy as np
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


def window(t, pad, fill=0.0):
    """t on the GPU, as a window of a buffer whose rows are `pad` wider."""
    b = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=torch.float32).to(t.dtype).to(dev())
    w = b[:, pad // 2: pad // 2 + t.shape[1]]
    w.copy_(t.to(dev()))
    return w


def some_ids(T, V, seed, kind="words", dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        ids = torch.full((T,), V // 2, dtype=torch.int64)
    elif kind == "even":
        ids = torch.randint(0, max(V, 1), (T,), generator=g)
    elif kind == "falling":
        ids = torch.arange(T - 1, -1, -1) % max(V, 1)
    else:
        ids = (torch.exp(torch.rand(T, generator=g, dtype=torch.float64) * np.log(max(V, 1))).long() - 1).clamp(0, max(V - 1, 0))
    out = torch.rand(T, generator=g) < 0.1
    odd = torch.tensor([-1, V, -100, 2 ** 31 - 1, -2 ** 31] + ([2 ** 40, -2 ** 40 + 3] if dtype == torch.int64 else []))
    ids[out] = odd[torch.arange(int(out.sum())) % len(odd)]
    return ids.to(dtype)


def sort(tide, ids, V, **kw):
    offsets = torch.full((V + 1,), -7, dtype=torch.int32, device=dev())
    order = torch.full((len(ids),), -7, dtype=torch.int32, device=dev())
    tide.sort_ids(ids.to(dev()), V, offsets, order, **kw)
    return offsets, order


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,V,kind", [
    (0, 5, "even"), (1, 1, "even"), (1, 70000, "even"), (7, 3, "words"), (64, 512, "even"), (65, 513, "even"),
    (1000, 1, "one"), (1000, 262144, "words"), (4095, 40000, "words"), (4096, 262145, "even"), (4097, 300, "falling"),
    (4097, 262144, "words"), (9000, 262145, "even"), (20000, 50001, "one"), (70001, 131072, "words"), (300000, 1000, "even"),
    (5000, 0, "even"), (10, 0, "even")])
def test_sort(tide, T, V, kind, dtype):
    say("sort", T, V, kind, dtype)
    ids = some_ids(T, V, T + V, kind, dtype)
    if V == 0:
        ids = ids.clamp(max=-1)
    want_off, want = step.sort_ids(ids, V)
    off, order = sort(tide, ids, V)
    assert np.array_equal(off.cpu().numpy(), want_off)
    assert np.array_equal(order.cpu().numpy()[: len(want)], want)
    assert (order.cpu().numpy()[len(want):] == -7).all()           # left as they were


def test_sort_of_a_vocabulary_in_four_passes(tide):
    V = (1 << 27) + 5
    for T in (3, 5000):
        ids = torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(T))
        ids[0], ids[1] = V - 1, 0
        off, order = sort(tide, ids, V)
        want = torch.sort(ids, stable=True).indices
        assert torch.equal(order.cpu().long(), want)
        assert int(off[V]) == T and int(off[0]) == 0 and int(off[1]) == int((ids == 0).sum())
        probe = ids[:50]
        assert torch.equal(off[probe.to(dev())].cpu().long(), torch.tensor([int((ids < i).sum()) for i in probe]))


def test_sort_with_a_given_workspace_and_twice_the_same(tide):
    ids = some_ids(30000, 99999, 5)
    need = tide.sort_ids_workspace_bytes(30000, 99999)
    first = sort(tide, ids, 99999, workspace=torch.full((need,), 255, dtype=torch.uint8, device=dev()))
    again = sort(tide, ids, 99999)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (3, 10, 7), (5, 10, 8), (33, 100, 257), (130, 50, 2048), (2, 4, 20001), (0, 4, 8), (4, 0, 8), (4, 3, 0)])
def test_lookup(tide, T, V, D, pad, dtype):
    say("lookup", T, V, D, pad, dtype)
    ids = some_ids(T, V, T + D, "even", torch.int32 if pad else torch.int64)
    if V == 0:
        ids = ids.clamp(max=-1)
    table = ref.normal((V, D), dtype, D)
    if V > 1 and D > 1:
        table[1, 0], table[0, D - 1] = float("nan"), float("inf")
    for scale in (1.0, 45.254834, -0.5):
        whole = torch.full((T, D + pad), 3.0, dtype=dtype, device=dev())
        out = whole[:, pad // 2: pad // 2 + D]
        tide.embed_tokens(ids.to(dev()), window(table, pad), out, scale=scale)
        got, want = out.cpu(), step.lookup(ids, table, torch.tensor(scale, dtype=F32))
        assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
        if pad:
            w = whole.cpu()
            assert (w[:, : pad // 2] == 3.0).all() and (w[:, pad // 2 + D:] == 3.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("T,V,D,kind", [
    (1, 1, 1, "even"), (3, 10, 7, "even"), (50, 20, 8, "words"), (64, 3, 9, "one"), (65, 3, 33, "one"), (200, 2, 40, "even"),
    (700, 5, 100, "words"), (1000, 300, 257, "words"), (0, 6, 16, "even"), (9, 6, 0, "even"), (9, 0, 8, "even"), (129, 4, 2056, "falling")])
def test_table_gradient(tide, T, V, D, kind, pad, dtype):
    say("table gradient", T, V, D, kind, pad, dtype)
    ids = some_ids(T, V, T + D, kind)
    if V == 0:
        ids = ids.clamp(max=-1)
    off, order = sort(tide, ids, V)
    dout, old = ref.normal((T, D), dtype, T), ref.normal((V, D), dtype, 1)
    for scale, more in ((1.0, False), (45.254834, True), (-2.0, False), (1.0, True)):
        whole = torch.full((V, D + pad), 3.0, dtype=dtype, device=dev())
        grad = whole[:, pad // 2: pad // 2 + D]
        if more:
            grad.copy_(old.to(dev()))
        tide.embed_tokens_grad(window(dout, pad, float("nan")), off, order, grad, scale=scale, accumulate=more)
        f = float(torch.tensor(scale, dtype=F32))
        want, lim = step.table_grad(dout, off.cpu(), order.cpu(), V, f, old if more else None)
        lim = torch.where(lim < 0, 0.0, lim + step.HALF[dtype] * want.abs())
        ref.close(grad, want, lim, "gradient")
        if pad:
            w = whole.cpu()
            assert (w[:, : pad // 2] == 3.0).all() and (w[:, pad // 2 + D:] == 3.0).all()


@pytest.mark.parametrize("T,V,kind,D", [
    (300, 7, "words", 72), (5000, 40, "words", 72), (9001, 3, "even", 72), (40000, 2, "one", 72), (17001, 90, "words", 1033),
    (4097, 4097, "even", 520), (16385, 3, "words", 1), (66000, 20, "falling", 72), (33, 5, "words", 600)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_whole_numbers_bit_for_bit(tide, T, V, kind, D, dtype):
    """Sums of whole numbers are exact in fp32 in any order: a token left out, one
    taken twice or a sum joined in bf16 would show."""
    ids = some_ids(T, V, T, kind)
    off, order = sort(tide, ids, V)
    dout, old = ref.whole((T, D), 9, T).to(dtype), ref.whole((V, D), 9, 3).to(dtype)
    for more in (False, True):
        grad = old.to(dev()).clone()
        tide.embed_tokens_grad(dout.to(dev()), off, order, grad, scale=2.0, accumulate=more)
        want = torch.zeros(V + 1, D, dtype=torch.float64)
        want.index_add_(0, torch.where((ids >= 0) & (ids < V), ids, V), 2.0 * dout.double())
        want = want[:V] + (old.double() if more else 0.0)
        assert float(want.abs().max()) < 2 ** 24
        assert torch.equal(grad.cpu(), want.float().to(dtype))


@pytest.mark.parametrize("V,kind", [(90, "words"), (5000, "even"), (20000, "even"), (3, "one")])
@pytest.mark.parametrize("dtype,D", [(BF16, 24), (F32, 9)])
def test_whole_numbers_of_a_million_tokens(tide, V, kind, dtype, D):
    """Over 2^20 tokens, of which a wave takes 256 in turns of 64: rows that end in a
    turn, cross several, and cross chunks. Sums below 2^24 in magnitude: exact."""
    T = (1 << 20) + 777
    say("a million tokens", V, kind, dtype)
    ids = some_ids(T, V, V, kind)
    off, order = sort(tide, ids, V)
    dout, old = ref.whole((T, D), 3, V).to(dtype), ref.whole((V, D), 9, 3).to(dtype)
    want = torch.zeros(V + 1, D, dtype=torch.float64)
    want.index_add_(0, torch.where((ids >= 0) & (ids < V), ids, V), 2.0 * dout.double())
    for more in (False, True):
        grad = old.to(dev()).clone()
        tide.embed_tokens_grad(dout.to(dev()), off, order, grad, scale=2.0, accumulate=more)
        assert torch.equal(grad.cpu(), (want[:V] + (old.double() if more else 0.0)).float().to(dtype)), more


@pytest.mark.parametrize("dtype,D", [(BF16, 11), (F32, 3)])
def test_a_table_of_many_short_rows(tide, dtype, D):
    """More rows than the waves that clear and join look at in one turn."""
    T, V = 70001, 9_000_011
    ids = torch.cat([some_ids(T - 20001, V, 1, "even"), some_ids(20001, V, 2, "words")])
    ids[::7] = V - 1
    off, order = sort(tide, ids, V)
    dout = ref.whole((T, D), 9, 1).to(dtype)
    want = torch.zeros(V + 1, D, dtype=torch.float64)
    want.index_add_(0, torch.where((ids >= 0) & (ids < V), ids, V), dout.double())
    for more in (False, True):
        grad = torch.full((V, D), 2.0, dtype=dtype, device=dev())
        tide.embed_tokens_grad(dout.to(dev()), off, order, grad, accumulate=more)
        assert torch.equal(grad.cpu(), (want[:V] + (2.0 if more else 0.0)).float().to(dtype)), more


@pytest.mark.parametrize("more", [False, True])
def test_places_without_a_token_cost_nothing(tide, more):
    """A batch of padding but for a few tokens: what sort_ids left of an earlier batch
    behind the last row is not gone through. With those places' rows of dout read, 1
    GiB, the calls took 1.9 and 1.6 times as long as with an order that holds none."""
    T, V, D = 65536, 300, 8192
    ids = torch.full((T,), -1)
    ids[::500] = torch.arange(len(ids[::500])) % V
    off, order = sort(tide, ids, V)
    n = int(off[V])
    assert n == len(ids[::500])
    stale = torch.randperm(T, generator=torch.Generator().manual_seed(1)).to(torch.int32).to(dev())
    stale[:n] = order[:n]
    dout = torch.randn(T, D, device=dev(), dtype=BF16)
    work = torch.empty(tide.embed_tokens_grad_workspace_bytes(T, D), dtype=torch.uint8, device=dev())
    grads, best = [torch.zeros(V, D, dtype=BF16, device=dev()) for _ in range(2)], [1e9, 1e9]
    for turn in range(20):
        for i, o in enumerate((order, stale)):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            grads[i].zero_()
            a.record()
            tide.embed_tokens_grad(dout, off, o, grads[i], accumulate=more, workspace=work)
            b.record()
            b.synchronize()
            best[i] = min(best[i], a.elapsed_time(b))
        assert torch.equal(*grads)
    say("padded batch", more, best)
    assert best[1] < 1.3 * best[0], best


def test_a_row_of_nan_stays_in_its_row(tide):
    T, V, D = 500, 6, 40
    ids = some_ids(T, V, 3, "even")
    dout = ref.normal((T, D), F32, 2)
    hit = int(torch.nonzero(ids == 4)[0])
    dout[hit] = float("nan")
    dout[ids == -1] = float("inf")                                  # tokens without an id: never read into a sum
    off, order = sort(tide, ids, V)
    grad = torch.empty(V, D, device=dev())
    tide.embed_tokens_grad(dout.to(dev()), off, order, grad)
    bad = torch.isnan(grad.cpu())
    assert bad[4].all() and not bad[[0, 1, 2, 3, 5]].any()


def test_offsets_and_order_of_other_making(tide):
    """Offsets outside the tokens are clamped, falling ones leave a row empty, an
    order outside the tokens adds nothing."""
    T, V, D = 100, 6, 24
    dout = ref.normal((T, D), F32, 2)
    off = torch.tensor([-5, 10, 90, 40, 200, 250, 2 ** 31 - 1], dtype=torch.int32)
    order = torch.randint(-20, 130, (T,), generator=torch.Generator().manual_seed(1)).to(torch.int32)
    order[:3] = torch.tensor([2 ** 31 - 1, -2 ** 31, T])
    grad = torch.full((V, D), 5.0, device=dev())
    tide.embed_tokens_grad(dout.to(dev()), off.to(dev()), order.to(dev()), grad)
    want, lim = step.table_grad(dout, off, order, V, 1.0)
    ref.close(grad, want, lim + step.U * want.abs(), "clamped")


@pytest.mark.parametrize("T", [17, 700, 5000, 17000])
@pytest.mark.parametrize("more", [False, True])
def test_offsets_that_do_not_rise(tide, T, more):
    """Rows that overlap, that are empty or that go back, over chunks of the order:
    each is the sum of its own places."""
    g = torch.Generator().manual_seed(T)
    V, D = 40, 40
    off = torch.randint(-50, T + 50, (V + 1,), generator=g).to(torch.int32)
    off[10:20] = torch.sort(off[10:20]).values
    off[20:25] = T // 3
    order = torch.randint(-5, T + 5, (T,), generator=g).to(torch.int32)
    dout, old = ref.whole((T, D), 9, T).float(), ref.whole((V, D), 9, 3).float()
    padded = torch.cat([dout.double(), torch.zeros(1, D, dtype=torch.float64)])
    rows = padded[torch.where((order >= 0) & (order < T), order.long(), T)]
    want = torch.stack([rows[max(int(off[v]), 0): max(min(int(off[v + 1]), T), 0)].sum(0)
                        for v in range(V)]) + (old.double() if more else 0.0)
    grad = old.to(dev()).clone()
    tide.embed_tokens_grad(dout.to(dev()), off.to(dev()), order.to(dev()), grad, accumulate=more)
    assert torch.equal(grad.cpu().double(), want)


def test_large_offsets(tide):
    """Rows past 2^31 elements, in the table and in its gradient."""
    V, D = 1 << 19, 4104
    table = torch.zeros(V, D, dtype=BF16, device=dev())
    ids = torch.tensor([0, V - 1, 5, V - 1, V // 2])
    row = ref.normal((5, D), BF16, 4)
    for i in range(5):
        table[ids[i]] = row[i].to(dev())
    out = torch.empty(5, D, dtype=BF16, device=dev())
    tide.embed_tokens(ids.to(dev()), table, out)
    assert torch.equal(out, table[ids.to(dev())])
    off, order = sort(tide, ids, V)
    tide.embed_tokens_grad(row.to(dev()), off, order, table)
    for i, rows in ((0, [0]), (V - 1, [1, 3]), (5, [2]), (V // 2, [4])):
        want = row[rows].double().sum(0)
        ref.close(table[i], want, (2.0 ** -8 + 4 * step.U) * want.abs() + 4 * step.U * row[rows].double().abs().sum(0), str(i))
    assert not table[V - 2].any() and not table[1].any() and not table[V // 2 + 1].any()
