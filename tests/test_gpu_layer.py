"""The training-layer operators together, as one mixture-of-experts layer's step
runs them, up to the reduce-scatter that reads their gradients; and captured,
replayed, on side streams and on two streams at once."""
import numpy as np
import pytest
import torch

import layer_reference as ref
from gpu_util import bits_of, dev, same_f32

pytestmark = pytest.mark.gpu
E4M3, E8M0, BF16 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.bfloat16


@pytest.fixture(scope="module")
def tide():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixed_precision_rs_amd as t
    return t


def saved(n, D):
    return torch.zeros(n, D, dtype=E4M3, device=dev()), torch.zeros(n, -(-D // 32), dtype=torch.uint8, device=dev()).view(E8M0)


class Layer:
    """Buffers of one layer's step and the calls between its matrix products."""

    def __init__(self, tide, T, k, E, H, F, seed, masked=0.1):
        self.tide, self.dims = tide, (T, k, E, H, F)
        n = T * k
        z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device=dev())  # noqa: E731
        self.fill(seed, masked)
        self.off, self.tok, self.slots = z(E + 1, dt=torch.int32), z(n, dt=torch.int32), z(T, k, dt=torch.int32)
        self.rows, self.h, self.y = z(n, H), z(n, F), z(n, H)
        self.out, self.dy, self.dw = z(T, H), z(n, H), z(T, k, dt=torch.float32)
        self.dg, self.du, self.h2, self.dx = z(n, F), z(n, F), z(n, F), z(T, H)
        self.xs, self.gs, self.us = saved(T, H), saved(n, F), saved(n, F)
        self.wg, self.wu, self.wd = z(E, F, H), z(E, F, H), z(E, H, F)

    def fill(self, seed, masked=0.1):
        T, k, E, H, F = self.dims
        new = {
            "ids": ref.experts(T, k, E, seed=seed, masked=masked), "x": ref.normal((T, H), BF16, seed),
            "w": torch.softmax(ref.normal((T, k), torch.float32, seed + 1), 1), "dout": ref.normal((T, H), BF16, seed + 2),
            # what the products between the calls give
            "g": ref.normal((T * k, F), BF16, seed + 3, 2.0), "u": ref.normal((T * k, F), BF16, seed + 4),
            "yp": ref.normal((T * k, H), BF16, seed + 5), "dh": ref.normal((T * k, F), BF16, seed + 6),
            "dxr": ref.normal((T * k, H), BF16, seed + 7)}
        for name, t in new.items():
            if hasattr(self, name):
                getattr(self, name).copy_(t)
            else:
                setattr(self, name, t.to(dev()))

    def step(self, stream=None):
        t, E = self.tide, self.dims[2]
        kw = {} if stream is None else {"stream": stream}
        t.route_tokens(self.ids, E, self.off, self.tok, self.slots, **kw)
        t.dispatch_tokens(self.x, self.slots, self.rows, **kw)
        t.checkpoint_pack(self.x, self.xs, **kw)
        t.gated_silu(self.g, self.u, self.h, gate_saved=self.gs, up_saved=self.us, **kw)
        t.combine_tokens(self.yp, self.slots, self.out, weights=self.w, **kw)
        t.combine_tokens_grad(self.dout, self.yp, self.slots, self.w, self.dy, self.dw, **kw)
        t.gated_silu_grad(self.dh, self.gs, self.us, self.dg, self.du, out=self.h2, **kw)
        t.weight_grads_bf16(self.dy, self.h2, self.wd, offsets=self.off, **kw)
        t.weight_grads_bf16(self.dg, self.xs, self.wg, offsets=self.off, token_of_row=self.tok, **kw)
        t.weight_grads_bf16(self.du, self.xs, self.wu, offsets=self.off, token_of_row=self.tok, **kw)
        t.combine_tokens(self.dxr, self.slots, self.dx, **kw)

    def results(self):
        return [t.clone() for t in (self.off, self.slots, self.rows, self.xs[0].view(torch.uint8), self.h, self.out,
                                    self.dy, self.dw, self.dg, self.du, self.h2, self.wd, self.wg, self.wu, self.dx)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_layer_step_and_the_reduce_scatter_of_its_gradients(tide, orc):
    """Every result of the step against the definition applied to the step's own
    inputs; then two contributors' gradients, where they lie, through the
    reduce-scatter, bit for bit against the oracle."""
    T, k, E, H, F = 200, 3, 6, 96, 136
    layers = [Layer(tide, T, k, E, H, F, seed) for seed in (1, 50)]
    for L in layers:
        L.step()
        cpu = lambda t: t.cpu()  # noqa: E731
        off, tok, slots = ref.route(cpu(L.ids).numpy(), E)
        assert np.array_equal(cpu(L.off), off) and np.array_equal(cpu(L.slots), slots)
        n, hs = int(off[-1]), cpu(L.slots)
        assert torch.equal(cpu(L.rows)[:n], cpu(L.x)[torch.from_numpy(tok)])
        want, mag = ref.combine(cpu(L.yp), hs, cpu(L.w))
        ref.close(L.out, want, 2.0 ** -8 * want.abs() + (k + 1) * 2.0 ** -24 * mag, "out")
        want, mag = ref.combine(cpu(L.dxr), hs, None)
        ref.close(L.dx, want, 2.0 ** -8 * want.abs() + (k + 1) * 2.0 ** -24 * mag, "dx")
        want = ref.gated(cpu(L.g), cpu(L.u))
        ref.close(L.h, want, (2.0 ** -8 + 2.0 ** -20) * want.abs(), "h")
        g, u = ref.unpack(*map(cpu, L.gs)), ref.unpack(*map(cpu, L.us))
        dg, du, h, mag = ref.gated_grad(cpu(L.dh), g, u)
        ref.close(L.dg, dg, 2.0 ** -8 * dg.abs() + 2.0 ** -20 * mag, "dg")
        ref.close(L.du, du, (2.0 ** -8 + 2.0 ** -20) * du.abs(), "du")
        ref.close(L.h2, h, (2.0 ** -8 + 2.0 ** -20) * h.abs(), "h again")
        o, t = torch.from_numpy(off), torch.from_numpy(tok)
        t = torch.cat([t, torch.full((T * k - n,), -1, dtype=t.dtype)])
        x = ref.unpack(*map(cpu, L.xs))
        for got, dy, xx, tt in ((L.wd, L.dy, cpu(L.h2), None), (L.wg, L.dg, x, t), (L.wu, L.du, x, t)):
            want, mag, cnt = ref.weight_grads(cpu(dy), xx, o, tt)
            for e in range(E):
                ref.close(got[e], want[e], 2.0 ** -8 * want[e].abs() + (cnt[e] + 2) * 2.0 ** -23 * mag[e], "expert")
    shapes = [(F, H), (F, H), (H, F)] * E
    grads = [[t for e in range(E) for t in (L.wg[e], L.wu[e], L.wd[e])] for L in layers]
    N = 5
    plan = tide.plan_create(shapes, N, 2)
    out = torch.full((N * plan.S,), float("nan"), device=dev())
    tide.reduce_scatter_bf16_fp32(plan, grads, out)
    host = [[bits_of(t) for t in g] for g in grads]
    same_f32(out.cpu().numpy(), orc.reduce_scatter(shapes, N, 2, host).reshape(-1), "shards")


def test_captured_and_replayed(tide):
    """The whole step in one graph, replayed on new inputs with eager work and
    waits between; every replay against the eager results."""
    eager, L = (Layer(tide, 300, 4, 16, 64, 96, 3) for _ in range(2))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        L.step()                                        # before the capture: nothing is first used in it
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        L.step()
    for seed in (3, 21, 22, 3, 40):
        for layer in (eager, L):
            layer.fill(seed)
            for t in (layer.rows, layer.dy):
                t.zero_()
        for t in (L.out, L.wg, L.wu, L.wd, L.dw):
            t.fill_(7.0)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert same(L.results(), eager.results()), seed


def test_two_graphs_with_split_sums_share_nothing(tide):
    """Two captured weight gradients whose rows are split keep a workspace
    each; replayed on two streams at once they give the eager bits."""
    n, O, I = 6000, 128, 128
    assert tide.weight_grads_workspace_bytes(n, O, I) > 0
    put = lambda s: (ref.normal((n, O), BF16, s).to(dev()), ref.normal((n, I), BF16, s + 1).to(dev()),  # noqa: E731
                     torch.zeros(1, O, I, dtype=BF16, device=dev()))
    sets, want, graphs = [put(1), put(9)], [], []
    streams = [torch.cuda.Stream() for _ in sets]
    for (dy, x, g), s in zip(sets, streams):
        tide.weight_grads_bf16(dy, x, g)
        want.append(g.clone())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            tide.weight_grads_bf16(dy, x, g)
        graphs.append(graph)
    for _ in range(10):
        for _, _, g in sets:
            g.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for (_, _, g), w in zip(sets, want))


@pytest.mark.parametrize("how", ["argument", "handle", "current"])
def test_on_side_streams_at_once(tide, how):
    """Two layers' steps on two streams, interleaved call by call by the GPU."""
    a, b = Layer(tide, 500, 4, 32, 128, 160, 5), Layer(tide, 333, 2, 8, 96, 64, 6)
    want = []
    for L in (a, b):
        L.step()
        torch.cuda.synchronize()
        want.append(L.results())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for L in (a, b):
            for t in (L.out, L.wg, L.wu, L.wd, L.rows, L.dy):
                t.zero_()
        torch.cuda.synchronize()
        for L, s in zip((a, b), streams):
            if how == "argument":
                L.step(stream=s)
            elif how == "handle":
                L.step(stream=int(s.cuda_stream))
            else:
                with torch.cuda.stream(s):
                    L.step()
        torch.cuda.synchronize()
        for L, w in zip((a, b), want):
            assert same(L.results(), w)


@pytest.mark.parametrize("null", [False, True])
def test_workspace_on_a_stream_handle(tide, null):
    """A call that allocates its workspace on a raw stream handle, also the null stream's."""
    n, O, I, T = 6000, 128, 128, 3000
    dy, x = ref.normal((n, O), BF16, 1).to(dev()), ref.normal((n, I), BF16, 2).to(dev())
    want, got = (torch.zeros(1, O, I, dtype=BF16, device=dev()) for _ in range(2))
    ids = ref.experts(T, 4, 16, seed=5).to(dev())
    outs = [[torch.zeros(s, dtype=torch.int32, device=dev()) for s in (17, T * 4, (T, 4))] for _ in range(2)]
    tide.weight_grads_bf16(dy, x, want)
    tide.route_tokens(ids, 16, *outs[0])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    handle = 0 if null else int(s.cuda_stream)
    for _ in range(3):
        got.zero_()
        torch.cuda.synchronize()
        tide.weight_grads_bf16(dy, x, got, stream=handle)
        tide.route_tokens(ids, 16, *outs[1], stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(*outs))


def test_x_without_rows(tide):
    """Every token out of range of an x that has no rows: zeros."""
    g = torch.full((2, 16, 24), 5.0, dtype=BF16, device=dev())
    off = torch.tensor([0, 3, 7], dtype=torch.int32, device=dev())
    tok = torch.full((7,), -1, dtype=torch.int32, device=dev())
    dy = torch.full((7, 16), float("nan"), dtype=BF16, device=dev())
    for x in (torch.empty(0, 24, dtype=BF16, device=dev()), saved(0, 24)):
        g.fill_(5.0)
        tide.weight_grads_bf16(dy, x, g, offsets=off, token_of_row=tok)
        assert (g.cpu() == 0).all()


def test_refused_on_the_gpu(tide):
    """Refusals that need GPU tensors: other types, sizes, overlaps, strides."""
    z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device=dev())  # noqa: E731
    x, slots, rows = z(4, 64), torch.full((4, 2), -1, dtype=torch.int32, device=dev()), z(8, 64)
    with pytest.raises(TypeError):
        tide.dispatch_tokens(z(4, 64, dt=torch.float16), slots, rows)
    with pytest.raises(TypeError):
        tide.dispatch_tokens(x, slots, rows.float())
    with pytest.raises(TypeError):
        tide.dispatch_tokens(x, slots.long(), rows)
    with pytest.raises(ValueError):
        tide.dispatch_tokens(x, slots[:3], rows)
    with pytest.raises(ValueError):
        tide.dispatch_tokens(x, slots, z(8, 63))
    with pytest.raises(ValueError):
        tide.dispatch_tokens(x[:, ::2], slots, z(8, 32))
    with pytest.raises(ValueError):
        tide.dispatch_tokens(x[:1].expand(4, 64), slots, rows)
    with pytest.raises(ValueError, match="not a GPU tensor"):
        tide.dispatch_tokens(x, slots.cpu(), rows)
    with pytest.raises(ValueError, match="not a GPU tensor"):
        tide.dispatch_tokens(x.cpu(), slots, rows)
    with pytest.raises(tide.TideError, match="overlaps"):
        tide.dispatch_tokens(rows[:4], slots, rows)
    with pytest.raises(ValueError, match="dweights needs rows"):
        tide.combine_tokens_grad(x, None, slots, None, rows, z(4, 2, dt=torch.float32))
    with pytest.raises(TypeError):
        tide.combine_tokens(rows, slots, x, weights=z(4, 2))
    with pytest.raises(TypeError):
        tide.route_tokens(z(4, 2, dt=torch.int16), 8, z(9, dt=torch.int32), z(8, dt=torch.int32), z(4, 2, dt=torch.int32))
    with pytest.raises(ValueError):
        tide.route_tokens(z(4, 2, dt=torch.int32), 8, z(8, dt=torch.int32), z(8, dt=torch.int32), z(4, 2, dt=torch.int32))
    with pytest.raises(tide.TideError, match="UNSUPPORTED"):
        tide.route_tokens(z(4, 2, dt=torch.int32), 600, z(601, dt=torch.int32), z(8, dt=torch.int32),
                          z(4, 2, dt=torch.int32))
    c, s = saved(4, 64)
    with pytest.raises(ValueError):
        tide.checkpoint_pack(x, (c, s[:, :1]))
    with pytest.raises(TypeError):
        tide.checkpoint_pack(x, (c.view(torch.uint8), s))
    with pytest.raises(tide.TideError, match="overlaps"):
        tide.gated_silu(x, x, x)
    with pytest.raises(tide.TideError, match="overlaps"):
        tide.gated_silu(x, x, z(4, 64), gate_saved=(c, s), up_saved=(c, s))
    dy, xx = z(10, 16), z(10, 24)
    with pytest.raises(tide.TideError, match="need offsets"):
        tide.weight_grads_bf16(dy, xx, z(2, 16, 24))
    with pytest.raises(ValueError):
        tide.weight_grads_bf16(dy, xx, z(1, 24, 16))
    with pytest.raises(ValueError):
        tide.weight_grads_bf16(dy, xx, z(2, 16, 24), offsets=z(2, dt=torch.int32))
    with pytest.raises(TypeError):
        tide.weight_grads_bf16(dy.float(), xx, z(1, 16, 24))
    with pytest.raises(tide.TideError, match="x has 9 rows"):
        tide.weight_grads_bf16(dy, xx[:9], z(1, 16, 24))
    g = z(16, 24)
    with pytest.raises(tide.TideError, match="overlap"):
        tide.weight_grads_bf16(dy, xx, [g, g], offsets=z(3, dt=torch.int32))


def test_list_of_transposed_gradients_is_refused(tide):
    dy, x = (torch.ones(10, c, dtype=BF16, device=dev()) for c in (16, 24))
    g = torch.full((24, 16), 3.0, dtype=BF16, device=dev())
    for grads in (g, g[None], [g], [g.view(-1)]):
        with pytest.raises(ValueError, match="shape"):
            tide.weight_grads_bf16(dy, x, grads)
    assert (g.cpu() == 3.0).all()
    tide.weight_grads_bf16(dy, x, [g.view(16, 24)])
    assert (g.cpu() == 10.0).all()


def test_an_earlier_error_of_the_caller_is_not_reported(tide):
    """An error that the program's own HIP call left behind is neither reported as
    a layer call's nor taken from the program."""
    import ctypes
    with open("/proc/self/maps") as f:
        hip = ctypes.CDLL(next(line.split()[-1] for line in f if "libamdhip64" in line))
    L = Layer(tide, 40, 2, 4, 64, 32, 7)
    L.step()
    torch.cuda.synchronize()
    want = L.results()
    bad = hip.hipSetDevice(1 << 20)                      # refused by the runtime on the host
    assert bad != 0
    try:
        L.step()
        left = hip.hipGetLastError()
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert left == bad and same(L.results(), want)
