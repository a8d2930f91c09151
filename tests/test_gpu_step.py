"""The operators of a step's ends together with the layer's and the collectives, as
a small model's training step runs them; captured, replayed, on side streams and
on two streams at once."""
import math

import pytest
import torch

import layer_reference as ref
import step_reference as step
from gpu_util import bits_of, dev, same_f32

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tide():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixed_precision_rs_amd as t
    return t


class Model:
    """Buffers of a step and the calls between its matrix products, whose results
    are inputs here: ids -> table rows; queries and keys normalised and rotated;
    logits -> log probabilities; their gradient -> the head's weight gradient (also
    the table's: they are tied), the norms' gradients, the lookups' added to it."""

    def __init__(self, tide, T, V, D, Hq, Hk, hd, seed):
        self.tide, self.dims = tide, (T, V, D, Hq, Hk, hd)
        z = lambda *s, dt=BF16: torch.zeros(*s, dtype=dt, device=dev())  # noqa: E731
        angle = torch.arange(T, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(hd // 2, dtype=torch.float64) / (hd // 2))
        self.cos, self.sin = torch.cos(angle).float().to(dev()), torch.sin(angle).float().to(dev())
        self.fill(seed)
        self.x, self.qo, self.ko = z(T, D), z(T, Hq, hd), z(T, Hk, hd)
        self.lp, self.st, self.H = z(T, dt=F32), z(T, 2, dt=F32), z(T, dt=F32)
        self.ids_top, self.lp_top = z(T, 3, dt=torch.int32), z(T, 3, dt=F32)
        self.dlogits, self.off, self.order = z(T, V), z(V + 1, dt=torch.int32), z(T, dt=torch.int32)
        self.dqkv = z(T, Hq + 2 * Hk, hd)
        self.gtable, self.gq, self.gk = z(V, D), z(hd), z(hd)
        self.total, self.norm = z(1, dt=torch.float64), z(1, dt=F32)
        self.clipped = [torch.zeros_like(t) for t in self.grads()]

    def grads(self):
        return [self.gtable, self.gq, self.gk]

    def fill(self, seed):
        T, V, D, Hq, Hk, hd = self.dims
        g = torch.Generator().manual_seed(seed)
        ids = torch.randint(-1, V, (T,), generator=g)
        ids[: T // 3] = seed % V                        # a word far more frequent than the others
        new = {
            "ids": ids, "targets": torch.where(torch.arange(T) % 4 == 0, -100, torch.randint(0, V, (T,), generator=g)),
            "table": ref.normal((V, D), BF16, seed), "qkv": ref.normal((T, Hq + 2 * Hk, hd), BF16, seed + 1),
            "qw": 1 + ref.normal((hd,), BF16, seed + 2, 0.1), "kw": 1 + ref.normal((hd,), BF16, seed + 3, 0.1),
            "h": ref.normal((T, D), BF16, seed + 4), "logits": ref.normal((T, V), BF16, seed + 5, 2.0),
            "dqo": ref.normal((T, Hq, hd), BF16, seed + 6), "dko": ref.normal((T, Hk, hd), BF16, seed + 7),
            "dx": ref.normal((T, D), BF16, seed + 8), "d": ref.normal((T,), F32, seed + 9),
            "positions": torch.arange(T).flip(0).to(torch.int32)}
        for name, t in new.items():
            if hasattr(self, name):
                getattr(self, name).copy_(t)
            else:
                setattr(self, name, t.to(dev()))

    def step(self, stream=None):
        t, (T, V, D, Hq, Hk, hd) = self.tide, self.dims
        kw = {} if stream is None else {"stream": stream}
        heads = lambda f: (f[:, :Hq], f[:, Hq: Hq + Hk])  # noqa: E731
        turn = dict(q_weight=self.qw, k_weight=self.kw, positions=self.positions, cos=self.cos, sin=self.sin, **kw)
        t.embed_tokens(self.ids, self.table, self.x, scale=math.sqrt(D), **kw)
        t.norm_rotate(*heads(self.qkv), self.qo, self.ko, **turn)
        t.token_logprobs(self.logits, self.targets, self.lp, stats=self.st, entropy=self.H, top_ids=self.ids_top, top_logprobs=self.lp_top, **kw)
        t.token_logprobs_grad(self.logits, self.targets, self.st, self.d, self.dlogits, **kw)
        t.weight_grads_bf16(self.dlogits, self.h, [self.gtable], **kw)
        t.norm_rotate_grad(self.dqo, self.dko, *heads(self.qkv), *heads(self.dqkv), dq_weight=self.gq, dk_weight=self.gk, **turn)
        t.sort_ids(self.ids, V, self.off, self.order, **kw)
        t.embed_tokens_grad(self.dx, self.off, self.order, self.gtable, scale=math.sqrt(D), accumulate=True, **kw)
        t.grad_squares(self.grads(), self.total, **kw)
        t.clip_grads(self.grads(), self.total, 1.0, out=self.clipped, norm=self.norm, **kw)

    def results(self):
        return [t.clone() for t in (self.x, self.qo, self.ko, self.lp, self.st, self.H, self.ids_top, self.lp_top, self.dlogits, self.off,
                                    self.dqkv, self.total, self.norm, *self.grads(), *self.clipped)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_step_and_the_collectives(tide, orc):
    """Every result against the definition applied to the step's own inputs; two
    contributors' gradients through the reduce-scatter, bit for bit against the
    oracle; the shards' norm and their clipping."""
    T, V, D, Hq, Hk, hd = 150, 40, 48, 4, 2, 16
    models = [Model(tide, T, V, D, Hq, Hk, hd, seed) for seed in (1, 50)]
    for m in models:
        m.step()
        cpu = lambda t: t.cpu()  # noqa: E731
        ids, targets = cpu(m.ids), cpu(m.targets)
        assert torch.equal(cpu(m.x), step.lookup(ids, cpu(m.table), torch.tensor(math.sqrt(D), dtype=F32)))
        where = (cpu(m.positions), cpu(m.cos), cpu(m.sin), 1e-6, False)
        for got, gd, gw, x, w, d in ((m.qo, m.dqkv[:, :Hq], m.gq, m.qkv[:, :Hq], m.qw, m.dqo),
                                     (m.ko, m.dqkv[:, Hq: Hq + Hk], m.gk, m.qkv[:, Hq: Hq + Hk], m.kw, m.dko)):
            want, lim = step.norm_rotate(cpu(x), cpu(w), *where)
            ref.close(got, want, lim + 2.0 ** -8 * want.abs(), "rotated")
            dx, lim, ww, lw = step.norm_rotate_grad(cpu(d), cpu(x), cpu(w), *where)
            ref.close(gd, dx, lim + 2.0 ** -8 * dx.abs(), "rotated gradient")
            ref.close(gw, ww, lw + 2.0 ** -8 * ww.abs(), "norm's weight")
        want = step.logprobs(cpu(m.logits), targets, 3)
        ref.close(m.lp, want["logprob"], want["d_logprob"], "logprob")
        ref.close(m.H, want["entropy"], want["d_entropy"], "entropy")
        assert torch.equal(cpu(m.ids_top), want["top_ids"])
        want, lim = step.logprobs_grad(cpu(m.logits), targets, cpu(m.st), cpu(m.d))
        ref.close(m.dlogits, want, lim + 2.0 ** -8 * want.abs(), "dlogits")
        # the table's gradient: the head's product, rounded to bf16, then the lookups added to it
        head, mag, _ = ref.weight_grads(cpu(m.dlogits), cpu(m.h), torch.tensor([0, T]), None)
        off, order = step.sort_ids(ids, V)
        assert cpu(m.off).tolist() == off.tolist()
        f = float(torch.tensor(math.sqrt(D), dtype=F32))
        want, lim = step.table_grad(cpu(m.dx), off, order, V, f, torch.zeros(V, D))
        first = 2.0 ** -8 * head[0].abs() + (T + 2) * 2.0 ** -23 * mag[0]
        ref.close(m.gtable, want + head[0], lim.clamp(min=0) + first + step.U * 4 * head[0].abs() + 2.0 ** -8 * ((want + head[0]).abs() + first),
                  "table")
        total = step.squares([cpu(t) for t in m.grads()])
        assert abs(float(m.total) - total) <= 1e-12 * total
        for t, c in zip(m.grads(), m.clipped):
            v, lim = step.clipped(cpu(t), float(m.total), 1.0)
            ref.close(c, v, lim + 2.0 ** -8 * v.abs(), "clipped")
    shapes = [(V, D), (hd, 1), (hd, 1)]
    N = 4
    plan = tide.plan_create(shapes, N, 2)
    out = torch.full((N * plan.S,), float("nan"), device=dev())
    tide.reduce_scatter_bf16_fp32(plan, [m.grads() for m in models], out)
    want = orc.reduce_scatter(shapes, N, 2, [[bits_of(t) for t in m.grads()] for m in models]).reshape(-1)
    same_f32(out.cpu().numpy(), want, "shards")
    # each rank its own shard; the ranks' totals added up, as an all-reduce would
    totals = []
    for r in range(N):
        t = torch.empty(1, dtype=torch.float64, device=dev())
        tide.grad_squares(out[r * plan.S: (r + 1) * plan.S], t)
        totals.append(t)
    total = torch.stack(totals).sum(0)
    exact = step.squares([torch.from_numpy(want)])
    assert abs(float(total) - exact) <= 1e-12 * exact
    before = out.clone()
    for r in range(N):
        tide.clip_grads(out[r * plan.S: (r + 1) * plan.S], total, 0.5)
    v, lim = step.clipped(before.cpu(), float(total), 0.5)
    ref.close(out, v, lim, "clipped shards")


def test_captured_and_replayed(tide):
    """The whole step in one graph, replayed on new inputs with eager work and
    waits between; every replay against the eager results."""
    dims = (300, 700, 64, 4, 1, 32)
    eager, m = Model(tide, *dims, 3), Model(tide, *dims, 3)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        m.step()                                        # before the capture: nothing is first used in it
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        m.step()
    for seed in (3, 21, 22, 3, 40):
        for one in (eager, m):
            one.fill(seed)
            one.order.zero_()
        for t in (*m.results(), m.x, m.gtable, m.gq, m.gk, m.lp, m.total, *m.clipped):
            t.fill_(7)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert same(m.results(), eager.results()), seed


def test_two_graphs_and_two_streams_share_nothing(tide):
    """Two captured steps, replayed on two streams at once, and two eager ones: the
    bits of each alone."""
    dims = (5000, 300, 40, 2, 1, 64)                    # a sort of several workgroups, long rows
    alone = []
    models = [Model(tide, *dims, seed) for seed in (5, 9)]
    for m in models:
        m.step()
        torch.cuda.synchronize()
        alone.append(m.results())
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for m, s in zip(models, streams):
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            m.step()
        graphs.append(g)
    for turn in range(4):
        for m in models:
            for t in (m.gtable, m.gq, m.x, m.dlogits, m.total):
                t.fill_(7)
        torch.cuda.synchronize()
        for m, s, g in zip(models, streams, graphs):
            with torch.cuda.stream(s):
                if turn % 2:
                    g.replay()
                else:
                    m.step()
        torch.cuda.synchronize()
        for m, want in zip(models, alone):
            assert same(m.results(), want), turn


def test_given_streams_and_raw_handles(tide):
    dims = (200, 100, 32, 2, 1, 16)
    m = Model(tide, *dims, 4)
    m.step()
    torch.cuda.synchronize()
    want = m.results()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        for t in (m.gtable, m.gq, m.x, m.dlogits, m.total):
            t.fill_(7)
        torch.cuda.synchronize()
        m.step(stream=stream)
        torch.cuda.synchronize()
        assert same(m.results(), want), stream


def test_refused_calls_on_gpu_tensors(tide):
    """What the binding refuses of real tensors, and that nothing was written."""
    d = dev()
    ids, table = torch.zeros(4, dtype=torch.int64, device=d), torch.zeros(8, 16, dtype=BF16, device=d)
    out = torch.full((4, 16), 5.0, dtype=BF16, device=d)
    with pytest.raises(ValueError, match="not adjacent"):
        tide.embed_tokens(ids, torch.zeros(16, 8, dtype=BF16, device=d).t(), out)
    with pytest.raises(ValueError, match="expected 4 x 16"):
        tide.embed_tokens(ids, table, out[:3])
    with pytest.raises(TypeError):
        tide.embed_tokens(ids, table, out.float())
    with pytest.raises(TypeError):
        tide.embed_tokens(ids.to(torch.int16), table, out)
    with pytest.raises(tide.TideError, match="overlaps"):
        tide.embed_tokens(ids, table, table[:4])
    logits, lp = torch.zeros(4, 10, device=d), torch.zeros(4, device=d)
    with pytest.raises(ValueError, match="go together"):
        tide.token_logprobs(logits, ids, lp, top_ids=torch.zeros(4, 2, dtype=torch.int32, device=d))
    with pytest.raises(tide.TideError, match="UNSUPPORTED"):
        tide.token_logprobs(logits, ids, lp, top_ids=torch.zeros(4, 33, dtype=torch.int32, device=d), top_logprobs=torch.zeros(4, 33, device=d))
    with pytest.raises(ValueError, match="needs entropy"):
        tide.token_logprobs_grad(logits, ids, torch.zeros(4, 2, device=d), lp, logits, dentropy=lp)
    with pytest.raises(ValueError, match="other sizes"):
        tide.clip_grads([lp], torch.ones(1, dtype=torch.float64, device=d), 1.0, out=[lp[:3]])
    with pytest.raises(TypeError):
        tide.grad_squares([lp, out], torch.ones(1, dtype=torch.float64, device=d))
    with pytest.raises(tide.TideError, match="overlaps"):
        tide.clip_grads([lp, lp], torch.ones(1, dtype=torch.float64, device=d), 1.0)
    assert (out == 5.0).all() and not lp.any()
