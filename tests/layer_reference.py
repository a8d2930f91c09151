"""The training-layer operators by their definitions, in 64 bits on the CPU
(torch and numpy only; none of the library's code), and seeded inputs for them.

Roundings are bounded by half a step: 2^-8 of the value for bf16, 2^-24 for
fp32, 2^-4 for e4m3."""
import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BLOCK = 32


def route(experts, E):
    """(offsets, token_of_row without the rows behind the last, slots)."""
    ids = np.asarray(experts)
    T, k = ids.shape
    flat = ids.reshape(-1)
    rows = [(int(e), i) for i, e in enumerate(flat) if 0 <= e < E]
    rows.sort()
    offsets = np.zeros(E + 1, np.int64)
    for e, _ in rows:
        offsets[e + 1] += 1
    slots = np.full(T * k, -1, np.int64)
    for p, (_, i) in enumerate(rows):
        slots[i] = p
    tokens = np.array([i // k for _, i in rows], np.int64)
    return np.cumsum(offsets), tokens, slots.reshape(T, k)


def combine(rows, slots, weights):
    """(sum, sum of magnitudes) in 64 bits; pairs without a row add nothing."""
    T, k = slots.shape
    out = torch.zeros(T, rows.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(out)
    for j in range(k):
        there = torch.nonzero((slots[:, j] >= 0) & (slots[:, j] < rows.shape[0])).reshape(-1)
        v = rows[slots[there, j].long()].double()
        if weights is not None:
            v = v * weights[there, j].double()[:, None]
        out[there] += v
        mag[there] += v.abs()
    return out, mag


def scale_exponents(x):
    """Exponent of each 32-element block of a row: the least e in [-117, 119]
    with amax <= 448 * 2^e over the finite elements (119 where none is)."""
    n, D = x.shape
    nb = -(-D // BLOCK)
    v = np.zeros((n, nb * BLOCK))
    v[:, :D] = x.double().numpy()
    v[~np.isfinite(v)] = 0
    top = np.abs(v).reshape(n, nb, BLOCK).max(-1)
    e = np.full(top.shape, -117, np.int64)
    for c in range(-117, 119):
        e = np.where(top > 448.0 * 2.0 ** c, c + 1, e)
    return e


def e4m3(q):
    """Nearest e4m3 value of |q| <= 448, ties to even, in 64 bits."""
    a = np.abs(q)
    ex = np.floor(np.log2(np.maximum(a, 2.0 ** -40)))
    ex = np.maximum(ex, -6.0)
    step = 2.0 ** (ex - 3)
    return np.sign(q) * np.rint(a / step) * step


def pack(x):
    """(code values, exponents): what the codes stand for before the scale."""
    n, D = x.shape
    e = scale_exponents(x)
    s = np.repeat(2.0 ** e.astype(np.float64), BLOCK, 1)[:, :D]
    v = x.double().numpy()
    fine = np.isfinite(v)
    q = e4m3(np.clip(np.where(fine, v, 0.0) / s, -448.0, 448.0))
    return np.where(fine, q, np.nan), e


def unpack(codes, scales):
    b = scales.view(torch.uint8).double()
    s = torch.exp2(b - 127).repeat_interleave(BLOCK, 1)[:, : codes.shape[1]]
    return codes.float().double() * s


def saved_of(x):
    """A checkpoint (codes, scales) on the CPU, from the definition."""
    q, e = pack(x)
    codes = torch.from_numpy(q).float().to(torch.float8_e4m3fn)
    scales = torch.from_numpy((e + 127).astype(np.uint8)).view(torch.float8_e8m0fnu)
    return codes, scales


def gated(g, u):
    g, u = g.double(), u.double()
    return g / (1 + torch.exp(-g)) * u


def gated_grad(d, g, u):
    """(dgate, dup, out, magnitude of dgate's two terms)."""
    d, g, u = d.double(), g.double(), u.double()
    s = 1 / (1 + torch.exp(-g))
    c = 1 / (1 + torch.exp(g))
    return d * u * (s + g * s * c), d * g * s, g * s * u, (d * u).abs() * (s + (g * s * c).abs())


def weight_grads(dy, x, offsets, tokens):
    """(gradients, sums of magnitudes, rows of each expert)."""
    dy, x = dy.double(), x.double()
    out, mag, cnt = [], [], []
    for e in range(len(offsets) - 1):
        r = torch.arange(int(offsets[e]), int(offsets[e + 1]))
        t = r if tokens is None else tokens[r].long()
        keep = (t >= 0) & (t < x.shape[0])
        a, b = dy[r[keep]], x[t[keep]]
        out.append(a.t() @ b)
        mag.append(a.abs().t() @ b.abs())
        cnt.append(int(keep.sum()))
    return torch.stack(out), torch.stack(mag), cnt


def experts(T, k, E, seed, masked=0.0, dtype=torch.int64):
    """Router-like ids: k different experts a token, some tokens with none."""
    g = torch.Generator().manual_seed(seed)
    score = torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g)
    ids = torch.topk(score, min(k, E), 1).indices
    if k > E:
        ids = torch.cat([ids, ids[:, : k - E]], 1)          # the same expert again
    ids[torch.rand(T, generator=g) < masked] = -1
    return ids.to(dtype)


def normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def close(got, want, bound, what=""):
    """|got - want| <= bound, elementwise, in 64 bits; NaN and infinities alike."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    off = (got - want).abs()[fine]
    lim = (bound + torch.zeros_like(want))[fine]
    bad = off > lim
    assert not bad.any(), "%s: %d of %d past the bound, worst %.3g over %.3g" % (
        what, int(bad.sum()), bad.numel(), float(off[bad].max()), float(lim[bad].min()))


def whole(shape, most, seed):
    """Whole numbers from -most to most as bf16 (exact up to 256)."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).to(torch.bfloat16)


def rounded_sum(dy, x, offsets, tokens, old=None):
    """Gradients of whole numbers below 2^24 in all: fp32 sums are exact in any
    order, so the result is the exact sum rounded once to bf16."""
    want, mag, _ = weight_grads(dy, x, offsets, tokens)
    if old is not None:
        want = want + old.double()
    assert float(mag.max()) + 256 < 2 ** 24
    return want.float().to(torch.bfloat16)
