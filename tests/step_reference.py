"""The operators at the ends of a training step and in front of its attention, by
their definitions, in 64 bits on the CPU (torch, numpy and the standard library;
none of the library's code), with bounds on what fp32 arithmetic may add.

u = 2^-24 is half a step of fp32. A function that returns a bound returns what the
arithmetic before the last rounding may be off by; the last rounding to bf16 adds
2^-8 of the value, to fp32 2^-24."""
import math

import numpy as np
import torch

from layer_reference import HALF  # noqa: F401

U = 2.0 ** -24


# ------------------------------------------------------------------ embedding

def sort_ids(ids, V):
    """(offsets, order): places of the ids in [0, V), stable."""
    flat = [int(i) for i in ids]
    order = sorted((t for t, i in enumerate(flat) if 0 <= i < V), key=lambda t: flat[t])
    count = np.zeros(V + 1, np.int64)
    for t in order:
        count[flat[t] + 1] += 1
    return np.cumsum(count), np.array(order, np.int64)


def lookup(ids, table, scale):
    """Exact: one product in fp32, rounded once to the table's type."""
    out = torch.zeros(len(ids), table.shape[1], dtype=table.dtype)
    for t, i in enumerate(int(i) for i in ids):
        if 0 <= i < table.shape[0]:
            out[t] = (table[i].float() * scale).to(table.dtype)
    return out


def table_grad(dout, offsets, order, V, scale, old=None):
    """(gradient, bound): a row of c tokens has c additions, a product, and one
    addition to what was there, each off by u of at most the sum of magnitudes."""
    T, D = dout.shape
    want, lim = torch.zeros(V, D, dtype=torch.float64), torch.zeros(V, D, dtype=torch.float64)
    for v in range(V):
        lo, hi = max(int(offsets[v]), 0), min(int(offsets[v + 1]), T)
        rows = [int(t) for t in order[lo:hi] if 0 <= int(t) < T] if lo < hi else []
        d = dout[rows].double() * scale
        want[v], mag = d.sum(0), d.abs().sum(0)
        if old is not None:
            want[v] += old[v].double()
            mag = mag + old[v].double().abs()
        lim[v] = (len(rows) + 2) * U * mag
        if old is not None and lo >= hi:
            lim[v] = -1.0                       # not touched: equal
    return want, lim


# ---------------------------------------------------------- log probabilities

def logprobs(x, targets, top=0):
    """dict of logprob, m, log_s, entropy, top_ids, top_logprobs and the bounds
    d_logprob, d_log_s, d_entropy, d_top.

    exp(x - m) is off by the rounding of x - m (u |z|), of the product with log2(e)
    and that constant (1.5 u |z|) and of the instruction (2 u). With 64 lanes a row or
    more, a sum takes at most V / 64 additions, and is brought to a new maximum at
    most once for each, each time off by the same as one exp at the rise, the rises
    adding up to at most the row's range; ten joins. So s is off by at most delta =
    (V / 64 * 4 + 30 + 5 range) u, range cut at 200, where exp is 0."""
    x = x.double()
    T, V = x.shape
    out = {k: [] for k in ("logprob", "m", "log_s", "entropy", "top_ids", "top_logprobs", "d_logprob", "d_log_s",
                           "d_entropy", "d_top")}
    for r in range(T):
        row, t = x[r], int(targets[r])
        bad = bool(torch.isnan(row).any() or (row == math.inf).any())
        some = row[row > -math.inf] if V else row
        m = float(some[~torch.isnan(some)].max()) if some.numel() and not torch.isnan(some).all() else -math.inf
        if bad:
            log_s = H = math.nan
            delta, Ez = 0.0, 0.0
        elif not some.numel():
            m = log_s = -math.inf
            H, delta, Ez = 0.0, 0.0, 0.0
        else:
            z = some - m
            e = torch.exp(z)
            s = float(e.sum())
            log_s = math.log(s)
            Ez = float((e * z.abs()).sum()) / s
            H = log_s + Ez
            span = min(float(some.max() - some.min()), 200.0)
            delta = (V / 16 + 30 + 5 * span) * U
        of = lambda v: math.nan if bad else -math.inf if m == -math.inf else v - m - log_s  # noqa: E731
        room = lambda v: delta + 4 * U * (abs(log_s) + abs(v - m)) if math.isfinite(of(v)) else 0.0  # noqa: E731
        inside = 0 <= t < V
        out["logprob"].append(of(float(row[t])) if inside else 0.0)
        out["d_logprob"].append(room(float(row[t])) if inside else 0.0)
        out["m"].append(m)
        out["log_s"].append(log_s)
        out["d_log_s"].append(delta + 4 * U * abs(log_s) if math.isfinite(log_s) else 0.0)
        out["entropy"].append(H)
        out["d_entropy"].append(0.0 if bad or m == -math.inf else delta * (1 + 3 * Ez) + 4 * U * (abs(log_s) + Ez))
        ids = [i for i in range(V) if float(row[i]) > -math.inf] if top else []
        ids = sorted(ids, key=lambda i: (-float(row[i]), i))[:top]
        out["top_ids"].append(ids + [-1] * (top - len(ids)))
        out["top_logprobs"].append([of(float(row[i])) for i in ids] + [-math.inf] * (top - len(ids)))
        out["d_top"].append([room(float(row[i])) for i in ids] + [0.0] * (top - len(ids)))
    kinds = {"top_ids": torch.int32}
    return {k: torch.tensor(v, dtype=kinds.get(k, torch.float64)).reshape((T, top) if "top" in k else (T,))
            for k, v in out.items()}


def logprobs_grad(x, targets, stats, d, H=None, h=None):
    """(gradient, bound) at the given stats. lp is off by 2 u (|x - m| + |log s|),
    p = exp(lp) by that and 2.5 u |lp| + 2 u of itself."""
    x, m, log_s = x.double(), stats[:, :1].double(), stats[:, 1:].double()
    T, V = x.shape
    lp = x - m - log_s
    p = torch.exp(lp)
    inside = (targets >= 0) & (targets < V)
    d = torch.where(inside, d.double(), 0.0)[:, None]
    want = -d * p
    lpf = torch.where(p > 0, lp, 0.0)
    off = 2.0 ** -21 * (1 + torch.where(p > 0, (x - m).abs() + log_s.abs(), 0.0))
    lim = off * d.abs() * p
    if h is not None:
        hh = h.double()[:, None]
        want = want - hh * p * (lpf + H.double()[:, None])
        lim = lim + off * hh.abs() * p * (1 + lpf.abs() + H.double()[:, None].abs())
    for r in range(T):
        if inside[r]:
            want[r, int(targets[r])] += d[r, 0]
            lim[r, int(targets[r])] += 2 * U * float(d[r, 0].abs())
        if not inside[r] and h is None or float(m[r]) == -math.inf:
            want[r] = 0.0
            lim[r] = 0.0
    return want, torch.nan_to_num(lim, 0.0, 0.0, 0.0)


# -------------------------------------------------------------- norm, rotation

def pair_index(D, pairs, adjacent):
    """(first, second) elements of each pair, the rotated ones first."""
    if adjacent:
        return list(range(0, D, 2)), list(range(1, D, 2))
    rest = D - 2 * pairs
    a = list(range(pairs)) + list(range(2 * pairs, 2 * pairs + rest // 2))
    b = list(range(pairs, 2 * pairs)) + list(range(2 * pairs + rest // 2, D))
    return a, b


def turn(x, cos, sin, at, adjacent, back=False):
    """Rotates (tokens, heads, D) by row at[t] of the tables (not where at[t] < 0);
    also what its terms add up to in magnitude."""
    if cos is None:
        return x, x.abs()
    T, _, D = x.shape
    pairs = cos.shape[1]
    a, b = pair_index(D, pairs, adjacent)
    c, s = torch.ones(T, D // 2, dtype=torch.float64), torch.zeros(T, D // 2, dtype=torch.float64)
    for t in range(T):
        if at[t] >= 0:
            c[t, :pairs], s[t, :pairs] = cos[at[t]].double(), sin[at[t]].double()
    c, s = c[:, None], (-s if back else s)[:, None]
    out, mag = x.clone(), x.abs()
    p, q = x[..., a], x[..., b]
    out[..., a], out[..., b] = p * c - q * s, p * s + q * c
    mag[..., a], mag[..., b] = (p * c).abs() + (q * s).abs(), (p * s).abs() + (q * c).abs()
    return out, mag


def rows_of(T, positions, cos):
    if cos is None:
        return [-1] * T
    p = range(T) if positions is None else [int(i) for i in positions]
    return [i if 0 <= i < cos.shape[0] else -1 for i in p]


def norm_rotate(x, w, positions, cos, sin, eps, adjacent):
    """(result, bound). A lane adds at most 16 squares and six exchanges join them
    (22 u), the mean, eps, the root and its inverse and two products: 20 u of each
    of a rotation's two terms covers them and the rotation."""
    x = x.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    out, mag = turn(y, cos, sin, rows_of(x.shape[0], positions, cos), adjacent)
    return out, 20 * U * mag


def norm_rotate_grad(dout, x, w, positions, cos, sin, eps, adjacent):
    """(dx, bound, dw, bound). g is off by 3 u of its terms' magnitudes G, n by 16
    u, the mean of g w n by 45 u of that of G w |n|: dx by 80 u of r (G w + |n|
    mean(G w |n|)), dw by u of the sum of G |n| for each of its additions."""
    x, d = x.double(), dout.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64) if w is None else w.double()
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    g, G = turn(d, cos, sin, rows_of(x.shape[0], positions, cos), adjacent, back=True)
    M = (G * w.abs() * n.abs()).mean(-1, keepdim=True)
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    count = x.shape[0] * x.shape[1]
    return dx, 80 * U * r * (G * w.abs() + n.abs() * M), (g * n).sum((0, 1)), (count + 40) * U * (G * n.abs()).sum((0, 1))


# ------------------------------------------------------------- norm, clipping

def squares(tensors):
    return math.fsum(float(v) * float(v) for t in tensors for v in t.reshape(-1).double().tolist())


def clipped(t, total, most):
    """(result, bound): the factor in 64 bits, the product rounded to fp32 (and, by
    the caller's allowance, to bf16)."""
    norm = math.sqrt(total)
    f = most / norm if most < norm < math.inf else 1.0
    want = t.double() * f
    return want, 2 * U * want.abs() + 2.0 ** -149
