"""The operators at the ends of a training step and in front of its attention, as cases for measurement.

Token ids looked up in the embedding table, and the table's gradient from tokens sorted by id; queries and keys
normalised head by head and rotated by position in one pass, and the gradient; log probabilities of given tokens with
entropy and the most probable alternatives, and the gradient to the logits; the gradient norm over many tensors, and
clipping by it. The gradients of the table and of the norms' weights are what the reduce-scatter reads, the clipped
tensors what it leaves. Layers are those of `workloads/configs.py` (width 2048 with 128 experts of 768, 32 heads of 128
for queries and 4 for keys; width 8192, 64 and 8 heads; width 5120), vocabularies are generic.

Each case runs in a plain form (elementary torch operations in 32 bits, 64 for the norm's long sums, rounded once) or,
where `own` is true, through the package's entry points."""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
IDS = {32: torch.int32, 64: torch.int64}


# ---------------------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # A few tokens looked up, as a short prompt or one decoding step of a batch does: the launch shows.
        {"name": "lookup, 33 tokens", "kind": "lookup", "T": 33, "V": 32768, "D": 2048, "type": "bf16", "ids": 64, "scale": 1.0, "masked": 0.0},
        # The table's gradient after a micro-batch of text: ids as unevenly used as words are, the table far larger than the batch.
        {"name": "table gradient, 16384 tokens", "kind": "table", "T": 16384, "V": 131072, "D": 2048, "type": "bf16", "ids": 64, "scale": 1.0, "masked": 0.0, "more": False},
        # An odd table in fp32 with scaled lookups, half of the batch padding, added to the micro-batch before it.
        {"name": "table gradient, fp32, half padded", "kind": "table", "T": 4095, "V": 50001, "D": 1000, "type": "fp32", "ids": 32, "scale": 32.0, "masked": 0.5, "more": True},
        # One decoding step: the sampled token's log probability, the entropy, eight alternatives.
        {"name": "log probabilities, one token", "kind": "logp", "T": 1, "V": 131072, "type": "bf16", "ids": 64, "entropy": True, "top": 8, "masked": 0.0},
        # The loss of a micro-batch, with the entropy that its reports show; some positions are prompt and do not count.
        {"name": "log probabilities, 4096 tokens", "kind": "logp", "T": 4096, "V": 131072, "type": "bf16", "ids": 64, "entropy": True, "top": 0, "masked": 0.1},
        # Scoring answers with their alternatives: fp32 logits over an odd vocabulary.
        {"name": "log probabilities, fp32, top 20", "kind": "logp", "T": 257, "V": 50001, "type": "fp32", "ids": 32, "entropy": False, "top": 20, "masked": 0.0},
        # The backward pass of that loss, to the logits.
        {"name": "log probability gradient, 4096", "kind": "logp_grad", "T": 4096, "V": 131072, "type": "bf16", "ids": 64, "entropy": False, "masked": 0.1},
        # One token in front of its attention.
        {"name": "norm and rotate, one token", "kind": "rotate", "T": 1, "Hq": 32, "Hk": 4, "D": 128, "R": 128, "adjacent": False, "P": 32768, "type": "bf16", "ids": 64},
        # Queries and keys of a long sequence, windows of the fused projection's rows.
        {"name": "norm and rotate, 8192 tokens", "kind": "rotate", "T": 8192, "Hq": 64, "Hk": 8, "D": 128, "R": 128, "adjacent": False, "P": 8192, "type": "bf16", "ids": 64},
        # Its backward pass over an odd number of tokens, with the weights' gradients.
        {"name": "norm and rotate gradient, 8191", "kind": "rotate_grad", "T": 8191, "Hq": 32, "Hk": 4, "D": 128, "R": 128, "adjacent": False, "P": 8192, "type": "bf16", "ids": 64},
        # One rank's fp32 shard of a dense layer (855.7 million parameters over 64 ranks), as the reduce-scatter leaves it.
        {"name": "norm and clip, one shard", "kind": "clip", "layer": "shard", "n": 13371392, "type": "fp32"},
        # Every gradient of a mixture-of-experts layer, tensor by tensor.
        {"name": "norm and clip, 391 tensors", "kind": "clip", "layer": "moe", "E": 128, "F": 768, "H": 2048, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def _width(rng, lo, hi):
    """A row length: most are multiples of 64 or 8, as layers have them, some are any number."""
    w = _log(rng, lo, hi)
    step = rng.choice([64, 64, 64, 8, 1])
    return max(lo, w // step * step)


def draw(rng):
    kind = rng.choice(["lookup", "table", "table", "logp", "logp", "logp_grad", "rotate", "rotate", "rotate_grad", "clip", "clip"])
    c = {"kind": kind, "type": rng.choice(["bf16", "bf16", "bf16", "fp32"])}
    if kind == "clip":
        c["layer"] = rng.choice(["shard", "moe", "list"])
        if c["layer"] == "shard":
            c["n"] = _log(rng, 1000, 100000000)
        elif c["layer"] == "moe":
            c.update(E=rng.choice([8, 16, 60, 64, 128]), F=_width(rng, 64, 1024), H=_width(rng, 256, 2048))
        else:
            c.update(n=rng.randint(1, 600), most=_log(rng, 100, 1000000))
        return c
    c["ids"] = rng.choice([32, 64])
    if kind in ("lookup", "table"):
        c.update(T=_log(rng, 1, 32768), V=_log(rng, 500, 262144), D=_width(rng, 64, 8192), scale=rng.choice([1.0, 1.0, 45.25]), masked=rng.choice([0.0, 0.02, 0.5]))
        while c["V"] * c["D"] > 131072 * 2048:
            c["V"] = c["V"] // 2
        while c["T"] * c["D"] > 16384 * 8192:
            c["T"] = c["T"] // 2
        if kind == "table":
            c["more"] = rng.random() < 0.3
        return c
    if kind in ("logp", "logp_grad"):
        c.update(T=_log(rng, 1, 8192), V=_width(rng, 1000, 262144), entropy=rng.random() < 0.5, masked=rng.choice([0.0, 0.1, 0.6]))
        if kind == "logp":
            c["top"] = rng.choice([0, 0, 1, 5, 20])
        while c["T"] * c["V"] > 2048 * 131072 // (4 if c.get("top") else 1):
            c["T"] = max(1, c["T"] // 2)
        return c
    c.update(T=_log(rng, 1, 16384), Hk=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 128, 256, 80]), P=rng.choice([16384, 131072]), adjacent=rng.random() < 0.25)
    c["Hq"] = c["Hk"] * rng.choice([1, 4, 8])
    c["R"] = rng.choice([c["D"], c["D"], c["D"] // 2])
    while c["T"] * (c["Hq"] + c["Hk"]) * c["D"] > 8192 * 72 * 128:
        c["T"] = c["T"] // 2
    return c


# ------------------------------------------------------------------------------------------------ plain operators

def plain_lookup(ids, table, scale):
    there = (ids >= 0) & (ids < table.shape[0])
    rows = table[torch.where(there, ids, 0).long()].float()
    return torch.where(there[:, None], rows * scale, 0.0).to(table.dtype)


def plain_sort(ids, V, order):
    """(offsets, order): tokens in the order of their ids, stably; an id outside 0 .. V - 1 has no place."""
    key = torch.where((ids >= 0) & (ids < V), ids.long(), V)
    by_id = torch.argsort(key, stable=True).int()
    offsets = torch.searchsorted(key[by_id.long()], torch.arange(V + 1, device=ids.device)).int()
    there = torch.arange(ids.numel(), device=ids.device) < offsets[V]
    return offsets, torch.where(there, by_id, order)


def plain_table_grad(ids, dout, V, scale, old):
    there = (ids >= 0) & (ids < V)
    total = torch.zeros(V + 1, dout.shape[1], device=dout.device)
    total.index_add_(0, torch.where(there, ids.long(), V), dout.float())
    total = total[:V] * scale
    return (total if old is None else total + old.float()).to(dout.dtype)


def plain_logp(logits, targets, top, entropy=True):
    """(log probability, (maximum, logarithm of the sum), entropy, alternatives' ids, their log probabilities), all in 32 bits."""
    x = logits.float()
    T, V = x.shape
    m = x.max(1).values
    z = x - m[:, None]
    e = torch.exp(z)
    s = e.sum(1)
    log_s = torch.log(s)
    there = (targets >= 0) & (targets < V)
    at = torch.where(there, targets.long(), 0)
    logp = torch.where(there, z.gather(1, at[:, None])[:, 0] - log_s, 0.0)
    H = log_s - (e * z).sum(1) / s if entropy else None
    if not top:
        return logp, torch.stack([m, log_s], 1), H, None, None
    bits = x.view(torch.int32).long()                                     # ordered as the floats are, then by lower index
    key = torch.where(bits >= 0, bits, -2 ** 31 - bits)
    key = key * 2 ** 20 + (2 ** 20 - 1 - torch.arange(V, device=x.device))
    ids = 2 ** 20 - 1 - torch.topk(key, top, 1).values % 2 ** 20
    return logp, torch.stack([m, log_s], 1), H, ids.int(), z.gather(1, ids) - log_s[:, None]


def plain_logp_grad(logits, targets, stats, dlogp, entropy, dentropy):
    x = logits.float()
    there = (targets >= 0) & (targets < x.shape[1])
    d = torch.where(there, dlogp, 0.0)[:, None]
    lp = x - stats[:, :1] - stats[:, 1:]
    p = torch.exp(lp)
    dx = -p * (d if dentropy is None else d + dentropy[:, None] * (lp + entropy[:, None]))
    dx.scatter_add_(1, torch.where(there, targets.long(), 0)[:, None], d)
    return dx.to(logits.dtype)


def _turn(x, c, s, R, adjacent):
    """The first R elements of each head as R / 2 pairs, each turned by its angle."""
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if adjacent else (x[..., : R // 2], x[..., R // 2: R])
    c, s = c[:, None, :], s[:, None, :]
    u, v = a * c - b * s, a * s + b * c
    turned = torch.stack([u, v], -1).flatten(-2) if adjacent else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., R:]], -1)


def plain_rotate(x, w, positions, cos, sin, eps, adjacent):
    v = x.float()
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + eps) * w.float()
    p = positions.long()
    return _turn(v, cos[p], sin[p], 2 * cos.shape[1], adjacent).to(x.dtype)


def plain_rotate_grad(dout, x, w, positions, cos, sin, eps, adjacent):
    """(gradient of x, gradient of the weight)."""
    p = positions.long()
    g = _turn(dout.float(), cos[p], -sin[p], 2 * cos.shape[1], adjacent)
    v = x.float()
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    v = v * r
    gw = g * w.float()
    dx = r * (gw - v * (gw * v).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * v).sum((0, 1)).to(w.dtype)


def plain_squares(grads):
    total = torch.zeros(1, dtype=torch.float64, device=grads[0].device)
    for g in grads:
        v = g.double()
        total += (v * v).sum()
    return total


def plain_clip(grads, total, most):
    norm = torch.sqrt(total)
    factor = torch.clamp(most / norm, max=1.0)
    return torch.cat([(g.float() * factor.float()).to(g.dtype).view(-1) for g in grads]), norm.float()


# ---------------------------------------------------------------------------------------------------- state and run

def _token_ids(T, V, masked, g, dev):
    """Ids whose use falls with their rank as words' does (the first takes some percent), some -1: padding."""
    u = torch.rand(T, generator=g, device=dev, dtype=torch.float64)
    ids = torch.clamp(torch.exp(u * math.log(V)).long() - 1, 0, V - 1)
    return torch.where(torch.rand(T, generator=g, device=dev) < masked, -1, ids)


def _sizes(c):
    if c["layer"] == "shard":
        return [(c["n"],)]
    if c["layer"] == "moe":
        E, F, H = c["E"], c["F"], c["H"]
        return [(F, H), (F, H), (H, F)] * E + [(E, H), (2 * H, H), (H // 4, H), (H // 4, H), (H, 2 * H), (H,), (H,)]
    rng = random.Random(c["n"] * 1000003 + c["most"])
    return [(_log(rng, 1, c["most"]),) for _ in range(c["n"])]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c, s, dtype = case, {"kind": case["kind"]}, TYPES[case["type"]]
    empty = lambda *shape, dt=dtype: torch.empty(*shape, dtype=dt, device=dev)  # noqa: E731
    normal = lambda *shape, dt=dtype: torch.randn(*shape, generator=g, device=dev, dtype=dt)  # noqa: E731
    if c["kind"] == "clip":
        s["grads"] = [1e-3 * normal(*shape) for shape in _sizes(c)]
        s["flat"] = empty(sum(t.numel() for t in s["grads"]))                                 # clipped into one buffer, tensor behind tensor
        s["out"] = [v.view(t.shape) for v, t in zip(s["flat"].split([t.numel() for t in s["grads"]]), s["grads"])]
        s["most"] = 0.37e-3 * math.sqrt(sum(t.numel() for t in s["grads"]))                   # about a third of the norm
        s["total"], s["norm"] = empty(1, dt=torch.float64), empty(1, dt=torch.float32)
        if own:
            import mixed_precision_rs_amd as tide
            s["grads_table"], s["out_table"] = tide.TensorTable(s["grads"]), tide.TensorTable(s["out"])
        return s
    T, ids = c["T"], IDS[c["ids"]]
    if c["kind"] in ("lookup", "table"):
        V, D = c["V"], c["D"]
        s.update(ids=_token_ids(T, V, c["masked"], g, dev).to(ids), scale=c["scale"])
        if c["kind"] == "lookup":
            s.update(table=0.02 * normal(V, D), out=empty(T, D))
            return s
        s.update(dout=1e-3 * normal(T, D), offsets=empty(V + 1, dt=torch.int32), order=torch.full((T,), -1, dtype=torch.int32, device=dev))
        s["old"] = 1e-3 * normal(V, D) if c["more"] else None
        s["grad"] = empty(V, D)
        return s
    if c["kind"] in ("logp", "logp_grad"):
        V = c["V"]
        s["logits"] = 2.0 * normal(T, V)
        targets = _token_ids(T, V, 0.0, g, dev)
        s["logits"].scatter_add_(1, targets[:, None], (10.0 + 2.0 * normal(T, 1)))             # the model has learned something
        hidden = torch.rand(T, generator=g, device=dev) < c["masked"]
        hidden[0] = False
        targets = torch.where(hidden, -100, targets)
        s["targets"] = targets.to(ids)
        f32 = lambda *shape: empty(*shape, dt=torch.float32)  # noqa: E731
        if c["kind"] == "logp":
            s.update(logp=f32(T), stats=f32(T, 2), entropy=f32(T) if c["entropy"] else None, top=c["top"])
            if c["top"]:
                s.update(top_ids=empty(T, c["top"], dt=torch.int32), top_logp=f32(T, c["top"]))
            return s
        _, s["stats"], s["entropy"], _, _ = plain_logp(s["logits"], targets, 0)
        s["dlogp"] = torch.where(hidden, 0.0, -1.0 / float((~hidden).sum()))                   # of the mean loss
        s["dentropy"] = torch.full((T,), -0.01 / T, device=dev) if c["entropy"] else None      # and of an entropy bonus
        s["dlogits"] = empty(T, V)
        return s
    Hq, Hk, D, R, P = c["Hq"], c["Hk"], c["D"], c["R"], c["P"]
    fused = normal(T, Hq + 2 * Hk, D) * torch.exp(0.5 * normal(1, Hq + 2 * Hk, 1))             # queries, keys and values of a token side by side
    s.update(q=fused[:, :Hq], k=fused[:, Hq: Hq + Hk], qw=1.0 + 0.1 * normal(D), kw=1.0 + 0.1 * normal(D), eps=1e-6, adjacent=c["adjacent"])
    turns = torch.arange(P, device=dev, dtype=torch.float64)[:, None] * 1e6 ** (-torch.arange(0, R, 2, device=dev, dtype=torch.float64) / R)
    s.update(cos=torch.cos(turns).float(), sin=torch.sin(turns).float())
    first = int(torch.randint(0, P, (1,), generator=g, device=dev))
    s["positions"] = ((first + torch.arange(T, device=dev)) % P).to(ids)
    if c["kind"] == "rotate":
        s.update(qo=empty(T, Hq, D), ko=empty(T, Hk, D))
        return s
    s.update(dqo=1e-3 * normal(T, Hq, D), dko=1e-3 * normal(T, Hk, D), dqw=empty(D), dkw=empty(D))
    dfused = torch.zeros_like(fused)
    s.update(dq=dfused[:, :Hq], dk=dfused[:, Hq: Hq + Hk])
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import mixed_precision_rs_amd as tide
    kind = s["kind"]
    if kind == "lookup":
        tide.embed_tokens(s["ids"], s["table"], s["out"], scale=s["scale"])
        return s["out"]
    if kind == "table":
        if s["old"] is not None:
            s["grad"].copy_(s["old"])
        tide.sort_ids(s["ids"], s["grad"].shape[0], s["offsets"], s["order"])
        tide.embed_tokens_grad(s["dout"], s["offsets"], s["order"], s["grad"], scale=s["scale"], accumulate=s["old"] is not None)
        return s["offsets"], s["order"], s["grad"]
    if kind == "logp":
        if not s["top"]:
            tide.token_logprobs(s["logits"], s["targets"], s["logp"], stats=s["stats"], entropy=s["entropy"])
            return s["logp"], s["stats"], s["entropy"]
        tide.token_logprobs(s["logits"], s["targets"], s["logp"], stats=s["stats"], entropy=s["entropy"], top_ids=s["top_ids"], top_logprobs=s["top_logp"])
        return s["logp"], s["stats"], s["entropy"], s["top_ids"], s["top_logp"]
    if kind == "logp_grad":
        with_entropy = {} if s["dentropy"] is None else {"entropy": s["entropy"], "dentropy": s["dentropy"]}
        tide.token_logprobs_grad(s["logits"], s["targets"], s["stats"], s["dlogp"], s["dlogits"], **with_entropy)
        return s["dlogits"]
    if kind == "rotate":
        tide.norm_rotate(s["q"], s["k"], s["qo"], s["ko"], q_weight=s["qw"], k_weight=s["kw"], positions=s["positions"], cos=s["cos"], sin=s["sin"], eps=s["eps"],
                         adjacent=s["adjacent"])
        return s["qo"], s["ko"]
    if kind == "rotate_grad":
        tide.norm_rotate_grad(s["dqo"], s["dko"], s["q"], s["k"], s["dq"], s["dk"], q_weight=s["qw"], k_weight=s["kw"], positions=s["positions"], cos=s["cos"],
                              sin=s["sin"], dq_weight=s["dqw"], dk_weight=s["dkw"], eps=s["eps"], adjacent=s["adjacent"])
        return s["dq"], s["dk"], s["dqw"], s["dkw"]
    tide.grad_squares(s["grads_table"], s["total"])
    tide.clip_grads(s["grads_table"], s["total"], s["most"], out=s["out_table"], norm=s["norm"])
    return s["total"], s["norm"], s["flat"]


def run_plain(s):
    kind = s["kind"]
    if kind == "lookup":
        return plain_lookup(s["ids"], s["table"], s["scale"])
    if kind == "table":
        V = s["grad"].shape[0]
        offsets, order = plain_sort(s["ids"], V, s["order"])
        return offsets, order, plain_table_grad(s["ids"], s["dout"], V, s["scale"], s["old"])
    if kind == "logp":
        logp, stats, entropy, ids, top = plain_logp(s["logits"], s["targets"], s["top"], s["entropy"] is not None)
        return (logp, stats, entropy, ids, top) if s["top"] else (logp, stats, entropy)
    if kind == "logp_grad":
        return plain_logp_grad(s["logits"], s["targets"], s["stats"], s["dlogp"], s["entropy"], s["dentropy"])
    if kind == "clip":
        total = plain_squares(s["grads"])
        clipped, norm = plain_clip(s["grads"], total, s["most"])
        return total, norm, clipped
    where = (s["positions"], s["cos"], s["sin"], s["eps"], s["adjacent"])
    if kind == "rotate":
        return plain_rotate(s["q"], s["qw"], *where), plain_rotate(s["k"], s["kw"], *where)
    (dq, dqw), (dk, dkw) = plain_rotate_grad(s["dqo"], s["q"], s["qw"], *where), plain_rotate_grad(s["dko"], s["k"], s["kw"], *where)
    return dq, dk, dqw, dkw


# ------------------------------------------------------------------------------------------------ work and exactness

def work(case):
    c, wide = case, 4 if case["type"] == "fp32" else 2
    if c["kind"] == "clip":
        n = sum(math.prod(shape) for shape in _sizes(c))
        return {"bytes": 2 * wide * n, "flops": 3 * n}
    T, ids = c["T"], c["ids"] // 8
    if c["kind"] == "lookup":
        return {"bytes": T * ids + wide * c["D"] * T * (2.0 - c["masked"]), "flops": T * c["D"] * (1.0 - c["masked"])}
    if c["kind"] == "table":
        V, D, rows = c["V"], c["D"], T * (1.0 - c["masked"])
        return {"bytes": T * (ids + 4) + 4 * (V + 1) + wide * D * (rows + V * (2 if c["more"] else 1)), "flops": rows * D}
    if c["kind"] == "logp":
        return {"bytes": wide * T * c["V"] + T * (ids + 12 + (4 if c["entropy"] else 0) + 8 * c["top"]), "flops": (6 if c["entropy"] else 4) * T * c["V"]}
    if c["kind"] == "logp_grad":
        rows = T * (1.0 if c["entropy"] else 1.0 - c["masked"])
        return {"bytes": wide * c["V"] * (T + rows) + T * (ids + 12), "flops": (7 if c["entropy"] else 4) * rows * c["V"]}
    n, table = T * (c["Hq"] + c["Hk"]) * c["D"], 4 * min(T, c["P"]) * c["R"] + T * ids
    if c["kind"] == "rotate":
        return {"bytes": 2 * wide * n + table, "flops": 7 * n}
    return {"bytes": 3 * wide * n + table, "flops": 14 * n}


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "clip":
        total = math.fsum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grads"])
        norm = math.sqrt(total)
        ratio = min(1.0, s["most"] / norm)
        one = lambda v: torch.tensor([v], dtype=torch.float64, device=s["norm"].device)  # noqa: E731
        return one(total), one(norm), torch.cat([t.double().view(-1) for t in s["grads"]]) * ratio
    if kind == "lookup":
        padded = torch.cat([s["table"].double() * s["scale"], torch.zeros(1, s["table"].shape[1], dtype=torch.float64, device=s["ids"].device)])
        return padded[s["ids"].long()]                                                             # -1 is the row of zeros
    if kind == "table":
        V, D = s["grad"].shape
        some = torch.nonzero(s["ids"] >= 0)[:, 0]
        out = torch.zeros(V, D, dtype=torch.float64, device=s["ids"].device)
        out.index_put_((s["ids"][some].long(),), s["dout"][some].double() * s["scale"], accumulate=True)
        return None, None, out if s["old"] is None else out + s["old"].double()
    if kind in ("logp", "logp_grad"):
        x = s["logits"].double()
        T, V = x.shape
        lse = torch.logsumexp(x, 1)
        rows = torch.nonzero(s["targets"] >= 0)[:, 0]
        cols = s["targets"][rows].long()
        if kind == "logp":
            logp = torch.zeros_like(lse)
            logp[rows] = x[rows, cols] - lse[rows]
            m = x.amax(1)
            entropy = None if s["entropy"] is None else torch.special.entr(torch.exp(x - lse[:, None])).sum(1)
            first = logp, torch.stack([m, lse - m], 1), entropy
            return first + (None, torch.topk(x, s["top"], 1).values - lse[:, None]) if s["top"] else first
        p = torch.exp(x - lse[:, None])
        out = torch.zeros_like(x)
        out[rows, cols] = s["dlogp"].double()[rows]
        out[rows] -= p[rows] * s["dlogp"].double()[rows, None]
        if s["dentropy"] is not None:
            H = torch.special.entr(p).sum(1, keepdim=True)
            out += s["dentropy"].double()[:, None] * (torch.special.entr(p) - p * H)
        return out
    at = s["positions"].long()
    angle = torch.complex(s["cos"][at].double(), s["sin"][at].double())[:, None]
    R = 2 * s["cos"].shape[1]

    def turned(x, w):
        y = x * w / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + s["eps"])
        pairs = y[..., :R].unflatten(-1, (R // 2, 2)) if s["adjacent"] else y[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * angle)
        z = z if s["adjacent"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), y[..., R:]], -1)

    if kind == "rotate":
        return turned(s["q"].double(), s["qw"].double()), turned(s["k"].double(), s["kw"].double())
    found = []
    for x, w, d in ((s["q"], s["qw"], s["dqo"]), (s["k"], s["kw"], s["dko"])):
        x, w = x.double().requires_grad_(), w.double().requires_grad_()
        found.append(torch.autograd.grad(turned(x, w), (x, w), d.double()))
    return found[0][0], found[1][0], found[0][1], found[1][1]
