"""ctypes binding of the calls at the ends of a training step and in front of
its attention (include/tide.h, "The ends of the step, and what stands before
its attention"): tokens sorted by id, embedding lookup and the table's gradient,
norm and rotation of queries and keys, log probabilities of given tokens and
their gradient, the gradient norm and clipping.

Argument marshalling only, as in _layer.py: tensors with unit column stride are
taken with their row strides, outputs are passed in.
"""
import ctypes
import struct
from typing import Optional, Sequence, Union

from ._lib import PointerTable, _check
from ._layer import (_SIGNATURES, _dtype_code, _flat, _fn, _mat, _on, _place, _run, _workspace)


# The structures as bytes, which ctypes passes as a pointer: a call of a few
# microseconds would spend two on objects of ctypes.Structure.
Heads = struct.Struct("@Pqqii").pack        # tide_heads: data, strides, heads, reserved
Rotation = struct.Struct("@PPPqqiiii").pack  # tide_rotation, in the header's order


_I32, _I64, _VP, _F32, _F64 = (ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float,
                               ctypes.c_double)
_SIGNATURES.update({
    "tide_sort_ids_workspace": [_I64, _I64, ctypes.POINTER(_I64)],
    "tide_sort_ids": [_VP, _I32, _I64, _I64, _VP, _VP, _VP, _I64, _VP],
    "tide_embed_tokens": [_I32, _VP, _I32, _I64, _VP, _I64, _I64, _I64, _F32, _VP, _I64, _VP],
    "tide_embed_tokens_grad_workspace": [_I64, _I64, ctypes.POINTER(_I64)],
    "tide_embed_tokens_grad": [_I32, _VP, _I64, _I64, _I64, _VP, _VP, _I64, _F32, _VP, _I64, _I32,
                               _VP, _I64, _VP],
    "tide_token_logprobs_workspace": [_I32, _I64, _I64, _I32, ctypes.POINTER(_I64)],
    "tide_token_logprobs": [_I32, _VP, _I64, _I64, _I64, _VP, _I32, _VP, _VP, _VP, _I32, _VP, _VP,
                            _VP, _I64, _VP],
    "tide_token_logprobs_grad": [_I32, _VP, _I64, _I64, _I64, _VP, _I32, _VP, _VP, _VP, _VP, _VP,
                                 _I64, _VP],
    "tide_norm_rotate": [_I32, _I64, _I32, _VP, _VP, _VP, _VP, _F32, _VP, _VP, _VP, _VP],
    "tide_norm_rotate_grad_workspace": [_I64, _I32, _I32, ctypes.POINTER(_I64)],
    "tide_norm_rotate_grad": [_I32, _I64, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _F32, _VP, _VP, _VP,
                              _VP, _VP, _I32, _VP, _I64, _VP],
    "tide_grad_squares_workspace": [_I32, _VP, _I32, ctypes.POINTER(_I64)],
    "tide_grad_squares": [_I32, _VP, _VP, _I32, _VP, _I32, _VP, _I64, _VP],
    "tide_clip_grads": [_I32, _VP, _VP, _I32, _VP, _F64, _VP, _VP, _VP],
})


def _ids(t, what: str, n: Optional[int], dev) -> int:
    """Address of a contiguous 1-D tensor of int32 or int64 ids."""
    import torch
    if t.dtype not in (torch.int32, torch.int64):
        raise TypeError("%s has dtype %s, expected torch.int32 or torch.int64" % (what, t.dtype))
    return _flat(t, what, t.dtype, (t.numel() if n is None else n,), dev)


def _bytes(name: str, *args) -> int:
    n = _I64()
    _check(_fn(name)(*args, ctypes.byref(n)), name)
    return int(n.value)


# ------------------------------------------------------------------ embedding

def sort_ids_workspace_bytes(tokens: int, vocab: int) -> int:
    """Bytes of workspace sort_ids needs (tide_sort_ids_workspace)."""
    return _bytes("tide_sort_ids_workspace", tokens, vocab)


def sort_ids(ids, vocab: int, offsets, order, workspace=None, stream=None) -> None:
    """Stable sort of tokens by id (tide_sort_ids). ids: (tokens,) int32 or
    int64, anything outside [0, vocab) for a token without an id; offsets:
    (vocab + 1,) int32; order: (tokens,) int32. workspace: uint8 tensor of
    sort_ids_workspace_bytes(), by default allocated for the call."""
    import torch
    sh, sobj, dev = _on(stream, ids)
    ip = _ids(ids, "ids", None, dev)
    n = ids.numel()
    op = _flat(offsets, "offsets", torch.int32, (vocab + 1,), dev)
    rp = _flat(order, "order", torch.int32, (n,), dev)
    need = sort_ids_workspace_bytes(n, vocab)
    wp, wn, w = _workspace(need, workspace, stream, dev)
    _run("tide_sort_ids", (ip, ids.element_size(), n, vocab, op, rp, wp, wn, sh), dev,
         [ids, offsets, order, w], sobj)


def embed_tokens(ids, table, out, scale: float = 1.0, stream=None) -> None:
    """out[t] = scale * table[ids[t]] (tide_embed_tokens); zeros where an id is
    outside the table. ids: (tokens,) int32 or int64; table: (vocab, width) and
    out: (tokens, width) bf16 or fp32."""
    sh, sobj, dev = _on(stream, table)
    code = _dtype_code(table, "table")
    tp, ts = _mat(table, "table", table.dtype, None, None, dev)
    V, D = table.shape
    ip = _ids(ids, "ids", None, dev)
    n = ids.numel()
    op, os_ = _mat(out, "out", table.dtype, n, D, dev)
    _run("tide_embed_tokens", (code, ip, ids.element_size(), n, tp, ts, V, D, scale, op, os_, sh),
         dev, [ids, table, out], sobj)


def embed_tokens_grad_workspace_bytes(tokens: int, width: int) -> int:
    """Bytes of workspace embed_tokens_grad needs (tide_embed_tokens_grad_workspace)."""
    return _bytes("tide_embed_tokens_grad_workspace", tokens, width)


def embed_tokens_grad(dout, offsets, order, grad, scale: float = 1.0, accumulate: bool = False,
                      workspace=None, stream=None) -> None:
    """Gradient of embed_tokens to the whole table, by the tokens that sort_ids
    sorted (tide_embed_tokens_grad): grad (vocab, width) is written completely,
    or, with accumulate, added to. dout: (tokens, width), of grad's type.
    workspace: uint8 tensor of embed_tokens_grad_workspace_bytes(), by default
    allocated for the call."""
    import torch
    sh, sobj, dev = _on(stream, dout)
    code = _dtype_code(dout, "dout")
    dp, ds = _mat(dout, "dout", dout.dtype, None, None, dev)
    n, D = dout.shape
    gp, gs = _mat(grad, "grad", dout.dtype, None, D, dev)
    V = grad.shape[0]
    op = _flat(offsets, "offsets", torch.int32, (V + 1,), dev)
    rp = _flat(order, "order", torch.int32, (n,), dev)
    need = embed_tokens_grad_workspace_bytes(n, D)
    wp, wn, w = _workspace(need, workspace, stream, dev)
    _run("tide_embed_tokens_grad", (code, dp, ds, n, D, op, rp, V, scale, gp, gs,
         1 if accumulate else 0, wp, wn, sh), dev, [dout, offsets, order, grad, w], sobj)


# ---------------------------------------------------------- log probabilities

def token_logprobs_workspace_bytes(logits, top: int = 0) -> int:
    """Bytes of workspace token_logprobs needs for these logits
    (tide_token_logprobs_workspace)."""
    return _bytes("tide_token_logprobs_workspace", _dtype_code(logits, "logits"), *logits.shape, top)


def token_logprobs(logits, targets, logprob, stats=None, entropy=None, top_ids=None,
                   top_logprobs=None, workspace=None, stream=None) -> None:
    """Log probabilities of the target tokens, entropies and the most probable
    alternatives in one pass over the logits (tide_token_logprobs). logits:
    (tokens, vocab) bf16 or fp32; targets: (tokens,) int32 or int64, anything
    outside [0, vocab) for a position that does not count; logprob, entropy:
    (tokens,) fp32; stats: (tokens, 2) fp32, for token_logprobs_grad; top_ids
    (tokens, top) int32 and top_logprobs (tokens, top) fp32, top up to 32.
    workspace: uint8 tensor of token_logprobs_workspace_bytes(), by default
    allocated for the call."""
    import torch
    sh, sobj, dev = _on(stream, logits)
    code = _dtype_code(logits, "logits")
    lp, ls = _mat(logits, "logits", logits.dtype, None, None, dev)
    n, V = logits.shape
    tp = _ids(targets, "targets", n, dev)
    pp = _flat(logprob, "logprob", torch.float32, (n,), dev)
    sp = 0 if stats is None else _flat(stats, "stats", torch.float32, (n, 2), dev)
    ep = 0 if entropy is None else _flat(entropy, "entropy", torch.float32, (n,), dev)
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs go together")
    top, ip, qp = 0, 0, 0
    if top_ids is not None:
        top = top_ids.shape[-1]
        ip = _flat(top_ids, "top_ids", torch.int32, (n, top), dev)
        qp = _flat(top_logprobs, "top_logprobs", torch.float32, (n, top), dev)
    need = _bytes("tide_token_logprobs_workspace", code, n, V, top)
    wp, wn, w = _workspace(need, workspace, stream, dev)
    _run("tide_token_logprobs", (code, lp, ls, n, V, tp, targets.element_size(), pp, sp, ep, top,
         ip, qp, wp, wn, sh), dev, [logits, targets, logprob, stats, entropy, top_ids,
         top_logprobs, w], sobj)


def token_logprobs_grad(logits, targets, stats, dlogprob, dlogits, entropy=None, dentropy=None,
                        stream=None) -> None:
    """Gradient of token_logprobs to the logits (tide_token_logprobs_grad).
    stats (and entropy, where dentropy is given) are token_logprobs' outputs;
    dlogprob, dentropy: (tokens,) fp32; dlogits: as logits, and may be logits."""
    import torch
    sh, sobj, dev = _on(stream, logits)
    code = _dtype_code(logits, "logits")
    lp, ls = _mat(logits, "logits", logits.dtype, None, None, dev)
    n, V = logits.shape
    tp = _ids(targets, "targets", n, dev)
    f32 = lambda t, what: _flat(t, what, torch.float32, (n,), dev)  # noqa: E731
    sp = _flat(stats, "stats", torch.float32, (n, 2), dev)
    dp = f32(dlogprob, "dlogprob")
    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs entropy")
    ep = 0 if entropy is None else f32(entropy, "entropy")
    hp = 0 if dentropy is None else f32(dentropy, "dentropy")
    op, os_ = _mat(dlogits, "dlogits", logits.dtype, n, V, dev)
    _run("tide_token_logprobs_grad", (code, lp, ls, n, V, tp, targets.element_size(), sp, dp, ep,
         hp, op, os_, sh), dev, [logits, targets, stats, dlogprob, entropy, dentropy, dlogits],
         sobj)


# -------------------------------------------------------------- norm, rotation

def _heads(t, what: str, dtype, tokens: Optional[int], heads: Optional[int], dim: Optional[int],
           dev) -> bytes:
    """tide_heads of a (tokens, heads, head_dim) tensor whose heads are contiguous."""
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (what, t.dtype, dtype))
    if t.dim() != 3:
        raise ValueError("%s has %d dimensions, expected 3" % (what, t.dim()))
    T, H, D = t.shape
    if T != tokens or H != heads or D != dim:
        for got, want, name in ((T, tokens, "tokens"), (H, heads, "heads"), (D, dim, "elements a head")):
            if want is not None and got != want:
                raise ValueError("%s has %d %s, expected %d" % (what, got, name, want))
    st, sh, sd = t.stride()
    if D > 1 and sd != 1 and t.numel():
        raise ValueError("%s: a head's elements are not adjacent" % what)
    _place(t, what, dev)
    return Heads(t.data_ptr(), st if T > 1 else max(H * D, 1), sh if H > 1 else D, H, 0)


def _rotation(positions, cos, sin, adjacent: bool, tokens: int, dev) -> Optional[bytes]:
    import torch
    if cos is None and sin is None:
        if positions is not None:
            raise ValueError("positions without cos and sin")
        return None
    if cos is None or sin is None:
        raise ValueError("cos and sin go together")
    cp, cs = _mat(cos, "cos", torch.float32, None, None, dev)
    sp, ss = _mat(sin, "sin", torch.float32, cos.shape[0], cos.shape[1], dev)
    if cs != ss:
        raise ValueError("cos and sin have row strides of %d and %d" % (cs, ss))
    pp = 0 if positions is None else _ids(positions, "positions", tokens, dev)
    size = 0 if positions is None else positions.element_size()
    return Rotation(pp, cp, sp, cos.shape[0], cs, size, cos.shape[1], 1 if adjacent else 0, 0)


def norm_rotate(q, k, q_out, k_out, q_weight=None, k_weight=None, positions=None, cos=None,
                sin=None, eps: float = 1e-6, adjacent: bool = False, stream=None) -> None:
    """Queries and keys normalised head by head (root mean square) and rotated
    by position, in one pass (tide_norm_rotate). q, k: (tokens, heads, head_dim)
    bf16 or fp32, windows of a wider tensor welcome; k and k_out may be None.
    q_weight, k_weight: (head_dim,), None for ones. cos, sin: (rows, pairs)
    fp32, the first 2 * pairs elements of a head are rotated, elements (i, i +
    pairs) or, with adjacent, (2i, 2i + 1) together; positions: (tokens,) int32
    or int64 rows of the tables, None for row t. Without cos and sin nothing is
    rotated."""
    sh, sobj, dev = _on(stream, q)
    code = _dtype_code(q, "q")
    hq = _heads(q, "q", q.dtype, None, None, None, dev)
    T, H, D = q.shape
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    oq = _heads(q_out, "q_out", q.dtype, T, H, D, dev)
    hk = ok = None
    if k is not None:
        hk = _heads(k, "k", q.dtype, T, None, D, dev)
        ok = _heads(k_out, "k_out", q.dtype, T, k.shape[1], D, dev)
    qw = 0 if q_weight is None else _flat(q_weight, "q_weight", q.dtype, (D,), dev)
    kw = 0 if k_weight is None else _flat(k_weight, "k_weight", q.dtype, (D,), dev)
    rot = _rotation(positions, cos, sin, adjacent, T, dev)
    _run("tide_norm_rotate", (code, T, D, hq, hk, qw, kw, eps, rot, oq, ok, sh), dev,
         [q, k, q_out, k_out, q_weight, k_weight, positions, cos, sin], sobj)


def norm_rotate_grad_workspace_bytes(tokens: int, heads: int, head_dim: int) -> int:
    """Bytes of workspace norm_rotate_grad needs for that many heads of queries
    and keys together (tide_norm_rotate_grad_workspace)."""
    return _bytes("tide_norm_rotate_grad_workspace", tokens, heads, head_dim)


def norm_rotate_grad(dq_out, dk_out, q, k, dq, dk, q_weight=None, k_weight=None, positions=None,
                     cos=None, sin=None, dq_weight=None, dk_weight=None, eps: float = 1e-6,
                     adjacent: bool = False, accumulate: bool = False, workspace=None,
                     stream=None) -> None:
    """Gradient of norm_rotate at the same q, k, weights and rotation
    (tide_norm_rotate_grad): dq, dk, and, where they are given, dq_weight and
    dk_weight (head_dim,), added to what they hold with accumulate. workspace:
    uint8 tensor of norm_rotate_grad_workspace_bytes(), by default allocated for
    the call."""
    sh, sobj, dev = _on(stream, q)
    code = _dtype_code(q, "q")
    hq = _heads(q, "q", q.dtype, None, None, None, dev)
    T, H, D = q.shape
    gq = _heads(dq_out, "dq_out", q.dtype, T, H, D, dev)
    xq = _heads(dq, "dq", q.dtype, T, H, D, dev)
    if k is None and (dk_out is not None or dk is not None or dk_weight is not None):
        raise ValueError("gradients of k without k")
    hk = gk = xk = None
    Hk = 0
    if k is not None:
        if dk_out is None or dk is None:
            raise ValueError("k needs dk_out and dk")
        Hk = k.shape[1]
        hk = _heads(k, "k", q.dtype, T, None, D, dev)
        gk = _heads(dk_out, "dk_out", q.dtype, T, Hk, D, dev)
        xk = _heads(dk, "dk", q.dtype, T, Hk, D, dev)
    ws = [0 if w is None else _flat(w, name, q.dtype, (D,), dev) for w, name in (
        (q_weight, "q_weight"), (k_weight, "k_weight"), (dq_weight, "dq_weight"),
        (dk_weight, "dk_weight"))]
    rot = _rotation(positions, cos, sin, adjacent, T, dev)
    wp, wn, w = 0, 0, None
    if dq_weight is not None or dk_weight is not None:
        wp, wn, w = _workspace(norm_rotate_grad_workspace_bytes(T, H + Hk, D), workspace, stream, dev)
    _run("tide_norm_rotate_grad", (code, T, D, gq, gk, hq, hk, ws[0], ws[1], eps, rot, xq, xk,
         ws[2], ws[3], 1 if accumulate else 0, wp, wn, sh), dev,
         [dq_out, dk_out, q, k, dq, dk, q_weight, k_weight, positions, cos, sin, dq_weight,
          dk_weight, w], sobj)


# ------------------------------------------------------------- norm, clipping

class TensorTable(PointerTable):
    """Addresses and sizes of contiguous tensors of one type (bf16 or fp32),
    marshalled once, for grad_squares and clip_grads (see PointerTable). Keeps
    the tensors alive."""

    def __init__(self, tensors: Sequence[object]):
        super().__init__(tensors)
        self.code, self.device = 0, None
        for i, t in enumerate(self.refs):
            code = _dtype_code(t, "tensor %d" % i)
            if i and code != self.code:
                raise TypeError("tensor %d has dtype %s, the first one %s" % (
                    i, t.dtype, self.refs[0].dtype))
            if not t.is_contiguous():
                raise ValueError("tensor %d is not contiguous" % i)
            _place(t, "tensor %d" % i, self.device)
            self.code, self.device = code, t.get_device()
        self.elems = (ctypes.c_int64 * max(self.n, 1))(*[t.numel() for t in self.refs])
        self.workspace_bytes = _bytes("tide_grad_squares_workspace", self.code, self.elems, self.n)


def _table(grads, what: str) -> TensorTable:
    if isinstance(grads, TensorTable):
        return grads
    if isinstance(grads, PointerTable):
        raise TypeError("%s: a table of addresses has no sizes; use a TensorTable" % what)
    return TensorTable(grads if isinstance(grads, (list, tuple)) else [grads])


def grad_squares_workspace_bytes(grads) -> int:
    """Bytes of workspace grad_squares needs for these tensors
    (tide_grad_squares_workspace)."""
    return _table(grads, "grads").workspace_bytes


def grad_squares(grads: Union[object, Sequence[object], TensorTable], total,
                 accumulate: bool = False, workspace=None, stream=None) -> None:
    """The square of the gradient norm, sum of x^2 over all tensors, into total,
    a (1,) float64 tensor (tide_grad_squares). grads: a tensor, a list, or a
    TensorTable, contiguous bf16 or fp32 of any shapes. accumulate: add to what
    total holds (other groups, other types). workspace: uint8 tensor of
    grad_squares_workspace_bytes(), by default allocated for the call."""
    import torch
    tab = _table(grads, "grads")
    sh, sobj, dev = _on(stream, total)
    tp = _flat(total, "total", torch.float64, (1,), dev)
    if tab.n and dev is not None and tab.device != dev:
        raise ValueError("grads are on GPU %d, the call on GPU %d" % (tab.device, dev))
    wp, wn, w = _workspace(tab.workspace_bytes, workspace, stream, dev)
    _run("tide_grad_squares", (tab.code, tab.arr, tab.elems, tab.n, tp, 1 if accumulate else 0, wp,
         wn, sh), dev, [*tab.refs, total, w], sobj)


def clip_grads(grads: Union[object, Sequence[object], TensorTable], total, max_norm: float,
               out: Union[object, Sequence[object], TensorTable, None] = None, norm=None,
               stream=None) -> None:
    """Scales the gradients by min(1, max_norm / sqrt(total)) (tide_clip_grads),
    in place, or into out (tensors of the same sizes). total: from grad_squares,
    added up over the ranks where the tensors are shards. norm: (1,) float32
    that receives the norm. Nothing waits for the GPU."""
    import torch
    tab = _table(grads, "grads")
    sh, sobj, dev = _on(stream, total)
    tp = _flat(total, "total", torch.float64, (1,), dev)
    np_ = 0 if norm is None else _flat(norm, "norm", torch.float32, (1,), dev)
    to = None if out is None else _table(out, "out")
    for t, what in ((tab, "grads"), (to, "out")):
        if t is not None and t.n and dev is not None and t.device != dev:
            raise ValueError("%s are on GPU %d, the call on GPU %d" % (what, t.device, dev))
    if to is not None:
        if to.n != tab.n or to.code != tab.code:
            raise ValueError("out holds %d tensors, grads %d, or of another type" % (to.n, tab.n))
        if bytes(to.elems) != bytes(tab.elems):
            raise ValueError("out's tensors have other sizes than grads'")
    _run("tide_clip_grads", (tab.code, tab.arr, tab.elems, tab.n, tp, float(max_norm),
         None if to is None else to.arr, np_, sh), dev,
         [*tab.refs, total, norm, *(() if to is None else to.refs)], sobj)
