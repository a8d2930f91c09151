"""ctypes binding of the training-layer calls of libtide.so (include/tide.h,
"The training layer beside the collectives"): tokens sorted by expert and back,
activation checkpoints in 8 bits, the gated activation over them, and weight
gradients taken from them.

Argument marshalling only. Matrices are 2-D GPU tensors with unit column
stride; a row stride is taken as it is, so column windows of a wider tensor
need no copy. Outputs are passed in, as with the collectives.
"""
import ctypes
from typing import Optional, Sequence, Tuple, Union

from ._lib import PointerTable, _check, _check_many, _load, _ptr, _record, _stream_handle

_DTYPES = {}             # torch dtype -> tide_dtype, filled when torch is first needed
SCALE_BLOCK = 32         # consecutive elements of a row that share a checkpoint scale


class Saved(ctypes.Structure):
    """tide_saved."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("codes_stride", ctypes.c_int64), ("scales_stride", ctypes.c_int64)]


_I32, _I64, _VP = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
_SP = ctypes.POINTER(Saved)
_SIGNATURES = {
    "tide_route_workspace": [_I64, _I32, _I32, ctypes.POINTER(_I64)],
    "tide_route_tokens": [_VP, _I32, _I64, _I32, _I32, _VP, _VP, _VP, _VP, _I64, _VP],
    "tide_dispatch_tokens": [_I32, _VP, _I64, _I64, _I64, _VP, _I32, _VP, _I64, _I64, _VP],
    "tide_combine_tokens": [_I32, _VP, _I64, _I64, _I64, _VP, _VP, _I64, _I32, _VP, _I64, _VP],
    "tide_combine_tokens_grad": [_I32, _VP, _I64, _VP, _I64, _I64, _I64, _VP, _VP, _I64, _I32,
                                 _VP, _I64, _VP, _VP],
    "tide_checkpoint_pack": [_I32, _VP, _I64, _I64, _I64, _SP, _VP],
    "tide_checkpoint_unpack": [_I32, _SP, _I64, _I64, _VP, _I64, _VP],
    "tide_gated_silu": [_I32, _VP, _I64, _VP, _I64, _I64, _I64, _VP, _I64, _SP, _SP, _VP],
    "tide_gated_silu_grad": [_I32, _VP, _I64, _SP, _SP, _I64, _I64, _VP, _I64, _VP, _I64, _VP,
                             _I64, _VP],
    "tide_weight_grads_workspace": [_I64, _I64, _I64, _I32, ctypes.POINTER(_I64)],
    "tide_weight_grads_bf16": [_VP, _I64, _I64, _I64, _VP, _I64, _SP, _I64, _I64, _VP, _VP, _I32,
                               _VP, _I32, _VP, _I64, _VP],
}
_fns = {}


def _fn(name: str):
    f = _fns.get(name)
    if f is None:
        f = getattr(_load(), name)
        f.argtypes = _SIGNATURES[name]
        f.restype = ctypes.c_int
        _fns[name] = f
    return f


def _dtype_code(t, what: str) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.bfloat16: 0, torch.float32: 1})
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s has dtype %s, expected torch.bfloat16 or torch.float32" % (what, t.dtype))
    return code


def _place(t, what: str, dev: Optional[int]) -> None:
    if not t.is_cuda:
        raise ValueError("%s is not a GPU tensor" % what)
    if dev is not None and t.get_device() != dev:
        raise ValueError("%s is on GPU %d, the call on GPU %d" % (what, t.get_device(), dev))


def _mat(t, what: str, dtype, rows: Optional[int], cols: Optional[int], dev) -> Tuple[int, int]:
    """(address, row stride) of a 2-D tensor of the given dtype and, where they
    are not None, sizes."""
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (what, t.dtype, dtype))
    if t.dim() != 2:
        raise ValueError("%s has %d dimensions, expected 2" % (what, t.dim()))
    r, c = t.shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError("%s is %d x %d, expected %s x %s" % (
            what, r, c, "any" if rows is None else rows, "any" if cols is None else cols))
    s0, s1 = t.stride()
    if r and c > 1 and s1 != 1:
        raise ValueError("%s: its columns are not adjacent" % what)
    if r > 1 and s0 < c:
        raise ValueError("%s: its rows overlap" % what)
    _place(t, what, dev)
    return t.data_ptr(), s0 if r > 1 else c


def _flat(t, what: str, dtype, shape, dev) -> int:
    """Address of a contiguous tensor of this dtype and shape."""
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (what, t.dtype, dtype))
    if tuple(t.shape) != shape:
        raise ValueError("%s has shape %s, expected %s" % (what, tuple(t.shape), shape))
    if not t.is_contiguous():
        raise ValueError("%s is not contiguous" % what)
    _place(t, what, dev)
    return t.data_ptr()


def _saved(saved, what: str, rows: Optional[int], cols: Optional[int], dev):
    """tide_saved of a (codes, scales) pair, and the codes' shape."""
    import torch
    codes, scales = saved
    cp, cs = _mat(codes, what + " codes", torch.float8_e4m3fn, rows, cols, dev)
    r, c = codes.shape
    sp, ss = _mat(scales, what + " scales", torch.float8_e8m0fnu, r, -(-c // SCALE_BLOCK), dev)
    return Saved(cp, sp, cs, ss), r, c


def _on(stream, t):
    """(handle, stream object or None, device or None) of a call whose first
    tensor is t. Without a stream: the current one of t's device, which need
    not be the current device. The object is there when the tensors have to be
    recorded on the stream. A raw handle does not tell its device: the call is
    on t's, where all its tensors and its workspace then have to be, and the
    null handle is that device's null stream."""
    dev = t.get_device() if t.get_device() >= 0 else None      # None: refused by the checks that follow
    if stream is None:
        import torch
        if dev is None:
            return 0, None, None
        h = torch._C._cuda_getCurrentRawStream(dev)
        return h, None if h == 0 else torch.cuda.current_stream(dev), dev
    h, obj = _stream_handle(stream)
    return h, obj, dev if obj is None else obj.device.index


def _run(name: str, args, dev: Optional[int], refs, sobj) -> None:
    """Calls the library with `dev` current (the null stream is the current
    device's) and records the tensors on the stream."""
    import torch
    if dev is None or dev == torch._C._cuda_getDevice():
        st = _fn(name)(*args)
    else:
        with torch.cuda.device(dev):
            st = _fn(name)(*args)
    if st:
        _check(st, name)
    if sobj is not None:
        _record(refs, sobj)


def _workspace(need: int, workspace, stream, dev):
    """(address, bytes, tensor) of the workspace: the caller's, or one allocated
    on the call's stream."""
    import torch
    if workspace is not None:
        if workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous torch.uint8 tensor")
        _place(workspace, "workspace", dev)
        return workspace.data_ptr(), workspace.numel(), workspace
    if need == 0:
        return 0, 0, None
    if stream is None:
        w = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        s = stream
        if isinstance(stream, int):
            s = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
        with torch.cuda.stream(s):
            w = torch.empty(need, dtype=torch.uint8, device=s.device)
    return w.data_ptr(), need, w


def route_workspace_bytes(tokens: int, k: int, num_experts: int) -> int:
    """Bytes of workspace route_tokens needs (tide_route_workspace)."""
    n = _I64()
    _check(_fn("tide_route_workspace")(tokens, k, num_experts, ctypes.byref(n)),
           "tide_route_workspace")
    return int(n.value)


def route_tokens(experts, num_experts: int, offsets, token_of_row, slots, workspace=None,
                 stream=None) -> None:
    """Stable sort of the (token, choice) pairs by expert (tide_route_tokens).
    experts: (tokens, k) int32 or int64 ids, anything outside [0, num_experts)
    for a pair without an expert; offsets: (num_experts + 1,) int32;
    token_of_row: (tokens * k,) int32; slots: (tokens, k) int32, -1 where a
    pair has no row. workspace: uint8 tensor of route_workspace_bytes(), by
    default allocated for the call."""
    import torch
    sh, sobj, dev = _on(stream, experts)
    if experts.dim() != 2:
        raise ValueError("experts has %d dimensions, expected 2" % experts.dim())
    T, k = experts.shape
    if experts.dtype not in (torch.int32, torch.int64):
        raise TypeError("experts has dtype %s, expected torch.int32 or torch.int64" % experts.dtype)
    ep = _flat(experts, "experts", experts.dtype, (T, k), dev)
    op = _flat(offsets, "offsets", torch.int32, (num_experts + 1,), dev)
    tp = _flat(token_of_row, "token_of_row", torch.int32, (T * k,), dev)
    sp = _flat(slots, "slots", torch.int32, (T, k), dev)
    need = route_workspace_bytes(T, k, num_experts)
    wp, wn, w = _workspace(need, workspace, stream, dev)
    _run("tide_route_tokens", (ep, experts.element_size(), T, k, num_experts, op, tp, sp, wp,
         wn, sh), dev, [experts, offsets, token_of_row, slots, w], sobj)


def dispatch_tokens(x, slots, rows, stream=None) -> None:
    """rows[slots[t, j]] = x[t] (tide_dispatch_tokens); x (tokens, width) and
    rows (capacity, width) bf16 or fp32, slots (tokens, k) from route_tokens.
    Its gradient is combine_tokens of the rows' gradients without weights."""
    import torch
    sh, sobj, dev = _on(stream, x)
    code = _dtype_code(x, "x")
    xp, xs = _mat(x, "x", x.dtype, None, None, dev)
    T, D = x.shape
    k = slots.shape[-1]
    sp = _flat(slots, "slots", torch.int32, (T, k), dev)
    rp, rs = _mat(rows, "rows", x.dtype, None, D, dev)
    _run("tide_dispatch_tokens", (code, xp, xs, T, D, sp, k, rp, rs, rows.shape[0], sh), dev,
         [x, slots, rows], sobj)


def combine_tokens(rows, slots, out, weights=None, stream=None) -> None:
    """out[t] = sum over j of weights[t, j] * rows[slots[t, j]] in fp32, rounded
    once (tide_combine_tokens); weights (tokens, k) fp32, or None for ones."""
    import torch
    sh, sobj, dev = _on(stream, rows)
    code = _dtype_code(rows, "rows")
    rp, rs = _mat(rows, "rows", rows.dtype, None, None, dev)
    n, D = rows.shape
    op, os_ = _mat(out, "out", rows.dtype, None, D, dev)
    T, k = out.shape[0], slots.shape[-1]
    sp = _flat(slots, "slots", torch.int32, (T, k), dev)
    wp = 0 if weights is None else _flat(weights, "weights", torch.float32, (T, k), dev)
    _run("tide_combine_tokens", (code, rp, rs, n, D, sp, wp, T, k, op, os_, sh), dev, [rows,
         slots, out, weights], sobj)


def combine_tokens_grad(dout, rows, slots, weights, drows, dweights, stream=None) -> None:
    """Gradient of combine_tokens (tide_combine_tokens_grad): drows[slots[t, j]]
    = weights[t, j] * dout[t], dweights[t, j] = dout[t] . rows[slots[t, j]].
    weights may be None (ones); with dweights None rows is not read and may be
    None."""
    import torch
    sh, sobj, dev = _on(stream, dout)
    code = _dtype_code(dout, "dout")
    dp, ds = _mat(dout, "dout", dout.dtype, None, None, dev)
    T, D = dout.shape
    k = slots.shape[-1]
    sp = _flat(slots, "slots", torch.int32, (T, k), dev)
    gp, gs = _mat(drows, "drows", dout.dtype, None, D, dev)
    n = drows.shape[0]
    if rows is None and dweights is not None:
        raise ValueError("dweights needs rows")
    rp, rs = (0, D) if rows is None else _mat(rows, "rows", dout.dtype, n, D, dev)
    wp = 0 if weights is None else _flat(weights, "weights", torch.float32, (T, k), dev)
    qp = 0 if dweights is None else _flat(dweights, "dweights", torch.float32, (T, k), dev)
    _run("tide_combine_tokens_grad", (code, dp, ds, rp, rs, n, D, sp, wp, T, k, gp, gs, qp,
         sh), dev, [dout, rows, slots, weights, drows, dweights], sobj)


def checkpoint_pack(x, saved, stream=None) -> None:
    """Packs x (rows, width), bf16 or fp32, into saved = (codes, scales): codes
    (rows, width) torch.float8_e4m3fn, scales (rows, ceil(width / 32))
    torch.float8_e8m0fnu (tide_checkpoint_pack)."""
    sh, sobj, dev = _on(stream, x)
    code = _dtype_code(x, "x")
    xp, xs = _mat(x, "x", x.dtype, None, None, dev)
    n, D = x.shape
    s, _, _ = _saved(saved, "saved", n, D, dev)
    _run("tide_checkpoint_pack", (code, xp, xs, n, D, ctypes.byref(s), sh), dev, [x, *saved], sobj)


def checkpoint_unpack(saved, out, stream=None) -> None:
    """The values a checkpoint stands for, in bf16 or fp32, exactly
    (tide_checkpoint_unpack)."""
    sh, sobj, dev = _on(stream, out)
    code = _dtype_code(out, "out")
    op, os_ = _mat(out, "out", out.dtype, None, None, dev)
    n, D = out.shape
    s, _, _ = _saved(saved, "saved", n, D, dev)
    _run("tide_checkpoint_unpack", (code, ctypes.byref(s), n, D, op, os_, sh), dev, [out,
         *saved], sobj)


def gated_silu(gate, up, out, gate_saved=None, up_saved=None, stream=None) -> None:
    """out = silu(gate) * up and, where they are given, the checkpoints of gate
    and up, in one pass (tide_gated_silu)."""
    sh, sobj, dev = _on(stream, gate)
    code = _dtype_code(gate, "gate")
    gp, gs = _mat(gate, "gate", gate.dtype, None, None, dev)
    n, D = gate.shape
    up_, us = _mat(up, "up", gate.dtype, n, D, dev)
    op, os_ = _mat(out, "out", gate.dtype, n, D, dev)
    a = None if gate_saved is None else _saved(gate_saved, "gate_saved", n, D, dev)[0]
    b = None if up_saved is None else _saved(up_saved, "up_saved", n, D, dev)[0]
    _run("tide_gated_silu", (code, gp, gs, up_, us, n, D, op, os_, a, b, sh), dev, [gate, up,
         out, *(gate_saved or ()), *(up_saved or ())], sobj)


def gated_silu_grad(dout, gate_saved, up_saved, dgate, dup, out=None, stream=None) -> None:
    """Gradient of gated_silu at the checkpoints' values; out, when given,
    receives the activation recomputed from them (tide_gated_silu_grad)."""
    sh, sobj, dev = _on(stream, dout)
    code = _dtype_code(dout, "dout")
    dp, ds = _mat(dout, "dout", dout.dtype, None, None, dev)
    n, D = dout.shape
    a = _saved(gate_saved, "gate_saved", n, D, dev)[0]
    b = _saved(up_saved, "up_saved", n, D, dev)[0]
    gp, gs = _mat(dgate, "dgate", dout.dtype, n, D, dev)
    up_, us = _mat(dup, "dup", dout.dtype, n, D, dev)
    op, os_ = (0, D) if out is None else _mat(out, "out", dout.dtype, n, D, dev)
    _run("tide_gated_silu_grad", (code, dp, ds, a, b, n, D, gp, gs, up_, us, op, os_, sh), dev,
         [dout, *gate_saved, *up_saved, dgate, dup, out], sobj)


def _grads_list(grads, out: int, in_: int, dev: Optional[int]):
    """Array of the addresses of a list of (out, in) gradients. A tensor of the
    transposed shape has as many elements, so the shape itself is compared."""
    want = (out, in_)
    for i, t in enumerate(grads):
        if t is None or isinstance(t, int):
            continue
        if t.shape != want:
            raise ValueError("grads[%d] has shape %s, expected %s" % (i, tuple(t.shape), want))
    _check_many(grads, "bfloat16", [out * in_] * len(grads), lambda i: "grads[%d]" % i)
    for i, t in enumerate(grads):
        if t is not None and not isinstance(t, int) and dev is not None and t.get_device() != dev:
            _place(t, "grads[%d]" % i, dev)
    return (ctypes.c_void_p * max(len(grads), 1))(*[_ptr(t) for t in grads])


def weight_grads_workspace_bytes(rows: int, out: int, in_: int, num_experts: int = 1) -> int:
    """Bytes of workspace weight_grads_bf16 needs (tide_weight_grads_workspace)."""
    n = _I64()
    _check(_fn("tide_weight_grads_workspace")(rows, out, in_, num_experts, ctypes.byref(n)),
           "tide_weight_grads_workspace")
    return int(n.value)


def weight_grads_bf16(dy, x, grads: Union[object, Sequence[object], PointerTable], offsets=None,
                      token_of_row=None, accumulate: bool = False, workspace=None,
                      stream=None) -> None:
    """Weight gradients dy^T x, one a parameter (tide_weight_grads_bf16).

    dy: (rows, out) bf16. x: (x_rows, in) bf16, or a checkpoint (codes, scales).
    grads: bf16 tensors (out, in), one an expert; or one contiguous tensor
    (experts, out, in); or a PointerTable of (out, in) tensors (the caller
    answers for their sizes). offsets, token_of_row: from
    route_tokens; without offsets there is one expert, with every row.
    accumulate: add to what grads holds. workspace: uint8 tensor of
    weight_grads_workspace_bytes(), by default allocated for the call."""
    import numpy as np
    import torch
    sh, sobj, dev = _on(stream, dy)
    dp, ds = _mat(dy, "dy", torch.bfloat16, None, None, dev)
    n, O = dy.shape
    keep = [dy, offsets, token_of_row]
    if isinstance(x, (tuple, list)):
        s, xr, I = _saved(x, "x", None, None, dev)
        xp, xs = 0, 0
        keep += list(x)
    else:
        s = None
        xp, xs = _mat(x, "x", torch.bfloat16, None, None, dev)
        xr, I = x.shape
        keep.append(x)
    if isinstance(grads, PointerTable):
        E, arr = grads.n, grads.arr
        keep += grads.refs
    elif isinstance(grads, (list, tuple)):
        E, arr = len(grads), _grads_list(grads, O, I, dev)
        keep += list(grads)
    else:
        E = grads.shape[0] if grads.dim() == 3 else -1
        base = _flat(grads, "grads", torch.bfloat16, (E, O, I), dev)
        table = np.arange(E, dtype=np.uint64) * (O * I * 2) + np.uint64(base)
        arr = table.ctypes.data
        keep.append(grads)
    op = 0 if offsets is None else _flat(offsets, "offsets", torch.int32, (E + 1,), dev)
    tp = 0 if token_of_row is None else _flat(token_of_row, "token_of_row", torch.int32, (n,), dev)
    need = weight_grads_workspace_bytes(n, O, I, E)
    wp, wn, w = _workspace(need, workspace, stream, dev)
    keep.append(w)
    _run("tide_weight_grads_bf16", (dp, ds, n, O, xp, xs, s, xr, I, op, tp, E, arr, 1 if
         accumulate else 0, wp, wn, sh), dev, keep, sobj)
