"""Operators around the matrix update of a training step (see include/ns.h).

``ns_embedding`` and its gradient, ``ns_rms_norm`` / ``ns_rms_norm_fp8`` and
their gradient, the preference loss on logits and its gradient, the log
probabilities of given tokens and their gradient, and the AdamW step of the
parameters that the Newton-Schulz update does not take. Argument
marshalling only, like the rest of the package, which exports every name of
this module: tensors become pointers, outputs and workspaces come from torch,
work goes to the current stream of the tensors' device. There is no autograd
wrapper: a backward pass calls the gradient functions.

Tensors of rows may have any number of leading dimensions, as long as those
collapse into one without a copy (a slice of the columns, or every k-th row,
of a larger tensor is fine; a transposed view is refused).
"""

from __future__ import annotations

import ctypes
import warnings
from typing import List, Optional, Sequence, Tuple

from . import (NS_DT_BF16, NS_DT_F16, NS_DT_F32, _check, _device_tensor, _dtype_code,
               _own_bytes, _workspace, library)


class _Torch:
    """torch, loaded where a call first needs it: the package and its build
    script import without it."""

    def __getattr__(self, name):
        global torch
        import torch
        return getattr(torch, name)


torch = _Torch()

NS_DT_E4M3 = 3
NS_IDS_I32, NS_IDS_I64 = 0, 1
NS_MAX_ROWS = 1 << 23
BF16_SLOWEST = 1 - 2.0 ** -8     # beta2 above which a bf16 second moment can stand still

_i64, _vp, _f32, _f64, _int = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_double,
                               ctypes.c_int)
_size = ctypes.c_size_t


class _RmsNormArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("x", "residual", "h", "weight", "y", "scales", "rstd")]
                + [(n, _i64) for n in ("rows", "dim", "ldx", "ld_residual", "ldh", "ldy")]
                + [(n, _int) for n in ("x_dtype", "h_dtype", "weight_dtype", "y_dtype")]
                + [("eps", _f32)])


class _RmsNormGradArgs(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("dy", "h", "weight", "rstd", "dh", "dx", "dweight")]
                + [(n, _i64) for n in ("rows", "dim", "lddy", "ldh", "lddh", "lddx")]
                + [(n, _int) for n in ("dy_dtype", "h_dtype", "weight_dtype", "dx_dtype",
                                       "dweight_dtype")])


class _PreferenceArgs(ctypes.Structure):
    _fields_ = [("logits", _vp), ("labels", _vp), ("pairs", _i64), ("length", _i64),
                ("vocab", _i64), ("ld", _i64), ("dtype", _int), ("label_type", _int),
                ("beta", _f32), ("label_smoothing", _f32), ("ld_sequence", _i64)]


class _TokenLogpsArgs(ctypes.Structure):
    _fields_ = [("logits", _vp), ("tokens", _vp), ("rows", _i64), ("vocab", _i64), ("ld", _i64),
                ("top", _i64), ("dtype", _int), ("token_type", _int), ("length", _i64),
                ("ld_sequence", _i64)]


class _AdamwTensor(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("param", "grad", "exp_avg", "exp_avg_sq", "master")]
                + [("elems", _i64)]
                + [(n, _int) for n in ("param_dtype", "grad_dtype", "exp_avg_dtype",
                                       "exp_avg_sq_dtype")]
                + [("weight_decay", _f32)])


SIGNATURES = {
    "ns_embedding": [_vp, _int, _i64, _i64, _i64, _vp, _int, _i64, _f32, _vp, _int, _i64, _vp],
    "ns_embedding_grad_workspace_size": [_i64, _i64, _i64, ctypes.POINTER(_size)],
    "ns_embedding_grad": [_vp, _int, _i64, _vp, _int, _i64, _i64, _i64, _f32, _i64, _int, _vp,
                          _int, _i64, _vp, _size, _vp],
    "ns_rms_norm": [ctypes.POINTER(_RmsNormArgs), _vp],
    "ns_rms_norm_grad_workspace_size": [_i64, _i64, ctypes.POINTER(_size)],
    "ns_rms_norm_grad": [ctypes.POINTER(_RmsNormGradArgs), _vp, _size, _vp],
    "ns_preference_loss_workspace_size": [_i64, _i64, _i64, ctypes.POINTER(_size)],
    "ns_preference_loss": [ctypes.POINTER(_PreferenceArgs), _vp, _vp, _vp, _vp, _vp, _vp, _size,
                           _vp],
    "ns_preference_loss_grad": [ctypes.POINTER(_PreferenceArgs), _vp, _vp, _vp, _vp, _i64, _vp],
    "ns_token_logps_workspace_size": [_i64, _i64, _i64, ctypes.POINTER(_size)],
    "ns_token_logps": [ctypes.POINTER(_TokenLogpsArgs), _vp, _vp, _vp, _vp, _vp, _vp, _size, _vp],
    "ns_token_logps_grad": [ctypes.POINTER(_TokenLogpsArgs), _vp, _vp, _vp, _vp, _vp, _i64, _vp],
    "ns_adamw_step": [ctypes.POINTER(_AdamwTensor), _int, _i64, _f64, _f64, _f64, _f64, _vp],
}


# Small calls take about as long as their launch: the helpers below run for
# every tensor of a call and are written for few steps.

_codes = {}      # of the tensor types met so far
_id_types = {}
_raw_stream = None


def _stream_of(dev: int) -> int:
    """The current stream of a device as a pointer; without a Stream object,
    where this torch can say it so."""
    global _raw_stream
    if _raw_stream is None:
        _raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
                       or (lambda index: torch.cuda.current_stream(index).cuda_stream))
    return _raw_stream(dev)


def _device_of(t, name: str) -> int:
    """Index of the device of a call: the first tensor's, which must be the current one."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        _device_tensor(t, name)   # says what is wrong
    return dev


def _code(t) -> int:
    code = _codes.get(t.dtype)
    if code is None:
        code = _codes[t.dtype] = _dtype_code(t.dtype)
    return code


def _ids_type(t, name: str) -> int:
    code = _id_types.get(t.dtype)
    if code is None:
        code = {torch.int32: NS_IDS_I32, torch.int64: NS_IDS_I64}.get(t.dtype)
        if code is None:
            raise TypeError(f"{name} must be int32 or int64, not {t.dtype}")
        _id_types[t.dtype] = code
    return code


def _rows_of(t, name: str, dev: int) -> Tuple[int, int, int]:
    """(rows, columns, leading dimension) of a tensor of rows on device `dev`."""
    if t.get_device() != dev:
        _device_tensor(t, name)
    shape = t.shape
    if len(shape) == 0:
        raise ValueError(f"{name} must have at least one dimension")
    cols = shape[-1]
    if t.is_contiguous():
        return (t.numel() // cols if cols else 0), cols, cols
    stride = t.stride()
    if cols > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: rows must be contiguous (stride(-1) == 1)")
    rows, ld = 1, None
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 0:
            return 0, cols, max(cols, 1)
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * rows:
            raise ValueError(f"{name}: the dimensions before the last do not collapse into rows of "
                             f"one stride (shape {tuple(shape)}, strides {tuple(stride)})")
        rows *= n
    if ld is None:
        ld = cols
    if ld < cols:
        raise ValueError(f"{name}: row stride {ld} is smaller than the row length {cols} "
                         f"(overlapping rows, e.g. an expanded view)")
    return rows, cols, ld


def _mismatch(t, shape, name: str, dtype):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    _device_tensor(t, name)
    raise ValueError(f"{name} must be contiguous")


def _like_rows(t, shape, name: str, dev: int, dtype=None) -> int:
    """Leading dimension of a tensor that must have this shape (and type)."""
    if t.shape != shape or (dtype is not None and t.dtype != dtype):
        _mismatch(t, shape, name, dtype)
    return _rows_of(t, name, dev)[2]


def _dense(t, shape, name: str, dev: int, dtype=None) -> int:
    """Pointer of a dense tensor that must have this shape (and type)."""
    if (t.shape != shape or t.get_device() != dev or not t.is_contiguous()
            or (dtype is not None and t.dtype != dtype)):
        _mismatch(t, shape, name, dtype)
    return t.data_ptr()


def _sized(name: str, *args) -> int:
    nbytes = _size(0)
    _check(getattr(library(), name)(*args, ctypes.byref(nbytes)), name)
    return nbytes.value


def _given_or_new(workspace, nbytes: int, device):
    if workspace is None or workspace.numel() * workspace.element_size() < nbytes:
        return _workspace(nbytes, device)
    return _own_bytes(workspace)


# ------------------------------------------------------------------ embedding

def ns_embedding(table, ids, scale: float = 1.0, out_dtype=None, out=None):
    """scale * table[ids], for ids (int32 or int64) of any shape; an id outside
    the table gives zeros. Returns a tensor of shape ids.shape + (dim,)."""
    if table.dim() != 2:
        raise ValueError("table must be 2-D")
    dev = _device_of(table, "table")
    rows, dim, ld = _rows_of(table, "table", dev)
    id_type = _ids_type(ids, "ids")
    if ids.get_device() != dev:
        _device_tensor(ids, "ids")
    ids = ids if ids.is_contiguous() else ids.contiguous()
    shape = ids.shape + (dim,)
    if out is None:
        out = torch.empty(shape, dtype=out_dtype or table.dtype, device=table.device)
        ld_out = dim
    else:
        ld_out = _like_rows(out, shape, "out", dev, out_dtype)
    _check(library().ns_embedding(table.data_ptr(), _code(table), rows, dim, ld, ids.data_ptr(),
                                  id_type, ids.numel(), scale, out.data_ptr(), _code(out), ld_out,
                                  _stream_of(dev)), "ns_embedding")
    return out


def ns_embedding_grad_workspace_size(rows: int, dim: int, count: int) -> int:
    return _sized("ns_embedding_grad_workspace_size", rows, dim, count)


def ns_embedding_grad(grad_out, ids, rows: int, scale: float = 1.0,
                      padding_idx: Optional[int] = None, out_dtype=None, out=None,
                      accumulate: bool = False, workspace=None):
    """Gradient of ns_embedding's table (rows, dim): scale times the sum of
    grad_out over the places that name each row. With accumulate it is added
    to out, which must then be given. ids outside the table and padding_idx
    contribute nothing."""
    dev = _device_of(grad_out, "grad_out")
    count, dim, ld = _rows_of(grad_out, "grad_out", dev)
    id_type = _ids_type(ids, "ids")
    if ids.get_device() != dev:
        _device_tensor(ids, "ids")
    if ids.shape != grad_out.shape[:-1]:
        raise ValueError(f"ids have shape {tuple(ids.shape)}, grad_out {tuple(grad_out.shape)}")
    if padding_idx is not None and not 0 <= padding_idx < rows:
        raise ValueError(f"padding_idx {padding_idx} is not a row of the table (0 to {rows - 1})")
    if accumulate and out is None:
        raise ValueError("accumulate adds to out: give it")
    ids = ids if ids.is_contiguous() else ids.contiguous()
    if out is None:
        out = torch.empty((rows, dim), dtype=out_dtype or grad_out.dtype, device=grad_out.device)
        ld_out = dim
    else:
        ld_out = _like_rows(out, (rows, dim), "out", dev, out_dtype)
    workspace = _given_or_new(workspace, ns_embedding_grad_workspace_size(rows, dim, count),
                              grad_out.device)
    _check(library().ns_embedding_grad(
        grad_out.data_ptr(), _code(grad_out), ld, ids.data_ptr(), id_type, count, rows, dim, scale,
        -1 if padding_idx is None else padding_idx, 1 if accumulate else 0, out.data_ptr(),
        _code(out), ld_out, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream_of(dev)), "ns_embedding_grad")
    return out


# ------------------------------------------------------------------- RMS norm

def _rms_norm(x, weight, residual, eps, y, y_code, scales, h, dev):
    rows, dim, ldx = _rows_of(x, "x", dev)
    code = h_code = _code(x)
    res_ptr, h_ptr, ld_residual, ldh = None, None, 0, 0
    if residual is None:
        if h is not None:
            raise ValueError("h is written only with a residual")
        h = x
    else:
        ld_residual = _like_rows(residual, x.shape, "residual", dev)
        res_ptr, h_code = residual.data_ptr(), _code(residual)
        if h is None:
            h = torch.empty(x.shape, dtype=residual.dtype, device=x.device)
            ldh = dim
        else:
            ldh = _like_rows(h, x.shape, "h", dev, residual.dtype)
        h_ptr = h.data_ptr()
    rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    args = _RmsNormArgs(x.data_ptr(), res_ptr, h_ptr, _dense(weight, (dim,), "weight", dev),
                        y.data_ptr(), scales.data_ptr() if scales is not None else None,
                        rstd.data_ptr(), rows, dim, ldx, ld_residual, ldh, dim, code, h_code,
                        _code(weight), y_code, eps)
    _check(library().ns_rms_norm(args, _stream_of(dev)), "ns_rms_norm")
    return h, rstd


def ns_rms_norm(x, weight, residual=None, eps: float = 1e-6, out_dtype=None, h=None):
    """RMS norm of the last dimension, of x + residual if that is given.
    Returns (y, h, rstd): y in out_dtype (x's by default), h the stored sum
    that was normalised (x itself without a residual) and 1 / rms of each row
    (fp32), both for ns_rms_norm_grad. The residual may be x's type or fp32;
    the sum has its type, and `h` may name its buffer (the residual's own, or
    x's where the types agree)."""
    dev = _device_of(x, "x")
    y = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
    h, rstd = _rms_norm(x, weight, residual, eps, y, _code(y), None, h, dev)
    return y, h, rstd


def ns_rms_norm_fp8(x, weight, residual=None, eps: float = 1e-6, h=None):
    """ns_rms_norm with the output as e4m3 codes and one fp32 scale for each
    row: codes are those of y * (1 / scale), code * scale stands for y.
    Returns (codes, scales, h, rstd)."""
    dev = _device_of(x, "x")
    q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    h, rstd = _rms_norm(x, weight, residual, eps, q, NS_DT_E4M3, scales, h, dev)
    return q, scales, h, rstd


def ns_rms_norm_grad_workspace_size(rows: int, dim: int) -> int:
    return _sized("ns_rms_norm_grad_workspace_size", rows, dim)


def ns_rms_norm_grad(dy, h, weight, rstd, dh=None, dx=None, dx_dtype=None, dweight_dtype=None,
                     workspace=None):
    """Gradients of ns_rms_norm (of ns_rms_norm_fp8 too): (dx, dweight), where
    dx is the gradient of x and of the residual. `h` and `rstd` are the norm's
    own; dh is the gradient that reaches h past the norm, of dx's type (dx may
    be its buffer). dweight has weight's type unless dweight_dtype says so."""
    dev = _device_of(dy, "dy")
    rows, dim, lddy = _rows_of(dy, "dy", dev)
    shape = dy.shape
    if dx is None:
        dx = torch.empty(shape, dtype=dx_dtype or (dh.dtype if dh is not None else dy.dtype),
                         device=dy.device)
        lddx = dim
    else:
        lddx = _like_rows(dx, shape, "dx", dev, dx_dtype)
    dh_ptr, lddh = None, 0
    if dh is not None:
        dh_ptr, lddh = dh.data_ptr(), _like_rows(dh, shape, "dh", dev, dx.dtype)
    dweight = torch.empty(dim, dtype=dweight_dtype or weight.dtype, device=dy.device)
    args = _RmsNormGradArgs(
        dy.data_ptr(), h.data_ptr(), _dense(weight, (dim,), "weight", dev),
        _dense(rstd, shape[:-1], "rstd", dev, torch.float32), dh_ptr, dx.data_ptr(),
        dweight.data_ptr(), rows, dim, lddy, _like_rows(h, shape, "h", dev), lddh, lddx, _code(dy),
        _code(h), _code(weight), _code(dx), _code(dweight))
    workspace = _given_or_new(workspace, ns_rms_norm_grad_workspace_size(rows, dim), dy.device)
    _check(library().ns_rms_norm_grad(args, workspace.data_ptr(),
                                      workspace.numel() * workspace.element_size(),
                                      _stream_of(dev)), "ns_rms_norm_grad")
    return dx, dweight


# ------------------------------------------------------------ preference loss

def _preference_args(logits, labels, beta, label_smoothing, dev):
    shape = logits.shape
    if len(shape) != 3 or shape[0] % 2:
        raise ValueError("logits must be (2 * pairs, length, vocab): the preferred sequences, then "
                         "the others")
    n, length, vocab = shape
    ld, sequence = vocab, 0
    if not logits.is_contiguous():   # positions and sequences may each lie further apart
        apart, step, one = logits.stride()
        if vocab > 1 and one != 1:
            raise ValueError("logits: rows must be contiguous (stride(-1) == 1)")
        ld = step if length > 1 else vocab
        sequence = apart if n > 1 else 0
        if n > 1 and length > 1 and vocab <= sequence and ld >= (n - 1) * sequence + vocab:
            raise ValueError(f"logits: sequences must lie one behind the other (shape {tuple(shape)}, "
                             f"strides {tuple(logits.stride())}): positions lie further apart than "
                             f"sequences here; pass logits.contiguous()")
        if ld < vocab or (n > 1 and sequence < (length - 1) * ld + vocab):
            raise ValueError(f"logits: overlapping rows (shape {tuple(shape)}, strides "
                             f"{tuple(logits.stride())})")
    args = _PreferenceArgs(logits.data_ptr(), _dense(labels, shape[:2], "labels", dev), n // 2, length,
                           vocab, ld, _code(logits), _ids_type(labels, "labels"), beta,
                           label_smoothing, sequence)
    return args


def ns_preference_loss_workspace_size(pairs: int, length: int, vocab: int) -> int:
    return _sized("ns_preference_loss_workspace_size", pairs, length, vocab)


def ns_preference_loss(logits, labels, ref_logps, beta: float = 0.1, label_smoothing: float = 0.0,
                       workspace=None):
    """Preference loss of paired sequences from the policy's logits (2 pairs,
    length, vocab; a slice such as logits[:, :-1] is fine, time-major logits
    are not), the labels (2 pairs, length; a position whose label is not in
    the vocabulary, such as -100, does not count) and the reference's log
    probability of each sequence (2 pairs, fp32). Returns fp32 tensors
    (losses, margins, logps, lse): the loss and margin of each pair, the
    policy's log probability of each sequence, and each position's log sum of
    exponentials, which the gradient needs."""
    dev = _device_of(logits, "logits")
    labels = labels if labels.is_contiguous() else labels.contiguous()
    args = _preference_args(logits, labels, beta, label_smoothing, dev)
    pairs, length, device = args.pairs, args.length, logits.device
    ref = _dense(ref_logps, (2 * pairs,), "ref_logps", dev, torch.float32)
    out = torch.empty(2 * pairs * (length + 2), dtype=torch.float32, device=device)
    losses, margins, logps, lse = out.split((pairs, pairs, 2 * pairs, 2 * pairs * length))
    workspace = _given_or_new(workspace,
                              ns_preference_loss_workspace_size(pairs, length, args.vocab), device)
    at = out.data_ptr()
    _check(library().ns_preference_loss(
        args, ref, at, at + 4 * pairs, at + 8 * pairs, at + 16 * pairs, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_of(dev)), "ns_preference_loss")
    return losses, margins, logps, lse.view(2 * pairs, length)


def ns_preference_loss_grad(logits, labels, margins, lse, dlosses, beta: float = 0.1,
                            label_smoothing: float = 0.0, out=None):
    """Gradient of ns_preference_loss's losses with respect to the logits, for
    margins and lse as it returned them and the gradient of each loss, dlosses
    (pairs, fp32). `out` may be the logits themselves."""
    dev = _device_of(logits, "logits")
    labels = labels if labels.is_contiguous() else labels.contiguous()
    args = _preference_args(logits, labels, beta, label_smoothing, dev)
    pairs, shape = args.pairs, logits.shape
    if out is None:
        out = torch.empty(shape, dtype=logits.dtype, device=logits.device)
        ld_out = args.vocab
    elif out.data_ptr() == logits.data_ptr():
        if out.dtype != logits.dtype or out.shape != shape or out.stride() != logits.stride():
            raise ValueError("out begins where the logits do, but is another view of that memory")
        ld_out = args.ld
    else:
        ld_out = _like_rows(out, shape, "out", dev, logits.dtype)
    _check(library().ns_preference_loss_grad(
        args, _dense(margins, (pairs,), "margins", dev, torch.float32),
        _dense(lse, shape[:2], "lse", dev, torch.float32),
        _dense(dlosses, (pairs,), "dlosses", dev, torch.float32), out.data_ptr(), ld_out,
        _stream_of(dev)), "ns_preference_loss_grad")
    return out


# --------------------------------------------------- token log probabilities

def _token_logps_args(logits, tokens, top, dev):
    shape = logits.shape
    if len(shape) < 1:
        raise ValueError("logits must have at least one dimension")
    length = sequence = 0
    if len(shape) < 3 or logits.is_contiguous() or 0 in shape:
        rows, vocab, ld = _rows_of(logits, "logits", dev)
    else:   # positions and what comes before them may each lie further apart
        length, vocab, ld = _rows_of(logits[(0,) * (len(shape) - 2)], "logits", dev)
        seqs, span, sequence = _rows_of(logits[..., 0, :1], "logits", dev)
        rows = seqs * length
        if seqs > 1 and sequence < (length - 1) * ld + vocab:
            raise ValueError(f"logits: overlapping sequences (shape {tuple(shape)}, strides "
                             f"{tuple(logits.stride())})")
    return _TokenLogpsArgs(logits.data_ptr(), _dense(tokens, shape[:-1], "tokens", dev), rows, vocab, ld, top,
                           _code(logits), _ids_type(tokens, "tokens"), length, sequence)


def ns_token_logps_workspace_size(rows: int, vocab: int, top: int = 0) -> int:
    return _sized("ns_token_logps_workspace_size", rows, vocab, top)


def ns_token_logps(logits, tokens, top: int = 0, workspace=None):
    """Log probabilities of the tokens (int32 or int64, of any shape) from
    logits of shape tokens.shape + (vocab,) (a slice such as logits[:, :-1] is
    fine). Returns (logps, lse, entropy,
    top_logps, top_ids): the first three are fp32 and of the tokens' shape, the
    log sum of exponentials and entropy of each row are also what the gradient
    needs; top_logps (fp32) and top_ids (of the tokens' type) are each row's
    `top` (0 to 64) likeliest entries, of equal ones the lowest index first, of
    shape tokens.shape + (top,), or None if top is 0. Rows whose token is not in
    the vocabulary, such as -100, do not count: 0, and -1 in top_ids."""
    dev = _device_of(logits, "logits")
    tokens = tokens if tokens.is_contiguous() else tokens.contiguous()
    args = _token_logps_args(logits, tokens, top, dev)
    rows, shape, device = args.rows, logits.shape[:-1], logits.device
    out = torch.empty((3,) + shape, dtype=torch.float32, device=device)
    top_logps = top_ids = logps_ptr = ids_ptr = ws_ptr = None
    if top > 0:
        top_logps = torch.empty(shape + (top,), dtype=torch.float32, device=device)
        top_ids = torch.empty(shape + (top,), dtype=tokens.dtype, device=device)
        logps_ptr, ids_ptr = top_logps.data_ptr(), top_ids.data_ptr()
    nbytes = ns_token_logps_workspace_size(rows, args.vocab, top)
    if nbytes:
        workspace = _given_or_new(workspace, nbytes, device)
        ws_ptr, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    at = out.data_ptr()
    _check(library().ns_token_logps(args, at, at + 4 * rows, at + 8 * rows, logps_ptr, ids_ptr, ws_ptr, nbytes,
                                    _stream_of(dev)), "ns_token_logps")
    logps, lse, entropy = out.unbind(0)
    return logps, lse, entropy, top_logps, top_ids


def ns_token_logps_grad(logits, tokens, lse, entropy, dlogps, dentropy=None, out=None):
    """Gradient of ns_token_logps's log probabilities and entropies with respect
    to the logits, for lse and entropy as it returned them and the gradient of
    each row's (fp32, of the tokens' shape; dlogps or dentropy may be None).
    `out` may be the logits themselves."""
    dev = _device_of(logits, "logits")
    tokens = tokens if tokens.is_contiguous() else tokens.contiguous()
    args = _token_logps_args(logits, tokens, 0, dev)
    shape = logits.shape
    if out is None:
        out = torch.empty_like(logits, memory_format=torch.contiguous_format)
        ld_out = args.vocab
    elif out.data_ptr() == logits.data_ptr() and args.rows > 0:
        if out.dtype != logits.dtype or out.shape != shape or out.stride() != logits.stride():
            raise ValueError("out begins where the logits do, but is another view of that memory")
        ld_out = args.ld
    else:
        ld_out = _like_rows(out, shape, "out", dev, logits.dtype)

    def row(t, name):
        return None if t is None else _dense(t, shape[:-1], name, dev, torch.float32)

    if dentropy is not None and entropy is None:
        raise ValueError("dentropy needs the entropy")
    _check(library().ns_token_logps_grad(args, row(lse, "lse"), row(entropy, "entropy"),
                                         row(dlogps, "dlogps"), row(dentropy, "dentropy"),
                                         out.data_ptr(), ld_out, _stream_of(dev)), "ns_token_logps_grad")
    return out


# ---------------------------------------------------------------------- AdamW

def ns_adamw_step(params: List, grads: List, exp_avgs: List, exp_avg_sqs: List, step: int,
                  lr: float, betas: Sequence[float] = (0.9, 0.999), eps: float = 1e-8,
                  weight_decays: Optional[Sequence[float]] = None,
                  masters: Optional[List] = None) -> None:
    """One AdamW step, in place, of the parameters that are not matrices of
    the Newton-Schulz update. Tensors are dense and of any shape; `masters`
    are fp32 copies that hold the weights, whose rounded values the params
    then receive (None entries: no copy). weight_decays: one for each tensor
    (0 by default).

    exp_avg_sqs may be fp32 or bf16. In bf16 a step that changes one by less
    than half a rounding step changes nothing: it settles within
    2^-8 / (1 - betas[1]) of g^2, relative to itself (8% at 0.95, 39% at 0.99),
    and above betas[1] = 1 - 2^-8 it stops falling under small gradients (at
    the default 0.999 at once); a RuntimeWarning says so. Keep it in fp32
    there."""
    count = len(params)
    if count == 0:
        return
    weight_decays = [0.0] * count if weight_decays is None else weight_decays
    masters = [None] * count if masters is None else masters
    if not (len(grads) == len(exp_avgs) == len(exp_avg_sqs) == len(weight_decays) == len(masters)
            == count):
        raise ValueError("params, grads, exp_avgs, exp_avg_sqs, weight_decays and masters must have "
                         "the same length")
    dev = _device_of(params[0], "param 0")
    shapes = [p.shape for p in params]
    columns = []
    for name, group in (("param", params), ("grad", grads), ("exp_avg", exp_avgs),
                        ("exp_avg_sq", exp_avg_sqs)):
        for t, shape in zip(group, shapes):
            if t.shape != shape or t.get_device() != dev or not t.is_contiguous():
                _mismatch(t, shape, name, None)
        columns.append([t.data_ptr() for t in group])
    columns.append([None if w is None else _dense(w, shape, "master", dev, torch.float32)
                    for w, shape in zip(masters, shapes)])
    columns.append([p.numel() for p in params])
    columns += [[_code(t) for t in group] for group in (params, grads, exp_avgs, exp_avg_sqs)]
    if betas[1] > BF16_SLOWEST and NS_DT_BF16 in columns[-1]:
        warnings.warn(f"a bf16 exp_avg_sq stops falling with beta2 = {betas[1]}: a step of 1 - beta2 of "
                      f"the value is below half a rounding step (up to 2^-8). Keep it in fp32, or take "
                      f"beta2 <= {BF16_SLOWEST}", RuntimeWarning, stacklevel=2)
    tensors = (_AdamwTensor * count)(*zip(*columns, weight_decays))
    _check(library().ns_adamw_step(tensors, count, step, lr, betas[0], betas[1], eps,
                                   _stream_of(dev)), "ns_adamw_step")


__all__ = ["NS_DT_E4M3", "NS_IDS_I32", "NS_IDS_I64", "NS_MAX_ROWS", "ns_embedding",
           "ns_embedding_grad", "ns_embedding_grad_workspace_size", "ns_rms_norm",
           "ns_rms_norm_fp8", "ns_rms_norm_grad", "ns_rms_norm_grad_workspace_size",
           "ns_preference_loss", "ns_preference_loss_grad", "ns_preference_loss_workspace_size",
           "ns_token_logps", "ns_token_logps_grad", "ns_token_logps_workspace_size",
           "ns_adamw_step"]
