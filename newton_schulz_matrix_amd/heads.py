"""Operators on heads, tensors of shape (tokens, heads, dim) (see include/ns.h):
the norm of queries and keys with the rotation of their positions, and causal
attention over packed sequences, with their gradients.

Argument marshalling in the manner of ``operators``; the package exports every
name of this module. Queries, keys and values may be views of one projection's
output, and the outputs that a call is given may be views of one buffer: any
strides of tokens and heads are taken as long as the last dimension is
contiguous and, in a tensor that is written, heads do not overlap.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence

from . import _check, _device_tensor, library
from .operators import (_code, _dense, _device_of, _f32, _given_or_new, _i64, _ids_type, _int, _mismatch,
                        _size, _sized, _stream_of, _vp, torch)

NS_MAX_HEADS = 1024
NS_MAX_HEAD_TILES = 1 << 22


class _Heads(ctypes.Structure):
    _fields_ = [("data", _vp), ("ld_token", _i64), ("ld_head", _i64)]


class _QkNormRopeArgs(ctypes.Structure):
    _fields_ = ([("q", _Heads), ("k", _Heads)]
                + [(n, _vp) for n in ("q_weight", "k_weight", "positions", "inv_freq")]
                + [(n, _i64) for n in ("tokens", "q_heads", "k_heads", "dim", "rotary", "ld_positions",
                                       "axes")]
                + [("sections", _i64 * 4)]
                + [(n, _int) for n in ("interleaved", "dtype", "weight_dtype", "position_type")]
                + [("eps", _f32)])


class _AttentionArgs(ctypes.Structure):
    _fields_ = ([(n, _Heads) for n in ("q", "k", "v")] + [("offsets", _vp)]
                + [(n, _i64) for n in ("tokens", "sequences", "q_heads", "k_heads", "dim")]
                + [("dtype", _int), ("clear_rest", _int), ("scale", _f32)])


SIGNATURES = {
    "ns_qk_norm_rope": [ctypes.POINTER(_QkNormRopeArgs), _Heads, _Heads, _vp],
    "ns_qk_norm_rope_grad_workspace_size": [_i64, _i64, ctypes.POINTER(_size)],
    "ns_qk_norm_rope_grad": [ctypes.POINTER(_QkNormRopeArgs), _Heads, _Heads, _Heads, _Heads, _vp, _vp,
                             _int, _vp, _size, _vp],
    "ns_attention_workspace_size": [_i64] * 5 + [ctypes.POINTER(_size)],
    "ns_attention": [ctypes.POINTER(_AttentionArgs), _Heads, _vp, _vp, _size, _vp],
    "ns_attention_grad_workspace_size": [_i64] * 5 + [ctypes.POINTER(_size)],
    "ns_attention_grad": [ctypes.POINTER(_AttentionArgs), _Heads, _Heads, _vp, _Heads, _Heads, _Heads,
                          _vp, _size, _vp],
}


# (data, ld_token, ld_head): a structure within another takes them as they are.

def _heads_of(t, name: str, dev: int):
    """Address and strides of a (tokens, heads, dim) tensor on device `dev`."""
    if t.get_device() != dev:
        _device_tensor(t, name)
    if t.dim() != 3:
        raise ValueError(f"{name} must be (tokens, heads, dim), not {tuple(t.shape)}")
    ld_token, ld_head, one = t.stride()
    if one != 1 and t.shape[2] > 1:
        raise ValueError(f"{name}: heads must be contiguous (stride(-1) == 1)")
    return t.data_ptr(), ld_token, ld_head


def _heads_like(t, name: str, dev: int, like) -> _Heads:
    """The same of a tensor that must have like's shape and type."""
    if t.shape != like.shape or t.dtype is not like.dtype:
        _mismatch(t, like.shape, name, like.dtype)
    return _Heads(*_heads_of(t, name, dev))


def _new_or_heads(t, name: str, dev: int, like):
    """An output of `like`'s shape and type: (tensor, its _Heads)."""
    if t is not None:
        return t, _heads_like(t, name, dev, like)
    t = torch.empty_like(like, memory_format=torch.contiguous_format)
    _, heads, dim = t.shape
    return t, _Heads(t.data_ptr(), heads * dim, dim)


# ------------------------------------- norm and rotation of queries and keys

_NO_SECTIONS = (_i64 * 4)()


def _qk_args(q, k, q_weight, k_weight, positions, inv_freq, eps, sections, interleaved, dev):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError(f"q and k must be (tokens, heads, dim), not {tuple(q.shape)} and {tuple(k.shape)}")
    tokens, q_heads, dim = q.shape
    k_tokens, k_heads, k_dim = k.shape
    if k_tokens != tokens or k_dim != dim:
        raise ValueError(f"q and k must be (tokens, heads, dim) of the same tokens and dim, not "
                         f"{tuple(q.shape)} and {tuple(k.shape)}")
    dtype = q.dtype
    if k.dtype is not dtype:
        _mismatch(k, k.shape, "k", dtype)
    heads_q, heads_k = _heads_of(q, "q", dev), _heads_of(k, "k", dev)
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight: give both or neither")
    q_ptr = k_ptr = None
    weight_code = 0
    if q_weight is not None:
        q_ptr = _dense(q_weight, (dim,), "q_weight", dev)
        k_ptr = _dense(k_weight, (dim,), "k_weight", dev, q_weight.dtype)
        weight_code = _code(q_weight)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be 1-D: one for each pair that turns")
    pairs = inv_freq.shape[0]
    place = positions.shape
    axes = 1 if len(place) == 1 else place[0] if len(place) == 2 else 5
    if axes > 4 or place[-1] != tokens:
        raise ValueError(f"positions must be (tokens,) or (axes, tokens) with up to 4 axes, not "
                         f"{tuple(place)} for {tokens} tokens")
    parts, ld_positions = _NO_SECTIONS, 0
    if axes > 1:
        if sections is None or len(sections) != axes or sum(sections) != pairs or min(sections) < 0:
            raise ValueError(f"sections must give the pairs of each of the {axes} axes, {pairs} in all")
        parts, ld_positions = (_i64 * 4)(*sections), positions.stride(0)
    elif sections is not None and list(sections) != [pairs]:
        raise ValueError(f"sections: one axis has all {pairs} pairs")
    if positions.get_device() != dev:
        _device_tensor(positions, "positions")
    if not positions.is_contiguous() and positions.stride(-1) != 1 and tokens > 1:
        raise ValueError("positions: an axis' positions must be contiguous")
    return _QkNormRopeArgs(heads_q, heads_k, q_ptr, k_ptr, positions.data_ptr(),
                           _dense(inv_freq, (pairs,), "inv_freq", dev, torch.float32), tokens, q_heads,
                           k_heads, dim, 2 * pairs, ld_positions, axes, parts, 1 if interleaved else 0,
                           _code(q), weight_code, _ids_type(positions, "positions"), eps)


def ns_qk_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps: float = 1e-6,
                    sections: Optional[Sequence[int]] = None, interleaved: bool = False, out_q=None,
                    out_k=None):
    """RMS norm of each query's and key's head (q (tokens, q_heads, dim), k
    (tokens, k_heads, dim)) with the rotation of its position in the same pass.
    The first 2 * len(inv_freq) columns turn, in pairs (i, i + half) or, with
    interleaved, (2 i, 2 i + 1), by the angle position * inv_freq[i] (taken in 64
    bits). positions is (tokens,), int32 or int64, or (axes, tokens) with
    `sections`, the number of pairs of each axis (such as time, height, width).
    Weights are (dim,), of q's type or fp32; None for both leaves out the norm.
    Returns (q, k); out_q may be q itself and out_k k, which the gradient then no
    longer has."""
    dev = _device_of(q, "q")
    args = _qk_args(q, k, q_weight, k_weight, positions, inv_freq, eps, sections, interleaved, dev)
    out_q, to_q = _new_or_heads(out_q, "out_q", dev, q)
    out_k, to_k = _new_or_heads(out_k, "out_k", dev, k)
    _check(library().ns_qk_norm_rope(args, to_q, to_k, _stream_of(dev)), "ns_qk_norm_rope")
    return out_q, out_k


def ns_qk_norm_rope_grad_workspace_size(tokens: int, dim: int) -> int:
    return _sized("ns_qk_norm_rope_grad_workspace_size", tokens, dim)


def ns_qk_norm_rope_grad(dout_q, dout_k, q, k, q_weight, k_weight, positions, inv_freq,
                         eps: float = 1e-6, sections: Optional[Sequence[int]] = None,
                         interleaved: bool = False, dq=None, dk=None, dweight_dtype=None,
                         workspace=None):
    """Gradients of ns_qk_norm_rope for the gradients of its outputs: (dq, dk,
    dq_weight, dk_weight), the last two None without weights and of weights' type
    unless dweight_dtype says so. q and k are the call's inputs. dq may be
    dout_q's buffer and dk dout_k's, or both views of one larger buffer."""
    dev = _device_of(q, "q")
    args = _qk_args(q, k, q_weight, k_weight, positions, inv_freq, eps, sections, interleaved, dev)
    g_q, g_k = _heads_like(dout_q, "dout_q", dev, q), _heads_like(dout_k, "dout_k", dev, k)
    dq, to_q = _new_or_heads(dq, "dq", dev, q)
    dk, to_k = _new_or_heads(dk, "dk", dev, k)
    if q_weight is None:
        _check(library().ns_qk_norm_rope_grad(args, g_q, g_k, to_q, to_k, None, None, 0, None, 0,
                                              _stream_of(dev)), "ns_qk_norm_rope_grad")
        return dq, dk, None, None
    dim = q.shape[2]
    dweights = torch.empty((2, dim), dtype=dweight_dtype or q_weight.dtype, device=q.device)
    dqw, dkw = dweights.unbind(0)
    workspace = _given_or_new(workspace, ns_qk_norm_rope_grad_workspace_size(q.shape[0], dim), q.device)
    _check(library().ns_qk_norm_rope_grad(args, g_q, g_k, to_q, to_k, dqw.data_ptr(), dkw.data_ptr(),
                                          _code(dweights), workspace.data_ptr(),
                                          workspace.numel() * workspace.element_size(),
                                          _stream_of(dev)), "ns_qk_norm_rope_grad")
    return dq, dk, dqw, dkw


# ------------------------------------------------------------------ attention

def _attention_args(q, k, v, offsets, scale, clear_rest, dev):
    shape, k_shape = q.shape, k.shape
    if len(shape) != 3 or len(k_shape) != 3 or k_shape != v.shape or shape[::2] != k_shape[::2]:
        raise ValueError(f"q (tokens, q_heads, dim) and k, v (tokens, k_heads, dim) do not go together: "
                         f"{tuple(shape)}, {tuple(k_shape)}, {tuple(v.shape)}")
    if k.dtype is not q.dtype or v.dtype is not q.dtype:
        _mismatch(k, k_shape, "k", q.dtype) if k.dtype is not q.dtype else _mismatch(v, k_shape, "v", q.dtype)
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError("offsets must be 1-D: where each sequence begins, and the end of the last")
    tokens, q_heads, dim = shape
    return _AttentionArgs(_heads_of(q, "q", dev), _heads_of(k, "k", dev), _heads_of(v, "v", dev),
                          _dense(offsets, offsets.shape, "offsets", dev, torch.int32), tokens,
                          offsets.shape[0] - 1, q_heads, k_shape[1], dim, _code(q),
                          1 if clear_rest else 0, dim ** -0.5 if scale is None else scale)


def ns_attention_workspace_size(tokens: int, sequences: int, q_heads: int, k_heads: int, dim: int) -> int:
    return _sized("ns_attention_workspace_size", tokens, sequences, q_heads, k_heads, dim)


def ns_attention(q, k, v, offsets, scale: Optional[float] = None, out=None, workspace=None):
    """Causal attention of packed sequences: q (tokens, q_heads, dim), k and v
    (tokens, k_heads, dim) in bf16 or fp16, q_heads a multiple of k_heads, dim a
    multiple of 8 up to 128; offsets (sequences + 1) int32 on the device, where
    each sequence begins and the last one ends (offsets[0] is 0);
    (tokens // 128 + sequences + 1) * q_heads up to NS_MAX_HEAD_TILES. scale is
    dim ** -0.5 by default. Returns (out, lse): out like q, and the log sum of
    exponentials of each row, (q_heads, tokens) fp32, for the gradient. Rows
    behind the last sequence are zeros in a new out, and left as they are in one
    that is given; lse is 0 there in the first case and unset in the second."""
    dev = _device_of(q, "q")
    args = _attention_args(q, k, v, offsets, scale, out is None, dev)
    out, to = _new_or_heads(out, "out", dev, q)
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    nbytes = ns_attention_workspace_size(args.tokens, args.sequences, args.q_heads, args.k_heads, args.dim)
    ws_ptr = None
    if nbytes:
        workspace = _given_or_new(workspace, nbytes, q.device)
        ws_ptr, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _check(library().ns_attention(args, to, lse.data_ptr(), ws_ptr, nbytes, _stream_of(dev)), "ns_attention")
    return out, lse


def ns_attention_grad_workspace_size(tokens: int, sequences: int, q_heads: int, k_heads: int, dim: int) -> int:
    return _sized("ns_attention_grad_workspace_size", tokens, sequences, q_heads, k_heads, dim)


def ns_attention_grad(dout, q, k, v, out, lse, offsets, scale: Optional[float] = None, dq=None, dk=None,
                      dv=None, workspace=None):
    """Gradients (dq, dk, dv) of ns_attention for the gradient of its out, with
    out and lse as it returned them. dq, dk and dv may be given, all three, for
    instance as views of one buffer: rows behind the last sequence are then left
    as they are, and are zeros in new ones."""
    dev = _device_of(q, "q")
    if (dq is None) != (dk is None) or (dq is None) != (dv is None):
        raise ValueError("dq, dk and dv: give all three or none")
    args = _attention_args(q, k, v, offsets, scale, dq is None, dev)
    tokens, q_heads, _ = q.shape
    dq, to_q = _new_or_heads(dq, "dq", dev, q)
    dk, to_k = _new_or_heads(dk, "dk", dev, k)
    dv, to_v = _new_or_heads(dv, "dv", dev, v)
    workspace = _given_or_new(workspace, ns_attention_grad_workspace_size(
        tokens, args.sequences, q_heads, args.k_heads, args.dim), q.device)
    _check(library().ns_attention_grad(
        args, _heads_like(dout, "dout", dev, q), _heads_like(out, "out", dev, q),
        _dense(lse, (q_heads, tokens), "lse", dev, torch.float32), to_q, to_k, to_v, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_of(dev)), "ns_attention_grad")
    return dq, dk, dv


__all__ = ["NS_MAX_HEADS", "NS_MAX_HEAD_TILES", "ns_qk_norm_rope", "ns_qk_norm_rope_grad",
           "ns_qk_norm_rope_grad_workspace_size", "ns_attention", "ns_attention_workspace_size",
           "ns_attention_grad", "ns_attention_grad_workspace_size"]
