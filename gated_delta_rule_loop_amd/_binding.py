"""ctypes binding of libgdr.so (include/gdr.h).

Argument marshalling only: torch tensors on the HIP device are described as
gdr_tensor structs (data pointer, dtype, shape, strides in elements) and the
call is enqueued on torch's current stream.  Every step of the recurrence runs
in the library's kernels; there is no fallback of any kind - if the library is
missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdr.so")

GDR_OK = 0
GDR_DTYPE_F32, GDR_DTYPE_BF16, GDR_DTYPE_U32, GDR_DTYPE_I32 = 0, 1, 2, 3
GDR_FLAG_L2NORM_QK = 1
GDR_FLAG_CONV_SILU = 2
GDR_FLAG_GATE_SIGMOID = 4
GDR_FLAG_GATE_SILU = 8
MAX_DIMS = 5

_DTYPES = {torch.float32: GDR_DTYPE_F32, torch.bfloat16: GDR_DTYPE_BF16,
           torch.int32: GDR_DTYPE_I32}
if hasattr(torch, "uint32"):
    _DTYPES[torch.uint32] = GDR_DTYPE_U32


class GdrTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * MAX_DIMS), ("stride", ctypes.c_int64 * MAX_DIMS)]


class GdrError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn} returned {code}: {msg}")
        self.code = code


_lib = None
EXPORTS = ("gdr_recurrence_fwd", "gdr_recurrence_verify_ring", "gdr_state_fold",
           "gdr_fused_recurrent_update", "gdr_snapshot_rollback", "gdr_causal_conv1d",
           "gdr_fwd_output_shape", "gdr_check_indices", "gdr_set_debug_checks",
           "gdr_linear_attention_fwd", "gdr_linear_attention_step", "gdr_linear_attention_bwd",
           "gdr_block_norm", "gdr_block_norm_bwd", "gdr_linear_attention_workspace",
           "gdr_block_norm_workspace", "gdr_ring_record_elements", "gdr_last_error_message", "gdr_version")


def lib():
    """Load libgdr.so (built by gated_delta_rule_loop_amd.build); raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m gated_delta_rule_loop_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(GdrTensor)
        i32, u32, f32, vp = ctypes.c_int32, ctypes.c_uint32, ctypes.c_float, ctypes.c_void_p
        L.gdr_recurrence_fwd.argtypes = [i32, i32, P, P, P, P, P, P, P, f32, u32, vp]
        L.gdr_recurrence_verify_ring.argtypes = [i32, i32, P, P, P, P, P, P, P, P, P, f32, u32, vp]
        L.gdr_state_fold.argtypes = [i32, i32, P, P, P, P, P, vp]
        L.gdr_fused_recurrent_update.argtypes = [P, P, P, P, P, f32, P, P, u32, P, P, P, P, i32,
                                                 P, vp]
        L.gdr_snapshot_rollback.argtypes = [P, P, P, P, vp]
        L.gdr_causal_conv1d.argtypes = [P, P, P, P, P, P, P, u32, vp]
        L.gdr_fwd_output_shape.argtypes = [P, P, ctypes.POINTER(ctypes.c_int64)]
        i64 = ctypes.c_int64
        L.gdr_check_indices.argtypes = [i64, vp, i64, vp, i64, vp, i64, i64, vp]
        L.gdr_set_debug_checks.argtypes = [ctypes.c_int]
        # these take their descriptors by address (_describe_all)
        L.gdr_linear_attention_fwd.argtypes = [vp] * 6 + [f32] + [vp] * 6
        L.gdr_linear_attention_step.argtypes = [vp] * 7 + [f32, vp]
        L.gdr_linear_attention_bwd.argtypes = [vp] * 6 + [f32] + [vp] * 9
        L.gdr_block_norm.argtypes = [vp] * 7 + [i64, f32, f32, u32, vp]
        L.gdr_block_norm_bwd.argtypes = [vp] * 12 + [i64, f32, f32, u32, vp, vp]
        L.gdr_linear_attention_workspace.argtypes = [i64, i64, i32, i32, i32, i32, ctypes.c_int]
        L.gdr_block_norm_workspace.argtypes = [i64, i64]
        for name in ("gdr_linear_attention_workspace", "gdr_block_norm_workspace"):
            getattr(L, name).restype = i64
        L.gdr_ring_record_elements.argtypes = [i32, i32, i32]
        L.gdr_ring_record_elements.restype = ctypes.c_int64
        L.gdr_last_error_message.restype = ctypes.c_char_p
        L.gdr_version.restype = ctypes.c_char_p
        for name in EXPORTS[:14]:
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def describe(t, *, allow_host=False):
    """gdr_tensor for a torch tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"expected a torch.Tensor, got {type(t)}")
    if not allow_host and not t.is_cuda:
        raise ValueError("gdr kernels take device tensors")
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    if t.dim() > MAX_DIMS:
        raise ValueError("rank above 5")
    d = GdrTensor()
    d.data = t.data_ptr() if t.numel() > 0 else (t.data_ptr() or None)
    d.dtype = _DTYPES[t.dtype]
    d.ndim = t.dim()
    for i, (s, st) in enumerate(zip(t.shape, t.stride())):
        d.shape[i] = s
        d.stride[i] = st
    return d


# gdr_tensor as struct.pack writes it, by rank.
_PACK = [struct.Struct(f"Pii{n}q{8 * (MAX_DIMS - n)}x{n}q{8 * (MAX_DIMS - n)}x").pack_into
         for n in range(MAX_DIMS + 1)]
_DESC_BYTES = ctypes.sizeof(GdrTensor)


def _describe_all(tensors):
    """(addresses of the tensors' gdr_tensors, None where a tensor is None, the
    buffer that holds them): describe() for a whole call, without a ctypes
    object for each tensor (a call's host time is a third of describe()'s)."""
    buf = bytearray(_DESC_BYTES * len(tensors))
    base = ctypes.addressof(ctypes.c_char.from_buffer(buf))
    refs, at = [], 0
    for t in tensors:
        if t is None:
            refs.append(None)
        else:
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"expected a torch.Tensor, got {type(t)}")
            if not t.is_cuda:
                raise ValueError("gdr kernels take device tensors")
            code = _DTYPES.get(t.dtype)
            if code is None:
                raise TypeError(f"unsupported dtype {t.dtype}")
            shape = t.shape
            n = len(shape)
            if n > MAX_DIMS:
                raise ValueError("rank above 5")
            _PACK[n](buf, at, t.data_ptr(), code, n, *shape, *t.stride())
            refs.append(base + at)
        at += _DESC_BYTES
    return refs, buf


def _ref(d):
    return None if d is None else ctypes.byref(d)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, rc):
    if rc != GDR_OK:
        raise GdrError(fn, rc, lib().gdr_last_error_message().decode())


def _scale(scale):
    return ctypes.c_float(-1.0 if scale is None or (isinstance(scale, float) and math.isnan(scale))
                          else float(scale))


def gdr_recurrence_fwd(recurrence_output, recurrent_state, slot_idx, qkv_conv_output,
                       decay_per_token, beta_per_token, input_row_offsets, *,
                       num_value_heads, num_key_heads, scale=None, l2norm=True, stream=None):
    """Slot-indexed ragged forward (page "gated_delta_recurrence_fwd_gpu").
    Writes recurrence_output and updates recurrent_state in place."""
    ds = [describe(x) for x in (recurrence_output, recurrent_state, slot_idx, qkv_conv_output,
                                decay_per_token, beta_per_token, input_row_offsets)]
    rc = lib().gdr_recurrence_fwd(num_value_heads, num_key_heads, *[_ref(d) for d in ds],
                                  _scale(scale), GDR_FLAG_L2NORM_QK if l2norm else 0,
                                  _stream(stream))
    _check("gdr_recurrence_fwd", rc)
    return recurrence_output


def gdr_recurrence_verify_ring(recurrence_output, recurrent_state, slot_idx, qkv_conv_output,
                               decay_per_token, beta_per_token, input_row_offsets, ring,
                               ring_slot_idx, *, num_value_heads, num_key_heads, scale=None,
                               l2norm=True, stream=None):
    """Verify window recording the ring (page "gated_delta_recurrence_verify_ring_gpu")."""
    ds = [describe(x) for x in (recurrence_output, recurrent_state, slot_idx, qkv_conv_output,
                                decay_per_token, beta_per_token, input_row_offsets, ring,
                                ring_slot_idx)]
    rc = lib().gdr_recurrence_verify_ring(num_value_heads, num_key_heads,
                                          *[_ref(d) for d in ds], _scale(scale),
                                          GDR_FLAG_L2NORM_QK if l2norm else 0, _stream(stream))
    _check("gdr_recurrence_verify_ring", rc)
    return recurrence_output


def gdr_state_fold(recurrent_state, slot_idx, ring, ring_slot_idx, accepted, *,
                   num_value_heads, num_key_heads, stream=None):
    """Fold accepted ring records into the live state."""
    ds = [describe(x) for x in (recurrent_state, slot_idx, ring, ring_slot_idx, accepted)]
    rc = lib().gdr_state_fold(num_value_heads, num_key_heads, *[_ref(d) for d in ds],
                              _stream(stream))
    _check("gdr_state_fold", rc)
    return recurrent_state


def gdr_fused_recurrent_update(q, k, v, g=None, beta=None, scale=None, initial_state=None,
                               output_final_state=False, use_qk_l2norm_in_kernel=False,
                               cu_seqlens=None, state=None, state_indices=None,
                               intermediate_states=None, steps_per_token=1, *, o=None,
                               final_state=None, stream=None):
    """Fused recurrent update (page "core.ssm.ops.gdp.fused_recurrent").

    Returns (o, final_state): final_state is `state` itself when a cache is
    given, the dense final state when output_final_state, else None.  o (of
    v's dtype) and a dense final state are allocated here with torch when not
    passed in."""
    if o is None:
        o = _new(v, stream=stream)
    if state is None and output_final_state and final_state is None:
        N = q.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
        dt = initial_state.dtype if initial_state is not None else torch.float32
        final_state = _new(v, (N, v.shape[2], q.shape[3], v.shape[3]), dt, stream)
    args = [describe(x) for x in (q, k, v, g, beta)]
    init_d, fin_d = describe(initial_state), describe(final_state)
    rest = [describe(x) for x in (cu_seqlens, state, state_indices, intermediate_states)]
    flags = GDR_FLAG_L2NORM_QK if use_qk_l2norm_in_kernel else 0
    rc = lib().gdr_fused_recurrent_update(*[_ref(d) for d in args], _scale(scale), _ref(init_d),
                                          _ref(fin_d), flags, *[_ref(d) for d in rest],
                                          int(steps_per_token), _ref(describe(o)),
                                          _stream(stream))
    _check("gdr_fused_recurrent_update", rc)
    return o, (state if state is not None else final_state)


def gdr_snapshot_rollback(state, state_indices, intermediate_states, accepted, *,
                          stream=None):
    """Roll each request's state back to its snapshot after `accepted` draft
    tokens (page "core.ssm.ops.gdp.fused_recurrent", intermediate_states)."""
    ds = [describe(x) for x in (state, state_indices, intermediate_states, accepted)]
    rc = lib().gdr_snapshot_rollback(*[_ref(d) for d in ds], _stream(stream))
    _check("gdr_snapshot_rollback", rc)
    return state


def gdr_causal_conv1d(x, weight, input_row_offsets, *, bias=None, conv_state=None,
                      slot_idx=None, silu=False, out=None, stream=None):
    """Pass-1 causal depthwise Conv1d producing qkv_conv_output (page
    "gated_delta_recurrence_fwd_gpu", Args).  Returns out (allocated here with
    torch, x's dtype and shape, when not passed in); conv_state is updated in
    place."""
    if out is None:
        out = _new(x, stream=stream)
    ds = [describe(t) for t in (out, x, weight, bias, conv_state, slot_idx, input_row_offsets)]
    rc = lib().gdr_causal_conv1d(*[_ref(d) for d in ds], GDR_FLAG_CONV_SILU if silu else 0,
                                 _stream(stream))
    _check("gdr_causal_conv1d", rc)
    return out


def gdr_fwd_output_shape(qkv_conv_output, recurrent_state):
    """Output shape of the forward (page "gated_delta_recurrence_fwd_shape")."""
    out = (ctypes.c_int64 * 2)()
    rc = lib().gdr_fwd_output_shape(_ref(describe(qkv_conv_output, allow_host=True)),
                                    _ref(describe(recurrent_state, allow_host=True)), out)
    _check("gdr_fwd_output_shape", rc)
    return (out[0], out[1])


def gdr_check_indices(rows, *, row_offsets=None, total_tokens=0, slots=None, num_slots=0,
                      ring_idx=None, ring_rows=0, ring_len=0, accepted=None):
    """Host-side index check (host arrays: NumPy or CPU tensors of 32-bit
    integers; -1 / 0xFFFFFFFF is padding).  Raises GdrError on a violation."""
    import numpy as np  # noqa: PLC0415
    keep = []

    def ptr(a):
        if a is None:
            return None
        if isinstance(a, torch.Tensor):
            a = a.detach().cpu().numpy()
        a = np.ascontiguousarray(a)
        if a.dtype.itemsize != 4 or a.dtype.kind not in "iu":
            raise TypeError("index arrays must hold 32-bit integers")
        keep.append(a)
        return a.ctypes.data_as(ctypes.c_void_p)

    rc = lib().gdr_check_indices(int(rows), ptr(row_offsets), int(total_tokens), ptr(slots),
                                 int(num_slots), ptr(ring_idx), int(ring_rows), int(ring_len),
                                 ptr(accepted))
    _check("gdr_check_indices", rc)


def gdr_set_debug_checks(enable):
    """Turn the per-call index checks on or off; returns the previous setting."""
    return bool(lib().gdr_set_debug_checks(1 if enable else 0))


_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(stream, t):
    """The stream's handle: the caller's, or torch's current one on t's device
    (asked for without building a Stream object where torch can)."""
    if stream is not None:
        return stream.cuda_stream
    if _current_handle is not None:
        return _current_handle(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _scale_value(scale):
    return -1.0 if scale is None else float(scale)  # not positive or NaN: the default


def _memory_of(stream):
    """Allocations inside come from `stream`'s own memory: a block that another
    stream has freed may still be in use there, and nothing makes `stream` wait
    for it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _scratch(floats, like, stream):
    """float32 workspace for a call on `stream` (torch's current one when None)."""
    if floats <= 0:
        return None
    with _memory_of(stream):
        return torch.empty(floats, dtype=torch.float32, device=like.device)


def _new(like, shape=None, dtype=None, stream=None):
    """An output allocated here, written on `stream` and handed to a program that
    may read it on its current one."""
    with _memory_of(stream):
        if shape is None and like.is_contiguous():
            t = torch.empty_like(like)
        else:
            t = torch.empty(like.shape if shape is None else shape, dtype=dtype or like.dtype,
                            device=like.device)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def gdr_linear_attention_workspace(tokens, rows, num_key_heads, num_value_heads, key_head_dim,
                                   value_head_dim, backward=False):
    """float32 elements of workspace that one call needs (0: none)."""
    return int(lib().gdr_linear_attention_workspace(tokens, rows, num_key_heads, num_value_heads,
                                                    key_head_dim, value_head_dim,
                                                    1 if backward else 0))


def _attention_scratch(q, v, offsets, backward, workspace, stream):
    if workspace is not None:
        return workspace
    T, nk, K = q.shape
    _, nv, V = v.shape
    n = lib().gdr_linear_attention_workspace(T, offsets.shape[0] - 1, nk, nv, K, V, backward)
    return _scratch(n, q, stream)


def gdr_linear_attention_fwd(q, k, v, g, input_row_offsets, *, state=None, slot_idx=None,
                             initial_state=None, final_state=None, output_final_state=False,
                             scale=None, o=None, workspace=None, stream=None):
    """Linear attention with a decay for each head over ragged prompts:
    S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q, k [T, nk, K]; v [T, nv, V]; g [T, nv] log decay (expanded for a fixed
    decay per head) or None.  Returns (o, final state): the pool itself,
    updated in place at slot_idx, when `state` is given, else final_state
    (allocated here when output_final_state is set), else None.  o and the
    workspace are allocated here with torch when not passed in.  Tokens outside
    the rows are not written: in an o allocated here they hold anything."""
    if o is None:
        o = _new(v, stream=stream)
    if state is None and output_final_state and final_state is None:
        dt = initial_state.dtype if initial_state is not None else torch.float32
        final_state = _new(v, (input_row_offsets.shape[0] - 1, v.shape[1], q.shape[2],
                               v.shape[2]), dt, stream)
    ws = _attention_scratch(q, v, input_row_offsets, 0, workspace, stream)
    r, _buf = _describe_all((o, q, k, v, g, input_row_offsets, initial_state, final_state, state,
                             slot_idx, ws))
    rc = lib().gdr_linear_attention_fwd(*r[:6], _scale_value(scale), *r[6:],
                                        _stream_of(stream, q))
    _check("gdr_linear_attention_fwd", rc)
    return o, (state if state is not None else final_state)


def gdr_linear_attention_step(q, k, v, g, state, slot_idx=None, *, scale=None, o=None,
                              stream=None):
    """One token for each row (q, k [B, nk, K]; v [B, nv, V]; g [B, nv] or
    None), with the row's state updated in place in its slot.  Returns o."""
    if o is None:
        o = _new(v, stream=stream)
    r, _buf = _describe_all((o, q, k, v, g, state, slot_idx))
    rc = lib().gdr_linear_attention_step(*r, _scale_value(scale), _stream_of(stream, q))
    _check("gdr_linear_attention_step", rc)
    return o


def gdr_linear_attention_bwd(do, q, k, v, g, input_row_offsets, *, initial_state=None,
                             dfinal_state=None, need_dg=True, need_dinitial_state=None,
                             scale=None, dq=None, dk=None, dv=None, dg=None, dinitial_state=None,
                             workspace=None, stream=None):
    """Gradients of gdr_linear_attention_fwd (dense states).  Returns (dq, dk,
    dv, dg, dinitial_state); dg is None without g or with need_dg=False,
    dinitial_state None unless there is an initial_state (or
    need_dinitial_state is set).  dg has one entry per token and head; a decay
    that tokens share gets their sum.  Outputs and the workspace are allocated
    here with torch when not passed in; tokens outside the rows are not written
    (in outputs allocated here they hold anything)."""
    dq = _new(q, stream=stream) if dq is None else dq
    dk = _new(k, stream=stream) if dk is None else dk
    dv = _new(v, stream=stream) if dv is None else dv
    if g is not None and need_dg and dg is None:
        dg = _new(g, stream=stream)
    if need_dinitial_state is None:
        need_dinitial_state = initial_state is not None
    if need_dinitial_state and dinitial_state is None:
        like = initial_state if initial_state is not None else dfinal_state
        dt = like.dtype if like is not None else torch.float32
        dinitial_state = _new(v, (input_row_offsets.shape[0] - 1, v.shape[1], q.shape[2],
                                  v.shape[2]), dt, stream)
    ws = _attention_scratch(q, v, input_row_offsets, 1, workspace, stream)
    r, _buf = _describe_all((do, q, k, v, g, input_row_offsets, initial_state, dfinal_state, dq,
                             dk, dv, dg, dinitial_state, ws))
    rc = lib().gdr_linear_attention_bwd(*r[:6], _scale_value(scale), *r[6:],
                                        _stream_of(stream, q))
    _check("gdr_linear_attention_bwd", rc)
    return dq, dk, dv, dg, dinitial_state


_ACTIVATIONS = {None: 0, "sigmoid": GDR_FLAG_GATE_SIGMOID, "silu": GDR_FLAG_GATE_SILU}


def gdr_block_norm(y, *, post_weight=None, group=0, gate=None, activation=None, residual=None,
                   residual_scale=1.0, pre_weight=None, eps=1e-6, h=None, n=None, stream=None):
    """The norms after and before a block, fused with its gate and residual
    scale: p = y / rms_group(y) * post_weight, h = residual + residual_scale *
    act(gate) * p, n = h / rms(h) * pre_weight.  y [T, D]; gate [T, D] or [D];
    post_weight [D] or [group].  Every argument but y is optional.  Returns
    (h, n), n None without pre_weight; both are allocated here with torch when
    not passed in."""
    if h is None:
        h = _new(y, stream=stream)
    if pre_weight is not None and n is None:
        n = _new(y, stream=stream)
    r, _buf = _describe_all((h, n, y, residual, gate, post_weight, pre_weight))
    rc = lib().gdr_block_norm(*r, group, residual_scale, eps, _ACTIVATIONS[activation],
                              _stream_of(stream, y))
    _check("gdr_block_norm", rc)
    return h, n


def gdr_block_norm_workspace(tokens, dim):
    """float32 elements of workspace that gdr_block_norm_bwd needs at most."""
    return int(lib().gdr_block_norm_workspace(tokens, dim))


def gdr_block_norm_bwd(dh, dn, y, h, *, post_weight=None, group=0, gate=None, activation=None,
                       residual=True, residual_scale=1.0, pre_weight=None, eps=1e-6,
                       dresidual=None, dy=None, dgate=None, dpost_weight=None, dpre_weight=None,
                       workspace=None, stream=None):
    """Gradients of gdr_block_norm given dh (of h, from everything but n) and
    dn (of n, with pre_weight); h is the forward's output, needed with
    pre_weight only.  Returns (dresidual, dgate, dy, dpost_weight,
    dpre_weight), None for what the forward did not have.  Without pre_weight
    dresidual is dh itself."""
    dx = dresidual
    if residual and dx is None and pre_weight is not None:
        dx = _new(y, stream=stream)
    dy = _new(y, stream=stream) if dy is None else dy
    dgate = _new(gate, stream=stream) if gate is not None and dgate is None else dgate
    if post_weight is not None and dpost_weight is None:
        dpost_weight = _new(post_weight, stream=stream)
    if pre_weight is not None and dpre_weight is None:
        dpre_weight = _new(pre_weight, stream=stream)
    ws = workspace
    if ws is None and y.dim() == 2:
        ws = _scratch(lib().gdr_block_norm_workspace(*y.shape), y, stream)
    r, _buf = _describe_all((dx, dy, dgate, dpost_weight, dpre_weight, dh, dn, y,
                             h if pre_weight is not None else None, gate, post_weight, pre_weight,
                             ws))
    rc = lib().gdr_block_norm_bwd(*r[:12], group, residual_scale, eps, _ACTIVATIONS[activation],
                                  r[12], _stream_of(stream, y))
    _check("gdr_block_norm_bwd", rc)
    return (dx if dx is not None else dh) if residual else None, dgate, dy, dpost_weight, \
        dpre_weight


def gdr_ring_record_elements(group, key_head_dim, value_head_dim):
    return int(lib().gdr_ring_record_elements(group, key_head_dim, value_head_dim))


def gdr_version():
    return lib().gdr_version().decode()


def gdr_last_error_message():
    return lib().gdr_last_error_message().decode()
