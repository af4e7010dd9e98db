"""Thin ctypes binding of libgdn.so (the C ABI declared in include/gdn.h).

Argument marshalling only: every step of the mixer runs in the library's
CUDA kernels.  Tensors are torch CUDA tensors (torch supplies device memory
and the current stream); they must be contiguous and on the current device.
There is no fallback: if libgdn.so is missing or a call fails, a
RuntimeError is raised.
"""

import collections
import ctypes
import functools
import math
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, 'libgdn.so')

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_DEVICE = range(5)
GDN_BF16, GDN_F32 = 0, 1

EXPORTS = ('gdn_version', 'gdn_last_error_string', 'gdn_check_device_error', 'gdn_conv_gating',
           'gdn_conv_state_steps',
           'gdn_gating', 'gdn_chunk_prefill_workspace_size', 'gdn_chunk_prefill',
           'gdn_chunk_prefill_fp32', 'gdn_chunk_prefill_static', 'gdn_chunk_prefill_gated_norm',
           'gdn_recurrent_decode', 'gdn_recurrent_decode_steps',
           'gdn_gated_rmsnorm', 'gdn_decode_fused',
           'gdn_qk_norm_rope', 'gdn_paged_kv_append', 'gdn_paged_attn_decode_workspace_size',
           'gdn_paged_attn_decode', 'gdn_paged_kv4_append', 'gdn_paged_kv4_read',
           'gdn_paged_kv4_attn_decode_workspace_size', 'gdn_paged_kv4_attn_decode', 'gdn_paged_plan',
           'gdn_draft_verify', 'gdn_test_chunk_wait_timeout', 'gdn_test_paged_attn_wait_timeout')


class gdn_dims(ctypes.Structure):
    _fields_ = [('num_seqs', ctypes.c_int32), ('total_tokens', ctypes.c_int32),
                ('num_k_heads', ctypes.c_int32), ('num_v_heads', ctypes.c_int32),
                ('head_k_dim', ctypes.c_int32), ('head_v_dim', ctypes.c_int32)]


class gdn_attn_dims(ctypes.Structure):
    _fields_ = [('num_seqs', ctypes.c_int32), ('total_tokens', ctypes.c_int32),
                ('num_q_heads', ctypes.c_int32), ('num_kv_heads', ctypes.c_int32),
                ('head_dim', ctypes.c_int32)]


class gdn_heads(ctypes.Structure):
    _fields_ = [('data', ctypes.c_void_p), ('token_stride', ctypes.c_int64), ('head_stride', ctypes.c_int64)]


class gdn_norm_rope(ctypes.Structure):
    _fields_ = [('q_norm_w', ctypes.c_void_p), ('k_norm_w', ctypes.c_void_p), ('norm_eps', ctypes.c_float),
                ('rotary_dim', ctypes.c_int32), ('interleaved', ctypes.c_int32),
                ('max_positions', ctypes.c_int32), ('cos_sin', ctypes.c_void_p),
                ('positions', ctypes.c_void_p)]


class gdn_paged_cache(ctypes.Structure):
    _fields_ = [('k', ctypes.c_void_p), ('v', ctypes.c_void_p), ('page_stride', ctypes.c_int64),
                ('head_stride', ctypes.c_int64), ('slot_stride', ctypes.c_int64),
                ('num_pages', ctypes.c_int32), ('page_size', ctypes.c_int32), ('max_pages', ctypes.c_int32),
                ('block_table', ctypes.c_void_p), ('kv_lens', ctypes.c_void_p)]


class gdn_paged_cache4(ctypes.Structure):
    _fields_ = [('k', ctypes.c_void_p), ('v', ctypes.c_void_p), ('k_scale', ctypes.c_void_p),
                ('v_scale', ctypes.c_void_p), ('page_stride', ctypes.c_int64), ('head_stride', ctypes.c_int64),
                ('slot_stride', ctypes.c_int64), ('scale_page_stride', ctypes.c_int64),
                ('scale_head_stride', ctypes.c_int64), ('scale_slot_stride', ctypes.c_int64),
                ('num_pages', ctypes.c_int32), ('page_size', ctypes.c_int32), ('max_pages', ctypes.c_int32),
                ('block_table', ctypes.c_void_p), ('kv_lens', ctypes.c_void_p)]


class gdn_page_plan(ctypes.Structure):
    _fields_ = [('num_seqs', ctypes.c_int32), ('total_tokens', ctypes.c_int32), ('num_pages', ctypes.c_int32),
                ('page_size', ctypes.c_int32), ('max_pages', ctypes.c_int32), ('new_lens', ctypes.c_void_p),
                ('kv_lens', ctypes.c_void_p), ('pages_held', ctypes.c_void_p), ('free_ring', ctypes.c_void_p),
                ('free_pages', ctypes.c_void_p), ('block_table', ctypes.c_void_p), ('cu_seqlens', ctypes.c_void_p),
                ('positions', ctypes.c_void_p), ('slots', ctypes.c_void_p), ('kv_lens_out', ctypes.c_void_p),
                ('pages_held_out', ctypes.c_void_p), ('free_ring_out', ctypes.c_void_p)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_DIMS = ctypes.POINTER(gdn_dims)
_ADIMS = ctypes.POINTER(gdn_attn_dims)
_HEADS = ctypes.POINTER(gdn_heads)
_NR = ctypes.POINTER(gdn_norm_rope)
_CACHE = ctypes.POINTER(gdn_paged_cache)
_CACHE4 = ctypes.POINTER(gdn_paged_cache4)
_PLAN = ctypes.POINTER(gdn_page_plan)
_I32 = ctypes.c_int32

_SIGS = {
    'gdn_version': ([], _I),
    'gdn_last_error_string': ([], ctypes.c_char_p),
    'gdn_check_device_error': ([_P], _I),
    'gdn_conv_gating': ([_DIMS, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _F, _F,
                         _P, _P, _P, _I, _P, _P, _P], _I),
    'gdn_gating': ([_I64, ctypes.c_int32, _P, _P, _I, _P, _P, _P, _P, _P], _I),
    'gdn_conv_state_steps': ([_DIMS, _P, _P, _I, _P, _P, _P], _I),
    'gdn_chunk_prefill_workspace_size': ([_DIMS, ctypes.POINTER(_SZ)], _I),
    'gdn_chunk_prefill': ([_DIMS, _P, _P, _P, _P, _I, _P, _P, _F, _P, _P, _P, _I, _P, _SZ, _P], _I),
    'gdn_chunk_prefill_fp32': ([_DIMS, _P, _P, _P, _P, _I, _P, _P, _F, _P, _P, _P, _I, _P], _I),
    'gdn_chunk_prefill_static': ([_DIMS, _P, _P, _P, _P, _I, _P, _P, _F, _P, _P, _P, _I, _P], _I),
    'gdn_chunk_prefill_gated_norm': ([_DIMS, _P, _P, _P, _P, _I, _P, _P, _F, _P, _P, _P, _I, _P, _F, _P, _I,
                                      _P, _SZ, _P], _I),
    'gdn_recurrent_decode': ([_DIMS, _P, _P, _P, _P, _I, _P, _P, _F, _P, _P, _I, _P], _I),
    'gdn_recurrent_decode_steps': ([_DIMS, _P, _P, _P, _P, _I, _P, _P, _F, _P, _P, _P, _I, _P], _I),
    'gdn_gated_rmsnorm': ([_I64, ctypes.c_int32, _P, _I, _P, _I, _P, _F, _P, _I, _P], _I),
    'gdn_decode_fused': ([_DIMS, _P, _I, _P, _P, _P, _P, _P, _P, _P, _F, _F, _P, _P, _P, _F,
                          _P, _I, _P], _I),
    'gdn_qk_norm_rope': ([_ADIMS, _P, _HEADS, _HEADS, _I, _NR, _P, _P, _I, _P], _I),
    'gdn_paged_kv_append': ([_ADIMS, _P, _HEADS, _HEADS, _HEADS, _I, _NR, _CACHE, _I, _P, _I, _P], _I),
    'gdn_paged_attn_decode_workspace_size': ([_ADIMS, _I, _I64, ctypes.POINTER(_SZ)], _I),
    'gdn_paged_attn_decode': ([_ADIMS, _P, _HEADS, _HEADS, _I, _CACHE, _F, _P, _I, _P, _SZ, _P], _I),
    'gdn_paged_kv4_append': ([_ADIMS, _P, _HEADS, _HEADS, _HEADS, _I, _NR, _CACHE4, _P, _I, _P], _I),
    'gdn_paged_kv4_read': ([_ADIMS, _P, _CACHE4, _P, _P, _I, _P], _I),
    'gdn_paged_kv4_attn_decode_workspace_size': ([_ADIMS, _I64, ctypes.POINTER(_SZ)], _I),
    'gdn_paged_kv4_attn_decode': ([_ADIMS, _P, _HEADS, _HEADS, _CACHE4, _F, _P, _P, _SZ, _P], _I),
    'gdn_paged_plan': ([_PLAN, _P], _I),
    'gdn_draft_verify': ([_I32, _I32, _I32, _I32, _P, _P, _I64, _P, _I64, _I64, _I, _P, _P, _P, _P, _P, _P, _P], _I),
    'gdn_test_paged_attn_wait_timeout': ([_ADIMS, _P, _HEADS, _I, _CACHE, _P, _P, _SZ, _I64, _I, _P], _I),
    'gdn_test_chunk_wait_timeout': ([_DIMS, _P, _P, _P, _P, _P, _P, _P, _SZ, _I64, _P], _I),
}


def lib():
    """Load libgdn.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError('libgdn.so is not built (%s); run __graft_entry__.build()' % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(status, name):
    if status != GDN_OK:
        msg = lib().gdn_last_error_string().decode()
        raise RuntimeError('%s failed (status %d): %s' % (name, status, msg))


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError('expected a CUDA tensor')
    if not t.is_contiguous():
        raise ValueError('expected a contiguous tensor')
    return t.data_ptr()


def _dt(t):
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float32:
        return GDN_F32
    raise ValueError('unsupported dtype %s' % t.dtype)


def _tdt(code):
    return torch.bfloat16 if code == GDN_BF16 else torch.float32


def _stream():
    # the handle of torch.cuda.current_stream() without its Stream object: 0.1 against 3.0 us on a Grace host
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _dims(num_seqs, total, Nk, Nv, Dk, Dv):
    return gdn_dims(int(num_seqs), int(total), int(Nk), int(Nv), int(Dk), int(Dv))


def _f32(t):
    if t is None or t.dtype == torch.float32:
        return t
    raise ValueError('expected a float32 tensor')


def check_device_error():
    """Synchronise the current stream and raise if a kernel flagged bad metadata."""
    _check(lib().gdn_check_device_error(_stream()), 'gdn_check_device_error')


def conv_gating(mixed_qkv, conv_w, a, b, A_log, dt_bias, Nk, Nv, Dk, Dv, cu_seqlens=None,
                num_seqs=1, conv_bias=None, conv_state_in=None, conv_state_out=None,
                q_scale=None, l2_eps=1e-6, out_dtype=torch.bfloat16, out=None):
    """gdn_conv_gating.  Returns (q, k, v, g, beta); ``out`` may supply them."""
    T = mixed_qkv.shape[0]
    if cu_seqlens is not None:
        num_seqs = cu_seqlens.numel() - 1
    if q_scale is None:
        q_scale = 1.0 / math.sqrt(Dk)
    dev = mixed_qkv.device
    if out is None:
        q = torch.empty(T, Nk, Dk, dtype=out_dtype, device=dev)
        k = torch.empty(T, Nk, Dk, dtype=out_dtype, device=dev)
        v = torch.empty(T, Nv, Dv, dtype=out_dtype, device=dev)
        g = torch.empty(T, Nv, dtype=torch.float32, device=dev)
        beta = torch.empty(T, Nv, dtype=torch.float32, device=dev)
    else:
        q, k, v, g, beta = out
    for t in (conv_w, a, b) + tuple(x for x in (conv_bias, conv_state_in, conv_state_out) if x is not None):
        if t.dtype != mixed_qkv.dtype:
            raise ValueError('conv_w, a, b, conv_bias and conv states share the dtype of mixed_qkv')
    d = _dims(num_seqs, T, Nk, Nv, Dk, Dv)
    st = lib().gdn_conv_gating(ctypes.byref(d), _ptr(cu_seqlens), _ptr(mixed_qkv), _dt(mixed_qkv),
                               _ptr(conv_w), _ptr(conv_bias), _ptr(conv_state_in),
                               _ptr(conv_state_out), _ptr(a), _ptr(b), _ptr(_f32(A_log)),
                               _ptr(_f32(dt_bias)), float(q_scale), float(l2_eps), _ptr(q), _ptr(k),
                               _ptr(v), _dt(q), _ptr(g), _ptr(beta), _stream())
    _check(st, 'gdn_conv_gating')
    return q, k, v, g, beta


def conv_state_steps(mixed_qkv, Nk, Nv, Dk, Dv, conv_state_in=None, cu_seqlens=None, num_seqs=1, out=None):
    """gdn_conv_state_steps: the conv state after every token, [tokens, C, 3]."""
    T, C = mixed_qkv.shape
    if cu_seqlens is not None:
        num_seqs = cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty(T, C, 3, dtype=mixed_qkv.dtype, device=mixed_qkv.device)
    if conv_state_in is not None and conv_state_in.dtype != mixed_qkv.dtype:
        raise ValueError('conv_state_in shares the dtype of mixed_qkv')
    d = _dims(num_seqs, T, Nk, Nv, Dk, Dv)
    st = lib().gdn_conv_state_steps(ctypes.byref(d), _ptr(cu_seqlens), _ptr(mixed_qkv), _dt(mixed_qkv),
                                    _ptr(conv_state_in), _ptr(out), _stream())
    _check(st, 'gdn_conv_state_steps')
    return out


def gating(a, b, A_log, dt_bias, out=None):
    """gdn_gating.  a, b [rows, Nv].  Returns (g, beta) fp32."""
    rows, Nv = a.shape
    if out is None:
        g = torch.empty(rows, Nv, dtype=torch.float32, device=a.device)
        beta = torch.empty_like(g)
    else:
        g, beta = out
    st = lib().gdn_gating(rows, Nv, _ptr(a), _ptr(b), _dt(a), _ptr(_f32(A_log)), _ptr(_f32(dt_bias)),
                          _ptr(g), _ptr(beta), _stream())
    _check(st, 'gdn_gating')
    return g, beta


def chunk_prefill_workspace_size(num_seqs, total, Nk, Nv, Dk, Dv):
    d = _dims(num_seqs, total, Nk, Nv, Dk, Dv)
    n = _SZ(0)
    _check(lib().gdn_chunk_prefill_workspace_size(ctypes.byref(d), ctypes.byref(n)),
           'gdn_chunk_prefill_workspace_size')
    return n.value


def chunk_prefill(q, k, v, g, beta, scale=1.0, initial_state=None, final_state=None,
                  cu_seqlens=None, num_seqs=1, out_dtype=torch.bfloat16, o=None, workspace=None,
                  fp32=False, want_final_state=True):
    """gdn_chunk_prefill (or gdn_chunk_prefill_fp32).  Returns (o, final_state)."""
    T, Nk, Dk = q.shape
    Nv, Dv = v.shape[1], v.shape[2]
    if cu_seqlens is not None:
        num_seqs = cu_seqlens.numel() - 1
    if o is None:
        o = torch.empty(T, Nv, Dv, dtype=out_dtype, device=q.device)
    if final_state is None and want_final_state:
        final_state = torch.empty(num_seqs, Nv, Dk, Dv, dtype=torch.float32, device=q.device)
    if q.dtype != k.dtype or q.dtype != v.dtype:
        raise ValueError('q, k, v must share a dtype')
    d = _dims(num_seqs, T, Nk, Nv, Dk, Dv)
    if fp32:
        st = lib().gdn_chunk_prefill_fp32(ctypes.byref(d), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v),
                                          _dt(q), _ptr(_f32(g)), _ptr(_f32(beta)), float(scale),
                                          _ptr(_f32(initial_state)), _ptr(_f32(final_state)), _ptr(o),
                                          _dt(o), _stream())
        _check(st, 'gdn_chunk_prefill_fp32')
        return o, final_state
    ws_bytes = chunk_prefill_workspace_size(num_seqs, T, Nk, Nv, Dk, Dv)
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    st = lib().gdn_chunk_prefill(ctypes.byref(d), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), _dt(q),
                                 _ptr(_f32(g)), _ptr(_f32(beta)), float(scale),
                                 _ptr(_f32(initial_state)), _ptr(_f32(final_state)), _ptr(o), _dt(o),
                                 _ptr(workspace), ws_bytes if workspace is not None else 0, _stream())
    _check(st, 'gdn_chunk_prefill')
    return o, final_state


def chunk_prefill_gated_norm(q, k, v, g, beta, z, norm_w, scale=1.0, initial_state=None,
                             final_state=None, cu_seqlens=None, num_seqs=1, norm_eps=1e-6,
                             out_dtype=torch.bfloat16, y=None, workspace=None, want_final_state=True):
    """gdn_chunk_prefill_gated_norm: chunk prefill with the gated RMSNorm fused into its
    output.  Returns (y, final_state)."""
    T, Nk, Dk = q.shape
    Nv, Dv = v.shape[1], v.shape[2]
    if cu_seqlens is not None:
        num_seqs = cu_seqlens.numel() - 1
    if y is None:
        y = torch.empty(T, Nv, Dv, dtype=out_dtype, device=q.device)
    if final_state is None and want_final_state:
        final_state = torch.empty(num_seqs, Nv, Dk, Dv, dtype=torch.float32, device=q.device)
    if q.dtype != k.dtype or q.dtype != v.dtype:
        raise ValueError('q, k, v must share a dtype')
    d = _dims(num_seqs, T, Nk, Nv, Dk, Dv)
    ws_bytes = chunk_prefill_workspace_size(num_seqs, T, Nk, Nv, Dk, Dv)
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    st = lib().gdn_chunk_prefill_gated_norm(
        ctypes.byref(d), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(_f32(g)),
        _ptr(_f32(beta)), float(scale), _ptr(_f32(initial_state)), _ptr(_f32(final_state)), _ptr(z),
        _dt(z), _ptr(_f32(norm_w)), float(norm_eps), _ptr(y), _dt(y), _ptr(workspace),
        ws_bytes if workspace is not None else 0, _stream())
    _check(st, 'gdn_chunk_prefill_gated_norm')
    return y, final_state


def recurrent_decode(q, k, v, g, beta, state, scale=1.0, cu_seqlens=None, num_seqs=None,
                     out_dtype=torch.bfloat16, o=None, step_states=None):
    """gdn_recurrent_decode: state [N, Nv, Dk, Dv] fp32 is updated in place.  Returns o.
    With ``step_states`` ([tokens, Nv, Dk, Dv] fp32) it calls gdn_recurrent_decode_steps,
    which also writes the state after every token."""
    T, Nk, Dk = q.shape
    Nv, Dv = v.shape[1], v.shape[2]
    if cu_seqlens is not None:
        num_seqs = cu_seqlens.numel() - 1
    if num_seqs is None:
        num_seqs = state.shape[0]
    if o is None:
        o = torch.empty(T, Nv, Dv, dtype=out_dtype, device=q.device)
    d = _dims(num_seqs, T, Nk, Nv, Dk, Dv)
    args = (ctypes.byref(d), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), _dt(q), _ptr(_f32(g)),
            _ptr(_f32(beta)), float(scale), _ptr(_f32(state)))
    if step_states is None:
        st = lib().gdn_recurrent_decode(*args, _ptr(o), _dt(o), _stream())
        _check(st, 'gdn_recurrent_decode')
    else:
        st = lib().gdn_recurrent_decode_steps(*args, _ptr(_f32(step_states)), _ptr(o), _dt(o), _stream())
        _check(st, 'gdn_recurrent_decode_steps')
    return o


def gated_rmsnorm(x, z, w, eps=1e-6, out_dtype=torch.bfloat16, y=None):
    """gdn_gated_rmsnorm over the last axis of x (any leading shape)."""
    dim = x.shape[-1]
    rows = x.numel() // dim
    if y is None:
        y = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    st = lib().gdn_gated_rmsnorm(rows, dim, _ptr(x), _dt(x), _ptr(z), _dt(z), _ptr(_f32(w)), float(eps),
                                 _ptr(y), _dt(y), _stream())
    _check(st, 'gdn_gated_rmsnorm')
    return y


def decode_fused(mixed_qkv, conv_w, conv_state, a, b, A_log, dt_bias, state, z, norm_w, Nk, Nv,
                 Dk, Dv, conv_bias=None, q_scale=None, l2_eps=1e-6, norm_eps=1e-6,
                 out_dtype=torch.bfloat16, y=None):
    """gdn_decode_fused: one token per sequence; conv_state and state updated in place."""
    B = mixed_qkv.shape[0]
    if q_scale is None:
        q_scale = 1.0 / math.sqrt(Dk)
    if y is None:
        y = torch.empty(B, Nv, Dv, dtype=out_dtype, device=mixed_qkv.device)
    d = _dims(B, B, Nk, Nv, Dk, Dv)
    st = lib().gdn_decode_fused(ctypes.byref(d), _ptr(mixed_qkv), _dt(mixed_qkv), _ptr(conv_w),
                                _ptr(conv_bias), _ptr(conv_state), _ptr(a), _ptr(b),
                                _ptr(_f32(A_log)), _ptr(_f32(dt_bias)), float(q_scale), float(l2_eps),
                                _ptr(_f32(state)), _ptr(z), _ptr(_f32(norm_w)), float(norm_eps), _ptr(y),
                                _dt(y), _stream())
    _check(st, 'gdn_decode_fused')
    return y


def mixer_prefill(mixed_qkv, conv_w, a, b, A_log, dt_bias, z, norm_w, Nk, Nv, Dk, Dv,
                  cu_seqlens=None, num_seqs=1, conv_bias=None, conv_state_in=None,
                  conv_state_out=None, initial_state=None, final_state=None, q_scale=None,
                  l2_eps=1e-6, norm_eps=1e-6, act_dtype=torch.bfloat16, out_dtype=torch.bfloat16,
                  bufs=None, fuse_norm=None):
    """The prefill path: conv_gating -> chunk_prefill -> gated_rmsnorm.  With ``fuse_norm``
    (and shapes that run on the tensor cores: bf16, 128-wide heads) the chunk prefill and
    the norm are one call (gdn_chunk_prefill_gated_norm).  By default (None) that call is
    taken for a single sequence, where the norm runs beside the sequential scan and the
    call measured faster than the two separate ones on a GB300 (119.2 vs 111.1 + 18.9 us at
    4096 tokens); packed batches take the two calls (their fused form applies the norm in
    the scan's output epilogue, which paces the scan).

    ``bufs`` (optional dict) supplies preallocated q, k, v, g, beta, o, y."""
    bufs = bufs or {}
    out = None
    if 'q' in bufs:
        out = (bufs['q'], bufs['k'], bufs['v'], bufs['g'], bufs['beta'])
    q, k, v, g, beta = conv_gating(mixed_qkv, conv_w, a, b, A_log, dt_bias, Nk, Nv, Dk, Dv,
                                   cu_seqlens, num_seqs, conv_bias, conv_state_in, conv_state_out,
                                   q_scale, l2_eps, act_dtype, out)
    if fuse_norm is None:
        fuse_norm = num_seqs == 1
    if fuse_norm and act_dtype == torch.bfloat16 and z.dtype == torch.bfloat16 and Dk == 128 and Dv == 128:
        return chunk_prefill_gated_norm(q, k, v, g, beta, z, norm_w, 1.0, initial_state, final_state,
                                        cu_seqlens, num_seqs, norm_eps, out_dtype, bufs.get('y'),
                                        bufs.get('workspace'))
    o, S = chunk_prefill(q, k, v, g, beta, 1.0, initial_state, final_state, cu_seqlens, num_seqs,
                         act_dtype, bufs.get('o'), bufs.get('workspace'))
    y = gated_rmsnorm(o, z, norm_w, norm_eps, out_dtype, bufs.get('y'))
    return y, S


# --- softmax attention over a paged cache ---------------------------------------------
#
# These calls take a few us on the GPU, so their marshalling is kept short: the C structs are
# packed as bytes (their layouts are those of the Structures above) and passed by address.

_pack_dims = struct.Struct('@5i').pack
_pack_heads = struct.Struct('@Pqq').pack
_pack_norm_rope = struct.Struct('@PPfiiiPP').pack
_pack_cache = struct.Struct('@PPqqqiiiPP').pack
_pack_cache4 = struct.Struct('@PPPPqqqqqqiiiPP').pack
_pack_plan = struct.Struct('@iiiiiPPPPPPPPPPPP').pack
_fast = {}


def _fn(name):
    """The library function with its struct arguments taken as addresses of packed bytes."""
    f = _fast.get(name)
    if f is None:
        f = lib()[name]                                       # a function object of its own
        args, f.restype = _SIGS[name]
        f.argtypes = [_P if hasattr(a, 'contents') else a for a in args]
        _fast[name] = f
    return f


def _device(t):
    """The library launches on the current device: the index of t's, which has to be that one."""
    dev = t.get_device()
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError('expected CUDA tensors on the current device')
    return dev


def _arg(t, dtype, dev, what):
    """Address of an optional contiguous tensor of the given type on device ``dev`` (0: none)."""
    if t is None:
        return 0
    if t.get_device() != dev:
        raise ValueError('%s must be on the device of the other tensors' % what)
    if t.dtype is not dtype:
        raise ValueError('%s must be %s' % (what, str(dtype)[6:]))
    if not t.is_contiguous():
        raise ValueError('%s must be contiguous' % what)
    return t.data_ptr()


def _heads(t, dev, what):
    """[tokens, heads, D] with contiguous head rows (a slice of a wider projection is fine)."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError('%s must be on the device of the other tensors' % what)
    shape = t.shape
    if len(shape) != 3:
        raise ValueError('%s must be [tokens, heads, head_dim]' % what)
    ts, hs, es = t.stride()
    if es != 1:
        raise ValueError('the head rows of %s must be contiguous' % what)
    T, H, D = shape
    # a stride over an axis of one entry is never used: any value may stand there
    return _pack_heads(t.data_ptr(), ts if T > 1 else H * D, hs if H > 1 else D)


def _norm_rope(q_norm_w, k_norm_w, norm_eps, cos_sin, positions, interleaved, T, D, dev):
    rot = maxpos = table = 0
    if cos_sin is not None:
        table = _arg(cos_sin, torch.float32, dev, 'cos_sin')
        if cos_sin.dim() != 2:
            raise ValueError('cos_sin must be [positions, rotary_dim]')
        maxpos, rot = cos_sin.shape
        if rot == 0:
            maxpos = table = 0
    if (q_norm_w is not None and q_norm_w.numel() != D) or (k_norm_w is not None and k_norm_w.numel() != D):
        raise ValueError('a norm weight has head_dim elements')
    if positions is not None and positions.numel() != T:
        raise ValueError('positions has one entry per token')
    return _pack_norm_rope(_arg(q_norm_w, torch.float32, dev, 'q_norm_w'), _arg(k_norm_w, torch.float32, dev, 'k_norm_w'),
                           norm_eps, rot, 1 if interleaved else 0, maxpos, table,
                           _arg(positions, torch.int32, dev, 'positions'))


def _cache(k_cache, v_cache, block_table, kv_lens, Nkv, D, num_seqs, dev):
    """Checks the cache's tensors against the call's sizes and packs them."""
    shape, stride = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape or k_cache.dtype is not v_cache.dtype:
        raise ValueError('k_cache and v_cache share the shape [pages, kv heads, page size, head_dim] and a dtype')
    if k_cache.get_device() != dev or v_cache.get_device() != dev:
        raise ValueError('the cache must be on the device of the other tensors')
    pages, H, P, E = shape
    if H != Nkv or E != D:
        raise ValueError('the cache holds %d heads of %d, the call has %d of %d' % (H, E, Nkv, D))
    v_stride = v_cache.stride()
    if pages == 1 or H == 1 or P == 1:
        # a stride over an axis of one entry is never used: any value may stand there
        def used(st):
            return (st[0] if pages > 1 else H * P * E, st[1] if H > 1 else P * E, st[2] if P > 1 else E, st[3])
        stride, v_stride = used(stride), used(v_stride)
    ps, hs, ss, es = stride
    if es != 1 or v_stride[3] != 1:
        raise ValueError('the head rows of the cache must be contiguous')
    if v_stride != stride:
        raise ValueError('k_cache and v_cache must have the same strides')
    rows = block_table.shape
    if len(rows) != 2 or rows[0] != num_seqs or kv_lens.numel() != num_seqs:
        raise ValueError('block_table is [sequences, pages] and kv_lens [sequences]')
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), ps, hs, ss, pages, P, rows[1],
                       _arg(block_table, torch.int32, dev, 'block_table'), _arg(kv_lens, torch.int32, dev, 'kv_lens'))


def _given(t, shape, dev, what):
    """An output the caller supplied."""
    if t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError('%s must be contiguous, on the device of the other tensors and of shape %s' % (what, shape))
    return t


def qk_norm_rope(q, k=None, cos_sin=None, q_norm_w=None, k_norm_w=None, positions=None, cu_seqlens=None,
                 num_seqs=1, norm_eps=1e-6, interleaved=False, out_dtype=torch.bfloat16, q_out=None, k_out=None):
    """gdn_qk_norm_rope: per-head RMSNorm and rotation of q [tokens, Nq, D] and k [tokens, Nkv, D].
    Returns (q_out, k_out); ``positions`` default to each token's index in its sequence."""
    T, Nq, D = shape = q.shape
    Nkv, k_shape = Nq, None
    if k is not None:
        Nkv = k.shape[1]
        k_shape = (T, Nkv, D)
        if k.shape != k_shape or k.dtype is not q.dtype:
            raise ValueError('q and k share tokens, head_dim and dtype')
    dev = _device(q)
    cu = 0
    if cu_seqlens is not None:
        cu = _arg(cu_seqlens, torch.int32, dev, 'cu_seqlens')
        num_seqs = cu_seqlens.numel() - 1
    q_out = torch.empty(shape, dtype=out_dtype, device=q.device) if q_out is None else _given(q_out, shape, dev, 'q_out')
    ko = 0
    if k is not None:
        k_out = (torch.empty(k_shape, dtype=q_out.dtype, device=q.device) if k_out is None
                 else _given(k_out, k_shape, dev, 'k_out'))
        if k_out.dtype is not q_out.dtype:
            raise ValueError('q_out and k_out share a dtype')
        ko = k_out.data_ptr()
    st = _fn('gdn_qk_norm_rope')(
        _pack_dims(num_seqs, T, Nq, Nkv, D), cu, _heads(q, dev, 'q'), _heads(k, dev, 'k'), _dt(q),
        _norm_rope(q_norm_w, k_norm_w, norm_eps, cos_sin, positions, interleaved, T, D, dev), q_out.data_ptr(),
        ko, _dt(q_out), _stream())
    if st:
        _check(st, 'gdn_qk_norm_rope')
    return q_out, k_out


def paged_kv_append(k, v, k_cache, v_cache, block_table, kv_lens, q=None, cos_sin=None, q_norm_w=None,
                    k_norm_w=None, positions=None, cu_seqlens=None, norm_eps=1e-6, interleaved=False,
                    out_dtype=torch.bfloat16, q_out=None):
    """gdn_paged_kv_append: k (normed and rotated on the way) and v of the new tokens into the cache, in place.
    k_cache, v_cache are [pages, Nkv, page size, D] (a [pages, page size, Nkv, D] cache goes in transposed);
    kv_lens include the new tokens.  Returns the normed and rotated q (None without q)."""
    T, Nkv, D = shape = k.shape
    if v.shape != shape or v.dtype is not k.dtype:
        raise ValueError('k and v share a shape and a dtype')
    dev = _device(k)
    num_seqs = kv_lens.numel()
    cu = 0
    if cu_seqlens is not None:
        cu = _arg(cu_seqlens, torch.int32, dev, 'cu_seqlens')
        if cu_seqlens.numel() != num_seqs + 1:
            raise ValueError('cu_seqlens has one entry more than kv_lens')
    cache = _cache(k_cache, v_cache, block_table, kv_lens, Nkv, D, num_seqs, dev)
    Nq, qo, qdt = Nkv, 0, GDN_BF16
    if q is not None:
        q_shape = q.shape
        Nq = q_shape[1]
        if q_shape != (T, Nq, D) or q.dtype is not k.dtype:
            raise ValueError('q shares tokens, head_dim and dtype with k')
        q_out = (torch.empty(q_shape, dtype=out_dtype, device=q.device) if q_out is None
                 else _given(q_out, q_shape, dev, 'q_out'))
        qo, qdt = q_out.data_ptr(), _dt(q_out)
    st = _fn('gdn_paged_kv_append')(
        _pack_dims(num_seqs, T, Nq, Nkv, D), cu, _heads(q, dev, 'q'), _heads(k, dev, 'k'), _heads(v, dev, 'v'), _dt(k),
        _norm_rope(q_norm_w, k_norm_w, norm_eps, cos_sin, positions, interleaved, T, D, dev), cache, _dt(k_cache),
        qo, qdt, _stream())
    if st:
        _check(st, 'gdn_paged_kv_append')
    return q_out if q is not None else None


def paged_attn_decode_workspace_size(num_seqs, total, Nq, Nkv, D, dtype, table_tokens):
    """Bytes for calls of these heads and type over tables of up to ``table_tokens`` cache entries (the numbers
    of sequences and tokens do not matter)."""
    n = _SZ(0)
    _check(lib().gdn_paged_attn_decode_workspace_size(gdn_attn_dims(num_seqs, total, Nq, Nkv, D),
                                                      GDN_BF16 if dtype == torch.bfloat16 else GDN_F32,
                                                      table_tokens, n), 'gdn_paged_attn_decode_workspace_size')
    return n.value


@functools.lru_cache(maxsize=256)
def _attn_workspace_size(device, *sizes):
    return paged_attn_decode_workspace_size(1, 1, *sizes)


def _attn_call(q, k_cache, v_cache, block_table, kv_lens, scale, gate, cu_seqlens, out_dtype, o, workspace):
    """Checks the arguments of paged_attn_decode; the library call's, the output and the workspace (to be held
    until the call is made)."""
    T, Nq, D = shape = q.shape
    dtype = q.dtype
    if k_cache.dtype is not dtype or (gate is not None and (gate.dtype is not dtype or gate.shape != shape)):
        raise ValueError('q, gate and the cache share a dtype; gate has the shape of q')
    dev = _device(q)
    num_seqs = kv_lens.numel()
    cu = 0
    if cu_seqlens is not None:
        cu = _arg(cu_seqlens, torch.int32, dev, 'cu_seqlens')
        if cu_seqlens.numel() != num_seqs + 1:
            raise ValueError('cu_seqlens has one entry more than kv_lens')
    Nkv = k_cache.shape[1]
    cache = _cache(k_cache, v_cache, block_table, kv_lens, Nkv, D, num_seqs, dev)
    o = torch.empty(shape, dtype=out_dtype, device=q.device) if o is None else _given(o, shape, dev, 'o')
    ws = 0
    if workspace is None:
        ws_bytes = _attn_workspace_size(dev, Nq, Nkv, D, dtype, block_table.shape[1] * k_cache.shape[2])
        if ws_bytes > 0:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
            ws = workspace.data_ptr()
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
        ws = _given(workspace, workspace.shape, dev, 'workspace').data_ptr()
    return (_pack_dims(num_seqs, T, Nq, Nkv, D), cu, _heads(q, dev, 'q'), _heads(gate, dev, 'gate'), _dt(q), cache,
            _F(1.0 / math.sqrt(D) if scale is None else scale), o.data_ptr(), _dt(o), ws, ws_bytes, _stream()), o, workspace


def paged_attn_decode(q, k_cache, v_cache, block_table, kv_lens, scale=None, gate=None, cu_seqlens=None,
                      out_dtype=torch.bfloat16, o=None, workspace=None):
    """gdn_paged_attn_decode: attention of the new tokens q [tokens, Nq, D] (one or a few per sequence, bounds
    from cu_seqlens, else equally many) over the cache, times sigmoid(gate) when given.  Returns o."""
    args, o, workspace = _attn_call(q, k_cache, v_cache, block_table, kv_lens, scale, gate, cu_seqlens, out_dtype, o,
                                    workspace)
    st = _fn('gdn_paged_attn_decode')(*args)
    if st:
        _check(st, 'gdn_paged_attn_decode')
    return o


def attention_decode(q, k, v, k_cache, v_cache, block_table, kv_lens, cos_sin=None, q_norm_w=None, k_norm_w=None,
                     gate=None, positions=None, cu_seqlens=None, scale=None, norm_eps=1e-6, interleaved=False,
                     out_dtype=torch.bfloat16, bufs=None, k_scale=None, v_scale=None):
    """One step of a full-attention layer from its projections to the input of its output projection, the
    counterpart of decode_fused in a hybrid decoder's other layers: paged_kv_append (k and v into the cache, q
    and k normed and rotated) -> paged_attn_decode (with the output gate).  What either call refuses is refused
    before the cache changes.  With k_scale and v_scale the cache is one in 4 bits: paged_kv4_append ->
    paged_kv4_attn_decode, in bf16.

    ``bufs`` (optional dict) supplies preallocated q, o, workspace."""
    bufs = bufs or {}
    four = k_scale is not None or v_scale is not None
    if four and (k_scale is None or v_scale is None or out_dtype is not torch.bfloat16):
        raise ValueError('a cache in 4 bits comes with k_scale and v_scale, its attention in bfloat16')
    qr = bufs.get('q')
    if qr is None:
        qr = torch.empty(q.shape, dtype=torch.bfloat16 if four else k_cache.dtype, device=q.device)
    elif qr.shape != q.shape or not qr.is_contiguous():
        raise ValueError('the q buffer is contiguous and has the shape of q')
    T, Nq, D = q.shape
    if four:
        args, o, workspace = _kv4_attn_call(qr, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, scale, gate,
                                            cu_seqlens, bufs.get('o'), bufs.get('workspace'))
        got, need = args[8], _kv4_workspace_size(qr.get_device(), D, block_table.shape[1] * k_cache.shape[2])
        if T * Nq >= 1 << 31:
            raise ValueError('tokens times query heads must be below 2^31')
    else:
        args, o, workspace = _attn_call(qr, k_cache, v_cache, block_table, kv_lens, scale, gate, cu_seqlens, out_dtype,
                                        bufs.get('o'), bufs.get('workspace'))
        got, need = args[10], _attn_workspace_size(qr.get_device(), Nq, k_cache.shape[1], D, qr.dtype,
                                                   block_table.shape[1] * k_cache.shape[2])
    # what only the library itself would find wrong with the attention's own arguments
    for t, what in ((o, 'o'), (workspace, 'workspace'), (gate, 'gate')):
        if t is not None and t.data_ptr() % 16:
            raise ValueError('%s must be 16-byte aligned' % what)
    if gate is not None and any(n > 1 and s * gate.element_size() % 16 for n, s in zip((T, Nq), gate.stride())):
        raise ValueError('the strides of gate must be multiples of 16 bytes')
    if T > 0 and got < need:
        raise ValueError('a workspace of %d bytes required, got %d' % (need, got))
    if four:
        paged_kv4_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, q, cos_sin, q_norm_w, k_norm_w,
                         positions, cu_seqlens, norm_eps, interleaved, q_out=qr)
    else:
        paged_kv_append(k, v, k_cache, v_cache, block_table, kv_lens, q, cos_sin, q_norm_w, k_norm_w, positions, cu_seqlens,
                        norm_eps, interleaved, q_out=qr)
    name = 'gdn_paged_kv4_attn_decode' if four else 'gdn_paged_attn_decode'
    st = _fn(name)(*args)
    if st:
        _check(st, name)
    return o


# --- the paged cache in 4 bits ---------------------------------------------------------

KV4_GROUP = 64


def _used(t):
    """The strides of a tensor, those over an axis of one entry (never used) as if it were contiguous."""
    out, span = list(t.stride()), 1
    for i in range(t.dim() - 1, -1, -1):
        if t.shape[i] == 1:
            out[i] = span
        span = max(span, out[i] * t.shape[i])
    return out


def _cache4(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, Nkv, D, num_seqs, dev):
    """Checks a 4-bit cache's tensors against the call's sizes and packs them."""
    shape = k_cache.shape
    u8, bf = torch.uint8, torch.bfloat16
    if len(shape) != 4 or v_cache.shape != shape or k_cache.dtype is not u8 or v_cache.dtype is not u8:
        raise ValueError('k_cache and v_cache share the shape [pages, kv heads, page size, head_dim / 2], in uint8')
    pages, H, P, E = shape
    scales = k_scale.shape
    if scales != (pages, H, P, E // (KV4_GROUP // 2), 2) or v_scale.shape != scales:
        raise ValueError('k_scale and v_scale are [pages, kv heads, page size, head_dim / 64, 2]')
    if k_scale.dtype is not bf or v_scale.dtype is not bf:
        raise ValueError('the scales must be bfloat16')
    if not k_cache.get_device() == v_cache.get_device() == k_scale.get_device() == v_scale.get_device() == dev:
        raise ValueError('the cache must be on the device of the other tensors')
    if H != Nkv or 2 * E != D:
        raise ValueError('the cache holds %d heads of %d, the call has %d of %d' % (H, 2 * E, Nkv, D))
    st, vt, ks, vs = k_cache.stride(), v_cache.stride(), k_scale.stride(), v_scale.stride()
    if pages == 1 or H == 1 or P == 1 or (ks[3] != 2 and scales[3] == 1):
        st, vt, ks, vs = _used(k_cache), _used(v_cache), _used(k_scale), _used(v_scale)
    if st[3] != 1 or ks[4] != 1 or ks[3] != 2:
        raise ValueError('the head rows of the cache and of its scales must be contiguous')
    if vt != st or vs != ks:
        raise ValueError('k_cache and v_cache, and k_scale and v_scale, must have the same strides')
    rows = block_table.shape
    if len(rows) != 2 or rows[0] != num_seqs or kv_lens.numel() != num_seqs:
        raise ValueError('block_table is [sequences, pages] and kv_lens [sequences]')
    return _pack_cache4(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), st[0], st[1], st[2],
                        ks[0], ks[1], ks[2], pages, P, rows[1], _arg(block_table, torch.int32, dev, 'block_table'),
                        _arg(kv_lens, torch.int32, dev, 'kv_lens'))


def _bounds(cu_seqlens, num_seqs, dev):
    if cu_seqlens is None:
        return 0
    if cu_seqlens.numel() != num_seqs + 1:
        raise ValueError('cu_seqlens has one entry more than there are sequences')
    return _arg(cu_seqlens, torch.int32, dev, 'cu_seqlens')


def paged_kv4_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, q=None, cos_sin=None, q_norm_w=None,
                     k_norm_w=None, positions=None, cu_seqlens=None, norm_eps=1e-6, interleaved=False,
                     out_dtype=torch.bfloat16, q_out=None):
    """gdn_paged_kv4_append: paged_kv_append into a cache in 4 bits, in place.  k_cache, v_cache are [pages, Nkv, page
    size, D / 2] uint8, k_scale, v_scale [pages, Nkv, page size, D / 64, 2] bf16 (either with its axes in another
    order in memory).  Returns the normed and rotated q (None without q)."""
    T, Nkv, D = shape = k.shape
    if v.shape != shape or v.dtype is not k.dtype:
        raise ValueError('k and v share a shape and a dtype')
    dev = _device(k)
    num_seqs = kv_lens.numel()
    cu = _bounds(cu_seqlens, num_seqs, dev)
    cache = _cache4(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, Nkv, D, num_seqs, dev)
    Nq, qo, qdt = Nkv, 0, GDN_BF16
    if q is not None:
        q_shape = q.shape
        Nq = q_shape[1]
        if q_shape != (T, Nq, D) or q.dtype is not k.dtype:
            raise ValueError('q shares tokens, head_dim and dtype with k')
        q_out = (torch.empty(q_shape, dtype=out_dtype, device=q.device) if q_out is None
                 else _given(q_out, q_shape, dev, 'q_out'))
        qo, qdt = q_out.data_ptr(), _dt(q_out)
    st = _fn('gdn_paged_kv4_append')(
        _pack_dims(num_seqs, T, Nq, Nkv, D), cu, _heads(q, dev, 'q'), _heads(k, dev, 'k'), _heads(v, dev, 'v'), _dt(k),
        _norm_rope(q_norm_w, k_norm_w, norm_eps, cos_sin, positions, interleaved, T, D, dev), cache, qo, qdt, _stream())
    if st:
        _check(st, 'gdn_paged_kv4_append')
    return q_out if q is not None else None


def paged_kv4_read(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, total_tokens, cu_seqlens=None,
                   out_dtype=torch.bfloat16, out=None):
    """gdn_paged_kv4_read: the last tokens of each sequence (bounds from cu_seqlens, else equally many of the
    total_tokens; as many as kv_lens says: all of it) as dense (k, v) [total_tokens, Nkv, D]; ``out`` may supply them."""
    dev = _device(k_cache)
    Nkv, D = k_cache.shape[1], 2 * k_cache.shape[3]
    num_seqs = kv_lens.numel()
    cu = _bounds(cu_seqlens, num_seqs, dev)
    cache = _cache4(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, Nkv, D, num_seqs, dev)
    shape = (total_tokens, Nkv, D)
    if out is None:
        k, v = (torch.empty(shape, dtype=out_dtype, device=k_cache.device) for _ in range(2))
    else:
        k, v = (_given(t, shape, dev, 'out') for t in out)
        if k.dtype is not v.dtype:
            raise ValueError('the outputs share a dtype')
    st = _fn('gdn_paged_kv4_read')(_pack_dims(num_seqs, total_tokens, Nkv, Nkv, D), cu, cache, k.data_ptr(), v.data_ptr(),
                                   _dt(k), _stream())
    if st:
        _check(st, 'gdn_paged_kv4_read')
    return k, v


def paged_kv4_attn_decode_workspace_size(D, table_tokens):
    """Bytes for calls with heads of D over tables of up to ``table_tokens`` cache entries (nothing else matters)."""
    n = _SZ(0)
    _check(lib().gdn_paged_kv4_attn_decode_workspace_size(gdn_attn_dims(1, 1, 1, 1, D), table_tokens, n),
           'gdn_paged_kv4_attn_decode_workspace_size')
    return n.value


@functools.lru_cache(maxsize=256)
def _kv4_workspace_size(device, D, table_tokens):
    return paged_kv4_attn_decode_workspace_size(D, table_tokens)


def _kv4_attn_call(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, scale, gate, cu_seqlens, o, workspace):
    """Checks the arguments of paged_kv4_attn_decode; the library call's, the output and the workspace (to be held
    until the call is made)."""
    T, Nq, D = shape = q.shape
    bf = torch.bfloat16
    if q.dtype is not bf or (gate is not None and (gate.dtype is not bf or gate.shape != shape)):
        raise ValueError('q and gate are bfloat16; gate has the shape of q')
    dev = _device(q)
    num_seqs = kv_lens.numel()
    cu = _bounds(cu_seqlens, num_seqs, dev)
    Nkv = k_cache.shape[1]
    cache = _cache4(k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, Nkv, D, num_seqs, dev)
    if o is None:
        o = torch.empty(shape, dtype=bf, device=q.device)
    elif _given(o, shape, dev, 'o').dtype is not bf:
        raise ValueError('o must be bfloat16')
    ws = 0
    if workspace is None:
        ws_bytes = _kv4_workspace_size(dev, D, block_table.shape[1] * k_cache.shape[2])
        if ws_bytes > 0:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
            ws = workspace.data_ptr()
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
        ws = _given(workspace, workspace.shape, dev, 'workspace').data_ptr()
    return (_pack_dims(num_seqs, T, Nq, Nkv, D), cu, _heads(q, dev, 'q'), _heads(gate, dev, 'gate'), cache,
            _F(1.0 / math.sqrt(D) if scale is None else scale), o.data_ptr(), ws, ws_bytes, _stream()), o, workspace


def paged_kv4_attn_decode(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, scale=None, gate=None,
                          cu_seqlens=None, o=None, workspace=None):
    """gdn_paged_kv4_attn_decode: paged_attn_decode over a cache in 4 bits; q, gate and o are bf16.  Returns o."""
    args, o, workspace = _kv4_attn_call(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, scale, gate, cu_seqlens,
                                        o, workspace)
    st = _fn('gdn_paged_kv4_attn_decode')(*args)
    if st:
        _check(st, 'gdn_paged_kv4_attn_decode')
    return o


# --- around the layers: the cache's metadata, and which drafted tokens stay ------------

PLAN_REST = 0x7fffffff                                   # GDN_PLAN_REST
PagedPlan = collections.namedtuple('PagedPlan', 'cu_seqlens positions slots kv_lens pages_held free_ring')


def paged_plan(new_lens, kv_lens, pages_held, free_ring, free_pages, block_table, page_size, total_tokens, out=None):
    """gdn_paged_plan: the step's metadata from its requests.  new_lens, kv_lens, pages_held [N], free_ring [2] and
    free_pages [num_pages] are int32; block_table [N, max_pages] and free_pages are updated in place.  Returns a
    PagedPlan of new tensors, or fills ``out`` (a PagedPlan; its kv_lens, pages_held and free_ring may be the inputs,
    its positions and slots None).  new_lens of the last sequence may be PLAN_REST: an inactive slot that takes the rows
    up to total_tokens."""
    dev = _device(new_lens)
    N = new_lens.numel()
    if kv_lens.numel() != N or pages_held.numel() != N or free_ring.numel() != 2:
        raise ValueError('new_lens, kv_lens and pages_held have one entry per sequence, free_ring two')
    table = block_table.shape
    if len(table) != 2 or table[0] != N:
        raise ValueError('block_table is [sequences, pages]')
    i32 = torch.int32
    ins = (_arg(new_lens, i32, dev, 'new_lens'), _arg(kv_lens, i32, dev, 'kv_lens'), _arg(pages_held, i32, dev, 'pages_held'),
           _arg(free_ring, i32, dev, 'free_ring'), _arg(free_pages, i32, dev, 'free_pages'),
           _arg(block_table, i32, dev, 'block_table'))
    if out is None:
        # six allocations take 9 us on a Grace host, one and its six views 14
        empty, on = torch.empty, new_lens.device
        out = PagedPlan(empty(N + 1, dtype=i32, device=on), empty(total_tokens, dtype=i32, device=on),
                        empty(total_tokens, dtype=torch.int64, device=on), empty(N, dtype=i32, device=on),
                        empty(N, dtype=i32, device=on), empty(2, dtype=i32, device=on))
        outs = [t.data_ptr() for t in out]
    else:
        for t, n in ((out.cu_seqlens, N + 1), (out.positions, total_tokens), (out.slots, total_tokens), (out.kv_lens, N),
                     (out.pages_held, N), (out.free_ring, 2)):
            if t is not None and t.numel() != n:
                raise ValueError('an output has %d entries, not %d' % (t.numel(), n))
        outs = (_arg(out.cu_seqlens, i32, dev, 'cu_seqlens'), _arg(out.positions, i32, dev, 'positions'),
                _arg(out.slots, torch.int64, dev, 'slots'), _arg(out.kv_lens, i32, dev, 'kv_lens'),
                _arg(out.pages_held, i32, dev, 'pages_held'), _arg(out.free_ring, i32, dev, 'free_ring'))
    st = _fn('gdn_paged_plan')(_pack_plan(N, total_tokens, free_pages.numel(), page_size, table[1], *ins, *outs), _stream())
    if st:
        _check(st, 'gdn_paged_plan')
    return out


def draft_verify(target_probs, tokens, uniform, draft_probs=None, cu_seqlens=None, num_seqs=1, kv_lens=None, out=None):
    """gdn_draft_verify: target_probs [T, V] (bf16 or float32; rows may be apart), tokens [T] int32 and uniform [T]
    float32 of a multi-token step (a prompt's last token alone, with bounds that count it as one row), draft_probs [N,
    drafts, V] (any strides over the first two axes; [N, 0, V] only where no sequence can have more than one row) or None.
    Returns (accepted [N], out_tokens [T], kv_lens [N] less the refused drafts, None without kv_lens); ``out`` may supply
    them (its kv_lens may be the input)."""
    T, V = target_probs.shape
    dev = _device(target_probs)
    if cu_seqlens is not None:
        num_seqs = cu_seqlens.numel() - 1
    if tokens.numel() != T or uniform.numel() != T or (kv_lens is not None and kv_lens.numel() != num_seqs):
        raise ValueError('tokens and uniform have one entry per row, kv_lens one per sequence')
    ld, es = target_probs.stride()
    if es != 1 and V > 1:
        raise ValueError('the rows of target_probs must be contiguous')
    drafts = ptr = ss = sr = 0
    if draft_probs is not None:
        if draft_probs.get_device() != dev:
            raise ValueError('draft_probs must be on the device of the other tensors')
        if draft_probs.dim() != 3 or draft_probs.shape[0] != num_seqs or draft_probs.shape[2] != V:
            raise ValueError('draft_probs is [sequences, drafts, vocabulary]')
        if draft_probs.dtype is not target_probs.dtype:
            raise ValueError('target_probs and draft_probs share a dtype')
        drafts = draft_probs.shape[1]
        ss, sr, es = draft_probs.stride()
        if es != 1 and V > 1:
            raise ValueError('the rows of draft_probs must be contiguous')
        ptr = draft_probs.data_ptr()
        if num_seqs == 1:
            ss = 0                                               # (a stride over one entry is never used)
        if drafts <= 1:
            sr = 0
        if drafts == 0:
            # fine for steps without drafts; None, which the library would get, is another rule for those that have some
            if T > 1 and (cu_seqlens is not None or T > num_seqs):
                raise ValueError('draft_probs of no drafts for sequences that may have some')
            ptr = 0
    i32 = torch.int32
    if out is None:
        empty, on = torch.empty, target_probs.device
        accepted, out_tokens = empty(num_seqs, dtype=i32, device=on), empty(T, dtype=i32, device=on)
        lens_out = None if kv_lens is None else empty(num_seqs, dtype=i32, device=on)
        out = (accepted, out_tokens, lens_out)
        outs = (0 if kv_lens is None else lens_out.data_ptr(), accepted.data_ptr(), out_tokens.data_ptr())
    else:
        accepted, out_tokens, lens_out = out
        if accepted.numel() != num_seqs or out_tokens.numel() != T or (kv_lens is not None and (
                lens_out is None or lens_out.numel() != num_seqs)):
            raise ValueError('the outputs are accepted [sequences], out_tokens [rows] and kv_lens [sequences]')
        if kv_lens is None:
            out = (accepted, out_tokens, None)
        outs = (_arg(out[2], i32, dev, 'the kv_lens output'), _arg(accepted, i32, dev, 'accepted'),
                _arg(out_tokens, i32, dev, 'out_tokens'))
    st = _fn('gdn_draft_verify')(
        num_seqs, T, V, drafts, _arg(cu_seqlens, i32, dev, 'cu_seqlens'), target_probs.data_ptr(), ld if T > 1 else V, ptr, ss,
        sr, _dt(target_probs), _arg(tokens, i32, dev, 'tokens'), _arg(uniform, torch.float32, dev, 'uniform'),
        _arg(kv_lens, i32, dev, 'kv_lens'), *outs, _stream())
    if st:
        _check(st, 'gdn_draft_verify')
    return out
