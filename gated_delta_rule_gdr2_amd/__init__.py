"""MI355X-native Gated Delta Rule-2 operator: thin Python binding of libgdr2.

The operator ("Gated DeltaNet-2: Decoupling Erase and Write in Linear
Attention", anthology record LIT-802, takeaway 1; paper Sec. 3.1 Eqs. 8-10)

    S_t = (I - k_t (b_t * k_t)^T) diag(exp g_t) S_{t-1} + k_t (w_t * v_t)^T
    o_t = S_t^T q_t

runs entirely in the HIP kernels of ``libgdr2.so`` (built from ``csrc/`` by
``python -m gated_delta_rule_gdr2_amd.build``); see ``include/gdr2.h`` for the
C ABI. So do the same recurrence with scalar gates (``gdr2_scalar_*``) and, for
the other layers of a hybrid decoder, attention over whole sequences with its
gradients (``gdr2_attn_fwd``, ``gdr2_attn_bwd``), over a paged key-value cache, of
one token (``gdr2_attn_step``) or of drafted ones (``gdr2_attn_tree``), and what
keeps the cache (``gdr2_kv_append``, ``gdr2_kv_keep``, ``gdr2_kv_pages``). This module
only marshals torch tensors (device memory and the current HIP stream) into
those calls. There is no fallback: if the library is missing every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch
from torch.autograd.forward_ad import unpack_dual
from torch.autograd.function import once_differentiable

__all__ = ["gdr2_fwd", "gdr2_bwd", "gdr2_step", "gdr2_fwd_logits", "gdr2_bwd_logits", "gdr2_step_logits",
           "gdr2_fwd_seg", "gdr2_bwd_seg", "gdr2_fwd_noalloc", "gdr2_fwd_workspace_bytes",
           "gdr2_bwd_workspace_bytes", "gdr2_seg_workspace_bytes", "gdr2_strerror", "gdr2_version", "GDR2Function",
           "gdr2_scalar_fwd", "gdr2_scalar_bwd", "gdr2_scalar_step", "gdr2_scalar_workspace_bytes",
           "GDR2ScalarFunction", "gdr2_attn_step", "gdr2_attn_workspace_bytes", "gdr2_kv_append",
           "gdr2_attn_fwd", "gdr2_attn_bwd", "gdr2_attn_bwd_workspace_bytes", "GDR2AttnFunction", "gdr2_attn_tree",
           "gdr2_attn_tree_workspace_bytes", "gdr2_kv_keep", "gdr2_kv_pages",
           "library_path", "load_library"]

_HERE = os.path.dirname(os.path.abspath(__file__))
# GDR2_LIB names another build of the same library (e.g. one with host-side sanitizers)
_LIB_PATH = os.environ.get("GDR2_LIB") or os.path.join(_HERE, "libgdr2.so")
_lib = None

DTYPE_F32, DTYPE_BF16 = 0, 1
_DT = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
EXPORTED = ["gdr2_fwd", "gdr2_bwd", "gdr2_step", "gdr2_fwd_logits", "gdr2_bwd_logits", "gdr2_step_logits",
            "gdr2_fwd_seg", "gdr2_bwd_seg", "gdr2_fwd_noalloc", "gdr2_fwd_workspace_bytes",
            "gdr2_bwd_workspace_bytes", "gdr2_seg_workspace_bytes", "gdr2_strerror", "gdr2_version",
            "gdr2_scalar_fwd", "gdr2_scalar_bwd", "gdr2_scalar_step", "gdr2_scalar_workspace_bytes",
            "gdr2_attn_step", "gdr2_attn_workspace_bytes", "gdr2_kv_append", "gdr2_attn_fwd", "gdr2_attn_bwd",
            "gdr2_attn_bwd_workspace_bytes", "gdr2_attn_tree", "gdr2_attn_tree_workspace_bytes", "gdr2_kv_keep",
            "gdr2_kv_pages"]
NOALLOC_SCRATCH_BYTES = 64 << 20  # GDR2_NOALLOC_SCRATCH_BYTES in include/gdr2.h


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libgdr2.so (raises RuntimeError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError("libgdr2.so not found at %s; build it with "
                           "`python -m gated_delta_rule_gdr2_amd.build`" % _LIB_PATH)
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.gdr2_fwd_workspace_bytes.argtypes = [i] * 8
    lib.gdr2_fwd_workspace_bytes.restype = sz
    lib.gdr2_bwd_workspace_bytes.argtypes = [i] * 7
    lib.gdr2_bwd_workspace_bytes.restype = sz
    lib.gdr2_fwd.argtypes = [vp] * 9 + [i] * 8 + [vp, sz, vp, vp]
    lib.gdr2_fwd.restype = i
    lib.gdr2_bwd.argtypes = [vp] * 16 + [i] * 8 + [vp, sz, vp, vp]
    lib.gdr2_bwd.restype = i
    lib.gdr2_step.argtypes = [vp] * 8 + [i] * 6 + [vp]
    lib.gdr2_step.restype = i
    f = ctypes.c_float
    lib.gdr2_fwd_logits.argtypes = [vp] * 6 + [f, f] + [vp] * 3 + [i] * 8 + [vp, sz, vp, vp]
    lib.gdr2_fwd_logits.restype = i
    lib.gdr2_bwd_logits.argtypes = [vp] * 6 + [f, f] + [vp] * 10 + [i] * 8 + [vp, sz, vp, vp]
    lib.gdr2_bwd_logits.restype = i
    lib.gdr2_step_logits.argtypes = [vp] * 6 + [f, f] + [vp] * 2 + [i] * 6 + [vp]
    lib.gdr2_step_logits.restype = i
    lib.gdr2_seg_workspace_bytes.argtypes = [i] * 9
    lib.gdr2_seg_workspace_bytes.restype = sz
    lib.gdr2_fwd_seg.argtypes = [vp] * 9 + [i] * 9 + [vp, sz, vp, vp]
    lib.gdr2_fwd_seg.restype = i
    lib.gdr2_bwd_seg.argtypes = [vp] * 16 + [i] * 9 + [vp, sz, vp, vp]
    lib.gdr2_bwd_seg.restype = i
    lib.gdr2_fwd_noalloc.argtypes = [vp] * 9 + [i] * 7 + [vp]
    lib.gdr2_fwd_noalloc.restype = i
    lib.gdr2_scalar_workspace_bytes.argtypes = [i] * 9
    lib.gdr2_scalar_workspace_bytes.restype = sz
    lib.gdr2_scalar_fwd.argtypes = [vp] * 9 + [i] * 9 + [vp, sz, vp]
    lib.gdr2_scalar_fwd.restype = i
    lib.gdr2_scalar_bwd.argtypes = [vp] * 15 + [i] * 9 + [vp, sz, vp]
    lib.gdr2_scalar_bwd.restype = i
    lib.gdr2_scalar_step.argtypes = [vp] * 8 + [i] * 8 + [vp]
    lib.gdr2_scalar_step.restype = i
    lib.gdr2_attn_workspace_bytes.argtypes = [i] * 5
    lib.gdr2_attn_workspace_bytes.restype = sz
    lib.gdr2_attn_step.argtypes = [vp] * 8 + [i] * 7 + [f] + [i] * 2 + [vp, sz, vp]
    lib.gdr2_attn_step.restype = i
    lib.gdr2_kv_append.argtypes = [vp] * 8 + [i] * 8 + [vp]
    lib.gdr2_kv_append.restype = i
    lib.gdr2_attn_fwd.argtypes = [vp] * 8 + [i] * 5 + [f] + [i] * 3 + [vp]
    lib.gdr2_attn_fwd.restype = i
    lib.gdr2_attn_bwd_workspace_bytes.argtypes = [i] * 7
    lib.gdr2_attn_bwd_workspace_bytes.restype = sz
    lib.gdr2_attn_bwd.argtypes = [vp] * 12 + [i] * 5 + [f] + [i] * 3 + [vp, sz, vp]
    lib.gdr2_attn_bwd.restype = i
    lib.gdr2_attn_tree_workspace_bytes.argtypes = [i] * 6
    lib.gdr2_attn_tree_workspace_bytes.restype = sz
    lib.gdr2_attn_tree.argtypes = [vp] * 9 + [i] * 8 + [f] + [i] * 2 + [vp, sz, vp]
    lib.gdr2_attn_tree.restype = i
    lib.gdr2_kv_keep.argtypes = [vp] * 7 + [i] * 8 + [vp]
    lib.gdr2_kv_keep.restype = i
    lib.gdr2_kv_pages.argtypes = [vp] * 8 + [i] * 5 + [vp]
    lib.gdr2_kv_pages.restype = i
    lib.gdr2_strerror.argtypes = [i]
    lib.gdr2_strerror.restype = ctypes.c_char_p
    lib.gdr2_version.argtypes = []
    lib.gdr2_version.restype = i
    _lib = lib
    return lib


def gdr2_strerror(status: int) -> str:
    return load_library().gdr2_strerror(int(status)).decode()


def gdr2_version() -> int:
    return int(load_library().gdr2_version())


def gdr2_fwd_workspace_bytes(B, T, H, dk, dv, chunk=64, dtype=DTYPE_BF16, save_for_bwd=False) -> int:
    return int(load_library().gdr2_fwd_workspace_bytes(B, T, H, dk, dv, chunk, dtype, int(bool(save_for_bwd))))


def gdr2_bwd_workspace_bytes(B, T, H, dk, dv, chunk=64, dtype=DTYPE_BF16) -> int:
    return int(load_library().gdr2_bwd_workspace_bytes(B, T, H, dk, dv, chunk, dtype))


def gdr2_seg_workspace_bytes(B, T, H, dk, dv, chunk=64, segments=1, dtype=DTYPE_BF16, save_for_bwd=False) -> int:
    return int(load_library().gdr2_seg_workspace_bytes(B, T, H, dk, dv, chunk, segments, dtype,
                                                       int(bool(save_for_bwd))))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, dtype, shape):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _raise(status, what):
    if status != 0:
        raise RuntimeError("%s failed: %s (status %d)" % (what, gdr2_strerror(status), status))


def _dims(q, v):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if q.dtype not in _DT:
        raise ValueError("unsupported dtype %s" % q.dtype)
    return B, T, H, dk, dv, _DT[q.dtype]


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _keep_for(stream, *tensors):
    """Tensors allocated here come from torch's current stream; when the kernels run on
    another stream, tell the caching allocator that this stream uses them too, so that their
    memory is not handed out again (after the caller, or this module, drops them) before the
    work enqueued on that stream has finished with it."""
    if stream is None or stream == torch.cuda.current_stream():
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def workspace(B, T, H, dk, dv, dtype, train, device="cuda", segments=None):
    """Allocate a workspace tensor (uint8) big enough for gdr2_fwd(save_for_bwd=train) / gdr2_bwd
    (segments=None), or for their _seg variants with that many segments."""
    dt = _DT[dtype] if isinstance(dtype, torch.dtype) else dtype
    if segments is None:
        n = gdr2_bwd_workspace_bytes(B, T, H, dk, dv, 64, dt) if train else \
            gdr2_fwd_workspace_bytes(B, T, H, dk, dv, 64, dt, False)
    else:
        n = gdr2_seg_workspace_bytes(B, T, H, dk, dv, 64, segments, dt, train)
    if n == 0 and B * T * H > 0:
        raise ValueError("unsupported shape/dtype for gdr2: B=%d T=%d H=%d dk=%d dv=%d" % (B, T, H, dk, dv))
    return torch.empty(n, dtype=torch.uint8, device=device)  # empty for a call without tokens


def gdr2_fwd(q, k, v, g, b, w, h0=None, *, chunk=64, save_for_bwd=False, ws=None, o=None,
             output_final_state=True, stream=None, stage_events=None):
    """Forward pass. q, k, g, b: [B,T,H,dk]; v, w: [B,T,H,dv] (bf16 or fp32, same dtype);
    h0: [B,H,dk,dv] fp32 or None. Returns (o, ht or None, ws). Pass ``ws`` back to
    gdr2_bwd(..., fwd_saved=True) when save_for_bwd is set. ``stage_events``: optional
    ctypes array of hipEvent_t handles recorded around the kernels (see include/gdr2.h)."""
    return _fwd(None, q, k, v, g, b, w, h0, chunk, save_for_bwd, ws, o, output_final_state, stream,
                stage_events)


def gdr2_fwd_seg(q, k, v, g, b, w, h0=None, *, segments, chunk=64, save_for_bwd=False, ws=None, o=None,
                 output_final_state=True, stream=None, stage_events=None):
    """gdr2_fwd with the state chains cut into ``segments`` pieces walked in parallel
    (chunk-parallel scan; see include/gdr2.h). The workspace must be sized for the same segments."""
    return _fwd(None, q, k, v, g, b, w, h0, chunk, save_for_bwd, ws, o, output_final_state, stream,
                stage_events, segments)


def gdr2_fwd_logits(q, k, v, zg, zb, zw, h0=None, *, g_scale=1.0, b_scale=1.0, chunk=64, save_for_bwd=False,
                    ws=None, o=None, output_final_state=True, stream=None, stage_events=None):
    """Forward pass with the gates given as logits, activated inside the kernels:
    g = -g_scale softplus(zg), b = b_scale sigmoid(zb), w = sigmoid(zw). Otherwise as gdr2_fwd."""
    return _fwd((g_scale, b_scale), q, k, v, zg, zb, zw, h0, chunk, save_for_bwd, ws, o, output_final_state,
                stream, stage_events)


def _fwd(scales, q, k, v, g, b, w, h0, chunk, save_for_bwd, ws, o, output_final_state, stream, stage_events,
         segments=None):
    lib = load_library()
    B, T, H, dk, dv, dt = _dims(q, v)
    for t, n, shp in ((q, "q", (B, T, H, dk)), (k, "k", (B, T, H, dk)), (g, "g", (B, T, H, dk)),
                      (b, "b", (B, T, H, dk)), (v, "v", (B, T, H, dv)), (w, "w", (B, T, H, dv))):
        _check(t, n, q.dtype, shp)
    _check(h0, "h0", torch.float32, (B, H, dk, dv))
    new = []
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
        new.append(o)
    _check(o, "o", q.dtype, (B, T, H, dv))
    ht = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device) if output_final_state else None
    new.append(ht)
    if ws is None:
        ws = workspace(B, T, H, dk, dv, dt, save_for_bwd, q.device, segments)
        new.append(ws)
    _keep_for(stream, *new)
    tail = (_ptr(h0), _ptr(o), _ptr(ht), B, T, H, dk, dv, chunk, dt, int(bool(save_for_bwd)), _ptr(ws),
            ws.numel(), _stream(stream), stage_events)
    if segments is not None:
        st = lib.gdr2_fwd_seg(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), *tail[:9], segments,
                              *tail[9:])
        _raise(st, "gdr2_fwd_seg")
        return o, ht, ws
    if scales is None:
        st = lib.gdr2_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), *tail)
    else:
        st = lib.gdr2_fwd_logits(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), *scales, *tail)
    _raise(st, "gdr2_fwd" if scales is None else "gdr2_fwd_logits")
    return o, ht, ws


def gdr2_fwd_noalloc(q, k, v, g, b, w, h0=None, *, chunk=64, o=None, output_final_state=True, stream=None):
    """Inference forward whose workspace is the library's fixed device array (for callers that
    cannot allocate device memory; see include/gdr2.h). The C call allocates nothing; this
    wrapper allocates o and ht only when they are not passed. Calls that overlap on one GPU race
    on the shared array. Returns (o, ht or None)."""
    lib = load_library()
    B, T, H, dk, dv, dt = _dims(q, v)
    for t, n, shp in ((q, "q", (B, T, H, dk)), (k, "k", (B, T, H, dk)), (g, "g", (B, T, H, dk)),
                      (b, "b", (B, T, H, dk)), (v, "v", (B, T, H, dv)), (w, "w", (B, T, H, dv))):
        _check(t, n, q.dtype, shp)
    _check(h0, "h0", torch.float32, (B, H, dk, dv))
    new = []
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
        new.append(o)
    _check(o, "o", q.dtype, (B, T, H, dv))
    ht = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device) if output_final_state else None
    new.append(ht)
    _keep_for(stream, *new)
    st = lib.gdr2_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), _ptr(h0), _ptr(o), _ptr(ht),
                              B, T, H, dk, dv, chunk, dt, _stream(stream))
    _raise(st, "gdr2_fwd_noalloc")
    return o, ht


def gdr2_step(q, k, v, g, b, w, state, *, o=None, stream=None):
    """Recurrent step (decoding): the T tokens of q, k, g, b [B,T,H,dk] and v, w [B,T,H,dv]
    one at a time from ``state`` ([B,H,dk,dv] fp32), which is updated in place. Returns o."""
    return _step(None, q, k, v, g, b, w, state, o, stream)


def gdr2_step_logits(q, k, v, zg, zb, zw, state, *, g_scale=1.0, b_scale=1.0, o=None, stream=None):
    """Recurrent step with the gates given as logits (activations as gdr2_fwd_logits)."""
    return _step((g_scale, b_scale), q, k, v, zg, zb, zw, state, o, stream)


def _step(scales, q, k, v, g, b, w, state, o, stream):
    lib = load_library()
    B, T, H, dk, dv, dt = _dims(q, v)
    for t, n, shp in ((q, "q", (B, T, H, dk)), (k, "k", (B, T, H, dk)), (g, "g", (B, T, H, dk)),
                      (b, "b", (B, T, H, dk)), (v, "v", (B, T, H, dv)), (w, "w", (B, T, H, dv))):
        _check(t, n, q.dtype, shp)
    if state is None:
        raise ValueError("state is required")
    _check(state, "state", torch.float32, (B, H, dk, dv))
    if o is None:
        o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device)
        _keep_for(stream, o)
    _check(o, "o", q.dtype, (B, T, H, dv))
    tail = (_ptr(state), _ptr(o), B, T, H, dk, dv, dt, _stream(stream))
    if scales is None:
        st = lib.gdr2_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), *tail)
    else:
        st = lib.gdr2_step_logits(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), *scales, *tail)
    _raise(st, "gdr2_step" if scales is None else "gdr2_step_logits")
    return o


def gdr2_bwd(q, k, v, g, b, w, h0, dout, dht=None, *, chunk=64, ws=None, fwd_saved=False,
             need_dh0=True, grads=None, stream=None, stage_events=None):
    """Backward pass. Returns a dict with dq, dk, dv, dg, db, dw (input dtype) and dh0 (fp32 or None).
    With fwd_saved=True, ``ws`` must be the workspace of a gdr2_fwd(..., save_for_bwd=True) call on
    the same inputs."""
    return _bwd(None, q, k, v, g, b, w, h0, dout, dht, chunk, ws, fwd_saved, need_dh0, grads, stream,
                stage_events)


def gdr2_bwd_seg(q, k, v, g, b, w, h0, dout, dht=None, *, segments, chunk=64, ws=None, fwd_saved=False,
                 need_dh0=True, grads=None, stream=None, stage_events=None):
    """gdr2_bwd with the reverse state chains cut into ``segments`` pieces (chunk-parallel scan).
    With fwd_saved=True, ``ws`` must come from gdr2_fwd_seg(save_for_bwd=True) with the same segments."""
    return _bwd(None, q, k, v, g, b, w, h0, dout, dht, chunk, ws, fwd_saved, need_dh0, grads, stream,
                stage_events, segments)


def gdr2_bwd_logits(q, k, v, zg, zb, zw, h0, dout, dht=None, *, g_scale=1.0, b_scale=1.0, chunk=64, ws=None,
                    fwd_saved=False, need_dh0=True, grads=None, stream=None, stage_events=None):
    """Backward with the gates given as logits: dg, db, dw of the returned dict are the gradients
    with respect to zg, zb, zw. With fwd_saved=True, ``ws`` must come from gdr2_fwd_logits on the
    same inputs and scales."""
    return _bwd((g_scale, b_scale), q, k, v, zg, zb, zw, h0, dout, dht, chunk, ws, fwd_saved, need_dh0, grads,
                stream, stage_events)


def _bwd(scales, q, k, v, g, b, w, h0, dout, dht, chunk, ws, fwd_saved, need_dh0, grads, stream, stage_events,
         segments=None):
    lib = load_library()
    B, T, H, dk, dv, dt = _dims(q, v)
    for t, n, shp in ((q, "q", (B, T, H, dk)), (k, "k", (B, T, H, dk)), (g, "g", (B, T, H, dk)),
                      (b, "b", (B, T, H, dk)), (v, "v", (B, T, H, dv)), (w, "w", (B, T, H, dv)),
                      (dout, "dout", (B, T, H, dv))):
        _check(t, n, q.dtype, shp)
    _check(h0, "h0", torch.float32, (B, H, dk, dv))
    _check(dht, "dht", torch.float32, (B, H, dk, dv))
    new = []
    if grads is None:
        grads = {n: torch.empty_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("db", b),
                                                     ("dw", w))}
        new += list(grads.values())
    grads["dh0"] = torch.empty(B, H, dk, dv, dtype=torch.float32, device=q.device) if need_dh0 else None
    new.append(grads["dh0"])
    if ws is None:
        if fwd_saved:
            raise ValueError("fwd_saved=True needs the forward's workspace")
        ws = workspace(B, T, H, dk, dv, dt, True, q.device, segments)
        new.append(ws)  # dropped on return: its memory must outlive the kernels on `stream`
    _keep_for(stream, *new)
    tail = (_ptr(h0), _ptr(dout), _ptr(dht), _ptr(grads["dq"]), _ptr(grads["dk"]), _ptr(grads["dv"]),
            _ptr(grads["dg"]), _ptr(grads["db"]), _ptr(grads["dw"]), _ptr(grads["dh0"]), B, T, H, dk, dv, chunk,
            dt, int(bool(fwd_saved)), _ptr(ws), ws.numel(), _stream(stream), stage_events)
    if segments is not None:
        st = lib.gdr2_bwd_seg(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), *tail[:16], segments,
                              *tail[16:])
        _raise(st, "gdr2_bwd_seg")
        return grads
    if scales is None:
        st = lib.gdr2_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), *tail)
    else:
        st = lib.gdr2_bwd_logits(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), *scales, *tail)
    _raise(st, "gdr2_bwd" if scales is None else "gdr2_bwd_logits")
    return grads


class GDR2Function(torch.autograd.Function):
    """Autograd wrapper: forward saves the per-chunk states in the workspace, backward reuses them."""

    @staticmethod
    def forward(ctx, q, k, v, g, b, w, h0=None):
        o, ht, ws = gdr2_fwd(q, k, v, g, b, w, h0, save_for_bwd=True)
        ctx.save_for_backward(q, k, v, g, b, w, h0, ws)
        ctx.has_h0 = h0 is not None
        return o, ht

    @staticmethod
    def backward(ctx, do, dht):
        q, k, v, g, b, w, h0, ws = ctx.saved_tensors
        gr = gdr2_bwd(q, k, v, g, b, w, h0, do.contiguous(),
                      None if dht is None else dht.contiguous(), ws=ws, fwd_saved=True,
                      need_dh0=ctx.has_h0)
        return gr["dq"], gr["dk"], gr["dv"], gr["dg"], gr["db"], gr["dw"], gr["dh0"]


# ---------------------------------------------------------------- gated delta rule with scalar gates


@functools.lru_cache(maxsize=256)
def gdr2_scalar_workspace_bytes(N, T, Hk, Hv, dk, dv, packed=False, dtype=DTYPE_BF16, save_for_bwd=False) -> int:
    return int(load_library().gdr2_scalar_workspace_bytes(N, T, Hk, Hv, dk, dv, int(bool(packed)), dtype,
                                                          int(bool(save_for_bwd))))


def _adr(t):
    return None if t is None else t.data_ptr()


def _want(t, name, dtype, shape, dev):
    """_check and one device for all, at a fraction of the calls into torch: a decode step's kernels take a
    few microseconds, and so do checks."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _check(t, name, dtype, shape)
        raise ValueError("all tensors must be on one device: %s is on %s, q or k on cuda:%d" % (name, t.device, dev))


def _device_of(t, name):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a GPU tensor" % name)
    return dev


# the current stream of a device as a number, without an object around it where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _launch(f, dev, stream, *args):
    """f(*args, stream) with device ``dev`` as the current one, on the given stream or the device's current one."""
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            return _launch(f, dev, stream, *args)
    return f(*args, _raw_stream(dev) if stream is None else stream.cuda_stream)


def _zero(stream, *tensors):
    """Sets tensors to zero on the stream that the call's kernels would run on."""
    with torch.cuda.stream(stream):  # None: the current one
        for t in tensors:
            t.zero_()


def _scalar_dims(q, k, v, g, beta, cu_seqlens):
    if cu_seqlens is None:  # what is as it should be is found so by one expression, at half the cost
        qs, vs, t, dev = q.shape, v.shape, q.dtype, q.get_device()
        if len(qs) == 4 and len(vs) == 4 and dev >= 0 and t in _DT:
            B, T, Hk, dk = qs
            _, _, Hv, dv = vs
            gs = (B, T, Hv)
            if (k.shape == qs and vs == (B, T, Hv, dv) and g.shape == gs and beta.shape == gs
                    and k.dtype is t and v.dtype is t and g.dtype is t and beta.dtype is t
                    and k.get_device() == dev and v.get_device() == dev and g.get_device() == dev
                    and beta.get_device() == dev and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
                    and g.is_contiguous() and beta.is_contiguous()):
                return B, T, Hk, Hv, dk, dv, B, _DT[t], dev
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q and v must have four dimensions [B,T,H,d]")
    B, T, Hk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    t = q.dtype
    if t not in _DT:
        raise ValueError("unsupported dtype %s" % t)
    dev = _device_of(q, "q")
    _want(q, "q", t, (B, T, Hk, dk), dev)
    _want(k, "k", t, (B, T, Hk, dk), dev)
    _want(v, "v", t, (B, T, Hv, dv), dev)
    _want(g, "g", t, (B, T, Hv), dev)
    _want(beta, "beta", t, (B, T, Hv), dev)
    N = B
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("packed sequences need B = 1, got B = %d" % B)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must have one dimension and at least one entry")
        _want(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, dev)
        N = cu_seqlens.numel() - 1
    return B, T, Hk, Hv, dk, dv, N, _DT[t], dev


def _scalar_workspace(N, T, Hk, Hv, dk, dv, packed, dt, train, device):
    n = gdr2_scalar_workspace_bytes(N, T, Hk, Hv, dk, dv, packed, dt, train)
    if n == 0 and N * T * Hv > 0:
        raise ValueError("unsupported shape/dtype: N=%d T=%d Hk=%d Hv=%d dk=%d dv=%d" % (N, T, Hk, Hv, dk, dv))
    return torch.empty(n, dtype=torch.uint8, device=device)


def gdr2_scalar_fwd(q, k, v, g, beta, h0=None, *, cu_seqlens=None, save_for_bwd=False, ws=None, o=None,
                    output_final_state=True, stream=None):
    """Gated delta rule with scalar gates, chunkwise forward (see include/gdr2.h). q, k: [B,T,Hk,dk];
    v: [B,T,Hv,dv]; g, beta: [B,T,Hv], all of one dtype (bf16 or fp32); Hv a multiple of Hk. h0:
    [N,Hv,dk,dv] fp32 or None. cu_seqlens: None (N = B sequences of T tokens) or int32 [N+1] on the
    device, the bounds of N sequences packed along T with B = 1. Returns (o, ht or None, ws); pass ``ws``
    back to gdr2_scalar_bwd(..., fwd_saved=True) when save_for_bwd is set. Rows of ``o`` that belong to
    no sequence are zero, or left as they were in an ``o`` that is passed in."""
    lib = load_library()
    B, T, Hk, Hv, dk, dv, N, dt, dev = _scalar_dims(q, k, v, g, beta, cu_seqlens)
    if h0 is not None:
        _want(h0, "h0", torch.float32, (N, Hv, dk, dv), dev)
    new = []
    own_o = o is None
    if own_o:
        o = torch.empty(B, T, Hv, dv, dtype=q.dtype, device=q.device)
        new.append(o)
    else:
        _want(o, "o", q.dtype, (B, T, Hv, dv), dev)
    ht = torch.empty(N, Hv, dk, dv, dtype=torch.float32, device=q.device) if output_final_state else None
    new.append(ht)
    if ws is None:
        ws = _scalar_workspace(N, T, Hk, Hv, dk, dv, cu_seqlens is not None, dt, save_for_bwd, q.device)
        new.append(ws)
    else:
        _want(ws, "ws", torch.uint8, ws.shape, dev)
    _keep_for(stream, *new)
    if own_o and N == 0:
        _zero(stream, o)  # no sequence, and no kernel
    st = _launch(lib.gdr2_scalar_fwd, dev, stream, _adr(q), _adr(k), _adr(v), _adr(g), _adr(beta), _adr(h0),
                 _adr(cu_seqlens), _adr(o), _adr(ht), N, T, Hk, Hv, dk, dv, dt, int(own_o), int(bool(save_for_bwd)),
                 _adr(ws), ws.numel())
    _raise(st, "gdr2_scalar_fwd")
    return o, ht, ws


def gdr2_scalar_bwd(q, k, v, g, beta, h0, dout, dht=None, *, cu_seqlens=None, ws=None, fwd_saved=False,
                    need_dh0=True, grads=None, stream=None):
    """Backward of gdr2_scalar_fwd. Returns a dict with dq, dk, dv, dg, dbeta (input dtype) and dh0 (fp32 or
    None). With fwd_saved=True, ``ws`` must be the workspace of a gdr2_scalar_fwd(..., save_for_bwd=True)
    call on the same inputs. ``grads``: a dict of the five token gradients to write into."""
    lib = load_library()
    B, T, Hk, Hv, dk, dv, N, dt, dev = _scalar_dims(q, k, v, g, beta, cu_seqlens)
    _want(dout, "dout", q.dtype, (B, T, Hv, dv), dev)
    for t, n in ((h0, "h0"), (dht, "dht")):
        if t is not None:
            _want(t, n, torch.float32, (N, Hv, dk, dv), dev)
    new = []
    names = (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))
    own = grads is None
    if own:
        grads = {n: torch.empty_like(x) for n, x in names}
        new += list(grads.values())
    else:
        grads = dict(grads)
        for n, x in names:
            if grads.get(n) is None:
                raise ValueError("grads must hold %s" % n)
            _want(grads[n], n, q.dtype, x.shape, dev)
    grads["dh0"] = torch.empty(N, Hv, dk, dv, dtype=torch.float32, device=q.device) if need_dh0 else None
    new.append(grads["dh0"])
    if ws is None:
        if fwd_saved:
            raise ValueError("fwd_saved=True needs the forward's workspace")
        ws = _scalar_workspace(N, T, Hk, Hv, dk, dv, cu_seqlens is not None, dt, True, q.device)
        new.append(ws)
    else:
        _want(ws, "ws", torch.uint8, ws.shape, dev)
    _keep_for(stream, *new)
    if own and N == 0:
        _zero(stream, *(grads[n] for n, _ in names))
    st = _launch(lib.gdr2_scalar_bwd, dev, stream, _adr(q), _adr(k), _adr(v), _adr(g), _adr(beta), _adr(h0),
                 _adr(dout), _adr(dht), _adr(cu_seqlens), _adr(grads["dq"]), _adr(grads["dk"]), _adr(grads["dv"]),
                 _adr(grads["dg"]), _adr(grads["dbeta"]), _adr(grads["dh0"]), N, T, Hk, Hv, dk, dv, dt, int(own),
                 int(bool(fwd_saved)), _adr(ws), ws.numel())
    _raise(st, "gdr2_scalar_bwd")
    return grads


def gdr2_scalar_step(q, k, v, g, beta, state, *, slots=None, o=None, stream=None):
    """Recurrent step (decoding) of the gated delta rule with scalar gates: the T tokens of q, k
    [B,T,Hk,dk], v [B,T,Hv,dv], g, beta [B,T,Hv], one at a time, on states in a pool: ``state``
    [S,Hv,dk,dv] fp32, updated in place. Row b uses state slots[b] (int32 [B] on the device), or b
    without slots. A slot outside the pool marks a padding row (o = 0, no state touched); rows with one
    slot in common are taken in order, as one sequence. Returns o."""
    lib = load_library()
    B, T, Hk, Hv, dk, dv, _, dt, dev = _scalar_dims(q, k, v, g, beta, None)
    if state is None:
        raise ValueError("state is required")
    if state.dim() != 4:
        raise ValueError("state must have four dimensions [S,Hv,dk,dv]")
    S = state.shape[0]
    _want(state, "state", torch.float32, (S, Hv, dk, dv), dev)
    if slots is not None:
        _want(slots, "slots", torch.int32, (B,), dev)
    elif S < B:
        raise ValueError("state holds %d states for %d rows" % (S, B))
    if o is None:
        o = torch.empty_like(v)
        _keep_for(stream, o)
    else:
        _want(o, "o", q.dtype, v.shape, dev)
    st = _launch(lib.gdr2_scalar_step, dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                 beta.data_ptr(), state.data_ptr(), _adr(slots), o.data_ptr(), B, T, Hk, Hv, dk, dv, S, dt)
    _raise(st, "gdr2_scalar_step")
    return o


def _accumulation_streams(leaves):
    """Of each leaf that wants a gradient, what its accumulation node carries. A node lives as long as any
    graph that was built on the leaf, and the engine runs it on the stream of the first."""
    if torch.is_inference_mode_enabled():
        return []  # no graph is built, and there are no nodes to ask for
    return [torch.autograd.graph.get_gradient_edge(t).node.metadata
            for t in leaves if t is not None and t.is_leaf and t.requires_grad]


def _refuse_tangents(*inputs):
    """A call that bypasses autograd.Function, since nothing wants a gradient, would drop the tangents of forward-mode
    differentiation where the function itself refuses them."""
    if any(t is not None and unpack_dual(t).tangent is not None for t in inputs):
        raise NotImplementedError("forward-mode differentiation is not supported: an input carries a tangent")


class GDR2ScalarFunction(torch.autograd.Function):
    """Autograd wrapper: forward saves the chunks' states in the workspace, backward reuses them. Where no
    gradient is wanted (no_grad, or no input that requires one) it is gdr2_scalar_fwd and saves nothing.
    Inputs with tangents (forward-mode differentiation) are refused.

    Forward and backward may be captured into a graph together, but not while an earlier graph of the same
    leaves, built on another stream, is still alive: their gradients would be accumulated on that stream,
    outside the capture. Such a backward is refused where the earlier graph went through this function; a
    graph that other operations built on the leaves, and leaves further back than the inputs, are not seen
    here and are the caller's to drop before a capture."""

    @classmethod
    def apply(cls, q, k, v, g, beta, h0=None, cu_seqlens=None):
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (q, k, v, g, beta, h0)):
            return super().apply(q, k, v, g, beta, h0, cu_seqlens)
        _refuse_tangents(q, k, v, g, beta, h0)
        return gdr2_scalar_fwd(q, k, v, g, beta, h0, cu_seqlens=cu_seqlens)[:2]

    @staticmethod
    def forward(ctx, q, k, v, g, beta, h0=None, cu_seqlens=None):
        here = torch.cuda.current_stream(q.device).cuda_stream
        for m in _accumulation_streams((q, k, v, g, beta, h0)):
            m.setdefault("gdr2_stream", here)
        o, ht, ws = gdr2_scalar_fwd(q, k, v, g, beta, h0, cu_seqlens=cu_seqlens, save_for_bwd=True)
        ctx.save_for_backward(q, k, v, g, beta, h0, cu_seqlens, ws)
        return o, ht

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dht):
        q, k, v, g, beta, h0, cu_seqlens, ws = ctx.saved_tensors
        if torch.cuda.is_current_stream_capturing():
            here = torch.cuda.current_stream(q.device).cuda_stream
            if any(m.get("gdr2_stream", here) != here for m in _accumulation_streams((q, k, v, g, beta, h0))):
                raise RuntimeError("cannot capture this backward: a graph of the same leaves from another stream is "
                                   "still alive (drop its outputs first, or capture gdr2_scalar_bwd)")
        gr = gdr2_scalar_bwd(q, k, v, g, beta, h0, do.contiguous(), None if dht is None else dht.contiguous(),
                             cu_seqlens=cu_seqlens, ws=ws, fwd_saved=True, need_dh0=h0 is not None)
        return gr["dq"], gr["dk"], gr["dv"], gr["dg"], gr["dbeta"], gr["dh0"], None


# ---------------------------------------------------------------- attention over a paged cache


@functools.lru_cache(maxsize=256)
def gdr2_attn_workspace_bytes(B, Hq, Hkv, D, dtype=DTYPE_BF16) -> int:
    return int(load_library().gdr2_attn_workspace_bytes(B, Hq, Hkv, D, dtype))


_Strides = ctypes.c_longlong * 6


@functools.lru_cache(maxsize=64)
def _strides(ks, vs):
    return _Strides(*ks[:3], *vs[:3])


def _cache_strides(k_cache, v_cache, block_table, dtype, D, dev):
    """Checks a cache. Returns its strides, pages, page size and heads."""
    shape, ks, vs = k_cache.shape, k_cache.stride(), v_cache.stride()
    if (len(shape) == 4 and v_cache.shape == shape and shape[3] == D and ks[3] == 1 and vs[3] == 1
            and k_cache.dtype is dtype and v_cache.dtype is dtype and k_cache.get_device() == dev
            and v_cache.get_device() == dev and shape[0] <= 0x7fffffff and shape[1] <= 0x7fffffff
            and block_table.dim() == 2):
        return _strides(ks, vs), shape[0], shape[1], shape[2]
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must have one shape [pages,page_size,Hkv,D], got %s and %s"
                         % (tuple(k_cache.shape), tuple(v_cache.shape)))
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.get_device() != dev:
            raise ValueError("%s must be on the GPU of the other tensors" % n)
        if t.dtype is not dtype:
            raise ValueError("%s must have dtype %s, got %s" % (n, dtype, t.dtype))
        if t.shape[3] != D:
            raise ValueError("%s must have %d channels, got %d" % (n, D, t.shape[3]))
        if t.stride(3) != 1:
            raise ValueError("the channels of %s must be contiguous" % n)
    if block_table.dim() != 2:
        raise ValueError("block_table must have two dimensions [B,max_pages]")
    raise ValueError("k_cache has too many pages or tokens a page")


def gdr2_attn_step(q, k_cache, v_cache, block_table, lengths, *, scale=None, window=0, o=None, lse=None,
                   return_lse=False, ws=None, stream=None):
    """Attention of one new token a sequence over a paged key-value cache (see include/gdr2.h). q:
    [B,Hq,D]; k_cache, v_cache: [pages,page_size,Hkv,D] with any strides but the last; block_table: int32
    [B,max_pages]; lengths: int32 [B], tokens held with the new one. scale: D ** -0.5 unless given;
    window: only the last ``window`` tokens (0: all). Returns o, or (o, lse) with return_lse or an
    ``lse`` tensor (fp32 [B,Hq]). ``ws``: a uint8 workspace of gdr2_attn_workspace_bytes."""
    lib = load_library()
    if q.dim() != 3:
        raise ValueError("q must have three dimensions [B,Hq,D]")
    B, Hq, D = q.shape
    if q.dtype not in _DT:
        raise ValueError("unsupported dtype %s" % q.dtype)
    dt, dev = _DT[q.dtype], _device_of(q, "q")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    strides, pages, page, Hkv = _cache_strides(k_cache, v_cache, block_table, q.dtype, D, dev)
    max_pages = block_table.shape[1]
    _want(block_table, "block_table", torch.int32, (B, max_pages), dev)
    _want(lengths, "lengths", torch.int32, (B,), dev)
    new = []
    if o is None:
        o = torch.empty_like(q)
        new.append(o)
    else:
        _want(o, "o", q.dtype, (B, Hq, D), dev)
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, Hq), dev)
    elif return_lse:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
        new.append(lse)
    if ws is None:
        ws = torch.empty(gdr2_attn_workspace_bytes(B, Hq, Hkv, D, dt), dtype=torch.uint8, device=q.device)
        new.append(ws)
    else:
        _want(ws, "ws", torch.uint8, ws.shape, dev)
    _keep_for(stream, *new)
    st = _launch(lib.gdr2_attn_step, dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), strides,
                 block_table.data_ptr(), lengths.data_ptr(), o.data_ptr(), _adr(lse), B, Hq, Hkv, D, pages, page,
                 max_pages, D ** -0.5 if scale is None else scale, max(-1, min(window, 0x7fffffff)), dt, ws.data_ptr(),
                 ws.numel())
    _raise(st, "gdr2_attn_step")
    return o if lse is None else (o, lse)


def gdr2_kv_append(k, v, k_cache, v_cache, block_table, starts, *, cu_seqlens=None, stream=None):
    """Writes the keys and values of new tokens, k and v [tokens,Hkv,D], into a paged cache (layout as
    gdr2_attn_step) behind the starts[s] tokens (int32 [B]) that each sequence holds. cu_seqlens: int32
    [B+1], the bounds of the sequences' tokens, or None for one token a sequence. Tokens without a place
    in block_table are dropped."""
    lib = load_library()
    if k.dim() != 3:
        raise ValueError("k must have three dimensions [tokens,Hkv,D]")
    tokens, Hkv, D = k.shape
    if k.dtype not in _DT:
        raise ValueError("unsupported dtype %s" % k.dtype)
    dev = _device_of(k, "k")
    if not k.is_contiguous():
        raise ValueError("k must be contiguous")
    _want(v, "v", k.dtype, (tokens, Hkv, D), dev)
    strides, pages, page, heads = _cache_strides(k_cache, v_cache, block_table, k.dtype, D, dev)
    if heads != Hkv:
        raise ValueError("k_cache must have %d heads, got %d" % (Hkv, heads))
    B, max_pages = block_table.shape
    _want(block_table, "block_table", torch.int32, (B, max_pages), dev)
    _want(starts, "starts", torch.int32, (B,), dev)
    if cu_seqlens is not None:
        _want(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,), dev)
    elif tokens != B:
        raise ValueError("without cu_seqlens there is one token a sequence, got %d tokens for %d sequences"
                         % (tokens, B))
    st = _launch(lib.gdr2_kv_append, dev, stream, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                 strides, block_table.data_ptr(), starts.data_ptr(), _adr(cu_seqlens), B, tokens, Hkv, D, pages, page,
                 max_pages, _DT[k.dtype])
    _raise(st, "gdr2_kv_append")


def gdr2_attn_tree(q, parents, k_cache, v_cache, block_table, starts, *, scale=None, window=0, o=None, lse=None,
                   return_lse=False, ws=None, stream=None):
    """Attention of a tree of drafted tokens over a paged key-value cache (see include/gdr2.h). q: [B,T,Hq,D],
    T at most 64; parents: int32 [B,T], the draft that each one continues, -1 where it continues the
    sequence itself (any other value: padding); cache and block_table as gdr2_attn_step; starts: int32 [B],
    tokens held before the drafts, which stand in the cache behind them (gdr2_kv_append with the same
    starts). Returns o, or (o, lse) with return_lse or an ``lse`` tensor (fp32 [B,T,Hq]). ``ws``: a uint8
    workspace of gdr2_attn_tree_workspace_bytes."""
    lib = load_library()
    if q.dim() != 4:
        raise ValueError("q must have four dimensions [B,T,Hq,D]")
    B, T, Hq, D = q.shape
    if q.dtype not in _DT:
        raise ValueError("unsupported dtype %s" % q.dtype)
    dt, dev = _DT[q.dtype], _device_of(q, "q")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous")
    strides, pages, page, Hkv = _cache_strides(k_cache, v_cache, block_table, q.dtype, D, dev)
    max_pages = block_table.shape[1]
    _want(parents, "parents", torch.int32, (B, T), dev)
    _want(block_table, "block_table", torch.int32, (B, max_pages), dev)
    _want(starts, "starts", torch.int32, (B,), dev)
    new = []
    if o is None:
        o = torch.empty_like(q)
        new.append(o)
    else:
        _want(o, "o", q.dtype, (B, T, Hq, D), dev)
    if lse is not None:
        _want(lse, "lse", torch.float32, (B, T, Hq), dev)
    elif return_lse:
        lse = torch.empty(B, T, Hq, dtype=torch.float32, device=q.device)
        new.append(lse)
    if ws is None:
        ws = torch.empty(gdr2_attn_tree_workspace_bytes(B, T, Hq, Hkv, D, dt), dtype=torch.uint8, device=q.device)
        new.append(ws)
    else:
        _want(ws, "ws", torch.uint8, ws.shape, dev)
    _keep_for(stream, *new)
    st = _launch(lib.gdr2_attn_tree, dev, stream, q.data_ptr(), parents.data_ptr(), k_cache.data_ptr(),
                 v_cache.data_ptr(), strides, block_table.data_ptr(), starts.data_ptr(), o.data_ptr(), _adr(lse), B, T,
                 Hq, Hkv, D, pages, page, max_pages, D ** -0.5 if scale is None else scale,
                 max(-1, min(window, 0x7fffffff)), dt, ws.data_ptr(), ws.numel())
    _raise(st, "gdr2_attn_tree")
    return o if lse is None else (o, lse)


def gdr2_kv_keep(k_cache, v_cache, block_table, starts, path, *, lengths=None, stream=None):
    """Keeps an accepted path of a tree of drafts: of each sequence the token at starts[b] + path[b][j] of
    the cache goes to starts[b] + j, for the entries of path (int32 [B,P], P at most 64) before its first
    negative one. Returns the tokens that each sequence then holds (int32 [B], in ``lengths`` if given)."""
    lib = load_library()
    if path.dim() != 2:
        raise ValueError("path must have two dimensions [B,P]")
    if k_cache.dim() != 4:
        raise ValueError("k_cache must have four dimensions [pages,page_size,Hkv,D]")
    if k_cache.dtype not in _DT:
        raise ValueError("unsupported dtype %s" % k_cache.dtype)
    dev, D = _device_of(k_cache, "k_cache"), k_cache.shape[3]
    strides, pages, page, Hkv = _cache_strides(k_cache, v_cache, block_table, k_cache.dtype, D, dev)
    B, max_pages = block_table.shape
    P = path.shape[1]
    _want(block_table, "block_table", torch.int32, (B, max_pages), dev)
    _want(starts, "starts", torch.int32, (B,), dev)
    _want(path, "path", torch.int32, (B, P), dev)
    if lengths is None:
        lengths = torch.empty_like(starts)
        _keep_for(stream, lengths)
    else:
        _want(lengths, "lengths", torch.int32, (B,), dev)
    st = _launch(lib.gdr2_kv_keep, dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), strides, block_table.data_ptr(),
                 starts.data_ptr(), path.data_ptr(), lengths.data_ptr(), B, P, Hkv, D, pages, page, max_pages,
                 _DT[k_cache.dtype])
    _raise(st, "gdr2_kv_keep")
    return lengths


def gdr2_kv_pages(lengths, counts, block_table, free_pages, num_free, *, page_size, max_tokens, new_lengths=None,
                  cu_seqlens=None, slots=None, stream=None):
    """Pages for the tokens to come (see include/gdr2.h). lengths, counts: int32 [B], the tokens that each
    request holds and how many come to it, negative where it ends; block_table: int32 [B,max_pages],
    free_pages: int32 [pages], a stack of which the first num_free (int32 [1]) entries are free: all three
    are updated. Returns (new_lengths int32 [B], cu_seqlens int32 [B+1], slots int64 [max_tokens]), in the
    tensors passed in if there are any."""
    lib = load_library()
    if block_table.dim() != 2:
        raise ValueError("block_table must have two dimensions [B,max_pages]")
    if free_pages.dim() != 1:
        raise ValueError("free_pages must have one dimension")
    B, max_pages = block_table.shape
    pages, i32, dev = free_pages.shape[0], torch.int32, _device_of(block_table, "block_table")
    if not (max_pages <= 0x7fffffff and pages <= 0x7fffffff and 0 <= max_tokens <= 0x7fffffff):
        raise ValueError("block_table, free_pages or max_tokens out of range")
    _want(lengths, "lengths", i32, (B,), dev)
    _want(counts, "counts", i32, (B,), dev)
    _want(block_table, "block_table", i32, (B, max_pages), dev)
    _want(free_pages, "free_pages", i32, (pages,), dev)
    _want(num_free, "num_free", i32, (1,), dev)
    new = []
    if new_lengths is None:
        new_lengths = torch.empty_like(lengths)
        new.append(new_lengths)
    else:
        _want(new_lengths, "new_lengths", i32, (B,), dev)
    if cu_seqlens is None:
        cu_seqlens = torch.empty(B + 1, dtype=i32, device=lengths.device)
        new.append(cu_seqlens)
    else:
        _want(cu_seqlens, "cu_seqlens", i32, (B + 1,), dev)
    if slots is None:
        slots = torch.empty(max_tokens, dtype=torch.int64, device=lengths.device)
        new.append(slots)
    else:
        _want(slots, "slots", torch.int64, (max_tokens,), dev)
    _keep_for(stream, *new)
    st = _launch(lib.gdr2_kv_pages, dev, stream, lengths.data_ptr(), counts.data_ptr(), block_table.data_ptr(),
                 free_pages.data_ptr(), num_free.data_ptr(), new_lengths.data_ptr(), cu_seqlens.data_ptr(),
                 slots.data_ptr(), B, max_tokens, pages, max(-1, min(page_size, 0x7fffffff)), max_pages)
    _raise(st, "gdr2_kv_pages")
    return new_lengths, cu_seqlens, slots


@functools.lru_cache(maxsize=256)
def gdr2_attn_tree_workspace_bytes(B, T, Hq, Hkv, D, dtype=DTYPE_BF16) -> int:
    return int(load_library().gdr2_attn_tree_workspace_bytes(B, T, Hq, Hkv, D, dtype))


# ---------------------------------------------------------------- attention over whole sequences


@functools.lru_cache(maxsize=256)
def gdr2_attn_bwd_workspace_bytes(N, T, Hq, Hkv, D, packed=False, dtype=DTYPE_BF16) -> int:
    return int(load_library().gdr2_attn_bwd_workspace_bytes(N, T, Hq, Hkv, D, int(bool(packed)), dtype))


def _attn_input(t, name, dtype, shape, dev):
    """Checks q, k or v of [B,T,H,D], which may be a part of a larger tensor's rows. Returns its token and head
    strides."""
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError("%s must be on the GPU of the other tensors" % name)
    if t.dtype is not dtype:
        raise ValueError("%s must have dtype %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    B, T, H, D = shape
    sb, st, sh, sd = t.stride()
    if t.is_contiguous():
        return H * D, D
    if T == 1:
        st = sb  # (the stride over tokens says nothing then)
    if sd != 1 or (B > 1 and T > 0 and sb != T * st):
        raise ValueError("the channels of %s must be contiguous, and its sequences T token strides apart" % name)
    return st, sh


def _like(x, contiguous):
    """A contiguous tensor of x's shape (empty_like is the quicker call, and keeps the strides of a dense x)."""
    return torch.empty_like(x) if contiguous else torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _attn_dims(q, k, v, cu_seqlens):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k and v must have four dimensions [B,T,H,D]")
    if q.dtype not in _DT:
        raise ValueError("unsupported dtype %s" % q.dtype)
    B, T, Hq, D = q.shape
    Hkv, dev, t = k.shape[2], _device_of(q, "q"), q.dtype
    strides = None
    if not (k.shape == v.shape == (B, T, Hkv, D) and k.dtype is t and v.dtype is t and k.get_device() == dev
            and v.get_device() == dev and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        qs, ks, vs = (_attn_input(x, n, t, (B, T, h, D), dev) for x, n, h in ((q, "q", Hq), (k, "k", Hkv), (v, "v", Hkv)))
        strides = _strides((*qs, ks[0]), (ks[1], *vs))
    N = B
    if cu_seqlens is not None:
        if B != 1:
            raise ValueError("packed sequences need B = 1, got B = %d" % B)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must have one dimension and at least one entry")
        _want(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, dev)
        N = cu_seqlens.numel() - 1
    return N, T, Hq, Hkv, D, _DT[t], dev, strides


def gdr2_attn_fwd(q, k, v, *, cu_seqlens=None, scale=None, window=0, o=None, lse=None, return_lse=False,
                  save_for_bwd=False, stream=None):
    """Causal attention over whole sequences (see include/gdr2.h). q: [B,T,Hq,D]; k, v: [B,T,Hkv,D], one dtype (bf16
    or fp32); they may be parts of the rows of a larger tensor. cu_seqlens: None (B sequences of T tokens) or
    int32 [N+1] on the device, the bounds of N sequences packed along T with B = 1. scale: D ** -0.5 unless
    given; window: only the last ``window`` tokens (0: all). Returns o, or (o, lse) with return_lse or an
    ``lse`` tensor (fp32 [B,T,Hq]), or with save_for_bwd (o, lse, rest) for gdr2_attn_bwd, rest (bf16; None
    for fp32) being what o's rounding left over. Rows of no sequence are zero (of lse and rest too), or, where an
    ``o`` is passed in, left as they were in each."""
    lib = load_library()
    N, T, Hq, Hkv, D, dt, dev, strides = _attn_dims(q, k, v, cu_seqlens)
    new, own_o, rest = [], o is None, None
    if own_o:
        o = _like(q, strides is None)
        new.append(o)
    else:
        _want(o, "o", q.dtype, q.shape, dev)
    if lse is not None:
        _want(lse, "lse", torch.float32, q.shape[:3], dev)
    elif return_lse or save_for_bwd:
        lse = torch.empty(q.shape[0], T, Hq, dtype=torch.float32, device=q.device)
        new.append(lse)
    if save_for_bwd and dt == DTYPE_BF16:
        rest = torch.empty_like(o)
        new.append(rest)
    _keep_for(stream, *new)
    if own_o and N == 0:
        _zero(stream, *(x for x in (o, lse, rest) if x is not None))  # no sequence, and no kernel
    st = _launch(lib.gdr2_attn_fwd, dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, _adr(cu_seqlens),
                 o.data_ptr(), _adr(lse), _adr(rest), N, T, Hq, Hkv, D, D ** -0.5 if scale is None else scale,
                 max(-1, min(window, 0x7fffffff)), dt, int(own_o))
    _raise(st, "gdr2_attn_fwd")
    return (o, lse, rest) if save_for_bwd else o if lse is None else (o, lse)


def gdr2_attn_bwd(q, k, v, o, lse, dout, *, rest=None, cu_seqlens=None, scale=None, window=0, grads=None, ws=None,
                  stream=None):
    """Backward of gdr2_attn_fwd, with its o, lse and (bf16) rest for the same arguments. Returns a dict with dq, dk
    and dv (contiguous), written into ``grads`` if given. ``ws``: a uint8 workspace of
    gdr2_attn_bwd_workspace_bytes."""
    lib = load_library()
    N, T, Hq, Hkv, D, dt, dev, strides = _attn_dims(q, k, v, cu_seqlens)
    _want(o, "o", q.dtype, q.shape, dev)
    _want(lse, "lse", torch.float32, q.shape[:3], dev)
    _want(dout, "dout", q.dtype, q.shape, dev)
    if rest is not None:
        _want(rest, "rest", q.dtype, q.shape, dev)
    new, own = [], grads is None
    if own:
        grads = {n: _like(x, strides is None) for n, x in (("dq", q), ("dk", k), ("dv", v))}
        new += list(grads.values())
    else:
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            if grads.get(n) is None:
                raise ValueError("grads must hold %s" % n)
            _want(grads[n], n, q.dtype, x.shape, dev)
    if ws is None:
        n = gdr2_attn_bwd_workspace_bytes(N, T, Hq, Hkv, D, cu_seqlens is not None, dt)
        ws = torch.empty(n, dtype=torch.uint8, device=q.device)
        new.append(ws)
    else:
        _want(ws, "ws", torch.uint8, ws.shape, dev)
    _keep_for(stream, *new)
    if own and N == 0:
        _zero(stream, *grads.values())
    st = _launch(lib.gdr2_attn_bwd, dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, o.data_ptr(),
                 lse.data_ptr(), _adr(rest), dout.data_ptr(), _adr(cu_seqlens), grads["dq"].data_ptr(),
                 grads["dk"].data_ptr(), grads["dv"].data_ptr(), N, T, Hq, Hkv, D, D ** -0.5 if scale is None else scale,
                 max(-1, min(window, 0x7fffffff)), dt, int(own), ws.data_ptr(), ws.numel())
    _raise(st, "gdr2_attn_bwd")
    return grads


class GDR2AttnFunction(torch.autograd.Function):
    """Autograd wrapper of gdr2_attn_fwd and gdr2_attn_bwd; apply(q, k, v, cu_seqlens, scale, window) returns o. Where no
    gradient is wanted it is gdr2_attn_fwd and saves nothing. Tangents, and capturing forward and backward into a graph:
    as GDR2ScalarFunction."""

    @classmethod
    def apply(cls, q, k, v, cu_seqlens=None, scale=None, window=0):
        if torch.is_grad_enabled() and any(t.requires_grad for t in (q, k, v)):
            return super().apply(q, k, v, cu_seqlens, scale, window)
        _refuse_tangents(q, k, v)
        return gdr2_attn_fwd(q, k, v, cu_seqlens=cu_seqlens, scale=scale, window=window)

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens=None, scale=None, window=0):
        here = torch.cuda.current_stream(q.device).cuda_stream
        for m in _accumulation_streams((q, k, v)):
            m.setdefault("gdr2_stream", here)
        o, lse, rest = gdr2_attn_fwd(q, k, v, cu_seqlens=cu_seqlens, scale=scale, window=window, save_for_bwd=True)
        ctx.save_for_backward(q, k, v, o, lse, rest, cu_seqlens)
        ctx.scale, ctx.window = scale, window
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, rest, cu_seqlens = ctx.saved_tensors
        if torch.cuda.is_current_stream_capturing():
            here = torch.cuda.current_stream(q.device).cuda_stream
            if any(m.get("gdr2_stream", here) != here for m in _accumulation_streams((q, k, v))):
                raise RuntimeError("cannot capture this backward: a graph of the same leaves from another stream is "
                                   "still alive (drop its outputs first, or capture gdr2_attn_bwd)")
        gr = gdr2_attn_bwd(q, k, v, o, lse, do.contiguous(), rest=rest, cu_seqlens=cu_seqlens, scale=ctx.scale,
                           window=ctx.window)
        return gr["dq"], gr["dk"], gr["dv"], None, None, None
