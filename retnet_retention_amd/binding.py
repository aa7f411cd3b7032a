"""ctypes binding of libretention.so: torch tensors in, C-ABI calls out.

This layer only marshals arguments (shapes, dtypes, device pointers and the
current HIP stream); every step of the computation runs in the library's
kernels. It raises when the library has not been built: there is no fallback.
"""

import contextlib
import ctypes
import functools
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libretention.so")

RET_F32 = 0
RET_BF16 = 1

STATUS = {
    0: "RET_OK",
    1: "RET_ERR_NULL",
    2: "RET_ERR_SHAPE",
    3: "RET_ERR_UNSUPPORTED",
    4: "RET_ERR_GAMMA",
    5: "RET_ERR_ALIGN",
    6: "RET_ERR_WORKSPACE",
    7: "RET_ERR_HIP",
    8: "RET_ERR_ALIAS",
    9: "RET_ERR_ARG",
    10: "RET_ERR_SCRATCH",
}

# names declared in include/retention.h
EXPORTS = (
    "retention_parallel_workspace_bytes",
    "retention_parallel_fwd",
    "retention_chunkwise_workspace_bytes",
    "retention_chunkwise_fwd",
    "retention_chunkwise_fwd_timed",
    "retention_chunkwise_fwd_noalloc",
    "retention_chunkwise_varlen_workspace_bytes",
    "retention_chunkwise_varlen_fwd",
    "retention_recurrent_step",
    "retention_recurrent_step_positions",
    "retention_parallel_bwd_workspace_bytes",
    "retention_parallel_bwd",
    "retention_chunkwise_bwd_workspace_bytes",
    "retention_chunkwise_bwd",
    "retention_chunkwise_bwd_state_workspace_bytes",
    "retention_chunkwise_bwd_state",
    "retention_score_map_workspace_bytes",
    "retention_score_map",
    "retention_chunkwise_error",
    "retention_delta_workspace_bytes",
    "retention_delta_fwd",
    "retention_delta_bwd_workspace_bytes",
    "retention_delta_bwd",
    "retention_delta_step",
    "retention_head_norm_fwd",
    "retention_head_norm_bwd_workspace_bytes",
    "retention_head_norm_bwd",
    "retention_residual_norm_fwd",
    "retention_residual_norm_bwd_workspace_bytes",
    "retention_residual_norm_bwd",
    "retention_status_string",
    "retention_abi_version",
)


class RetDesc(ctypes.Structure):
    """Mirror of ret_desc_t."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("seqlen", ctypes.c_int32),
        ("heads", ctypes.c_int32),
        ("dk", ctypes.c_int32),
        ("dv", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("gamma", ctypes.POINTER(ctypes.c_double)),
        ("rotary_base", ctypes.c_double),
        ("pos_offset", ctypes.c_int64),
        ("gn_eps", ctypes.c_float),
    ]


class DeltaDesc(ctypes.Structure):
    """Mirror of ret_delta_desc_t."""

    _fields_ = [
        ("batch", ctypes.c_int32),
        ("seqlen", ctypes.c_int32),
        ("k_heads", ctypes.c_int32),
        ("v_heads", ctypes.c_int32),
        ("dk", ctypes.c_int32),
        ("dv", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class NormDesc(ctypes.Structure):
    """Mirror of ret_norm_desc_t."""

    _fields_ = [
        ("rows", ctypes.c_int64),
        ("width", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("center", ctypes.c_int32),
        ("eps", ctypes.c_float),
    ]


class RetentionError(RuntimeError):
    """A call's status was not RET_OK, or a chunkwise call's control word
    reported an error (status "control", word in .word)."""

    def __init__(self, status, text, word=0):
        super().__init__(f"{STATUS.get(status, status)}: {text}")
        self.status = status
        self.word = word


_lib = None


def lib():
    """The loaded library (loads it on first use; raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                f"{LIB_PATH} is missing: build it first (python -m retnet_retention_amd.build); "
                "there is no fallback implementation"
            )
        h = ctypes.CDLL(LIB_PATH)
        vp, sz, st, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int32
        pd = ctypes.POINTER(RetDesc)
        h.retention_parallel_workspace_bytes.argtypes = [pd]
        h.retention_parallel_workspace_bytes.restype = sz
        h.retention_parallel_fwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, sz, vp]
        h.retention_parallel_fwd.restype = st
        h.retention_chunkwise_workspace_bytes.argtypes = [pd, i32]
        h.retention_chunkwise_workspace_bytes.restype = sz
        h.retention_chunkwise_fwd.argtypes = [pd, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        h.retention_chunkwise_fwd.restype = st
        h.retention_chunkwise_fwd_timed.argtypes = [pd, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp]
        h.retention_chunkwise_fwd_timed.restype = st
        h.retention_chunkwise_fwd_noalloc.argtypes = [pd, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        h.retention_chunkwise_fwd_noalloc.restype = st
        h.retention_chunkwise_varlen_workspace_bytes.argtypes = [pd, i32]
        h.retention_chunkwise_varlen_workspace_bytes.restype = sz
        h.retention_chunkwise_varlen_fwd.argtypes = [pd, i32, vp, ctypes.c_int64] + [vp] * 8 + [sz, vp]
        h.retention_chunkwise_varlen_fwd.restype = st
        h.retention_recurrent_step.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp]
        h.retention_recurrent_step.restype = st
        h.retention_recurrent_step_positions.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp]
        h.retention_recurrent_step_positions.restype = st
        h.retention_parallel_bwd_workspace_bytes.argtypes = [pd, i32]
        h.retention_parallel_bwd_workspace_bytes.restype = sz
        h.retention_parallel_bwd.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        h.retention_parallel_bwd.restype = st
        h.retention_chunkwise_bwd_workspace_bytes.argtypes = [pd, i32, i32]
        h.retention_chunkwise_bwd_workspace_bytes.restype = sz
        h.retention_chunkwise_bwd.argtypes = [pd, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        h.retention_chunkwise_bwd.restype = st
        h.retention_chunkwise_bwd_state_workspace_bytes.argtypes = [pd, i32, i32]
        h.retention_chunkwise_bwd_state_workspace_bytes.restype = sz
        h.retention_chunkwise_bwd_state.argtypes = [pd, i32] + [vp] * 13 + [sz, vp]
        h.retention_chunkwise_bwd_state.restype = st
        h.retention_score_map_workspace_bytes.argtypes = [pd]
        h.retention_score_map_workspace_bytes.restype = sz
        h.retention_score_map.argtypes = [pd, vp, vp, i32, vp, vp, sz, vp]
        h.retention_score_map.restype = st
        h.retention_chunkwise_error.argtypes = [vp, sz, ctypes.POINTER(i32), vp]
        h.retention_chunkwise_error.restype = st
        pdd, i64 = ctypes.POINTER(DeltaDesc), ctypes.c_int64
        h.retention_delta_workspace_bytes.argtypes = [pdd, i32, i64]
        h.retention_delta_workspace_bytes.restype = sz
        h.retention_delta_fwd.argtypes = [pdd, vp, i64] + [vp] * 9 + [sz, vp]
        h.retention_delta_fwd.restype = st
        h.retention_delta_bwd_workspace_bytes.argtypes = [pdd, i32, i64]
        h.retention_delta_bwd_workspace_bytes.restype = sz
        h.retention_delta_bwd.argtypes = [pdd, vp, i64] + [vp] * 15 + [sz, vp]
        h.retention_delta_bwd.restype = st
        h.retention_delta_step.argtypes = [pdd] + [vp] * 8 + [i64, vp]
        h.retention_delta_step.restype = st
        pnd, f32 = ctypes.POINTER(NormDesc), ctypes.c_float
        h.retention_head_norm_fwd.argtypes = [pnd] + [vp] * 5
        h.retention_head_norm_fwd.restype = st
        h.retention_head_norm_bwd_workspace_bytes.argtypes = [pnd]
        h.retention_head_norm_bwd_workspace_bytes.restype = sz
        h.retention_head_norm_bwd.argtypes = [pnd] + [vp] * 8 + [sz, vp]
        h.retention_head_norm_bwd.restype = st
        h.retention_residual_norm_fwd.argtypes = [pnd, f32] + [vp] * 8
        h.retention_residual_norm_fwd.restype = st
        h.retention_residual_norm_bwd_workspace_bytes.argtypes = [pnd]
        h.retention_residual_norm_bwd_workspace_bytes.restype = sz
        h.retention_residual_norm_bwd.argtypes = [pnd, f32] + [vp] * 13 + [sz, vp]
        h.retention_residual_norm_bwd.restype = st
        h.retention_status_string.argtypes = [st]
        h.retention_status_string.restype = ctypes.c_char_p
        h.retention_abi_version.argtypes = []
        h.retention_abi_version.restype = i32
        _lib = h
    return _lib


def _check(status):
    if status != 0:
        raise RetentionError(status, lib().retention_status_string(status).decode())


def make_desc(batch, seqlen, heads, dk, dv, dtype, gammas=None, rotary_base=0.0, pos_offset=0, eps=1e-5):
    """Build a RetDesc; returns (desc, keepalive) -- keep the second alive
    while the descriptor is in use (it owns the gamma array)."""
    gam = None
    if gammas is not None:
        gam = (ctypes.c_double * heads)(*[float(x) for x in gammas])
    d = RetDesc(batch, seqlen, heads, dk, dv, dtype,
                ctypes.cast(gam, ctypes.POINTER(ctypes.c_double)) if gam is not None else None,
                float(rotary_base), int(pos_offset), float(eps))
    return d, gam


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return RET_BF16
    if t.dtype == torch.float32:
        return RET_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on_device(name, t, like):
    """t (may be None) must be a GPU tensor on the device of `like`: its
    pointer goes to the kernels as a device address."""
    if t is not None and (not t.is_cuda or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must be a GPU tensor on {like.device}")


def _workspace(ws, need, like):
    """The caller's workspace (checked), or a new one; returns (workspace,
    bytes, whether it is the binding's own)."""
    if ws is None:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=like.device)
        return ws, ws.numel(), True
    _on_device("workspace", ws, like)
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ws, ws.numel() * ws.element_size(), False


_CTRL_BITS = {1: "a wait between the chunk-to-chunk state workgroups gave up after its bound",
              2: "packed-sequence bounds (cu_seqlens) had to be clamped"}


def chunkwise_error(workspace):
    """Control word 1 of a chunkwise call's workspace (synchronizes the
    current stream first): 0 when the call that used it completed without an
    error, else bit 0 (1) a wait that gave up, bit 1 (2) clamped packed
    bounds; the outputs are then not valid."""
    stream = _stream(workspace)
    word = ctypes.c_int32(0)
    _check(lib().retention_chunkwise_error(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                           ctypes.byref(word), stream))
    return int(word.value)


def check_chunkwise(workspace):
    """Raise RetentionError when the chunkwise call that used `workspace`
    reported an error in its control word (synchronizes)."""
    w = chunkwise_error(workspace)
    if w:
        why = "; ".join(t for b, t in _CTRL_BITS.items() if w & b) or "unknown bits"
        raise RetentionError("control", f"chunkwise control word 1 = {w} ({why}); the outputs are not valid", w)


# The stream's handle without a Stream object around it (a microsecond of a
# decode call), where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream(t):
    """The current stream of a GPU tensor's device. A CPU tensor is refused: its
    device number, -1, would mean the current device."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("the call takes GPU tensors")
    return _raw_stream(dev)


def _validate(q, k, v, g, out):
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("out", out)):
        if t is None:
            continue
        if not t.is_cuda or t.device != q.device:
            raise ValueError(f"{name} must be a GPU tensor on q's device")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.dtype != q.dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {q.dtype}")
        if t.dim() != 4:
            raise ValueError(f"{name} must be [batch, seqlen, heads, d]")
    if k.shape != q.shape:
        raise ValueError("k must have the shape of q")
    if v.shape[:3] != q.shape[:3]:
        raise ValueError("v must agree with q on [batch, seqlen, heads]")
    for name, t in (("g", g), ("out", out)):
        if t is not None and t.shape != v.shape:
            raise ValueError(f"{name} must have the shape of v")


def _desc_for(q, v, gammas, rotary_base, pos_offset, eps):
    b, n, h, dk = q.shape
    return make_desc(b, n, h, dk, v.shape[-1], _dtype_code(q), gammas, rotary_base, pos_offset, eps)


def parallel_fwd(q, k, v, g=None, *, gammas=None, rotary_base=0.0, pos_offset=0, eps=1e-5, out=None,
                 workspace=None):
    """Parallel form over whole sequences; returns the output tensor."""
    out = torch.empty_like(v) if out is None else out
    _validate(q, k, v, g, out)
    desc, keep = _desc_for(q, v, gammas, rotary_base, pos_offset, eps)
    L = lib()
    need = L.retention_parallel_workspace_bytes(ctypes.byref(desc))
    ws_bytes = 0
    if need or workspace is not None:
        workspace, ws_bytes, _ = _workspace(workspace, need, q)
    _check(L.retention_parallel_fwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(out),
                                    _ptr(workspace), ws_bytes, _stream(q)))
    del keep
    return out


def parallel_bwd(q, k, v, dout, g=None, *, gammas=None, rotary_base=0.0, pos_offset=0, eps=1e-5, workspace=None):
    """Gradients of sum(dout * parallel_fwd(q, k, v, g, ...)) with respect to
    q, k, v and g; returns (dq, dk, dv, dg), dg None without a gate."""
    _validate(q, k, v, g, dout)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty_like(g) if g is not None else None
    desc, keep = _desc_for(q, v, gammas, rotary_base, pos_offset, eps)
    L = lib()
    need = L.retention_parallel_bwd_workspace_bytes(ctypes.byref(desc), int(g is not None))
    workspace, ws_bytes, _ = _workspace(workspace, need, q)
    _check(L.retention_parallel_bwd(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(dout), _ptr(dq),
                                    _ptr(dk), _ptr(dv), _ptr(dg), _ptr(workspace), ws_bytes, _stream(q)))
    del keep
    return dq, dk, dv, dg


def chunkwise_bwd(q, k, v, dout, g=None, *, chunk=512, state_in=None, d_state_out=None, gammas=None,
                  rotary_base=0.0, pos_offset=0, eps=1e-5, workspace=None, check=None):
    """Gradients of sum(dout * out) (+ sum(d_state_out * state_out)) with
    out, state_out = chunkwise_fwd(q, k, v, g, chunk=chunk, state_in=state_in,
    ...), with respect to q, k, v, g and state_in. Returns (dq, dk, dv, dg)
    without a carried state, (dq, dk, dv, dg, d_state_in) with one; dg is
    None without a gate. check: as chunkwise_fwd (the control word covers
    all of the call's chunkwise launches)."""
    _validate(q, k, v, g, dout)
    if state_in is not None or d_state_out is not None:
        return _chunkwise_bwd_state(q, k, v, dout, g, chunk, state_in, d_state_out, gammas, rotary_base,
                                    pos_offset, eps, workspace, check)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty_like(g) if g is not None else None
    desc, keep = _desc_for(q, v, gammas, rotary_base, pos_offset, eps)
    L = lib()
    need = L.retention_chunkwise_bwd_workspace_bytes(ctypes.byref(desc), int(chunk), int(g is not None))
    workspace, ws_bytes, own = _workspace(workspace, need, q)
    _check(L.retention_chunkwise_bwd(ctypes.byref(desc), int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(dout),
                                     _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(workspace), ws_bytes, _stream(q)))
    del keep
    if check or (check is None and own):
        check_chunkwise(workspace)
    return dq, dk, dv, dg


def score_map(q, k, *, query=-1, gammas=None, rotary_base=0.0, pos_offset=0, workspace=None):
    """Retention score map of query token `query` (-1: the last) over the
    tokens before it, summed over heads; returns fp32 [batch, seqlen]."""
    _validate(q, k, k, None, k)
    out = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
    desc, keep = _desc_for(q, k, gammas, rotary_base, pos_offset, 1e-5)
    L = lib()
    need = L.retention_score_map_workspace_bytes(ctypes.byref(desc))
    ws_bytes = 0
    if need or workspace is not None:
        workspace, ws_bytes, _ = _workspace(workspace, need, q)
    _check(L.retention_score_map(ctypes.byref(desc), _ptr(q), _ptr(k), int(query), _ptr(out), _ptr(workspace),
                                 ws_bytes, _stream(q)))
    del keep
    return out


def _chunkwise_bwd_state(q, k, v, dout, g, chunk, state_in, d_state_out, gammas, rotary_base, pos_offset, eps,
                         workspace, check):
    b, _, h, dk = q.shape
    for name, t in (("state_in", state_in), ("d_state_out", d_state_out)):
        _on_device(name, t, q)
        if t is not None and (t.dtype != torch.float32 or not t.is_contiguous()
                              or tuple(t.shape) != (b, h, dk, v.shape[-1])):
            raise ValueError(f"{name} must be a contiguous fp32 [batch, heads, dk, dv] tensor")
    dq, dk_, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty_like(g) if g is not None else None
    ds0 = torch.empty_like(state_in) if state_in is not None else None
    desc, keep = _desc_for(q, v, gammas, rotary_base, pos_offset, eps)
    L = lib()
    need = L.retention_chunkwise_bwd_state_workspace_bytes(ctypes.byref(desc), int(chunk), int(g is not None))
    workspace, ws_bytes, own = _workspace(workspace, need, q)
    _check(L.retention_chunkwise_bwd_state(ctypes.byref(desc), int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                           _ptr(dout), _ptr(state_in), _ptr(d_state_out), _ptr(dq), _ptr(dk_),
                                           _ptr(dv), _ptr(dg), _ptr(ds0), _ptr(workspace), ws_bytes, _stream(q)))
    del keep
    if check or (check is None and own):
        check_chunkwise(workspace)
    return (dq, dk_, dv, dg) if state_in is None else (dq, dk_, dv, dg, ds0)


def chunkwise_workspace_bytes(q, v, chunk, rotary_base=0.0):
    desc, keep = _desc_for(q, v, None, rotary_base, 0, 1e-5)
    return lib().retention_chunkwise_workspace_bytes(ctypes.byref(desc), int(chunk))


def chunkwise_fwd(q, k, v, g=None, *, chunk=512, state_in=None, state_out=None, gammas=None, rotary_base=0.0,
                  pos_offset=0, eps=1e-5, out=None, workspace=None, kernel_events=None, check=None):
    """Chunkwise form; returns the output tensor (state_out, if given, is
    filled with the state after the last token). kernel_events: optional pair
    of torch.cuda.Event (timing enabled) recorded around the chunkwise kernel
    alone. check: synchronize and raise RetentionError if the call's control
    word reports an error; None checks only when the binding allocated the
    workspace (a caller's workspace can be checked later with
    check_chunkwise)."""
    out = torch.empty_like(v) if out is None else out
    _validate(q, k, v, g, out)
    for name, s in (("state_in", state_in), ("state_out", state_out)):
        if s is not None:
            b, _, h, dk = q.shape
            _on_device(name, s, q)
            if s.dtype != torch.float32 or not s.is_contiguous() or tuple(s.shape) != (b, h, dk, v.shape[-1]):
                raise ValueError(f"{name} must be a contiguous fp32 [batch, heads, dk, dv] tensor")
    desc, keep = _desc_for(q, v, gammas, rotary_base, pos_offset, eps)
    L = lib()
    need = L.retention_chunkwise_workspace_bytes(ctypes.byref(desc), int(chunk))
    workspace, ws_bytes, own = _workspace(workspace, need, q)
    if kernel_events is None:
        _check(L.retention_chunkwise_fwd(ctypes.byref(desc), int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                         _ptr(out), _ptr(state_in), _ptr(state_out), _ptr(workspace), ws_bytes,
                                         _stream(q)))
    else:
        before, after = (ctypes.c_void_p(e.cuda_event) for e in kernel_events)
        _check(L.retention_chunkwise_fwd_timed(ctypes.byref(desc), int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                               _ptr(out), _ptr(state_in), _ptr(state_out), _ptr(workspace),
                                               ws_bytes, _stream(q), before, after))
    del keep
    if check or (check is None and own):
        check_chunkwise(workspace)
    return out


def chunkwise_fwd_noalloc(q, k, v, g=None, *, chunk=512, state_in=None, state_out=None, gammas=None,
                          rotary_base=0.0, pos_offset=0, eps=1e-5, out=None, error_word=None):
    """The chunkwise form through the entry point that allocates nothing: the
    library's static scratch replaces the workspace (calls on one device must
    not overlap in time). `out` must be given (nothing is allocated here
    either); error_word: optional GPU int32 tensor [1] that receives the
    call's control word 1 in stream order."""
    if out is None:
        raise ValueError("chunkwise_fwd_noalloc allocates nothing: pass `out`")
    _validate(q, k, v, g, out)
    for name, t in (("state_in", state_in), ("state_out", state_out)):
        if t is not None:
            b, _, h, dk = q.shape
            _on_device(name, t, q)
            if t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != (b, h, dk, v.shape[-1]):
                raise ValueError(f"{name} must be a contiguous fp32 [batch, heads, dk, dv] tensor")
    if error_word is not None:
        _on_device("error_word", error_word, q)
        if error_word.dtype != torch.int32 or error_word.numel() < 1 or not error_word.is_contiguous():
            raise ValueError("error_word must be a contiguous GPU int32 tensor of at least one element")
    desc, keep = _desc_for(q, v, gammas, rotary_base, pos_offset, eps)
    _check(lib().retention_chunkwise_fwd_noalloc(ctypes.byref(desc), int(chunk), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                                 _ptr(out), _ptr(state_in), _ptr(state_out), _ptr(error_word),
                                                 _stream(q)))
    del keep
    return out


def chunkwise_varlen_fwd(q, k, v, cu_seqlens, max_seqlen, g=None, *, chunk=512, state_in=None, state_out=None,
                         gammas=None, rotary_base=0.0, pos_offset=0, eps=1e-5, out=None, workspace=None, check=None):
    """Chunkwise form over packed sequences of different lengths: q, k, v, g
    are [total_tokens, heads, d], sequence b holds rows cu_seqlens[b] ..
    cu_seqlens[b+1]-1 (cu_seqlens: GPU int32 [batch + 1]); max_seqlen bounds
    every length. state_in / state_out: fp32 [batch, heads, dk, dv] or None.
    Returns the output (rows outside every sequence are left as they were).
    check: as chunkwise_fwd (clamped cu_seqlens raise RetentionError)."""
    out = torch.empty_like(v) if out is None else out
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("out", out)):
        if t is None:
            continue
        if not t.is_cuda or t.device != q.device or not t.is_contiguous() or t.dtype != q.dtype or t.dim() != 3:
            raise ValueError(f"{name} must be a contiguous GPU [total_tokens, heads, d] tensor of q's dtype")
    if k.shape != q.shape or v.shape[:2] != q.shape[:2] or (g is not None and g.shape != v.shape) \
            or out.shape != v.shape:
        raise ValueError("q, k, v, g and out must agree on [total_tokens, heads]")
    _on_device("cu_seqlens", cu_seqlens, q)
    if not cu_seqlens.is_cuda or cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 \
            or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous GPU int32 tensor [batch + 1]")
    batch = cu_seqlens.numel() - 1
    total, h, dk = q.shape
    for name, st in (("state_in", state_in), ("state_out", state_out)):
        _on_device(name, st, q)
        if st is not None and (st.dtype != torch.float32 or not st.is_contiguous()
                               or tuple(st.shape) != (batch, h, dk, v.shape[-1])):
            raise ValueError(f"{name} must be a contiguous fp32 [batch, heads, dk, dv] tensor")
    desc, keep = make_desc(batch, int(max_seqlen), h, dk, v.shape[-1], _dtype_code(q), gammas, rotary_base,
                           pos_offset, eps)
    L = lib()
    need = L.retention_chunkwise_varlen_workspace_bytes(ctypes.byref(desc), int(chunk))
    workspace, ws_bytes, own = _workspace(workspace, need, q)
    _check(L.retention_chunkwise_varlen_fwd(ctypes.byref(desc), int(chunk), _ptr(cu_seqlens), int(total), _ptr(q),
                                            _ptr(k), _ptr(v), _ptr(g), _ptr(out), _ptr(state_in), _ptr(state_out),
                                            _ptr(workspace), ws_bytes, _stream(q)))
    del keep
    if check or (check is None and own):
        check_chunkwise(workspace)
    return out


def chunkwise_varlen_workspace_bytes(batch, max_seqlen, heads, d, dtype, chunk, rotary_base=0.0):
    """Workspace bytes of chunkwise_varlen_fwd for `batch` sequences of at
    most max_seqlen tokens (dtype: torch.bfloat16 or torch.float32)."""
    code = RET_BF16 if dtype == torch.bfloat16 else RET_F32
    desc, keep = make_desc(batch, max_seqlen, heads, d, d, code, rotary_base=rotary_base)
    return lib().retention_chunkwise_varlen_workspace_bytes(ctypes.byref(desc), int(chunk))


def recurrent_step(q, k, v, state, g=None, *, gammas=None, rotary_base=0.0, pos=0, eps=1e-5, out=None,
                   positions=None):
    """One decode step (q, k: [batch, 1, heads, dk]); updates `state` in place
    and returns the output [batch, 1, heads, dv]. `positions` (optional, a GPU
    int64 tensor [batch]): each sequence's rotation position, in place of
    `pos`."""
    out = torch.empty_like(v) if out is None else out
    _validate(q, k, v, g, out)
    if q.shape[1] != 1:
        raise ValueError("recurrent_step takes one token per sequence (seqlen 1)")
    b, _, h, dk = q.shape
    _on_device("state", state, q)
    if state.dtype != torch.float32 or not state.is_contiguous() or tuple(state.shape) != (b, h, dk, v.shape[-1]):
        raise ValueError("state must be a contiguous fp32 [batch, heads, dk, dv] tensor")
    desc, keep = _desc_for(q, v, gammas, rotary_base, pos, eps)
    if positions is None:
        _check(lib().retention_recurrent_step(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(out),
                                              _ptr(state), _stream(q)))
    else:
        _on_device("positions", positions, q)
        if (positions.dtype != torch.int64 or not positions.is_cuda or not positions.is_contiguous()
                or tuple(positions.shape) != (b,)):
            raise ValueError("positions must be a contiguous GPU int64 tensor [batch]")
        _check(lib().retention_recurrent_step_positions(ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                                        _ptr(out), _ptr(state), _ptr(positions), _stream(q)))
    del keep
    return out


# ---------------------------------------------------------------------------
# Gated delta rule
# ---------------------------------------------------------------------------
# The decode calls' kernels take a few microseconds, so these checks read each
# property once and build nothing they do not need.
def _delta_inputs(q, k, v, log_decay, beta, name, other, cu_seqlens, max_seqlen):
    """Checks of the chunkwise calls' tensors; returns (batch, seqlen,
    total_tokens). `other` (called `name`): a further tensor like v."""
    packed = cu_seqlens is not None
    dims = 3 if packed else 4
    dev, dtype = q.get_device(), q.dtype
    if dev < 0:
        raise ValueError("q must be a GPU tensor")
    for n, t in (("q", q), ("k", k), ("v", v), (name, other)):
        if t.get_device() != dev:
            raise ValueError(f"{n} must be a GPU tensor on {q.device}")
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
        if t.dtype != dtype:
            raise ValueError(f"{n} has dtype {t.dtype}, expected {dtype}")
        if t.dim() != dims:
            raise ValueError(f"{n} must be " + ("[total_tokens, heads, d]" if packed else "[batch, seqlen, heads, d]"))
    qs, vs = q.shape, v.shape
    if k.shape != qs:
        raise ValueError("k must have the shape of q")
    if vs[:-2] != qs[:-2]:
        raise ValueError("v must agree with q on its tokens")
    if other.shape != vs:
        raise ValueError(f"{name} must have the shape of v")
    gates = vs[:-1]
    for n, t in (("log_decay", log_decay), ("beta", beta)):
        if t.get_device() != dev or t.dtype != torch.float32 or not t.is_contiguous() or t.shape != gates:
            raise ValueError(f"{n} must be a contiguous fp32 tensor {list(gates)} on {q.device}")
    if not packed:
        if max_seqlen is not None:
            raise ValueError("max_seqlen goes with cu_seqlens")
        return qs[0], qs[1], 0
    if (cu_seqlens.get_device() != dev or cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1
            or not cu_seqlens.is_contiguous()):
        raise ValueError("cu_seqlens must be a contiguous GPU int32 tensor [batch + 1]")
    if max_seqlen is None:
        raise ValueError("max_seqlen (a bound on every length) goes with cu_seqlens")
    return cu_seqlens.numel() - 1, int(max_seqlen), qs[0]


@functools.lru_cache(maxsize=1024)
def _delta_desc_of(batch, seqlen, k_heads, v_heads, dk, dv, dtype, scale):
    """(descriptor, reference to it): calls only read it."""
    d = DeltaDesc(batch, seqlen, k_heads, v_heads, dk, dv, dtype, scale)
    return d, ctypes.byref(d)


def _delta_desc(batch, seqlen, q, v, scale):
    qs, vs = q.shape, v.shape
    return _delta_desc_of(batch, seqlen, qs[-2], vs[-2], qs[-1], vs[-1], _dtype_code(q), float(scale))[1]


def _delta_state(name, t, batch, q, v):
    if t is None:
        return
    if (t.get_device() != q.get_device() or t.dtype != torch.float32 or not t.is_contiguous()
            or t.shape != (batch, v.shape[-2], q.shape[-1], v.shape[-1])):
        raise ValueError(f"{name} must be a contiguous fp32 [batch, v_heads, dk, dv] tensor on {q.device}")


_here = contextlib.nullcontext()


def _current(t):
    """The tensor's device as the current one (kernels launch there)."""
    dev = t.get_device()
    return _here if dev == torch.cuda.current_device() else torch.cuda.device(dev)


def delta_chunkwise_fwd(q, k, v, log_decay, beta, *, scale=1.0, state_in=None, state_out=None, cu_seqlens=None,
                        max_seqlen=None, out=None, workspace=None, check=False):
    """Gated delta rule over whole sequences: q, k [batch, seqlen, k_heads, d],
    v [batch, seqlen, v_heads, d], log_decay and beta fp32 [batch, seqlen,
    v_heads]; returns the output (v's shape) and fills state_out (fp32 [batch,
    v_heads, d, d], may be state_in itself) if it is given. Packed sequences:
    [total_tokens, heads, d] tensors with cu_seqlens (GPU int32 [batch + 1])
    and max_seqlen; rows outside every sequence are left as they were. A first
    token with log decay -infinity forgets whatever state_in holds. check:
    synchronize and raise RetentionError if cu_seqlens had to be clamped
    (check_chunkwise does the same later for a caller's workspace)."""
    out = torch.empty_like(v) if out is None else out
    batch, seqlen, total = _delta_inputs(q, k, v, log_decay, beta, "out", out, cu_seqlens, max_seqlen)
    _delta_state("state_in", state_in, batch, q, v)
    _delta_state("state_out", state_out, batch, q, v)
    desc = _delta_desc(batch, seqlen, q, v, scale)
    L = lib()
    need = L.retention_delta_workspace_bytes(desc, int(cu_seqlens is not None), total)
    workspace, ws_bytes, _ = _workspace(workspace, need, q)
    with _current(q):
        _check(L.retention_delta_fwd(desc, _ptr(cu_seqlens), total, _ptr(q), _ptr(k), _ptr(v),
                                     _ptr(log_decay), _ptr(beta), _ptr(out), _ptr(state_in), _ptr(state_out),
                                     _ptr(workspace), ws_bytes, _stream(q)))
    if check:
        check_chunkwise(workspace)
    return out


def delta_chunkwise_bwd(q, k, v, log_decay, beta, dout, *, scale=1.0, state_in=None, d_state_out=None,
                        cu_seqlens=None, max_seqlen=None, workspace=None, check=False):
    """Gradients of sum(dout * out) (+ sum(d_state_out * state_out)) with out,
    state_out = delta_chunkwise_fwd(q, k, v, log_decay, beta, ...). Returns
    (dq, dk, dv, dlog_decay, dbeta), and d_state_in after them when state_in
    is given. Packed sequences and check as in the forward; gradient rows
    outside every sequence are zero."""
    batch, seqlen, total = _delta_inputs(q, k, v, log_decay, beta, "dout", dout, cu_seqlens, max_seqlen)
    _delta_state("state_in", state_in, batch, q, v)
    _delta_state("d_state_out", d_state_out, batch, q, v)
    new = torch.empty_like if cu_seqlens is None else torch.zeros_like
    grads = [new(t) for t in (q, k, v, log_decay, beta)]
    if state_in is not None:
        grads.append(torch.empty_like(state_in))
    desc = _delta_desc(batch, seqlen, q, v, scale)
    L = lib()
    need = L.retention_delta_bwd_workspace_bytes(desc, int(cu_seqlens is not None), total)
    workspace, ws_bytes, _ = _workspace(workspace, need, q)
    with _current(q):
        _check(L.retention_delta_bwd(desc, _ptr(cu_seqlens), total, _ptr(q), _ptr(k), _ptr(v),
                                     _ptr(log_decay), _ptr(beta), _ptr(dout), _ptr(state_in), _ptr(d_state_out),
                                     *(_ptr(t) for t in grads[:5]), _ptr(grads[5]) if state_in is not None else None,
                                     _ptr(workspace), ws_bytes, _stream(q)))
    if check:
        check_chunkwise(workspace)
    return tuple(grads)


def delta_recurrent_step(q, k, v, log_decay, beta, state, *, scale=1.0, slots=None, out=None):
    """One decode step of the gated delta rule (q, k: [batch, 1, k_heads, d],
    v: [batch, 1, v_heads, d]); updates `state` in place and returns the
    output. state: fp32 [batch, v_heads, d, d], or with `slots` (GPU int32
    [batch]) a pool [num_slots, v_heads, d, d] of which sequence b uses slot
    slots[b]; a slot that is negative, outside the pool or named by an earlier
    sequence is inactive (its output is zero). Log decay -infinity forgets
    whatever the slot holds."""
    out = torch.empty_like(v) if out is None else out
    batch, seqlen, _ = _delta_inputs(q, k, v, log_decay, beta, "out", out, None, None)
    if seqlen != 1:
        raise ValueError("delta_recurrent_step takes one token per sequence (seqlen 1)")
    _delta_state("state", state, batch if slots is None else state.shape[0], q, v)
    if slots is not None:
        if (slots.get_device() != q.get_device() or slots.dtype != torch.int32 or not slots.is_contiguous()
                or slots.shape != (batch,)):
            raise ValueError("slots must be a contiguous GPU int32 tensor [batch]")
    desc = _delta_desc(batch, 1, q, v, scale)
    with _current(q):
        _check(lib().retention_delta_step(desc, _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(beta),
                                          _ptr(out), _ptr(state), _ptr(slots), state.shape[0], _stream(q)))
    return out


# ---------------------------------------------------------------------------
# Norms around a token mixer
# ---------------------------------------------------------------------------
def _norm_inputs(x, rows, weights):
    """Checks of a norm call's tensors: `rows` like x, `weights` fp32 [width]."""
    dev, dtype, shape = x.get_device(), x.dtype, x.shape
    if dev < 0 or not x.is_contiguous() or x.dim() < 1:
        raise ValueError("x must be a contiguous GPU tensor [..., width]")
    for name, t in rows:
        if t is not None and (t.get_device() != dev or t.dtype != dtype or not t.is_contiguous() or t.shape != shape):
            raise ValueError(f"{name} must be a contiguous tensor of x's shape and dtype on {x.device}")
    width = shape[-1:]
    for name, t in weights:
        if t is not None and (t.get_device() != dev or t.dtype != torch.float32 or not t.is_contiguous()
                              or t.shape != width):
            raise ValueError(f"{name} must be a contiguous fp32 tensor [{shape[-1]}] on {x.device}")


@functools.lru_cache(maxsize=1024)
def _norm_desc_of(rows, width, dtype, center, eps):
    """(descriptor, reference to it): calls only read it."""
    d = NormDesc(rows, width, dtype, center, eps)
    return d, ctypes.byref(d)


def _norm_desc(x, center, eps):
    width = x.shape[-1]
    return _norm_desc_of(x.numel() // width if width else 0, width, _dtype_code(x), int(bool(center)), float(eps))[1]


def head_norm_fwd(x, weight=None, gate=None, *, center=False, eps=1e-5, out=None):
    """Norm over the last dimension (a head of a token), times weight (fp32
    [d]) and swish(gate) where given; center: subtract the mean (GroupNorm, one
    group per head), else the root mean square alone."""
    out = torch.empty_like(x) if out is None else out
    _norm_inputs(x, (("gate", gate), ("out", out)), (("weight", weight),))
    desc = _norm_desc(x, center, eps)
    with _current(x):
        _check(lib().retention_head_norm_fwd(desc, _ptr(x), _ptr(weight), _ptr(gate), _ptr(out),
                                             _stream(x)))
    return out


def head_norm_bwd(x, dout, weight=None, gate=None, *, center=False, eps=1e-5, workspace=None):
    """Gradients of sum(dout * head_norm_fwd(x, weight, gate, ...)): (dx,
    dweight, dgate), None where there is no such input."""
    _norm_inputs(x, (("dout", dout), ("gate", gate)), (("weight", weight),))
    dx = torch.empty_like(x)
    dweight = torch.empty_like(weight) if weight is not None else None
    dgate = torch.empty_like(gate) if gate is not None else None
    desc = _norm_desc(x, center, eps)
    L = lib()
    need = L.retention_head_norm_bwd_workspace_bytes(desc) if weight is not None else 0
    workspace, ws_bytes, _ = _workspace(workspace, need, x)
    with _current(x):
        _check(L.retention_head_norm_bwd(desc, _ptr(x), _ptr(weight), _ptr(gate), _ptr(dout), _ptr(dx),
                                         _ptr(dweight), _ptr(dgate), _ptr(workspace), ws_bytes, _stream(x)))
    return dx, dweight, dgate


def residual_norm_fwd(x, y, weight, *, post_weight=None, scale=None, skip=1.0, center=False, eps=1e-5, out=None,
                      residual=None):
    """The step from one block to the next over rows [..., width]: z = norm(y)
    post_weight (or y), residual = skip x + scale z, out = norm(residual)
    weight; returns (out, residual). residual may be x itself. post_weight,
    scale, weight: fp32 [width]."""
    out = torch.empty_like(x) if out is None else out
    residual = torch.empty_like(x) if residual is None else residual
    _norm_inputs(x, (("y", y), ("out", out), ("residual", residual)),
                 (("weight", weight), ("post_weight", post_weight), ("scale", scale)))
    desc = _norm_desc(x, center, eps)
    with _current(x):
        _check(lib().retention_residual_norm_fwd(desc, float(skip), _ptr(x), _ptr(y), _ptr(weight),
                                                 _ptr(post_weight), _ptr(scale), _ptr(out), _ptr(residual), _stream(x)))
    return out, residual


def residual_norm_bwd(x, y, weight, dout, dresidual=None, *, post_weight=None, scale=None, skip=1.0, center=False,
                      eps=1e-5, workspace=None):
    """Gradients of sum(dout * out) (+ sum(dresidual * residual)) with out,
    residual = residual_norm_fwd(x, y, weight, ...): (dx, dy, dweight,
    dpost_weight, dscale), None where there is no such input. x and y are the
    forward's inputs (x before a residual written over it)."""
    _norm_inputs(x, (("y", y), ("dout", dout), ("dresidual", dresidual)),
                 (("weight", weight), ("post_weight", post_weight), ("scale", scale)))
    dx, dy, dweight = torch.empty_like(x), torch.empty_like(y), torch.empty_like(weight)
    dpost = torch.empty_like(post_weight) if post_weight is not None else None
    dscale = torch.empty_like(scale) if scale is not None else None
    desc = _norm_desc(x, center, eps)
    L = lib()
    need = L.retention_residual_norm_bwd_workspace_bytes(desc)
    workspace, ws_bytes, _ = _workspace(workspace, need, x)
    with _current(x):
        _check(L.retention_residual_norm_bwd(desc, float(skip), _ptr(x), _ptr(y), _ptr(weight),
                                             _ptr(post_weight), _ptr(scale), _ptr(dout), _ptr(dresidual), _ptr(dx),
                                             _ptr(dy), _ptr(dweight), _ptr(dpost), _ptr(dscale), _ptr(workspace),
                                             ws_bytes, _stream(x)))
    return dx, dy, dweight, dpost, dscale
