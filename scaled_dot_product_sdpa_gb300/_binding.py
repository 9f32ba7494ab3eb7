"""ctypes binding of libgbattn.so: argument marshalling only.

Every function here converts torch tensors to raw device pointers and sizes, calls the
C entry point of the same name (include/gbattn.h), and turns a nonzero return code into
a GbattnError.  There is no fallback: if the library is missing or the tensors are not
on a CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgbattn.so")
_lib = None

FLAG_P_SMEM = 1
FLAG_SINGLE_TILE = 2
FLAG_TWO_TILE = 4
FLAG_DSPLIT = 8
FLAG_SPLIT_KV = 16


class GbattnError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: gbattn error {code}: {attn_strerror(code)}")


def load_library(path: str | None = None):
    """Load libgbattn.so (built by scaled_dot_product_sdpa_gb300.build).  Raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libgbattn.so not built ({path} missing); run "
                           "`python -m scaled_dot_product_sdpa_gb300.build` or __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
    lib.attn_fwd.restype = i
    lib.attn_fwd_ex.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, i, i]
    lib.attn_fwd_ex.restype = i
    lib.attn_debug_scores.argtypes = [vp, vp, vp, i, i, i, i, f, vp]
    lib.attn_debug_scores.restype = i
    lib.attn_last_device_error.argtypes = []
    lib.attn_last_device_error.restype = i
    lib.attn_debug_wait_probe.argtypes = [ctypes.c_longlong, vp]
    lib.attn_debug_wait_probe.restype = i
    lib.attn_strerror.argtypes = [i]
    lib.attn_strerror.restype = ctypes.c_char_p
    ip = ctypes.POINTER(ctypes.c_int)
    lib.attn_debug_schedule.argtypes = [i, i, i, i, i, i, i, ip, ip, i]
    lib.attn_debug_schedule.restype = i
    sz = ctypes.c_size_t
    lib.attn_fwd_host.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, vp, sz, vp]
    lib.attn_fwd_host.restype = i
    lib.attn_fwd_host_workspace_size.argtypes = [i, i, i, i]
    lib.attn_fwd_host_workspace_size.restype = sz
    lib.attn_debug_plan.argtypes = [i, i, i, i, i, i, i, i, ip]
    lib.attn_debug_plan.restype = i
    lib.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
    lib.attn_bwd.restype = i
    lib.attn_bwd_workspace_bytes.argtypes = [i, i, i]
    lib.attn_bwd_workspace_bytes.restype = ctypes.c_longlong
    lib.attn_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, vp]
    lib.attn_bwd_noalloc.restype = i
    lib.attn_bwd_noalloc_max_bytes.argtypes = []
    lib.attn_bwd_noalloc_max_bytes.restype = ctypes.c_longlong
    lib.attn_decode.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, vp]
    lib.attn_decode.restype = i
    lib.attn_decode_workspace_bytes.argtypes = [i, i, i]
    lib.attn_decode_workspace_bytes.restype = ctypes.c_longlong
    lib.attn_debug_decode_plan.argtypes = [i, i, i, i, i, i, i, ip]
    lib.attn_debug_decode_plan.restype = i
    ll = ctypes.c_longlong
    rows = [vp, ll, ll, ll]
    lib.attn_rope.argtypes = rows + rows + [vp, vp, vp, i, i, f, vp, ll, vp, vp, f, i, i, i, i, i, i, vp]
    lib.attn_rope.restype = i
    lib.attn_rope_bwd.argtypes = (4 * rows + [vp, vp, vp, vp, vp, i, i, f, vp, ll, vp, vp, f, vp, i, i, i, i, i, i, vp])
    lib.attn_rope_bwd.restype = i
    lib.attn_rope_bwd_workspace_bytes.argtypes = [i]
    lib.attn_rope_bwd_workspace_bytes.restype = ll
    lib.attn_cache_append.argtypes = (3 * rows + [vp, vp, vp, ll, ll, ll, i, i, vp, ll, i, vp, vp, vp, i, i, f, vp, vp, f,
                                                  i, i, i, i, i, i, vp])
    lib.attn_cache_append.restype = i
    lib.attn_cache_copy.argtypes = [vp, vp, ll, ll, ll, i, i, i, i, vp, vp, i, vp]
    lib.attn_cache_copy.restype = i
    lib.attn_decode_paged.argtypes = [vp, ll, ll, vp, vp, ll, ll, ll, i, i, vp, ll, i, vp, vp, vp, vp, i, i, i, i, i, f, vp]
    lib.attn_decode_paged.restype = i
    lib.attn_decode_paged_workspace_bytes.argtypes = [i, i, i]
    lib.attn_decode_paged_workspace_bytes.restype = ll
    lib.attn_version.argtypes = []
    lib.attn_version.restype = i
    _lib = lib
    return lib


def attn_strerror(code: int) -> str:
    return load_library().attn_strerror(int(code)).decode()


def attn_version() -> int:
    return load_library().attn_version()


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check_qkv(q, k, v=None):
    ts = [q, k] + ([v] if v is not None else [])
    for t in ts:
        if not t.is_cuda:
            raise ValueError("gbattn: tensors must be on a CUDA device (no CPU path exists)")
        if t.dtype != torch.float16:
            raise ValueError("gbattn: q, k, v must be float16")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError("gbattn: q, k, v must be contiguous [B, H, L, d]")
        if t.shape != q.shape:
            raise ValueError("gbattn: q, k, v must have the same shape")
    return q.shape


def attn_fwd(q, k, v, causal: bool = False, scale: float | None = None, o=None, lse=None, stream=None,
             flags: int = 0, grid_limit: int = 0):
    """O, LSE = SDPA forward of fp16 [B, H, L, d] q, k, v.  Outputs are allocated by torch
    on q's device unless given.  Enqueued on `stream` (default: torch's current stream)."""
    B, H, L, d = _check_qkv(q, k, v)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    if o.shape != q.shape or o.dtype != torch.float16 or not o.is_contiguous():
        raise ValueError("gbattn: o must be contiguous float16 like q")
    if lse.shape != (B, H, L) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("gbattn: lse must be contiguous float32 [B, H, L]")
    lib = load_library()
    with torch.cuda.device(q.device):
        rc = lib.attn_fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                             B, H, L, d, int(bool(causal)), float(scale), _stream_handle(stream),
                             int(flags), int(grid_limit))
    if rc != 0:
        raise GbattnError(rc, "attn_fwd")
    return o, lse


def attn_bwd_workspace_bytes(B: int, H: int, L: int) -> int:
    """Bytes of device workspace attn_bwd needs (8 per query row, rows padded to 128)."""
    n = load_library().attn_bwd_workspace_bytes(int(B), int(H), int(L))
    if n < 0:
        raise GbattnError(int(n), "attn_bwd_workspace_bytes")
    return int(n)


def attn_bwd(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None, dq=None, dk=None, dv=None,
             stream=None, workspace=None):
    """Gradients (dq, dk, dv) of O = SDPA(q, k, v) for the upstream gradient dout, from the
    forward pass's o and lse (as attn_fwd returns them).  fp16 [B, H, L, d] tensors, d 64 or
    128; outputs allocated by torch on q's device unless given, and so is the workspace
    (attn_bwd_workspace_bytes(B, H, L) bytes) unless `workspace` (a contiguous CUDA tensor
    at least that large) is given.  Enqueued on `stream`."""
    B, H, L, d = _check_qkv(q, k, v)
    for t in (o, dout):
        if not t.is_cuda or t.dtype != torch.float16 or t.shape != q.shape or not t.is_contiguous():
            raise ValueError("gbattn: o and dout must be contiguous float16 like q")
    if not lse.is_cuda or lse.dtype != torch.float32 or lse.shape != (B, H, L) or not lse.is_contiguous():
        raise ValueError("gbattn: lse must be contiguous float32 [B, H, L]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    for t in (dq, dk, dv):
        if t.shape != q.shape or t.dtype != torch.float16 or not t.is_contiguous():
            raise ValueError("gbattn: dq, dk, dv must be contiguous float16 like q")
    lib = load_library()
    nbytes = attn_bwd_workspace_bytes(B, H, L)
    if workspace is None:
        workspace = torch.empty(nbytes // 4, dtype=torch.float32, device=q.device)
        if isinstance(stream, torch.cuda.Stream):
            workspace.record_stream(stream)  # freed only once the kernels on `stream` are done
    elif (not workspace.is_cuda or not workspace.is_contiguous()
          or workspace.numel() * workspace.element_size() < nbytes):
        raise ValueError(f"gbattn: workspace must be a contiguous CUDA tensor of at least {nbytes} bytes")
    with torch.cuda.device(q.device):
        rc = lib.attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), dout.data_ptr(),
                          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), B, H, L, d,
                          int(bool(causal)), float(scale), _stream_handle(stream))
    if rc != 0:
        raise GbattnError(rc, "attn_bwd")
    return dq, dk, dv


def attn_decode(q, k, v, scale: float | None = None, o=None, lse=None, stream=None, grouped: bool = True):
    """Decode: O [B, H, d] and LSE [B, H] for one fp16 query row q ([B, H, d] or
    [B, H, 1, d]) per head against fp16 k, v [B, H, L, d], every key visible.  Outputs are
    allocated by torch on q's device unless given, and so is the small workspace that lets
    a head's keys be split over several clusters (`grouped`; without it, one cluster per
    head).  Enqueued on `stream`."""
    for t in (q, k, v):
        if not t.is_cuda:
            raise ValueError("gbattn: tensors must be on a CUDA device (no CPU path exists)")
        if t.dtype != torch.float16 or not t.is_contiguous():
            raise ValueError("gbattn: q, k, v must be contiguous float16")
    if k.dim() != 4 or v.shape != k.shape:
        raise ValueError("gbattn: k and v must share one [B, H, L, d] shape")
    B, H, L, d = k.shape
    if tuple(q.shape) not in ((B, H, d), (B, H, 1, d)):
        raise ValueError("gbattn: q must be [B, H, d] or [B, H, 1, d]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty((B, H, d), dtype=torch.float16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if o.numel() != B * H * d or o.dtype != torch.float16 or not o.is_contiguous():
        raise ValueError("gbattn: o must be contiguous float16 with B*H*d elements")
    if lse.numel() != B * H or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("gbattn: lse must be contiguous float32 [B, H]")
    lib = load_library()
    ws = None
    if grouped:
        nbytes = lib.attn_decode_workspace_bytes(B, H, d)
        if nbytes < 0:
            raise GbattnError(int(nbytes), "attn_decode_workspace_bytes")
        ws = torch.empty(nbytes // 4, dtype=torch.float32, device=q.device)
        if isinstance(stream, torch.cuda.Stream):
            ws.record_stream(stream)  # freed only once the kernels on `stream` are done
    with torch.cuda.device(q.device):
        rc = lib.attn_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                             ws.data_ptr() if ws is not None else None, B, H, L, d, float(scale),
                             _stream_handle(stream))
    if rc != 0:
        raise GbattnError(rc, "attn_decode")
    return o, lse


def attn_debug_decode_plan(B: int, H: int, L: int, d: int, sm_count: int, max_ranks: int = 16,
                           grouped: bool = False) -> dict:
    """The split attn_decode uses (host-only): CTAs per cluster, keys per CTA and clusters
    per head (more than one only with a workspace, `grouped`)."""
    out = (ctypes.c_int * 3)()
    rc = load_library().attn_debug_decode_plan(B, H, L, d, sm_count, max_ranks, int(bool(grouped)), out)
    if rc != 0:
        raise GbattnError(rc, "attn_debug_decode_plan")
    return {"ranks": out[0], "keys_per_rank": out[1], "groups": out[2]}


def attn_debug_scores(q, k, scale: float | None = None, s=None, stream=None):
    """Raw scaled logits scale * Q K^T as fp32 [B, H, L, L] (test hook, no mask)."""
    B, H, L, d = _check_qkv(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if s is None:
        s = torch.empty((B, H, L, L), dtype=torch.float32, device=q.device)
    lib = load_library()
    with torch.cuda.device(q.device):
        rc = lib.attn_debug_scores(q.data_ptr(), k.data_ptr(), s.data_ptr(), B, H, L, d, float(scale),
                                   _stream_handle(stream))
    if rc != 0:
        raise GbattnError(rc, "attn_debug_scores")
    return s


def attn_last_device_error() -> int:
    """Synchronise the current device, then read and clear its device status word."""
    return load_library().attn_last_device_error()


def attn_debug_wait_probe(limit_cycles: int, stream=None) -> None:
    rc = load_library().attn_debug_wait_probe(int(limit_cycles), _stream_handle(stream))
    if rc != 0:
        raise GbattnError(rc, "attn_debug_wait_probe")


def attn_debug_schedule(B: int, H: int, L: int, d: int, causal: bool, grid: int, flags: int = 0):
    """The static work schedule attn_fwd would use (host-only): a list with, per CTA, the
    work-item indices it runs in order; None when the kernels use their fixed order.  With
    FLAG_SPLIT_KV an index >= the item count names a query tile whose key range the two
    CTAs of a cluster (CTAs 2c, 2c + 1) share."""
    max_items = 1 << 16
    start = (ctypes.c_int * (grid + 1))()
    items = (ctypes.c_int * max_items)()
    n = load_library().attn_debug_schedule(B, H, L, d, int(bool(causal)), grid, flags, start, items, max_items)
    if n < 0:
        raise GbattnError(n, "attn_debug_schedule")
    if n == 0:
        return None
    return [list(items[start[c]:start[c + 1]]) for c in range(grid)]


def attn_debug_plan(B: int, H: int, L: int, d: int, causal: bool, sm_count: int, flags: int = 0,
                    grid_limit: int = 0) -> dict:
    """The kernel attn_fwd would launch on a GPU with `sm_count` SMs (host-only):
    kind 0 single-tile, 1 two-tile, 2 single-tile with the head_dim split, 3 single-tile
    with key-range splits (CTAs in clusters of two)."""
    out = (ctypes.c_int * 4)()
    rc = load_library().attn_debug_plan(B, H, L, d, int(bool(causal)), sm_count, flags, grid_limit, out)
    if rc != 0:
        raise GbattnError(rc, "attn_debug_plan")
    return {"kind": out[0], "items": out[1], "grid": out[2], "makespan": out[3] / 100.0}


# Device workspaces of attn_fwd_host, one per (device, stream): calls on one stream never
# overlap on the GPU, calls on different streams may.
_host_workspaces: dict = {}


def attn_fwd_host(q, k, v, causal: bool = False, scale: float | None = None, o=None, lse=None,
                  device=None, stream=None):
    """O, LSE = SDPA forward of fp16 [B, H, L, d] CPU tensors q, k, v (pin them for the
    copies to overlap), computed on `device` (default: the current CUDA device) in
    chunks whose host<->device copies overlap the kernels.  Outputs are CPU tensors
    (pinned, allocated here unless given).  Enqueued on `stream` (default: the device's
    current stream); synchronise it before reading the outputs."""
    for t in (q, k, v):
        if t.is_cuda:
            raise ValueError("gbattn: attn_fwd_host takes CPU tensors (use attn_fwd for CUDA tensors)")
        if t.dtype != torch.float16 or t.dim() != 4 or not t.is_contiguous() or t.shape != q.shape:
            raise ValueError("gbattn: q, k, v must be contiguous float16 [B, H, L, d] of one shape")
    B, H, L, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q).pin_memory()
    if lse is None:
        lse = torch.empty((B, H, L), dtype=torch.float32).pin_memory()
    if o.is_cuda or o.shape != q.shape or o.dtype != torch.float16 or not o.is_contiguous():
        raise ValueError("gbattn: o must be a contiguous float16 CPU tensor like q")
    if lse.is_cuda or lse.shape != (B, H, L) or lse.dtype != torch.float32 or not lse.is_contiguous():
        raise ValueError("gbattn: lse must be a contiguous float32 CPU tensor [B, H, L]")
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    lib = load_library()
    with torch.cuda.device(device):
        sh = _stream_handle(stream)
        need = int(lib.attn_fwd_host_workspace_size(B, H, L, d))
        key = (device.index, sh)
        ws = _host_workspaces.get(key)
        if ws is None or ws.numel() < need:
            ws = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
            _host_workspaces[key] = ws
        rc = lib.attn_fwd_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                               B, H, L, d, int(bool(causal)), float(scale), ws.data_ptr(), ws.numel(), sh)
    if rc != 0:
        raise GbattnError(rc, "attn_fwd_host")
    return o, lse


# ---------------------------------------------------------------------------------------
# Rotary positions and the paged cache.  Tensors of a call share one device and, but for the
# integer and frequency tensors, one type (float16 or bfloat16).  What a call allocates
# belongs to the stream that it runs on.
_DTYPES = {torch.float16: 0, torch.bfloat16: 1}


def _empty(shape, dtype, device, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _launch(what, fn, device, stream, *args):
    """Call the C entry point `fn` with the device current and its stream as last argument."""
    if device.index == torch.cuda.current_device():
        rc = fn(*args, _stream_handle(stream))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _stream_handle(stream))
    if rc != 0:
        raise GbattnError(rc, what)


def _check_like(t, name, q, shape=None):
    if not t.is_cuda or t.device != q.device:
        raise ValueError(f"gbattn: {name} must be on the CUDA device of the other tensors (no CPU path exists)")
    if t.dtype != q.dtype:
        raise ValueError(f"gbattn: {name} must be {q.dtype} like the other tensors")
    if shape is not None and t.shape != shape:
        raise ValueError(f"gbattn: {name} must have the shape {tuple(shape)}")


def _dtype_code(t, name):
    if not t.is_cuda:
        raise ValueError("gbattn: tensors must be on a CUDA device (no CPU path exists)")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"gbattn: {name} must be float16 or bfloat16")
    return code


def _rows(t, name):
    """(pointer, strides of batch, head and row) of [B, H, L, d] rows; the last dimension must be
    contiguous, the strides of dimensions of one element do not matter."""
    sb, sh, sl, sd = t.stride()
    B, H, L, _ = t.shape
    if sd != 1:
        raise ValueError(f"gbattn: the last dimension of {name} must be contiguous")
    return t.data_ptr(), sb if B > 1 else 0, sh if H > 1 else 0, sl if L > 1 else 0


_NO_ROWS = (None, 0, 0, 0)


def _out(t, name, shape, dtype, like, stream):
    if t is None:
        return _empty(shape, dtype, like.device, stream)
    if t.shape != shape or t.dtype != dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"gbattn: {name} must be contiguous {dtype} {tuple(shape)} on the device of the other tensors")
    return t


def _ints(t, name, shape, like):
    """(pointer, row stride) of an int32 device tensor whose last dimension is contiguous."""
    if t.dtype != torch.int32 or t.device != like.device or t.shape != shape:
        raise ValueError(f"gbattn: {name} must be int32 {tuple(shape)} on the device of the other tensors")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"gbattn: the last dimension of {name} must be contiguous")
    return t.data_ptr(), (t.stride(0) if t.dim() == 2 and t.shape[0] > 1 else 0)


def _frequencies(inv_freq, d, like):
    """(pointer, rotary width) of the inverse frequencies (None: nothing is rotated)."""
    if inv_freq is None:
        return None, 0
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or inv_freq.device != like.device or not inv_freq.is_contiguous():
        raise ValueError("gbattn: inv_freq must be contiguous float64 [rotary / 2] on the device of the other tensors")
    n = 2 * inv_freq.shape[0]
    return (inv_freq.data_ptr() if n else None), n


def _norm_weights(q_weight, k_weight, d, q, has_q, has_k):
    if q_weight is None and k_weight is None:
        return None, None
    if (q_weight is None) == has_q or (k_weight is None) == has_k:
        raise ValueError("gbattn: norms need a weight for each tensor that is normalised")
    for t, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _check_like(t, name, q, (d,))
            if not t.is_contiguous():
                raise ValueError(f"gbattn: {name} must be contiguous")
    return q_weight.data_ptr() if has_q else None, k_weight.data_ptr() if has_k else None


def _rope_positions(positions, B, L, like):
    if positions is None:
        return None, 0
    if positions.dim() == 1:
        return _ints(positions, "positions", (L,), like)[0], 0
    return _ints(positions, "positions", (B, L), like)


def attn_rope(q, k, inv_freq, positions=None, interleaved: bool = False, factor: float = 1.0, q_weight=None,
              k_weight=None, eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """Rotary positions, and with q_weight and k_weight ([d]) per-head RMS norms before them, of
    q [B, Hq, L, d] and k [B, Hkv, L, d] (k None: q alone), fp16 or bf16, in one pass.  Rows may
    lie anywhere (a transposed [B, L, H, d] projection, a slice of a joint one) as long as each
    is contiguous; the outputs (q_out, k_out) are contiguous [B, H, L, d], as attn_fwd takes them.
    inv_freq: float64 [rotary / 2] (attn_rope_frequencies), rotary a multiple of 16 up to d;
    positions: int32 [B, L] or [L], default 0 .. L-1; interleaved: pairs (2r, 2r + 1) instead of
    (r, r + rotary / 2); factor multiplies cosine and sine.  Enqueued on `stream`."""
    code = _dtype_code(q, "q")
    if q.dim() != 4:
        raise ValueError("gbattn: q must be [B, H, L, d]")
    B, Hq, L, d = q.shape
    Hkv = 0
    kr = _NO_ROWS
    if k is not None:
        if k.dim() != 4 or k.shape[0] != B or k.shape[2] != L or k.shape[3] != d:
            raise ValueError("gbattn: k must be [B, Hkv, L, d] like q")
        _check_like(k, "k", q)
        Hkv = k.shape[1]
        kr = _rows(k, "k")
        k_out = _out(k_out, "k_out", k.shape, q.dtype, q, stream)
    fp, rotary = _frequencies(inv_freq, d, q)
    pp, ps = _rope_positions(positions, B, L, q)
    wq, wk = _norm_weights(q_weight, k_weight, d, q, True, k is not None)
    q_out = _out(q_out, "q_out", q.shape, q.dtype, q, stream)
    _launch("attn_rope", load_library().attn_rope, q.device, stream, *_rows(q, "q"), *kr, q_out.data_ptr(),
            k_out.data_ptr() if k is not None else None, fp, rotary, int(bool(interleaved)), float(factor), pp, ps, wq, wk,
            float(eps), code, B, Hq, Hkv, L, d)
    return q_out, (k_out if k is not None else None)


def attn_rope_bwd(dq, dk, inv_freq, positions=None, interleaved: bool = False, factor: float = 1.0, q=None, k=None,
                  q_weight=None, k_weight=None, eps: float = 1e-6, dq_out=None, dk_out=None, dq_weight=None,
                  dk_weight=None, stream=None, workspace=None):
    """Gradients of attn_rope: from dq [B, Hq, L, d] and dk [B, Hkv, L, d] (of its outputs; attn_bwd's
    results; dk None without keys) those of its inputs, contiguous: (dq_out, dk_out).  With norms, q and k
    are attn_rope's inputs and the result is (dq_out, dk_out, dq_weight, dk_weight), the weights'
    gradients in float32 [d].  The other arguments are attn_rope's."""
    code = _dtype_code(dq, "dq")
    if dq.dim() != 4:
        raise ValueError("gbattn: dq must be [B, H, L, d]")
    B, Hq, L, d = dq.shape
    Hkv = 0
    kr = _NO_ROWS
    if dk is not None:
        if dk.dim() != 4 or dk.shape[0] != B or dk.shape[2] != L or dk.shape[3] != d:
            raise ValueError("gbattn: dk must be [B, Hkv, L, d] like dq")
        _check_like(dk, "dk", dq)
        Hkv = dk.shape[1]
        kr = _rows(dk, "dk")
        dk_out = _out(dk_out, "dk_out", dk.shape, dq.dtype, dq, stream)
    fp, rotary = _frequencies(inv_freq, d, dq)
    pp, ps = _rope_positions(positions, B, L, dq)
    wq, wk = _norm_weights(q_weight, k_weight, d, dq, True, dk is not None)
    lib = load_library()
    xq = xk = _NO_ROWS
    norm = wq is not None
    if norm:
        if q is None or (dk is not None) != (k is not None):
            raise ValueError("gbattn: the gradients of norms need attn_rope's inputs q and k")
        _check_like(q, "q", dq, dq.shape)
        xq = _rows(q, "q")
        dq_weight = _out(dq_weight, "dq_weight", (d,), torch.float32, dq, stream)
        if k is not None:
            _check_like(k, "k", dq, dk.shape)
            xk = _rows(k, "k")
            dk_weight = _out(dk_weight, "dk_weight", (d,), torch.float32, dq, stream)
        nbytes = lib.attn_rope_bwd_workspace_bytes(d)
        if nbytes < 0:
            raise GbattnError(int(nbytes), "attn_rope_bwd_workspace_bytes")
        workspace = _workspace(workspace, nbytes, dq, stream)
    dq_out = _out(dq_out, "dq_out", dq.shape, dq.dtype, dq, stream)
    _launch("attn_rope_bwd", lib.attn_rope_bwd, dq.device, stream, *_rows(dq, "dq"), *kr, *xq, *xk, dq_out.data_ptr(),
            dk_out.data_ptr() if dk is not None else None, dq_weight.data_ptr() if norm else None,
            dk_weight.data_ptr() if norm and dk is not None else None, fp, rotary, int(bool(interleaved)), float(factor), pp,
            ps, wq, wk, float(eps), workspace.data_ptr() if norm else None, code, B, Hq, Hkv, L, d)
    if dk is None:
        dk_out = None
    return (dq_out, dk_out, dq_weight, dk_weight if dk is not None else None) if norm else (dq_out, dk_out)


def attn_rope_bwd_workspace_bytes(d: int) -> int:
    """Bytes of device workspace attn_rope_bwd needs with norms."""
    n = load_library().attn_rope_bwd_workspace_bytes(int(d))
    if n < 0:
        raise GbattnError(int(n), "attn_rope_bwd_workspace_bytes")
    return int(n)


def _workspace(workspace, nbytes, like, stream):
    if workspace is None:
        return _empty((nbytes // 4,), torch.float32, like.device, stream)
    if (workspace.device != like.device or not workspace.is_contiguous()
            or workspace.numel() * workspace.element_size() < nbytes):
        raise ValueError(f"gbattn: workspace must be a contiguous CUDA tensor of at least {nbytes} bytes on the device "
                         "of the other tensors")
    return workspace


def _cache(k_pages, v_pages, like=None):
    """(k pointer, v pointer, page, head and slot strides, pages, slots of a page), and the shape."""
    code = _dtype_code(k_pages, "k_pages")
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("gbattn: k_pages and v_pages must share one [pages, Hkv, page, d] shape")
    if v_pages.dtype != k_pages.dtype or v_pages.device != k_pages.device:
        raise ValueError("gbattn: k_pages and v_pages must share their type and device")
    if like is not None:
        _check_like(like, "q, k and v", k_pages)
    P, H, page, d = k_pages.shape
    sp, sh, ss, sd = k_pages.stride()
    vp, vh, vs, vd = v_pages.stride()
    if sd != 1 or vd != 1:
        raise ValueError("gbattn: the last dimension of k_pages and v_pages must be contiguous")
    if (P > 1 and sp != vp) or (H > 1 and sh != vh) or (page > 1 and ss != vs):
        raise ValueError("gbattn: k_pages and v_pages must share their strides")
    sh = sh if H > 1 else 0
    if P <= 1:
        sp = 0
    return code, (k_pages.data_ptr(), v_pages.data_ptr(), sp, sh, ss, P, page), (H, d)


def attn_cache_append(k, v, k_pages, v_pages, table, lengths, counts=None, q=None, inv_freq=None,
                      interleaved: bool = False, factor: float = 1.0, q_weight=None, k_weight=None, eps: float = 1e-6,
                      q_out=None, stream=None):
    """Write new tokens' keys and values (k, v [B, Hkv, L, d]) into the pages of a cache
    (k_pages, v_pages [pages, Hkv, page, d], or the same with another order in memory).
    table: int32 [B, width], the pages of each sequence; lengths: int32 [B], the tokens of each
    sequence AFTER the call; counts: int32 [B], how many of the L rows are new tokens (default
    all), at positions lengths - counts ...  With inv_freq (and q_weight, k_weight) the keys
    are rotated (and normalised) on the way as by attn_rope, and so is q [B, Hq, L, d], whose
    result is returned (q_out; zeros in rows behind counts).  Enqueued on `stream`."""
    code, cache, (Hkv, d) = _cache(k_pages, v_pages, k)
    if k.dim() != 4 or k.shape[1] != Hkv or k.shape[3] != d:
        raise ValueError("gbattn: k must be [B, Hkv, L, d] with the cache's Hkv and d")
    _check_like(v, "v", k, k.shape)
    B, _, L, _ = k.shape
    Hq = 0
    qr = _NO_ROWS
    if q is not None:
        if q.dim() != 4 or q.shape[0] != B or q.shape[2] != L or q.shape[3] != d:
            raise ValueError("gbattn: q must be [B, Hq, L, d] like k")
        _check_like(q, "q", k)
        Hq = q.shape[1]
        qr = _rows(q, "q")
        q_out = _out(q_out, "q_out", q.shape, q.dtype, q, stream)
    if table.dim() != 2:
        raise ValueError("gbattn: table must be [B, width]")
    tp, ts = _ints(table, "table", (B, table.shape[1]), k)
    lp, _ = _ints(lengths, "lengths", (B,), k)
    cp = _ints(counts, "counts", (B,), k)[0] if counts is not None else None
    fp, rotary = _frequencies(inv_freq, d, k)
    wq, wk = _norm_weights(q_weight, k_weight, d, k, q is not None, True)
    _launch("attn_cache_append", load_library().attn_cache_append, k.device, stream, *_rows(k, "k"), *_rows(v, "v"), *qr,
            q_out.data_ptr() if q is not None else None, *cache, tp, ts, table.shape[1], lp, cp, fp, rotary,
            int(bool(interleaved)), float(factor), wq, wk, float(eps), code, B, Hq, Hkv, L, d)
    return q_out if q is not None else None


def _page_list(x, name):
    if not isinstance(x, torch.Tensor):
        x = torch.tensor(list(x), dtype=torch.int32)
    if x.is_cuda or x.dtype != torch.int32 or x.dim() != 1 or not x.is_contiguous():
        raise ValueError(f"gbattn: {name} must be a list of page numbers or a contiguous int32 CPU tensor")
    return x


def attn_cache_copy(k_pages, v_pages, src, dst, stream=None) -> None:
    """Copy pages of a cache, keys and values: page src[i] to page dst[i], one after the other (also
    where a page occurs more than once).  src and dst are page numbers on the host (lists or
    int32 CPU tensors), read before the call returns.  Enqueued on `stream`."""
    _, cache, (Hkv, d) = _cache(k_pages, v_pages)
    src, dst = _page_list(src, "src"), _page_list(dst, "dst")
    if src.shape != dst.shape:
        raise ValueError("gbattn: src and dst must have the same length")
    _launch("attn_cache_copy", load_library().attn_cache_copy, k_pages.device, stream, *cache, Hkv, d, src.data_ptr(),
            dst.data_ptr(), src.shape[0])


def attn_decode_paged_workspace_bytes(Hq: int, Hkv: int, d: int) -> int:
    """Bytes of device workspace attn_decode_paged needs."""
    n = load_library().attn_decode_paged_workspace_bytes(int(Hq), int(Hkv), int(d))
    if n < 0:
        raise GbattnError(int(n), "attn_decode_paged_workspace_bytes")
    return int(n)


def attn_decode_paged(q, k_pages, v_pages, table, lengths, scale: float | None = None, o=None, lse=None, stream=None,
                      workspace=None):
    """Decode over a paged cache: O [B, Hq, d] and LSE [B, Hq] for one query row q ([B, Hq, d] or
    [B, Hq, 1, d]) per sequence and head against the lengths[b] tokens that table (int32
    [B, width]) finds in k_pages, v_pages [pages, Hkv, page, d]; Hq a multiple of Hkv.  An empty
    sequence gives zeros and -inf.  Outputs, and the workspace unless given (a contiguous CUDA
    tensor of attn_decode_paged_workspace_bytes bytes), are allocated by torch.  Enqueued on
    `stream`."""
    code, cache, (Hkv, d) = _cache(k_pages, v_pages, q)
    if q.dim() == 4 and q.shape[2] == 1:
        q = q[:, :, 0]
    if q.dim() != 3 or q.shape[2] != d:
        raise ValueError("gbattn: q must be [B, Hq, d] or [B, Hq, 1, d] with the cache's d")
    B, Hq, _ = q.shape
    if q.stride(2) != 1:
        raise ValueError("gbattn: the last dimension of q must be contiguous")
    if table.dim() != 2:
        raise ValueError("gbattn: table must be [B, width]")
    tp, ts = _ints(table, "table", (B, table.shape[1]), q)
    lp, _ = _ints(lengths, "lengths", (B,), q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    o = _out(o, "o", (B, Hq, d), q.dtype, q, stream)
    lse = _out(lse, "lse", (B, Hq), torch.float32, q, stream)
    lib = load_library()
    nbytes = lib.attn_decode_paged_workspace_bytes(Hq, Hkv, d)
    if nbytes < 0:
        raise GbattnError(int(nbytes), "attn_decode_paged_workspace_bytes")
    workspace = _workspace(workspace, nbytes, q, stream)
    _launch("attn_decode_paged", lib.attn_decode_paged, q.device, stream, q.data_ptr(), q.stride(0) if B > 1 else 0,
            q.stride(1) if Hq > 1 else 0, *cache, tp, ts, table.shape[1], lp, o.data_ptr(), lse.data_ptr(),
            workspace.data_ptr(), code, B, Hq, Hkv, d, float(scale))
    return o, lse
