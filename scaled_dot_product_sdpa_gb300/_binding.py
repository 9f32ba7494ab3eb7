"""ctypes binding of libgbattn.so: argument marshalling only.

Every function here converts torch tensors to raw device pointers and sizes, calls the
C entry point of the same name (include/gbattn.h), and turns a nonzero return code into
a GbattnError.  There is no fallback: if the library is missing or the tensors are not
on a CUDA device, the call raises.
"""
from __future__ import annotations

import array
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
# belongs to the stream that it runs on.  A decoding step makes several of these calls, each
# worth a few microseconds on the GPU, so the checks read each property of a tensor once.
_DTYPES = {torch.float16: 0, torch.bfloat16: 1}
# Private names of torch, each with the public way beside it (a torch without CUDA lacks them).
# Of a device index; torch.cuda.current_stream costs 3 us.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# torch.empty without its argument parser, on the current device (0.9 us a tensor instead of 1.5, and more between
# launches: attn_decode_paged 22.0 us a call, with this 18.8, attn_rope 16.7 and 13.4); None: torch.empty.
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


def _empty(shape, dtype, like, stream):
    """An uninitialised tensor of 1 to 4 dimensions on the device of `like` that belongs to `stream`."""
    if stream is None:
        if _empty_strided is not None and like.get_device() == _current_device():
            n = len(shape)
            if n == 4:
                a, b, c, d = shape
                return _empty_strided((a, b, c, d), (b * c * d, c * d, d, 1), dtype)
            if n == 3:
                a, b, c = shape
                return _empty_strided((a, b, c), (b * c, c, 1), dtype)
            return _empty_strided(shape, (shape[1], 1) if n == 2 else (1,), dtype)
        return torch.empty(shape, dtype=dtype, device=like.device)
    device = like.device
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device) if int(stream) else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _launch(what, fn, dev, stream, *args):
    """Call the C entry point `fn` with device `dev` current and its stream as last argument."""
    handle = _current_stream(dev) if stream is None else _stream_handle(stream)
    if dev == _current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    if rc != 0:
        raise GbattnError(rc, what)


def _device_and_type(t, name):
    """Device index and type code of a call's first tensor."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("gbattn: tensors must be on a CUDA device (no CPU path exists)")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"gbattn: {name} must be float16 or bfloat16")
    return dev, code


def _check_like(t, name, dev, dtype):
    if t.get_device() != dev:
        raise ValueError(f"gbattn: {name} must be on the CUDA device of the other tensors (no CPU path exists)")
    if t.dtype != dtype:
        raise ValueError(f"gbattn: {name} must be {dtype} like the other tensors")


def _rows(t, name, shape):
    """Pointer and strides of batch, head and row of [B, H, L, d] rows; the last dimension must be
    contiguous, the strides of dimensions of one element do not matter."""
    sb, sh, sl, sd = t.stride()
    if sd != 1:
        raise ValueError(f"gbattn: the last dimension of {name} must be contiguous")
    B, H, L, _ = shape
    return t.data_ptr(), (sb if B > 1 else 0), (sh if H > 1 else 0), (sl if L > 1 else 0)


_NO_ROWS = (None, 0, 0, 0)


def _check_out(t, name, shape, dtype, dev):
    if t.shape != shape or t.dtype != dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"gbattn: {name} must be contiguous {dtype} {tuple(shape)} on the device of the other tensors")
    return t


def _ints(t, name, n, dev):
    """Pointer of an int32 [n] device tensor."""
    if t.dtype != torch.int32 or t.get_device() != dev or t.shape != (n,):
        raise ValueError(f"gbattn: {name} must be int32 {(n,)} on the device of the other tensors")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"gbattn: {name} must be contiguous")
    return t.data_ptr()


def _int_rows(t, name, B, dev, width=None):
    """Pointer, row stride and width of an int32 [B, width] device tensor with contiguous rows."""
    shape = t.shape
    if t.dtype != torch.int32 or t.get_device() != dev or len(shape) != 2 or shape[0] != B or (width is not None and shape[1] != width):
        raise ValueError(f"gbattn: {name} must be int32 [{B}, {'width' if width is None else width}] on the device of the other tensors")
    sr, sc = t.stride()
    if sc != 1 and shape[1] > 1:
        raise ValueError(f"gbattn: the last dimension of {name} must be contiguous")
    return t.data_ptr(), (sr if B > 1 else 0), shape[1]


def _frequencies(inv_freq, dev):
    """Pointer and rotary width of the inverse frequencies (None: nothing is rotated)."""
    if inv_freq is None:
        return None, 0
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or inv_freq.get_device() != dev or not inv_freq.is_contiguous():
        raise ValueError("gbattn: inv_freq must be contiguous float64 [rotary / 2] on the device of the other tensors")
    n = 2 * inv_freq.shape[0]
    return (inv_freq.data_ptr() if n else None), n


def _weight(t, name, d, dev, dtype):
    _check_like(t, name, dev, dtype)
    if t.shape != (d,) or not t.is_contiguous():
        raise ValueError(f"gbattn: {name} must be contiguous [{d}]")
    return t.data_ptr()


def _norm_weights(q_weight, k_weight, d, dev, dtype, has_q, has_k):
    if q_weight is None and k_weight is None:
        return None, None
    if (q_weight is None) == has_q or (k_weight is None) == has_k:
        raise ValueError("gbattn: norms need a weight for each tensor that is normalised")
    return (_weight(q_weight, "q_weight", d, dev, dtype) if has_q else None,
            _weight(k_weight, "k_weight", d, dev, dtype) if has_k else None)


def _rope_positions(positions, B, L, dev):
    if positions is None:
        return None, 0
    if positions.dim() == 1:
        return _ints(positions, "positions", L, dev), 0
    return _int_rows(positions, "positions", B, dev, L)[:2]


def _workspace(workspace, nbytes, like, dev, stream):
    if workspace is None:
        return _empty((nbytes // 4,), torch.float32, like, stream)
    if (workspace.get_device() != dev or not workspace.is_contiguous()
            or workspace.numel() * workspace.element_size() < nbytes):
        raise ValueError(f"gbattn: workspace must be a contiguous CUDA tensor of at least {nbytes} bytes on the device "
                         "of the other tensors")
    return workspace


def attn_rope(q, k, inv_freq, positions=None, interleaved: bool = False, factor: float = 1.0, q_weight=None,
              k_weight=None, eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """Rotary positions, and with q_weight and k_weight ([d]) per-head RMS norms before them, of
    q [B, Hq, L, d] and k [B, Hkv, L, d] (k None: q alone), fp16 or bf16, in one pass.  Rows may
    lie anywhere (a transposed [B, L, H, d] projection, a slice of a joint one) as long as each
    is contiguous; the outputs (q_out, k_out) are contiguous [B, H, L, d], as attn_fwd takes them.
    inv_freq: float64 [rotary / 2] (attn_rope_frequencies), rotary a multiple of 16 up to d;
    positions: int32 [B, L] or [L], default 0 .. L-1; interleaved: pairs (2r, 2r + 1) instead of
    (r, r + rotary / 2); factor multiplies cosine and sine.  Enqueued on `stream`."""
    dev, code = _device_and_type(q, "q")
    dtype, shape = q.dtype, q.shape
    if len(shape) != 4:
        raise ValueError("gbattn: q must be [B, H, L, d]")
    B, Hq, L, d = shape
    Hkv, kr, k_to = 0, _NO_ROWS, None
    if k is not None:
        k_shape = k.shape
        if len(k_shape) != 4 or k_shape[0] != B or k_shape[2] != L or k_shape[3] != d:
            raise ValueError("gbattn: k must be [B, Hkv, L, d] like q")
        _check_like(k, "k", dev, dtype)
        Hkv, kr = k_shape[1], _rows(k, "k", k_shape)
        k_out = _empty(k_shape, dtype, q, stream) if k_out is None else _check_out(k_out, "k_out", k_shape, dtype, dev)
        k_to = k_out.data_ptr()
    else:
        k_out = None
    fp, rotary = _frequencies(inv_freq, dev)
    pp, ps = _rope_positions(positions, B, L, dev)
    wq, wk = _norm_weights(q_weight, k_weight, d, dev, dtype, True, k is not None)
    q_out = _empty(shape, dtype, q, stream) if q_out is None else _check_out(q_out, "q_out", shape, dtype, dev)
    _launch("attn_rope", (_lib or load_library()).attn_rope, dev, stream, *_rows(q, "q", shape), *kr, q_out.data_ptr(), k_to,
            fp, rotary, bool(interleaved), float(factor), pp, ps, wq, wk, float(eps), code, B, Hq, Hkv, L, d)
    return q_out, k_out


def attn_rope_bwd(dq, dk, inv_freq, positions=None, interleaved: bool = False, factor: float = 1.0, q=None, k=None,
                  q_weight=None, k_weight=None, eps: float = 1e-6, dq_out=None, dk_out=None, dq_weight=None,
                  dk_weight=None, stream=None, workspace=None):
    """Gradients of attn_rope: from dq [B, Hq, L, d] and dk [B, Hkv, L, d] (of its outputs; attn_bwd's
    results; dk None without keys) those of its inputs, contiguous: (dq_out, dk_out).  With norms, q and k
    are attn_rope's inputs and the result is (dq_out, dk_out, dq_weight, dk_weight), the weights'
    gradients in float32 [d].  The other arguments are attn_rope's."""
    dev, code = _device_and_type(dq, "dq")
    dtype, shape = dq.dtype, dq.shape
    if len(shape) != 4:
        raise ValueError("gbattn: dq must be [B, H, L, d]")
    B, Hq, L, d = shape
    Hkv, kr, k_to = 0, _NO_ROWS, None
    if dk is not None:
        k_shape = dk.shape
        if len(k_shape) != 4 or k_shape[0] != B or k_shape[2] != L or k_shape[3] != d:
            raise ValueError("gbattn: dk must be [B, Hkv, L, d] like dq")
        _check_like(dk, "dk", dev, dtype)
        Hkv, kr = k_shape[1], _rows(dk, "dk", k_shape)
        dk_out = _empty(k_shape, dtype, dq, stream) if dk_out is None else _check_out(dk_out, "dk_out", k_shape, dtype, dev)
        k_to = dk_out.data_ptr()
    else:
        dk_out = None
    fp, rotary = _frequencies(inv_freq, dev)
    pp, ps = _rope_positions(positions, B, L, dev)
    wq, wk = _norm_weights(q_weight, k_weight, d, dev, dtype, True, dk is not None)
    lib = _lib or load_library()
    xq = xk = _NO_ROWS
    wq_to = wk_to = ws = None
    if wq is not None:
        if q is None or (dk is not None) != (k is not None):
            raise ValueError("gbattn: the gradients of norms need attn_rope's inputs q and k")
        _check_like(q, "q", dev, dtype)
        if q.shape != shape or (k is not None and k.shape != k_shape):
            raise ValueError("gbattn: q and k must have the shapes of dq and dk")
        xq = _rows(q, "q", shape)
        dq_weight = _empty((d,), torch.float32, dq, stream) if dq_weight is None else _check_out(dq_weight, "dq_weight", (d,), torch.float32, dev)
        wq_to = dq_weight.data_ptr()
        if k is not None:
            _check_like(k, "k", dev, dtype)
            xk = _rows(k, "k", k_shape)
            dk_weight = _empty((d,), torch.float32, dq, stream) if dk_weight is None else _check_out(dk_weight, "dk_weight", (d,), torch.float32, dev)
            wk_to = dk_weight.data_ptr()
        nbytes = lib.attn_rope_bwd_workspace_bytes(d)
        if nbytes < 0:
            raise GbattnError(int(nbytes), "attn_rope_bwd_workspace_bytes")
        workspace = _workspace(workspace, nbytes, dq, dev, stream)
        ws = workspace.data_ptr()
    dq_out = _empty(shape, dtype, dq, stream) if dq_out is None else _check_out(dq_out, "dq_out", shape, dtype, dev)
    _launch("attn_rope_bwd", lib.attn_rope_bwd, dev, stream, *_rows(dq, "dq", shape), *kr, *xq, *xk, dq_out.data_ptr(), k_to,
            wq_to, wk_to, fp, rotary, bool(interleaved), float(factor), pp, ps, wq, wk, float(eps), ws, code, B, Hq, Hkv, L, d)
    if wq is None:
        return dq_out, dk_out
    return dq_out, dk_out, dq_weight, (dk_weight if dk is not None else None)


def attn_rope_bwd_workspace_bytes(d: int) -> int:
    """Bytes of device workspace attn_rope_bwd needs with norms."""
    n = load_library().attn_rope_bwd_workspace_bytes(int(d))
    if n < 0:
        raise GbattnError(int(n), "attn_rope_bwd_workspace_bytes")
    return int(n)


def _cache(k_pages, v_pages):
    """Device index, type code, shape, and (k pointer, v pointer, page, head and slot strides, pages, slots of a page)."""
    dev, code = _device_and_type(k_pages, "k_pages")
    shape = k_pages.shape
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("gbattn: k_pages and v_pages must share one [pages, Hkv, page, d] shape")
    if v_pages.dtype != k_pages.dtype or v_pages.get_device() != dev:
        raise ValueError("gbattn: k_pages and v_pages must share their type and device")
    P, H, page, _ = shape
    strides, v_strides = k_pages.stride(), v_pages.stride()
    sp, sh, ss, sd = strides
    if sd != 1 or v_strides[3] != 1:
        raise ValueError("gbattn: the last dimension of k_pages and v_pages must be contiguous")
    if v_strides != strides and any(n > 1 and a != b for n, a, b in zip(shape, strides, v_strides)):
        raise ValueError("gbattn: k_pages and v_pages must share their strides")
    return dev, code, shape, (k_pages.data_ptr(), v_pages.data_ptr(), sp if P > 1 else 0, sh if H > 1 else 0, ss, P, page)


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
    dev, code, (_, Hkv, _, d), cache = _cache(k_pages, v_pages)
    dtype, shape = k_pages.dtype, k.shape
    if len(shape) != 4 or shape[1] != Hkv or shape[3] != d or v.shape != shape:
        raise ValueError("gbattn: k and v must be [B, Hkv, L, d] with the cache's Hkv and d")
    _check_like(k, "k", dev, dtype)
    _check_like(v, "v", dev, dtype)
    B, _, L, _ = shape
    Hq, qr, q_to = 0, _NO_ROWS, None
    if q is not None:
        q_shape = q.shape
        if len(q_shape) != 4 or q_shape[0] != B or q_shape[2] != L or q_shape[3] != d:
            raise ValueError("gbattn: q must be [B, Hq, L, d] like k")
        _check_like(q, "q", dev, dtype)
        Hq, qr = q_shape[1], _rows(q, "q", q_shape)
        q_out = _empty(q_shape, dtype, q, stream) if q_out is None else _check_out(q_out, "q_out", q_shape, dtype, dev)
        q_to = q_out.data_ptr()
    tp, ts, tw = _int_rows(table, "table", B, dev)
    lp = _ints(lengths, "lengths", B, dev)
    cp = _ints(counts, "counts", B, dev) if counts is not None else None
    fp, rotary = _frequencies(inv_freq, dev)
    wq, wk = _norm_weights(q_weight, k_weight, d, dev, dtype, q is not None, True)
    _launch("attn_cache_append", (_lib or load_library()).attn_cache_append, dev, stream, *_rows(k, "k", shape),
            *_rows(v, "v", shape), *qr, q_to, *cache, tp, ts, tw, lp, cp, fp, rotary, bool(interleaved), float(factor), wq, wk, float(eps),
            code, B, Hq, Hkv, L, d)
    return q_out if q is not None else None


def _page_list(x, name):
    """Address and length of page numbers on the host, and what keeps them there."""
    if not isinstance(x, torch.Tensor):
        x = array.array("i", x if type(x) is list else list(x))
        return x.buffer_info()[0], len(x), x
    if x.is_cuda or x.dtype != torch.int32 or x.dim() != 1 or not x.is_contiguous():
        raise ValueError(f"gbattn: {name} must be a list of page numbers or a contiguous int32 CPU tensor")
    return x.data_ptr(), x.shape[0], x


def attn_cache_copy(k_pages, v_pages, src, dst, stream=None) -> None:
    """Copy pages of a cache, keys and values: page src[i] to page dst[i], one after the other (also
    where a page occurs more than once).  src and dst are page numbers on the host (lists or
    int32 CPU tensors), read before the call returns.  Enqueued on `stream`."""
    dev, _, (_, Hkv, _, d), cache = _cache(k_pages, v_pages)
    (src_at, n, src), (dst_at, m, dst) = _page_list(src, "src"), _page_list(dst, "dst")
    if n != m:
        raise ValueError("gbattn: src and dst must have the same length")
    _launch("attn_cache_copy", (_lib or load_library()).attn_cache_copy, dev, stream, *cache, Hkv, d, src_at, dst_at, n)


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
    sequence gives zeros and -inf.  Sums in float32; the weights that meet the values keep 22 bits
    with float16 and 16 with bfloat16.  Outputs, and the workspace unless given (a contiguous CUDA
    tensor of attn_decode_paged_workspace_bytes bytes), are allocated by torch.  Enqueued on
    `stream`."""
    dev, code, (_, Hkv, _, d), cache = _cache(k_pages, v_pages)
    shape, strides = q.shape, q.stride()
    if len(shape) not in (3, 4) or shape[-1] != d or (len(shape) == 4 and shape[2] != 1):
        raise ValueError("gbattn: q must be [B, Hq, d] or [B, Hq, 1, d] with the cache's d")
    _check_like(q, "q", dev, k_pages.dtype)
    B, Hq = shape[0], shape[1]
    if strides[-1] != 1:
        raise ValueError("gbattn: the last dimension of q must be contiguous")
    tp, ts, tw = _int_rows(table, "table", B, dev)
    lp = _ints(lengths, "lengths", B, dev)
    o = _empty((B, Hq, d), q.dtype, q, stream) if o is None else _check_out(o, "o", (B, Hq, d), q.dtype, dev)
    lse = _empty((B, Hq), torch.float32, q, stream) if lse is None else _check_out(lse, "lse", (B, Hq), torch.float32, dev)
    lib = _lib or load_library()
    nbytes = lib.attn_decode_paged_workspace_bytes(Hq, Hkv, d)
    if nbytes < 0:
        raise GbattnError(int(nbytes), "attn_decode_paged_workspace_bytes")
    workspace = _workspace(workspace, nbytes, q, dev, stream)
    _launch("attn_decode_paged", lib.attn_decode_paged, dev, stream, q.data_ptr(), strides[0] if B > 1 else 0,
            strides[1] if Hq > 1 else 0, *cache, tp, ts, tw, lp, o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), code, B, Hq,
            Hkv, d, 1.0 / math.sqrt(d) if scale is None else float(scale))
    return o, lse
