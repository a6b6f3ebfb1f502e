"""ctypes binding of libltxattn.so (the C ABI in include/ltxattn.h).

Argument marshalling only: torch tensors are checked for dtype, device, shape and
contiguity, and their device pointers are passed to the library together with
the current CUDA stream.  There is no fallback: if the library is missing or a
call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import re
import struct
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
# LTXATTN_DEBUG=1 selects the guard-word build (libltxattn_debug.so, see build.build(debug=True))
LIB_PATH = os.path.join(_PKG, "libltxattn_debug.so" if os.environ.get("LTXATTN_DEBUG") == "1"
                        else "libltxattn.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "ltxattn.h")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_MISALIGNED, ERR_CUDA, ERR_DEVICE_TIMEOUT, \
    ERR_NOT_INITIALIZED, ERR_WORKSPACE_GUARD = range(8)

_lock = threading.Lock()
_lib = None


class LtxAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class _RopeCall(ctypes.Structure):
    """``ltxattn_rope_call`` of include/ltxattn.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "q_out", "k_out")]
                + [(n, ctypes.c_longlong * 3)
                   for n in ("q_stride", "k_stride", "q_out_stride", "k_out_stride")]
                + [("positions", ctypes.c_void_p), ("inv_freq", ctypes.POINTER(ctypes.c_double)),
                   ("axis_dims", ctypes.c_int * 4)]
                + [(n, ctypes.c_int) for n in ("axes", "positions_batch", "batch", "len", "heads",
                                               "kv_heads", "head_dim", "dtype", "layout",
                                               "inverse")])


class _MaskedCall(ctypes.Structure):
    """``ltxattn_masked_call`` of include/ltxattn.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("q", "k", "v", "out", "lse")]
                + [(n, ctypes.c_longlong * 3)
                   for n in ("q_stride", "k_stride", "v_stride", "out_stride")]
                + [(n, ctypes.c_int) for n in ("batch", "q_len", "kv_len", "heads", "kv_heads",
                                               "head_dim")]
                + [("scale", ctypes.c_float), ("softcap", ctypes.c_float)]
                + [(n, ctypes.c_void_p) for n in ("slopes", "prefix", "q_starts", "kv_starts")]
                + [("docs", ctypes.c_int), ("causal", ctypes.c_int)])


class _MaskedGrad(ctypes.Structure):
    """``ltxattn_masked_grad`` of include/ltxattn.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("d_out", "dq", "dk", "dv")]
                + [(n, ctypes.c_longlong * 3)
                   for n in ("d_out_stride", "dq_stride", "dk_stride", "dv_stride")])


def _packer(cls):
    """``struct.Struct`` of a ctypes structure's fields, arrays spelled out: packing a call's
    arguments into bytes takes a third of the time of filling the structure."""
    codes = {ctypes.c_void_p: "P", ctypes.c_longlong: "q", ctypes.c_int: "i",
             ctypes.c_float: "f"}
    fmt = "@"
    for _, kind in cls._fields_:
        if issubclass(kind, ctypes.Array):
            fmt += f"{kind._length_}{codes[kind._type_]}"
        else:
            fmt += codes.get(kind, "P")
    packer = struct.Struct(fmt)
    assert packer.size <= ctypes.sizeof(cls)  # a trailing pad at most
    return packer.pack


_pack_rope, _pack_masked, _pack_grad = (_packer(c) for c in (_RopeCall, _MaskedCall, _MaskedGrad))


def load() -> ctypes.CDLL:
    """Load libltxattn.so (built by ``joint_audio_video_flash_b200.build``); raise if absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"{LIB_PATH} is missing: run joint_audio_video_flash_b200.build"
                                  + (" with debug=True" if LIB_PATH.endswith("_debug.so") else ""))
            lib = ctypes.CDLL(LIB_PATH)
            vp, ci, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
            lib.ltxattn_create.argtypes = []
            lib.ltxattn_forward.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, vp]
            lib.ltxattn_forward_ex.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci,
                                               ctypes.POINTER(ci), vp]
            lib.ltxattn_check.argtypes = [vp]
            lib.ltxattn_destroy.argtypes = []
            lib.ltxattn_status_string.argtypes = [ci]
            lib.ltxattn_status_string.restype = ctypes.c_char_p
            lib.ltxattn_selftest_wait_timeout.argtypes = [ctypes.c_ulonglong, vp]
            lib.ltxattn_num_entry_points.argtypes = []
            lib.ltxattn_qk_norm_rope.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci,
                                                 cf, vp]
            lib.ltxattn_na3d_forward.argtypes = [vp, vp, vp, vp] + [ci] * 9 + [cf, vp]
            lib.ltxattn_na3d_plan.argtypes = [ci] * 6 + [vp, vp]
            lib.ltxattn_forward_plan.argtypes = [ci] * 8 + [vp, vp]
            lib.ltxattn_forward_partial.argtypes = [vp, vp, vp, vp, vp] + [ci] * 6 + [cf, vp]
            lib.ltxattn_combine.argtypes = [vp, vp, vp] + [ci] * 5 + [vp]
            lib.ltxattn_forward_grouped.argtypes = [vp, ci, vp]
            ll, ull = ctypes.c_longlong, ctypes.c_ulonglong
            lib.ltxattn_rope_axes.argtypes = [vp, vp]  # the structs: packed bytes
            lib.ltxattn_layer_norm.argtypes = [vp] * 6 + [ll, ci, ll, ll, ll, cf, ci, vp]
            lib.ltxattn_layer_norm_workspace.argtypes = [ll, ci, ll, ci, ctypes.POINTER(ull)]
            lib.ltxattn_layer_norm_backward.argtypes = ([vp] * 8 + [ll, ci] + [ll] * 4
                                                        + [ci, vp, ull, vp])
            lib.ltxattn_masked_forward.argtypes = [vp, vp, ull, vp]
            lib.ltxattn_masked_backward.argtypes = [vp, vp, vp, ull, vp]
            lib.ltxattn_masked_workspace.argtypes = [vp, ci, ctypes.POINTER(ull)]
            lib.ltxattn_entry_point_name.argtypes = [ci]
            lib.ltxattn_entry_point_name.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def header_entry_points() -> list[str]:
    """Function names declared in include/ltxattn.h."""
    with open(HEADER) as f:
        text = f.read()
    return re.findall(r"^\s*(?:LTXATTN_API\s+)?(?:int|const char\*)\s+(ltxattn_\w+)\s*\(", text, flags=re.M)


def status_string(status: int) -> str:
    return load().ltxattn_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != OK:
        raise LtxAttnError(status, where)


def create() -> None:
    _check((_lib or load()).ltxattn_create(), "ltxattn_create")


def destroy() -> None:
    _check(load().ltxattn_destroy(), "ltxattn_destroy")


def _stream_handle(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def check(stream=None) -> None:
    """Synchronise the stream and raise if a kernel recorded a stalled wait."""
    _check(load().ltxattn_check(ctypes.c_void_p(_stream_handle(stream))), "ltxattn_check")


def selftest_wait_timeout(timeout_ns: int = 1_000_000, stream=None) -> int:
    """Run the bounded-wait self-test; returns the raw status (DEVICE_TIMEOUT expected)."""
    return int(load().ltxattn_selftest_wait_timeout(ctypes.c_ulonglong(int(timeout_ns)),
                                                      ctypes.c_void_p(_stream_handle(stream))))


def _check_attention_tensors(q, k, v, out) -> None:
    """Checks the library cannot make from raw pointers: bf16, contiguous 4-D BSHD, k and v
    shaped [batch, kv_len, heads, head_dim] like q, out shaped like q, every tensor on the
    current CUDA device (the C ABI works on the current device's context).  `out` may be
    None (checked later, once allocated)."""
    import torch
    named = [("q", q), ("k", k), ("v", v)] + ([("out", out)] if out is not None else [])
    for name, t in named:
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [batch, len, heads, head_dim] tensor")
        if t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, not on the current device "
                             f"cuda:{torch.cuda.current_device()}")
    batch, _, heads, head_dim = q.shape
    kv_len = k.shape[1]
    if tuple(k.shape) != (batch, kv_len, heads, head_dim) or v.shape != k.shape:
        raise ValueError("k and v must be [batch, kv_len, heads, head_dim] matching q")
    if out is not None and out.shape != q.shape:
        raise ValueError("out must be shaped like q")


def forward(q, k, v, out=None, *, kv_valid_len: int | None = None, scale: float | None = None,
            num_splits: int = 0, stream=None, return_splits: bool = False):
    """O = softmax(scale q k^T, keys < kv_valid_len) v for bf16 BSHD CUDA tensors.

    q: [B, Lq, H, D]; k, v: [B, Lkv, H, D]; out (optional): [B, Lq, H, D].
    """
    import torch
    if out is None:
        _check_attention_tensors(q, k, v, None)
        out = torch.empty_like(q)
    _check_attention_tensors(q, k, v, out)
    batch, q_len, heads, head_dim = q.shape
    kv_len = k.shape[1]
    if kv_valid_len is None:
        kv_valid_len = kv_len
    if scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    used = ctypes.c_int(0)
    st = load().ltxattn_forward_ex(
        ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
        ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()), int(q_len), int(kv_len),
        int(kv_valid_len), int(batch), int(heads), int(head_dim), ctypes.c_float(scale),
        int(num_splits), ctypes.byref(used), ctypes.c_void_p(_stream_handle(stream)))
    _check(st, "ltxattn_forward")
    return (out, used.value) if return_splits else out


class _Call(ctypes.Structure):
    """``ltxattn_call`` of include/ltxattn.h."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("q_len", ctypes.c_int), ("kv_len", ctypes.c_int),
                ("kv_valid_len", ctypes.c_int), ("batch", ctypes.c_int),
                ("heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("scale", ctypes.c_float)]


def forward_grouped(calls, *, stream=None):
    """Several independent attention calls through ``ltxattn_forward_grouped``.

    ``calls``: a sequence of dicts with keys q, k, v, out (tensors as for ``forward``; out
    required) and optional kv_valid_len and scale.  Calls at head_dim 64 whose valid keys
    fit in one 128-key tile (a2v, audio self-attention) share one launch.  Returns the
    list of outputs.
    """
    arr = (_Call * len(calls))()
    outs = []
    for i, c in enumerate(calls):
        q, k, v, out = c["q"], c["k"], c["v"], c["out"]
        _check_attention_tensors(q, k, v, out)
        batch, q_len, heads, head_dim = q.shape
        kv_len = k.shape[1]
        kv_valid = c.get("kv_valid_len")
        scale = c.get("scale")
        arr[i] = _Call(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), int(q_len),
                       int(kv_len), int(kv_len if kv_valid is None else kv_valid), int(batch),
                       int(heads), int(head_dim),
                       float(1.0 / math.sqrt(head_dim) if scale is None else scale))
        outs.append(out)
    st = load().ltxattn_forward_grouped(ctypes.cast(arr, ctypes.c_void_p), len(calls),
                                        ctypes.c_void_p(_stream_handle(stream)))
    _check(st, "ltxattn_forward_grouped")
    return outs


def forward_split_noalloc(q, k, v, out, *, kv_valid_len: int | None = None,
                          scale: float | None = None, num_splits: int = 0, stream=None) -> int:
    """Key-split forward that allocates no device memory (``ltxattn_forward_split_noalloc``).

    For callers that must not let the library allocate (a plugin host that owns all
    device memory, a serving loop with a fixed memory plan, a hard memory quota):
    key-split fp32 partials go to the library's built-in 16 MiB scratch array (one key
    part needs none).  ``out`` is required (this call allocates nothing, not even the
    output).  Tensors are checked as for ``forward``.  Returns the raw status; calls whose
    GPU work overlaps race on the shared scratch; ``check()`` reports a kernel wait that
    ran out in the last such call.
    """
    _check_attention_tensors(q, k, v, out)
    lib = load()
    fn = lib.ltxattn_forward_split_noalloc
    vp, ci = ctypes.c_void_p, ctypes.c_int
    fn.argtypes = [vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ctypes.c_float, ci, vp]
    batch, q_len, heads, head_dim = q.shape
    kv_len = k.shape[1]
    if kv_valid_len is None:
        kv_valid_len = kv_len
    if scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    return int(fn(vp(q.data_ptr()), vp(k.data_ptr()), vp(v.data_ptr()), vp(out.data_ptr()),
                  int(q_len), int(kv_len), int(kv_valid_len), int(batch), int(heads),
                  int(head_dim), ctypes.c_float(scale), int(num_splits),
                  vp(_stream_handle(stream))))


def qk_norm_rope(q, k, q_weight, k_weight, cos, sin, q_out=None, k_out=None, *,
                 eps: float = 1e-6, stream=None):
    """Norm and rotary step of queries and keys (``ltxattn_qk_norm_rope``); returns (q', k').

    q, k: bf16 CUDA [B, L, H, D]; weights: bf16 [H * D]; cos, sin: fp32 [L, D / 2].  The
    outputs may be the inputs (in place).
    """
    import torch
    for name, t in (("q", q), ("k", k)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda \
                or t.dim() != 4 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous bf16 CUDA [batch, len, heads, dim] tensor")
    if k.shape != q.shape:
        raise ValueError("q and k must have the same shape")
    batch, seq_len, heads, head_dim = q.shape
    for name, t, dt, shape in (("q_weight", q_weight, torch.bfloat16, (heads * head_dim,)),
                               ("k_weight", k_weight, torch.bfloat16, (heads * head_dim,)),
                               ("cos", cos, torch.float32, (seq_len, head_dim // 2)),
                               ("sin", sin, torch.float32, (seq_len, head_dim // 2))):
        if (not isinstance(t, torch.Tensor) or t.dtype != dt or not t.is_cuda
                or tuple(t.shape) != shape or not t.is_contiguous()):
            raise TypeError(f"{name} must be a contiguous {dt} CUDA tensor of shape {shape}")
    q_out = torch.empty_like(q) if q_out is None else q_out
    k_out = torch.empty_like(k) if k_out is None else k_out
    for name, t in (("q_out", q_out), ("k_out", k_out)):
        if t.dtype != torch.bfloat16 or t.shape != q.shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 tensor shaped like q")
    st = load().ltxattn_qk_norm_rope(
        ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
        ctypes.c_void_p(q_out.data_ptr()), ctypes.c_void_p(k_out.data_ptr()),
        ctypes.c_void_p(q_weight.data_ptr()), ctypes.c_void_p(k_weight.data_ptr()),
        ctypes.c_void_p(cos.data_ptr()), ctypes.c_void_p(sin.data_ptr()), int(batch),
        int(seq_len), int(heads), int(head_dim), ctypes.c_float(eps),
        ctypes.c_void_p(_stream_handle(stream)))
    _check(st, "ltxattn_qk_norm_rope")
    return q_out, k_out


def na3d_forward(q, k, v, grid, window, out=None, *, scale: float | None = None, stream=None):
    """3-D neighbourhood attention (``ltxattn_na3d_forward``) of bf16 CUDA tensors.

    q, k, v: [B, T*Y*X, H, D] with tokens in raster order of the grid (T, Y, X); window
    (kT, kY, kX): odd sizes, each at most its grid axis.  Returns out [B, T*Y*X, H, D].
    """
    import torch
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
        if t.dim() != 4 or not t.is_contiguous() or t.shape != q.shape:
            raise ValueError(f"{name} must be a contiguous [batch, tokens, heads, head_dim] "
                             "tensor shaped like q")
    grid_t, grid_y, grid_x = (int(x) for x in grid)
    win_t, win_y, win_x = (int(x) for x in window)
    batch, tokens, heads, head_dim = q.shape
    if tokens != grid_t * grid_y * grid_x:
        raise ValueError(f"{tokens} tokens but grid {tuple(grid)}")
    if out is None:
        out = torch.empty_like(q)
    elif (out.dtype != torch.bfloat16 or out.shape != q.shape or not out.is_contiguous()
          or out.device != q.device):
        raise ValueError("out must be a contiguous bf16 tensor shaped like q on q's device")
    if scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    st = load().ltxattn_na3d_forward(
        ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
        ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(out.data_ptr()), int(batch), grid_t,
        grid_y, grid_x, int(heads), int(head_dim), win_t, win_y, win_x, ctypes.c_float(scale),
        ctypes.c_void_p(_stream_handle(stream)))
    _check(st, "ltxattn_na3d_forward")
    return out


# ltxattn_kernel values
KERNEL_ONE_TILE, KERNEL_TWO_TILES, KERNEL_ONE_TILE_DUAL = 0, 1, 2
KERNEL_SHORT_KV, KERNEL_A2V, KERNEL_PAIR = 3, 4, 5


def forward_plan(q_len: int, kv_len: int, kv_valid_len: int, batch: int, heads: int,
                 head_dim: int, num_splits: int = 0, num_sms: int = 148):
    """The kernel ``ltxattn_forward`` runs for these sizes and its key-range parts
    (``ltxattn_forward_plan``, host only): (one of the KERNEL_* values, parts)."""
    kernel = ctypes.c_int()
    parts = ctypes.c_int()
    st = load().ltxattn_forward_plan(int(q_len), int(kv_len), int(kv_valid_len), int(batch),
                                     int(heads), int(head_dim), int(num_splits), int(num_sms),
                                     ctypes.cast(ctypes.pointer(kernel), ctypes.c_void_p),
                                     ctypes.cast(ctypes.pointer(parts), ctypes.c_void_p))
    _check(st, "ltxattn_forward_plan")
    return kernel.value, parts.value


def na3d_plan(grid, window):
    """The blocking ``ltxattn_na3d_forward`` uses (``ltxattn_na3d_plan``, host only): the
    query brick (t, y, x), the key tile (t, y, x) and the key tiles per (batch, head)."""
    shape = (ctypes.c_int * 6)()
    tiles = ctypes.c_longlong()
    st = load().ltxattn_na3d_plan(*(int(x) for x in grid), *(int(x) for x in window),
                                  ctypes.cast(shape, ctypes.c_void_p),
                                  ctypes.cast(ctypes.pointer(tiles), ctypes.c_void_p))
    _check(st, "ltxattn_na3d_plan")
    return tuple(shape[:3]), tuple(shape[3:]), int(tiles.value)


def rows_pad(q_len: int) -> int:
    """Query rows per (batch, head) in the partial-result layout: q_len rounded up to 128."""
    return -(-int(q_len) // 128) * 128


def forward_partial(q, k, v, o_part=None, lse=None, *, kv_valid_len: int | None = None,
                    scale: float | None = None, stream=None):
    """Attention over one key range (``ltxattn_forward_partial``): returns (o_part, lse).

    q: [B, Lq, H, D]; k, v: [B, Lkv, H, D] (bf16 CUDA).  o_part: fp32 [B, H, rows_pad, D],
    lse: fp32 [B, H, rows_pad] base-2 log-sum-exp; rows past Lq are left unwritten.
    """
    import torch
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [batch, len, heads, head_dim] tensor")
    batch, q_len, heads, head_dim = q.shape
    kv_len = k.shape[1]
    if tuple(k.shape) != (batch, kv_len, heads, head_dim) or v.shape != k.shape:
        raise ValueError("k and v must be [batch, kv_len, heads, head_dim] matching q")
    rp = rows_pad(q_len)
    if o_part is None:
        o_part = torch.empty(batch, heads, rp, head_dim, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty(batch, heads, rp, dtype=torch.float32, device=q.device)
    if (o_part.dtype != torch.float32 or tuple(o_part.shape) != (batch, heads, rp, head_dim)
            or not o_part.is_contiguous() or lse.dtype != torch.float32
            or tuple(lse.shape) != (batch, heads, rp) or not lse.is_contiguous()):
        raise ValueError("o_part / lse must be contiguous fp32 [B, H, rows_pad, D] / [B, H, rows_pad]")
    if kv_valid_len is None:
        kv_valid_len = kv_len
    if scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    st = load().ltxattn_forward_partial(
        ctypes.c_void_p(q.data_ptr()), ctypes.c_void_p(k.data_ptr()),
        ctypes.c_void_p(v.data_ptr()), ctypes.c_void_p(o_part.data_ptr()),
        ctypes.c_void_p(lse.data_ptr()), int(q_len), int(kv_len), int(kv_valid_len), int(batch),
        int(heads), int(head_dim), ctypes.c_float(scale), ctypes.c_void_p(_stream_handle(stream)))
    _check(st, "ltxattn_forward_partial")
    return o_part, lse


def combine(o_parts, lses, q_len: int, out=None, *, stream=None):
    """Merge of key-range partial results (``ltxattn_combine``) into bf16 [B, q_len, H, D].

    o_parts: fp32 [P, B, H, rows_pad, D]; lses: fp32 [P, B, H, rows_pad].
    """
    import torch
    if (not isinstance(o_parts, torch.Tensor) or o_parts.dtype != torch.float32
            or o_parts.dim() != 5 or not o_parts.is_contiguous() or not o_parts.is_cuda):
        raise TypeError("o_parts must be a contiguous fp32 CUDA [P, B, H, rows_pad, D] tensor")
    parts, batch, heads, rp, head_dim = o_parts.shape
    if rp != rows_pad(q_len):
        raise ValueError(f"rows_pad {rp} does not match q_len {q_len}")
    if (lses.dtype != torch.float32 or tuple(lses.shape) != (parts, batch, heads, rp)
            or not lses.is_contiguous()):
        raise ValueError("lses must be a contiguous fp32 [P, B, H, rows_pad] tensor")
    if out is None:
        out = torch.empty(batch, q_len, heads, head_dim, dtype=torch.bfloat16,
                          device=o_parts.device)
    st = load().ltxattn_combine(
        ctypes.c_void_p(o_parts.data_ptr()), ctypes.c_void_p(lses.data_ptr()),
        ctypes.c_void_p(out.data_ptr()), int(parts), int(q_len), int(batch), int(heads),
        int(head_dim), ctypes.c_void_p(_stream_handle(stream)))
    _check(st, "ltxattn_combine")
    return out


# ltxattn_dtype and ltxattn_rope_layout values
BF16, FP16, FP32 = 0, 1, 2
ROPE_LAYOUTS = {"pairs": 0, "halves": 1}

_NO_STRIDES = (0, 0, 0)

# The calls below run at the size of one token too, where the host's time is the call's time:
# a tensor is looked at once, one that is made here not at all, and the current device and stream
# are asked for once a call.


def _raw_stream(device: int) -> int:
    """The current stream's handle."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device)


@functools.lru_cache(maxsize=1)
def _dtype_codes() -> dict:
    import torch
    return {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}


def _dtype_code(t) -> int:
    code = _dtype_codes().get(t.dtype)
    if code is None:
        raise TypeError(f"dtype {t.dtype} is none of bfloat16, float16, float32")
    return code


def _on_stream(stream, call, *args, **kw):
    """``call`` on another stream than the current one: allocations inside belong to that stream
    (torch's allocator reuses their memory in that stream's order), and the tensors it was given
    are not handed out again before the work queued on it is done."""
    import torch
    with torch.cuda.stream(stream):
        result = call(*args, **kw)
    if stream != torch.cuda.current_stream():
        for t in (*args, *kw.values()):
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    return result


def _not_here(name: str, t, dtype, device: int):
    """The error for a tensor that is not of this dtype on this CUDA device."""
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (dtype is not None and t.dtype != dtype):
        return TypeError(f"{name} must be a {dtype or ''} CUDA tensor".replace("  ", " "))
    return ValueError(f"{name} is on {t.device}, not on the current device cuda:{device}")


def _check_cuda(name: str, t, device: int, dtype=None, shape=None) -> None:
    """A contiguous CUDA tensor on `device`, of this dtype and shape where they are given."""
    try:
        here = t.get_device() == device and (dtype is None or t.dtype == dtype)
    except AttributeError:
        here = False
    if not here:
        raise _not_here(name, t, dtype, device)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _heads_strides(name: str, t, device: int, dtype, shape=None):
    """Strides of a [batch, len, heads, head_dim] CUDA tensor with contiguous channels."""
    try:
        here = t.get_device() == device and (dtype is None or t.dtype == dtype)
    except AttributeError:
        here = False
    if not here:
        raise _not_here(name, t, dtype, device)
    size = t.shape
    if shape is not None and size != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(size)}")
    if len(size) != 4 or 0 in size:
        raise ValueError(f"{name} must be a non-empty [batch, len, heads, head_dim] tensor")
    strides = t.stride()
    if strides[3] != 1 and size[3] > 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    return strides


def rope_frequencies(axis_dims, base: float = 10000.0) -> list[float]:
    """base^(-2i/d) for the pairs i of every axis of d channels, axis after axis: the
    ``inv_freq`` of :func:`rope_axes` that turns each axis as a one-axis embedding of d
    channels turns."""
    return [float(base) ** (-2.0 * i / d) for d in axis_dims for i in range(d // 2)]


@functools.lru_cache(maxsize=16)
def _rope_axes_arrays(inv_freq: tuple, axis_dims: tuple):
    """The frequencies as a C array, its address, and four axes' channels."""
    dims = tuple(int(x) for x in axis_dims)
    if not 1 <= len(dims) <= 4:
        raise ValueError("axis_dims must name one to four axes")
    if len(inv_freq) != sum(dims) // 2:
        raise ValueError(f"{len(inv_freq)} frequencies for {sum(dims) // 2} rotated pairs")
    freq = (ctypes.c_double * len(inv_freq))(*inv_freq)
    return freq, ctypes.addressof(freq), dims + (0,) * (4 - len(dims))


def rope_axes(q, k, positions, inv_freq, axis_dims, q_out=None, k_out=None, *,
              layout: str = "pairs", inverse: bool = False, stream=None):
    """Rotary positions with several axes (``ltxattn_rope_axes``); returns (q', k').

    q: [B, L, H, D], k: [B, L, Hkv, D] or None (bf16, fp16 or fp32 CUDA, channels contiguous,
    other strides free); positions: fp32 [B or 1, L, axes]; inv_freq: host numbers, one per
    rotated pair, axis after axis (see :func:`rope_frequencies`); axis_dims: channels of each
    axis.  layout "pairs" turns (2i, 2i+1), "halves" (i, i + D/2).  ``inverse`` turns back:
    the gradient.  The outputs may be the inputs (in place).
    """
    import torch
    if stream is not None:
        return _on_stream(stream, rope_axes, q, k, positions, inv_freq, axis_dims, q_out, k_out,
                          layout=layout, inverse=inverse)
    freq, freq_at, dims = _rope_axes_arrays(tuple(inv_freq), tuple(axis_dims))
    axes = len(axis_dims)
    code_layout = ROPE_LAYOUTS.get(layout)
    if code_layout is None:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}")
    device = torch.cuda.current_device()
    q_strides = _heads_strides("q", q, device, None)
    code = _dtype_code(q)
    shape = q.shape
    batch, length, heads, head_dim = shape
    _check_cuda("positions", positions, device, torch.float32)
    pos_shape = positions.shape
    pos_batch = pos_shape[0]
    if len(pos_shape) != 3 or pos_batch not in (1, batch) or pos_shape[1] != length \
            or pos_shape[2] != axes:
        raise ValueError(f"positions must be [{batch} or 1, {length}, {axes}]")
    if q_out is None:
        q_out = torch.empty_like(q)
        q_out_strides = q_out.stride()
    else:
        q_out_strides = _heads_strides("q_out", q_out, device, q.dtype, shape)
    if k is not None:
        k_strides = _heads_strides("k", k, device, None)
        k_shape = k.shape
        kv_heads = k_shape[2]
        if k.dtype != q.dtype or k_shape[0] != batch or k_shape[1] != length \
                or k_shape[3] != head_dim:
            raise ValueError("k must have q's dtype, batch, length and head_dim")
        if k_out is None:
            k_out = torch.empty_like(k)
            k_out_strides = k_out.stride()
        else:
            k_out_strides = _heads_strides("k_out", k_out, device, q.dtype, k_shape)
        k_at, k_out_at = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    else:
        kv_heads, k_strides, k_out_strides, k_at, k_out_at = 1, _NO_STRIDES, _NO_STRIDES, 0, 0
    call = _pack_rope(
        q.data_ptr(), k_at, q_out.data_ptr(), k_out_at, *q_strides[:3], *k_strides[:3],
        *q_out_strides[:3], *k_out_strides[:3], positions.data_ptr(), freq_at, *dims, axes,
        pos_batch, batch, length, heads, kv_heads, head_dim, code, code_layout, bool(inverse))
    status = (_lib or load()).ltxattn_rope_axes(call, _raw_stream(device))
    if status:
        _check(status, "ltxattn_rope_axes")
    return q_out, k_out


def _norm_rows(name: str, t, device: int, dtype=None, shape=None):
    """(rows, cols, row stride) of a [..., cols] CUDA tensor whose rows lie at one stride."""
    try:
        here = t.get_device() == device and (dtype is None or t.dtype == dtype)
    except AttributeError:
        here = False
    if not here:
        raise _not_here(name, t, dtype, device)
    size = t.shape
    if shape is not None and size != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(size)}")
    n = t.numel()
    if len(size) < 1 or n == 0:
        raise ValueError(f"{name} must be a non-empty [..., cols] tensor")
    cols = size[-1]
    if t.is_contiguous():
        return n // cols, cols, cols
    steps = t.stride()
    if cols > 1 and steps[-1] != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    stride, want = None, None
    for count, step in zip(reversed(size[:-1]), reversed(steps[:-1])):
        if count == 1:
            continue
        if stride is None:
            stride = step
        elif step != want:
            raise ValueError(f"the rows of {name} must lie at one stride")
        want = step * count
    return n // cols, cols, cols if stride is None else stride


def _norm_affine(weight, bias, x, rows: int, cols: int, device: int) -> int:
    """Groups of a weight (and bias) of shape [cols] or [groups, cols]."""
    if weight is None:
        if bias is not None:
            raise ValueError("a bias needs a weight")
        return 1
    _check_cuda("weight", weight, device, x.dtype)
    shape = weight.shape
    if len(shape) not in (1, 2) or shape[-1] != cols:
        raise ValueError(f"weight must be [{cols}] or [groups, {cols}]")
    if bias is not None:
        _check_cuda("bias", bias, device, x.dtype, shape)
    groups = shape[0] if len(shape) == 2 else 1
    if groups < 1 or rows % groups:
        raise ValueError(f"{rows} rows do not fall into {groups} equal groups")
    return groups


def layer_norm(x, weight=None, bias=None, out=None, *, eps: float = 1e-6,
               return_stats: bool = False, stream=None):
    """Layer norm over the last axis (``ltxattn_layer_norm``); returns out, or (out, mean,
    rstd) with ``return_stats`` (fp32, one per row: what :func:`layer_norm_backward` reads).

    x: [..., C] (bf16, fp16 or fp32 CUDA; rows at one stride); weight, bias: [C], or [G, C]
    with one row for each G-th of x's rows in order (the scale and shift of every sample).
    ``out`` may be x.
    """
    import torch
    if stream is not None:
        return _on_stream(stream, layer_norm, x, weight, bias, out, eps=eps,
                          return_stats=return_stats)
    device = torch.cuda.current_device()
    rows, cols, x_stride = _norm_rows("x", x, device)
    code = _dtype_code(x)
    groups = _norm_affine(weight, bias, x, rows, cols, device)
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        out_stride = cols
    else:
        out_stride = _norm_rows("out", out, device, x.dtype, x.shape)[2]
    mean = rstd = None
    if return_stats:
        mean, rstd = torch.empty(2, *x.shape[:-1], dtype=torch.float32, device=x.device)
    status = (_lib or load()).ltxattn_layer_norm(
        x.data_ptr(), _ptr(weight), _ptr(bias), out.data_ptr(), _ptr(mean), _ptr(rstd), rows,
        cols, groups, x_stride, out_stride, eps, code, _raw_stream(device))
    if status:
        _check(status, "ltxattn_layer_norm")
    return (out, mean, rstd) if return_stats else out


def layer_norm_backward(dy, x, mean, rstd, weight=None, dx=None, *, stream=None):
    """Gradients of :func:`layer_norm` (``ltxattn_layer_norm_backward``): (dx, dweight, dbias).

    dy: like x; mean, rstd: as the forward call returned them; weight as given to it.
    dweight and dbias are fp32 of weight's shape, or None without a weight.  ``dx`` may be dy
    or x.
    """
    import torch
    if stream is not None:
        return _on_stream(stream, layer_norm_backward, dy, x, mean, rstd, weight, dx)
    lib = _lib or load()
    device = torch.cuda.current_device()
    rows, cols, x_stride = _norm_rows("x", x, device)
    code = _dtype_code(x)
    dy_stride = _norm_rows("dy", dy, device, x.dtype, x.shape)[2]
    stats = x.shape[:-1]
    _check_cuda("mean", mean, device, torch.float32, stats)
    _check_cuda("rstd", rstd, device, torch.float32, stats)
    groups = _norm_affine(weight, None, x, rows, cols, device)
    if dx is None:
        dx = torch.empty_like(x, memory_format=torch.contiguous_format)
        dx_stride = cols
    else:
        dx_stride = _norm_rows("dx", dx, device, x.dtype, x.shape)[2]
    dweight = dbias = workspace = None
    need = ctypes.c_ulonglong(0)
    if weight is not None:
        dweight = torch.empty_like(weight, dtype=torch.float32)
        dbias = torch.empty_like(dweight)
        _check(lib.ltxattn_layer_norm_workspace(rows, cols, groups, code, need),
               "ltxattn_layer_norm_workspace")
        if need.value:
            workspace = torch.empty(need.value, dtype=torch.uint8, device=x.device)
    status = lib.ltxattn_layer_norm_backward(
        dy.data_ptr(), x.data_ptr(), _ptr(weight), mean.data_ptr(), rstd.data_ptr(),
        dx.data_ptr(), _ptr(dweight), _ptr(dbias), rows, cols, groups, dy_stride, x_stride,
        dx_stride, code, _ptr(workspace), need.value, _raw_stream(device))
    if status:
        _check(status, "ltxattn_layer_norm_backward")
    return dx, dweight, dbias


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _masked_call(device, q, k, v, out, lse, scale, softcap, slopes, causal, prefix, q_starts,
                 kv_starts) -> bytes:
    """Checks what the library cannot see from raw pointers; returns the ltxattn_masked_call."""
    import torch
    bf16 = torch.bfloat16
    q_strides = _heads_strides("q", q, device, bf16)
    k_strides = _heads_strides("k", k, device, bf16)
    q_shape, k_shape = q.shape, k.shape
    batch, q_len, heads, head_dim = q_shape
    kv_batch, kv_len, kv_heads, kv_dim = k_shape
    if kv_batch != batch or kv_dim != head_dim or v.shape != k_shape:
        raise ValueError("k and v must be [batch, kv_len, kv_heads, head_dim] matching q")
    v_strides = _heads_strides("v", v, device, bf16)
    out_strides = _heads_strides("out", out, device, bf16, q_shape)
    _check_cuda("lse", lse, device, torch.float32, (batch, heads, q_len))
    docs = 0
    if q_starts is not None or kv_starts is not None:
        if q_starts is None or kv_starts is None:
            raise ValueError("q_starts and kv_starts come together")
        if q_starts.dim() != 2 or q_starts.shape[1] < 2:
            raise ValueError("q_starts must be [batch, documents + 1]")
        docs = q_starts.shape[1] - 1
        _check_cuda("q_starts", q_starts, device, torch.int32, (batch, docs + 1))
        _check_cuda("kv_starts", kv_starts, device, torch.int32, (batch, docs + 1))
    if prefix is not None:
        if not causal:
            raise ValueError("a prefix needs causal=True (without it every key is visible)")
        _check_cuda("prefix", prefix, device, torch.int32, (batch, max(docs, 1)))
    if slopes is not None:
        _check_cuda("slopes", slopes, device, torch.float32, (heads,))
    return _pack_masked(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), *q_strides[:3],
        *k_strides[:3], *v_strides[:3], *out_strides[:3], batch, q_len, kv_len, heads, kv_heads,
        head_dim, 1.0 / math.sqrt(head_dim) if scale is None else scale, softcap,
        0 if slopes is None else slopes.data_ptr(), 0 if prefix is None else prefix.data_ptr(),
        0 if docs == 0 else q_starts.data_ptr(), 0 if docs == 0 else kv_starts.data_ptr(), docs,
        bool(causal))


def _masked_workspace(lib, call, backward: bool, device):
    """Workspace of the call, and its bytes."""
    import torch
    need = ctypes.c_ulonglong(0)
    _check(lib.ltxattn_masked_workspace(call, backward, need), "ltxattn_masked_workspace")
    n = need.value
    return (torch.empty(n, dtype=torch.uint8, device=device) if n else None), n


def masked_forward(q, k, v, out=None, lse=None, *, scale: float | None = None,
                   softcap: float = 0.0, slopes=None, causal: bool = False, prefix=None,
                   q_starts=None, kv_starts=None, stream=None):
    """Attention with masked, capped and distance-biased scores (``ltxattn_masked_forward``);
    returns (out, lse), lse fp32 [B, H, Lq] in base 2.

    q: [B, Lq, H, D]; k, v: [B, Lkv, Hkv, D], H a multiple of Hkv (bf16 CUDA, channels
    contiguous, other strides free).  softcap: s = softcap * tanh(s / softcap).  slopes: fp32
    [H], subtracts slopes[h] times the token distance.  causal: query i of nq sees the keys up
    to i + nkv - nq, and the first prefix[b, d] keys (int32 [B, documents or 1]).  q_starts,
    kv_starts: int32 [B, documents + 1] offsets of packed documents, whose queries see their
    own document's keys only; rows of no document keep what out and lse held (zeros and -inf
    when they are allocated here).
    """
    import torch
    if stream is not None:
        return _on_stream(stream, masked_forward, q, k, v, out, lse, scale=scale, softcap=softcap,
                          slopes=slopes, causal=causal, prefix=prefix, q_starts=q_starts,
                          kv_starts=kv_starts)
    device = torch.cuda.current_device()
    if out is None or lse is None:  # rows of no document stay as they are made here
        _heads_strides("q", q, device, torch.bfloat16)
        if out is None:
            out = torch.empty_like(q) if q_starts is None else torch.zeros_like(q)
        if lse is None:
            shape = (q.shape[0], q.shape[2], q.shape[1])
            lse = torch.empty(shape, dtype=torch.float32, device=q.device) \
                if q_starts is None else \
                torch.full(shape, -math.inf, dtype=torch.float32, device=q.device)
    call = _masked_call(device, q, k, v, out, lse, scale, softcap, slopes, causal, prefix,
                        q_starts, kv_starts)
    lib = _lib or load()
    workspace, need = _masked_workspace(lib, call, False, q.device)
    status = lib.ltxattn_masked_forward(call, None if workspace is None else workspace.data_ptr(),
                                        need, _raw_stream(device))
    if status:
        _check(status, "ltxattn_masked_forward")
    return out, lse


def masked_backward(d_out, q, k, v, out, lse, dq=None, dk=None, dv=None, *,
                    scale: float | None = None, softcap: float = 0.0, slopes=None,
                    causal: bool = False, prefix=None, q_starts=None, kv_starts=None,
                    stream=None):
    """Gradients of :func:`masked_forward` (``ltxattn_masked_backward``): (dq, dk, dv), bf16.

    d_out: like q; out, lse: what the forward call returned; the options as given to it.  Rows
    of no document keep what dq, dk and dv held (zeros when they are allocated here).
    """
    import torch
    if out is None or lse is None:
        raise ValueError("out and lse of the forward call are needed")
    if stream is not None:
        return _on_stream(stream, masked_backward, d_out, q, k, v, out, lse, dq, dk, dv,
                          scale=scale, softcap=softcap, slopes=slopes, causal=causal,
                          prefix=prefix, q_starts=q_starts, kv_starts=kv_starts)
    device, bf16 = torch.cuda.current_device(), torch.bfloat16
    call = _masked_call(device, q, k, v, out, lse, scale, softcap, slopes, causal, prefix,
                        q_starts, kv_starts)
    d_out_strides = _heads_strides("d_out", d_out, device, bf16, q.shape)
    make = torch.empty_like if q_starts is None else torch.zeros_like
    grads, strides = [], []
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is None:
            t = make(like)
            strides.append(t.stride())
        else:
            strides.append(_heads_strides(name, t, device, bf16, like.shape))
        grads.append(t)
    dq, dk, dv = grads
    grad = _pack_grad(d_out.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                      *d_out_strides[:3], *strides[0][:3], *strides[1][:3], *strides[2][:3])
    lib = _lib or load()
    workspace, need = _masked_workspace(lib, call, True, q.device)
    status = lib.ltxattn_masked_backward(call, grad, workspace.data_ptr(), need,
                                         _raw_stream(device))
    if status:
        _check(status, "ltxattn_masked_backward")
    return dq, dk, dv
