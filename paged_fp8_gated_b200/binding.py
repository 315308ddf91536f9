"""Python binding of libgad_attn.so (argument marshalling only).

Every step of the computation runs in the library's CUDA kernels; this module
only checks torch tensors' dtypes and layouts, allocates the output and the
workspace with torch when the caller does not pass them, and forwards raw
device pointers and the current CUDA stream to the C ABI (include/gad_attn.h).

Importing it fails loudly when the library has not been built: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgad_attn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python -m paged_fp8_gated_b200.build` (nvcc, sm_100a)")

_lib = ctypes.CDLL(LIB_PATH)
_vp = ctypes.c_void_p
_lib.gad_attn_workspace_bytes.restype = ctypes.c_size_t
_lib.gad_attn_workspace_bytes.argtypes = [ctypes.c_int, ctypes.c_int]
_lib.gad_attn_decode.restype = ctypes.c_int
_lib.gad_attn_decode.argtypes = [
    _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,            # qkv .. v_scale
    ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64,  # B, L, max_pages, num_rows
    ctypes.c_int, ctypes.c_int, ctypes.c_int,               # page_size, window, use_rope
    _vp, _vp, ctypes.c_size_t, _vp]                         # out, workspace, bytes, stream
_lib.gad_attn_workspace_bytes_heads.restype = ctypes.c_size_t
_lib.gad_attn_workspace_bytes_heads.argtypes = [ctypes.c_int] * 4
_lib.gad_attn_decode_heads.restype = ctypes.c_int
_lib.gad_attn_decode_heads.argtypes = (list(_lib.gad_attn_decode.argtypes[:11])
                                       + [ctypes.c_int, ctypes.c_int]  # hq, hkv
                                       + list(_lib.gad_attn_decode.argtypes[11:]))
_lib.gad_attn_decode_heads_timed.restype = ctypes.c_int
_lib.gad_attn_decode_heads_timed.argtypes = list(_lib.gad_attn_decode_heads.argtypes) + [_vp]
_lib.gad_attn_prefill.restype = ctypes.c_int
_lib.gad_attn_prefill.argtypes = list(_lib.gad_attn_decode.argtypes)
_lib.gad_attn_prefill_workspace_bytes.restype = ctypes.c_size_t
_lib.gad_attn_prefill_workspace_bytes.argtypes = [ctypes.c_int, ctypes.c_int]
_lib.gad_attn_prefill_timed.restype = ctypes.c_int
_lib.gad_attn_prefill_timed.argtypes = list(_lib.gad_attn_decode.argtypes) + [_vp]
_lib.gad_oproj.restype = ctypes.c_int
_lib.gad_oproj.argtypes = [_vp, _vp, _vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp]
_lib.gad_attn_decode_oproj.restype = ctypes.c_int
_lib.gad_attn_decode_oproj.argtypes = (list(_lib.gad_attn_decode.argtypes[:19])
                                       + [_vp, ctypes.c_int, _vp, _vp])  # o_weight, hidden, a, stream
_lib.gad_attn_decode_timed.restype = ctypes.c_int
_lib.gad_attn_decode_timed.argtypes = list(_lib.gad_attn_decode.argtypes) + [_vp]
_lib.gad_attn_decode_noalloc.restype = ctypes.c_int
_lib.gad_attn_decode_noalloc.argtypes = list(_lib.gad_attn_decode.argtypes[:17]) + [_vp]
_lib.gad_attn_step_status.restype = ctypes.c_int
_lib.gad_attn_step_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_int), _vp]
_lib.gad_oproj_status.restype = ctypes.c_int
_lib.gad_oproj_status.argtypes = [ctypes.POINTER(ctypes.c_int), _vp]
_i64 = ctypes.c_int64
_lib.gad_linear.restype = ctypes.c_int
_lib.gad_linear.argtypes = [_vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64] + [ctypes.c_int] * 6 + [_vp]
_lib.gad_linear_status.restype = ctypes.c_int
_lib.gad_linear_status.argtypes = [ctypes.POINTER(ctypes.c_int), _vp]
_lib.gad_beam_workspace_bytes.restype = ctypes.c_size_t
_lib.gad_beam_workspace_bytes.argtypes = [ctypes.c_int] * 4
_lib.gad_beam_select.restype = ctypes.c_int
_lib.gad_beam_select.argtypes = ([_vp, ctypes.c_int, _i64, _vp, _vp] + [ctypes.c_int] * 5
                                 + [_vp, _vp, _vp, _vp, ctypes.c_size_t, _vp])
_lib.gad_pages_workspace_bytes.restype = ctypes.c_size_t
_lib.gad_pages_workspace_bytes.argtypes = [ctypes.c_int, _i64]
_lib.gad_pages_copy.restype = ctypes.c_int
_lib.gad_pages_copy.argtypes = [_vp, ctypes.c_int, ctypes.c_size_t, _i64, _vp, _vp, ctypes.c_int, _vp]
_lib.gad_pages_fork.restype = ctypes.c_int
_lib.gad_pages_fork.argtypes = ([_vp, _vp, ctypes.c_int, _vp] + [ctypes.c_int] * 3 + [_vp, _i64]
                                + [_vp] * 5 + [ctypes.c_size_t, _vp])
_lib.gad_pages_extend.restype = ctypes.c_int
_lib.gad_pages_extend.argtypes = ([_vp, _vp] + [ctypes.c_int] * 4 + [_vp, _i64]
                                  + [_vp] * 3 + [ctypes.c_size_t, _vp])
_lib.gad_pages_free.restype = ctypes.c_int
_lib.gad_pages_free.argtypes = [_vp, _vp, ctypes.c_int, _vp, ctypes.c_int, ctypes.c_int, _vp, _i64, _vp]
_lib.gad_pages_compact.restype = ctypes.c_int
_lib.gad_pages_compact.argtypes = ([_vp, _vp] + [ctypes.c_int] * 3 + [_vp, _i64, _vp, _vp, ctypes.c_int]
                                   + [_vp] * 2 + [ctypes.c_size_t, _vp])


class GadTensor(ctypes.Structure):
    """gad_tensor: data pointer, element type code, rank, extents, strides (elements)."""
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


_GT = ctypes.POINTER(GadTensor)
_lib.gad_attn_set_workspace.restype = ctypes.c_int
_lib.gad_attn_set_workspace.argtypes = [_vp, ctypes.c_size_t]
_lib.gad_attn_workspace_bytes_t.restype = ctypes.c_size_t
_lib.gad_attn_workspace_bytes_t.argtypes = [ctypes.c_int] * 5
_lib.gad_attn_decode_t.restype = ctypes.c_int
_lib.gad_attn_decode_t.argtypes = [_GT] * 9 + [ctypes.c_int] * 3 + [_GT, _vp]
_lib.gad_last_error.restype = ctypes.c_char_p
_lib.gad_last_error.argtypes = []
_lib.gad_status_string.restype = ctypes.c_char_p
_lib.gad_status_string.argtypes = [ctypes.c_int]

HQ, HKV, D = 16, 2, 64
QKV_COLS, OUT_COLS, ROW_BYTES = 2304, 1024, 128
MAX_L, MAX_PREFILL_L = 8, 65536
HIDDEN = 8192

EXPORTED = ("gad_attn_decode", "gad_attn_decode_heads", "gad_attn_decode_timed",
            "gad_attn_decode_heads_timed", "gad_attn_prefill", "gad_attn_prefill_timed",
            "gad_attn_prefill_workspace_bytes", "gad_oproj", "gad_attn_decode_oproj",
            "gad_attn_decode_noalloc", "gad_attn_workspace_bytes",
            "gad_attn_workspace_bytes_heads", "gad_last_error", "gad_status_string",
            "gad_attn_step_status", "gad_oproj_status", "gad_attn_set_workspace",
            "gad_attn_workspace_bytes_t", "gad_attn_decode_t",
            "gad_linear", "gad_linear_status", "gad_beam_select", "gad_beam_workspace_bytes",
            "gad_pages_workspace_bytes", "gad_pages_copy", "gad_pages_fork", "gad_pages_extend",
            "gad_pages_free", "gad_pages_compact")
# gad_dtype codes (include/gad_attn.h)
DTYPE_BF16, DTYPE_E4M3, DTYPE_U8, DTYPE_I32, DTYPE_I64, DTYPE_F32, DTYPE_F16 = 1, 2, 3, 4, 5, 6, 7
_DTYPE_CODES = {torch.bfloat16: DTYPE_BF16, torch.uint8: DTYPE_U8, torch.int32: DTYPE_I32,
                torch.int64: DTYPE_I64, torch.float32: DTYPE_F32, torch.float16: DTYPE_F16}
if hasattr(torch, "float8_e4m3fn"):
    _DTYPE_CODES[torch.float8_e4m3fn] = DTYPE_E4M3
NOALLOC_SCRATCH_BYTES = 16 << 20
# gad_activation codes
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
# GAD_STATUS_* bits
STATUS_ATTN_WAIT, STATUS_OPROJ_WAIT, STATUS_PAGES_POOL, STATUS_PAGES_ROW, STATUS_LINEAR_WAIT = 1, 2, 4, 8, 16


class GadError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _lib.gad_last_error().decode(errors="replace")
        name = _lib.gad_status_string(status).decode()
        super().__init__(f"{where}: {name} ({status}): {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    return _lib


def workspace_bytes(B: int, L: int, hq: int = HQ, hkv: int = HKV) -> int:
    """Workspace of one step; blocks longer than MAX_L tokens go to the prefill
    entry point (16 and 2 heads)."""
    if L > MAX_L and (hq, hkv) == (HQ, HKV):
        n = _lib.gad_attn_prefill_workspace_bytes(int(B), int(L))
    elif (hq, hkv) == (HQ, HKV):
        n = _lib.gad_attn_workspace_bytes(int(B), int(L))
    else:
        n = _lib.gad_attn_workspace_bytes_heads(int(B), int(L), int(hq), int(hkv))
    if n == 0:
        raise GadError(-2, "gad_attn_workspace_bytes")
    return int(n)


def alloc_workspace(B: int, L: int, device=None, hq: int = HQ, hkv: int = HKV) -> torch.Tensor:
    """Caller-owned scratch for gad_attn_decode (256-byte aligned by torch's allocator)."""
    return torch.empty(workspace_bytes(B, L, hq, hkv), dtype=torch.uint8,
                       device=device or "cuda")


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def attn_decode(qkv: torch.Tensor, positions: torch.Tensor, seq_lens: torch.Tensor | None,
                page_table: torch.Tensor, cache_loc: torch.Tensor, k_cache: torch.Tensor,
                v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                page_size: int, window: int, use_rope: bool, L: int = 1,
                out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None,
                events: list | None = None, hq: int = HQ, hkv: int = HKV) -> torch.Tensor:
    """One decode step (L = 1), verify block (L <= 8) or prefill block (L up to
    MAX_PREFILL_L, through gad_attn_prefill, 16 and 2 heads); returns out bf16
    [B, L, 64 hq].

    Shapes: qkv bf16 [B*L, 64 (2 hq + 2 hkv)]; positions, cache_loc int64 [B*L];
    seq_lens int32 [B] (optional); page_table int32 [B, max_pages]; k_cache / v_cache
    uint8 [num_pages, page_size, hkv, 64] (mutated in the rows cache_loc); k_scale /
    v_scale float32 [1] on the device.  hq, hkv: head counts (16, 2 by default; other
    counts go through gad_attn_decode_heads).  With ``events`` (four torch.cuda.Event
    with timing), the profiling entry point records them around the three kernels.
    """
    _need(qkv, "qkv", torch.bfloat16, 2)
    _need(positions, "positions", torch.int64, 1)
    _need(page_table, "page_table", torch.int32, 2)
    _need(cache_loc, "cache_loc", torch.int64, 1)
    _need(k_cache, "k_cache", torch.uint8)
    _need(v_cache, "v_cache", torch.uint8)
    _need(k_scale, "k_scale", torch.float32)
    _need(v_scale, "v_scale", torch.float32)
    if seq_lens is not None:
        _need(seq_lens, "seq_lens", torch.int32, 1)
    B, max_pages = page_table.shape
    T = qkv.shape[0]
    qkv_cols, out_cols, row_bytes = (2 * hq + 2 * hkv) * D, hq * D, hkv * D
    if qkv.shape[1] != qkv_cols or T != B * L:
        raise ValueError(f"qkv must be [B*L={B * L}, {qkv_cols}], got {tuple(qkv.shape)}")
    if positions.numel() != T or cache_loc.numel() != T:
        raise ValueError("positions and cache_loc need one entry per token")
    if k_cache.shape != v_cache.shape or k_cache.numel() % row_bytes:
        raise ValueError(f"k_cache and v_cache must have the same shape, {row_bytes} bytes per row")
    num_rows = k_cache.numel() // row_bytes
    if out is None:
        out = torch.empty(B, L, out_cols, dtype=torch.bfloat16, device=qkv.device)
    else:
        _need(out, "out", torch.bfloat16)
        if out.numel() != T * out_cols:
            raise ValueError(f"out must hold B*L*{out_cols} values")
    if workspace is None:
        workspace = alloc_workspace(B, L, qkv.device, hq, hkv)
    else:
        _need(workspace, "workspace", torch.uint8)
    s = (stream or torch.cuda.current_stream(qkv.device)).cuda_stream
    head = (_ptr(qkv), _ptr(positions), _ptr(seq_lens), _ptr(page_table), _ptr(cache_loc),
            _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), int(B), int(L))
    tail = (int(max_pages), int(num_rows), int(page_size), int(window), int(bool(use_rope)),
            _ptr(out), _ptr(workspace), int(workspace.numel()), ctypes.c_void_p(s))
    args = head + tail
    tp8 = (hq, hkv) == (HQ, HKV)
    prefill = L > MAX_L
    if prefill and not tp8:
        raise ValueError(f"blocks longer than {MAX_L} tokens take 16 query and 2 KV heads")
    if events is None:
        if prefill:
            st = _lib.gad_attn_prefill(*args)
        else:
            st = _lib.gad_attn_decode(*args) if tp8 else \
                _lib.gad_attn_decode_heads(*head, int(hq), int(hkv), *tail)
    else:
        if len(events) != 4:
            raise ValueError("events must hold four torch.cuda.Event")
        for ev in events:   # materialise the underlying cudaEvent_t
            if ev.cuda_event == 0:
                ev.record()
        arr = (ctypes.c_void_p * 4)(*[ctypes.c_void_p(ev.cuda_event) for ev in events])
        if prefill:
            st = _lib.gad_attn_prefill_timed(*args, arr)
        else:
            st = _lib.gad_attn_decode_timed(*args, arr) if tp8 else \
                _lib.gad_attn_decode_heads_timed(*head, int(hq), int(hkv), *tail, arr)
    if st != 0:
        raise GadError(st, "gad_attn_prefill" if prefill else "gad_attn_decode")
    return out


def attn_decode_noalloc(qkv: torch.Tensor, positions: torch.Tensor,
                        seq_lens: torch.Tensor | None, page_table: torch.Tensor,
                        cache_loc: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        k_scale: torch.Tensor, v_scale: torch.Tensor, page_size: int, window: int,
                        use_rope: bool, L: int = 1, out: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The step through gad_attn_decode_noalloc: no workspace argument, the library's
    built-in 16 MiB device scratch is used instead (for callers that cannot allocate
    device memory themselves).  Calls on one device must not overlap on the GPU."""
    for t, n, dt in ((qkv, "qkv", torch.bfloat16), (positions, "positions", torch.int64),
                     (page_table, "page_table", torch.int32), (cache_loc, "cache_loc", torch.int64),
                     (k_cache, "k_cache", torch.uint8), (v_cache, "v_cache", torch.uint8),
                     (k_scale, "k_scale", torch.float32), (v_scale, "v_scale", torch.float32)):
        _need(t, n, dt)
    B, max_pages = page_table.shape
    T = qkv.shape[0]
    if qkv.shape[1] != QKV_COLS or T != B * L:
        raise ValueError(f"qkv must be [B*L={B * L}, {QKV_COLS}], got {tuple(qkv.shape)}")
    if positions.numel() != T or cache_loc.numel() != T:
        raise ValueError("positions and cache_loc need one entry per token")
    if k_cache.shape != v_cache.shape or k_cache.numel() % ROW_BYTES:
        raise ValueError(f"k_cache and v_cache must have the same shape, {ROW_BYTES} bytes per row")
    num_rows = k_cache.numel() // ROW_BYTES
    if out is None:
        out = torch.empty(B, L, OUT_COLS, dtype=torch.bfloat16, device=qkv.device)
    else:
        _need(out, "out", torch.bfloat16)
        if out.numel() != T * OUT_COLS:
            raise ValueError(f"out must hold B*L*{OUT_COLS} values")
    s = (stream or torch.cuda.current_stream(qkv.device)).cuda_stream
    st = _lib.gad_attn_decode_noalloc(
        _ptr(qkv), _ptr(positions), _ptr(seq_lens), _ptr(page_table), _ptr(cache_loc),
        _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), int(B), int(L),
        int(max_pages), int(num_rows), int(page_size), int(window), int(bool(use_rope)),
        _ptr(out), ctypes.c_void_p(s))
    if st != 0:
        raise GadError(st, "gad_attn_decode_noalloc")
    return out


def oproj(out: torch.Tensor, o_weight: torch.Tensor, a: torch.Tensor | None = None,
          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """a = out @ o_weight^T through gad_oproj: out bf16 [T, K], o_weight bf16 [N, K]
    (both CUDA, contiguous); returns a bf16 [T, N]."""
    _need(out, "out", torch.bfloat16)
    _need(o_weight, "o_weight", torch.bfloat16, 2)
    K = out.shape[-1]
    T = out.numel() // K
    N = o_weight.shape[0]
    if o_weight.shape[1] != K:
        raise ValueError(f"o_weight must be [N, {K}], got {tuple(o_weight.shape)}")
    if a is None:
        a = torch.empty(T, N, dtype=torch.bfloat16, device=out.device)
    else:
        _need(a, "a", torch.bfloat16)
        if a.numel() != T * N:
            raise ValueError(f"a must hold {T}x{N} values")
    s = (stream or torch.cuda.current_stream(out.device)).cuda_stream
    st = _lib.gad_oproj(_ptr(out), _ptr(o_weight), _ptr(a), int(T), int(K), int(N), ctypes.c_void_p(s))
    if st != 0:
        raise GadError(st, "gad_oproj")
    return a


def attn_decode_oproj(qkv, positions, seq_lens, page_table, cache_loc, k_cache, v_cache, k_scale,
                      v_scale, page_size: int, window: int, use_rope: bool, o_weight: torch.Tensor,
                      L: int = 1, out: torch.Tensor | None = None, a: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """The step and its output projection in one call (gad_attn_decode_oproj);
    returns (out bf16 [B, L, 1024], a bf16 [B * L, hidden])."""
    for t, n, dt in ((qkv, "qkv", torch.bfloat16), (positions, "positions", torch.int64),
                     (page_table, "page_table", torch.int32), (cache_loc, "cache_loc", torch.int64),
                     (k_cache, "k_cache", torch.uint8), (v_cache, "v_cache", torch.uint8),
                     (k_scale, "k_scale", torch.float32), (v_scale, "v_scale", torch.float32)):
        _need(t, n, dt)
    _need(o_weight, "o_weight", torch.bfloat16, 2)
    B, max_pages = page_table.shape
    T = qkv.shape[0]
    if qkv.shape[1] != QKV_COLS or T != B * L:
        raise ValueError(f"qkv must be [B*L={B * L}, {QKV_COLS}], got {tuple(qkv.shape)}")
    hidden = o_weight.shape[0]
    num_rows = k_cache.numel() // ROW_BYTES
    if out is None:
        out = torch.empty(B, L, OUT_COLS, dtype=torch.bfloat16, device=qkv.device)
    if a is None:
        a = torch.empty(T, hidden, dtype=torch.bfloat16, device=qkv.device)
    if workspace is None:
        n = _lib.gad_attn_prefill_workspace_bytes(int(B), int(L))
        if n == 0:
            raise GadError(-2, "gad_attn_prefill_workspace_bytes")
        workspace = torch.empty(int(n), dtype=torch.uint8, device=qkv.device)
    s = (stream or torch.cuda.current_stream(qkv.device)).cuda_stream
    st = _lib.gad_attn_decode_oproj(
        _ptr(qkv), _ptr(positions), _ptr(seq_lens), _ptr(page_table), _ptr(cache_loc), _ptr(k_cache),
        _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), int(B), int(L), int(max_pages), int(num_rows),
        int(page_size), int(window), int(bool(use_rope)), _ptr(out), _ptr(workspace),
        int(workspace.numel()), _ptr(o_weight), int(hidden), _ptr(a), ctypes.c_void_p(s))
    if st != 0:
        raise GadError(st, "gad_attn_decode_oproj")
    return out, a


def raw_call(**kw) -> int:
    """Call the C entry point with raw values (for boundary tests); returns the status."""
    args = [kw.get(k) for k in ("qkv", "positions", "seq_lens", "page_table", "cache_loc",
                                "k_cache", "v_cache", "k_scale", "v_scale")]
    args = [a if (a is None or isinstance(a, ctypes.c_void_p)) else ctypes.c_void_p(a) for a in args]
    args += [kw.get("B", 1), kw.get("L", 1)]
    rest = [kw.get("max_pages", 1), kw.get("num_rows", 1), kw.get("page_size", 1),
            kw.get("window", 0), kw.get("use_rope", 0), kw.get("out"), kw.get("workspace"),
            kw.get("workspace_bytes", 0), kw.get("stream")]
    if kw.get("prefill"):           # through gad_attn_prefill
        return _lib.gad_attn_prefill(*args, *rest)
    if "hq" in kw or "hkv" in kw:   # through gad_attn_decode_heads
        return _lib.gad_attn_decode_heads(*args, kw.get("hq", HQ), kw.get("hkv", HKV), *rest)
    return _lib.gad_attn_decode(*args, *rest)


def last_error() -> str:
    return _lib.gad_last_error().decode(errors="replace")


# ---------------------------------------------------------------------------
# Status words and the tensor-descriptor form
# ---------------------------------------------------------------------------

def step_status(workspace: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> int:
    """GAD_STATUS_* bits of the last step run with `workspace` (None: the
    allocation-free entry point's built-in scratch); waits for `stream`."""
    st = ctypes.c_int(-1)
    dev = workspace.device if workspace is not None else torch.device("cuda", torch.cuda.current_device())
    s = stream or torch.cuda.current_stream(dev)
    rc = _lib.gad_attn_step_status(_ptr(workspace), ctypes.byref(st), ctypes.c_void_p(s.cuda_stream))
    if rc != 0:
        raise GadError(rc, "gad_attn_step_status")
    s.synchronize()
    return int(st.value)


def oproj_status(stream: torch.cuda.Stream | None = None) -> int:
    """GAD_STATUS_* bits of the standalone projections since the last read (then cleared)."""
    st = ctypes.c_int(-1)
    s = stream or torch.cuda.current_stream()
    rc = _lib.gad_oproj_status(ctypes.byref(st), ctypes.c_void_p(s.cuda_stream))
    if rc != 0:
        raise GadError(rc, "gad_oproj_status")
    s.synchronize()
    return int(st.value)


def tensor_desc(t: torch.Tensor | None, dtype: int | None = None, data: int | None = None,
                shape=None, stride=None) -> GadTensor | None:
    """gad_tensor for a torch tensor (its pointer, element type, extents and
    strides); the keyword overrides let tests describe malformed tensors."""
    if t is None and data is None:
        return None
    d = GadTensor()
    d.data = data if data is not None else t.data_ptr()
    d.dtype = dtype if dtype is not None else _DTYPE_CODES.get(t.dtype, 0)
    shp = list(shape if shape is not None else t.shape)
    std = list(stride if stride is not None else t.stride())
    d.ndim = len(shp)
    for i in range(min(4, len(shp))):
        d.shape[i] = int(shp[i])
        d.stride[i] = int(std[i])
    return d


def set_workspace(workspace: torch.Tensor | None) -> None:
    """Register (None: unregister) the scratch gad_attn_decode_t uses on the current device."""
    rc = _lib.gad_attn_set_workspace(_ptr(workspace), 0 if workspace is None else int(workspace.numel()))
    if rc != 0:
        raise GadError(rc, "gad_attn_set_workspace")


def workspace_bytes_t(B: int, L: int, max_pages: int, page_size: int, window: int) -> int:
    n = _lib.gad_attn_workspace_bytes_t(int(B), int(L), int(max_pages), int(page_size), int(window))
    if n == 0:
        raise GadError(-2, "gad_attn_workspace_bytes_t")
    return int(n)


def raw_call_t(descs: dict, page_size: int = 1, window: int = 0, use_rope: int = 0, stream=None) -> int:
    """gad_attn_decode_t on prepared descriptors (missing names pass NULL); returns the status."""
    names = ("qkv", "positions", "seq_lens", "page_table", "cache_loc", "k_cache", "v_cache",
             "k_scale", "v_scale")
    ptrs = [ctypes.byref(descs[n]) if descs.get(n) is not None else None for n in names]
    out = descs.get("out")
    return _lib.gad_attn_decode_t(*ptrs, int(page_size), int(window), int(use_rope),
                                  ctypes.byref(out) if out is not None else None, stream)


def attn_decode_t(qkv, positions, seq_lens, page_table, cache_loc, k_cache, v_cache, k_scale, v_scale,
                  page_size: int, window: int, use_rope: bool, out: torch.Tensor,
                  stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The step through the descriptor entry point (scratch from set_workspace):
    the tensors are described as they are; the library checks them."""
    descs = dict(qkv=tensor_desc(qkv), positions=tensor_desc(positions), seq_lens=tensor_desc(seq_lens),
                 page_table=tensor_desc(page_table), cache_loc=tensor_desc(cache_loc),
                 k_cache=tensor_desc(k_cache), v_cache=tensor_desc(v_cache), k_scale=tensor_desc(k_scale),
                 v_scale=tensor_desc(v_scale), out=tensor_desc(out))
    s = (stream or torch.cuda.current_stream(out.device)).cuda_stream
    rc = raw_call_t(descs, page_size, window, int(bool(use_rope)), ctypes.c_void_p(s))
    if rc != 0:
        raise GadError(rc, "gad_attn_decode_t")
    return out


# ---------------------------------------------------------------------------
# Linear layer, beam selection and page operations
# ---------------------------------------------------------------------------

def _call(fn, dev: torch.device, stream: torch.cuda.Stream | None, *args) -> None:
    """Calls a C entry point with the tensors' device current, on ``stream`` (by default that
    device's current one; a stream of another device is refused)."""
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev.index)
    elif stream.device != dev:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {dev}")
    else:
        s = stream.cuda_stream
    if dev.index == torch._C._cuda_getDevice():
        st = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, s)
    if st != 0:
        raise GadError(st, fn.__name__)


def _make(stream: torch.cuda.Stream | None, make):
    """make(), a call that creates tensors, on the stream that will use them."""
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        return make()


def _dev_of(t, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _cuda(t, name: str, dev: torch.device, dtype, shape=None):
    """A contiguous CUDA tensor of `dtype` (and `shape`) on `dev`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        _need(t, name, dtype)
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _rows(t, name: str, dev, dtype, shape):
    """A matrix whose rows are contiguous; returns its row stride in values."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == dev and t.shape == shape):
        if _dev_of(t, name) != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return ld if shape[0] > 1 else max(ld, shape[1])   # a single row's stride is never followed


def linear(x: torch.Tensor, w: torch.Tensor, bias: torch.Tensor | None = None,
           residual: torch.Tensor | None = None, activation: str = "none",
           out_dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
           stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """act(x @ w^T + bias) + residual through gad_linear.

    x [T, K] and w [N, K] bf16 or fp16 (rows contiguous, a multiple of 8 values
    apart, so with room behind them if K is no multiple of 8); bias [N] of their type; residual and the result [T, N] of
    ``out_dtype`` (that of x, or float32).  ``activation``: one of ACTIVATIONS.
    ``out`` may be the residual itself.
    """
    dev = _dev_of(x, "x")
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"x must be bfloat16 or float16, got {x.dtype}")
    if x.dim() != 2 or not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("x and w must be matrices [T, K] and [N, K]")
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    (T, K), N = x.shape, w.shape[0]
    dt = x.dtype
    if out_dtype is None:
        out_dtype = dt if out is None else out.dtype
    if out_dtype is not dt and out_dtype is not torch.float32:
        raise TypeError(f"the result must be {dt} or float32, got {out_dtype}")
    ldx, one = x.stride()
    if one != 1 and K > 1:
        raise ValueError("x must have contiguous rows")
    ldw = _rows(w, "w", dev, dt, (N, K))
    if T == 1:     # a single row's stride is never followed
        ldx = -(-K // 8) * 8
    if N == 1:
        ldw = -(-ldw // 8) * 8
    if bias is not None:
        bias = _cuda(bias, "bias", dev, dt, (N,)).data_ptr()
    ldr = 0
    if residual is not None:
        ldr = _rows(residual, "residual", dev, out_dtype, (T, N))
        residual = residual.data_ptr()
    if out is None:
        out = _make(stream, lambda: torch.empty(T, N, dtype=out_dtype, device=dev))
    ldy = _rows(out, "out", dev, out_dtype, (T, N))
    _call(_lib.gad_linear, dev, stream, x.data_ptr(), ldx, w.data_ptr(), ldw, bias, residual, ldr,
          out.data_ptr(), ldy, T, K, N, _DTYPE_CODES[dt], _DTYPE_CODES[out_dtype], act)
    return out


def linear_status(stream: torch.cuda.Stream | None = None) -> int:
    """GAD_STATUS_* bits of the linear layers since the last read (then cleared)."""
    st = ctypes.c_int(-1)
    s = stream or torch.cuda.current_stream()
    _call(_lib.gad_linear_status, s.device, s, ctypes.byref(st))
    s.synchronize()
    return int(st.value)


def beam_workspace_bytes(G: int, W: int, V: int, K: int) -> int:
    n = _lib.gad_beam_workspace_bytes(int(G), int(W), int(V), int(K))
    if n == 0:
        raise GadError(-2, "gad_beam_workspace_bytes")
    return int(n)


def alloc_beam_workspace(G: int, W: int, V: int, K: int, device=None) -> torch.Tensor:
    """Scratch for beam_select with these sizes (256-byte aligned by torch's allocator)."""
    return torch.empty(beam_workspace_bytes(G, W, V, K), dtype=torch.uint8, device=device or "cuda")


def beam_select(logits: torch.Tensor, scores: torch.Tensor, K: int, finished: torch.Tensor | None = None,
                pad_token: int = 0, out: tuple | None = None, workspace: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The K best (beam, token) candidates of every request through gad_beam_select.

    logits [G, W, V] bf16, fp16 or float32 (each beam's row contiguous, rows evenly
    apart); scores float32 [G, W]; finished uint8 or bool [G, W].  Returns scores
    float32, parent rows int32 (as pages_fork takes them) and tokens int32, each [G, K].
    """
    dev = _dev_of(logits, "logits")
    if logits.dim() != 3:
        raise ValueError("logits must be [G, W, V]")
    if logits.dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise TypeError(f"logits must be bfloat16, float16 or float32, got {logits.dtype}")
    G, W, V = logits.shape
    sg, sw, sv = logits.stride()
    ld = V if G * W <= 1 else sw if W > 1 else sg
    if (V > 1 and sv != 1) or (G > 1 and W > 1 and sg != W * ld):
        raise ValueError("logits must have contiguous rows that lie evenly apart")
    _cuda(scores, "scores", dev, torch.float32, (G, W))
    if finished is not None:
        _cuda(finished, "finished", dev, torch.bool if finished.dtype == torch.bool else torch.uint8, (G, W))
    if out is None:
        out = _make(stream, lambda: tuple(torch.empty(G, K, dtype=dt, device=dev)
                                          for dt in (torch.float32, torch.int32, torch.int32)))
    else:
        best, parent, token = out
        _cuda(best, "out scores", dev, torch.float32, (G, K))
        _cuda(parent, "out parent", dev, torch.int32, (G, K))
        _cuda(token, "out token", dev, torch.int32, (G, K))
    if workspace is None:
        workspace = _make(stream, lambda: alloc_beam_workspace(G, W, V, K, dev))
    else:
        _cuda(workspace, "workspace", dev, torch.uint8)
    _call(_lib.gad_beam_select, dev, stream, logits.data_ptr(), _DTYPE_CODES[logits.dtype], ld,
          scores.data_ptr(), None if finished is None else finished.data_ptr(), int(pad_token), G, W, V,
          int(K), out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), workspace.data_ptr(),
          workspace.numel())
    return tuple(out)


def pages_workspace_bytes(rows: int, num_pages: int) -> int:
    n = _lib.gad_pages_workspace_bytes(int(rows), int(num_pages))
    if n == 0:
        raise GadError(-2, "gad_pages_workspace_bytes")
    return int(n)


def alloc_pages_workspace(rows: int, num_pages: int, device=None) -> torch.Tensor:
    """Scratch for the page operations on a pool of num_pages; its first word is
    their status (step_status).  A call that is given no workspace takes one of its
    own, whose status nobody can read: a pool without a page left then shows only in
    what the call returns (extend: cache_loc -1; fork: shorter lens)."""
    return torch.empty(pages_workspace_bytes(rows, num_pages), dtype=torch.uint8, device=device or "cuda")


def _pool(page_table, lens, refs):
    """Checks the pool's state; returns (device, rows, max_pages, num_pages)."""
    dev = _dev_of(page_table, "page_table")
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [rows, max_pages], got {list(page_table.shape)}")
    rows, max_pages = _cuda(page_table, "page_table", dev, torch.int32).shape
    _cuda(lens, "lens", dev, torch.int32, (rows,))
    num_pages = _cuda(refs, "refs", dev, torch.int32).numel()
    return dev, rows, max_pages, num_pages


def _pages_ws(workspace, rows, num_pages, dev, stream):
    if workspace is None:
        return _make(stream, lambda: alloc_pages_workspace(rows, num_pages, dev))
    return _cuda(workspace, "workspace", dev, torch.uint8)


_CACHE_DTYPES = (torch.uint8, torch.float8_e4m3fn)


def pages_copy(caches: list[torch.Tensor], src: torch.Tensor, dst: torch.Tensor,
               stream: torch.cuda.Stream | None = None) -> None:
    """Copies page src[i] to page dst[i] in every cache of the list (uint8 or E4M3
    [num_pages, page_size, hkv, 64], all of one shape) through gad_pages_copy; pairs
    with an id outside the pool (-1) are skipped."""
    dev, n = _dev_of(src, "src"), src.numel()
    _cuda(src, "src", dev, torch.int32, (n,))
    _cuda(dst, "dst", dev, torch.int32, (n,))
    if not caches:
        raise ValueError("caches must hold at least one tensor")
    shape = caches[0].shape
    ptrs = []
    for c in caches:
        if not (c.shape == shape and c.dtype in _CACHE_DTYPES and c.is_contiguous() and c.device == dev):
            _cuda(c, f"caches[{len(ptrs)}]", dev, torch.uint8, shape)
        ptrs.append(c.data_ptr())
    num_pages = shape[0] if shape else 0
    page_bytes = caches[0].numel() // num_pages if num_pages else 0
    ptrs = (ctypes.c_void_p * len(ptrs))(*ptrs)
    _call(_lib.gad_pages_copy, dev, stream, ptrs, len(caches), page_bytes, num_pages, src.data_ptr(),
          dst.data_ptr(), n)


def pages_fork(page_table: torch.Tensor, lens: torch.Tensor, parent: torch.Tensor, refs: torch.Tensor,
               page_size: int, out: tuple | None = None, workspace: torch.Tensor | None = None,
               stream: torch.cuda.Stream | None = None) -> tuple:
    """New rows that continue the old rows ``parent`` (int32, any shape; -1: empty) through
    gad_pages_fork.  Returns (page_table [n, max_pages], lens [n], copy_src [n], copy_dst [n]),
    all int32; refs is updated in place.  Entries behind a row's last page are not written
    (without ``out`` they are -1)."""
    dev, rows, max_pages, num_pages = _pool(page_table, lens, refs)
    _cuda(parent, "parent", dev, torch.int32)
    n = parent.numel()
    if out is None:
        out = _make(stream, lambda: (torch.full((n, max_pages), -1, dtype=torch.int32, device=dev),
                                     *(torch.empty(n, dtype=torch.int32, device=dev) for _ in range(3))))
    else:
        table, new_lens, src, dst = out
        _cuda(table, "out table", dev, torch.int32, (n, max_pages))
        _cuda(new_lens, "out lens", dev, torch.int32, (n,))
        _cuda(src, "copy_src", dev, torch.int32, (n,))
        _cuda(dst, "copy_dst", dev, torch.int32, (n,))
    ws = _pages_ws(workspace, max(rows, n), num_pages, dev, stream)
    _call(_lib.gad_pages_fork, dev, stream, page_table.data_ptr(), lens.data_ptr(), rows, parent.data_ptr(),
          n, max_pages, int(page_size), refs.data_ptr(), num_pages, *(t.data_ptr() for t in out),
          ws.data_ptr(), ws.numel())
    return tuple(out)


def pages_extend(page_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_size: int, L: int = 1,
                 out: tuple | None = None, workspace: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Room for L more tokens in every row that holds a request, through gad_pages_extend:
    page_table, lens and refs are updated in place; returns (positions, cache_loc) int64
    [rows * L] as attn_decode takes them."""
    dev, rows, max_pages, num_pages = _pool(page_table, lens, refs)
    if out is None:
        out = _make(stream, lambda: tuple(torch.empty(rows * max(int(L), 0), dtype=torch.int64, device=dev)
                                          for _ in range(2)))
    else:
        positions, cache_loc = out
        _cuda(positions, "positions", dev, torch.int64, (rows * L,))
        _cuda(cache_loc, "cache_loc", dev, torch.int64, (rows * L,))
    ws = _pages_ws(workspace, rows, num_pages, dev, stream)
    _call(_lib.gad_pages_extend, dev, stream, page_table.data_ptr(), lens.data_ptr(), rows, int(L),
          max_pages, int(page_size), refs.data_ptr(), num_pages, out[0].data_ptr(), out[1].data_ptr(),
          ws.data_ptr(), ws.numel())
    return tuple(out)


def pages_free(page_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_size: int,
               leave: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> None:
    """Releases the pages of the rows with leave[r] != 0 (uint8 or bool; None: all rows) and
    marks them empty, through gad_pages_free; lens and refs are updated in place.

    To shorten rows (tokens that were not accepted), release the pages behind their new
    ends before lowering lens, as rows of a table of their own:

        keep, had = -(-new // page_size), -(-lens // page_size)     # pages; new <= lens
        tail = page_table.gather(1, (keep[:, None] + cols).clamp(0, page_table.shape[1] - 1).long())
        pages_free(tail, (had - keep) * page_size, refs, page_size)
        lens.copy_(new)

    with cols = arange(the most pages that a row gives back)."""
    dev, rows, max_pages, num_pages = _pool(page_table, lens, refs)
    if leave is not None:
        _cuda(leave, "leave", dev, torch.bool if leave.dtype == torch.bool else torch.uint8, (rows,))
    _call(_lib.gad_pages_free, dev, stream, page_table.data_ptr(), lens.data_ptr(), rows, None if leave is
          None else leave.data_ptr(), max_pages, int(page_size), refs.data_ptr(), num_pages)


def pages_compact(page_table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, page_size: int,
                  max_moves: int | None = None, out: tuple | None = None, workspace: torch.Tensor | None = None,
                  stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Moves pages in use to the front of the pool through gad_pages_compact: page_table and
    refs are updated in place; returns (copy_src, copy_dst, used) int32 for pages_copy
    (max_moves pairs, -1 behind the last; by default enough for any pool)."""
    dev, rows, max_pages, num_pages = _pool(page_table, lens, refs)
    if out is None:
        m = max(1, num_pages // 2) if max_moves is None else int(max_moves)
        out = _make(stream, lambda: tuple(torch.empty(max(n, 0), dtype=torch.int32, device=dev)
                                          for n in (m, m, 1)))
    else:
        m = out[0].numel() if max_moves is None else int(max_moves)
        src, dst, used = out
        _cuda(src, "copy_src", dev, torch.int32, (m,))
        _cuda(dst, "copy_dst", dev, torch.int32, (m,))
        _cuda(used, "used", dev, torch.int32, (1,))
    ws = _pages_ws(workspace, rows, num_pages, dev, stream)
    _call(_lib.gad_pages_compact, dev, stream, page_table.data_ptr(), lens.data_ptr(), rows, max_pages,
          int(page_size), refs.data_ptr(), num_pages, out[0].data_ptr(), out[1].data_ptr(), m,
          out[2].data_ptr(), ws.data_ptr(), ws.numel())
    return tuple(out)
