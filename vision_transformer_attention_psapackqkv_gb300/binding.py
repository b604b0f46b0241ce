"""Thin Python binding of libpsa_gb300.so (the C ABI declared in include/psa.h).

Every function carries the C entry point's name and only marshals arguments:
torch tensors become device pointers, the current torch CUDA stream becomes the
cudaStream_t, and a non-OK status raises PsaError.  All computation happens in
the library's kernels; there is no fallback of any kind.  If the shared library
has not been built, the first call raises RuntimeError.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

PSA_OK = 0
PSA_DTYPE_F32 = 0
PSA_DTYPE_BF16 = 1

_lib = None


class PsaError(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn} failed with status {status}: {message}")
        self.status = status


class PsaShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("num_heads", ctypes.c_int), ("key_dim", ctypes.c_int),
                ("H", ctypes.c_int), ("W", ctypes.c_int), ("dtype", ctypes.c_int)]


class PsaRows(ctypes.Structure):
    """A view [B, heads, N, d]: base pointer and the strides of its first three dimensions."""
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_longlong), ("stride_h", ctypes.c_longlong),
                ("stride_n", ctypes.c_longlong)]


class PsaNormRope(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("num_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("N", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("rotary_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("max_pos", ctypes.c_int),
                ("eps", ctypes.c_float)]


class PsaWindow(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("num_heads", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("n_q", ctypes.c_int), ("n_k", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("window_left", ctypes.c_int), ("window_right", ctypes.c_int), ("sinks", ctypes.c_int)]


class PsaCache(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("num_kv_heads", ctypes.c_int), ("N", ctypes.c_int),
                ("max_len", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int)]


EXPORTED = (
    "psa_qkv_conv", "psa_pack_qkv", "psa_unpack_qkv", "psa_extract_v", "psa_merge_attn", "psa_unmerge_attn",
    "flash_attn2_fwd", "flash_attn2_bwd_dq", "flash_attn2_bwd_dkdv", "psa_attention_fwd",
    "psa_attention_fwd_residual", "psa_attention_bwd", "psa_attention_bwd_dq", "psa_attention_bwd_dkdv", "psa_attention_bwd_noalloc",
    "psa_attention_bwd_workspace_size", "psa_qk_norm_rope_fwd", "psa_qk_norm_rope_bwd",
    "psa_qk_norm_rope_bwd_workspace_size", "psa_window_attn_fwd", "psa_window_attn_bwd",
    "psa_window_attn_bwd_workspace_size", "psa_window_attn_decode", "psa_window_attn_decode_workspace_size",
    "psa_kv_append", "psa_kv4_append", "psa_kv4_read", "psa_window_attn_decode_kv4", "psa_status_string",
    "psa_get_last_device_error", "psa_debug_wait_timeout",
)


def library_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None):
    """Loads the shared library (built by ``_build.build()`` / ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libpsa_gb300.so is not built ({path}); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    P, I, F, S, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, PsaShape, ctypes.c_size_t
    R, NR, WN, CA = PsaRows, PsaNormRope, PsaWindow, PsaCache
    sigs = {
        "psa_qkv_conv": [P, P, P, P, I, I, I, I, I, P],
        "psa_pack_qkv": [P, P, S, P],
        "psa_unpack_qkv": [P, P, S, P],
        "psa_extract_v": [P, P, S, P],
        "psa_merge_attn": [P, P, P, S, P],
        "psa_unmerge_attn": [P, P, P, S, P],
        "flash_attn2_fwd": [P, P, P, P, P, I, I, I, F, I, P],
        "flash_attn2_bwd_dq": [P, P, P, P, P, P, P, P, I, I, I, F, I, P],
        "flash_attn2_bwd_dkdv": [P, P, P, P, P, P, P, P, I, I, I, F, I, P],
        "psa_attention_fwd": [P, P, P, P, S, F, P],
        "psa_attention_fwd_residual": [P, P, P, P, S, F, P],
        "psa_attention_bwd": [P, P, P, P, P, P, P, Z, S, F, P],
        "psa_attention_bwd_dq": [P, P, P, P, P, P, S, F, P],
        "psa_attention_bwd_dkdv": [P, P, P, P, P, P, S, F, P],
        "psa_attention_bwd_noalloc": [P, P, P, P, P, P, S, F, P],
        "psa_attention_bwd_workspace_size": [S],
        "psa_qk_norm_rope_fwd": [R, R, P, P, P, P, P, R, R, NR, P],
        "psa_qk_norm_rope_bwd": [R, R, P, P, P, P, P, R, R, R, R, P, P, P, Z, NR, P],
        "psa_qk_norm_rope_bwd_workspace_size": [NR],
        "psa_window_attn_fwd": [R, R, R, P, R, P, WN, F, P],
        "psa_window_attn_bwd": [R, R, R, R, R, P, P, R, R, R, P, Z, WN, F, P],
        "psa_window_attn_bwd_workspace_size": [WN],
        "psa_window_attn_decode": [R, R, R, P, R, P, Z, WN, F, P],
        "psa_window_attn_decode_workspace_size": [WN],
        "psa_kv_append": [R, R, P, P, R, R, CA, P],
        "psa_kv4_append": [R, R, P, P, P, P, P, P, CA, P],
        "psa_kv4_read": [P, P, P, P, R, R, CA, P],
        "psa_window_attn_decode_kv4": [R, P, P, P, P, P, R, P, Z, WN, F, P],
        "psa_status_string": [I],
        "psa_get_last_device_error": [P],
        "psa_debug_wait_timeout": [ctypes.c_ulonglong, P],
    }
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    for name in ("psa_attention_bwd", "psa_qk_norm_rope_bwd", "psa_window_attn_bwd", "psa_window_attn_decode"):
        getattr(lib, name + "_workspace_size").restype = ctypes.c_size_t
    lib.psa_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(fn: str, status: int):
    if status != PSA_OK:
        raise PsaError(fn, status, load().psa_status_string(status).decode())


def dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return PSA_DTYPE_BF16
    if t.dtype == torch.float32:
        return PSA_DTYPE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def shape_of(qkv, num_heads: int, key_dim: int) -> PsaShape:
    B, C, H, W = qkv.shape
    if C != num_heads * 4 * key_dim:
        raise ValueError(f"QKV has {C} channels, expected num_heads*4*key_dim = {num_heads * 4 * key_dim}")
    return PsaShape(B, num_heads, key_dim, H, W, dtype_code(qkv))


# ------------------------------------------------------------------ QKV convolution
def psa_qkv_conv(x, weight, bias, qkv, stream=None):
    """x [B, cin, H, W] bf16, weight [cout, cin] bf16, bias [cout] fp32 or None -> qkv."""
    Bn, cin, H, W = x.shape
    cout = weight.shape[0]
    _check("psa_qkv_conv", load().psa_qkv_conv(_ptr(x), _ptr(weight), _ptr(bias), _ptr(qkv), Bn, cin,
                                                cout, H, W, _stream(stream)))


# ------------------------------------------------------------------ layout
def psa_pack_qkv(qkv, packed, shape: PsaShape, stream=None):
    _check("psa_pack_qkv", load().psa_pack_qkv(_ptr(qkv), _ptr(packed), shape, _stream(stream)))


def psa_unpack_qkv(packed, qkv, shape: PsaShape, stream=None):
    _check("psa_unpack_qkv", load().psa_unpack_qkv(_ptr(packed), _ptr(qkv), shape, _stream(stream)))


def psa_extract_v(qkv, v_nchw, shape: PsaShape, stream=None):
    _check("psa_extract_v", load().psa_extract_v(_ptr(qkv), _ptr(v_nchw), shape, _stream(stream)))


def psa_merge_attn(o_lo, o_hi, out, shape: PsaShape, stream=None):
    _check("psa_merge_attn", load().psa_merge_attn(_ptr(o_lo), _ptr(o_hi), _ptr(out), shape, _stream(stream)))


def psa_unmerge_attn(dout, do_lo, do_hi, shape: PsaShape, stream=None):
    _check("psa_unmerge_attn",
           load().psa_unmerge_attn(_ptr(dout), _ptr(do_lo), _ptr(do_hi), shape, _stream(stream)))


# ------------------------------------------------------------------ Flash Attention 2
def flash_attn2_fwd(q, k, v, o, lse, scale: float, stream=None):
    BH, N, d = q.shape
    _check("flash_attn2_fwd", load().flash_attn2_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), BH, N, d, float(scale), dtype_code(q),
        _stream(stream)))


def flash_attn2_bwd_dq(q, k, v, o, do, lse, delta, dq, scale: float, stream=None):
    BH, N, d = q.shape
    _check("flash_attn2_bwd_dq", load().flash_attn2_bwd_dq(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(delta), _ptr(dq), BH, N, d,
        float(scale), dtype_code(q), _stream(stream)))


def flash_attn2_bwd_dkdv(q, k, v, do, lse, delta, dk, dv, scale: float, stream=None):
    BH, N, d = q.shape
    _check("flash_attn2_bwd_dkdv", load().flash_attn2_bwd_dkdv(
        _ptr(q), _ptr(k), _ptr(v), _ptr(do), _ptr(lse), _ptr(delta), _ptr(dk), _ptr(dv), BH, N, d,
        float(scale), dtype_code(q), _stream(stream)))


# ------------------------------------------------------------------ fused PSA
def psa_attention_fwd(qkv, out, lse, v_nchw, shape: PsaShape, scale: float, stream=None):
    _check("psa_attention_fwd", load().psa_attention_fwd(
        _ptr(qkv), _ptr(out), _ptr(lse), _ptr(v_nchw), shape, float(scale), _stream(stream)))


def psa_attention_fwd_residual(qkv, out_res, out, lse, shape: PsaShape, scale: float, stream=None):
    _check("psa_attention_fwd_residual", load().psa_attention_fwd_residual(
        _ptr(qkv), _ptr(out_res), _ptr(out), _ptr(lse), shape, float(scale), _stream(stream)))


def psa_attention_bwd_workspace_size(shape: PsaShape) -> int:
    return int(load().psa_attention_bwd_workspace_size(shape))


def psa_attention_bwd(qkv, out, dout, lse, dvres, dqkv, workspace, shape: PsaShape, scale: float,
                      stream=None):
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("psa_attention_bwd", load().psa_attention_bwd(
        _ptr(qkv), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dvres), _ptr(dqkv), _ptr(workspace),
        ws_bytes, shape, float(scale), _stream(stream)))


def psa_attention_bwd_dq(qkv, out, dout, lse, delta, dqkv, shape: PsaShape, scale: float, stream=None):
    _check("psa_attention_bwd_dq", load().psa_attention_bwd_dq(
        _ptr(qkv), _ptr(out), _ptr(dout), _ptr(lse), _ptr(delta), _ptr(dqkv), shape, float(scale),
        _stream(stream)))


def psa_attention_bwd_dkdv(qkv, dout, lse, delta, dvres, dqkv, shape: PsaShape, scale: float, stream=None):
    _check("psa_attention_bwd_dkdv", load().psa_attention_bwd_dkdv(
        _ptr(qkv), _ptr(dout), _ptr(lse), _ptr(delta), _ptr(dvres), _ptr(dqkv), shape, float(scale),
        _stream(stream)))


def psa_attention_bwd_noalloc(qkv, out, dout, lse, dvres, dqkv, shape: PsaShape, scale: float, stream=None):
    _check("psa_attention_bwd_noalloc", load().psa_attention_bwd_noalloc(
        _ptr(qkv), _ptr(out), _ptr(dout), _ptr(lse), _ptr(dvres), _ptr(dqkv), shape, float(scale),
        _stream(stream)))


# ------------------------------------------------------------------ token sequences
# Views are torch tensors [B, heads, N, d] of any strides whose channels are contiguous.
# The calls run on the tensors' device, on its current stream unless one is given.
# A decoding step's calls are as long on the host as on the device, so their checks go over
# plain tuples and integers.
def _wrong(t, shape, dtype, what: str):
    """Raises what is wrong with an argument that failed its check."""
    if t is None:
        raise ValueError(f"{what} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{what} is {t.dtype}, expected {dtype}")
    raise ValueError(f"{what} must be contiguous")


def _rows(t, shape, dtype, what: str) -> PsaRows:
    if t is None or t.shape != shape or t.dtype != dtype:
        _wrong(t, shape, dtype, what)
    sb, sh, sn, sc = t.stride()
    if sc != 1 and shape[3] != 1:
        raise ValueError(f"{what}: the channels of a row must be contiguous")
    return PsaRows(t.data_ptr(), sb, sh, sn)


def _dense(t, shape, dtype, what: str):
    """Address of a dense array of that shape and type; None for None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        _wrong(t, shape, dtype, what)
    return t.data_ptr()


def _type_of(p, t):
    """The type of t, which problem p has to have been made for: its kernels read rows of that type."""
    if dtype_code(t) != p.dtype:
        raise TypeError(f"the problem was made for another type than {t.dtype}")
    return t.dtype


def _on_device(fn: str, tensors, stream, *args):
    """Calls entry point `fn` with its arguments on the tensors' one CUDA device."""
    import torch

    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"{fn}: tensors on {tensors[0].device} and {t.device}")
    if index < 0:
        raise ValueError(f"{fn}: tensors must be on a CUDA device, got {tensors[0].device}")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    call = getattr(_lib or load(), fn)
    if torch._C._cuda_getDevice() == index:
        status = call(*args, raw)
    else:
        with torch.cuda.device(index):
            status = call(*args, raw)
    if status != PSA_OK:
        _check(fn, status)


def _workspace(t, fn: str):
    if t is None or not t.is_contiguous():
        raise ValueError(f"{fn}: the workspace must be a contiguous tensor")
    return t.data_ptr(), t.numel() * t.element_size()


def norm_rope_of(q, k, cos, eps: float = 1e-6, interleaved: bool = False) -> PsaNormRope:
    """The problem of q [B, num_heads, N, d], k [B, num_kv_heads, N, d] and a table cos
    [max_pos, rotary_dim / 2] (None: no rotation)."""
    B, nh, N, d = q.shape
    rot, max_pos = (0, 2 ** 31 - 1) if cos is None else (2 * cos.shape[1], cos.shape[0])
    return PsaNormRope(B, nh, k.shape[1], N, d, dtype_code(q), rot, int(bool(interleaved)), max_pos, float(eps))


def _norm_rope_inputs(q, k, q_weight, k_weight, cos, sin, positions, p):
    import torch

    B, N, d, f32, t = p.B, p.N, p.head_dim, torch.float32, _type_of(p, q)
    table, by_q, by_k = (p.max_pos, p.rotary_dim // 2), (B, p.num_heads, N, d), (B, p.num_kv_heads, N, d)
    return by_q, by_k, (_rows(q, by_q, t, "q"), _rows(k, by_k, t, "k"), _dense(q_weight, (d,), f32, "q_weight"),
                        _dense(k_weight, (d,), f32, "k_weight"), _dense(cos, table, f32, "cos"),
                        _dense(sin, table, f32, "sin"), _dense(positions, (B, N), torch.int32, "positions"))


def psa_qk_norm_rope_fwd(q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out, p: PsaNormRope,
                         stream=None):
    by_q, by_k, args = _norm_rope_inputs(q, k, q_weight, k_weight, cos, sin, positions, p)
    _on_device("psa_qk_norm_rope_fwd", (q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out), stream,
               *args, _rows(q_out, by_q, q.dtype, "q_out"), _rows(k_out, by_k, q.dtype, "k_out"), p)


def psa_qk_norm_rope_bwd_workspace_size(p: PsaNormRope) -> int:
    return int(load().psa_qk_norm_rope_bwd_workspace_size(p))


def psa_qk_norm_rope_bwd(q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, dq, dk, dq_weight,
                         dk_weight, workspace, p: PsaNormRope, stream=None):
    import torch

    by_q, by_k, args = _norm_rope_inputs(q, k, q_weight, k_weight, cos, sin, positions, p)
    t, d = q.dtype, (p.head_dim,)
    _on_device("psa_qk_norm_rope_bwd",
               (q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, dq, dk, dq_weight, dk_weight,
                workspace), stream, *args, _rows(dq_out, by_q, t, "dq_out"), _rows(dk_out, by_k, t, "dk_out"),
               _rows(dq, by_q, t, "dq"), _rows(dk, by_k, t, "dk"), _dense(dq_weight, d, torch.float32, "dq_weight"),
               _dense(dk_weight, d, torch.float32, "dk_weight"), *_workspace(workspace, "psa_qk_norm_rope_bwd"), p)


def window_of(q, k, window_left: int = -1, window_right: int = 0, sinks: int = 0) -> PsaWindow:
    """The problem of q [B, num_heads, n_q, d] against keys, a cache or its codes k
    [B, num_kv_heads, n_k, ...]; a negative window has no limit on that side.  The last query
    stands at the last key's position: with n_q > n_k the first n_q - n_k see nothing."""
    B, nh, n_q, d = q.shape
    n_k = k.shape[2]
    # nothing is past n_k, and all that is negative is alike; a C int would drop the upper bits
    left, right, sinks = (max(-1, min(int(w), n_k)) for w in (window_left, window_right, sinks))
    return PsaWindow(B, nh, k.shape[1], n_q, n_k, d, dtype_code(q), left, right, sinks)


def _window_shapes(win: PsaWindow):
    """Shapes of what goes by the queries, and by the keys."""
    B, d = win.B, win.head_dim
    return (B, win.num_heads, win.n_q, d), (B, win.num_kv_heads, win.n_k, d)


def _lens(lens, win: PsaWindow):
    import torch

    return _dense(lens, (win.B,), torch.int32, "lens")


def psa_window_attn_fwd(q, k, v, lens, o, lse, win: PsaWindow, scale: float, stream=None):
    import torch

    by_q, by_k = _window_shapes(win)
    t = _type_of(win, q)
    _on_device("psa_window_attn_fwd", (q, k, v, lens, o, lse), stream, _rows(q, by_q, t, "q"), _rows(k, by_k, t, "k"),
               _rows(v, by_k, t, "v"), _lens(lens, win), _rows(o, by_q, t, "o"),
               _dense(lse, by_q[:3], torch.float32, "lse"), win, scale)


def psa_window_attn_bwd_workspace_size(win: PsaWindow) -> int:
    return int(load().psa_window_attn_bwd_workspace_size(win))


def psa_window_attn_bwd(q, k, v, o, do, lse, lens, dq, dk, dv, workspace, win: PsaWindow, scale: float,
                        stream=None):
    import torch

    by_q, by_k = _window_shapes(win)
    t = _type_of(win, q)
    _on_device("psa_window_attn_bwd", (q, k, v, o, do, lse, lens, dq, dk, dv, workspace), stream,
               _rows(q, by_q, t, "q"), _rows(k, by_k, t, "k"), _rows(v, by_k, t, "v"), _rows(o, by_q, t, "o"),
               _rows(do, by_q, t, "do"), _dense(lse, by_q[:3], torch.float32, "lse"), _lens(lens, win),
               _rows(dq, by_q, t, "dq"), _rows(dk, by_k, t, "dk"), _rows(dv, by_k, t, "dv"),
               *_workspace(workspace, "psa_window_attn_bwd"), win, scale)


def psa_window_attn_decode_workspace_size(win: PsaWindow) -> int:
    return int(load().psa_window_attn_decode_workspace_size(win))


def psa_window_attn_decode(q, k_cache, v_cache, lens, o, workspace, win: PsaWindow, scale: float, stream=None):
    by_q, by_k = _window_shapes(win)
    t = _type_of(win, q)
    _on_device("psa_window_attn_decode", (q, k_cache, v_cache, lens, o, workspace), stream, _rows(q, by_q, t, "q"),
               _rows(k_cache, by_k, t, "k_cache"), _rows(v_cache, by_k, t, "v_cache"), _lens(lens, win),
               _rows(o, by_q, t, "o"), *_workspace(workspace, "psa_window_attn_decode"), win, scale)


def cache_of(k, max_len: int) -> PsaCache:
    """Rows k [B, num_kv_heads, N, d] next to a cache of max_len rows."""
    B, nkv, N, d = k.shape
    return PsaCache(B, nkv, N, int(max_len), d, dtype_code(k))


def _cache_rows(starts, counts, p: PsaCache):
    import torch

    return (_dense(starts, (p.B,), torch.int32, "starts"), _dense(counts, (p.B,), torch.int32, "counts"))


def _kv4(k_codes, k_scales, v_codes, v_scales, B, nkv, max_len, d):
    import torch

    codes, scales = (B, nkv, max_len, d // 2), (B, nkv, max_len, d // 32)
    return (_dense(k_codes, codes, torch.uint8, "k_codes"), _dense(k_scales, scales, torch.bfloat16, "k_scales"),
            _dense(v_codes, codes, torch.uint8, "v_codes"), _dense(v_scales, scales, torch.bfloat16, "v_scales"))


def psa_kv_append(k, v, starts, counts, k_cache, v_cache, stream=None):
    p = cache_of(k, k_cache.shape[2])
    rows, cache = (p.B, p.num_kv_heads, p.N, p.head_dim), (p.B, p.num_kv_heads, p.max_len, p.head_dim)
    _on_device("psa_kv_append", (k, v, starts, counts, k_cache, v_cache), stream, _rows(k, rows, k.dtype, "k"),
               _rows(v, rows, k.dtype, "v"), *_cache_rows(starts, counts, p),
               _rows(k_cache, cache, k.dtype, "k_cache"), _rows(v_cache, cache, k.dtype, "v_cache"), p)


def psa_kv4_append(k, v, starts, counts, k_codes, k_scales, v_codes, v_scales, stream=None):
    p = cache_of(k, k_codes.shape[2])
    rows, cache = (p.B, p.num_kv_heads, p.N, p.head_dim), (k_codes, k_scales, v_codes, v_scales)
    _on_device("psa_kv4_append", (k, v, starts, counts, *cache), stream, _rows(k, rows, k.dtype, "k"),
               _rows(v, rows, k.dtype, "v"), *_cache_rows(starts, counts, p),
               *_kv4(*cache, p.B, p.num_kv_heads, p.max_len, p.head_dim), p)


def psa_kv4_read(k_codes, k_scales, v_codes, v_scales, k, v, stream=None):
    """Rows 0 .. N - 1 of the cache into k and v [B, num_kv_heads, N, d]."""
    p = cache_of(k, k_codes.shape[2])
    rows, cache = (p.B, p.num_kv_heads, p.N, p.head_dim), (k_codes, k_scales, v_codes, v_scales)
    _on_device("psa_kv4_read", (k, v, *cache), stream, *_kv4(*cache, p.B, p.num_kv_heads, p.max_len, p.head_dim),
               _rows(k, rows, k.dtype, "k"), _rows(v, rows, k.dtype, "v"), p)


def psa_window_attn_decode_kv4(q, k_codes, k_scales, v_codes, v_scales, lens, o, workspace, win: PsaWindow,
                               scale: float, stream=None):
    cache = (k_codes, k_scales, v_codes, v_scales)
    by_q, (B, nkv, max_len, d) = _window_shapes(win)
    t = _type_of(win, q)
    _on_device("psa_window_attn_decode_kv4", (q, *cache, lens, o, workspace), stream, _rows(q, by_q, t, "q"),
               *_kv4(*cache, B, nkv, max_len, d), _lens(lens, win), _rows(o, by_q, t, "o"),
               *_workspace(workspace, "psa_window_attn_decode_kv4"), win, scale)


def psa_get_last_device_error(stream=None) -> int:
    return int(load().psa_get_last_device_error(_stream(stream)))


def psa_debug_wait_timeout(limit_ns: int, stream=None):
    _check("psa_debug_wait_timeout", load().psa_debug_wait_timeout(int(limit_ns), _stream(stream)))


def psa_status_string(status: int) -> str:
    return load().psa_status_string(int(status)).decode()
