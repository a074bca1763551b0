"""Python binding of the CSA2 C ABI (``include/csa2.h``, ``libcsa2.so``).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (torch supplies device memory and
streams); calls are enqueued on torch's current stream.  Importing this
package raises if the library has not been built -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

from ._build import LIB, bind_path

__all__ = ["Csa2Error", "lib", "csa2_cache", "csa2_window", "csa2_model", "csa2_step_in",
           "csa2_step_out", "pack_cache", "index_topk", "index_topk_workspace", "index_pool_workspace",
           "index_topk_pool", "index_topk_in_pool", "POOL_BLOCK", "MAX_POOL_BLOCKS", "WIN_BF16", "WIN_FP8",
           "sparse_attn",
           "sparse_attn_workspace", "window_append", "layer_step", "layer_step_workspace", "layer_step_launches", "seq_image_bytes", "cache_export",
           "cache_import", "csa2_heads", "csa2_rotary", "csa2_kv_cache", "rotary", "rotate", "kv_cache", "kv_append",
           "kv_attn", "kv_attn_workspace", "KV_BF16", "KV_F16", "KV_E4M3",
           "SWA_ONLY", "FULL", "REINDEX", "REUSE", "DTYPE_BF16", "DTYPE_F32", "DTYPE_F16"]

SWA_ONLY, FULL, REINDEX, REUSE = 0, 1, 2, 3
DTYPE_BF16, DTYPE_F32, DTYPE_F16 = 0, 1, 2
POOL_BLOCK, MAX_POOL_BLOCKS = 8, 8192
WIN_BF16, WIN_FP8 = 0, 1
KV_BF16, KV_F16, KV_E4M3 = 0, 1, 2
MAX_ROT = 256
DEVERR_CAPACITY, DEVERR_PAGE, DEVERR_COUNT, DEVERR_TIMEOUT, DEVERR_IMAGE = 1, 2, 4, 8, 16

_vp, _i32, _f32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t


class Csa2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {lib().csa2_strerror(status).decode()} ({status})")
        self.status = status


class csa2_cache(ctypes.Structure):
    _fields_ = [("main_codes", _vp), ("main_scales", _vp), ("idx_codes", _vp), ("idx_scales", _vp),
                ("page_table", _vp), ("n_entries", _vp), ("pend_x", _vp), ("pend_g", _vp),
                ("pend_valid", _vp), ("status", _vp), ("batch", _i32), ("max_pages", _i32),
                ("num_pages", _i32), ("ratio", _i32)]


class csa2_window(ctypes.Structure):
    _fields_ = [("tokens", _vp), ("count", _vp), ("batch", _i32), ("dtype", _i32)]


class csa2_model(ctypes.Structure):
    _fields_ = [("n_layers", _i32), ("n_sources", _i32), ("mode", ctypes.POINTER(_i32)),
                ("src", ctypes.POINTER(_i32)), ("idx_src", ctypes.POINTER(_i32)),
                ("caches", ctypes.POINTER(csa2_cache)), ("w_idx", ctypes.POINTER(_vp)),
                ("windows", ctypes.POINTER(csa2_window)), ("batch", _i32), ("H", _i32),
                ("H_idx", _i32), ("K", _i32), ("scale", _f32), ("pool_blocks", _i32)]


class csa2_step_in(ctypes.Structure):
    _fields_ = [("x_new", ctypes.POINTER(_vp)), ("g_new", ctypes.POINTER(_vp)),
                ("q", ctypes.POINTER(_vp)), ("q_idx", ctypes.POINTER(_vp)), ("w", ctypes.POINTER(_vp)),
                ("win_tok", ctypes.POINTER(_vp))]


class csa2_step_out(ctypes.Structure):
    _fields_ = [("out", ctypes.POINTER(_vp)), ("idx", ctypes.POINTER(_vp))]


class csa2_heads(ctypes.Structure):
    _fields_ = [("data", _vp), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class csa2_rotary(ctypes.Structure):
    _fields_ = [("inv_freq", _vp), ("axis", ctypes.POINTER(ctypes.c_uint8)), ("rot_dim", _i32),
                ("rot_offset", _i32), ("neighbours", _i32), ("n_axes", _i32)]


class csa2_kv_cache(ctypes.Structure):
    _fields_ = [("k_pages", _vp), ("v_pages", _vp), ("page_table", _vp), ("n_tokens", _vp), ("status", _vp),
                ("batch", _i32), ("max_pages", _i32), ("num_pages", _i32), ("kv_heads", _i32),
                ("head_dim", _i32), ("dtype", _i32)]


_lib = None


def lib():
    """The loaded libcsa2.so (raises if it is missing: no CPU fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise ImportError(f"{LIB} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB)
        P = ctypes.POINTER
        for name, res, args in [
            ("csa2_version", ctypes.c_int, []),
            ("csa2_strerror", ctypes.c_char_p, [ctypes.c_int]),
            ("csa2_pack_cache", ctypes.c_int, [P(csa2_cache), _vp, ctypes.c_int, _vp, _vp, ctypes.c_int, _vp]),
            ("csa2_index_topk_workspace", _sz, [ctypes.c_int] * 4),
            ("csa2_index_topk", ctypes.c_int, [P(csa2_cache), _vp, _vp, ctypes.c_int, ctypes.c_int, _vp,
                                               _vp, _vp, _sz, _vp]),
            ("csa2_index_pool_workspace", _sz, [ctypes.c_int] * 5),
            ("csa2_index_topk_pool", ctypes.c_int, [P(csa2_cache), _vp, _vp, ctypes.c_int, ctypes.c_int, _vp,
                                                    _vp, ctypes.c_int, _vp, _vp, _sz, _vp]),
            ("csa2_index_topk_in_pool", ctypes.c_int, [P(csa2_cache), _vp, _vp, ctypes.c_int, ctypes.c_int,
                                                       _vp, ctypes.c_int, _vp, _vp, _vp, _sz, _vp]),
            ("csa2_sparse_attn_workspace", _sz, [ctypes.c_int] * 3),
            ("csa2_sparse_attn", ctypes.c_int, [P(csa2_cache), _vp, ctypes.c_int, _vp, ctypes.c_int,
                                                P(csa2_window), ctypes.c_float, _vp, _vp, _sz, _vp]),
            ("csa2_window_append", ctypes.c_int, [P(csa2_window), _vp, _vp]),
            ("csa2_layer_step_workspace", _sz, [P(csa2_model)]),
            ("csa2_layer_step", ctypes.c_int, [P(csa2_model), P(csa2_step_in), P(csa2_step_out), _vp,
                                               _sz, _vp]),
            ("csa2_layer_step_launches", ctypes.c_int, [P(csa2_model), P(csa2_step_in)]),
            ("csa2_seq_image_bytes", _sz, [ctypes.c_int]),
            ("csa2_cache_export", ctypes.c_int, [P(csa2_cache), ctypes.c_int, _vp, ctypes.c_int, _vp]),
            ("csa2_cache_import", ctypes.c_int, [P(csa2_cache), ctypes.c_int, _vp, ctypes.c_int, _vp]),
            ("csa2_rotate", ctypes.c_int, [P(csa2_rotary), P(csa2_heads), P(csa2_heads), ctypes.c_int,
                                           ctypes.c_int64, ctypes.c_int, ctypes.c_int, _vp, ctypes.c_int, _vp]),
            ("csa2_kv_append", ctypes.c_int, [P(csa2_kv_cache), P(csa2_heads), P(csa2_heads), ctypes.c_int, _vp,
                                              ctypes.c_int, ctypes.c_int, _vp, P(csa2_rotary), _vp, _vp]),
            ("csa2_kv_attn_workspace", _sz, [P(csa2_kv_cache), ctypes.c_int, ctypes.c_int, ctypes.c_int]),
            ("csa2_kv_attn", ctypes.c_int, [P(csa2_kv_cache), P(csa2_heads), ctypes.c_int, ctypes.c_int, _vp,
                                            ctypes.c_int, ctypes.c_int, _f32, ctypes.c_int, P(csa2_heads), _vp,
                                            _vp, _sz, _vp]),
        ]:
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ok(rc: int, what: str):
    if rc != 0:
        raise Csa2Error(rc, what)


def pack_cache(cache: csa2_cache, x, gates, w_idx, stream=None):
    """Append x [batch][T][512] (bf16 or fp32) with gate logits [batch][T]."""
    import torch
    dt = DTYPE_F32 if x.dtype == torch.float32 else DTYPE_BF16
    T = x.shape[1]
    _ok(lib().csa2_pack_cache(ctypes.byref(cache), _ptr(x), dt, _ptr(gates), _ptr(w_idx), T,
                              _stream(stream)), "csa2_pack_cache")


def index_topk_workspace(batch: int, max_entries: int, H_idx: int, K: int) -> int:
    return int(lib().csa2_index_topk_workspace(batch, max_entries, H_idx, K))


def index_topk(cache: csa2_cache, q_idx, w, K: int, idx_out, ws, score_out=None, stream=None):
    H_idx = q_idx.shape[1]
    _ok(lib().csa2_index_topk(ctypes.byref(cache), _ptr(q_idx), _ptr(w), H_idx, K, _ptr(idx_out),
                              _ptr(score_out), _ptr(ws), ws.numel() * ws.element_size(),
                              _stream(stream)), "csa2_index_topk")


def index_pool_workspace(batch: int, max_entries: int, H_idx: int, K: int, pool_blocks: int) -> int:
    return int(lib().csa2_index_pool_workspace(batch, max_entries, H_idx, K, pool_blocks))


def index_topk_pool(cache: csa2_cache, q_idx, w, K: int, idx_out, pool_out, ws, score_out=None,
                    stream=None):
    """Full-layer scan: Top-K into idx_out and the block pool into pool_out
    [batch][pool_blocks]."""
    H_idx = q_idx.shape[1]
    _ok(lib().csa2_index_topk_pool(ctypes.byref(cache), _ptr(q_idx), _ptr(w), H_idx, K, _ptr(idx_out),
                                   _ptr(score_out), pool_out.shape[1], _ptr(pool_out), _ptr(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)), "csa2_index_topk_pool")


def index_topk_in_pool(cache: csa2_cache, q_idx, w, K: int, pool, idx_out, ws, score_out=None, stream=None):
    """Scan restricted to pool [batch][pool_blocks]; Top-K into idx_out."""
    H_idx = q_idx.shape[1]
    _ok(lib().csa2_index_topk_in_pool(ctypes.byref(cache), _ptr(q_idx), _ptr(w), H_idx, K, _ptr(pool),
                                      pool.shape[1], _ptr(idx_out), _ptr(score_out), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream)),
        "csa2_index_topk_in_pool")


def sparse_attn_workspace(batch: int, H: int, K: int) -> int:
    return int(lib().csa2_sparse_attn_workspace(batch, H, K))


def sparse_attn(cache, q, idx, K: int, win: csa2_window, scale: float, out, ws, stream=None):
    H = q.shape[1]
    cp = ctypes.byref(cache) if cache is not None else None
    _ok(lib().csa2_sparse_attn(cp, _ptr(q), H, _ptr(idx), K, ctypes.byref(win), float(scale), _ptr(out),
                               _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
        "csa2_sparse_attn")


def selftest_wait_timeout(status, timeout_us: int, stream=None):
    """Make one bounded device wait run out (see csa2_selftest_wait_timeout):
    CSA2_DEVERR_TIMEOUT is ORed into status[0] after timeout_us microseconds."""
    f = lib().csa2_selftest_wait_timeout
    f.restype = ctypes.c_int
    f.argtypes = [_vp, ctypes.c_uint, _vp]
    _ok(f(_ptr(status), int(timeout_us), _stream(stream)), "csa2_selftest_wait_timeout")


def window_append(win: csa2_window, tok, stream=None):
    _ok(lib().csa2_window_append(ctypes.byref(win), _ptr(tok), _stream(stream)), "csa2_window_append")


def layer_step_workspace(model: csa2_model) -> int:
    return int(lib().csa2_layer_step_workspace(ctypes.byref(model)))


def layer_step(model: csa2_model, step_in: csa2_step_in, step_out: csa2_step_out, ws, stream=None):
    _ok(lib().csa2_layer_step(ctypes.byref(model), ctypes.byref(step_in), ctypes.byref(step_out),
                              _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
        "csa2_layer_step")


def layer_step_launches(model: csa2_model, step_in: csa2_step_in) -> int:
    """Kernel launches one layer_step call enqueues (no work is enqueued)."""
    n = int(lib().csa2_layer_step_launches(ctypes.byref(model), ctypes.byref(step_in)))
    if n < 0:
        raise Csa2Error(n, "csa2_layer_step_launches")
    return n


def seq_image_bytes(capacity: int) -> int:
    """Bytes of a one-sequence cache image with room for `capacity` entries."""
    return int(lib().csa2_seq_image_bytes(capacity))


def cache_export(cache: csa2_cache, seq: int, image, capacity: int, stream=None):
    """Copy sequence `seq` of `cache` into `image` (a uint8 tensor the device can
    address: CUDA memory or pinned host memory) in logical entry order."""
    _ok(lib().csa2_cache_export(ctypes.byref(cache), seq, _ptr(image), capacity, _stream(stream)),
        "csa2_cache_export")


def cache_import(cache: csa2_cache, seq: int, image, capacity: int, stream=None):
    """Write an image made by cache_export into sequence `seq` of `cache`."""
    _ok(lib().csa2_cache_import(ctypes.byref(cache), seq, _ptr(image), capacity, _stream(stream)),
        "csa2_cache_import")


def index_topk_noalloc(cache: csa2_cache, q_idx, w, K: int, idx_out, score_out=None, stream=None):
    """csa2_index_topk without a workspace: for callers that cannot allocate
    device memory (a fixed memory pool, no allocation on the decode path).  The
    scratch is a fixed 8 MiB array inside the library; see include/csa2.h."""
    f = lib().csa2_index_topk_noalloc
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.POINTER(csa2_cache), _vp, _vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp]
    H_idx = q_idx.shape[1]
    _ok(f(ctypes.byref(cache), _ptr(q_idx), _ptr(w), H_idx, K, _ptr(idx_out), _ptr(score_out),
          _stream(stream)), "csa2_index_topk_noalloc")


# ---------------------------------------------------------------- paged key/value cache
#
# The calls themselves (checks of the tensors, device guard, stream) are csrc/bind.cpp's.

_bind = None


def _calls():
    """The loaded module with the calls (raises if it is missing)."""
    global _bind
    if _bind is None:
        import importlib.util
        import torch  # noqa: F401  (its libraries are loaded first)
        path = bind_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is not built; run __graft_entry__.build() first")
        spec = importlib.util.spec_from_file_location("_bind", path)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        L = lib()
        m.init(*[ctypes.cast(f, _vp).value for f in (L.csa2_rotate, L.csa2_kv_append, L.csa2_kv_attn)])
        _bind = m
    return _bind


def _want(t, what, dtype, shape, index=None):
    """A contiguous CUDA tensor of this dtype and shape (the library sees only its address); its device index."""
    at = t.get_device()
    if at < 0 or (index is not None and at != index):
        raise ValueError(f"{what} is on {t.device}, not on the call's CUDA device")
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"not {t.dtype} {tuple(t.shape)}")
    return at


def _int32(**numbers) -> None:
    """ctypes would keep the low bits only."""
    for what, n in numbers.items():
        if not -(1 << 31) <= n < 1 << 31:
            raise ValueError(f"{what} = {n} is out of range")


def rotary(inv_freq, rot_dim: int, offset: int = 0, neighbours: bool = False, n_axes: int = 1, axis=None) -> csa2_rotary:
    """A rotation: channels offset .. offset + rot_dim - 1 of a head turn in pairs (neighbours, or half the
    rotation apart) by position * inv_freq[pair] (fp32 CUDA tensor).  axis (a list, one entry per pair) says
    which of the n_axes positions turns it."""
    import torch
    _int32(rot_dim=rot_dim, offset=offset, n_axes=n_axes)
    if axis is not None and not all(0 <= a < n_axes for a in axis):
        raise ValueError(f"axis has entries outside 0 .. {n_axes - 1}")
    index = _want(inv_freq, "inv_freq", torch.float32, (rot_dim // 2,))
    r = csa2_rotary(inv_freq.data_ptr(), None, rot_dim, offset, int(neighbours), n_axes)
    if axis is not None:
        if len(axis) != rot_dim // 2:
            raise ValueError(f"axis has {len(axis)} entries, not one for each of the {rot_dim // 2} pairs")
        r.axis = (ctypes.c_uint8 * len(axis))(*axis)
    r._keep, r._index = inv_freq, index  # the descriptor holds its address
    return r


def rotate(rot: csa2_rotary, x, pos, out, inverse: bool = False, stream=None):
    """out = x [tokens][heads][channels] rotated at pos int32 [n_axes][tokens] (out may be x); inverse turns back."""
    rc = (_bind or _calls()).rotate(rot, x, pos, out, inverse, stream)
    if rc:
        raise Csa2Error(rc, "csa2_rotate")


def kv_cache(k_pages, v_pages, page_table, n_tokens, status) -> csa2_kv_cache:
    """Descriptor of a paged key/value cache: pools [pages][kv_heads][64][head_dim] (bf16, fp16 or float8_e4m3fn),
    page_table int32 [batch][max_pages], n_tokens int32 [batch], status int32 (one word or more)."""
    import torch
    types = {torch.bfloat16: KV_BF16, torch.float16: KV_F16, torch.float8_e4m3fn: KV_E4M3}
    pages, heads, rows, dim = k_pages.shape
    if rows != 64:
        raise ValueError(f"a page has 64 rows, not {rows}")
    if k_pages.dtype not in types:
        raise ValueError(f"k_pages: {k_pages.dtype} is not supported")
    index = _want(k_pages, "k_pages", k_pages.dtype, k_pages.shape)
    _want(v_pages, "v_pages", k_pages.dtype, k_pages.shape, index)
    batch, max_pages = page_table.shape
    _want(page_table, "page_table", torch.int32, (batch, max_pages), index)
    _want(n_tokens, "n_tokens", torch.int32, (batch,), index)
    if status.get_device() != index or status.element_size() != 4 or status.numel() < 1:
        raise ValueError("status must be a tensor of 32-bit words on the cache's device")
    c = csa2_kv_cache(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), n_tokens.data_ptr(),
                      status.data_ptr(), batch, max_pages, pages, heads, dim, types[k_pages.dtype])
    c._keep, c._index = (k_pages, v_pages, page_table, n_tokens, status), index  # the descriptor holds their addresses
    return c


def kv_append(cache: csa2_kv_cache, k, v, cu, max_new: int, start=None, rotary=None, pos=None, stream=None):
    """Write the new tokens k, v [total][kv_heads][head_dim] (sequence b: rows cu[b] .. cu[b + 1] - 1) behind
    start (int32 [batch]; None: behind the tokens held), the keys rotated at pos int32 [n_axes][total]
    (None: their slots)."""
    rc = (_bind or _calls()).kv_append(cache, k, v, cu, max_new, start, rotary, pos, stream)
    if rc:
        raise Csa2Error(rc, "csa2_kv_append")


def kv_attn_workspace(cache: csa2_kv_cache, total: int, max_new: int, H: int) -> int:
    """Bytes of workspace for kv_attn calls of these sizes; what does for max_new does for fewer."""
    import torch
    _int32(total=total, max_new=max_new, H=H)
    with torch.cuda.device(getattr(cache, "_index", -1)):
        return int(lib().csa2_kv_attn_workspace(ctypes.byref(cache), total, max_new, H))


def kv_attn(cache: csa2_kv_cache, q, cu, max_new: int, scale: float, out, ws, lse=None, window: int = 0, stream=None):
    """out [total][H][head_dim] = attention of the new tokens' queries q over the cache (their own keys appended
    before); lse fp32 [total][H] (optional); window > 0: each token sees its last `window` keys only."""
    rc = (_bind or _calls()).kv_attn(cache, q, cu, max_new, scale, out, ws, lse, window, stream)
    if rc:
        raise Csa2Error(rc, "csa2_kv_attn")
