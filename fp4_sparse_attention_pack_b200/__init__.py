"""Python binding of the CSA2 C ABI (``include/csa2.h``, ``libcsa2.so``).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Tensors are torch CUDA tensors (torch supplies device memory and
streams); calls are enqueued on torch's current stream.  Importing this
package raises if the library has not been built -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

from ._build import LIB

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
# A decode step makes these calls with a few microseconds of device work each, so
# their checks compare attributes only and the device guard is taken when needed.

class _Names:
    """torch's objects that every call compares with, looked up once."""

    def __init__(self):
        import torch
        self.int32, self.float32 = torch.int32, torch.float32
        self.heads = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}
        self.pools = {torch.bfloat16: KV_BF16, torch.float16: KV_F16, torch.float8_e4m3fn: KV_E4M3}
        self.device = torch.cuda.device
        self.current_device = torch.cuda.current_device
        # the current stream's handle without a Stream object
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.stream = raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)


_n = None


def _names():
    global _n
    if _n is None:
        _n = _Names()
    return _n


def _want(t, what, dtype, shape, index=None):
    """A contiguous CUDA tensor of this dtype and shape (the library sees only its address); its device index."""
    at = t.get_device()
    if at < 0 or (index is not None and at != index):
        raise ValueError(f"{what} is on {t.device}, not on the call's CUDA device")
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"not {t.dtype} {tuple(t.shape)}")
    return at


def _heads(t, what, shape, dtype, index):
    """csa2_heads of a [tokens][heads][channels] tensor with contiguous channels."""
    if t.get_device() != index or index < 0 or t.dtype is not dtype:
        raise ValueError(f"{what} is {t.dtype} on {t.device}: it must be {dtype}, on the call's CUDA device")
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    ts, hs, cs = t.stride()
    if cs != 1 and shape[2] > 1:
        raise ValueError(f"{what}: the channels must be contiguous")
    return csa2_heads(t.data_ptr(), ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0)


def _code(codes, t, what):
    code = codes.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: {t.dtype} is not supported")
    return code


def _on_cache(cache, index, what):
    at = getattr(cache, "_index", index)
    if at != index:
        raise ValueError(f"{what} is on CUDA device {index}, the cache on {at}")


def _call(f, index, stream, args, what):
    """f(*args, stream) with tensor device `index` current."""
    n = _names()
    if n.current_device() == index:
        rc = f(*args, n.stream(index) if stream is None else stream.cuda_stream)
    else:
        with n.device(index):
            rc = f(*args, n.stream(index) if stream is None else stream.cuda_stream)
    if rc != 0:
        raise Csa2Error(rc, what)


def rotary(inv_freq, rot_dim: int, offset: int = 0, neighbours: bool = False, n_axes: int = 1, axis=None) -> csa2_rotary:
    """A rotation: channels offset .. offset + rot_dim - 1 of a head turn in pairs (neighbours, or half the
    rotation apart) by position * inv_freq[pair] (fp32 CUDA tensor).  axis (a list, one entry per pair) says
    which of the n_axes positions turns it."""
    index = _want(inv_freq, "inv_freq", _names().float32, (rot_dim // 2,))
    r = csa2_rotary(inv_freq.data_ptr(), None, rot_dim, offset, int(neighbours), n_axes)
    if axis is not None:
        if len(axis) != rot_dim // 2:
            raise ValueError(f"axis has {len(axis)} entries, not one for each of the {rot_dim // 2} pairs")
        r.axis = (ctypes.c_uint8 * len(axis))(*axis)
    r._keep, r._index = inv_freq, index  # the descriptor holds its address
    return r


def rotate(rot: csa2_rotary, x, pos, out, inverse: bool = False, stream=None):
    """out = x [tokens][heads][channels] rotated at pos int32 [n_axes][tokens] (out may be x); inverse turns back."""
    n, index, shape = _names(), x.get_device(), x.shape
    if len(shape) != 3:
        raise ValueError(f"x must be [tokens][heads][channels], not {tuple(shape)}")
    xd = _heads(x, "x", shape, x.dtype, index)
    yd = _heads(out, "out", shape, x.dtype, index)
    _want(pos, "pos", n.int32, (rot.n_axes, shape[0]), index)
    _on_cache(rot, index, "x")
    _call(lib().csa2_rotate, index, stream,
          (ctypes.byref(rot), ctypes.byref(xd), ctypes.byref(yd), _code(n.heads, x, "x"), shape[0], shape[1], shape[2],
           pos.data_ptr(), int(inverse)), "csa2_rotate")


def kv_cache(k_pages, v_pages, page_table, n_tokens, status) -> csa2_kv_cache:
    """Descriptor of a paged key/value cache: pools [pages][kv_heads][64][head_dim] (bf16, fp16 or float8_e4m3fn),
    page_table int32 [batch][max_pages], n_tokens int32 [batch], status int32 (one word or more)."""
    n = _names()
    pages, heads, rows, dim = k_pages.shape
    if rows != 64:
        raise ValueError(f"a page has 64 rows, not {rows}")
    index = _want(k_pages, "k_pages", k_pages.dtype, k_pages.shape)
    _want(v_pages, "v_pages", k_pages.dtype, k_pages.shape, index)
    batch, max_pages = page_table.shape
    _want(page_table, "page_table", n.int32, (batch, max_pages), index)
    _want(n_tokens, "n_tokens", n.int32, (batch,), index)
    if status.get_device() != index or status.element_size() != 4 or status.numel() < 1:
        raise ValueError("status must be a tensor of 32-bit words on the cache's device")
    c = csa2_kv_cache(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(), n_tokens.data_ptr(),
                      status.data_ptr(), batch, max_pages, pages, heads, dim, _code(n.pools, k_pages, "k_pages"))
    c._keep, c._index = (k_pages, v_pages, page_table, n_tokens, status), index  # the descriptor holds their addresses
    return c


def kv_append(cache: csa2_kv_cache, k, v, cu, max_new: int, start=None, rotary=None, pos=None, stream=None):
    """Write the new tokens k, v [total][kv_heads][head_dim] (sequence b: rows cu[b] .. cu[b + 1] - 1) behind
    start (int32 [batch]; None: behind the tokens held), the keys rotated at pos int32 [n_axes][total]
    (None: their slots)."""
    n, index, total, batch = _names(), k.get_device(), k.shape[0], cache.batch
    shape = (total, cache.kv_heads, cache.head_dim)
    kd, vd = _heads(k, "k", shape, k.dtype, index), _heads(v, "v", shape, k.dtype, index)
    _on_cache(cache, index, "k")
    _want(cu, "cu", n.int32, (batch + 1,), index)
    if start is not None:
        _want(start, "start", n.int32, (batch,), index)
    if rotary is not None:
        _on_cache(rotary, index, "k")
    if pos is not None:
        _want(pos, "pos", n.int32, (rotary.n_axes if rotary is not None else 0, total), index)
    _call(lib().csa2_kv_append, index, stream,
          (ctypes.byref(cache), ctypes.byref(kd), ctypes.byref(vd), _code(n.heads, k, "k"), cu.data_ptr(), total, max_new,
           _ptr(start), ctypes.byref(rotary) if rotary is not None else None, _ptr(pos)), "csa2_kv_append")


def kv_attn_workspace(cache: csa2_kv_cache, total: int, max_new: int, H: int) -> int:
    return int(lib().csa2_kv_attn_workspace(ctypes.byref(cache), total, max_new, H))


def kv_attn(cache: csa2_kv_cache, q, cu, max_new: int, scale: float, out, ws, lse=None, window: int = 0, stream=None):
    """out [total][H][head_dim] = attention of the new tokens' queries q over the cache (their own keys appended
    before); lse fp32 [total][H] (optional); window > 0: each token sees its last `window` keys only."""
    n, index = _names(), q.get_device()
    shape = (q.shape[0], q.shape[1], cache.head_dim)
    qd, od = _heads(q, "q", shape, q.dtype, index), _heads(out, "out", shape, q.dtype, index)
    _on_cache(cache, index, "q")
    _want(cu, "cu", n.int32, (cache.batch + 1,), index)
    if lse is not None:
        _want(lse, "lse", n.float32, shape[:2], index)
    if ws is not None and ws.get_device() != index:
        raise ValueError(f"ws is on {ws.device}, not on the call's CUDA device")
    _call(lib().csa2_kv_attn, index, stream,
          (ctypes.byref(cache), ctypes.byref(qd), shape[1], _code(n.heads, q, "q"), cu.data_ptr(), shape[0], max_new, scale,
           window, ctypes.byref(od), _ptr(lse), _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0),
          "csa2_kv_attn")
