"""Thin ctypes binding of libmasw (include/masw.h), same names as the C calls.

Argument marshalling only: torch tensors contribute device pointers, the
current CUDA stream is passed as the stream, and a non-zero status becomes a
MaswError carrying masw_last_error().  Every step of the computation runs in
the library's CUDA kernels; there is no fallback if the library is missing.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmasw.so")

MASW_OK, MASW_EINVAL, MASW_ENOMEM, MASW_ECAPACITY, MASW_ESTATE, MASW_ECUDA, MASW_ETIMEOUT = 0, -1, -2, -3, -4, -5, -6
MASW_EGUARD = -7
MASW_F32, MASW_BF16, MASW_E4M3 = 0, 1, 2
MASW_MAX_BATCH, MASW_MAX_GROUP = 512, 8

# every symbol include/masw.h declares
EXPORTS = [
    "masw_mem_create", "masw_mem_destroy", "masw_last_error", "masw_append_kv",
    "masw_materialize_slot", "masw_rollback", "masw_draft_attn", "masw_full_attn",
    "masw_draft_step", "masw_full_step", "masw_draft_step_slot",
    "masw_verify_attn", "masw_verify_workspace_bytes", "masw_verify_attn_noalloc", "masw_mem_load", "masw_mem_export",
    "masw_query", "masw_sync", "masw_index", "masw_version", "masw_check_guards",
    "masw_greedy_accept", "masw_greedy_workspace_bytes", "masw_eq1_speedup", "masw_prefill",
    "masw_selftest_timeout", "masw_paged_append", "masw_paged_attn", "masw_paged_workspace_bytes",
]


class MaswError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libmasw status {code}: {msg}")
        self.code = code


class masw_opts_t(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("dtype", ctypes.c_int), ("max_seq_len", ctypes.c_int),
                ("softmax_scale", ctypes.c_float), ("slot_self_attend", ctypes.c_int),
                ("full_kv", ctypes.c_int), ("rollback_reserve", ctypes.c_int)]


class masw_state_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("t", "n_sink", "n_local", "m", "dev_t", "dev_m",
                                            "ring_rows", "rows", "slot_capacity")]


class masw_paged_t(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("page_stride", ctypes.c_longlong)] + \
               [(n, ctypes.c_int) for n in ("dtype", "n_pages", "page_size", "n_kv_heads", "head_dim", "batch",
                                            "table_stride")]


class masw_rope_t(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p)] + [(n, ctypes.c_int) for n in ("n_pos", "rot_dim", "interleaved")]


_lib = None


def load() -> ctypes.CDLL:
    """Load the in-tree libmasw.so; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmasw.so not built at {LIB_PATH}; run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L = ctypes.c_longlong
    IP = ctypes.POINTER(ctypes.c_int)
    sig = {
        "masw_mem_create": [I, I, I, I, I, I, ctypes.POINTER(masw_opts_t), ctypes.POINTER(P)],
        "masw_mem_destroy": [P],
        "masw_check_guards": [P],
        "masw_append_kv": [P, I, P, P, P, P],
        "masw_materialize_slot": [P, I, IP, I, P, P, P, P, P, I, P],
        "masw_rollback": [P, IP, IP, I, P],
        "masw_draft_attn": [P, I, P, I, P, P, P],
        "masw_full_attn": [P, I, P, I, P, P, P],
        "masw_draft_step": [P, I, P, P, P, P, I, P, P, P],
        "masw_full_step": [P, I, P, P, P, P, I, P, P, P],
        "masw_draft_step_slot": [P, I, P, P, P, P, I, P, P, IP, I, P, P, P, P, P, P],
        "masw_prefill": [P, I, I, I, P, P, P, P, P, P, I, P, P, P, P, P],
        "masw_selftest_timeout": [P, I, P],
        "masw_verify_attn": [P, P, P, P, I, I, I, I, I, I, I, F, P, P, P, Z, P],
        "masw_verify_workspace_bytes": [I, I, I, I, I, I, ctypes.POINTER(Z)],
        "masw_verify_attn_noalloc": [P, P, P, P, I, I, I, I, I, I, I, F, P, P, P, P],
        "masw_mem_load": [P, I, I, I, P, P, P, P, I],
        "masw_mem_export": [P, I, I, P, P, IP],
        "masw_query": [P, I, I, ctypes.POINTER(masw_state_t)],
        "masw_sync": [P, P],
        "masw_index": [I, I, I, I, I, I],
        "masw_greedy_accept": [P, P, I, I, I, I, P, P, P, Z, P],
        "masw_greedy_workspace_bytes": [I, I, I, ctypes.POINTER(Z)],
        "masw_paged_append": [P, P, P, I, P, P, L, L, P, P, P, P, I, L, P, P],
        "masw_paged_attn": [P, P, P, I, I, P, I, L, I, F, P, I, P, P, P, Z, P],
        "masw_paged_workspace_bytes": [P, I, I, I, ctypes.POINTER(Z)],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = I
    lib.masw_last_error.argtypes = [P]
    lib.masw_last_error.restype = ctypes.c_char_p
    lib.masw_eq1_speedup.argtypes = [ctypes.c_double, I, ctypes.c_double, ctypes.c_double]
    lib.masw_eq1_speedup.restype = ctypes.c_double
    lib.masw_version.argtypes = []
    lib.masw_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(rc: int, handle=None):
    if rc != MASW_OK:
        msg = load().masw_last_error(handle)
        raise MaswError(rc, msg.decode() if msg else "")


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def _int_array(xs):
    xs = [int(x) for x in xs]
    return (ctypes.c_int * len(xs))(*xs), len(xs)


# ---------------------------------------------------------------- lifetime --

def masw_mem_create(S, W, r, n_kv_heads, head_dim, layers, batch=1, dtype=MASW_BF16, max_seq_len=32768,
                    softmax_scale=0.0, slot_self_attend=False, full_kv=False, rollback_reserve=0):
    lib = load()
    opts = masw_opts_t(batch, dtype, max_seq_len, softmax_scale, int(slot_self_attend), int(full_kv),
                       rollback_reserve)
    h = ctypes.c_void_p()
    _check(lib.masw_mem_create(S, W, r, n_kv_heads, head_dim, layers, ctypes.byref(opts), ctypes.byref(h)))
    return h.value


def masw_mem_destroy(handle):
    _check(load().masw_mem_destroy(handle))


def masw_check_guards(handle):
    """Raise MaswError(MASW_EGUARD) if a guard band around one of the handle's
    device buffers was overwritten (synchronises the device)."""
    _check(load().masw_check_guards(handle), handle)


def masw_last_error(handle=None) -> str:
    msg = load().masw_last_error(handle)
    return msg.decode() if msg else ""


# ------------------------------------------------------------- maintenance --

def masw_append_kv(handle, layer, k, v, active=None, stream=None):
    act = None
    if active is not None:
        act = (ctypes.c_uint8 * len(active))(*[1 if a else 0 for a in active])
    _check(load().masw_append_kv(handle, layer, _ptr(k), _ptr(v),
                                 ctypes.cast(act, ctypes.c_void_p) if act is not None else None,
                                 _stream(stream)), handle)


def masw_materialize_slot(handle, layer, seq_ids, q_g, k_g, v_g, o_g, lse_g=None, stream=None):
    ids, n = _int_array(seq_ids)
    _check(load().masw_materialize_slot(handle, layer, ids, n, _ptr(q_g), _ptr(k_g), _ptr(v_g), _ptr(o_g),
                                        _ptr(lse_g), q_g.shape[1], _stream(stream)), handle)


def masw_rollback(handle, seq_ids, t_new, stream=None):
    ids, n = _int_array(seq_ids)
    tn, n2 = _int_array(t_new)
    if n != n2:
        raise ValueError("seq_ids and t_new differ in length")
    _check(load().masw_rollback(handle, ids, tn, n, _stream(stream)), handle)


# --------------------------------------------------------------- attention --

def masw_draft_attn(handle, layer, q, o, lse=None, stream=None):
    _check(load().masw_draft_attn(handle, layer, _ptr(q), q.shape[1], _ptr(o), _ptr(lse), _stream(stream)), handle)


def masw_full_attn(handle, layer, q, o, lse=None, stream=None):
    _check(load().masw_full_attn(handle, layer, _ptr(q), q.shape[1], _ptr(o), _ptr(lse), _stream(stream)), handle)


def _active(active):
    if active is None:
        return None, None
    arr = (ctypes.c_uint8 * len(active))(*[1 if a else 0 for a in active])
    return arr, ctypes.cast(arr, ctypes.c_void_p)


def masw_draft_step(handle, layer, q, k, v, o, lse=None, active=None, stream=None):
    keep, act = _active(active)
    _check(load().masw_draft_step(handle, layer, _ptr(q), _ptr(k), _ptr(v), act, q.shape[1], _ptr(o), _ptr(lse),
                                  _stream(stream)), handle)


def masw_full_step(handle, layer, q, k, v, o, lse=None, active=None, stream=None):
    keep, act = _active(active)
    _check(load().masw_full_step(handle, layer, _ptr(q), _ptr(k), _ptr(v), act, q.shape[1], _ptr(o), _ptr(lse),
                                 _stream(stream)), handle)


def masw_draft_step_slot(handle, layer, q, k, v, o, seq_ids, q_g, k_g, v_g, o_g, lse=None, lse_g=None,
                         active=None, stream=None):
    keep, act = _active(active)
    ids, n = _int_array(seq_ids)
    _check(load().masw_draft_step_slot(handle, layer, _ptr(q), _ptr(k), _ptr(v), act, q.shape[1], _ptr(o), _ptr(lse),
                                       ids, n, _ptr(q_g), _ptr(k_g), _ptr(v_g), _ptr(o_g), _ptr(lse_g),
                                       _stream(stream)), handle)


def masw_verify_workspace_bytes(B, Lq, Hq, Hkv, D, Tmax) -> int:
    out = ctypes.c_size_t()
    _check(load().masw_verify_workspace_bytes(B, Lq, Hq, Hkv, D, Tmax, ctypes.byref(out)))
    return out.value


def masw_verify_attn(q, k_cache, v_cache, kv_len, o, lse=None, workspace=None, scale=0.0, stream=None):
    """q [B, Lq, Hq, D] bf16, caches [B, Hkv, Tmax, D] bf16, kv_len [B] int32 -> o [B, Lq, Hq, D] fp32.
    A caller's workspace (uint8, at least masw_verify_workspace_bytes) must be zero-filled before its first
    use; every completed call leaves it zero-filled.  Without one, a zero-filled workspace is allocated."""
    B, Lq, Hq, D = q.shape
    Hkv, Tmax = k_cache.shape[1], k_cache.shape[2]
    need = masw_verify_workspace_bytes(B, Lq, Hq, Hkv, D, Tmax)
    if workspace is None:
        import torch
        workspace = torch.zeros(need, dtype=torch.uint8, device=q.device)   # zero-filled before first use
    _check(load().masw_verify_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_len), B, Lq, Hq, Hkv, D, Tmax,
                                   MASW_BF16, scale, _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(),
                                   _stream(stream)))


def masw_verify_attn_noalloc(q, k_cache, v_cache, kv_len, o, lse=None, scale=0.0, status=None, stream=None):
    """masw_verify_attn for callers that cannot allocate: no workspace, the
    library's own fixed device array holds the split partials.  status: an
    optional device int32 tensor that receives the call's status word."""
    B, Lq, Hq, D = q.shape
    Hkv, Tmax = k_cache.shape[1], k_cache.shape[2]
    _check(load().masw_verify_attn_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(kv_len), B, Lq, Hq, Hkv, D,
                                           Tmax, MASW_BF16, scale, _ptr(o), _ptr(lse), _ptr(status),
                                           _stream(stream)))


def masw_greedy_accept(logits, draft, tokens, n_emit, workspace=None, stream=None):
    """logits [B, L+1, V] (bf16 or fp32), draft [B, L] int32 -> tokens [B, L+1], n_emit [B] (int32)."""
    import torch
    B, L1, V = logits.shape
    L = L1 - 1
    need = ctypes.c_size_t()
    _check(load().masw_greedy_workspace_bytes(B, L, V, ctypes.byref(need)))
    if workspace is None:   # zero-filled once; every call leaves it zero-filled
        workspace = torch.zeros(need.value, dtype=torch.uint8, device=logits.device)
    dt = MASW_BF16 if logits.dtype == torch.bfloat16 else MASW_F32
    _check(load().masw_greedy_accept(_ptr(logits), _ptr(draft), B, L, V, dt, _ptr(tokens), _ptr(n_emit),
                                     _ptr(workspace), workspace.numel(), _stream(stream)))


def masw_greedy_workspace_bytes(B, L, V) -> int:
    out = ctypes.c_size_t()
    _check(load().masw_greedy_workspace_bytes(B, L, V, ctypes.byref(out)))
    return out.value


def masw_eq1_speedup(l_acc, l_draft, t_draft, t_target) -> float:
    return load().masw_eq1_speedup(l_acc, l_draft, t_draft, t_target)


# ------------------------------------------------------------ paged caches --

def masw_paged_cache(k, v, page_table, k_scale=None, v_scale=None) -> masw_paged_t:
    """Describe a paged cache to the calls below: k, v [n_pages, Hkv, page_size, D] (bf16, or float8_e4m3fn / uint8
    bytes of e4m3 with fp32 scales [n_pages, Hkv]), page_table [batch, stride] int32.  Pages may lie apart (a view of
    a larger array), their inside is dense.  The description holds the tensors; make it once per cache."""
    import torch
    e4 = k.dtype in (torch.float8_e4m3fn, torch.uint8)
    if not e4 and k.dtype != torch.bfloat16:
        raise ValueError("pages must be bfloat16 or float8_e4m3fn")
    n, h, p, d = k.shape
    if v.shape != k.shape or v.dtype != k.dtype or (n > 1 and v.stride(0) != k.stride(0)):
        raise ValueError("k and v pages must have the same shape, type and page stride")
    for x in (k, v):
        if tuple(x.stride()[1:]) != (p * d, d, 1):
            raise ValueError("a page must be dense")
        if n > 1 and x.stride(0) < h * p * d:
            raise ValueError("pages must not overlap")
    if e4:
        for x in (k_scale, v_scale):
            if x is None or x.dtype != torch.float32 or tuple(x.shape) != (n, h) or not x.is_contiguous():
                raise ValueError("e4m3 pages need contiguous fp32 scales [n_pages, Hkv] for k and v")
    elif k_scale is not None or v_scale is not None:
        raise ValueError("bf16 pages have no scales")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.stride(1) != 1:
        raise ValueError("page_table must be int32 [batch, stride] with dense rows")
    tensors = [x for x in (k, v, page_table, k_scale, v_scale) if x is not None]
    if len({x.device for x in tensors}) != 1:
        raise ValueError("the cache's tensors must lie on one device")
    B = page_table.shape[0]
    c = masw_paged_t(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(page_table), k.stride(0) if n > 1 else 0,
                     MASW_E4M3 if e4 else MASW_BF16, n, p, h, d, B,
                     page_table.stride(0) if B > 1 else page_table.shape[1])
    c.tensors = tensors
    # what the calls below need on every step, looked up once
    c.address = ctypes.addressof(c)
    c.device, c.bf16, c.int32, c.f32 = k.device, torch.bfloat16, torch.int32, torch.float32
    c.cuda_index = k.device.index if k.device.type == "cuda" else None
    return c


def masw_rope(cos_sin, interleaved=False) -> masw_rope_t:
    """Rotary table for masw_paged_append: cos_sin [n_pos, rot_dim] fp32, each row the cosines, then the sines."""
    import torch
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise ValueError("cos_sin must be contiguous fp32 [n_pos, rot_dim]")
    r = masw_rope_t(_ptr(cos_sin), cos_sin.shape[0], cos_sin.shape[1], int(interleaved))
    r.tensors = [cos_sin]
    r.address, r.device = ctypes.addressof(r), cos_sin.device
    return r


def _token_rows(name, x, heads, dim, cache):
    """Token stride of x [rows, heads, dim] (bf16 on the cache's device; heads and elements dense)."""
    shape, st = x.shape, x.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim or x.dtype is not cache.bf16 or x.device != cache.device:
        raise ValueError(f"{name} must be bfloat16 [rows, {heads}, {dim}] on the cache's device")
    if st[2] != 1 or (st[1] != dim and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be dense")
    if shape[0] < 2:
        return 0
    if st[0] < heads * dim:
        raise ValueError(f"{name}: tokens must not overlap")
    return st[0]


def _ints(name, x, n, cache):
    if x is None:
        return None
    if x.dtype is not cache.int32 or x.numel() < n or x.device != cache.device or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 with at least {n} elements on the cache's device")
    return x.data_ptr()


def _cache_stream(stream, cache):
    """The stream to launch on, as a handle; the cache's device has to be the current one."""
    if cache.cuda_index is None:
        return stream or 0
    import torch
    if torch.cuda.current_device() != cache.cuda_index:
        raise ValueError("the cache lies on another device than the current one")
    return torch._C._cuda_getCurrentRawStream(cache.cuda_index) if stream is None else stream


def masw_paged_append(cache, kv_len, k, v, rope=None, pos=None, q=None, q_out=None, row_start=None, status=None,
                      stream=None):
    """Append the K/V rows [rows, Hkv, D] of new tokens to a paged cache, K (and q -> q_out [rows, Hq, D]) rotated by
    `rope` on the way.  kv_len [batch] counts them already; row_start [batch + 1] says whose rows are whose (None:
    rows / batch each).  k, v and q may be slices of a fused projection.  status: optional int32 word."""
    rows, B, H, D = k.shape[0], cache.batch, cache.n_kv_heads, cache.head_dim
    ks, vs = _token_rows("k", k, H, D, cache), _token_rows("v", v, H, D, cache)
    hq = qs = 0
    q_ptr = q_out_ptr = None
    if q is not None:
        hq = q.shape[1]
        qs = _token_rows("q", q, hq, D, cache)
        if q_out is None or q_out.dtype is not cache.bf16 or q_out.shape != q.shape or not q_out.is_contiguous() or q_out.device != cache.device:
            raise ValueError("q_out must be contiguous bfloat16 of q's shape on the cache's device")
        q_ptr, q_out_ptr = q.data_ptr(), q_out.data_ptr()
    if v.shape[0] != rows or (q is not None and q.shape[0] != rows):
        raise ValueError("k, v and q differ in rows")
    if rope is not None and rope.device != cache.device:
        raise ValueError("the rotary table lies on another device than the cache")
    _check(load().masw_paged_append(cache.address, _ints("kv_len", kv_len, B, cache), _ints("row_start", row_start, B + 1, cache),
                                    rows, k.data_ptr(), v.data_ptr(), ks, vs, None if rope is None else rope.address,
                                    _ints("pos", pos, rows, cache), q_ptr, q_out_ptr, hq, qs,
                                    _ints("status", status, 1, cache), _cache_stream(stream, cache)))


def masw_paged_workspace_bytes(cache, rows, max_rows, n_q_heads) -> int:
    out = ctypes.c_size_t()
    _check(load().masw_paged_workspace_bytes(cache.address, rows, max_rows, n_q_heads, ctypes.byref(out)))
    return out.value


def masw_paged_attn(cache, kv_len, q, o, lse=None, row_start=None, max_rows=None, window=0, scale=0.0, status=None,
                    workspace=None, stream=None):
    """Causal attention of q [rows, Hq, D] bf16 over a paged cache -> o [rows, Hq, D] (bf16 or fp32), lse [rows, Hq]
    fp32.  With row_start, max_rows bounds the rows of one sequence (None: all of them).  Without a workspace (uint8,
    masw_paged_workspace_bytes), one is allocated."""
    rows, hq, _ = q.shape
    B = cache.batch
    qs = _token_rows("q", q, hq, cache.head_dim, cache)
    if o.shape != q.shape or not o.is_contiguous() or o.device != cache.device or (o.dtype is not cache.bf16 and o.dtype is not cache.f32):
        raise ValueError("o must be contiguous bfloat16 or float32 of q's shape on the cache's device")
    lse_ptr = None
    if lse is not None:
        if lse.shape != (rows, hq) or lse.dtype is not cache.f32 or not lse.is_contiguous() or lse.device != cache.device:
            raise ValueError("lse must be contiguous float32 [rows, Hq]")
        lse_ptr = lse.data_ptr()
    mr = rows // B if row_start is None else (rows if max_rows is None else max_rows)
    if workspace is None:
        import torch
        if stream is not None and cache.cuda_index is not None and stream != torch._C._cuda_getCurrentRawStream(cache.cuda_index):
            raise ValueError("on a stream other than the current one the call needs a workspace")   # it would be reused too early
        workspace = torch.empty(masw_paged_workspace_bytes(cache, rows, mr, hq), dtype=torch.uint8, device=cache.device)
    elif workspace.device != cache.device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the cache's device")
    _check(load().masw_paged_attn(cache.address, _ints("kv_len", kv_len, B, cache), _ints("row_start", row_start, B + 1, cache),
                                  rows, mr, q.data_ptr(), hq, qs, window, scale, o.data_ptr(),
                                  MASW_BF16 if o.dtype is cache.bf16 else MASW_F32, lse_ptr,
                                  _ints("status", status, 1, cache), workspace.data_ptr(), workspace.nbytes,
                                  _cache_stream(stream, cache)))


# ---------------------------------------------------------------- plumbing --

def masw_prefill(handle, layer, seq, q_raw, k_raw, v_raw, q_slot, k_slot, v_slot, o_raw, lse_raw=None,
                 o_slot=None, lse_slot=None, stream=None):
    """Prefill one (layer, seq): q_raw [T, Hq, D], k_raw/v_raw [T, Hkv, D], the slot
    tokens' q/k/v [M, ...] (None when M = 0), outputs fp32 o [.., Hq, D], lse [.., Hq]."""
    T, Hq = q_raw.shape[0], q_raw.shape[1]
    _check(load().masw_prefill(handle, layer, seq, T, _ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(q_slot),
                               _ptr(k_slot), _ptr(v_slot), Hq, _ptr(o_raw), _ptr(lse_raw), _ptr(o_slot),
                               _ptr(lse_slot), _stream(stream)), handle)


def masw_selftest_timeout(handle, polls=1000, stream=None):
    """Launch the failure-detection self-test (a bounded wait that runs out);
    the next masw_sync raises MaswError with MASW_ETIMEOUT."""
    _check(load().masw_selftest_timeout(handle, polls, _stream(stream)), handle)


def masw_mem_load(handle, layer, seq, k_raw, v_raw, k_slots=None, v_slots=None):
    """k_raw, v_raw: [t, Hkv, D] torch tensors (CPU or CUDA), contiguous."""
    t = k_raw.shape[0]
    n = 0 if k_slots is None else k_slots.shape[0]
    for x in (k_raw, v_raw, k_slots, v_slots):
        if x is not None and not x.is_contiguous():
            raise ValueError("load inputs must be contiguous")
    _check(load().masw_mem_load(handle, layer, seq, t, _ptr(k_raw), _ptr(v_raw), _ptr(k_slots), _ptr(v_slots), n),
           handle)


def masw_mem_export(handle, layer, seq, k_out, v_out, slot_capacity=0):
    pos = (ctypes.c_int * max(1, slot_capacity))()
    _check(load().masw_mem_export(handle, layer, seq, _ptr(k_out), _ptr(v_out), pos), handle)
    return list(pos)[:slot_capacity]


def masw_query(handle, layer, seq) -> dict:
    st = masw_state_t()
    _check(load().masw_query(handle, layer, seq, ctypes.byref(st)), handle)
    return {name: getattr(st, name) for name, _ in masw_state_t._fields_}


def masw_sync(handle, stream=None):
    _check(load().masw_sync(handle, _stream(stream)), handle)


def masw_index(which, t, S, W, r, R=0) -> int:
    return load().masw_index(which, t, S, W, r, R)


def masw_version() -> str:
    return load().masw_version().decode()
