"""Block-quantized-weight matmul on GB300 (sm_103a): Python binding.

A thin ctypes layer over libcq.so: each function takes torch tensors (or
numpy arrays for host-side helpers), checks nothing itself, and passes
pointers and sizes to the C entry point of the same name.  Every step of
the computation runs in the library's CUDA kernels; there is no fallback,
and the functions raise if the library is missing.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcq.so")
INCLUDE = os.path.join(os.path.dirname(_HERE), "include", "cq.h")

CQ_F16, CQ_BF16, CQ_F32 = 0, 1, 2
CQ_OPT_SMALL_T_MAX, CQ_OPT_FORCE_PATH, CQ_OPT_WAIT_NS, CQ_OPT_TEST_STALL, CQ_OPT_TRACE, CQ_OPT_TC_BN, CQ_OPT_TC_KSPLIT, \
    CQ_OPT_TC_AMODE, CQ_OPT_TC_PAIR, CQ_OPT_STREAM_KERNEL = 0, 1, 2, 3, 4, 5, 6, 7, 8, 9
CQ_ROPE_HALF, CQ_ROPE_PAIRS = 0, 1
CQ_ROPE_PLAIN, CQ_ROPE_LINEAR, CQ_ROPE_BASE, CQ_ROPE_RAMP, CQ_ROPE_BANDS = 0, 1, 2, 3, 4
STATUS = {0: "CQ_OK", 1: "CQ_ERR_NULL", 2: "CQ_ERR_DTYPE", 3: "CQ_ERR_SHAPE", 4: "CQ_ERR_ALIGN",
          5: "CQ_ERR_INDEX", 6: "CQ_ERR_WORKSPACE", 7: "CQ_ERR_CUDA", 8: "CQ_ERR_TIMEOUT", 9: "CQ_ERR_ARCH",
          10: "CQ_ERR_ARG"}

_lib = None

_c_p, _c_i64, _c_int, _c_sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_SIGS = {
    "cq_gemm_q4_workspace_bytes": (_c_sz, [_c_i64, _c_i64]),
    "cq_gemm_q4": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_int, _c_p, _c_sz, _c_p]),
    "cq_gemm_q4_noalloc": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_int, _c_p]),
    "cq_gemm_q8row": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_int, _c_p]),
    "cq_moe_workspace_bytes": (_c_sz, [_c_i64] * 5),
    "cq_ffn_q4_workspace_bytes": (_c_sz, [_c_i64] * 3),
    "cq_gemm_q8b_workspace_bytes": (_c_sz, [_c_i64, _c_i64]),
    "cq_gemm_q8b": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_int, _c_p, _c_sz, _c_p]),
    "cq_gemm_q4a_workspace_bytes": (_c_sz, [_c_i64] * 4),
    "cq_gemm_q4a": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_p, _c_int, _c_p, _c_sz,
                             _c_p]),
    "cq_gemm_q8_2f_workspace_bytes": (_c_sz, [_c_i64, _c_i64]),
    "cq_gemm_q8_2f": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_p, _c_int, _c_p, _c_sz, _c_p]),
    "cq_gemm_q4_batched_workspace_bytes": (_c_sz, [_c_i64, _c_i64, _c_int]),
    "cq_gemm_q4_batched": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_int, _c_i64, _c_p, _c_int, _c_i64,
                                    _c_p, _c_sz, _c_p]),
    "cq_ffn_q4": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_sz,
                           _c_p]),
    "cq_moe_panels": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p,
                               _c_p, _c_p, _c_p, _c_int, _c_p, _c_sz, _c_p]),
    "cq_moe_route": (_c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_int, _c_p, _c_p, _c_p]),
    "cq_moe_layout": (_c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p]),
    "cq_kv8_write": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p]),
    "cq_kv8_read": (_c_int, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p]),
    "cq_attn_kv8_workspace_bytes": (_c_sz, [_c_i64] * 6),
    "cq_attn_kv8": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_i64, ctypes.c_float, _c_int,
                             _c_i64, _c_p, _c_int, _c_i64, _c_p, _c_p, _c_sz, _c_p]),
    "cq_rope": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_int, _c_i64, _c_p]),
    "cq_rope_freqs": (_c_int, [_c_i64, ctypes.c_double, _c_int] + [ctypes.c_double] * 4 + [_c_p, _c_p]),
    "cq_kv8_write_rope": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "cq_attn_kv8_tree": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_i64, ctypes.c_float, _c_p,
                                  _c_i64, _c_p, _c_int, _c_i64, _c_p, _c_p, _c_sz, _c_p]),
    "cq_verify": (_c_int, [_c_p, _c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_i64, _c_p, _c_p, _c_i64, _c_p, _c_i64, _c_i64,
                           _c_p, _c_p, _c_p, _c_p, _c_i64, _c_p, _c_p]),
    "cq_dequant_q4": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p]),
    "cq_dequant_q8row": (_c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p]),
    "cq_get_device_error": (_c_int, [_c_p]),
    "cq_last_error": (ctypes.c_char_p, []),
    "cq_last_launches": (_c_int, []),
    "cq_set_option": (_c_int, [_c_int, _c_i64]),
    "cq_get_option": (_c_i64, [_c_int]),
    "cq_version": (_c_int, []),
}


class CQError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


def lib():
    """The loaded libcq.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libcq.so is not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(st: int):
    if st != 0:
        raise CQError(st, lib().cq_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _xt(t):
    import torch
    if t.dtype == torch.float16:
        return CQ_F16
    if t.dtype == torch.bfloat16:
        return CQ_BF16
    if t.dtype == torch.float32:
        return CQ_F32
    return -1


# ---- entry points (same names as the C ABI) -----------------------------

def cq_gemm_q4_workspace_bytes(T: int, K: int) -> int:
    return lib().cq_gemm_q4_workspace_bytes(T, K)


def cq_gemm_q4(X, Wq, Ws, Y, ws, stream=None, raise_on_error=True):
    """Y[T][N] = X[T][K] . dequant(Wq, Ws)^T.  X fp16/bf16, Wq uint8 [N][K/2],
    Ws int16/uint16-bits fp16 [N][K/32], Y f32/bf16 [T][N], ws uint8."""
    T, K = X.shape
    N = Wq.shape[0]
    st = lib().cq_gemm_q4(_ptr(X), _xt(X), T, K, _ptr(Wq), _ptr(Ws), N, _ptr(Y), _xt(Y), _ptr(ws),
                          0 if ws is None else ws.numel() * ws.element_size(), _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_gemm_q4_noalloc(X, Wq, Ws, Y, stream=None, raise_on_error=True):
    """cq_gemm_q4 without a caller workspace: for callers that cannot
    allocate device memory; the scratch is a fixed array inside the library
    (see include/cq.h for the size limit and the sharing rules)."""
    T, K = X.shape
    N = Wq.shape[0]
    st = lib().cq_gemm_q4_noalloc(_ptr(X), _xt(X), T, K, _ptr(Wq), _ptr(Ws), N, _ptr(Y), _xt(Y), _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_gemm_q8row(X, Wq, rs, Y, stream=None, raise_on_error=True):
    T, K = X.shape
    N = Wq.shape[0]
    st = lib().cq_gemm_q8row(_ptr(X), _xt(X), T, K, _ptr(Wq), _ptr(rs), N, _ptr(Y), _xt(Y), _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_moe_workspace_bytes(T, H, I, E, topk) -> int:
    return lib().cq_moe_workspace_bytes(T, H, I, E, topk)


def cq_moe_panels(X, idx, w, Wgu_q, Wgu_s, Wd_q, Wd_s, Y, ws, stream=None, raise_on_error=True):
    T, H = X.shape
    E, twoI = Wgu_q.shape[0], Wgu_q.shape[1]
    topk = idx.shape[1]
    st = lib().cq_moe_panels(_ptr(X), _xt(X), T, H, E, twoI // 2, topk, _ptr(idx), _ptr(w), _ptr(Wgu_q),
                             _ptr(Wgu_s), _ptr(Wd_q), _ptr(Wd_s), _ptr(Y), _xt(Y), _ptr(ws),
                             ws.numel() * ws.element_size(), _stream(stream))
    if raise_on_error:
        _check(st)
    return st


class cq_q4_job(ctypes.Structure):
    """One job of cq_gemm_q4_batched (the C struct of the same name)."""
    _fields_ = [("Wq", ctypes.c_void_p), ("Ws", ctypes.c_void_p), ("x_off", ctypes.c_int64), ("y_off", ctypes.c_int64)]


def cq_gemm_q4_batched_workspace_bytes(T, K, z) -> int:
    return lib().cq_gemm_q4_batched_workspace_bytes(T, K, z)


def cq_gemm_q4_batched(X, K, jobs, N, Y, ws, stream=None, raise_on_error=True):
    """jobs: list of (Wq, Ws, x_off, y_off) with device tensors; X [T][ldx],
    Y [T][ldy] (the pitches are the tensors' row strides)."""
    T = X.shape[0]
    arr = (cq_q4_job * len(jobs))(*[cq_q4_job(Wq.data_ptr(), Ws.data_ptr(), xo, yo) for Wq, Ws, xo, yo in jobs])
    st = lib().cq_gemm_q4_batched(_ptr(X), _xt(X), T, K, X.stride(0), ctypes.cast(arr, ctypes.c_void_p), len(jobs), N,
                                  _ptr(Y), _xt(Y), Y.stride(0), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_gemm_q8b_workspace_bytes(T, K) -> int:
    return lib().cq_gemm_q8b_workspace_bytes(T, K)


def cq_gemm_q8b(X, Wq, Ws, Y, ws, stream=None, raise_on_error=True):
    """Q8 per 32-k block: Wq int8 [N][K], Ws f32 [N][K/32]."""
    T, K = X.shape
    st = lib().cq_gemm_q8b(_ptr(X), _xt(X), T, K, _ptr(Wq), _ptr(Ws), Wq.shape[0], _ptr(Y), _xt(Y), _ptr(ws),
                           ws.numel() * ws.element_size(), _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_gemm_q4a_workspace_bytes(T, K, N, gk) -> int:
    return lib().cq_gemm_q4a_workspace_bytes(T, K, N, gk)


def cq_gemm_q4a(X, Wq, Ws, Wo, gk, Y, ws, stream=None, raise_on_error=True):
    """Affine Q4: the Q4 split plane plus Wo bf16-bit offsets [N][K/32/gk]."""
    T, K = X.shape
    st = lib().cq_gemm_q4a(_ptr(X), _xt(X), T, K, _ptr(Wq), _ptr(Ws), _ptr(Wo), gk, Wq.shape[0], _ptr(Y), _xt(Y),
                           _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_gemm_q8_2f_workspace_bytes(T, K) -> int:
    return lib().cq_gemm_q8_2f_workspace_bytes(T, K)


def cq_gemm_q8_2f(X, Wq, rs, col, Y, ws, stream=None, raise_on_error=True):
    """q8_2f: Wq int8 [N][K], rs f32 [N], col f32 [K]."""
    T, K = X.shape
    st = lib().cq_gemm_q8_2f(_ptr(X), _xt(X), T, K, _ptr(Wq), _ptr(rs), _ptr(col), Wq.shape[0], _ptr(Y), _xt(Y),
                             _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_ffn_q4_workspace_bytes(T, H, I) -> int:
    return lib().cq_ffn_q4_workspace_bytes(T, H, I)


def cq_ffn_q4(X, Wgu_q, Wgu_s, Wd_q, Wd_s, Y, ws, stream=None, raise_on_error=True):
    """Y[T][H] = Wd . (silu(Wg . x) * (Wu . x)) per token; Wgu_q uint8 [2I][H/2]
    (gate rows then up rows), Wd_q uint8 [H][I/2], fp16-bit scales."""
    T, H = X.shape
    I = Wgu_q.shape[0] // 2
    st = lib().cq_ffn_q4(_ptr(X), _xt(X), T, H, I, _ptr(Wgu_q), _ptr(Wgu_s), _ptr(Wd_q), _ptr(Wd_s), _ptr(Y), _xt(Y),
                         _ptr(ws), ws.numel() * ws.element_size(), _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_moe_route(logits, topk, idx, w, shared=False, stream=None):
    """idx [T][topk + shared] int32, w [T][topk + shared] f32 from logits [T][E + shared] f32."""
    T, cols = logits.shape
    E = cols - (1 if shared else 0)
    _check(lib().cq_moe_route(_ptr(logits), T, E, topk, 1 if shared else 0, _ptr(idx), _ptr(w), _stream(stream)))


def cq_moe_layout(ws, T, H, I, E, topk, perm_out, seg_out, stream=None):
    _check(lib().cq_moe_layout(_ptr(ws), T, H, I, E, topk, _ptr(perm_out), _ptr(seg_out), _stream(stream)))


# ---- 8-bit key/value cache (include/cq_kv8.h) ---------------------------

class _kv8_desc(ctypes.Structure):
    _fields_ = [("Kq", _c_p), ("Ks", _c_p), ("Vq", _c_p), ("Vs", _c_p), ("pages", _c_i64), ("Hkv", _c_i64),
                ("page", _c_i64), ("D", _c_i64), ("table", _c_p), ("ldt", _c_i64), ("B", _c_i64)]


def _described(name):
    return property(lambda self: self._held[name], lambda self, t: self._describe(**{**self._held, name: t}))


class cq_kv8_cache:
    """One layer's 8-bit cache: Kq, Vq int8 [pages][Hkv][page][D], Ks, Vs f32
    [pages][Hkv][page / 32], table int32 [B][ldt].  Holds the tensors (which
    must be dense; a table's rows may be a slice of a wider one
    that holds the last row's pitch too) and the C
    descriptor of the same name.  A tensor that is assigned to one of these
    names is checked like the first ones and takes its place in the descriptor."""

    def __init__(self, Kq, Ks, Vq, Vs, table):
        self._describe(Kq, Ks, Vq, Vs, table)

    def _describe(self, Kq, Ks, Vq, Vs, table):
        import torch
        pages, Hkv, page, D = Kq.shape
        for t, dt, shape in ((Kq, torch.int8, (pages, Hkv, page, D)), (Vq, torch.int8, (pages, Hkv, page, D)),
                             (Ks, torch.float32, (pages, Hkv, page // 32)), (Vs, torch.float32, (pages, Hkv, page // 32))):
            if t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"a dense {dt} tensor of shape {shape} is needed, got {t.dtype} {tuple(t.shape)}")
        if table.dtype != torch.int32 or table.dim() != 2 or table.stride(1) != 1:
            raise ValueError("the table must be int32 [B][ldt]")
        ldt = table.stride(0) if table.shape[0] > 1 else table.shape[1]
        if table.storage_offset() + table.shape[0] * ldt > table.untyped_storage().nbytes() // 4:
            raise ValueError(f"a table's rows must be readable up to their pitch, also the last one: {table.shape[0]} rows of {ldt}"
                             f" from entry {table.storage_offset()} on leave their memory")
        self._held = {"Kq": Kq, "Ks": Ks, "Vq": Vq, "Vs": Vs, "table": table}
        self.desc = _kv8_desc(Kq.data_ptr(), Ks.data_ptr(), Vq.data_ptr(), Vs.data_ptr(), pages, Hkv, page, D,
                              table.data_ptr(), ldt, table.shape[0])
        # read on every call: plain attributes cost less than the descriptor's fields
        self.Hkv, self.D, self.B, self._ref = Hkv, D, table.shape[0], ctypes.byref(self.desc)
        self._types = {torch.float16: CQ_F16, torch.bfloat16: CQ_BF16, torch.float32: CQ_F32}
        self._int32, self._float32, self._cuda = torch.int32, torch.float32, torch._C
        self._device = Kq.get_device()

    Kq, Ks, Vq, Vs, table = map(_described, ("Kq", "Ks", "Vq", "Vs", "table"))

    @staticmethod
    def empty(pages, Hkv, page, D, table, device="cuda"):
        """A cache of zeroed pools over `table`."""
        import torch
        q = lambda: torch.zeros(pages, Hkv, page, D, dtype=torch.int8, device=device)
        s = lambda: torch.zeros(pages, Hkv, page // 32, dtype=torch.float32, device=device)
        return cq_kv8_cache(q(), s(), q(), s(), table)

    def _rows(self, t, what, heads):
        """(T, row pitch) of a [T][heads][D] tensor whose rows are dense."""
        sh, st = t.shape, t.stride()
        if len(sh) != 3 or sh[1] != heads or sh[2] != self.D or st[2] != 1 or (heads > 1 and st[1] != self.D):
            raise ValueError(f"{what} must be [T][{heads}][{self.D}] with dense rows, got shape {tuple(sh)}, strides {st}")
        return sh[0], (st[0] if sh[0] > 1 else heads * self.D)

    def _index(self, t, what, n):
        if t.dtype is not self._int32 or t.shape != (n,) or not t.is_contiguous():
            raise ValueError(f"{what} must be a dense int32 tensor of {n} entries, got {t.dtype} {tuple(t.shape)}")
        return t.data_ptr()

    def _kv(self, K, V):
        T, ldk = self._rows(K, "K", self.Hkv)
        T2, ldv = self._rows(V, "V", self.Hkv)
        if T != T2 or V.dtype != K.dtype:
            raise ValueError("K and V must have one type and shape")
        return K.data_ptr(), V.data_ptr(), self._types.get(K.dtype, -1), T, ldk, ldv

    def _stream(self, stream):
        """The given stream, else the current one of the current device (as a handle: a tenth of the time of a stream object)."""
        return self._cuda._cuda_getCurrentRawStream(self._cuda._cuda_getDevice()) if stream is None else _stream(stream)


def cq_kv8_write(cache, K, V, q_start, lens, stream=None, raise_on_error=True):
    """The rows of K, V ([T][Hkv][D], fp16/bf16/f32; rows q_start[b] .. q_start[b+1]
    - 1 of sequence b) become the last tokens of their sequences, which hold
    lens[b] tokens afterwards."""
    k, v, xt, T, ldk, ldv = cache._kv(K, V)
    st = lib().cq_kv8_write(cache._ref, k, v, xt, T, ldk, ldv, cache._index(q_start, "q_start", cache.B + 1),
                            cache._index(lens, "lens", cache.B), cache._stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_kv8_read(cache, first, out_start, K, V, stream=None, raise_on_error=True):
    """Rows out_start[b] .. out_start[b+1] - 1 of K, V ([T][Hkv][D], fp16/bf16/f32)
    become the values of tokens first[b] .. of sequence b (first None: from 0)."""
    k, v, yt, T, ldk, ldv = cache._kv(K, V)
    st = lib().cq_kv8_read(cache._ref, None if first is None else cache._index(first, "first", cache.B),
                           cache._index(out_start, "out_start", cache.B + 1), k, v, yt, T, ldk, ldv, cache._stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_attn_kv8_workspace_bytes(T, Hq, Hkv, D, B, max_q) -> int:
    return lib().cq_attn_kv8_workspace_bytes(T, Hq, Hkv, D, B, max_q)


def cq_attn_kv8(Q, cache, q_start, lens, max_q, O, ws, scale=None, causal=True, window=0, lse=None, stream=None,
                raise_on_error=True):
    """O[T][Hq][D] = softmax attention of Q [T][Hq][D] (fp16/bf16) over the cache;
    the rows of sequence b are the last of its lens[b] tokens.  scale None:
    1 / sqrt(D).  lse (f32 [T][Hq]) takes each row's log of the sum of exponentials."""
    if Q.dim() != 3:
        raise ValueError(f"Q must be [T][Hq][{cache.D}], got shape {tuple(Q.shape)}")
    Hq = Q.shape[1]
    T, ldq = cache._rows(Q, "Q", Hq)
    T2, ldo = cache._rows(O, "O", Hq)
    if T != T2:
        raise ValueError("O must have the shape of Q")
    if lse is not None and (lse.dtype is not cache._float32 or lse.shape != (T, Hq) or not lse.is_contiguous()):
        raise ValueError("lse must be a dense f32 tensor [T][Hq]")
    st = lib().cq_attn_kv8(Q.data_ptr(), cache._types.get(Q.dtype, -1), T, Hq, ldq, cache._ref,
                           cache._index(q_start, "q_start", cache.B + 1), cache._index(lens, "lens", cache.B), max_q,
                           cache.D ** -0.5 if scale is None else scale, 1 if causal else 0, window, O.data_ptr(),
                           cache._types.get(O.dtype, -1), ldo, None if lse is None else lse.data_ptr(),
                           None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel() * ws.element_size(),
                           cache._stream(stream))
    if raise_on_error:
        _check(st)
    return st


# ---- a step of drafting (include/cq_draft.h) ----------------------------

class _rope_desc(ctypes.Structure):
    _fields_ = [("freq", _c_p), ("rot", _c_i64), ("layout", _c_int), ("mag", ctypes.c_float)]


class cq_rope_spec:
    """Rotary positions: freq f32 [rot / 2] radians per position on the device, the
    layout of the pairs, a factor on the rotated channels.  Holds the tensor and
    the C descriptor of the same name.  What is assigned to one of the three names
    is checked like the first ones and takes its place in the descriptor."""

    def __init__(self, freq, layout=CQ_ROPE_HALF, mag=1.0):
        self._describe(freq, layout, mag)

    def _describe(self, freq, layout, mag):
        import torch
        if freq.dtype != torch.float32 or freq.dim() != 1 or not freq.is_contiguous():
            raise ValueError(f"freq must be a dense f32 tensor [rot / 2], got {freq.dtype} {tuple(freq.shape)}")
        self.desc = _rope_desc(freq.data_ptr(), 2 * freq.shape[0], layout, mag)
        self._held = {"freq": freq, "layout": layout, "mag": mag}
        self._ref, self._device = ctypes.byref(self.desc), freq.get_device()

    freq, layout, mag = map(_described, ("freq", "layout", "mag"))

    @staticmethod
    def make(rot, base=10000.0, kind=CQ_ROPE_PLAIN, factor=1.0, low=1.0, high=32.0, trained=8192.0, layout=CQ_ROPE_HALF, device="cuda"):
        """The spec of cq_rope_freqs' frequencies."""
        freq, mag = cq_rope_freqs(rot, base, kind, factor, low, high, trained)
        return cq_rope_spec(freq.to(device), layout, mag)


def cq_rope_freqs(rot, base=10000.0, kind=CQ_ROPE_PLAIN, factor=1.0, low=1.0, high=32.0, trained=8192.0):
    """(frequencies f32 [rot / 2] on the host, mag) of one of the kinds CQ_ROPE_PLAIN .. CQ_ROPE_BANDS."""
    import torch
    freq, mag = torch.empty(max(rot, 0) // 2, dtype=torch.float32), ctypes.c_float()
    _check(lib().cq_rope_freqs(rot, base, kind, factor, low, high, trained, freq.data_ptr(), ctypes.byref(mag)))
    return freq, mag.value


_T = None


def _types():
    """{torch type: CQ_F16 ..}, and torch's int32, f32, uint32 and its raw stream calls (looked up once: a call's time counts)."""
    global _T
    if _T is None:
        import torch
        _T = ({torch.float16: CQ_F16, torch.bfloat16: CQ_BF16, torch.float32: CQ_F32}, torch.int32, torch.float32, torch.uint32, torch._C)
    return _T


def _here(d, *tensors):
    """The current device's current stream, for tensors that all lie on that device, d (None: left out)."""
    if d >= 0:
        C = (_T or _types())[4]
        for t in tensors:
            if t is not None and t.get_device() != d:
                break
        else:
            if d == C._cuda_getDevice():
                return C._cuda_getCurrentRawStream(d)
    if d < 0 or any(t is not None and t.get_device() < 0 for t in tensors):
        raise ValueError("the tensors must be on a GPU")
    raise ValueError("the tensors must be on the current device")


def _dense(t, what, dtype, n):
    """The address of a dense tensor of n entries (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a dense {dtype} tensor of {n} entries, got {t.dtype} {tuple(t.shape)}, strides {t.stride()}")
    return t.data_ptr()


def _rows3(sh, st, what):
    """Row pitch of a [T][H][D] tensor whose rows are dense."""
    if len(sh) != 3 or (sh[2] > 1 and st[2] != 1) or (sh[1] > 1 and st[1] != sh[2]):
        raise ValueError(f"{what} must be [T][H][D] with dense rows, got shape {tuple(sh)}, strides {st}")
    return st[0] if sh[0] > 1 else sh[1] * sh[2]


def _mask(mask, T, bits):
    """(address, row pitch) of a tree's mask [T][words], int32 or uint32, rows dense and of so many bits at least."""
    sh, st, dt = mask.shape, mask.stride(), mask.dtype
    ty = _T or _types()
    if (dt is not ty[1] and dt is not ty[3]) or len(sh) != 2 or sh[0] != T or (sh[1] > 1 and st[1] != 1) or 32 * sh[1] < bits:
        raise ValueError(f"mask must be int32 [{T}][words] with dense rows of {bits} bits, got {dt} {tuple(sh)}, strides {st}")
    return mask.data_ptr(), st[0] if T > 1 else sh[1]


def cq_rope(X, rope, pos, Y=None, stream=None, raise_on_error=True):
    """Y (None: X itself) = the rows of X [T][H][D] (fp16/bf16/f32) at positions pos
    (int32 [T]), their first rot channels rotated.  Y may have another type."""
    types, i32, _, _, _ = _T or _types()
    sh = X.shape
    ldx = ldy = _rows3(sh, X.stride(), "X")
    if Y is None:
        Y = X
    elif Y is not X:
        if Y.shape != sh:
            raise ValueError("Y must have the shape of X")
        ldy = _rows3(sh, Y.stride(), "Y")
    T, H, D = sh
    s = _here(rope._device, X, Y, pos)
    st = lib().cq_rope(X.data_ptr(), types.get(X.dtype, -1), T, H, D, ldx, rope._ref, _dense(pos, "pos", i32, T), Y.data_ptr(),
                       types.get(Y.dtype, -1), ldy, s if stream is None else _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_kv8_write_rope(cache, K, V, q_start, lens, rope, pos=None, stream=None, raise_on_error=True):
    """cq_kv8_write of keys that are rotated on the way: by pos (int32 [T]), or (None)
    by their rows' places in their sequences."""
    k, v, xt, T, ldk, ldv = cache._kv(K, V)
    s = _here(cache._device, K, V, q_start, lens, pos, rope.freq)
    st = lib().cq_kv8_write_rope(cache._ref, k, v, xt, T, ldk, ldv, cache._index(q_start, "q_start", cache.B + 1),
                                 cache._index(lens, "lens", cache.B), rope._ref, _dense(pos, "pos", cache._int32, T),
                                 s if stream is None else _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_attn_kv8_tree(Q, cache, q_start, lens, max_q, mask, O, ws, scale=None, lse=None, stream=None, raise_on_error=True):
    """cq_attn_kv8 for drafted trees: a row sees every token before its sequence's rows, and of
    those the ones whose bits are set in its row of mask (int32 [T][words])."""
    if Q.dim() != 3:
        raise ValueError(f"Q must be [T][Hq][{cache.D}], got shape {tuple(Q.shape)}")
    Hq = Q.shape[1]
    T, ldq = cache._rows(Q, "Q", Hq)
    T2, ldo = cache._rows(O, "O", Hq)
    if T != T2:
        raise ValueError("O must have the shape of Q")
    bits, ldm = _mask(mask, T, min(max_q, T))
    l = _dense(lse, "lse", cache._float32, T * Hq)
    s = _here(cache._device, Q, O, q_start, lens, mask, lse, ws)
    st = lib().cq_attn_kv8_tree(Q.data_ptr(), cache._types.get(Q.dtype, -1), T, Hq, ldq, cache._ref,
                                cache._index(q_start, "q_start", cache.B + 1), cache._index(lens, "lens", cache.B), max_q,
                                cache.D ** -0.5 if scale is None else scale, bits, ldm, O.data_ptr(),
                                cache._types.get(O.dtype, -1), ldo, l, None if ws is None else ws.data_ptr(),
                                0 if ws is None else ws.numel() * ws.element_size(), s if stream is None else _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_verify(P, tokens, q_start, max_q, u, u_last, out, path, count, Q=None, mask=None, stream=None, raise_on_error=True):
    """Which of the drafted tokens stand against the target's probabilities P [T][V], and the
    token after them.  tokens int32 [T], u f32 [T], u_last f32 [B]; Q [T][V]: the draft's
    probabilities that the tokens were drawn from (None: chosen ones); mask: the
    trees (None: chains).  out, path int32 [B][max_q or more], count int32 [B]."""
    types, i32, f32, _, _ = _T or _types()
    sh, st, dt = P.shape, P.stride(), P.dtype
    if len(sh) != 2 or (sh[1] > 1 and st[1] != 1):
        raise ValueError(f"P must be [T][V] with dense rows, got shape {tuple(sh)}, strides {st}")
    T, V = sh
    ldp = ldq = st[0] if T > 1 else (V + 7) // 8 * 8             # (of one row any pitch will do)
    q = None
    if Q is not None:
        sq = Q.stride()
        if Q.shape != sh or Q.dtype is not dt or (V > 1 and sq[1] != 1):
            raise ValueError(f"Q must have the type and shape of P and dense rows, got {Q.dtype} {tuple(Q.shape)}, strides {sq}")
        q = Q.data_ptr()
        if T > 1:
            ldq = sq[0]
    B = u_last.numel()
    so, st = out.shape, out.stride()
    if out.dtype is not i32 or path.dtype is not i32 or len(so) != 2 or so[0] != B or so[1] < max_q or (so[1] > 1 and st[1] != 1) \
            or path.shape != so or path.stride() != st:
        raise ValueError(f"out and path must be int32 [{B}][{max_q} or more] with dense rows of one pitch, got {out.dtype} {tuple(so)}, strides {st}, "
                         f"and {path.dtype} {tuple(path.shape)}, strides {path.stride()}")
    bits, ldm = (None, 0) if mask is None else _mask(mask, T, max_q)
    s = _here(P.get_device(), tokens, q_start, u, u_last, out, path, count, Q, mask)
    st = lib().cq_verify(P.data_ptr(), types.get(dt, -1), T, V, ldp, q, ldq, _dense(tokens, "tokens", i32, T), bits, ldm,
                         _dense(q_start, "q_start", i32, B + 1), B, max_q, _dense(u, "u", f32, T), _dense(u_last, "u_last", f32, B),
                         out.data_ptr(), path.data_ptr(), st[0] if B > 1 else so[1], _dense(count, "count", i32, B),
                         s if stream is None else _stream(stream))
    if raise_on_error:
        _check(st)
    return st


def cq_dequant_q4(Wq, Ws, W, stream=None):
    N, K = W.shape
    _check(lib().cq_dequant_q4(_ptr(Wq), _ptr(Ws), N, K, _ptr(W), _stream(stream)))


def cq_dequant_q8row(Wq, rs, W, stream=None):
    N, K = W.shape
    _check(lib().cq_dequant_q8row(_ptr(Wq), _ptr(rs), N, K, _ptr(W), _stream(stream)))


def cq_get_device_error(stream=None) -> int:
    return lib().cq_get_device_error(_stream(stream))


def cq_last_error() -> str:
    return lib().cq_last_error().decode(errors="replace")


def cq_last_launches() -> int:
    """Kernel launches of the calling thread's most recent library call."""
    return lib().cq_last_launches()


def cq_set_option(option: int, value: int):
    _check(lib().cq_set_option(option, value))


def cq_get_option(option: int) -> int:
    return lib().cq_get_option(option)


def cq_version() -> int:
    return lib().cq_version()
