"""CSA2 sparse-attention decode over an FP4 global KV cache, GB300 (sm_103a).

Thin binding over the C ABI of ``libcsa2.so`` (declared in include/csa2.h):
argument marshalling only, by ctypes and, for the operators whose calls are short
(csa2_linear_fp4, csa2_norm_rope, csa2_dense_attn, csa2_tree_attn, csa2_cache_append, csa2_cache_read),
by the C++ module ``_native``, which is loaded at the first of them.  Every step runs in the library's CUDA kernels; PyTorch supplies device memory and
the current stream.  There is no CPU fallback: if the library is not built, every call raises.

Entry points (same names as the C ABI):
    csa2_cache_write, csa2_quantize_fp4, csa2_indexer_topk, csa2_reindex, csa2_reindex_f32,
    csa2_sparse_attn, csa2_dense_attn, csa2_tree_attn, csa2_linear_fp4, csa2_norm_rope, csa2_cache_append,
    csa2_cache_read, csa2_workspace_size, csa2_poll_error, csa2_selftest_wait_timeout
plus ``Cache``, which owns the four cache planes as torch tensors.
"""
import ctypes
import importlib.machinery
import importlib.util
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa2.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE, ERR_TIMEOUT = 0, 1, 2, 3, 4, 5
FULL, REINDEX, REUSE = 0, 1, 2
OP_INDEXER_TOPK, OP_REINDEX, OP_SPARSE_ATTN, OP_DENSE_ATTN, OP_LINEAR_FP4, OP_TREE_ATTN = 1, 2, 3, 4, 5, 6
ROPE_HALVES, ROPE_INVERSE, ROPE_NO_NORM = 1, 2, 4
WINDOW_AT_QUERY = -(1 << 63)
EVERY_ENTRY = -1
LATENTS, INDEXER_KEYS = 0, 1
D_LAT = 512


class Csa2Error(RuntimeError):
    def __init__(self, status, fn):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (fn, _status_string(status), status))


class _CacheStruct(ctypes.Structure):
    _fields_ = [("lat_codes", ctypes.c_void_p), ("lat_scales", ctypes.c_void_p),
                ("ikey_codes", ctypes.c_void_p), ("ikey_scales", ctypes.c_void_p),
                ("batch", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("d_lat", ctypes.c_int32), ("d_idx", ctypes.c_int32), ("ratio", ctypes.c_int32)]


class _HeadRows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("x_tok", ctypes.c_int64), ("x_head", ctypes.c_int64), ("y_tok", ctypes.c_int64),
                ("y_head", ctypes.c_int64), ("n_heads", ctypes.c_int32)]


_native = None
_lib = None
EXPORTS = ("csa2_cache_write", "csa2_quantize_fp4", "csa2_indexer_topk", "csa2_reindex", "csa2_sparse_attn",
           "csa2_workspace_size", "csa2_status_string", "csa2_abi_version", "csa2_launch_count",
           "csa2_reindex_noalloc", "csa2_reindex_f32", "csa2_poll_error", "csa2_selftest_wait_timeout",
           "csa2_cache_write_projected", "csa2_linear_fp4", "csa2_norm_rope", "csa2_dense_attn",
           "csa2_tree_attn", "csa2_cache_append", "csa2_cache_read")


def load(path=None):
    """Load libcsa2.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError("libcsa2.so is not built (%s); run __graft_entry__.build()" % p)
    lib = ctypes.CDLL(p)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    cp = ctypes.POINTER(_CacheStruct)
    lib.csa2_cache_write.argtypes = [cp, vp, i64, i32, vp, vp, vp, vp]
    lib.csa2_cache_write_projected.argtypes = [cp, vp, i64, i32, vp, vp, vp, vp, vp]
    lib.csa2_cache_write_projected.restype = ctypes.c_int
    lib.csa2_quantize_fp4.argtypes = [vp, i64, i32, vp, vp, vp]
    lib.csa2_indexer_topk.argtypes = [cp, vp, vp, vp, i32, vp, i32, i32, vp, i32, i32, vp, vp, sz, vp]
    lib.csa2_reindex.argtypes = [i32, cp, vp, vp, vp, i32, i32, vp, i32, vp, i32, vp, vp, sz, vp]
    lib.csa2_reindex_f32.argtypes = [cp, vp, vp, i32, i32, vp, i32, i32, vp, vp, sz, vp]
    lib.csa2_sparse_attn.argtypes = [cp, vp, i32, i32, vp, vp, i32, vp, i64, i32, ctypes.c_float, vp, vp, vp, sz, vp]
    lib.csa2_linear_fp4.argtypes = [vp, i32, i64, i64, i32, i32, i32, i32, vp, vp, ctypes.c_float, vp, i32, i64,
                                    i64, vp, sz, vp]
    hp = ctypes.POINTER(_HeadRows)
    lib.csa2_norm_rope.argtypes = [hp, hp, i32, i32, i32, i32, i32, vp, vp, ctypes.c_float, i32, vp]
    lib.csa2_dense_attn.argtypes = [cp, vp, i32, i32, vp, vp, vp, i32, ctypes.c_float, vp, i32, vp, vp, sz, vp]
    lib.csa2_tree_attn.argtypes = [cp, vp, i32, i32, vp, vp, vp, vp, i32, vp, vp, i32, ctypes.c_float, vp, i32, vp, vp, sz, vp]
    lib.csa2_cache_append.argtypes = [cp, vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.csa2_cache_read.argtypes = [cp, i32, vp, i64, i64, vp, i32, vp]
    lib.csa2_reindex_noalloc.argtypes = [cp, vp, vp, vp, i32, i32, vp, i32, i32, vp, vp]
    lib.csa2_reindex_noalloc.restype = ctypes.c_int
    lib.csa2_poll_error.argtypes = [vp, sz, vp]
    lib.csa2_poll_error.restype = ctypes.c_int
    lib.csa2_selftest_wait_timeout.argtypes = [ctypes.c_uint32, vp, sz, vp]
    lib.csa2_selftest_wait_timeout.restype = ctypes.c_int
    lib.csa2_workspace_size.argtypes = [i32, i32, i32, i32, i32, i64]
    lib.csa2_workspace_size.restype = sz
    lib.csa2_status_string.argtypes = [ctypes.c_int]
    lib.csa2_status_string.restype = ctypes.c_char_p
    lib.csa2_abi_version.restype = i32
    lib.csa2_launch_count.restype = i64
    for name in ("csa2_cache_write", "csa2_quantize_fp4", "csa2_indexer_topk", "csa2_reindex", "csa2_reindex_f32",
                 "csa2_sparse_attn", "csa2_linear_fp4", "csa2_norm_rope", "csa2_dense_attn", "csa2_tree_attn",
                 "csa2_cache_append", "csa2_cache_read"):
        getattr(lib, name).restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def _load_native():
    """the C++ part of the binding, for the operators that go through it (nothing else needs it)"""
    global _native
    lib = load()
    p = os.path.join(_HERE, "_native.so")
    if not os.path.exists(p):
        raise RuntimeError("_native.so is not built (%s); run __graft_entry__.build()" % p)
    spec = importlib.util.spec_from_file_location("_native", p, loader=importlib.machinery.ExtensionFileLoader("_native", p))
    native = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(native)
    native.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in
                  (lib.csa2_linear_fp4, lib.csa2_norm_rope, lib.csa2_dense_attn, lib.csa2_tree_attn, lib.csa2_cache_append,
                   lib.csa2_cache_read, lib.csa2_workspace_size)))
    _native = native


def _status_string(s):
    try:
        return load().csa2_status_string(s).decode()
    except Exception:
        return "status %d" % s


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    """the cudaStream_t of `stream`, or of PyTorch's current stream (asked for as a plain pointer:
    building a torch.cuda.Stream takes longer than a launch)"""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _check(status, fn):
    if status != OK:
        raise Csa2Error(status, fn)


class Cache:
    """The four planes of the FP4 global KV cache (device tensors, uint8); ratio
    raw positions per entry (2: an encoder copy, 1: the decoder's)."""

    def __init__(self, batch, capacity, d_idx=128, device="cuda", ratio=2):
        self.batch, self.capacity, self.d_idx, self.ratio = batch, capacity, d_idx, ratio
        self.lat_codes = torch.zeros((batch, capacity, D_LAT // 2), dtype=torch.uint8, device=device)
        self.lat_scales = torch.zeros((batch, capacity, D_LAT // 16), dtype=torch.uint8, device=device)
        self.ikey_codes = torch.zeros((batch, capacity, d_idx // 2), dtype=torch.uint8, device=device)
        self.ikey_scales = torch.zeros((batch, capacity, d_idx // 16), dtype=torch.uint8, device=device)

    @classmethod
    def of(cls, lat_codes, lat_scales, ikey_codes=None, ikey_scales=None, ratio=2):
        """a cache over planes that exist already (uint8, contiguous): lat_codes [B, n, 256],
        lat_scales [B, n, 32] and, for the indexer, ikey_codes [B, n, d_idx/2] and ikey_scales"""
        c = object.__new__(cls)
        c.batch, c.capacity = lat_codes.shape[0], lat_codes.shape[1]
        c.d_idx = 128 if ikey_codes is None else 2 * ikey_codes.shape[-1]
        c.ratio = ratio
        c.lat_codes, c.lat_scales, c.ikey_codes, c.ikey_scales = lat_codes, lat_scales, ikey_codes, ikey_scales
        return c

    def struct(self):
        ik, iks = self.ikey_codes, self.ikey_scales
        return _CacheStruct(self.lat_codes.data_ptr(), self.lat_scales.data_ptr(), ik.data_ptr() if ik is not None else 0,
                            iks.data_ptr() if iks is not None else 0, self.batch, self.capacity, D_LAT, self.d_idx,
                            getattr(self, "ratio", 2))

    def nbytes(self):
        return sum(t.numel() for t in (self.lat_codes, self.lat_scales, self.ikey_codes, self.ikey_scales)
                   if t is not None)


def csa2_launch_count():
    return load().csa2_launch_count()


def csa2_workspace_size(op, batch, n_q, n_heads, k, capacity):
    return load().csa2_workspace_size(op, batch, n_q, n_heads, k, capacity)


def workspace(op, batch, n_q, n_heads, k, capacity, device="cuda"):
    """a workspace for the operation, its error word cleared"""
    n = csa2_workspace_size(op, batch, n_q, n_heads, k, capacity)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=device)
    ws[:16].zero_()
    return ws


def csa2_poll_error(ws, stream=None):
    """reads and clears the error word of a workspace: OK, or ERR_TIMEOUT if a
    kernel that used it gave up on a bounded wait (synchronises the stream)"""
    return load().csa2_poll_error(_ptr(ws), ws.numel(), _stream(stream))


def csa2_selftest_wait_timeout(max_polls, ws, stream=None):
    """a kernel waits on a barrier nothing signals, with at most max_polls polls,
    gives up and records it in ws's error word"""
    _check(load().csa2_selftest_wait_timeout(int(max_polls), _ptr(ws), ws.numel(), _stream(stream)),
           "csa2_selftest_wait_timeout")


def csa2_cache_write(cache, h, pos0, w0, w1, ikey_raw=None, stream=None):
    """h: bf16 [B, n_pos, 512] (as torch.bfloat16 or int16 bits); w0/w1 fp32 [512];
    ikey_raw bf16 [B, n_pos/2, d_idx] or None."""
    c = cache.struct()
    st = load().csa2_cache_write(ctypes.byref(c), _ptr(h), int(pos0), int(h.shape[1]), _ptr(w0), _ptr(w1),
                                 _ptr(ikey_raw), _stream(stream))
    _check(st, "csa2_cache_write")


def csa2_cache_write_projected(cache, h, pos0, w0, w1, wik_codes, wik_scales, stream=None):
    """as csa2_cache_write, with the indexer keys projected from the entries:
    wik_codes uint8 [d_idx, 256], wik_scales uint8 [d_idx, 32] (FP4 W)"""
    c = cache.struct()
    st = load().csa2_cache_write_projected(ctypes.byref(c), _ptr(h), int(pos0), int(h.shape[1]), _ptr(w0), _ptr(w1),
                                           _ptr(wik_codes), _ptr(wik_scales), _stream(stream))
    _check(st, "csa2_cache_write_projected")


def csa2_quantize_fp4(x, codes=None, scales=None, stream=None):
    """fp32 [..., d] -> (codes uint8 [..., d/2], scales uint8 [..., d/16])"""
    d = x.shape[-1]
    if codes is None:
        codes = torch.empty(x.shape[:-1] + (d // 2,), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(x.shape[:-1] + (d // 16,), dtype=torch.uint8, device=x.device)
    st = load().csa2_quantize_fp4(_ptr(x), x.numel() // d, d, _ptr(codes), _ptr(scales), _stream(stream))
    _check(st, "csa2_quantize_fp4")
    return codes, scales


def csa2_indexer_topk(cache, iq_codes, iq_scales, w_head, q_pos, k, pool_blocks=0, pool_block_size=8,
                      idx_out=None, pool_out=None, ws=None, stream=None):
    """Full-mode indexer + top-k (+ HSI pool).  iq_codes [B, n_q, H_I, d_idx/2] ...
    Returns (idx [B, n_q, k] int32, pool [B, n_q, P] int32 or None)."""
    B, n_q, H = iq_codes.shape[0], iq_codes.shape[1], iq_codes.shape[2]
    dev = iq_codes.device
    if idx_out is None:
        idx_out = torch.empty((B, n_q, k), dtype=torch.int32, device=dev)
    if pool_blocks and pool_out is None:
        P = pool_blocks * pool_block_size if pool_block_size else pool_blocks   # 0: the pure pool
        pool_out = torch.empty((B, n_q, P), dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(OP_INDEXER_TOPK, cache.batch, n_q, H, k, cache.capacity, dev)
    c = cache.struct()
    st = load().csa2_indexer_topk(ctypes.byref(c), _ptr(iq_codes), _ptr(iq_scales), _ptr(w_head), n_q, _ptr(q_pos),
                                  H, k, _ptr(idx_out), pool_blocks, pool_block_size,
                                  _ptr(pool_out) if pool_blocks else None, _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "csa2_indexer_topk")
    return idx_out, (pool_out if pool_blocks else None)


def csa2_reindex(mode, cache, k, iq_codes=None, iq_scales=None, w_head=None, pool=None, prev_idx=None,
                 idx_out=None, ws=None, stream=None, n_q=None):
    """mode REINDEX: top-k inside the pool with this layer's indexer queries;
    mode REUSE: copy prev_idx."""
    if n_q is None:
        n_q = (iq_codes if iq_codes is not None else prev_idx).shape[1]
    dev = (iq_codes if iq_codes is not None else prev_idx).device
    if idx_out is None:
        idx_out = torch.empty((cache.batch, n_q, k), dtype=torch.int32, device=dev)
    H = iq_codes.shape[2] if iq_codes is not None else 0
    pool_len = pool.shape[-1] if pool is not None else 0
    if mode == REINDEX and ws is None:
        ws = workspace(OP_REINDEX, cache.batch, n_q, H, k, pool_len, dev)
    c = cache.struct()
    st = load().csa2_reindex(mode, ctypes.byref(c), _ptr(iq_codes), _ptr(iq_scales), _ptr(w_head), n_q, H,
                             _ptr(pool), pool_len, _ptr(prev_idx), k, _ptr(idx_out), _ptr(ws),
                             ws.numel() if ws is not None else 0, _stream(stream))
    _check(st, "csa2_reindex")
    return idx_out


def csa2_reindex_f32(cache, k, iq, w_head, pool, idx_out=None, ws=None, stream=None):
    """Reindex from fp32 indexer queries iq [B, n_q, H, d_idx]: the query
    quantisation runs inside the Reindex kernels (same results as
    csa2_quantize_fp4 followed by csa2_reindex)."""
    B, n_q, H = iq.shape[0], iq.shape[1], iq.shape[2]
    if idx_out is None:
        idx_out = torch.empty((B, n_q, k), dtype=torch.int32, device=iq.device)
    pool_len = pool.shape[-1]
    if ws is None:
        ws = workspace(OP_REINDEX, cache.batch, n_q, H, k, pool_len, iq.device)
    c = cache.struct()
    st = load().csa2_reindex_f32(ctypes.byref(c), _ptr(iq), _ptr(w_head), n_q, H, _ptr(pool), pool_len, k,
                                 _ptr(idx_out), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "csa2_reindex_f32")
    return idx_out


def csa2_reindex_noalloc(cache, k, iq_codes, iq_scales, w_head, pool, idx_out=None, stream=None):
    """Reindex with the library's built-in scratch instead of a workspace (for
    callers that cannot allocate device memory; see include/csa2.h)."""
    B, n_q, H = iq_codes.shape[0], iq_codes.shape[1], iq_codes.shape[2]
    if idx_out is None:
        idx_out = torch.empty((B, n_q, k), dtype=torch.int32, device=iq_codes.device)
    c = cache.struct()
    st = load().csa2_reindex_noalloc(ctypes.byref(c), _ptr(iq_codes), _ptr(iq_scales), _ptr(w_head), n_q, H,
                                     _ptr(pool), pool.shape[-1], k, _ptr(idx_out), _stream(stream))
    _check(st, "csa2_reindex_noalloc")
    return idx_out


def csa2_sparse_attn(cache, q, q_pos, idx, swa, swa_pos0, scale=D_LAT ** -0.5, out=None, lse=None,
                     want_lse=False, ws=None, stream=None):
    """q bf16 [B, n_q, H, 512]; idx int32 [B, n_q, k]; swa bf16 [B, swa_len, 512], row r at raw position
    swa_pos0 + r, or with swa_pos0 = WINDOW_AT_QUERY the last row at each sequence's last query.
    Returns (out fp32 [B, n_q, H, 512], lse fp32 [B, n_q, H] or None)."""
    B, n_q, H = q.shape[0], q.shape[1], q.shape[2]
    k = idx.shape[-1] if idx is not None else 0
    if out is None:
        out = torch.empty((B, n_q, H, D_LAT), dtype=torch.float32, device=q.device)
    if want_lse and lse is None:
        lse = torch.empty((B, n_q, H), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = workspace(OP_SPARSE_ATTN, cache.batch, n_q, H, k, cache.capacity, q.device)
    c = cache.struct()
    st = load().csa2_sparse_attn(ctypes.byref(c), _ptr(q), n_q, H, _ptr(q_pos), _ptr(idx), k, _ptr(swa),
                                 int(swa_pos0), int(swa.shape[1]) if swa is not None else 0, float(scale), _ptr(out),
                                 _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "csa2_sparse_attn")
    return out, lse


def csa2_linear_fp4(x, codes, scales, alpha=1.0, out=None, out_dtype=None, ws=None, stream=None):
    """y = alpha * W x with FP4 weights (csa2_quantize_fp4's format), for every token.
    x bf16 / fp16 / fp32 [T, n_in] with codes uint8 [n_out, n_in/2] and scales uint8 [n_out, n_in/16], or
    x [T, G, n_in] with codes [G, n_out, n_in/2] and scales [G, n_out, n_in/16] (a product per group).
    Rows of x and out are contiguous, their other strides free.  Returns [T, n_out] or [T, G, n_out]
    of out_dtype (default: that of x).  With a stream other than the current one, give `out` (a new one
    belongs to the current stream); without ws the scratch is taken for the call's own stream."""
    if _native is None:
        _load_native()
    r = _native.linear_fp4(x, codes, scales, alpha, out, out_dtype, ws, None if stream is None else stream.cuda_stream)
    if type(r) is int:
        raise Csa2Error(r, "csa2_linear_fp4")
    return r


def csa2_norm_rope(q, pos, inv_freq, q_weight=None, k=None, k_weight=None, eps=1e-6, norm=True, halves=False,
                   inverse=False, q_out=None, k_out=None, out_dtype=None, stream=None):
    """RMS norm of every head row of q [T, Hq, d] (and k [T, Hk, d]) with the rotation of its last
    2 * len(inv_freq) values by pos int64 [T] * inv_freq fp32; norm=False rotates only, inverse=True
    turns back, halves=True pairs value i with i + d_rot/2 (default: 2i with 2i+1).  pos and inv_freq
    may both be None (no rotation).  bf16 / fp16 / fp32, rows contiguous, other strides free; q_out may
    be q.  Returns (q_out, k_out or None)."""
    if _native is None:
        _load_native()
    r = _native.norm_rope(q, pos, inv_freq, q_weight, k, k_weight, eps, norm, halves, inverse, q_out, k_out, out_dtype,
                          None if stream is None else stream.cuda_stream)
    if type(r) is int:
        raise Csa2Error(r, "csa2_norm_rope")
    return r


def csa2_dense_attn(cache, q, q_pos, swa, swa_pos0, scale=D_LAT ** -0.5, out=None, out_dtype=torch.bfloat16, lse=None,
                    want_lse=False, ws=None, stream=None):
    """Attention over every visible entry of the cache and the window: q bf16 [B, n_q, H, 512]; q_pos
    int64 [B, n_q]; swa bf16 [B, swa_len, 512] or None, row r of sequence b at raw position
    swa_pos0[b] + r (int64 [B] on the device, or None: zeros).  Returns (out [B, n_q, H, 512], lse
    fp32 [B, n_q, H] or None).  With a stream other than the current one, give out and lse (new ones
    belong to the current stream); without ws the scratch is taken for the call's own stream, and a
    bounded wait that gave up cannot be polled."""
    if _native is None:
        _load_native()
    r = _native.dense_attn(cache.lat_codes, cache.lat_scales, cache.ratio, q, q_pos, swa, swa_pos0, scale, out, out_dtype,
                           lse, want_lse, ws, None if stream is None else stream.cuda_stream)
    if type(r) is int:
        raise Csa2Error(r, "csa2_dense_attn")
    return r


def csa2_tree_attn(cache, q, q_pos, parent, draft, swa, swa_pos0, idx=None, scale=D_LAT ** -0.5, out=None,
                   out_dtype=torch.bfloat16, lse=None, want_lse=False, ws=None, stream=None):
    """Attention of drafted trees: q bf16 [B, n, H, 512] and draft bf16 [B, n, 512] of up to 128 nodes a
    sequence, q_pos int64 [B, n] their raw positions, parent int32 [B, n] (an earlier node, -1: a child of
    the last committed token, anything else: not there).  A node sees every visible entry, or with idx int32
    [B, n, k] those of its list; the committed rows of its window (swa and swa_pos0 as in csa2_dense_attn); its
    ancestors' and its own draft rows.  Returns (out [B, n, H, 512], lse fp32 [B, n, H] or None), zeros
    and -inf for nodes that are not there.  Streams, out, lse and ws as in csa2_dense_attn; a workspace is
    workspace(OP_TREE_ATTN, B, n, H, k, capacity), with k EVERY_ENTRY where there is no idx."""
    if _native is None:
        _load_native()
    r = _native.tree_attn(cache.lat_codes, cache.lat_scales, cache.ratio, q, q_pos, parent, draft, swa, swa_pos0, idx, scale,
                          out, out_dtype, lse, want_lse, ws, None if stream is None else stream.cuda_stream)
    if type(r) is int:
        raise Csa2Error(r, "csa2_tree_attn")
    return r


def csa2_cache_append(cache, rows, pos0, path=None, prev=None, prev_out=None, w0=None, w1=None, wik_codes=None,
                      wik_scales=None, stream=None):
    """Rows into the cache, each sequence at its own position pos0 int64 [B]: rows bf16 [B, n, 512] in their
    order, or those that path int32 [B, m] names (up to its first number that is no row).  A ratio-2 cache
    takes prev bf16 [B, 512], the row of position pos0 - 1, leaves the last one in prev_out (may be prev; None:
    not wanted) and takes w0, w1 as csa2_cache_write does.  With wik_codes and wik_scales the indexer keys are
    projected from the entries."""
    if _native is None:
        _load_native()
    r = _native.cache_append(cache.lat_codes, cache.lat_scales, cache.ikey_codes, cache.ikey_scales, cache.ratio, rows, pos0, path,
                             prev, prev_out, w0, w1, wik_codes, wik_scales, None if stream is None else stream.cuda_stream)
    if type(r) is int:
        raise Csa2Error(r, "csa2_cache_append")


def csa2_cache_read(cache, idx=None, first=0, count=None, keys=False, out=None, out_dtype=torch.bfloat16, stream=None):
    """Entries as values, bf16, fp16 or fp32: those that idx int32 [B, ..] names (zeros for -1 and for numbers
    outside the cache), or count of them from `first` on (default: all).  Latents [.., 512], or with
    keys=True indexer keys [.., d_idx].  With a stream other than the current one, give out."""
    if _native is None:
        _load_native()
    r = _native.cache_read(cache.lat_codes, cache.lat_scales, cache.ikey_codes, cache.ikey_scales, cache.ratio, idx, first, count,
                           keys, out, out_dtype, None if stream is None else stream.cuda_stream)
    if type(r) is int:
        raise Csa2Error(r, "csa2_cache_read")
    return r
