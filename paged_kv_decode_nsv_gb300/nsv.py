"""Thin ctypes binding of libnsv.so (declared in include/nsv.h).

Argument marshalling only: every step of the decode read and the KV append
runs in the library's CUDA kernels.  Tensors are torch tensors on the current
CUDA device, C-contiguous, in the layouts nsv.h documents:

  q, out          [rows, num_heads, head_dim]               float32 | bfloat16
                  or [rows, query_len, num_heads, head_dim] (several query
                  tokens per row, causal among themselves)
  k_pool, v_pool  [num_blocks + 1, num_kv_heads, 16, head_dim]  (last = sink)
  k_new, v_new    [rows, num_kv_heads, head_dim] or [rows, query_len, ...]
  write_slots     [rows] or [rows, query_len] int64
  block_tables    [rows, max_blocks] int32
  context_lens    [rows] int32

The chunk attention (paged_chunk, chunk_step) takes ragged batches instead:

  q, out          [tokens, num_heads, head_dim]
  k_new, v_new    [tokens, num_kv_heads, head_dim], write_slots [tokens] int64
  chunk_starts    [rows + 1] int32: row r's tokens are chunk_starts[r] ..
                  chunk_starts[r + 1] - 1
  slopes          [num_heads] float32; see_begin, see_end [tokens] int32

The page operators (blocks_copy, rows_fork, rows_extend, rows_free,
blocks_compact) keep block_refs [num_blocks] int32, the references to each
block (0: free), with the tables and lengths, and change them in place.

Importing this module loads the library and raises ImportError if it has not
been built (``python -m paged_kv_decode_nsv_gb300.build``); there is no
fallback path.
"""

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libnsv.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libnsv.so is not built (%s); run python -m paged_kv_decode_nsv_gb300.build"
                      % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)

ABI_VERSION = 102  # the layout of Shape and Plan below
F32, BF16 = 0, 1
(CONSUMER_AUTO, CONSUMER_CUDA, CONSUMER_TENSOR, CONSUMER_TENSOR_VECTOR_ROWS,
 CONSUMER_TENSOR_TMEM) = 0, 1, 2, 3, 4
DEV_BAD_CTX, DEV_BAD_BLOCK, DEV_BAD_SLOT, DEV_TIMEOUT = 1, 2, 4, 8
DEV_BAD_CHUNK, DEV_BAD_ROW, DEV_NO_BLOCKS = 16, 32, 64
ERRORS = {0: "NSV_OK", -1: "NSV_ERR_NULLPTR", -2: "NSV_ERR_DTYPE", -3: "NSV_ERR_SHAPE",
          -4: "NSV_ERR_ALIGN", -5: "NSV_ERR_RANGE", -6: "NSV_ERR_CAPTURE", -7: "NSV_ERR_CUDA",
          -8: "NSV_ERR_WORKSPACE", -10: "NSV_ERR_UNSUPPORTED"}


class Shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("max_blocks", ctypes.c_int32),
                ("num_blocks", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("query_len", ctypes.c_int32)]


class Plan(ctypes.Structure):
    _fields_ = [("kv_heads_per_cta", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("ctas_per_sm", ctypes.c_int32), ("grid", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("smem_bytes", ctypes.c_int32),
                ("num_sms", ctypes.c_int32), ("vectors_per_warp", ctypes.c_int32),
                ("consumer", ctypes.c_int32), ("blocks_per_stage", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_int64)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


class Scores(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("see_begin", ctypes.c_void_p), ("see_end", ctypes.c_void_p)]


_vp, _i32, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_SP, _PP = ctypes.POINTER(Shape), ctypes.POINTER(Plan)

_lib.nsv_abi_version.restype = _i32
_lib.nsv_abi_version.argtypes = []
if _lib.nsv_abi_version() != ABI_VERSION:
    raise ImportError("libnsv.so has ABI version %d, this binding expects %d; rebuild it"
                      % (_lib.nsv_abi_version(), ABI_VERSION))
_lib.nsv_strerror.restype = ctypes.c_char_p
_lib.nsv_strerror.argtypes = [_i32]
_lib.nsv_plan_split.restype = _i32
_lib.nsv_plan_split.argtypes = [_SP, _i32, _PP]
_lib.nsv_plan_custom.restype = _i32
_lib.nsv_plan_custom.argtypes = [_SP, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _PP]
_lib.nsv_plan_resident_ctas.restype = _i32
_lib.nsv_plan_resident_ctas.argtypes = [_SP, _PP, ctypes.POINTER(ctypes.c_int)]
_lib.nsv_kv_write.restype = _i32
_lib.nsv_kv_write.argtypes = [_SP, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.nsv_paged_decode.restype = _i32
_lib.nsv_paged_decode.argtypes = [_SP, _vp, _vp, _vp, _vp, _vp, _f, _vp, _vp]
_lib.nsv_paged_decode_ws.restype = _i32
_lib.nsv_paged_decode_ws.argtypes = [_SP, _PP, _vp, _vp, _vp, _vp, _vp, _f, _vp, _vp, _sz, _vp]
_lib.nsv_decode_step.restype = _i32
_lib.nsv_decode_step.argtypes = [_SP, _PP, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _f, _vp,
                                 _vp, _sz, _vp]
_lib.nsv_paged_decode_slots.restype = _i32
_lib.nsv_paged_decode_slots.argtypes = [_SP, _PP, _vp, _vp, _vp, _vp, ctypes.c_int64,
                                        ctypes.c_int64, _vp, _f, _vp, _vp, _sz, _vp]
_lib.nsv_paged_decode_noalloc.restype = _i32
_lib.nsv_paged_decode_noalloc.argtypes = [_SP, _vp, _vp, _vp, _vp, _vp, _f, _vp, _vp]
_i64 = ctypes.c_int64
_lib.nsv_chunk_workspace.restype = _i32
_lib.nsv_chunk_workspace.argtypes = [_SP, _i64, _i32, ctypes.POINTER(_i64)]
_lib.nsv_paged_chunk.restype = _i32
_lib.nsv_paged_chunk.argtypes = [_SP, ctypes.POINTER(Scores), _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _f, _vp, _vp, _sz, _vp]
_lib.nsv_chunk_step.restype = _i32
_lib.nsv_chunk_step.argtypes = [_SP, ctypes.POINTER(Scores), _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                _vp, _vp, _vp, _f, _vp, _vp, _sz, _vp]
_lib.nsv_pages_workspace.restype = _i32
_lib.nsv_pages_workspace.argtypes = [_SP, ctypes.POINTER(_i64)]
_i32c = ctypes.c_int32
for _name, _args in (("blocks_copy", [_i32c, _vp, _vp, _vp, _vp, _vp]),
                     ("rows_fork", [_i32c, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
                     ("rows_extend", [_i64, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
                     ("rows_free", [_i32c, _vp, _vp, _vp, _vp, _vp]),
                     ("blocks_compact", [_vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp])):
    getattr(_lib, "nsv_" + _name).restype = _i32
    getattr(_lib, "nsv_" + _name).argtypes = [_SP] + _args
_lib.nsv_device_status.restype = _i32
_lib.nsv_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint32),
                                   ctypes.POINTER(ctypes.c_uint64), _i32]
_lib.nsv_status_async.restype = _i32
_lib.nsv_status_async.argtypes = [_vp, _i32, _vp]
_lib.nsv_selftest_bounded_wait.restype = _i32
_lib.nsv_selftest_bounded_wait.argtypes = [ctypes.c_uint64, ctypes.POINTER(ctypes.c_int),
                                           ctypes.POINTER(ctypes.c_uint64), _vp]


class NsvError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__("%s: %s (%s)" % (where, ERRORS.get(code, code),
                                          _lib.nsv_strerror(code).decode()))


def _check(rc, where):
    if rc != 0:
        raise NsvError(rc, where)


def lib_path():
    return LIB_PATH


def abi_version():
    return _lib.nsv_abi_version()


def strerror(code):
    return _lib.nsv_strerror(code).decode()


def make_shape(rows, num_heads, num_kv_heads, head_dim, max_blocks, num_blocks, dtype,
               block_size=16, query_len=1):
    return Shape(rows, num_heads, num_kv_heads, head_dim, block_size, max_blocks, num_blocks,
                 dtype, query_len)


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("nsv tensors must be float32 or bfloat16, got %s" % t.dtype)


def _ptr(t, what):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % what)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return t.data_ptr()


def shape_of(q, k_pool, block_tables):
    """nsv_shape from the read's tensors (q is [R, H, D] or [R, NQ, H, D])."""
    if q.dim() == 4:
        R, NQ, H, D = q.shape
    else:
        (R, H, D), NQ = q.shape, 1
    NB1, Hkv, B, D2 = k_pool.shape
    if D2 != D:
        raise ValueError("q head_dim %d != pool head_dim %d" % (D, D2))
    if block_tables.shape[0] != R:
        raise ValueError("block_tables rows %d != q rows %d" % (block_tables.shape[0], R))
    if q.dtype != k_pool.dtype:
        raise ValueError("q and the pool must share one dtype")
    return make_shape(R, H, Hkv, D, block_tables.shape[1], NB1 - 1, _dtype_code(k_pool), B,
                      query_len=NQ)


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def plan_split(shape, num_sms=0):
    p = Plan()
    _check(_lib.nsv_plan_split(ctypes.byref(shape), int(num_sms), ctypes.byref(p)),
           "nsv_plan_split")
    return p


def plan_custom(shape, num_sms=0, kv_heads_per_cta=0, stages=0, ctas_per_sm=0, grid=0,
                vectors_per_warp=0, consumer=CONSUMER_AUTO, blocks_per_stage=0):
    p = Plan()
    _check(_lib.nsv_plan_custom(ctypes.byref(shape), int(num_sms), int(kv_heads_per_cta),
                                int(stages), int(ctas_per_sm), int(grid), int(vectors_per_warp),
                                int(consumer), int(blocks_per_stage), ctypes.byref(p)),
           "nsv_plan_custom")
    return p


def plan_resident_ctas(shape, plan):
    """CTAs of the plan's kernel that one SM of the current device holds."""
    n = ctypes.c_int(0)
    _check(_lib.nsv_plan_resident_ctas(ctypes.byref(shape), ctypes.byref(plan), ctypes.byref(n)),
           "nsv_plan_resident_ctas")
    return n.value


def workspace_for(plan, device=None):
    """A caller-owned workspace tensor for `plan` (None when it needs none)."""
    import torch
    if plan.workspace_bytes == 0:
        return None
    return torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=device or "cuda")


def kv_write(k_new, v_new, write_slots, k_pool, v_pool, stream=None):
    if k_new.dim() == 4:
        k_new = k_new.reshape(-1, k_new.shape[2], k_new.shape[3])
        v_new = v_new.reshape(-1, v_new.shape[2], v_new.shape[3])
        write_slots = write_slots.reshape(-1)
    R, Hkv, D = k_new.shape
    NB1, Hkv2, B, D2 = k_pool.shape
    if (Hkv, D) != (Hkv2, D2) or k_new.dtype != k_pool.dtype or v_new.dtype != k_pool.dtype:
        raise ValueError("k_new/v_new do not match the pool")
    shape = make_shape(R, Hkv2, Hkv2, D2, 1, NB1 - 1, _dtype_code(k_pool), B)
    _check(_lib.nsv_kv_write(ctypes.byref(shape), _ptr(k_new, "k_new"), _ptr(v_new, "v_new"),
                             _ptr(write_slots, "write_slots"), _ptr(k_pool, "k_pool"),
                             _ptr(v_pool, "v_pool"), _stream(stream)), "nsv_kv_write")


def paged_decode(q, k_pool, v_pool, block_tables, context_lens, scale, out, stream=None):
    """Decode read with the default plan and the library-owned workspace."""
    shape = shape_of(q, k_pool, block_tables)
    _check(_lib.nsv_paged_decode(ctypes.byref(shape), _ptr(q, "q"), _ptr(k_pool, "k_pool"),
                                 _ptr(v_pool, "v_pool"), _ptr(block_tables, "block_tables"),
                                 _ptr(context_lens, "context_lens"), float(scale),
                                 _ptr(out, "out"), _stream(stream)), "nsv_paged_decode")
    return out


def paged_decode_noalloc(q, k_pool, v_pool, block_tables, context_lens, scale, out,
                         stream=None):
    """Decode read that allocates no device memory (scratch from the library's
    fixed buffer; see nsv_paged_decode_noalloc in nsv.h for the size limit)."""
    shape = shape_of(q, k_pool, block_tables)
    _check(_lib.nsv_paged_decode_noalloc(ctypes.byref(shape), _ptr(q, "q"),
                                         _ptr(k_pool, "k_pool"), _ptr(v_pool, "v_pool"),
                                         _ptr(block_tables, "block_tables"),
                                         _ptr(context_lens, "context_lens"), float(scale),
                                         _ptr(out, "out"), _stream(stream)),
           "nsv_paged_decode_noalloc")
    return out


def paged_decode_ws(q, k_pool, v_pool, block_tables, context_lens, scale, out, workspace=None,
                    plan=None, stream=None):
    """Decode read with an explicit plan (None: default) and caller workspace."""
    shape = shape_of(q, k_pool, block_tables)
    ws_ptr = _ptr(workspace, "workspace")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.nsv_paged_decode_ws(ctypes.byref(shape), ctypes.byref(plan) if plan else None,
                                    _ptr(q, "q"), _ptr(k_pool, "k_pool"), _ptr(v_pool, "v_pool"),
                                    _ptr(block_tables, "block_tables"),
                                    _ptr(context_lens, "context_lens"), float(scale),
                                    _ptr(out, "out"), ws_ptr, ws_bytes, _stream(stream)),
           "nsv_paged_decode_ws")
    return out


def paged_decode_slots(q, k_pool, v_pool, slot_table, context_lens, scale, out, workspace=None,
                       plan=None, max_blocks=None, stream=None):
    """Decode read through a per-token slot table.

    slot_table is an int64 [rows, width] tensor whose rows may be strided (a
    window of a wider table, as slots[:rows, :width] of a persistent buffer);
    its last dimension must be contiguous.  max_blocks defaults to
    cdiv(width, 16) and only sizes the plan.
    """
    import torch
    if slot_table.dtype != torch.int64 or slot_table.dim() != 2 or \
            (slot_table.shape[1] > 1 and slot_table.stride(1) != 1):
        raise ValueError("slot_table must be an int64 [rows, width] tensor with unit column stride")
    if not slot_table.is_cuda:
        raise ValueError("slot_table must be a CUDA tensor")
    rows, width = slot_table.shape
    mb = max_blocks or (width + 15) // 16
    if q.dim() == 4:
        R, NQ, H, D = q.shape
    else:
        (R, H, D), NQ = q.shape, 1
    NB1, Hkv, B, _ = k_pool.shape
    shape = make_shape(R, H, Hkv, D, mb, NB1 - 1, _dtype_code(k_pool), B, query_len=NQ)
    ws_ptr = _ptr(workspace, "workspace")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.nsv_paged_decode_slots(ctypes.byref(shape), ctypes.byref(plan) if plan else None,
                                       _ptr(q, "q"), _ptr(k_pool, "k_pool"),
                                       _ptr(v_pool, "v_pool"), slot_table.data_ptr(), int(width),
                                       int(slot_table.stride(0)),
                                       _ptr(context_lens, "context_lens"), float(scale),
                                       _ptr(out, "out"), ws_ptr, ws_bytes, _stream(stream)),
           "nsv_paged_decode_slots")
    return out


def decode_step(q, k_new, v_new, write_slots, k_pool, v_pool, block_tables, context_lens, scale,
                out, workspace=None, plan=None, stream=None):
    """Append then read, on one stream (workspace None: the library's)."""
    shape = shape_of(q, k_pool, block_tables)
    ws_ptr = _ptr(workspace, "workspace")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.nsv_decode_step(ctypes.byref(shape), ctypes.byref(plan) if plan else None,
                                _ptr(q, "q"), _ptr(k_new, "k_new"), _ptr(v_new, "v_new"),
                                _ptr(write_slots, "write_slots"), _ptr(k_pool, "k_pool"),
                                _ptr(v_pool, "v_pool"), _ptr(block_tables, "block_tables"),
                                _ptr(context_lens, "context_lens"), float(scale),
                                _ptr(out, "out"), ws_ptr, ws_bytes, _stream(stream)),
           "nsv_decode_step")
    return out


def _arg(t, what, dtype, shape, device):
    """The pointer of an argument that must be a contiguous CUDA tensor of this
    type and shape on device number `device`; None passes as NULL."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape:
        raise ValueError("%s must be %s %s, got %s %s" % (what, dtype, list(shape), t.dtype,
                                                          list(t.shape)))
    if t.get_device() != device:
        raise ValueError("%s is on %s, not on the current CUDA device %d"
                         % (what, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    return t.data_ptr()


def _raw_stream(stream, device):
    """The handle of a torch stream (None: the current one on `device`)."""
    import torch
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device)


def _call(what, args, need, workspace, stream, device):
    """Calls `what` of the library with a workspace: the caller's, or memory that
    torch's caching allocator lends for the call on its stream.  (A raw allocation:
    a tensor around it costs a call 5 us more.)"""
    import torch
    fn, raw = getattr(_lib, what), _raw_stream(stream, device)
    if workspace is None:
        ptr = torch._C._cuda_cudaCachingAllocator_raw_alloc(need, raw)
        try:
            rc = fn(*args, ptr, need, raw)
        finally:
            torch._C._cuda_cudaCachingAllocator_raw_delete(ptr)
    else:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous, on the current CUDA device")
        rc = fn(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), raw)
    _check(rc, what)


def chunk_workspace_bytes(shape, tokens, num_sms=0):
    """Workspace bytes of paged_chunk and chunk_step for up to `tokens` tokens."""
    n = _i64(0)
    _check(_lib.nsv_chunk_workspace(ctypes.byref(shape), int(tokens), int(num_sms),
                                    ctypes.byref(n)), "nsv_chunk_workspace")
    return n.value


@functools.lru_cache(maxsize=4096)
def _chunk_sizes(device, rows, heads, kv_heads, head_dim, max_blocks, num_blocks, dtype,
                 block_size, tokens):
    """A reference to the nsv_shape of these sizes, and its workspace bytes."""
    shape = make_shape(rows, heads, kv_heads, head_dim, max_blocks, num_blocks, dtype, block_size)
    return ctypes.byref(shape), chunk_workspace_bytes(shape, tokens)


def _chunk_args(q, k_pool, v_pool, block_tables, chunk_starts, context_lens, out, softcap, slopes,
                see_begin, see_end):
    import torch
    dev = torch.cuda.current_device()
    qs, ks, bs, dt, i32 = q.shape, k_pool.shape, block_tables.shape, k_pool.dtype, torch.int32
    if len(qs) != 3 or len(ks) != 4 or len(bs) != 2:
        raise ValueError("q must be [tokens, heads, head_dim], the pools [blocks + 1, kv_heads, "
                         "16, head_dim] and block_tables [rows, max_blocks]")
    (T, H, D), (NB1, Hkv, B, D2), (R, MB) = qs, ks, bs
    if D2 != D:
        raise ValueError("q head_dim %d != pool head_dim %d" % (D, D2))
    ptrs = (_arg(q, "q", dt, qs, dev), _arg(k_pool, "k_pool", dt, ks, dev),
            _arg(v_pool, "v_pool", dt, ks, dev), _arg(block_tables, "block_tables", i32, bs, dev),
            _arg(chunk_starts, "chunk_starts", i32, (R + 1,), dev),
            _arg(context_lens, "context_lens", i32, (R,), dev))
    out_ptr = _arg(out, "out", dt, qs, dev)
    shape, need = _chunk_sizes(dev, R, H, Hkv, D, MB, NB1 - 1, _dtype_code(k_pool), B, T)
    scores = None
    if softcap or slopes is not None or see_begin is not None or see_end is not None:
        scores = ctypes.byref(Scores(float(softcap),
                                     _arg(slopes, "slopes", torch.float32, (H,), dev),
                                     _arg(see_begin, "see_begin", i32, (T,), dev),
                                     _arg(see_end, "see_end", i32, (T,), dev)))
    return shape, scores, T, ptrs, out_ptr, need, dev


def paged_chunk(q, k_pool, v_pool, block_tables, chunk_starts, context_lens, scale, out,
                softcap=0.0, slopes=None, see_begin=None, see_end=None, workspace=None,
                stream=None):
    """Attention of each row's new tokens over its paged context (nsv_paged_chunk
    in nsv.h): causal, or with capped and biased scores and visibility bounds.
    workspace: chunk_workspace_bytes() of uint8, or None to allocate it."""
    shape, scores, T, ptrs, out_ptr, need, dev = _chunk_args(
        q, k_pool, v_pool, block_tables, chunk_starts, context_lens, out, softcap, slopes,
        see_begin, see_end)
    _call("nsv_paged_chunk", (shape, scores, T, *ptrs, float(scale), out_ptr),
          need, workspace, stream, dev)
    return out


def chunk_step(q, k_new, v_new, write_slots, k_pool, v_pool, block_tables, chunk_starts,
               context_lens, scale, out, softcap=0.0, slopes=None, see_begin=None, see_end=None,
               workspace=None, stream=None):
    """Append the new tokens' keys and values, then paged_chunk, on one stream."""
    import torch
    shape, scores, T, ptrs, out_ptr, need, dev = _chunk_args(
        q, k_pool, v_pool, block_tables, chunk_starts, context_lens, out, softcap, slopes,
        see_begin, see_end)
    new = (T, k_pool.shape[1], q.shape[2])
    new_ptrs = (_arg(k_new, "k_new", q.dtype, new, dev), _arg(v_new, "v_new", q.dtype, new, dev),
                _arg(write_slots, "write_slots", torch.int64, (T,), dev))
    args = (shape, scores, T, ptrs[0], *new_ptrs, *ptrs[1:], float(scale), out_ptr)
    _call("nsv_chunk_step", args, need, workspace, stream, dev)
    return out


def pages_workspace_bytes(rows, num_blocks):
    """Workspace bytes of rows_fork, rows_extend and blocks_compact."""
    n = _i64(0)
    shape = make_shape(rows, 1, 1, 64, 1, num_blocks, F32)
    _check(_lib.nsv_pages_workspace(ctypes.byref(shape), ctypes.byref(n)), "nsv_pages_workspace")
    return n.value


@functools.lru_cache(maxsize=4096)
def _page_sizes(rows, max_blocks, num_blocks, kv_heads, head_dim, dtype, block_size):
    """A reference to the nsv_shape of these sizes, and its workspace bytes."""
    shape = make_shape(rows, kv_heads, kv_heads, head_dim, max_blocks, num_blocks, dtype,
                       block_size)
    return ctypes.byref(shape), pages_workspace_bytes(rows, num_blocks)


def _pool_args(k_pool, v_pool, num_blocks, dev):
    ks, dt = k_pool.shape, k_pool.dtype
    if len(ks) != 4:
        raise ValueError("the pools must be [blocks + 1, kv_heads, 16, head_dim]")
    if num_blocks is not None and ks[0] != num_blocks + 1:
        raise ValueError("the pools have %d blocks and the sink, block_refs %d"
                         % (ks[0] - 1, num_blocks))
    return _arg(k_pool, "k_pool", dt, ks, dev), _arg(v_pool, "v_pool", dt, ks, dev)


def _cache_args(block_tables, context_lens, block_refs, dev):
    import torch
    i32, bs, n = torch.int32, block_tables.shape, block_refs.numel()
    if len(bs) != 2:
        raise ValueError("block_tables must be [rows, max_blocks]")
    return (_arg(block_tables, "block_tables", i32, bs, dev),
            _arg(context_lens, "context_lens", i32, bs[:1], dev),
            _arg(block_refs, "block_refs", i32, (n,), dev)), bs[0], bs[1], n


def _pool_sizes(rows, max_blocks, k_pool):
    NB1, Hkv, B, D = k_pool.shape
    return _page_sizes(rows, max_blocks, NB1 - 1, Hkv, D, _dtype_code(k_pool), B)


def blocks_copy(src_blocks, dst_blocks, k_pool, v_pool, stream=None):
    """Copy blocks src_blocks[i] of both pools to dst_blocks[i] (int32 tensors)."""
    import torch
    dev, i32, n = torch.cuda.current_device(), torch.int32, src_blocks.numel()
    pools = _pool_args(k_pool, v_pool, None, dev)
    shape, _ = _pool_sizes(0, 1, k_pool)
    _check(_lib.nsv_blocks_copy(shape, n, _arg(src_blocks, "src_blocks", i32, (n,), dev),
                                _arg(dst_blocks, "dst_blocks", i32, (n,), dev), *pools,
                                _raw_stream(stream, dev)), "nsv_blocks_copy")


def rows_fork(parents, children, block_tables, context_lens, block_refs, k_pool, v_pool,
              workspace=None, stream=None):
    """Make empty rows children[i] copies of rows parents[i] (int32 tensors):
    full blocks are shared, a partly filled last one is copied."""
    import torch
    dev, i32, n = torch.cuda.current_device(), torch.int32, parents.numel()
    cache, rows, width, blocks = _cache_args(block_tables, context_lens, block_refs, dev)
    pools = _pool_args(k_pool, v_pool, blocks, dev)
    shape, need = _pool_sizes(rows, width, k_pool)
    ids = _arg(parents, "parents", i32, (n,), dev), _arg(children, "children", i32, (n,), dev)
    _call("nsv_rows_fork", (shape, n, *ids, *cache, *pools), need, workspace, stream, dev)


def rows_extend(chunk_starts, block_tables, context_lens, block_refs, write_slots, workspace=None,
                stream=None):
    """Grow each row by its new tokens: blocks, lengths, and the tokens' write
    slots (int64 [tokens]), as chunk_step takes them."""
    import torch
    dev, T = torch.cuda.current_device(), write_slots.numel()
    cache, rows, width, blocks = _cache_args(block_tables, context_lens, block_refs, dev)
    starts = _arg(chunk_starts, "chunk_starts", torch.int32, (rows + 1,), dev)
    slots = _arg(write_slots, "write_slots", torch.int64, (T,), dev)
    shape, need = _page_sizes(rows, width, blocks, 1, 64, F32, 16)
    _call("nsv_rows_extend", (shape, T, starts, *cache, slots), need, workspace, stream, dev)
    return write_slots


def rows_free(rows, block_tables, context_lens, block_refs, stream=None):
    """Free the rows listed in `rows` (an int32 tensor)."""
    import torch
    dev, n = torch.cuda.current_device(), rows.numel()
    cache, R, width, blocks = _cache_args(block_tables, context_lens, block_refs, dev)
    shape, _ = _page_sizes(R, width, blocks, 1, 64, F32, 16)
    _check(_lib.nsv_rows_free(shape, n, _arg(rows, "rows", torch.int32, (n,), dev), *cache,
                              _raw_stream(stream, dev)), "nsv_rows_free")


def blocks_compact(block_tables, context_lens, block_refs, k_pool, v_pool, workspace=None,
                   stream=None):
    """Move the blocks in use to the front of the pool; tables and references
    follow."""
    import torch
    dev = torch.cuda.current_device()
    cache, rows, width, blocks = _cache_args(block_tables, context_lens, block_refs, dev)
    pools = _pool_args(k_pool, v_pool, blocks, dev)
    shape, need = _pool_sizes(rows, width, k_pool)
    _call("nsv_blocks_compact", (shape, *cache, *pools), need, workspace, stream, dev)


def selftest_bounded_wait(limit_ns, stream=None):
    """Run the decode kernel's bounded wait on a barrier nothing completes;
    returns (gave_up, waited_ns).  Synchronises the stream."""
    gave_up = ctypes.c_int(0)
    waited = ctypes.c_uint64(0)
    _check(_lib.nsv_selftest_bounded_wait(int(limit_ns), ctypes.byref(gave_up),
                                          ctypes.byref(waited), _stream(stream)),
           "nsv_selftest_bounded_wait")
    return gave_up.value, waited.value


def status_async(dst, clear=True, stream=None):
    """Enqueue a copy of the device status word into `dst` (a uint32/int32
    tensor of at least one element, on the device or in pinned host memory)
    and, with `clear`, zero the word, both on `stream`; no synchronisation.
    Read `dst` once the stream has reached the copy."""
    import torch
    if dst.dtype not in (torch.int32, torch.uint32) or dst.numel() < 1:
        raise ValueError("dst must be an int32 or uint32 tensor of at least one element")
    if not dst.is_cuda and not dst.is_pinned():
        raise ValueError("dst must be device memory or pinned host memory")
    _check(_lib.nsv_status_async(dst.data_ptr(), 1 if clear else 0, _stream(stream)),
           "nsv_status_async")
    return dst


def device_status(clear=True):
    """(status bits, walked (row, block) pairs) of the current device; synchronises."""
    st = ctypes.c_uint32(0)
    w = ctypes.c_uint64(0)
    _check(_lib.nsv_device_status(ctypes.byref(st), ctypes.byref(w), 1 if clear else 0),
           "nsv_device_status")
    return st.value, w.value
