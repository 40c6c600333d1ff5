"""GB300 (sm_103a) group-wise affine-quantized multi-row matmul.

Thin ctypes binding of the C ABI in ``include/qmm.h`` (``libqmm.so`` in this
directory). It only marshals arguments: every step of the computation runs in
the library's CUDA kernels. PyTorch is used for device memory and streams.

    import bit_affine_quantized_group_gb300 as qmm
    plan = qmm.Plan(K=5120, N=17408, bits=4, group=32, max_M=16, out_dtype="bf16")
    qmm.forward(plan, x, w, s, b, out)        # tensors on the plan's device

The library is built by ``bit_affine_quantized_group_gb300._build`` (nvcc for
sm_103a). There is no fallback: if the library is missing, the first call
raises ImportError.
"""
from __future__ import annotations

import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqmm.so")

QMM_OK = 0
QMM_ERR_INVALID_ARG = 1
QMM_ERR_UNSUPPORTED = 2
QMM_ERR_PLAN_MISMATCH = 3
QMM_ERR_CUDA = 4
QMM_ERR_ALLOC = 5
QMM_ERR_TIMEOUT = 6
QMM_ERR_SCRATCH_LIMIT = 7
NOALLOC_SCRATCH_BYTES = 4 << 20
QMM_OUT_F32 = 0
QMM_OUT_BF16 = 1
MAX_ROWS = 16
MAX_BANKS = 64
MAX_SPLITS = 16
QMM_IN_F32 = 0
QMM_IN_BF16 = 1
KV_TIMEOUT = 7
KV_BAD_PAGE = 16
KV_BAD_LENGTH = 32
KV_BAD_POSITION = 64
SAMPLE_MAX_VOCAB = 393216

# Every entry point declared in include/qmm.h.
EXPORTS = (
    "qmm_validate_desc", "qmm_workspace_bytes", "qmm_plan", "qmm_plan_get_info",
    "qmm_check_forward_args", "qmm_forward", "qmm_forward_banked", "qmm_unpack_codes",
    "qmm_plan_error", "qmm_destroy", "qmm_status_string", "qmm_forward_noalloc", "qmm_forward_swiglu",
    "qmm_kv_validate_desc", "qmm_kv_workspace_bytes", "qmm_kv_plan", "qmm_kv_error", "qmm_kv_destroy",
    "qmm_check_qk_norm_rope_args", "qmm_qk_norm_rope", "qmm_check_attention_args", "qmm_attention", "qmm_sample",
)


class QmmDesc(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int64), ("N", ctypes.c_int64), ("bits", ctypes.c_int32),
                ("group", ctypes.c_int32), ("max_M", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("splits", ctypes.c_int32), ("max_banks", ctypes.c_int32)]


class QmmPlanInfo(ctypes.Structure):
    _fields_ = [("splits", ctypes.c_int32), ("chunks", ctypes.c_int32), ("stages", ctypes.c_int32 * 2),
                ("smem_bytes", ctypes.c_int32 * 2), ("num_sms", ctypes.c_int32), ("device", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_int64)]


class QmmKvDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("q_heads", "kv_heads", "head_dim", "page_size", "max_seqs", "max_rows",
                                              "max_pages", "window", "sinks", "rot_dim", "interleaved")] + \
               [("scale", ctypes.c_float), ("eps", ctypes.c_float)]


class QmmKvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("num_pages", ctypes.c_int64)] + \
               [(f"{s}_{d}_stride", ctypes.c_int64) for s in "kv" for d in ("page", "head", "slot")]


class QmmAttentionArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lengths", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64),
                ("seqs", ctypes.c_int32), ("rows", ctypes.c_int32)]


class QmmAppendArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("rope", ctypes.c_void_p),
                ("rope_len", ctypes.c_int64), ("lengths", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("q_out_stride", ctypes.c_int64),
                ("seqs", ctypes.c_int32), ("rows", ctypes.c_int32), ("in_dtype", ctypes.c_int32)]


class QmmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"qmm CUDA library not built ({LIB_PATH} missing); run "
                          "`python -m bit_affine_quantized_group_gb300._build` (needs nvcc, sm_103a)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    pp = ctypes.POINTER(ctypes.c_void_p)
    lib.qmm_validate_desc.argtypes = [ctypes.POINTER(QmmDesc)]
    lib.qmm_workspace_bytes.argtypes = [ctypes.POINTER(QmmDesc)]
    lib.qmm_workspace_bytes.restype = sz
    lib.qmm_plan.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(QmmDesc), vp, sz]
    lib.qmm_plan_get_info.argtypes = [vp, ctypes.POINTER(QmmPlanInfo)]
    lib.qmm_check_forward_args.argtypes = [ctypes.POINTER(QmmDesc), vp, i32, i32, pp, pp, pp, i64, i64, i32, i32, pp]
    lib.qmm_forward.argtypes = [vp, vp, i32, vp, vp, vp, i64, i64, i32, i32, vp, vp]
    lib.qmm_forward_banked.argtypes = [vp, vp, i32, i32, pp, pp, pp, i64, i64, i32, i32, pp, vp]
    lib.qmm_forward_swiglu.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, vp, vp]
    lib.qmm_unpack_codes.argtypes = [vp, i64, i64, i32, vp, vp]
    lib.qmm_forward_noalloc.argtypes = [vp, i32, vp, vp, vp, i64, i64, i32, i32, i32, vp, vp]
    lib.qmm_plan_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.qmm_destroy.argtypes = [vp]
    lib.qmm_destroy.restype = None
    kvd, kvc = ctypes.POINTER(QmmKvDesc), ctypes.POINTER(QmmKvCache)
    lib.qmm_kv_validate_desc.argtypes = [kvd]
    lib.qmm_kv_workspace_bytes.argtypes = [kvd]
    lib.qmm_kv_workspace_bytes.restype = sz
    lib.qmm_kv_plan.argtypes = [ctypes.POINTER(vp), kvd, vp, sz]
    lib.qmm_kv_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.qmm_kv_destroy.argtypes = [vp]
    lib.qmm_kv_destroy.restype = None
    lib.qmm_check_qk_norm_rope_args.argtypes = [kvd, kvc, vp]
    lib.qmm_qk_norm_rope.argtypes = [vp, kvc, vp, vp]
    lib.qmm_check_attention_args.argtypes = [kvd, kvc, vp]
    lib.qmm_attention.argtypes = [vp, kvc, vp, vp]
    lib.qmm_sample.argtypes = [vp, i32, i32, i64, i32, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.qmm_status_string.argtypes = [i32]
    lib.qmm_status_string.restype = ctypes.c_char_p
    for name in EXPORTS:
        if name not in ("qmm_workspace_bytes", "qmm_destroy", "qmm_status_string", "qmm_kv_workspace_bytes",
                        "qmm_kv_destroy"):
            getattr(lib, name).restype = i32
    return lib


_LIB = None


def _lib() -> ctypes.CDLL:
    """The loaded libqmm.so (loaded on first use; ImportError if it was never built)."""
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def __getattr__(name):
    if name == "lib":
        return _lib()
    raise AttributeError(name)


def status_string(status: int) -> str:
    return _lib().qmm_status_string(int(status)).decode()


def _out_code(out_dtype) -> int:
    if out_dtype in ("f32", "float32", QMM_OUT_F32):
        return QMM_OUT_F32
    if out_dtype in ("bf16", "bfloat16", QMM_OUT_BF16):
        return QMM_OUT_BF16
    try:
        import torch
        if out_dtype is torch.float32:
            return QMM_OUT_F32
        if out_dtype is torch.bfloat16:
            return QMM_OUT_BF16
    except ImportError:
        pass
    raise ValueError(f"unsupported out_dtype {out_dtype!r}")


def make_desc(K, N, bits, group, max_M=16, out_dtype="bf16", splits=0, max_banks=1) -> QmmDesc:
    return QmmDesc(int(K), int(N), int(bits), int(group), int(max_M), _out_code(out_dtype), int(splits),
                   int(max_banks))


def validate_desc(desc: QmmDesc) -> int:
    return int(_lib().qmm_validate_desc(ctypes.byref(desc)))


def workspace_bytes(desc: QmmDesc) -> int:
    return int(_lib().qmm_workspace_bytes(ctypes.byref(desc)))


def _stream_handle(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


# What calls of a few microseconds take from torch, looked up once (torch is imported when it is first needed).
_F32 = _BF16 = _I32 = _RAW_STREAM = _CURRENT_DEVICE = None


def _bind_torch() -> None:
    global _F32, _BF16, _I32, _RAW_STREAM, _CURRENT_DEVICE
    import torch
    _F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
    _RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _CURRENT_DEVICE = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_on(stream, device: int) -> int:
    """_stream_handle without a Stream object for the current stream: calls of a few microseconds notice it."""
    if stream is None and _RAW_STREAM is not None and device >= 0:
        return _RAW_STREAM(device)
    return _stream_handle(stream)


def _wait_for_block(dev) -> None:
    """A block from the allocator may still be written by what was launched before on the current stream; the library clears a
    workspace on another one."""
    import torch
    torch.cuda.current_stream(dev).synchronize()


class Plan:
    """A qmm plan (qmm_plan / qmm_destroy). By default its workspace is a
    PyTorch-allocated device buffer (so PyTorch's allocator owns the memory);
    pass ``torch_workspace=False`` to let the library cudaMalloc it."""

    def __init__(self, K, N, bits, group, max_M=16, out_dtype="bf16", splits=0, max_banks=1,
                 torch_workspace: bool = True, device=None):
        import torch
        self.desc = make_desc(K, N, bits, group, max_M, out_dtype, splits, max_banks)
        st = validate_desc(self.desc)
        if st != QMM_OK:
            raise QmmError(st, "qmm_validate_desc")
        self.K, self.N, self.bits, self.group = int(K), int(N), int(bits), int(group)
        self.max_M, self.max_banks = int(max_M), int(max_banks)
        self.out_dtype = torch.float32 if self.desc.out_dtype == QMM_OUT_F32 else torch.bfloat16
        self._handle = ctypes.c_void_p()
        self.workspace = None
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        with torch.cuda.device(dev):
            if torch_workspace:
                nbytes = workspace_bytes(self.desc)
                self.workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device=dev)
                base = self.workspace.data_ptr()
                aligned = (base + 255) // 256 * 256
                _wait_for_block(dev)
                st = _lib().qmm_plan(ctypes.byref(self._handle), ctypes.byref(self.desc), ctypes.c_void_p(aligned),
                                  ctypes.c_size_t(nbytes))
            else:
                st = _lib().qmm_plan(ctypes.byref(self._handle), ctypes.byref(self.desc), None, ctypes.c_size_t(0))
        if st != QMM_OK:
            raise QmmError(st, "qmm_plan")
        self.device = dev

    @property
    def handle(self):
        return self._handle

    def info(self) -> dict:
        inf = QmmPlanInfo()
        st = _lib().qmm_plan_get_info(self._handle, ctypes.byref(inf))
        if st != QMM_OK:
            raise QmmError(st, "qmm_plan_get_info")
        return {"splits": inf.splits, "chunks": inf.chunks, "stages": list(inf.stages),
                "smem_bytes": list(inf.smem_bytes), "num_sms": inf.num_sms, "device": inf.device,
                "workspace_bytes": inf.workspace_bytes}

    def error_flags(self) -> int:
        v = ctypes.c_uint32(0)
        st = _lib().qmm_plan_error(self._handle, ctypes.byref(v))
        if st not in (QMM_OK, QMM_ERR_TIMEOUT):
            raise QmmError(st, "qmm_plan_error")
        return int(v.value)

    def close(self):
        if self._handle is not None and self._handle.value:
            _lib().qmm_destroy(self._handle)
            self._handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _ptr(t) -> int:
    return int(t.data_ptr()) if t is not None else 0


def forward(plan: Plan, x, w, s, b, out, stream=None) -> None:
    """out[M, N] = qmm(x[M, K], w, s, b) via qmm_forward (asynchronous on `stream`)."""
    M = int(x.shape[0]) if x.dim() == 2 else 1
    st = _lib().qmm_forward(plan.handle, ctypes.c_void_p(_ptr(x)), M, ctypes.c_void_p(_ptr(w)),
                         ctypes.c_void_p(_ptr(s)), ctypes.c_void_p(_ptr(b)), plan.K, plan.N, plan.bits,
                         plan.group, ctypes.c_void_p(_ptr(out)), ctypes.c_void_p(_stream_handle(stream)))
    if st != QMM_OK:
        raise QmmError(st, "qmm_forward")


def _ptr_array(ts):
    arr = (ctypes.c_void_p * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = _ptr(t)
    return arr


def forward_banked(plan: Plan, x, ws, ss, bs, outs, stream=None) -> None:
    """One launch for len(ws) projections sharing x (qmm_forward_banked)."""
    n = len(ws)
    M = int(x.shape[0]) if x.dim() == 2 else 1
    st = _lib().qmm_forward_banked(plan.handle, ctypes.c_void_p(_ptr(x)), M, n, _ptr_array(ws), _ptr_array(ss),
                                _ptr_array(bs), plan.K, plan.N, plan.bits, plan.group, _ptr_array(outs),
                                ctypes.c_void_p(_stream_handle(stream)))
    if st != QMM_OK:
        raise QmmError(st, "qmm_forward_banked")


def forward_swiglu(plan: Plan, x, w_gate, s_gate, b_gate, w_up, s_up, b_up, out, stream=None) -> None:
    """out[M, N] = silu(qmm(x, gate weights)) * qmm(x, up weights) in one main-kernel
    launch (qmm_forward_swiglu; the plan needs max_banks >= 2)."""
    M = int(x.shape[0]) if x.dim() == 2 else 1
    vp = ctypes.c_void_p
    st = _lib().qmm_forward_swiglu(plan.handle, vp(_ptr(x)), M, vp(_ptr(w_gate)), vp(_ptr(s_gate)),
                                   vp(_ptr(b_gate)), vp(_ptr(w_up)), vp(_ptr(s_up)), vp(_ptr(b_up)), plan.K,
                                   plan.N, plan.bits, plan.group, vp(_ptr(out)), vp(_stream_handle(stream)))
    if st != QMM_OK:
        raise QmmError(st, "qmm_forward_swiglu")


def check_forward_args(desc: QmmDesc, x_ptr: int, M: int, w_ptrs, s_ptrs, b_ptrs, K, N, bits, group,
                       out_ptrs) -> int:
    """Host-only argument check (qmm_check_forward_args); pointers are plain integers."""
    def arr(ps):
        if ps is None:
            return None
        a = (ctypes.c_void_p * len(ps))()
        for i, p in enumerate(ps):
            a[i] = p
        return a
    n = len(w_ptrs) if w_ptrs is not None else 1
    return int(_lib().qmm_check_forward_args(ctypes.byref(desc), ctypes.c_void_p(x_ptr), int(M), n, arr(w_ptrs),
                                          arr(s_ptrs), arr(b_ptrs), int(K), int(N), int(bits), int(group),
                                          arr(out_ptrs)))


def unpack_codes(w, K: int, N: int, bits: int, stream=None):
    """Run the kernels' in-register unpacking on packed words; returns uint8 [N, K]."""
    import torch
    codes = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    st = _lib().qmm_unpack_codes(ctypes.c_void_p(_ptr(w)), int(K), int(N), int(bits), ctypes.c_void_p(_ptr(codes)),
                              ctypes.c_void_p(_stream_handle(stream)))
    if st != QMM_OK:
        raise QmmError(st, "qmm_unpack_codes")
    return codes


def make_kv_desc(q_heads, kv_heads, head_dim, page_size, max_seqs, max_rows, max_pages, window=0, sinks=0, rot_dim=None,
                 interleaved=False, scale=None, eps=1e-6) -> QmmKvDesc:
    """Descriptor of a KVPlan; rot_dim defaults to head_dim and scale to head_dim ** -0.5."""
    return QmmKvDesc(int(q_heads), int(kv_heads), int(head_dim), int(page_size), int(max_seqs), int(max_rows),
                     int(max_pages), int(window), int(sinks), int(head_dim if rot_dim is None else rot_dim),
                     int(bool(interleaved)), float(head_dim ** -0.5 if scale is None else scale), float(eps))


def kv_validate_desc(desc: QmmKvDesc) -> int:
    return int(_lib().qmm_kv_validate_desc(ctypes.byref(desc)))


def kv_workspace_bytes(desc: QmmKvDesc) -> int:
    return int(_lib().qmm_kv_workspace_bytes(ctypes.byref(desc)))


class KVPlan:
    """A plan of the cache operators (qmm_kv_plan / qmm_kv_destroy) for one kind of attention layer. Its workspace
    is a PyTorch-allocated device buffer unless ``torch_workspace=False``; keep the plan until its calls have run.
    Arguments as for `make_kv_desc`."""

    def __init__(self, *args, torch_workspace: bool = True, device=None, **kwargs):
        import torch
        _bind_torch()
        self.desc = d = make_kv_desc(*args, **kwargs)
        st = kv_validate_desc(d)
        if st != QMM_OK:
            raise QmmError(st, "qmm_kv_validate_desc")
        self._handle = ctypes.c_void_p()
        self.workspace = None
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        if dev.index is None:
            dev = torch.device(dev.type, torch.cuda.current_device())
        with torch.cuda.device(dev):
            ws, nbytes = None, 0
            if torch_workspace:
                nbytes = kv_workspace_bytes(d)
                self.workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device=dev)
                ws = (self.workspace.data_ptr() + 255) // 256 * 256
                _wait_for_block(dev)
            st = _lib().qmm_kv_plan(ctypes.byref(self._handle), ctypes.byref(d), ws, nbytes)
        if st != QMM_OK:
            raise QmmError(st, "qmm_kv_plan")
        self.device, self._device_index = dev, dev.index
        self.q_width, self.kv_width = d.q_heads * d.head_dim, d.kv_heads * d.head_dim
        self.page_shape = (d.kv_heads, d.page_size, d.head_dim)
        self.max_pages, self.head_dim, self.rot_dim = d.max_pages, d.head_dim, d.rot_dim

    @property
    def handle(self):
        return self._handle

    def error_flags(self) -> int:
        """The KV_BAD_* bits of the calls since the last read, cleared. Waits for the device, whatever streams they are on."""
        v = ctypes.c_uint32(0)
        st = _lib().qmm_kv_error(self._handle, ctypes.byref(v))
        if st not in (QMM_OK, QMM_ERR_INVALID_ARG, QMM_ERR_TIMEOUT):
            raise QmmError(st, "qmm_kv_error")
        return int(v.value)

    def close(self):
        if self._handle is not None and self._handle.value:
            _lib().qmm_kv_destroy(self._handle)
            self._handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KVCache:
    """The pages of keys and values as the cache operators take them: two bfloat16 tensors
    [pages, kv_heads, page_size, head_dim] of any strides with adjacent elements in the last dimension (a pool laid
    out [pages, page_size, kv_heads, head_dim] is passed as its transpose(1, 2))."""

    def __init__(self, k, v):
        import torch
        for t in (k, v):
            if t.get_device() != k.get_device():
                raise ValueError("k and v are on the same device")
            if t.dim() != 4 or t.dtype != torch.bfloat16 or t.shape != k.shape or t.stride(3) != 1:
                raise ValueError("k and v are bfloat16 tensors [pages, kv_heads, page_size, head_dim] of the same shape")
        self.k, self.v = k, v
        self.device_index = k.get_device()
        self.page_shape = tuple(k.shape[1:])
        self.struct = QmmKvCache(k.data_ptr(), v.data_ptr(), k.shape[0], *k.stride()[:3], *v.stride()[:3])
        self.ref = ctypes.byref(self.struct)


# What a call passes to the library, packed for each call: threads may share a plan.
_APPEND_ARGS = struct.Struct("@3P3q3Pq4Pq3i4x")      # QmmAppendArgs
_ATTENTION_ARGS = struct.Struct("@4P2q2i")           # QmmAttentionArgs
assert _APPEND_ARGS.size == ctypes.sizeof(QmmAppendArgs) and _ATTENTION_ARGS.size == ctypes.sizeof(QmmAttentionArgs)


def _rows(t, tokens, width, dtype, what):
    """Elements between the rows of a tensor [tokens, width] or [tokens, heads, head_dim] of adjacent heads. One token's row may
    be any contiguous tensor."""
    shape, st = t.shape, t.stride()
    if t.dtype is dtype:
        n = len(shape)
        if n > 1 and shape[0] == tokens and st[-1] == 1 and \
                (shape[1] == width if n == 2 else
                 n == 3 and shape[1] * shape[2] == width and (st[1] == shape[2] or shape[1] == 1)):
            return st[0]
        if tokens == 1 and t.numel() == width and t.is_contiguous():
            return width
    raise ValueError(f"{what}: {tokens} {dtype} rows of {width} adjacent elements are needed")


def _check_step(plan, cache, page_table, lengths, tokens, *others):
    device = plan._device_index
    if cache.device_index != device or page_table.get_device() != device or lengths.get_device() != device:
        raise ValueError(f"cache, page_table and lengths are on the plan's device {plan.device}")
    for t in others:
        if t is not None and t.get_device() != device:
            raise ValueError(f"all tensors are on the plan's device {plan.device}")
    seqs = lengths.numel()
    if cache.page_shape != plan.page_shape:
        raise ValueError("the cache's pages are not the plan's [kv_heads, page_size, head_dim]")
    if lengths.dtype is not _I32 or page_table.dtype is not _I32 or not page_table.is_contiguous() or \
            not lengths.is_contiguous() or page_table.shape != (seqs, plan.max_pages):
        raise ValueError("lengths [seqs] and page_table [seqs, max_pages] are contiguous int32 tensors")
    rows, rest = divmod(tokens, seqs) if seqs else (0, tokens)
    if rest:
        raise ValueError("every sequence has the same number of rows")
    return seqs, rows


def qk_norm_rope(plan: KVPlan, q, k, v, q_weight, k_weight, rope, lengths, page_table, cache: KVCache, out,
                 positions=None, stream=None) -> None:
    """Norms of q and k for each head, rotation, and the append of k and v to the cache (qmm_qk_norm_rope). q, k, v:
    [tokens, heads * head_dim] of float32 or bfloat16, rows of any stride; out: the queries, bfloat16. q_weight and
    k_weight: float32 [head_dim] or None; rope: float32 [positions, rot_dim], cosines then sines."""
    dtype, tokens = q.dtype, q.shape[0]
    seqs, rows = _check_step(plan, cache, page_table, lengths, tokens, q, k, v, out, q_weight, k_weight, rope, positions)
    if dtype is not _F32 and dtype is not _BF16:
        raise ValueError("q, k and v are float32 or bfloat16")
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype is not _F32 or w.numel() != plan.head_dim or not w.is_contiguous()):
            raise ValueError("q_weight and k_weight are float32 [head_dim] or None")
    if plan.rot_dim and (rope is None or rope.dtype is not _F32 or not rope.is_contiguous() or rope.dim() != 2 or
                         rope.shape[1] != plan.rot_dim):
        raise ValueError("rope is a float32 tensor [positions, rot_dim]")
    if positions is not None and (positions.dtype is not _I32 or positions.numel() != tokens or
                                  not positions.is_contiguous()):
        raise ValueError("positions is an int32 tensor [tokens]")
    args = _APPEND_ARGS.pack(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _rows(q, tokens, plan.q_width, dtype, "q"),
        _rows(k, tokens, plan.kv_width, dtype, "k"), _rows(v, tokens, plan.kv_width, dtype, "v"),
        0 if q_weight is None else q_weight.data_ptr(), 0 if k_weight is None else k_weight.data_ptr(),
        rope.data_ptr() if plan.rot_dim else 0, rope.shape[0] if plan.rot_dim else 0, lengths.data_ptr(),
        0 if positions is None else positions.data_ptr(), page_table.data_ptr(), out.data_ptr(),
        _rows(out, tokens, plan.q_width, _BF16, "out"), seqs, rows, QMM_IN_F32 if dtype is _F32 else QMM_IN_BF16)
    st = _LIB.qmm_qk_norm_rope(plan._handle, cache.ref, args, _stream_on(stream, plan._device_index))
    if st != QMM_OK:
        raise QmmError(st, "qmm_qk_norm_rope")


def attention(plan: KVPlan, q, cache: KVCache, page_table, lengths, out, stream=None) -> None:
    """Attention of the new tokens over the cache (qmm_attention): q and out [tokens, q_heads, head_dim] bfloat16 (or
    [tokens, q_heads * head_dim]), tokens = seqs * rows with 1 to max_rows rows for each sequence."""
    tokens = q.shape[0]
    seqs, rows = _check_step(plan, cache, page_table, lengths, tokens, q, out)
    args = _ATTENTION_ARGS.pack(q.data_ptr(), out.data_ptr(), lengths.data_ptr(), page_table.data_ptr(),
                                _rows(q, tokens, plan.q_width, _BF16, "q"), _rows(out, tokens, plan.q_width, _BF16, "out"),
                                seqs, rows)
    st = _LIB.qmm_attention(plan._handle, cache.ref, args, _stream_on(stream, plan._device_index))
    if st != QMM_OK:
        raise QmmError(st, "qmm_attention")


def sample(logits, temperature, top_k, top_p, min_p, u, tokens, probs=None, stream=None) -> None:
    """Draw a token for each row of logits [M, vocab] (float32 or bfloat16, rows of any stride) from the uniform
    numbers u (qmm_sample): tokens int32 [M], probs float32 [M] or None. temperature, top_p, min_p: float32 [M];
    top_k: int32 [M]."""
    if _F32 is None:
        _bind_torch()
    f32, i32, dtype = _F32, _I32, logits.dtype
    shape, strides = logits.shape, logits.stride()
    if len(shape) != 2 or (dtype is not f32 and dtype is not _BF16) or strides[1] != 1:
        raise ValueError("logits are float32 or bfloat16 rows of adjacent elements")
    M, device = shape[0], logits.get_device()
    for t, want in ((temperature, f32), (top_k, i32), (top_p, f32), (min_p, f32), (u, f32), (tokens, i32)):
        if t.dtype is not want or t.numel() != M or not t.is_contiguous():
            raise ValueError("temperature, top_p, min_p and u are float32 [M], top_k and tokens int32 [M]")
        if t.get_device() != device:
            raise ValueError("all tensors are on the device of the logits")
    if probs is not None and (probs.dtype is not f32 or probs.numel() != M or not probs.is_contiguous() or
                              probs.get_device() != device):
        raise ValueError("probs is float32 [M] on the device of the logits, or None")
    if device < 0:
        raise ValueError("logits are on a CUDA device")
    args = (logits.data_ptr(), M, shape[1], strides[0], QMM_IN_F32 if dtype is f32 else QMM_IN_BF16,
            temperature.data_ptr(), top_k.data_ptr(), top_p.data_ptr(), min_p.data_ptr(), u.data_ptr(),
            tokens.data_ptr(), None if probs is None else probs.data_ptr(), _stream_on(stream, device))
    if device == _CURRENT_DEVICE():
        st = _lib().qmm_sample(*args)
    else:
        import torch
        with torch.cuda.device(device):   # the library launches on the current one
            st = _lib().qmm_sample(*args)
    if st != QMM_OK:
        raise QmmError(st, "qmm_sample")
