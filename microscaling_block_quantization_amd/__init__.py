"""Python binding of libmx.so, the gfx950 microscaling block-quantization library.

Argument marshalling only: the functions below take torch tensors (device
memory and streams come from PyTorch), pass raw pointers through the C ABI of
``include/mx.h`` and return.  Every step of quantization, dequantization, the
QSNR reduction and the block-scaled GEMM runs in the library's HIP kernels.
There is no fallback: if ``libmx.so`` is missing or fails to load, importing
the entry points raises.

The method (cited by page title and section): MXFP4 = E2M1 elements + one
E8M0 scale per 32; NVFP4 = E2M1 + E4M3 per 16 + an fp32 per-tensor scale
("Unveiling the Potential of Quantization with MXFP4", Sec. 2); QSNR eq. (1),
(2) (same page, Sec. 3); OAS and Macro Block Scaling (Sec. 4); UE5M3 scales
("Is Finer Better?", technical summary); block Hadamard rotation ("Bridging
the Gap ... Microscaling FP4 Quantization", Sec. 2.2); INT4 / E3M0 elements,
RTNE / stochastic / ceil rounding, asymmetric scaling and row / column / 2D
blocks (ARITH 2025 MX-training report, main results).
"""
import ctypes
import os
import struct
from dataclasses import dataclass, field

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmx.so")

MX_OK, MX_ERR_ARG, MX_ERR_UNSUPPORTED, MX_ERR_ALIGN, MX_ERR_WORKSPACE, MX_ERR_HIP, MX_ERR_TOO_LARGE = range(7)
NOALLOC_SCRATCH_BYTES = 4 << 20      # MX_NOALLOC_SCRATCH_BYTES of include/mx.h
ELEM_E2M1, ELEM_INT4, ELEM_FP6_E2M3, ELEM_FP6_E3M2, ELEM_E3M0, ELEM_FP8_E4M3, ELEM_FP8_E5M2 = range(7)
SCALE_E8M0, SCALE_UE4M3, SCALE_NVFP4, SCALE_UE5M3, SCALE_E3M0 = range(5)
RULE_FLOOR, RULE_CEIL, RULE_OAS = range(3)
ROUND_RTNE, ROUND_SR, ROUND_CEIL = range(3)
DTYPE_F32, DTYPE_BF16 = range(2)

EXPORTS = ["mx_query_sizes", "mx_quantize", "mx_quantize_noalloc", "mx_quantize_many", "mx_dequantize",
           "mx_qsnr_workspace_size", "mx_qsnr", "mx_gemm", "mx_matvec", "mx_qk_rope",
           "mx_qk_rope_workspace_size", "mx_qk_rope_backward", "mx_cache_write", "mx_attend_workspace_size",
           "mx_attend", "mx_status_string"]


class MxFormat(ctypes.Structure):
    _fields_ = [("elem", ctypes.c_int32), ("scale", ctypes.c_int32), ("rule", ctypes.c_int32),
                ("round", ctypes.c_int32), ("block_rows", ctypes.c_int32),
                ("block_cols", ctypes.c_int32), ("asymmetric", ctypes.c_int32),
                ("hadamard", ctypes.c_int32), ("macro_cols", ctypes.c_int32),
                ("oas_tau", ctypes.c_float), ("seed", ctypes.c_uint64),
                ("rng_offset", ctypes.c_uint64)]


class MxQTensor(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("macro_scales", ctypes.c_void_p),
                ("tensor_scale", ctypes.c_void_p), ("ref_exp", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class MxStats(ctypes.Structure):
    _fields_ = [("sig2", ctypes.c_double), ("err2", ctypes.c_double), ("n", ctypes.c_int64),
                ("nonzero", ctypes.c_int64), ("flushed", ctypes.c_int64),
                ("zero_blocks", ctypes.c_int64)]


class MxQJob(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("out", ctypes.POINTER(MxQTensor)), ("stats", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t)]


class MxSizes(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_size_t), ("scales", ctypes.c_size_t),
                ("offsets", ctypes.c_size_t), ("macro_scales", ctypes.c_size_t),
                ("tensor_scale", ctypes.c_size_t), ("ref_exp", ctypes.c_size_t),
                ("workspace", ctypes.c_size_t)]


class MxHeads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class MxRope(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p),
                ("table_rows", ctypes.c_int64), ("positions", ctypes.c_void_p), ("eps", ctypes.c_float)]


class MxKVCache(ctypes.Structure):
    _fields_ = [("format", ctypes.POINTER(MxFormat)), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32)]


class MxError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {mx_status_string(status)} (status {status})")


_lib = None


def lib():
    """Load libmx.so.  Raises if it has not been built: there is no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "python microscaling_block_quantization_amd/build.py")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        P = ctypes.POINTER
        L.mx_query_sizes.argtypes = [P(MxFormat), i64, i64, P(MxSizes)]
        L.mx_quantize.argtypes = [P(MxFormat), i32, vp, i64, i64, i64, P(MxQTensor), vp, i32, vp,
                                  vp, ctypes.c_size_t, vp]
        L.mx_quantize_noalloc.argtypes = [P(MxFormat), i32, vp, i64, i64, i64, P(MxQTensor), vp, i32, vp, vp]
        L.mx_quantize_many.argtypes = [P(MxFormat), i32, P(MxQJob), i32, vp]
        L.mx_dequantize.argtypes = [P(MxFormat), P(MxQTensor), i32, vp, i64, vp]
        L.mx_qsnr_workspace_size.argtypes = [i64]
        L.mx_qsnr_workspace_size.restype = ctypes.c_size_t
        L.mx_qsnr.argtypes = [i32, vp, vp, i64, P(MxStats), P(ctypes.c_double), vp,
                              ctypes.c_size_t, vp]
        L.mx_gemm.argtypes = [P(MxFormat), P(MxQTensor), P(MxFormat), P(MxQTensor), vp, i64, i32, vp]
        # structs of these calls are passed as packed bytes or by reference
        sz = ctypes.c_size_t
        L.mx_matvec.argtypes = [vp, vp, i32, vp, i64, i64, vp, vp, i64, i32, vp]
        L.mx_qk_rope.argtypes = [vp] * 6
        L.mx_qk_rope_workspace_size.argtypes = [vp]
        L.mx_qk_rope_workspace_size.restype = sz
        L.mx_qk_rope_backward.argtypes = [vp] * 10 + [sz, vp]
        L.mx_cache_write.argtypes = [vp, vp, vp, i64, vp, vp]
        L.mx_attend_workspace_size.argtypes = [vp, i64, ctypes.c_int32, i64]
        L.mx_attend_workspace_size.restype = sz
        L.mx_attend.argtypes = [vp, vp, i64, vp, i64, i64, vp, ctypes.c_float, vp, vp, vp, sz, vp]
        L.mx_status_string.argtypes = [i32]
        L.mx_status_string.restype = ctypes.c_char_p
        for name in ("mx_query_sizes", "mx_quantize", "mx_quantize_noalloc", "mx_quantize_many",
                     "mx_dequantize", "mx_qsnr", "mx_gemm", "mx_matvec", "mx_qk_rope", "mx_qk_rope_backward",
                     "mx_cache_write", "mx_attend"):
            getattr(L, name).restype = ctypes.c_int
        _lib = L
    return _lib


def mx_status_string(status):
    return lib().mx_status_string(int(status)).decode()


@dataclass
class Format:
    elem: int = ELEM_E2M1
    scale: int = SCALE_E8M0
    rule: int = RULE_FLOOR
    round: int = ROUND_RTNE
    block_rows: int = 1
    block_cols: int = 32
    asymmetric: int = 0
    hadamard: int = 0
    macro_cols: int = 0
    oas_tau: float = 0.0
    seed: int = 0
    rng_offset: int = 0

    def c(self):
        return MxFormat(self.elem, self.scale, self.rule, self.round, self.block_rows,
                        self.block_cols, self.asymmetric, self.hadamard, self.macro_cols,
                        self.oas_tau, self.seed, self.rng_offset)


MXFP4 = Format()
MXFP6_E2M3 = Format(elem=ELEM_FP6_E2M3)
MXFP6_E3M2 = Format(elem=ELEM_FP6_E3M2)
MXFP8_E4M3 = Format(elem=ELEM_FP8_E4M3)
MXFP8_E5M2 = Format(elem=ELEM_FP8_E5M2)


@dataclass
class QTensor:
    """A quantized tensor: device buffers laid out as include/mx.h describes."""
    rows: int
    cols: int
    codes: torch.Tensor
    scales: torch.Tensor
    offsets: torch.Tensor = None
    macro_scales: torch.Tensor = None
    tensor_scale: torch.Tensor = None
    ref_exp: torch.Tensor = None
    _keep: list = field(default_factory=list)

    def c(self):
        p = lambda t: None if t is None else t.data_ptr()
        return MxQTensor(p(self.codes), p(self.scales), p(self.offsets), p(self.macro_scales),
                         p(self.tensor_scale), p(self.ref_exp), self.rows, self.cols)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _on(stream, call, *args):
    """call(*args) with `stream` as the current stream, so that what the call
    allocates belongs to the stream its kernels run on: a workspace freed at
    the return, and an output, are given out again in that stream's order.  The
    outputs' use on the caller's stream is recorded."""
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = call(*args)
    if stream != caller:
        _record(out, caller)
    return out


def _record(out, stream):
    if isinstance(out, torch.Tensor):
        out.record_stream(stream)
    elif isinstance(out, QTensor):
        _record((out.codes, out.scales, out.offsets, out.macro_scales, out.tensor_scale, out.ref_exp), stream)
    elif isinstance(out, (tuple, list)):
        for o in out:
            _record(o, stream)


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(rc, where):
    if rc != MX_OK:
        raise MxError(rc, where)


def _dtype_code(t):
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _empty(nbytes, device):
    # 16-byte aligned: the caching allocator hands out 512-byte aligned blocks
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def mx_query_sizes(fmt: Format, rows, cols):
    s = MxSizes()
    f = fmt.c()
    _check(lib().mx_query_sizes(ctypes.byref(f), rows, cols, ctypes.byref(s)), "mx_query_sizes")
    return {k: getattr(s, k) for k, _ in MxSizes._fields_}


def alloc_qtensor(fmt: Format, rows, cols, device="cuda"):
    s = mx_query_sizes(fmt, rows, cols)
    q = QTensor(rows, cols, _empty(s["codes"], device), _empty(s["scales"], device))
    if s["offsets"]:
        q.offsets = torch.empty(s["offsets"] // 2, dtype=torch.int16, device=device)
    if s["macro_scales"]:
        q.macro_scales = _empty(s["macro_scales"], device)
    if s["tensor_scale"]:
        q.tensor_scale = torch.empty(1, dtype=torch.float32, device=device)
    if s["ref_exp"]:
        q.ref_exp = torch.empty(1, dtype=torch.int32, device=device)
    return q


def alloc_workspace(fmt: Format, rows, cols, device="cuda"):
    return _empty(mx_query_sizes(fmt, rows, cols)["workspace"], device)


def stats_to_dict(t):
    """Read a device mx_stats (48 bytes) into a dict."""
    raw = t.detach().to("cpu").numpy().tobytes()[:ctypes.sizeof(MxStats)]
    st = MxStats.from_buffer_copy(raw)
    return {k: getattr(st, k) for k, _ in MxStats._fields_}


def mx_quantize(fmt: Format, x: torch.Tensor, out: QTensor = None, dequant=None, stats=None,
                workspace=None, stream=None):
    """Quantize a 2-D fp32 / bf16 device tensor.

    dequant: None, a dtype (torch.float32 / torch.bfloat16) to allocate, or a tensor.
    stats: None, True (allocate), or a 48-byte device uint8 tensor.
    Returns (qtensor, dequant tensor or None, stats tensor or None)."""
    if stream is not None:
        return _on(stream, mx_quantize, fmt, x, out, dequant, stats, workspace)
    assert x.dim() == 2 and x.is_cuda
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    assert x.stride(1) == 1
    if out is None:
        out = alloc_qtensor(fmt, rows, cols, x.device)
    if isinstance(dequant, torch.dtype):
        dequant = torch.empty((rows, cols), dtype=dequant, device=x.device)
    if stats is True:
        stats = _empty(ctypes.sizeof(MxStats), x.device)
    need_ws = stats is not None or fmt.scale in (SCALE_NVFP4, SCALE_E3M0)
    if workspace is None and need_ws:
        workspace = alloc_workspace(fmt, rows, cols, x.device)
    f = fmt.c()
    q = out.c()
    rc = lib().mx_quantize(ctypes.byref(f), _dtype_code(x), _ptr(x), rows, cols, ld, ctypes.byref(q),
                           _ptr(dequant), DTYPE_F32 if dequant is None else _dtype_code(dequant),
                           _ptr(stats), _ptr(workspace),
                           0 if workspace is None else workspace.numel(), _stream())
    _check(rc, "mx_quantize")
    return out, dequant, stats


def mx_quantize_noalloc(fmt: Format, x: torch.Tensor, out: QTensor, dequant=None, stats=None, stream=None):
    """mx_quantize without a workspace: the library's static scratch array on
    this GPU holds what its kernels need beyond the outputs (at most
    NOALLOC_SCRATCH_BYTES; larger calls raise MxError MX_ERR_TOO_LARGE).  The
    outputs are the caller's: `out` (a QTensor), `dequant` (None or a tensor)
    and `stats` (None or a 48-byte device tensor).  Calls that overlap on one
    GPU share the array and race."""
    if stream is not None:
        return _on(stream, mx_quantize_noalloc, fmt, x, out, dequant, stats)
    assert x.dim() == 2 and x.is_cuda and x.stride(1) == 1
    rows, cols = x.shape
    ld = x.stride(0) if rows > 1 else cols
    f = fmt.c()
    q = out.c()
    rc = lib().mx_quantize_noalloc(ctypes.byref(f), _dtype_code(x), _ptr(x), rows, cols, ld, ctypes.byref(q),
                                   _ptr(dequant), DTYPE_F32 if dequant is None else _dtype_code(dequant),
                                   _ptr(stats), _stream())
    _check(rc, "mx_quantize_noalloc")
    return out, dequant, stats


def mx_quantize_many(fmt: Format, xs, outs=None, stats=None, workspaces=None, stream=None):
    """Quantize several 2-D device tensors of one dtype in one format (one
    call of mx_quantize_many).  outs: None or a list of QTensors; stats: None,
    True (allocate one per tensor) or a list of 48-byte device tensors (or
    None entries); workspaces: None (allocated where needed) or a list.
    Returns (list of qtensors, list of stats tensors or None)."""
    if stream is not None:
        return _on(stream, mx_quantize_many, fmt, xs, outs, stats, workspaces)
    xs = list(xs)
    n = len(xs)
    outs = [None] * n if outs is None else list(outs)
    if stats is True:
        stats = [_empty(ctypes.sizeof(MxStats), x.device) for x in xs]
    stats = [None] * n if stats is None else list(stats)
    workspaces = [None] * n if workspaces is None else list(workspaces)
    assert len(outs) == n and len(stats) == n and len(workspaces) == n
    dt = _dtype_code(xs[0]) if n else DTYPE_BF16
    keep = []
    jobs = (MxQJob * max(n, 1))()
    for i, x in enumerate(xs):
        assert x.dim() == 2 and x.is_cuda and _dtype_code(x) == dt
        assert x.numel() == 0 or x.stride(1) == 1
        rows, cols = x.shape
        if outs[i] is None:
            outs[i] = alloc_qtensor(fmt, rows, cols, x.device)
        if workspaces[i] is None and (stats[i] is not None or fmt.scale in (SCALE_NVFP4, SCALE_E3M0)):
            workspaces[i] = alloc_workspace(fmt, rows, cols, x.device)
        q = outs[i].c()
        keep.append(q)
        ws = workspaces[i]
        jobs[i] = MxQJob(x.data_ptr(), rows, cols, x.stride(0) if rows > 1 and x.numel() else cols,
                         ctypes.pointer(q),
                         None if stats[i] is None else stats[i].data_ptr(),
                         None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel())
    f = fmt.c()
    rc = lib().mx_quantize_many(ctypes.byref(f), dt, jobs, n, _stream())
    _check(rc, "mx_quantize_many")
    return outs, stats


def mx_dequantize(fmt: Format, q: QTensor, out_dtype=torch.float32, y=None, stream=None):
    if stream is not None:
        return _on(stream, mx_dequantize, fmt, q, out_dtype, y)
    if y is None:
        y = torch.empty((q.rows, q.cols), dtype=out_dtype, device=q.codes.device)
    f = fmt.c()
    qc = q.c()
    ld = y.stride(0) if q.rows > 1 else q.cols
    rc = lib().mx_dequantize(ctypes.byref(f), ctypes.byref(qc), _dtype_code(y), _ptr(y), ld, _stream())
    _check(rc, "mx_dequantize")
    return y


def mx_qsnr_workspace_size(n):
    return int(lib().mx_qsnr_workspace_size(int(n)))


def mx_qsnr(ref: torch.Tensor, approx: torch.Tensor, workspace=None, stream=None):
    """QSNR (dB) of eq. (1)/(2) between two device tensors; returns (stats, dB)."""
    if stream is not None:
        return _on(stream, mx_qsnr, ref, approx, workspace)
    assert ref.dtype == approx.dtype and ref.numel() == approx.numel()
    assert ref.is_contiguous() and approx.is_contiguous()
    n = ref.numel()
    if workspace is None:
        workspace = _empty(mx_qsnr_workspace_size(n), ref.device)
    st = MxStats()
    d = ctypes.c_double()
    rc = lib().mx_qsnr(_dtype_code(ref), _ptr(ref), _ptr(approx), n, ctypes.byref(st), ctypes.byref(d),
                       _ptr(workspace), workspace.numel(), _stream())
    _check(rc, "mx_qsnr")
    return {k: getattr(st, k) for k, _ in MxStats._fields_}, d.value


def mx_gemm(fa: Format, a: QTensor, fb: Format, b: QTensor, c=None, out_dtype=torch.bfloat16, stream=None):
    """C = deq(A) . deq(B)^T for A (M x K) and B (N x K): MXFP4, MXFP6 (E2M3 /
    E3M2) or MXFP8 (E4M3 / E5M2) with E8M0 scales per 1 x 32 block, in any pairing (MXFP4 operands may
    carry 1 x 128 macro-block scales, macro_cols=128); or E2M1 under UE4M3,
    NVFP4, UE5M3 or E8M0 scales on other row blocks.  c: an M x N view (any
    row stride) to write into, else a new tensor of out_dtype."""
    if stream is not None:
        return _on(stream, mx_gemm, fa, a, fb, b, c, out_dtype)
    if c is None:
        c = torch.empty((a.rows, b.rows), dtype=out_dtype, device=a.codes.device)
    ldc = c.stride(0) if a.rows > 1 else b.rows
    f1, f2 = fa.c(), fb.c()
    qa, qb = a.c(), b.c()
    rc = lib().mx_gemm(ctypes.byref(f1), ctypes.byref(qa), ctypes.byref(f2), ctypes.byref(qb), _ptr(c), ldc,
                       _dtype_code(c), _stream())
    _check(rc, "mx_gemm")
    return c


# ---- one decode step with quantized weights and a quantized cache ------------
# These kernels take a few microseconds, so the host's share of a call counts:
# each check is one cheap comparison whose message is only formed when it
# fails, and structs are packed as bytes.  `stream`: the stream to launch on
# (default: the current one), see _on.  The calls record nothing for autograd
# (mx_qk_rope_backward is the gradient to put into a Function).
_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
_PACK_FORMAT = struct.Struct("@9if2Q").pack
_PACK_QTENSOR = struct.Struct("@6P2q").pack
_PACK_HEADS = struct.Struct("@Pqqii").pack
_PACK_ROPE = struct.Struct("@q4i4PqPf4x").pack


def _code(dtype):
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _stream_ptr(dev, where):
    """The current stream, for a launch whose operands lie on device `dev`:
    kernels run on the current device."""
    if dev < 0:
        raise ValueError(f"{where}: the operands must be GPU tensors")
    if torch._C._cuda_getDevice() != dev:
        raise ValueError(f"{where}: the operands lie on device {dev}, the call (or its stream) runs on {torch._C._cuda_getDevice()}")
    return torch._C._cuda_getCurrentRawStream(dev)


def _raw(t):
    return 0 if t is None else t.data_ptr()


def _changed(*ts):
    """Tensors of the caller's that a launch writes into: autograd's count of
    their changes goes up, as torch's own in-place operations do."""
    torch._C._increment_version([t for t in ts if t is not None and not t.is_inference()])


def _heads(t, dim, dev, what):
    """The mx_heads of a tokens x heads x dim tensor whose last dimension is contiguous."""
    sh, st = t.shape, t.stride()
    if len(sh) != 3 or sh[2] != dim or st[2] != 1 or t.get_device() != dev:
        raise ValueError(f"{what}: expected tokens x heads x {dim} on one device, the last dimension contiguous")
    return _PACK_HEADS(t.data_ptr(), st[0], st[1], sh[1], _code(t.dtype))


def _vector(t, n, dtype, dev, where, name):
    """The address of n contiguous values (of dtype, unless None)."""
    if t.shape != (n,) or not t.is_contiguous() or t.get_device() != dev or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{where}: {name} must be {n} contiguous values{'' if dtype is None else f' of {dtype}'} on the inputs' device")
    return t.data_ptr()


def _buffer(t, nbytes, dev, where, name):
    """The address of a caller's buffer of at least nbytes."""
    if t.nbytes < nbytes or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be {nbytes} contiguous bytes at least, on the inputs' device")
    return t.data_ptr()


def mx_matvec(fmt: Format, w: QTensor, x: torch.Tensor, bias=None, y=None, out_dtype=None, stream=None):
    """y = x . deq(W)^T + bias for a few unquantized tokens x (tokens x K, bf16
    or fp32, any row stride) and a 4-bit weight W (N x K: E2M1 or INT4 in row
    blocks, see include/mx.h).  bias: None or N values of x's dtype.  y: a
    tokens x N view to write into, else a new tensor of out_dtype (default: x's)."""
    if stream is not None:
        return _on(stream, mx_matvec, fmt, w, x, bias, y, out_dtype)
    n, k, codes, scales, dev, shape = w.rows, w.cols, w.codes, w.scales, x.get_device(), x.shape
    if len(shape) != 2 or shape[1] != k or codes.get_device() != dev:
        raise ValueError(f"mx_matvec: x must be tokens x {k} on the weight's device")
    tokens = shape[0]
    ldx, last = x.stride()
    if last != 1 and k > 1 and tokens:
        raise ValueError("mx_matvec: the rows of x must be contiguous")
    bp = 0 if bias is None else _vector(bias, n, x.dtype, dev, "mx_matvec", "bias")
    given = y is not None
    if not given:
        y = x.new_empty((tokens, n)) if out_dtype is None or out_dtype is x.dtype else x.new_empty((tokens, n), dtype=out_dtype)
        ldy = n
    else:
        if y.shape != (tokens, n) or (y.stride(1) != 1 and n > 1 and tokens) or y.get_device() != dev:
            raise ValueError(f"mx_matvec: y must be {tokens} x {n} with contiguous rows")
        ldy = y.stride(0)
    if tokens <= 1:
        ldx, ldy = k, n
    # row blocks of 4-bit codes: any other format is the library's to refuse
    bc, asym, offsets, macro, ts = fmt.block_cols, fmt.asymmetric, w.offsets, w.macro_scales, w.tensor_scale
    held = n * k if bc > 0 and fmt.block_rows == 1 and fmt.elem in (ELEM_E2M1, ELEM_INT4) else 0
    blocks = held // (bc or 1)
    if (codes.nbytes < held // 2 or scales.nbytes < blocks or scales.get_device() != dev or not codes.is_contiguous() or
            not scales.is_contiguous()):
        _buffer(codes, held // 2, dev, "mx_matvec", "codes")
        _buffer(scales, blocks, dev, "mx_matvec", "scales")
    if offsets is not None:
        if offsets.get_device() != dev or not offsets.is_contiguous() or (asym and offsets.nbytes < 2 * blocks):
            _buffer(offsets, 2 * blocks if asym else 0, dev, "mx_matvec", "offsets")
        offsets = offsets.data_ptr()
    if macro is not None:
        macro = _buffer(macro, held // 128 if fmt.macro_cols else 0, dev, "mx_matvec", "macro_scales")
    if ts is not None:
        if ts.dtype is not torch.float32:
            raise ValueError("mx_matvec: tensor_scale must be fp32")
        ts = _buffer(ts, 4, dev, "mx_matvec", "tensor_scale")
    f = _PACK_FORMAT(fmt.elem, fmt.scale, fmt.rule, fmt.round, fmt.block_rows, bc, asym, fmt.hadamard, fmt.macro_cols, fmt.oas_tau,
                     fmt.seed, fmt.rng_offset)
    q = _PACK_QTENSOR(codes.data_ptr(), scales.data_ptr(), offsets or 0, macro or 0, ts or 0, 0, n, k)
    _check(lib().mx_matvec(f, q, _code(x.dtype), x.data_ptr(), tokens, ldx, bp, y.data_ptr(), ldy, _code(y.dtype),
                           _stream_ptr(dev, "mx_matvec")), "mx_matvec")
    if given:
        _changed(y)
    return y


def _rope_args(q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved, where):
    """The mx_rope of a call, its shapes checked."""
    tokens, _, dim = q.shape
    dev = q.get_device()
    if (cos.dim() != 2 or cos.shape != sin.shape or cos.dtype != torch.float32 or sin.dtype != torch.float32 or
            not cos.is_contiguous() or not sin.is_contiguous() or cos.get_device() != dev or sin.get_device() != dev):
        raise ValueError(f"{where}: cos and sin must be contiguous fp32 tables of positions x rot_dim/2")
    rows, half = cos.shape
    pos = _vector(positions, tokens, torch.int32, dev, where, "positions")
    wd = DTYPE_F32
    qp = kp = 0
    if q_weight is not None:
        qp, wd = _vector(q_weight, dim, None, dev, where, "q_weight"), _code(q_weight.dtype)
    if k_weight is not None:
        if k is None or (q_weight is not None and q_weight.dtype != k_weight.dtype):
            raise ValueError(f"{where}: k_weight needs k, and the dtype of q_weight")
        kp, wd = _vector(k_weight, dim, None, dev, where, "k_weight"), _code(k_weight.dtype)
    if k is not None and k.size(0) != tokens:
        raise ValueError(f"{where}: q and k differ in tokens")
    return _PACK_ROPE(tokens, dim, 2 * half, 1 if interleaved else 0, wd, qp, kp, cos.data_ptr(), sin.data_ptr(), rows, pos, eps)


def _out_heads(out, like, dim, dev, what):
    """An output of `like`'s shape (a new tensor when None) and its mx_heads."""
    if out is None:
        out = torch.empty_like(like, memory_format=torch.contiguous_format)
        n = like.size(1)
        return out, _PACK_HEADS(out.data_ptr(), n * dim, dim, n, _DTYPES[like.dtype])
    if out.shape != like.shape:
        raise ValueError(f"{what}: expected the shape {tuple(like.shape)}")
    return out, _heads(out, dim, dev, what)


def mx_qk_rope(q, k, cos, sin, positions, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None,
               k_out=None, stream=None):
    """RMS norm (where a weight is given) and rotation of query and key heads
    in one pass.  q, k: tokens x heads x dim, bf16 or fp32, any token and head
    strides (views of a fused projection); k may be None.  cos, sin: fp32
    tables of positions x rot_dim/2; positions: int32 per token.  interleaved:
    pairs (2i, 2i+1) instead of (i, i + rot_dim/2).  q_out, k_out: tensors to
    write into (q and k themselves included), else new ones.
    Returns (q_out, k_out)."""
    if stream is not None:
        return _on(stream, mx_qk_rope, q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved, q_out, k_out)
    if q.dim() != 3:
        raise ValueError("mx_qk_rope: q must be tokens x heads x dim")
    dev, dim, given = q.get_device(), q.size(2), (q_out, k_out)
    r = _rope_args(q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved, "mx_qk_rope")
    hq = _heads(q, dim, dev, "mx_qk_rope: q")
    q_out, oq = _out_heads(q_out, q, dim, dev, "mx_qk_rope: q_out")
    hk = ok = None
    if k is not None:
        hk = _heads(k, dim, dev, "mx_qk_rope: k")
        k_out, ok = _out_heads(k_out, k, dim, dev, "mx_qk_rope: k_out")
    _check(lib().mx_qk_rope(r, hq, hk, oq, ok, _stream_ptr(dev, "mx_qk_rope")), "mx_qk_rope")
    if given[0] is not None or given[1] is not None:
        _changed(*given)
    return q_out, k_out


def mx_qk_rope_workspace_size(tokens, dim, rot_dim, weights=True):
    """Workspace bytes of mx_qk_rope_backward (0 without norm weights)."""
    a = 256 if weights else 0                  # any aligned address: only whether it is set counts here
    r = _PACK_ROPE(tokens, dim, rot_dim, 0, DTYPE_F32, a, a, 256, 256, 1, 256, 0.0)
    return int(lib().mx_qk_rope_workspace_size(r))


def mx_qk_rope_backward(dy_q, dy_k, q, k, cos, sin, positions, q_weight=None, k_weight=None, eps=1e-6,
                        interleaved=False, dq=None, dk=None, workspace=None, stream=None):
    """Gradient of mx_qk_rope: dy_q, dy_k are the gradients of its outputs, the
    rest are its arguments.  Returns (dq, dk, dq_weight, dk_weight); the weight
    gradients are fp32 (None without that weight).  dq, dk may be dy_q, dy_k."""
    if stream is not None:
        return _on(stream, mx_qk_rope_backward, dy_q, dy_k, q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved, dq, dk,
                   workspace)
    if q.dim() != 3 or (k is None) != (dy_k is None):
        raise ValueError("mx_qk_rope_backward: q must be tokens x heads x dim, and dy_k and k go together")
    dev, dim, given = q.get_device(), q.size(2), (dq, dk)
    r = _rope_args(q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved, "mx_qk_rope_backward")
    if dy_q.shape != q.shape or (k is not None and dy_k.shape != k.shape):
        raise ValueError("mx_qk_rope_backward: gradients must have their heads' shape")
    gq, xq = _heads(dy_q, dim, dev, "mx_qk_rope_backward: dy_q"), _heads(q, dim, dev, "mx_qk_rope_backward: q")
    dq, oq = _out_heads(dq, q, dim, dev, "mx_qk_rope_backward: dq")
    gk = xk = ok = None
    if k is not None:
        gk, xk = _heads(dy_k, dim, dev, "mx_qk_rope_backward: dy_k"), _heads(k, dim, dev, "mx_qk_rope_backward: k")
        dk, ok = _out_heads(dk, k, dim, dev, "mx_qk_rope_backward: dk")
    dqw = None if q_weight is None else cos.new_empty((dim,))
    dkw = None if k_weight is None else cos.new_empty((dim,))
    if workspace is not None:
        _buffer(workspace, 0, dev, "mx_qk_rope_backward", "workspace")
    elif dqw is not None or dkw is not None:
        workspace = cos.new_empty((lib().mx_qk_rope_workspace_size(r),), dtype=torch.uint8)
    _check(lib().mx_qk_rope_backward(r, gq, gk, xq, xk, oq, ok, _raw(dqw), _raw(dkw), _raw(workspace),
                                     0 if workspace is None else workspace.nbytes, _stream_ptr(dev, "mx_qk_rope_backward")),
           "mx_qk_rope_backward")
    if given[0] is not None or given[1] is not None:
        _changed(*given)
    return dq, dk, dqw, dkw


@dataclass(frozen=True, eq=False)
class KVCache:
    """A paged cache of keys and values.  fmt None: k and v are bf16, pages x
    heads x page_size x dim.  fmt MXFP8_E4M3 or MXFP4: uint8 codes, pages x
    heads x page_size x (dim or dim/2), with uint8 E8M0 scales pages x heads x
    page_size x dim/32.  Fixed once made: its C struct is packed here."""
    fmt: Format
    k: torch.Tensor
    v: torch.Tensor
    k_scales: torch.Tensor = None
    v_scales: torch.Tensor = None

    def __post_init__(self):
        bits = 16 if self.fmt is None else {ELEM_FP8_E4M3: 8, ELEM_E2M1: 4}.get(self.fmt.elem)
        if bits is None:
            raise ValueError("KVCache: the format must have E4M3 or E2M1 elements")
        if self.k.dim() != 4:
            raise ValueError("KVCache: k must be pages x heads x page_size x dim")
        put = lambda name, v: object.__setattr__(self, name, v)
        pages, heads, page_size, last = self.k.shape
        dim = last * 2 if bits == 4 else last
        dtype = torch.bfloat16 if self.fmt is None else torch.uint8
        need = [(self.k, self.k.shape, dtype), (self.v, self.k.shape, dtype)]
        if self.fmt is not None:
            grid = (pages, heads, page_size, dim // 32)
            need += [(self.k_scales, grid, torch.uint8), (self.v_scales, grid, torch.uint8)]
        for t, shape, dt in need:
            if t is None or t.shape != shape or t.dtype != dt or not t.is_contiguous() or t.get_device() != self.k.get_device():
                raise ValueError(f"KVCache: expected a contiguous {dt} buffer of {tuple(shape)}")
        for name, v in (("pages", pages), ("heads", heads), ("page_size", page_size), ("dim", dim)):
            put(name, v)
        f = None if self.fmt is None else self.fmt.c()
        put("_format", f)
        c = MxKVCache(None if f is None else ctypes.pointer(f), self.k.data_ptr(), self.v.data_ptr(),
                      None if f is None else self.k_scales.data_ptr(), None if f is None else self.v_scales.data_ptr(), pages,
                      page_size, heads, dim)
        put("_c", c)
        put("_ref", ctypes.byref(c))

    def c(self):
        return self._c


def alloc_kv_cache(fmt, pages, page_size, heads, dim, device="cuda"):
    """A KVCache of zeros: fmt None (bf16), MXFP8_E4M3 or MXFP4."""
    z = lambda last, dtype: torch.zeros((pages, heads, page_size, last), dtype=dtype, device=device)
    if fmt is None:
        return KVCache(None, z(dim, torch.bfloat16), z(dim, torch.bfloat16))
    last = dim // 2 if fmt.elem == ELEM_E2M1 else dim
    return KVCache(fmt, z(last, torch.uint8), z(last, torch.uint8), z(dim // 32, torch.uint8), z(dim // 32, torch.uint8))


def mx_cache_write(cache: KVCache, k, v, slots, stream=None):
    """Write the keys and values of new tokens (tokens x heads x dim, bf16 or
    fp32, any token and head strides) to the cache, quantized to its format.
    slots: int64 per token, page * page_size + position in the page; a slot
    outside the cache skips its token.  Returns the cache."""
    if stream is not None:
        return _on(stream, mx_cache_write, cache, k, v, slots)
    dev, dim = cache.k.get_device(), cache.dim
    hk, hv = _heads(k, dim, dev, "mx_cache_write: k"), _heads(v, dim, dev, "mx_cache_write: v")
    tokens = k.size(0)
    if v.size(0) != tokens:
        raise ValueError("mx_cache_write: k and v differ in tokens")
    at = _vector(slots, tokens, torch.int64, dev, "mx_cache_write", "slots")
    _check(lib().mx_cache_write(cache._ref, hk, hv, tokens, at, _stream_ptr(dev, "mx_cache_write")), "mx_cache_write")
    return cache


def mx_attend_workspace_size(cache: KVCache, batch, q_heads, table_cols):
    """Workspace bytes of mx_attend for at most `batch` sequences of at most
    `table_cols` pages."""
    return int(lib().mx_attend_workspace_size(cache._ref, batch, q_heads, table_cols))


def alloc_attend_workspace(cache: KVCache, batch, q_heads, table_cols):
    """A workspace for calls of at most `batch` sequences of at most `table_cols` pages."""
    return _empty(mx_attend_workspace_size(cache, batch, q_heads, table_cols), cache.k.device)


def mx_attend(q, cache: KVCache, page_table, lengths, scale=None, out=None, lse=None, workspace=None, stream=None):
    """Attention of one new token per sequence over the paged cache.  q: batch x
    heads x dim (bf16 or fp32; heads a multiple of the cache's); page_table:
    int32, batch x columns (rows may be strided); lengths: int32 per sequence,
    0 allowed (out 0, lse -inf).  scale: default dim^-1/2.  lse: None, True
    (allocate) or a batch x heads fp32 tensor.  workspace: as
    alloc_attend_workspace gives (allocated when None).
    Returns out, or (out, lse) when lse is asked for."""
    if stream is not None:
        return _on(stream, mx_attend, q, cache, page_table, lengths, scale, out, lse, workspace)
    dev, dim = cache.k.get_device(), cache.dim
    hq = _heads(q, dim, dev, "mx_attend: q")
    batch, heads = q.size(0), q.size(1)
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.size(0) != batch or page_table.get_device() != dev:
        raise ValueError(f"mx_attend: page_table must be {batch} rows of int32 on the cache's device")
    cols = page_table.size(1)
    stride, last = page_table.stride()
    if last != 1 and cols > 1 and batch:
        raise ValueError("mx_attend: the rows of page_table must be contiguous")
    n = _vector(lengths, batch, torch.int32, dev, "mx_attend", "lengths")
    given = (out, None if lse is True else lse)
    out, ho = _out_heads(out, q, dim, dev, "mx_attend: out")
    if lse is True:
        lse = q.new_empty((batch, heads), dtype=torch.float32)
    elif lse is not None and (lse.shape != (batch, heads) or lse.dtype != torch.float32 or not lse.is_contiguous() or
                              lse.get_device() != dev):
        raise ValueError(f"mx_attend: lse must be a contiguous fp32 {batch} x {heads}")
    if workspace is None:
        workspace = cache.k.new_empty((lib().mx_attend_workspace_size(cache._ref, batch, heads, cols),), dtype=torch.uint8)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _buffer(workspace, 0, dev, "mx_attend", "workspace")
    _check(lib().mx_attend(cache._ref, hq, batch, page_table.data_ptr(), cols, cols if batch <= 1 else stride, n,
                           dim ** -0.5 if scale is None else scale, ho, _raw(lse), workspace.data_ptr(), workspace.nbytes,
                           _stream_ptr(dev, "mx_attend")), "mx_attend")
    if given[0] is not None or given[1] is not None:
        _changed(*given)
    return out if lse is None else (out, lse)
