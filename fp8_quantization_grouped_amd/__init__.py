"""MI355X (gfx950) MoE FP8 training hot path: fused FP8 quantization and scaled grouped GEMM.

Thin ctypes binding over the C ABI in ``include/fp8_quant_grouped.h`` (library
``libfp8qg.so`` next to this file, built by ``_build.build()``).  Each Python function has the
name of the C entry point it calls and only marshals arguments: it takes torch tensors for
device memory, allocates outputs with torch on the input's device, passes raw pointers and the
current HIP stream, and raises on a non-zero status.  Every step of the computation runs in
the HIP kernels; there is no fallback.  If the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfp8qg.so")

E4M3FNUZ = 0  # AMD e4m3fnuz: largest value 240
E4M3FN = 1    # OCP e4m3fn: largest value 448
FMAX = {E4M3FNUZ: 240.0, E4M3FN: 448.0}
GEMM_FWD_MGROUPED = 0
GEMM_WGRAD_KGROUPED = 1
OUT_BF16 = 0
OUT_FP32 = 1

_lib = None

# name -> (restype, argtypes)
_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
_I = ctypes.c_int
SIGNATURES = {
    "fp8q_abi_version": (_I, []),
    "fp8q_status_string": (ctypes.c_char_p, [_I]),
    "fp8_abi_version": (_I, []),
    "fp8_status_string": (ctypes.c_char_p, [_I]),
    "fp8_grouped_gemm_workspace_size": (_SZ, [_I, _I64, _I64, _I64, _I32]),
    "fp8_quant_rowwise": (_I, [_P, _I64, _I64, _I64, _I, _P, _I64, _P, _P]),
    "fp8_quant_rowwise_gather": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I, _P, _I64, _P, _P]),
    "fp8_quant_colwise_grouped_workspace_size": (_SZ, [_I64, _I64, _I32]),
    "fp8_quant_colwise_grouped": (_I, [_P, _I64, _I64, _I64, _P, _I32, _I, _P, _I64, _P, _P, _SZ,
                                       _P]),
    "fp8_quant_dual_grouped_workspace_size": (_SZ, [_I64, _I64, _I32]),
    "fp8_quant_dual_grouped": (_I, [_P, _I64, _I64, _I64, _P, _I32, _I, _P, _I64, _P, _P, _I64, _P,
                                    _P, _SZ, _P]),
    "fp8_quant_colwise_grouped_noalloc": (_I, [_P, _I64, _I64, _I64, _P, _I32, _I, _P, _I64, _P,
                                               _P]),
    "fp8_quant_weights_dual_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "fp8_quant_weights_dual": (_I, [_P, _I64, _I64, _I64, _I64, _I, _P, _I64, _P, _P, _I64, _P, _P,
                                    _SZ, _P]),
    "fp8_grouped_gemm": (_I, [_I, _I, _P, _I64, _P, _P, _I64, _I64, _P, _P, _I32, _I64, _I64,
                              _I64, _P, _I64, _I, _P, _SZ, _P]),
    "fp8_mx_quant_rowwise": (_I, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P]),
    "fp8_mx_quant_colwise": (_I, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P]),
    "fp8_mx_grouped_gemm": (_I, [_P, _I64, _P, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I32,
                                 _I64, _I64, _I64, _P, _I64, _I, _P, _SZ, _P]),
    "fp8_mx_grouped_gemm_wgrad": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I32, _I64,
                                       _I64, _I64, _P, _I64, _I, _P, _SZ, _P]),
    "fp8_block_quant_rowwise": (_I, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P]),
    "fp8_block_quant_dual": (_I, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                                  _P]),
    "fp8_block_quant_weights": (_I, [_P, _I64, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _P]),
    "fp8_block_grouped_gemm": (_I, [_I, _P, _I64, _P, _I64, _P, _I64, _I64, _P, _I64, _I64, _I64,
                                    _P, _I32, _I64, _I64, _I64, _P, _I64, _I, _P, _SZ, _P]),
    "moe_route_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "moe_route": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I64, _P, _I, _I32, _I, ctypes.c_float, _P,
                       _P, _P, _SZ, _P]),
    "fp8_moe_few_tokens_workspace_size": (_SZ, [_I64, _I64, _I64, _I32]),
    "fp8_moe_few_tokens": (_I, [_P, _I64, _I64, _I64, _P, _P, _I32, _P, _I64, _I64, _P, _I64, _I64,
                                _I64, _P, _I64, _I64, _P, _I64, _I64, _I64, _I64, _I64, _P, _I64,
                                _P, _SZ, _P]),
}


def lib() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "fp8_quantization_grouped_amd._build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(name: str, status: int) -> None:
    if status != 0:
        msg = lib().fp8q_status_string(status).decode()
        raise RuntimeError(f"{name} failed: status {status} ({msg})")


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(t: torch.Tensor, what: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a device tensor")


def fp8_quant_rowwise(x: torch.Tensor, fmt: int, q: torch.Tensor | None = None,
                      scales: torch.Tensor | None = None):
    """x: bf16 [rows, cols] (row stride may exceed cols).  Returns (q uint8 [rows, cols],
    scales float32 [rows])."""
    _dev(x, "x")
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows,), dtype=torch.float32, device=x.device)
    st = lib().fp8_quant_rowwise(_ptr(x), rows, cols, x.stride(0), fmt, _ptr(q), q.stride(0),
                                 _ptr(scales), _stream(x))
    _check("fp8_quant_rowwise", st)
    return q, scales


def fp8_quant_rowwise_gather(x: torch.Tensor, row_index: torch.Tensor, fmt: int,
                             q: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """Rowwise quantization of the rows x[row_index[r]] (indices clamped into range).
    x: bf16 [src_rows, cols]; row_index: int32 [rows] on the device.  Returns (q uint8
    [rows, cols], scales float32 [rows])."""
    _dev(x, "x")
    _dev(row_index, "row_index")
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    assert row_index.dtype == torch.int32 and row_index.dim() == 1 and row_index.is_contiguous()
    src_rows, cols = x.shape
    rows = row_index.numel()
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((rows,), dtype=torch.float32, device=x.device)
    st = lib().fp8_quant_rowwise_gather(_ptr(x), src_rows, cols, x.stride(0), _ptr(row_index),
                                        rows, fmt, _ptr(q), q.stride(0), _ptr(scales), _stream(x))
    _check("fp8_quant_rowwise_gather", st)
    return q, scales


def fp8_quant_colwise_grouped_workspace_size(rows: int, cols: int, groups: int) -> int:
    return int(lib().fp8_quant_colwise_grouped_workspace_size(rows, cols, groups))


def fp8_quant_colwise_grouped(x: torch.Tensor, offsets: torch.Tensor, fmt: int,
                              q_t: torch.Tensor | None = None,
                              scales: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None):
    """x: bf16 [rows, cols]; offsets: int32 device [groups] (cumulative group ends).
    Returns (q_t uint8 [cols, rows] column-major copy, scales float32 [groups, cols])."""
    _dev(x, "x")
    _dev(offsets, "offsets")
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    assert offsets.dtype == torch.int32 and offsets.is_contiguous()
    rows, cols = x.shape
    groups = offsets.numel()
    if q_t is None:
        q_t = torch.empty((cols, rows), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((groups, cols), dtype=torch.float32, device=x.device)
    need = fp8_quant_colwise_grouped_workspace_size(rows, cols, groups)
    if workspace is None:
        workspace = torch.empty((max(need, 256),), dtype=torch.uint8, device=x.device)
    st = lib().fp8_quant_colwise_grouped(_ptr(x), rows, cols, x.stride(0), _ptr(offsets), groups,
                                         fmt, _ptr(q_t), q_t.stride(0), _ptr(scales),
                                         _ptr(workspace), workspace.numel(), _stream(x))
    _check("fp8_quant_colwise_grouped", st)
    return q_t, scales


def fp8_quant_dual_grouped_workspace_size(rows: int, cols: int, groups: int) -> int:
    return int(lib().fp8_quant_dual_grouped_workspace_size(rows, cols, groups))


def fp8_quant_dual_grouped(x: torch.Tensor, offsets: torch.Tensor, fmt: int,
                           q: torch.Tensor | None = None, s_rows: torch.Tensor | None = None,
                           q_t: torch.Tensor | None = None, s_cols: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None):
    """Both layouts of x [rows, cols] at once: returns ((q uint8 [rows, cols], s_rows float32
    [rows]) as fp8_quant_rowwise would, (q_t uint8 [cols, rows], s_cols float32 [groups, cols])
    as fp8_quant_colwise_grouped with these token offsets would)."""
    _dev(x, "x")
    _dev(offsets, "offsets")
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    assert offsets.dtype == torch.int32 and offsets.is_contiguous()
    rows, cols = x.shape
    groups = offsets.numel()
    e = lambda *s, dt=torch.uint8: torch.empty(s, dtype=dt, device=x.device)
    q = e(rows, cols) if q is None else q
    s_rows = e(rows, dt=torch.float32) if s_rows is None else s_rows
    q_t = e(cols, rows) if q_t is None else q_t
    s_cols = e(groups, cols, dt=torch.float32) if s_cols is None else s_cols
    need = fp8_quant_dual_grouped_workspace_size(rows, cols, groups)
    if workspace is None:
        workspace = e(max(need, 256))
    st = lib().fp8_quant_dual_grouped(_ptr(x), rows, cols, x.stride(0), _ptr(offsets), groups, fmt,
                                      _ptr(q), q.stride(0), _ptr(s_rows), _ptr(q_t), q_t.stride(0),
                                      _ptr(s_cols), _ptr(workspace), workspace.numel(), _stream(x))
    _check("fp8_quant_dual_grouped", st)
    return (q, s_rows), (q_t, s_cols)


def fp8_quant_colwise_grouped_noalloc(x: torch.Tensor, offsets: torch.Tensor, fmt: int,
                                      q_t: torch.Tensor | None = None,
                                      scales: torch.Tensor | None = None):
    """fp8_quant_colwise_grouped through the entry point that allocates nothing (its maxima
    live in the library's static per-GPU array; sizes beyond it raise).  The C call allocates
    nothing; pass q_t and scales to allocate nothing here either."""
    _dev(x, "x")
    _dev(offsets, "offsets")
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    assert offsets.dtype == torch.int32 and offsets.is_contiguous()
    rows, cols = x.shape
    groups = offsets.numel()
    if q_t is None:
        q_t = torch.empty((cols, rows), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((groups, cols), dtype=torch.float32, device=x.device)
    st = lib().fp8_quant_colwise_grouped_noalloc(_ptr(x), rows, cols, x.stride(0), _ptr(offsets),
                                                 groups, fmt, _ptr(q_t), q_t.stride(0),
                                                 _ptr(scales), _stream(x))
    _check("fp8_quant_colwise_grouped_noalloc", st)
    return q_t, scales


def fp8_quant_weights_dual_workspace_size(experts: int, K: int, N: int) -> int:
    return int(lib().fp8_quant_weights_dual_workspace_size(experts, K, N))


def fp8_quant_weights_dual(w: torch.Tensor, experts: int, fmt: int,
                           q_rows: torch.Tensor | None = None,
                           s_rows: torch.Tensor | None = None,
                           q_t: torch.Tensor | None = None, s_cols: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None):
    """Expert weights w: bf16 [experts*K, N] in both layouts at once.  Returns
    (q_rows uint8 [experts*K, N], s_rows float32 [experts*K]) as fp8_quant_rowwise would and
    (q_t uint8 [N, experts*K], s_cols float32 [experts, N]) as fp8_quant_colwise_grouped with
    offsets K, 2K, .. would."""
    _dev(w, "w")
    assert w.dtype == torch.bfloat16 and w.dim() == 2 and w.stride(1) == 1
    rows, N = w.shape
    assert experts > 0 and rows % experts == 0
    K = rows // experts
    if q_rows is None:
        q_rows = torch.empty((rows, N), dtype=torch.uint8, device=w.device)
    if s_rows is None:
        s_rows = torch.empty((rows,), dtype=torch.float32, device=w.device)
    if q_t is None:
        q_t = torch.empty((N, rows), dtype=torch.uint8, device=w.device)
    if s_cols is None:
        s_cols = torch.empty((experts, N), dtype=torch.float32, device=w.device)
    need = fp8_quant_weights_dual_workspace_size(experts, K, N)
    if workspace is None:
        workspace = torch.empty((max(need, 256),), dtype=torch.uint8, device=w.device)
    st = lib().fp8_quant_weights_dual(_ptr(w), experts, K, N, w.stride(0), fmt, _ptr(q_rows),
                                      q_rows.stride(0), _ptr(s_rows), _ptr(q_t), q_t.stride(0),
                                      _ptr(s_cols), _ptr(workspace), workspace.numel(),
                                      _stream(w))
    _check("fp8_quant_weights_dual", st)
    return (q_rows, s_rows), (q_t, s_cols)


def fp8_grouped_gemm_workspace_size(mode: int, M: int, N: int, K: int, groups: int) -> int:
    return int(lib().fp8_grouped_gemm_workspace_size(mode, M, N, K, groups))


_OUT = {torch.bfloat16: OUT_BF16, torch.float32: OUT_FP32}


def _gemm_out(c, shape, out_dtype, dev):
    if c is None:
        c = torch.empty(shape, dtype=out_dtype, device=dev)
    if c.dtype not in _OUT:
        raise ValueError("the GEMM output must be bfloat16 or float32")
    if c.dim() != len(shape) or tuple(c.shape) != tuple(shape) or c.stride(-1) != 1:
        raise ValueError(f"the GEMM output must be {tuple(shape)} with unit column stride")
    if len(shape) == 3 and c.stride(0) != shape[1] * c.stride(1):
        raise ValueError("a weight-gradient output's group stride must be K * ldc")
    return c


def _gemm_ws(workspace, mode, M, N, K, groups, dev):
    need = fp8_grouped_gemm_workspace_size(mode, M, N, K, groups)
    if workspace is None:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    return workspace


def gemm_offsets_status(workspace: torch.Tensor):
    """The offsets check a grouped GEMM wrote into its workspace: (status, first bad group);
    (0, -1) for valid offsets.  Synchronises with the device to read it."""
    w = workspace[:8].view(torch.int32).cpu()
    return int(w[0]), int(w[1])


def fp8_grouped_gemm(mode: int, fmt: int, a: torch.Tensor, a_scales: torch.Tensor,
                     b: torch.Tensor, b_scales: torch.Tensor, offsets: torch.Tensor, M: int,
                     N: int, K: int, ldb: int | None = None, b_group_stride: int = 0,
                     c: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                     workspace: torch.Tensor | None = None):
    """Scaled FP8 grouped GEMM (see the C header for the two modes).
    Forward: a [M, lda], b holds every group's [N, K] rows at ldb / b_group_stride; returns
    [M, N].  Weight gradient: a [K, lda >= M], b [N, ldb >= M]; returns [G, K, N].  The output
    is bfloat16 or float32 (out_dtype, or the dtype of a given c)."""
    _dev(a, "a")
    groups = offsets.numel()
    if ldb is None:
        ldb = b.stride(0)
    shape = (M, N) if mode == GEMM_FWD_MGROUPED else (groups, K, N)
    c = _gemm_out(c, shape, out_dtype, a.device)
    ws = _gemm_ws(workspace, mode, M, N, K, groups, a.device)
    st = lib().fp8_grouped_gemm(mode, fmt, _ptr(a), a.stride(0), _ptr(a_scales), _ptr(b), ldb,
                                b_group_stride, _ptr(b_scales), _ptr(offsets), groups, M, N, K,
                                _ptr(c), c.stride(-2), _OUT[c.dtype], _ptr(ws), ws.numel(),
                                _stream(a))
    _check("fp8_grouped_gemm", st)
    return c


def fp8_mx_quant_rowwise(x: torch.Tensor, q: torch.Tensor | None = None,
                         e8m0: torch.Tensor | None = None):
    """Returns (q uint8 [rows, cols] OCP e4m3fn, e8m0 uint8 [rows, cols/32])."""
    _dev(x, "x")
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device)
    if e8m0 is None:
        e8m0 = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
    st = lib().fp8_mx_quant_rowwise(_ptr(x), rows, cols, x.stride(0), _ptr(q), q.stride(0),
                                    _ptr(e8m0), e8m0.stride(0), _stream(x))
    _check("fp8_mx_quant_rowwise", st)
    return q, e8m0


def fp8_mx_quant_colwise(x: torch.Tensor, q_t: torch.Tensor | None = None,
                         e8m0: torch.Tensor | None = None):
    """Blocks of 32 rows per column, transposed output.  Returns (q_t uint8 [cols, rows],
    e8m0 uint8 [cols, rows/32])."""
    _dev(x, "x")
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    rows, cols = x.shape
    if q_t is None:
        q_t = torch.empty((cols, rows), dtype=torch.uint8, device=x.device)
    if e8m0 is None:
        e8m0 = torch.empty((cols, rows // 32), dtype=torch.uint8, device=x.device)
    st = lib().fp8_mx_quant_colwise(_ptr(x), rows, cols, x.stride(0), _ptr(q_t), q_t.stride(0),
                                    _ptr(e8m0), e8m0.stride(0), _stream(x))
    _check("fp8_mx_quant_colwise", st)
    return q_t, e8m0


def fp8_mx_grouped_gemm(a: torch.Tensor, a_e8m0: torch.Tensor, b: torch.Tensor,
                        b_e8m0: torch.Tensor, offsets: torch.Tensor, M: int, N: int, K: int,
                        ldb: int, b_group_stride: int, ld_sb: int, sb_group_stride: int,
                        c: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                        workspace: torch.Tensor | None = None):
    """MX grouped GEMM forward; returns [M, N] (bfloat16 or float32)."""
    _dev(a, "a")
    groups = offsets.numel()
    c = _gemm_out(c, (M, N), out_dtype, a.device)
    ws = _gemm_ws(workspace, GEMM_FWD_MGROUPED, M, N, K, groups, a.device)
    st = lib().fp8_mx_grouped_gemm(_ptr(a), a.stride(0), _ptr(a_e8m0), a_e8m0.stride(0), _ptr(b),
                                   ldb, b_group_stride, _ptr(b_e8m0), ld_sb, sb_group_stride,
                                   _ptr(offsets), groups, M, N, K, _ptr(c), c.stride(0),
                                   _OUT[c.dtype], _ptr(ws), ws.numel(), _stream(a))
    _check("fp8_mx_grouped_gemm", st)
    return c


def fp8_mx_grouped_gemm_wgrad(a: torch.Tensor, a_e8m0: torch.Tensor, b: torch.Tensor,
                              b_e8m0: torch.Tensor, offsets: torch.Tensor, M: int, N: int,
                              K: int, c: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                              workspace: torch.Tensor | None = None):
    """MX weight gradient: a = XqT [K, lda >= M], b = dYqT [N, ldb >= M] with E8M0 per 32
    tokens (fp8_mx_quant_colwise outputs).  Returns [G, K, N] (bfloat16 or float32)."""
    _dev(a, "a")
    groups = offsets.numel()
    c = _gemm_out(c, (groups, K, N), out_dtype, a.device)
    ws = _gemm_ws(workspace, GEMM_WGRAD_KGROUPED, M, N, K, groups, a.device)
    st = lib().fp8_mx_grouped_gemm_wgrad(_ptr(a), a.stride(0), _ptr(a_e8m0), a_e8m0.stride(0),
                                         _ptr(b), b.stride(0), _ptr(b_e8m0), b_e8m0.stride(0),
                                         _ptr(offsets), groups, M, N, K, _ptr(c), c.stride(-2),
                                         _OUT[c.dtype], _ptr(ws), ws.numel(), _stream(a))
    _check("fp8_mx_grouped_gemm_wgrad", st)
    return c


# ------------------------------------------------------------- block-scaled FP8 (blocks of 128)

BLOCK = 128
_BYTES = (torch.uint8, torch.float8_e4m3fn)  # how e4m3fn bytes may be held


def _want(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _rows_of(t: torch.Tensor, what: str, dtypes, shape, dev) -> None:
    """Checks that t is a tensor on device dev of one of dtypes and of the given shape, with unit
    stride in its last dimension."""
    if (t.dtype in dtypes and t.device == dev and t.shape == shape
            and (t.stride()[-1] == 1 or shape[-1] <= 1) and t.is_cuda):
        return
    _want(t.is_cuda and t.device == dev, f"{what} must be on the operands' GPU")
    _want(t.dtype in dtypes, f"{what} must be {' or '.join(map(str, dtypes))}, not {t.dtype}")
    _want(t.shape == shape, f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise ValueError(f"{what} must have unit stride in its last dimension")


def _matrix(t: torch.Tensor, what: str, dtypes):
    """Checks the first operand of a call, a matrix of any size; returns its rows, columns and
    device."""
    dev = t.device
    if t.dtype not in dtypes or t.dim() != 2 or not t.is_cuda:
        _want(t.dim() == 2, f"{what} must be a matrix")
        _rows_of(t, what, dtypes, t.shape, dev)
    rows, cols = t.shape
    if cols > 1 and t.stride()[1] != 1:
        raise ValueError(f"{what} must have unit stride in its last dimension")
    return rows, cols, dev


def _one_row(ld: int, cols: int) -> int:
    """Leading dimension for a matrix of one row, whose stride ld says nothing but where it covers
    the row's end up to whole 16 elements (padding that the products may read)."""
    return min(max(ld, cols), -(-cols // 16) * 16)


def _ld(t: torch.Tensor, rows: int, cols: int) -> int:
    """Leading dimension of rows x cols elements (groups of matrices: rows of all of them); the
    stride of a single or an empty row says nothing.  Any other is handed on as it is: rows that
    overlap (an expanded tensor) are for the C entry point to refuse."""
    ld = t.stride()[-2]
    return ld if rows > 1 and cols > 0 else _one_row(ld, cols)


# the current stream's handle without a Stream object made for it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
# the current device, for callers that hold a tensor of a GPU already
_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name: str, dev: torch.device, *args) -> None:
    """The C entry point on the current stream of dev, with dev the current device."""
    index = dev.index
    if index == _device_now():
        status = getattr(_lib or lib(), name)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = getattr(_lib or lib(), name)(*args, _raw_stream(index))
    if status:
        _check(name, status)


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _padded_bytes(rows: int, cols: int, dev) -> torch.Tensor:
    """[rows, cols] bytes whose rows start on 16 bytes, as the GEMMs take them."""
    if cols % 16 == 0:
        return torch.empty(rows, cols, dtype=torch.uint8, device=dev)
    return torch.empty(rows, -(-cols // 16) * 16, dtype=torch.uint8, device=dev)[:, :cols]


_BF16, _F32, _I32T = (torch.bfloat16,), (torch.float32,), (torch.int32,)


def _factors(s: torch.Tensor, what: str, shape, dev) -> None:
    """Checks block factors, of any strides."""
    if s.dtype is not torch.float32 or s.device != dev or s.shape != shape:
        raise ValueError(f"{what} must be float32 {shape} on the operands' GPU")


def _workspace(ws: torch.Tensor, dev):
    """Pointer and bytes of a caller's workspace: one run of memory on the operands' GPU."""
    if not (ws.is_cuda and ws.device == dev and ws.is_contiguous()):
        raise ValueError("workspace must be contiguous and on the operands' GPU")
    return ws.data_ptr(), ws.nbytes


def fp8_block_quant_rowwise(x: torch.Tensor, q: torch.Tensor | None = None,
                            scales: torch.Tensor | None = None):
    """x: bf16 [rows, cols] in blocks of 1 x 128.  Returns (q [rows, cols] e4m3fn bytes, scales
    float32 [ceil(cols/128), rows], the factors d with x ~ q * d).  Rows of a new q start on 16
    bytes."""
    rows, cols, dev = _matrix(x, "x", _BF16)
    if q is None:
        q = _padded_bytes(rows, cols, dev)
    else:
        _rows_of(q, "q", _BYTES, x.shape, dev)
    blocks = -(-cols // BLOCK)
    if scales is None:
        scales = torch.empty(blocks, rows, dtype=torch.float32, device=dev)
        ld_s = rows
    else:
        _rows_of(scales, "scales", _F32, (blocks, rows), dev)
        ld_s = _ld(scales, blocks, rows)
    _call("fp8_block_quant_rowwise", dev, x.data_ptr(), rows, cols, _ld(x, rows, cols),
          q.data_ptr(), _ld(q, rows, cols), scales.data_ptr(), ld_s)
    return q, scales


def fp8_block_quant_dual(x: torch.Tensor, q: torch.Tensor | None = None,
                         s_rows: torch.Tensor | None = None, q_t: torch.Tensor | None = None,
                         s_cols: torch.Tensor | None = None, transposed_only: bool = False):
    """x: bf16 [rows, cols] in both layouts from one read.  Returns ((q [rows, cols], s_rows
    [ceil(cols/128), rows]) as fp8_block_quant_rowwise would, (q_t [cols, rows], s_cols float32
    [ceil(rows/128), cols]) in blocks of 128 rows of a column).  transposed_only: the second pair
    alone is made, and the first is (None, None)."""
    rows, cols, dev = _matrix(x, "x", _BF16)
    f32 = torch.float32
    if transposed_only:
        _want(q is None and s_rows is None, "transposed_only takes no q and s_rows")
        row_args = (None, 0, None, 0)
    else:
        if q is None:
            q = _padded_bytes(rows, cols, dev)
        else:
            _rows_of(q, "q", _BYTES, x.shape, dev)
        if s_rows is None:
            s_rows = torch.empty(_blocks(cols), rows, dtype=f32, device=dev)
        else:
            _rows_of(s_rows, "s_rows", _F32, (_blocks(cols), rows), dev)
        row_args = (q.data_ptr(), _ld(q, rows, cols), s_rows.data_ptr(),
                    _ld(s_rows, _blocks(cols), rows))
    if q_t is None:
        q_t = _padded_bytes(cols, rows, dev)
    else:
        _rows_of(q_t, "q_t", _BYTES, (cols, rows), dev)
    if s_cols is None:
        s_cols = torch.empty(_blocks(rows), cols, dtype=f32, device=dev)
    else:
        _rows_of(s_cols, "s_cols", _F32, (_blocks(rows), cols), dev)
    _call("fp8_block_quant_dual", dev, x.data_ptr(), rows, cols, _ld(x, rows, cols), *row_args,
          q_t.data_ptr(), _ld(q_t, cols, rows), s_cols.data_ptr(),
          _ld(s_cols, _blocks(rows), cols))
    return (q, s_rows), (q_t, s_cols)


def fp8_block_quant_weights(w: torch.Tensor, experts: int, q: torch.Tensor | None = None,
                            q_t: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """w: bf16 [experts * rows, cols], each expert's matrix in blocks of 128 x 128.  Returns (q
    [experts * rows, cols], q_t [cols, experts * rows] with the experts' transposes side by side,
    scales float32 [experts, ceil(rows/128), ceil(cols/128)], which serve both)."""
    total, cols, dev = _matrix(w, "w", _BF16)
    _want(experts > 0 and total % experts == 0, "w must hold experts matrices of equal size")
    rows = total // experts
    if q is None:
        q = _padded_bytes(total, cols, dev)
    else:
        _rows_of(q, "q", _BYTES, w.shape, dev)
    if q_t is None:
        q_t = _padded_bytes(cols, total, dev)
    else:
        _rows_of(q_t, "q_t", _BYTES, (cols, total), dev)
    shape = (experts, _blocks(rows), _blocks(cols))
    if scales is None:
        scales = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _rows_of(scales, "scales", _F32, shape, dev)
        _want(scales.is_contiguous(), "scales must be contiguous")
    _call("fp8_block_quant_weights", dev, w.data_ptr(), experts, rows, cols, _ld(w, total, cols),
          q.data_ptr(), _ld(q, total, cols), q_t.data_ptr(), _ld(q_t, cols, total),
          scales.data_ptr())
    return q, q_t, scales


def fp8_block_grouped_gemm(mode: int, a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor,
                           b_scales: torch.Tensor, offsets: torch.Tensor | None = None,
                           c: torch.Tensor | None = None, out_dtype=torch.bfloat16,
                           workspace: torch.Tensor | None = None):
    """Block-scaled FP8 grouped GEMM (see the C header for the two modes).
    Forward: a [M, K] with a_scales [ceil(K/128), M], b [groups, N, K] with b_scales [groups,
    ceil(N/128), ceil(K/128)] (any strides: a transpose of the quantizer's factors, with b a view
    of its transposed bytes, gives the data gradient); returns [M, N].
    Weight gradient: a [K, M] with a_scales [ceil(M/128), K], b [N, M] with b_scales [ceil(M/128),
    N]; returns [groups, K, N].
    offsets: int32 [groups] cumulative group ends, None for one group.  The output is bfloat16 or
    float32 (out_dtype, or the dtype of a given c).  gemm_offsets_status reads the offsets check
    from a given workspace."""
    _want(mode in (GEMM_FWD_MGROUPED, GEMM_WGRAD_KGROUPED), "unknown mode")
    fwd = mode == GEMM_FWD_MGROUPED
    rows, inner, dev = _matrix(a, "a", _BYTES)  # forward M, K; weight gradient K, M
    groups, off = 1, None
    if offsets is not None:
        _want(offsets.dim() == 1, "offsets must have one dimension")
        groups = offsets.shape[0]
        _rows_of(offsets, "offsets", _I32T, (groups,), dev)
        off = offsets.data_ptr()
    _want(b.dim() == (3 if fwd else 2), "b must be [groups, N, K] in the forward, [N, M] else")
    N = b.shape[-2]
    _rows_of(b, "b", _BYTES, (groups, N, inner) if fwd else (N, inner), dev)
    kb = -(-inner // BLOCK)
    _rows_of(a_scales, "a_scales", _F32, (kb, rows), dev)
    ld_sa = _ld(a_scales, kb, rows)
    if fwd:
        nb = -(-N // BLOCK)
        _factors(b_scales, "b_scales", (groups, nb, kb), dev)
        # a dimension of one entry has no stride that means anything
        sbg, sbn, sbk = b_scales.stride()
        bgs, ldb, _ = b.stride()
        if groups == 1:
            bgs = sbg = 0
        if nb <= 1:
            sbn = 0
        if kb <= 1:
            sbk = 0
        if N <= 1:
            ldb = _one_row(ldb, inner)
        if inner == 0:  # nothing is read, and the strides of no elements are no strides
            bgs = ldb = 0
        M, K, shape = rows, inner, (rows, N)
    else:
        _rows_of(b_scales, "b_scales", _F32, (kb, N), dev)
        bgs, ldb, sbg, sbn = 0, _ld(b, N, inner), 0, 1
        sbk = _ld(b_scales, kb, N)
        M, K, shape = inner, rows, (groups, rows, N)
    if c is None:
        _want(out_dtype in _OUT, "the output must be bfloat16 or float32")
        c = torch.empty(*shape, dtype=out_dtype, device=dev)
        ldc = N
    else:
        c = _gemm_out(c, shape, out_dtype, dev)
        _want(c.device == dev, "c must be on the operands' GPU")
        ldc = _ld(c, c.shape[-2] if fwd else groups * c.shape[-2], N)
    ws, ws_bytes = (None, 0) if workspace is None else _workspace(workspace, dev)
    _call("fp8_block_grouped_gemm", dev, mode, a.data_ptr(), _ld(a, rows, inner),
          a_scales.data_ptr(), ld_sa, b.data_ptr(), ldb, bgs, b_scales.data_ptr(), sbn, sbk, sbg,
          off, groups, M, N, K, c.data_ptr(), ldc, _OUT[c.dtype], ws, ws_bytes)
    return c


# ------------------------------------------------- a mixture-of-experts layer for a few tokens

def _no_grad(what: str, *tensors) -> None:
    """Refuses operands whose gradient the call would lose."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(f"{what} has no gradient: detach its operands, or call it under torch.no_grad()")


SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
_SCORING = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}


def moe_route_workspace_size(T: int, H: int, E: int) -> int:
    return int(lib().moe_route_workspace_size(T, H, E))


def moe_route(x: torch.Tensor, router: torch.Tensor, top_k: int,
              bias: torch.Tensor | None = None, scoring: str = "softmax",
              renormalize: bool = True, scale: float = 1.0, ids: torch.Tensor | None = None,
              weights: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """The experts of each token: x bf16 [T, H], router bf16 [E, H], bias float32 [E] (added to the
    scores for the choice alone).  scoring: "softmax" or "sigmoid".  Returns (ids int32 [T, top_k],
    weights float32 [T, top_k]) in descending order; ties go to the lowest index.  No gradient:
    operands that require one are refused while torch records."""
    T, H, dev = _matrix(x, "x", _BF16)
    _no_grad("moe_route", x, router, bias)
    E = router.shape[0]
    _rows_of(router, "router", _BF16, (E, H), dev)
    _want(scoring in _SCORING, "scoring must be softmax or sigmoid")
    _want(1 <= top_k <= E, "top_k must lie in [1, number of experts]")
    if bias is not None:
        _rows_of(bias, "bias", _F32, (E,), dev)
    if ids is None:
        ids = torch.empty(T, top_k, dtype=torch.int32, device=dev)
    else:
        _rows_of(ids, "ids", _I32T, (T, top_k), dev)
        _want(ids.is_contiguous(), "ids must be contiguous")
    if weights is None:
        weights = torch.empty(T, top_k, dtype=torch.float32, device=dev)
    else:
        _rows_of(weights, "weights", _F32, (T, top_k), dev)
        _want(weights.is_contiguous(), "weights must be contiguous")
    ws = None
    if workspace is None:
        need = lib().moe_route_workspace_size(T, H, E)
        if need:  # a small router takes none
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            ws = workspace.data_ptr()
    else:
        ws, need = _workspace(workspace, dev)
    _call("moe_route", dev, x.data_ptr(), T, H, _ld(x, T, H), router.data_ptr(), E,
          _ld(router, E, H),
          None if bias is None else bias.data_ptr(), _SCORING[scoring], top_k, int(renormalize),
          scale, ids.data_ptr(), weights.data_ptr(),
          ws, need)
    return ids, weights


def fp8_moe_few_tokens_workspace_size(T: int, H: int, I: int, top_k: int) -> int:
    return int(lib().fp8_moe_few_tokens_workspace_size(T, H, I, top_k))


def _expert_weights(w, s, what, shape, dev):
    """The pointers and strides of block-scaled expert weights, as the C entry point takes them."""
    _rows_of(w, what, _BYTES, shape, dev)
    E, n, k = shape
    _factors(s, f"the factors of {what}", (E, _blocks(n), _blocks(k)), dev)
    sg, sn, sk = s.stride()
    gs, ld, _ = w.stride()
    if E == 1:
        gs = sg = 0
    if n <= BLOCK:
        sn = 0
        if n <= 1:
            ld = max(ld, k)
    if k <= BLOCK:
        sk = 0
    return w.data_ptr(), ld, gs, s.data_ptr(), sn, sk, sg


def fp8_moe_few_tokens(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                       w13: torch.Tensor, s13: torch.Tensor, w2: torch.Tensor, s2: torch.Tensor,
                       y: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """The experts' feed-forward of a few tokens (at most 128): x bf16 [T, H]; ids int32 and
    weights float32 [T, top_k] (moe_route's); w13 [E, 2I, H] and w2 [E, H, I] e4m3fn bytes with
    scales [E, ceil(2I/128), ceil(H/128)] and [E, ceil(H/128), ceil(I/128)]
    (fp8_block_quant_weights').  Returns y bf16 [T, H].  An id outside [0, E) adds nothing.  No
    gradient: operands that require one are refused while torch records."""
    T, H, dev = _matrix(x, "x", _BF16)
    _no_grad("fp8_moe_few_tokens", x, weights)
    _want(ids.dim() == 2, "ids must be a matrix")
    top_k = ids.shape[1]
    _rows_of(ids, "ids", _I32T, (T, top_k), dev)
    _rows_of(weights, "weights", _F32, (T, top_k), dev)
    _want(ids.is_contiguous() and weights.is_contiguous(), "ids and weights must be contiguous")
    _want(w13.dim() == 3 and w13.shape[1] % 2 == 0, "w13 must be [E, 2I, H]")
    E, I = w13.shape[0], w13.shape[1] // 2
    args13 = _expert_weights(w13, s13, "w13", (E, 2 * I, H), dev)
    args2 = _expert_weights(w2, s2, "w2", (E, H, I), dev)
    if y is None:
        y = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
    else:
        _rows_of(y, "y", _BF16, (T, H), dev)
    if workspace is None:
        need = fp8_moe_few_tokens_workspace_size(T, H, I, top_k)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        ws = workspace.data_ptr()
    else:
        ws, need = _workspace(workspace, dev)
    _call("fp8_moe_few_tokens", dev, x.data_ptr(), T, H, _ld(x, T, H), ids.data_ptr(),
          weights.data_ptr(), top_k, *args13, *args2, E, I, y.data_ptr(), _ld(y, T, H),
          ws, need)
    return y
