"""Python binding of libgptq_mi355x.so (argument marshalling only).

Every step of the hot path runs in the library's HIP kernels. PyTorch supplies
device memory (torch.empty on a ROCm device) and the current stream. There is
no CPU fallback: if the library is missing, loading raises.

Entry points (same names as include/gptq.h):
    accumulate_hessian(H, X, accumulate)      H (+)= 2 X^T X, lower triangle
    prepare_hinv(H, damp)                      U = chol_upper((H + lambda I)^-1)
    quantize_layer(W, U, bits, group_size, grid)
    act_order(H)                               column order of descending diag(H)
    permute_hessian(H, perm)                   H gathered into that order
    quantize_layer_ordered(W, U, perm, bits, group_size, grid, static_groups)
    dequant_gemv(qcodes, scales, zeros, bits, group_size, x)   y = W_hat x, one token
    pack_codes(codes, bits)
    kv_append(k, v, page_table, lens, k_new, v_new, cu_seqlens)   new rows into a paged key-value cache
    paged_attention(q, k, v, page_table, lens, ...)   one new token per sequence over its pages
    paged_prefill(q, k, v, page_table, lens, cu_seqlens, ...)   prompts, or the next chunks of them
    kv_evict(k, v, page_table, lens, weights, budget, new_pages, ...)   the least attended slots leave
    trace_start(), trace_stop()                device time per kernel family (instrumentation)
and quantize(W, x_chunks, ...) which runs the stages of one layer (natural
order, or act-order with act_order=True).
"""

from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# GPTQ_MI355X_LIB may name another build of the library (the debug build,
# libgptq_mi355x_debug.so, for instance)
LIB_PATH = os.environ.get("GPTQ_MI355X_LIB") or os.path.join(_HERE, "libgptq_mi355x.so")

GPTQ_OK, GPTQ_ERR_INVALID_ARG, GPTQ_ERR_WORKSPACE, GPTQ_ERR_HIP, GPTQ_ERR_UNSUPPORTED = range(5)
GPTQ_F16, GPTQ_F32, GPTQ_F64, GPTQ_BF16 = 0, 1, 2, 3
GPTQ_GRID_ASYM_MINMAX, GPTQ_GRID_TERNARY, GPTQ_GRID_SYM_MINMAX = 0, 1, 2
WS_ACCUMULATE_HESSIAN, WS_PREPARE_HINV, WS_QUANTIZE_LAYER = 0, 1, 2

EXPORTED = ["gptq_abi_version", "gptq_status_string", "gptq_workspace_bytes", "gptq_accumulate_hessian",
            "gptq_prepare_hinv", "gptq_quantize_layer", "gptq_act_order", "gptq_permute_hessian",
            "gptq_quantize_layer_ordered", "gptq_dequant_gemv", "gptq_pack_codes", "gptq_trace_start",
            "gptq_trace_stop", "gptq_trace_family", "gptq_accumulate_hessian_noalloc", "gptq_prepare_hchol",
            "gptq_gemv_prepare_act_order", "gptq_dequant_gemv_perm", "gptq_kv_append", "gptq_kv_workspace_bytes",
            "gptq_paged_attention", "gptq_paged_prefill", "gptq_kv_evict"]
TRACE_FAMILIES = 18


GPTQ_FACTOR_HINV_CHOL, GPTQ_FACTOR_H_CHOL = 0, 1
_FACTOR = {"U": GPTQ_FACTOR_HINV_CHOL, "R": GPTQ_FACTOR_H_CHOL}


class QCfg(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int32), ("grid", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("factor", ctypes.c_int32)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("n_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64)]


class KvSeqs(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("ld_table", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("lens", ctypes.c_void_p), ("n_seqs", ctypes.c_int64)]


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the HIP library (raises when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m post_weight_quantization_18_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.gptq_abi_version.restype = i32
    lib.gptq_abi_version.argtypes = []
    lib.gptq_status_string.restype = ctypes.c_char_p
    lib.gptq_status_string.argtypes = [i32]
    lib.gptq_workspace_bytes.restype = sz
    lib.gptq_workspace_bytes.argtypes = [i32, i64, i64, i64, ctypes.POINTER(QCfg)]
    lib.gptq_accumulate_hessian.restype = i32
    lib.gptq_accumulate_hessian.argtypes = [vp, i32, i64, i64, vp, i64, i64, i32, vp, sz, vp]
    lib.gptq_prepare_hinv.restype = i32
    lib.gptq_prepare_hinv.argtypes = [vp, i32, i64, i64, ctypes.c_double, vp, i32, i64, vp, vp, vp, sz, vp]
    lib.gptq_prepare_hchol.restype = i32
    lib.gptq_prepare_hchol.argtypes = [vp, i32, i64, i64, ctypes.c_double, vp, i32, i64, vp, vp, vp, sz, vp]
    lib.gptq_quantize_layer.restype = i32
    lib.gptq_quantize_layer.argtypes = [vp, i32, i64, i64, i64, vp, i32, i64, ctypes.POINTER(QCfg), vp, vp, vp, vp,
                                        vp, vp, sz, vp]
    lib.gptq_act_order.restype = i32
    lib.gptq_act_order.argtypes = [vp, i32, i64, i64, vp, vp]
    lib.gptq_permute_hessian.restype = i32
    lib.gptq_permute_hessian.argtypes = [vp, i32, i64, i64, vp, vp, i64, vp]
    lib.gptq_quantize_layer_ordered.restype = i32
    lib.gptq_quantize_layer_ordered.argtypes = [vp, i32, i64, i64, i64, vp, i32, i64, ctypes.POINTER(QCfg), vp, i32,
                                                vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.gptq_dequant_gemv.restype = i32
    lib.gptq_dequant_gemv.argtypes = [vp, vp, vp, i64, i64, i32, i32, vp, vp, vp]
    lib.gptq_gemv_prepare_act_order.restype = i32
    lib.gptq_gemv_prepare_act_order.argtypes = [vp, vp, i64, i64, i32, i32, vp, vp, vp, vp]
    lib.gptq_dequant_gemv_perm.restype = i32
    lib.gptq_dequant_gemv_perm.argtypes = [vp, vp, vp, i64, i64, i32, i32, vp, vp, vp, vp, vp]
    lib.gptq_pack_codes.restype = i32
    lib.gptq_pack_codes.argtypes = [vp, i64, i64, i32, vp, vp]
    lib.gptq_accumulate_hessian_noalloc.restype = i32
    lib.gptq_accumulate_hessian_noalloc.argtypes = [vp, i32, i64, i64, vp, i64, i64, i32, vp]
    f32, pc, ps = ctypes.c_float, ctypes.POINTER(KvCache), ctypes.POINTER(KvSeqs)
    lib.gptq_kv_append.restype = i32
    lib.gptq_kv_append.argtypes = [pc, ps, vp, i64, vp, i64, vp, i64, vp]
    lib.gptq_kv_workspace_bytes.restype = sz
    lib.gptq_kv_workspace_bytes.argtypes = [pc, ps, i64, i64, i64, i64, i32]
    lib.gptq_paged_attention.restype = i32
    lib.gptq_paged_attention.argtypes = [pc, ps, vp, i64, i64, f32, i64, i64, vp, i64, vp, i64, vp, sz, vp]
    lib.gptq_paged_prefill.restype = i32
    lib.gptq_paged_prefill.argtypes = [pc, ps, vp, i64, vp, i64, i64, f32, i64, i64, vp, i64, vp, i64, vp, sz, vp]
    lib.gptq_kv_evict.restype = i32
    lib.gptq_kv_evict.argtypes = [pc, ps, vp, i64, i64, i64, i64, vp, i64, vp, i64, vp, vp, i64, vp, vp]
    lib.gptq_trace_start.restype = i32
    lib.gptq_trace_start.argtypes = []
    lib.gptq_trace_stop.restype = i32
    lib.gptq_trace_stop.argtypes = [vp, vp, vp, i32]
    lib.gptq_trace_family.restype = ctypes.c_char_p
    lib.gptq_trace_family.argtypes = [i32]
    _lib = lib
    return lib


class GPTQError(RuntimeError):
    def __init__(self, status: int, what: str):
        msg = load_library().gptq_status_string(status).decode()
        super().__init__(f"{what}: {msg}")
        self.status = status


def _check(status: int, what: str):
    if status != GPTQ_OK:
        raise GPTQError(status, what)


_DT = {torch.float16: GPTQ_F16, torch.float32: GPTQ_F32, torch.float64: GPTQ_F64}


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need_cuda(t, name):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a tensor on a ROCm device")


def _rowmajor_ld(t, name):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a row-major 2-D tensor (unit column stride)")
    return t.stride(0)


def make_qcfg(bits: int, group_size: int = 0, grid: str = "asym", block_size: int = 128,
              factor: str = "U") -> QCfg:
    g = {"asym": GPTQ_GRID_ASYM_MINMAX, "ternary": GPTQ_GRID_TERNARY, "sym": GPTQ_GRID_SYM_MINMAX}[grid]
    return QCfg(bits, g, group_size, block_size, _FACTOR[factor])


def workspace_bytes(which: int, m: int = 0, d: int = 0, n: int = 0, cfg: QCfg | None = None) -> int:
    lib = load_library()
    return int(lib.gptq_workspace_bytes(which, m, d, n, ctypes.byref(cfg) if cfg is not None else None))


def _workspace(nbytes: int, device, workspace):
    if nbytes == 0:
        return None
    if workspace is not None and workspace.numel() * workspace.element_size() >= nbytes:
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def accumulate_hessian(H: torch.Tensor, X: torch.Tensor, accumulate: bool = True, workspace=None):
    """H[i][j] (+)= 2 sum_t X[t][i] X[t][j] for i >= j. H fp64 or fp32 [d, d]; X fp16 [n, d]."""
    lib = load_library()
    _need_cuda(H, "H")
    _need_cuda(X, "X")
    if X.dtype != torch.float16:
        raise ValueError("X must be fp16")
    d = H.shape[0]
    ldh = _rowmajor_ld(H, "H")
    ldx = _rowmajor_ld(X, "X") if X.shape[0] > 0 else d
    n = X.shape[0]
    # a caller's workspace is passed as it is: the call accepts any size (a
    # smaller one selects the token-major form, then fewer split partials)
    ws = workspace if workspace is not None else _workspace(workspace_bytes(WS_ACCUMULATE_HESSIAN, 0, d, n),
                                                           H.device, None)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.gptq_accumulate_hessian(_ptr(H), _DT[H.dtype], d, ldh, _ptr(X) if n else ctypes.c_void_p(0), n, ldx,
                                       int(bool(accumulate)), _ptr(ws), nbytes, _stream(H.device)),
           "gptq_accumulate_hessian")
    return H


def prepare_hinv(H: torch.Tensor, damp: float = 0.01, U: torch.Tensor | None = None,
                 u_dtype: torch.dtype = torch.float32, workspace=None):
    """Returns (U, info, lam): U upper [d, d] with U^T U = (H + lam I)^-1, info a
    1-element int32 device tensor (0 = ok), lam a 1-element fp64 device tensor."""
    lib = load_library()
    _need_cuda(H, "H")
    d = H.shape[0]
    if U is None:
        U = torch.empty(d, d, dtype=u_dtype, device=H.device)
    info = torch.empty(1, dtype=torch.int32, device=H.device)
    lam = torch.empty(1, dtype=torch.float64, device=H.device)
    ws = _workspace(workspace_bytes(WS_PREPARE_HINV, 0, d), H.device, workspace)
    _check(lib.gptq_prepare_hinv(_ptr(H), _DT[H.dtype], d, _rowmajor_ld(H, "H"), float(damp), _ptr(U), _DT[U.dtype],
                                 _rowmajor_ld(U, "U"), _ptr(info), _ptr(lam), _ptr(ws), ws.numel(),
                                 _stream(H.device)), "gptq_prepare_hinv")
    return U, info, lam


def prepare_hchol(H: torch.Tensor, damp: float = 0.01, R: torch.Tensor | None = None,
                  r_dtype: torch.dtype = torch.float64, workspace=None):
    """Returns (R, info, lam): R upper [d, d] with R R^T = H + lam I (R = U^-1), info
    and lam as prepare_hinv. Pass R to the quantize calls with factor="R"."""
    lib = load_library()
    _need_cuda(H, "H")
    d = H.shape[0]
    if R is None:
        R = torch.empty(d, d, dtype=r_dtype, device=H.device)
    info = torch.empty(1, dtype=torch.int32, device=H.device)
    lam = torch.empty(1, dtype=torch.float64, device=H.device)
    ws = _workspace(workspace_bytes(WS_PREPARE_HINV, 0, d), H.device, workspace)
    _check(lib.gptq_prepare_hchol(_ptr(H), _DT[H.dtype], d, _rowmajor_ld(H, "H"), float(damp), _ptr(R), _DT[R.dtype],
                                  _rowmajor_ld(R, "R"), _ptr(info), _ptr(lam), _ptr(ws), ws.numel(),
                                  _stream(H.device)), "gptq_prepare_hchol")
    return R, info, lam


def quantize_layer(W: torch.Tensor, U: torch.Tensor, bits: int, group_size: int = 0, grid: str = "asym",
                   block_size: int = 128, want_w_hat: bool = True, workspace=None, out=None, factor: str = "U"):
    """Returns dict(qcodes uint32 [m, d*bits/32] (as int32 storage), scales fp32 [m, ng],
    zeros uint8 [m, ng], w_hat fp32 [m, d] or None, err_sq fp32 [m]). factor "U": U =
    chol(H_d^-1) from prepare_hinv; "R": R from prepare_hchol (passed as U)."""
    lib = load_library()
    _need_cuda(W, "W")
    _need_cuda(U, "U")
    m, d = W.shape
    cfg = make_qcfg(bits, group_size, grid, block_size, factor)
    ng = d // group_size if group_size else 1
    dev = W.device
    if out is None:
        out = {
            "qcodes": torch.empty(m, d * bits // 32, dtype=torch.int32, device=dev),
            "scales": torch.empty(m, ng, dtype=torch.float32, device=dev),
            "zeros": torch.empty(m, ng, dtype=torch.uint8, device=dev),
            "w_hat": torch.empty(m, d, dtype=torch.float32, device=dev) if want_w_hat else None,
            "err_sq": torch.empty(m, dtype=torch.float32, device=dev),
        }
    ws = _workspace(workspace_bytes(WS_QUANTIZE_LAYER, m, d, 0, cfg), dev, workspace)
    _check(lib.gptq_quantize_layer(_ptr(W), _DT[W.dtype], m, d, _rowmajor_ld(W, "W"), _ptr(U), _DT[U.dtype],
                                   _rowmajor_ld(U, "U"), ctypes.byref(cfg), _ptr(out["qcodes"]), _ptr(out["scales"]),
                                   _ptr(out["zeros"]), _ptr(out["w_hat"]), _ptr(out["err_sq"]), _ptr(ws), ws.numel(),
                                   _stream(dev)), "gptq_quantize_layer")
    return out


def act_order(H: torch.Tensor, perm: torch.Tensor | None = None) -> torch.Tensor:
    """int32 device [d]: perm[j] = the column with the j-th largest H_jj (ties in index order)."""
    lib = load_library()
    _need_cuda(H, "H")
    d = H.shape[0]
    if perm is None:
        perm = torch.empty(d, dtype=torch.int32, device=H.device)
    elif perm.dtype != torch.int32 or not perm.is_contiguous() or perm.numel() != d:
        raise ValueError("perm must be contiguous int32 [d]")
    _check(lib.gptq_act_order(_ptr(H), _DT[H.dtype], d, _rowmajor_ld(H, "H"), _ptr(perm), _stream(H.device)),
           "gptq_act_order")
    return perm


_act_order = act_order  # `quantize` takes a flag of the same name


def permute_hessian(H: torch.Tensor, perm: torch.Tensor, Hp: torch.Tensor | None = None) -> torch.Tensor:
    """Hp[i][j] = H[perm[i]][perm[j]] for j <= i (lower triangles), same dtype as H."""
    lib = load_library()
    _need_cuda(H, "H")
    _need_cuda(perm, "perm")
    if perm.dtype != torch.int32 or not perm.is_contiguous():
        raise ValueError("perm must be contiguous int32")
    d = H.shape[0]
    if Hp is None:
        Hp = torch.empty(d, d, dtype=H.dtype, device=H.device)
    _check(lib.gptq_permute_hessian(_ptr(H), _DT[H.dtype], d, _rowmajor_ld(H, "H"), _ptr(perm), _ptr(Hp),
                                    _rowmajor_ld(Hp, "Hp"), _stream(H.device)), "gptq_permute_hessian")
    return Hp


def quantize_layer_ordered(W: torch.Tensor, U: torch.Tensor, perm: torch.Tensor, bits: int, group_size: int = 0,
                           grid: str = "asym", static_groups: bool = False, block_size: int = 128,
                           want_w_hat: bool = True, workspace=None, out=None, factor: str = "U"):
    """quantize_layer with the columns quantized in the order perm (U: the factor of
    the Hessian in that order). Outputs in natural column order, plus g_idx int32 [d]."""
    lib = load_library()
    _need_cuda(W, "W")
    _need_cuda(U, "U")
    _need_cuda(perm, "perm")
    if perm.dtype != torch.int32 or not perm.is_contiguous():
        raise ValueError("perm must be contiguous int32")
    m, d = W.shape
    cfg = make_qcfg(bits, group_size, grid, block_size, factor)
    ng = d // group_size if group_size else 1
    dev = W.device
    if out is None:
        out = {
            "qcodes": torch.empty(m, d * bits // 32, dtype=torch.int32, device=dev),
            "scales": torch.empty(m, ng, dtype=torch.float32, device=dev),
            "zeros": torch.empty(m, ng, dtype=torch.uint8, device=dev),
            "g_idx": torch.empty(d, dtype=torch.int32, device=dev),
            "w_hat": torch.empty(m, d, dtype=torch.float32, device=dev) if want_w_hat else None,
            "err_sq": torch.empty(m, dtype=torch.float32, device=dev),
        }
    ws = _workspace(workspace_bytes(WS_QUANTIZE_LAYER, m, d, 0, cfg), dev, workspace)
    _check(lib.gptq_quantize_layer_ordered(_ptr(W), _DT[W.dtype], m, d, _rowmajor_ld(W, "W"), _ptr(U), _DT[U.dtype],
                                           _rowmajor_ld(U, "U"), ctypes.byref(cfg), _ptr(perm),
                                           int(bool(static_groups)), _ptr(out["qcodes"]), _ptr(out["scales"]),
                                           _ptr(out["zeros"]), _ptr(out["g_idx"]), _ptr(out["w_hat"]),
                                           _ptr(out["err_sq"]), _ptr(ws), ws.numel(), _stream(dev)),
           "gptq_quantize_layer_ordered")
    return out


def dequant_gemv(qcodes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, bits: int, group_size: int,
                 x: torch.Tensor, y: torch.Tensor | None = None) -> torch.Tensor:
    """y fp32 [m] = W_hat x with W_hat dequantized on the fly from the packed
    codes (the quantize_layer outputs); x fp16 [d]."""
    lib = load_library()
    for t, n in ((qcodes, "qcodes"), (scales, "scales"), (zeros, "zeros"), (x, "x")):
        _need_cuda(t, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if x.dtype != torch.float16 or scales.dtype != torch.float32 or zeros.dtype != torch.uint8:
        raise ValueError("x fp16, scales fp32, zeros uint8")
    m, d = qcodes.shape[0], x.shape[0]
    if y is None:
        y = torch.empty(m, dtype=torch.float32, device=x.device)
    _check(lib.gptq_dequant_gemv(_ptr(qcodes), _ptr(scales), _ptr(zeros), m, d, bits, group_size, _ptr(x), _ptr(y),
                                 _stream(x.device)), "gptq_dequant_gemv")
    return y


def gemv_prepare_act_order(qcodes: torch.Tensor, g_idx: torch.Tensor, bits: int, group_size: int):
    """Act-order codes (natural column order, group index g_idx) rewritten with
    the columns sorted by group. Returns (qcodes in col_perm order, col_perm
    int32 [d], info int32 device scalar: 0 when every group holds group_size
    columns)."""
    lib = load_library()
    for t, n in ((qcodes, "qcodes"), (g_idx, "g_idx")):
        _need_cuda(t, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if g_idx.dtype != torch.int32:
        raise ValueError("g_idx must be int32")
    m, d = qcodes.shape[0], g_idx.shape[0]
    out = torch.empty_like(qcodes)
    col_perm = torch.empty(d, dtype=torch.int32, device=qcodes.device)
    info = torch.empty(1, dtype=torch.int32, device=qcodes.device)
    _check(lib.gptq_gemv_prepare_act_order(_ptr(qcodes), _ptr(g_idx), m, d, bits, group_size, _ptr(out),
                                           _ptr(col_perm), _ptr(info), _stream(qcodes.device)),
           "gptq_gemv_prepare_act_order")
    return out, col_perm, info


def dequant_gemv_perm(qcodes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, bits: int, group_size: int,
                      col_perm: torch.Tensor, x: torch.Tensor, x_perm: torch.Tensor | None = None,
                      y: torch.Tensor | None = None) -> torch.Tensor:
    """y fp32 [m] = W x for codes in col_perm order (gemv_prepare_act_order), x
    fp16 [d] in natural order; x_perm is the fp16 [d] buffer the gather uses."""
    lib = load_library()
    for t, n in ((qcodes, "qcodes"), (scales, "scales"), (zeros, "zeros"), (col_perm, "col_perm"), (x, "x")):
        _need_cuda(t, n)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if x.dtype != torch.float16 or scales.dtype != torch.float32 or zeros.dtype != torch.uint8:
        raise ValueError("x fp16, scales fp32, zeros uint8")
    m, d = qcodes.shape[0], x.shape[0]
    if x_perm is None:
        x_perm = torch.empty(d, dtype=torch.float16, device=x.device)
    if y is None:
        y = torch.empty(m, dtype=torch.float32, device=x.device)
    _check(lib.gptq_dequant_gemv_perm(_ptr(qcodes), _ptr(scales), _ptr(zeros), m, d, bits, group_size,
                                      _ptr(col_perm), _ptr(x), _ptr(x_perm), _ptr(y), _stream(x.device)),
           "gptq_dequant_gemv_perm")
    return y


def pack_codes(codes: torch.Tensor, bits: int) -> torch.Tensor:
    """codes uint8 [m, d] -> int32 storage of the uint32 bitstream [m, d*bits/32]."""
    lib = load_library()
    _need_cuda(codes, "codes")
    if codes.dtype != torch.uint8 or not codes.is_contiguous():
        raise ValueError("codes must be contiguous uint8")
    m, d = codes.shape
    out = torch.empty(m, d * bits // 32, dtype=torch.int32, device=codes.device)
    _check(lib.gptq_pack_codes(_ptr(codes), m, d, bits, _ptr(out), _stream(codes.device)), "gptq_pack_codes")
    return out


_KV_DT = {torch.float16: GPTQ_F16, torch.bfloat16: GPTQ_BF16}


def _kv(k, v, page_table, lens):
    """The cache and its sequences as the library takes them, dtypes and shapes checked."""
    _need_cuda(k, "k")
    dt = _KV_DT.get(k.dtype)
    if dt is None or v.dtype != k.dtype:
        raise ValueError("k and v must be fp16 or bf16, both the same")
    shape, strides = k.shape, k.stride()
    if len(shape) != 4 or v.shape != shape:
        raise ValueError("k and v must be [n_pages, n_kv_heads, page_size, head_dim]")
    n_pages, n_kv, ps, dim = shape
    if v.stride() != strides or strides[3] != 1 or strides[2] != dim or strides[1] != ps * dim:
        raise ValueError("k and v: equal strides, contiguous within a page")
    if page_table.dtype != torch.int32 or lens.dtype != torch.int32:
        raise ValueError("page_table and lens must be int32")
    rows = page_table.shape
    if len(rows) != 2 or lens.shape != rows[:1]:
        raise ValueError("page_table [n_seqs, max_pages], lens [n_seqs]")
    n_seqs, max_pages = rows
    ld, one = page_table.stride()
    if (one != 1 and max_pages > 1) or (n_seqs > 1 and lens.stride(0) != 1):
        raise ValueError("page_table rows and lens must be contiguous")
    # the stride of a single page or row says nothing
    return (KvCache(k.data_ptr(), v.data_ptr(), dt, ps, n_kv, dim, n_pages,
                    strides[0] if n_pages > 1 else n_kv * ps * dim),
            KvSeqs(page_table.data_ptr(), ld if n_seqs > 1 else max_pages, max_pages, lens.data_ptr(), n_seqs))


def _one_device(k, *others):
    dev = k.get_device()
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError("every tensor must be on the cache's device")
    return dev


def _rows(t, name, dtype, heads, dim):
    """Row stride of new tokens' rows [n, heads, dim], contiguous within a row."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must have the cache's dtype")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [n, heads, head_dim] of the cache's head_dim")
    s = t.stride()
    if s[2] != 1 or (s[1] != dim and shape[1] > 1):
        raise ValueError(f"{name} rows must be contiguous")
    return s[0] if shape[0] > 1 else shape[1] * dim


def _cu(cu, n_seqs):
    if cu.dtype != torch.int32 or cu.dim() != 1 or cu.shape[0] != n_seqs + 1 or not cu.is_contiguous():
        raise ValueError("cu_seqlens must be contiguous int32 [n_seqs + 1]")
    return cu.data_ptr()


def _weights(w, name, n_seqs, n_kv, slots):
    """Row stride of accumulated weights [n_seqs, n_kv, >= slots]."""
    if w.dtype != torch.float32 or w.dim() != 3 or w.shape[0] != n_seqs or w.shape[1] != n_kv or w.shape[2] < slots:
        raise ValueError(f"{name} must be fp32 [n_seqs, n_kv_heads, >= max_pages * page_size]")
    if not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return w.shape[2]


def _launch(dev, fn, what, *args):
    """fn(*args, stream) on device dev and its current stream."""
    # (the raw handle: a Stream object around it costs a microsecond)
    if torch.cuda.current_device() == dev:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        raise GPTQError(status, what)


def kv_append(k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, k_new: torch.Tensor,
              v_new: torch.Tensor, cu_seqlens: torch.Tensor | None = None):
    """New tokens' keys and values into the pages of their sequences. k, v [n_pages,
    n_kv_heads, page_size, head_dim] fp16 or bf16; page_table int32 [n_seqs,
    max_pages]; lens int32 [n_seqs], the new tokens counted; k_new, v_new [n,
    n_kv_heads, head_dim], sequence b's rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1
    (int32 [n_seqs + 1]; None: one row per sequence)."""
    lib = _lib or load_library()
    cache, seqs = _kv(k, v, page_table, lens)
    dev = _one_device(k, v, page_table, lens, k_new, v_new, cu_seqlens)
    ldk = _rows(k_new, "k_new", k.dtype, cache.n_kv_heads, cache.head_dim)
    ldv = _rows(v_new, "v_new", k.dtype, cache.n_kv_heads, cache.head_dim)
    n = k_new.shape[0]
    if v_new.shape[0] != n:
        raise ValueError("k_new and v_new must have the same tokens")
    cu = _cu(cu_seqlens, seqs.n_seqs) if cu_seqlens is not None else None
    _launch(dev, lib.gptq_kv_append, "gptq_kv_append", cache, seqs, k_new.data_ptr(), ldk, v_new.data_ptr(), ldv, cu, n)


def kv_workspace_bytes(k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, n_heads: int,
                       window: int = 0, sinks: int = 0, n_tokens: int = 0, weights: bool = False) -> int:
    """Workspace of paged_attention (n_tokens = 0) or of paged_prefill with n_tokens rows."""
    cache, seqs = _kv(k, v, page_table, lens)
    return int(load_library().gptq_kv_workspace_bytes(cache, seqs, n_heads, window, sinks, n_tokens, int(weights)))


def _attend(fn, name, lib, q, k, v, page_table, lens, cu_seqlens, scale, window, sinks, weights, out, workspace):
    cache, seqs = _kv(k, v, page_table, lens)
    dev = _one_device(k, v, page_table, lens, q, cu_seqlens, weights, out, workspace)
    dim, dtype = cache.head_dim, k.dtype
    ldq = _rows(q, "q", dtype, None, dim)
    n, heads = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty(n, heads, dim, dtype=dtype, device=q.device)
        ldo = heads * dim
    else:
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
        ldo = _rows(out, "out", dtype, heads, dim)
    wp, ldw, summed = None, 0, 0
    if weights is not None:
        ldw = _weights(weights, "weights", seqs.n_seqs, cache.n_kv_heads, seqs.max_pages * cache.page_size)
        wp, summed = weights.data_ptr(), 1
    if scale is None:
        scale = dim ** -0.5
    if cu_seqlens is None:
        if n != seqs.n_seqs:
            raise ValueError("q must have one row per sequence")
        rows = ()
        nbytes = lib.gptq_kv_workspace_bytes(cache, seqs, heads, window, sinks, 0, summed)
    else:
        rows = (_cu(cu_seqlens, seqs.n_seqs), n)
        nbytes = lib.gptq_kv_workspace_bytes(cache, seqs, heads, window, sinks, n, summed) if n else 0
    ws = None
    if nbytes:
        workspace = _workspace(nbytes, q.device, workspace)
        ws = workspace.data_ptr()
    _launch(dev, fn, name, cache, seqs, q.data_ptr(), ldq, *rows, heads, scale, window, sinks, wp, ldw, out.data_ptr(),
            ldo, ws, nbytes)
    return out


def paged_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                    scale: float | None = None, window: int = 0, sinks: int = 0, weights: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of one new token per sequence (its key and value already appended):
    out [n_seqs, n_heads, head_dim] in q's dtype. The token sees its whole sequence,
    or with a window the last `window` slots and the first `sinks`. scale defaults
    to head_dim^-0.5. weights fp32 [n_seqs, n_kv_heads, slots] (slots >= max_pages *
    page_size): every visible slot's attention weight is added, summed over the heads
    that share its key."""
    lib = _lib or load_library()
    return _attend(lib.gptq_paged_attention, "gptq_paged_attention", lib, q, k, v, page_table, lens, None, scale, window,
                   sinks, weights, out, workspace)


def paged_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor,
                  cu_seqlens: torch.Tensor, scale: float | None = None, window: int = 0, sinks: int = 0,
                  weights: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Causal attention of prompts, or of the next chunks of longer ones, over the
    pages: rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of q [n, n_heads, head_dim] are
    the last tokens of sequence b. Rows behind the last sequence stay as `out` held
    them. Other arguments as paged_attention."""
    lib = _lib or load_library()
    if cu_seqlens is None:
        raise ValueError("cu_seqlens must be int32 [n_seqs + 1]")
    return _attend(lib.gptq_paged_prefill, "gptq_paged_prefill", lib, q, k, v, page_table, lens, cu_seqlens, scale,
                   window, sinks, weights, out, workspace)


def kv_evict(k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, weights: torch.Tensor,
             budget: int, new_pages: torch.Tensor, sinks: int = 0, recent: int = 0):
    """Sequences longer than budget keep, per kv head, the first `sinks`, the last
    `recent` and the most attended other slots (weights, as the attention calls add
    them), in order, moved to new_pages int32 [n_seqs, >= ceil(budget / page_size)]
    (free pages). Returns (page_table, lens, weights, kept): the table and lengths
    to go on with, the weights in the new order (0 behind the last slot), and
    int32 [n_seqs, n_kv_heads, budget] the old slot of every new one (-1 behind the
    last)."""
    lib = _lib or load_library()
    cache, seqs = _kv(k, v, page_table, lens)
    dev = _one_device(k, v, page_table, lens, weights, new_pages)
    n_seqs, max_pages, n_kv = seqs.n_seqs, seqs.max_pages, cache.n_kv_heads
    slots = max_pages * cache.page_size
    ldw = _weights(weights, "weights", n_seqs, n_kv, slots)
    if new_pages.dtype != torch.int32 or new_pages.dim() != 2 or new_pages.shape[0] != n_seqs or \
            (new_pages.stride(1) != 1 and new_pages.shape[1] > 1):
        raise ValueError("new_pages must be int32 [n_seqs, pages], rows contiguous")
    if budget < 1:
        raise ValueError("budget must be positive")
    table_out = torch.empty_like(page_table, memory_format=torch.contiguous_format)
    lens_out = torch.empty_like(lens)
    weights_out = torch.empty_like(weights)
    kept = torch.empty(n_seqs, n_kv, budget, dtype=torch.int32, device=k.device)
    _launch(dev, lib.gptq_kv_evict, "gptq_kv_evict", cache, seqs, weights.data_ptr(), ldw, budget, sinks, recent,
            new_pages.data_ptr(), new_pages.stride(0) if n_seqs > 1 else new_pages.shape[1], table_out.data_ptr(),
            max_pages, lens_out.data_ptr(), weights_out.data_ptr(), ldw, kept.data_ptr())
    return table_out, lens_out, weights_out, kept


def trace_start():
    """Start recording HIP events around every library launch from this thread."""
    _check(load_library().gptq_trace_start(), "gptq_trace_start")


def trace_stop() -> dict:
    """End the trace; {family: {"launches": n, "ms": summed device ms, "work": executed
    matrix-core flops}} for the families that launched anything."""
    lib = load_library()
    n = TRACE_FAMILIES
    launches = (ctypes.c_int64 * n)()
    ms = (ctypes.c_double * n)()
    work = (ctypes.c_double * n)()
    _check(lib.gptq_trace_stop(ctypes.cast(launches, ctypes.c_void_p), ctypes.cast(ms, ctypes.c_void_p),
                               ctypes.cast(work, ctypes.c_void_p), n), "gptq_trace_stop")
    return {lib.gptq_trace_family(k).decode(): {"launches": int(launches[k]), "ms": float(ms[k]),
                                                   "work": float(work[k])}
            for k in range(n) if launches[k]}


def quantize(W: torch.Tensor, x_chunks, bits: int, group_size: int = 0, grid: str = "asym", damp: float = 0.01,
             h_dtype: torch.dtype = torch.float64, u_dtype: torch.dtype = torch.float32, want_w_hat: bool = True,
             act_order: bool = False, static_groups: bool = False, factor: str = "U"):
    """The whole hot path of one layer: H over the chunks, U, then the column loop.
    Returns (result dict, H, U, lam). Raises when H + lam I is not positive definite.
    With act_order the columns go in descending diag(H) (result["perm"]), U is the
    factor of the permuted H, and the outputs are still in natural column order."""
    if isinstance(x_chunks, torch.Tensor):
        x_chunks = [x_chunks]
    d = W.shape[1]
    H = torch.empty(d, d, dtype=h_dtype, device=W.device)
    for i, xc in enumerate(x_chunks):
        accumulate_hessian(H, xc, accumulate=i > 0)
    perm = None
    prep = prepare_hchol if factor == "R" else prepare_hinv
    kw = {"r_dtype": torch.float64} if factor == "R" else {"u_dtype": u_dtype}
    if act_order:
        perm = _act_order(H)
        U, info, lam = prep(permute_hessian(H, perm), damp, **kw)
    else:
        U, info, lam = prep(H, damp, **kw)
    bad = int(info.item())
    if bad:
        raise GPTQError(GPTQ_ERR_INVALID_ARG, f"H + lambda I is not positive definite (reversed minor {bad})")
    if act_order:
        res = quantize_layer_ordered(W, U, perm, bits, group_size, grid, static_groups, want_w_hat=want_w_hat,
                                     factor=factor)
        res["perm"] = perm
    else:
        res = quantize_layer(W, U, bits, group_size, grid, want_w_hat=want_w_hat, factor=factor)
    return res, H, U, lam
