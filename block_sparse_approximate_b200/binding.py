"""ctypes binding of libsparseattn (argument marshalling only).

Every function here validates tensor placement, allocates the outputs with
torch on the inputs' device, passes raw device pointers and the current CUDA
stream to the C entry point of the same name, and raises ``SparseAttnError``
on a non-OK status.  All computation happens in the library's CUDA kernels;
there is no fallback: if ``libsparseattn.so`` has not been built, ``load()``
raises.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsparseattn.so")

SA_OK, SA_ERR_INVALID_ARG, SA_ERR_UNSUPPORTED, SA_ERR_ALIGNMENT, SA_ERR_CUDA, SA_ERR_WORKSPACE = range(6)
SA_FP32, SA_BF16 = 0, 1
ROUTE = {"dot": 0, "proj": 1, "taylor2": 2, "cov": 3}
TAIL = {"drop": 0, "zero_order": 1, "linear_mix": 2, "first_order": 3, "residual_linear": 4}

# every entry point declared in include/sparseattn.h
EXPORTS = ("sa_block_pool", "sa_route", "sa_sparse_attn_fwd", "sa_decode_workspace_size",
           "sa_decode_fwd", "sa_decode_fwd_static", "sa_quantize_e4m3", "sa_sparse_attn_fwd_fp8",
           "sa_sfa_encode", "sa_sfa_densify", "sa_sfa_workspace_size", "sa_sfa_attn_fwd",
           "sa_sparse_attn_bwd_workspace_size", "sa_sparse_attn_bwd", "sa_sparse_attn_fwd_lse",
           "sa_sparse_attn_bwd_lse", "sa_sparse_attn_bwd_linear_mix_workspace_size", "sa_sparse_attn_bwd_linear_mix",
           "sa_paged_plan", "sa_paged_append", "sa_paged_attn_workspace_size", "sa_paged_attn_fwd",
           "sa_device_error", "sa_last_error", "sa_version")


class SparseAttnError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("N", ctypes.c_int32),
                ("d", ctypes.c_int32), ("block", ctypes.c_int32)]


class DecodeShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("N", ctypes.c_int32), ("d", ctypes.c_int32), ("block", ctypes.c_int32)]


class PagedShape(ctypes.Structure):
    _fields_ = [("S", ctypes.c_int32), ("T", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("page", ctypes.c_int32), ("P", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


_STAT_FIELDS = ("qmean", "kmean", "vsum", "kvar", "zrelu", "htot", "ztot", "kmean_bf16", "vmean_bf16",
                "hbar", "hbarT_bf16", "covnorm", "sexp", "kvar_bf16")


class BlockStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _STAT_FIELDS]


_FP8_FIELDS = ("q", "k", "v", "q_scale", "k_scale", "v_scale", "v_scale_max", "kbar", "vbar",
               "kbar_scale", "vbar_scale")


class Fp8Operands(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _FP8_FIELDS]


_lib = None


def load():
    """Loads libsparseattn.so (built in-tree) and declares its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: run `python -m block_sparse_approximate_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    lib.sa_block_pool.argtypes = [vp, vp, vp, ctypes.c_int, Shape, ctypes.POINTER(BlockStats), vp]
    lib.sa_route.argtypes = [ctypes.POINTER(BlockStats), Shape, ctypes.c_int, vp, vp, f32, i32, vp, vp, vp]
    lib.sa_sparse_attn_fwd.argtypes = [vp, vp, vp, ctypes.c_int, Shape, vp, i32, ctypes.c_int, vp,
                                       ctypes.POINTER(BlockStats), f32, vp, vp]
    lib.sa_decode_workspace_size.argtypes = [DecodeShape, i32]
    lib.sa_decode_workspace_size.restype = sz
    lib.sa_decode_fwd.argtypes = [vp, vp, vp, ctypes.c_int, DecodeShape, ctypes.POINTER(BlockStats),
                                  i32, f32, ctypes.c_int, vp, vp, vp, vp, sz, vp]
    lib.sa_decode_fwd_static.argtypes = [vp, vp, vp, ctypes.c_int, DecodeShape, ctypes.POINTER(BlockStats),
                                         i32, f32, ctypes.c_int, vp, vp, vp, vp]
    lib.sa_quantize_e4m3.argtypes = [vp, ctypes.c_int64, i32, i32, i32, vp, vp, vp, vp]
    lib.sa_sparse_attn_fwd_fp8.argtypes = [ctypes.POINTER(Fp8Operands), Shape, vp, i32, ctypes.c_int, f32, vp, vp]
    i64 = ctypes.c_int64
    lib.sa_sfa_encode.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp]
    lib.sa_sfa_densify.argtypes = [vp, vp, i64, i32, i32, vp, vp]
    lib.sa_sfa_workspace_size.argtypes = [Shape]
    lib.sa_sfa_workspace_size.restype = sz
    lib.sa_sfa_attn_fwd.argtypes = [vp, vp, vp, ctypes.c_int, Shape, f32, vp, vp, sz, vp]
    lib.sa_sparse_attn_bwd_workspace_size.argtypes = [Shape, i32]
    lib.sa_sparse_attn_bwd_workspace_size.restype = sz
    lib.sa_sparse_attn_bwd.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, Shape, vp, i32, ctypes.c_int,
                                       ctypes.POINTER(BlockStats), f32, vp, vp, vp, vp, sz, vp]
    lib.sa_sparse_attn_fwd_lse.argtypes = [vp, vp, vp, ctypes.c_int, Shape, vp, i32, ctypes.c_int,
                                           ctypes.POINTER(BlockStats), f32, vp, vp, vp]
    lib.sa_sparse_attn_bwd_lse.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_int, Shape, vp, i32, ctypes.c_int,
                                           ctypes.POINTER(BlockStats), f32, vp, vp, vp, vp, sz, vp]
    lib.sa_sparse_attn_bwd_linear_mix_workspace_size.argtypes = [Shape, i32]
    lib.sa_sparse_attn_bwd_linear_mix_workspace_size.restype = sz
    lib.sa_sparse_attn_bwd_linear_mix.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, Shape, vp, i32, vp,
                                                  ctypes.POINTER(BlockStats), f32, vp, vp, vp, vp, sz, vp]
    lib.sa_paged_plan.argtypes = [vp, vp, PagedShape, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.sa_paged_append.argtypes = [vp, vp, i64, i64, ctypes.c_int, PagedShape, vp, vp, vp, vp]
    lib.sa_paged_attn_workspace_size.argtypes = [PagedShape]
    lib.sa_paged_attn_workspace_size.restype = sz
    lib.sa_paged_attn_fwd.argtypes = [vp, i64, vp, vp, ctypes.c_int, PagedShape, vp, vp, vp, i32, f32, vp, vp, sz, vp]
    for fn in ("sa_paged_plan", "sa_paged_append", "sa_paged_attn_fwd",
               "sa_block_pool", "sa_route", "sa_sparse_attn_fwd", "sa_decode_fwd", "sa_decode_fwd_static",
               "sa_quantize_e4m3", "sa_sparse_attn_fwd_fp8", "sa_sfa_encode", "sa_sfa_densify", "sa_sfa_attn_fwd",
               "sa_sparse_attn_bwd", "sa_sparse_attn_fwd_lse", "sa_sparse_attn_bwd_lse",
               "sa_sparse_attn_bwd_linear_mix"):
        getattr(lib, fn).restype = ctypes.c_int
    lib.sa_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32)]
    lib.sa_device_error.restype = ctypes.c_int
    lib.sa_last_error.restype = ctypes.c_char_p
    lib.sa_version.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(fn: str, status: int):
    if status != SA_OK:
        raise SparseAttnError(fn, status, load().sa_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SA_FP32
    if t.dtype == torch.bfloat16:
        return SA_BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


def _stats_struct(stats: dict) -> BlockStats:
    return BlockStats(*[_ptr(stats.get(n)) for n in _STAT_FIELDS])


def device_error() -> int:
    """Reads and clears the device-side error word (0 = no kernel gave up)."""
    v = ctypes.c_uint32(0)
    _check("sa_device_error", load().sa_device_error(ctypes.byref(v)))
    return int(v.value)


def version() -> str:
    return load().sa_version().decode()


def block_pool(Q: Optional[torch.Tensor], K: torch.Tensor, V: torch.Tensor, block: int, *,
               variance: bool = False, linear: bool = False, centroids_bf16: bool = False,
               first_order: bool = False, covariance: bool = False, residual: bool = False,
               stream=None) -> dict:
    """Block statistics of (Q,) K, V [B,H,N,d]; returns a dict of float32 tensors."""
    lib = load()
    Bsz, H, N, d = K.shape
    nb = N // block
    dev = K.device
    f = dict(device=dev, dtype=torch.float32)
    st = {"kmean": torch.empty(Bsz, H, nb, d, **f), "vsum": torch.empty(Bsz, H, nb, d, **f)}
    if Q is not None:
        st["qmean"] = torch.empty(Bsz, H, nb, d, **f)
    if variance:
        st["kvar"] = torch.empty(Bsz, H, nb, d, **f)
    if linear:
        st["zrelu"] = torch.empty(Bsz, H, nb, d, **f)
        st["htot"] = torch.empty(Bsz, H, d, d, **f)
        st["ztot"] = torch.empty(Bsz, H, d, **f)
    if centroids_bf16:
        st["kmean_bf16"] = torch.empty(Bsz, H, nb, d, device=dev, dtype=torch.bfloat16)
        st["vmean_bf16"] = torch.empty(Bsz, H, nb, d, device=dev, dtype=torch.bfloat16)
        if variance:
            st["kvar_bf16"] = torch.empty(Bsz, H, nb, d, device=dev, dtype=torch.bfloat16)
    if first_order or covariance:
        st["hbar"] = torch.empty(Bsz, H, d, d, **f)
        if centroids_bf16 and first_order:
            st["hbarT_bf16"] = torch.empty(Bsz, H, d, d, device=dev, dtype=torch.bfloat16)
    if covariance:
        st["covnorm"] = torch.empty(Bsz, H, nb, **f)
    if residual:
        st["sexp"] = torch.empty(Bsz, H, d, d, **f)
    cst = _stats_struct(st)
    _check("sa_block_pool", lib.sa_block_pool(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(K),
                                              Shape(Bsz, H, N, d, block), ctypes.byref(cst),
                                              _stream(stream)))
    return st


def route(stats: dict, shape, mode: str, topk: int, *, proj_q=None, proj_k=None,
          scale: float = 1.0, want_scores: bool = False, stream=None):
    """Top-k KV blocks per query block: returns (block_idx int32 [B,H,nqb,topk], scores or None)."""
    lib = load()
    Bsz, H, N, d, block = shape
    nb = N // block
    dev = stats["kmean"].device
    idx = torch.empty(Bsz, H, nb, topk, device=dev, dtype=torch.int32)
    sc = torch.empty(Bsz, H, nb, nb, device=dev, dtype=torch.float32) if want_scores else None
    cst = _stats_struct(stats)
    _check("sa_route", lib.sa_route(ctypes.byref(cst), Shape(Bsz, H, N, d, block), ROUTE[mode],
                                    _ptr(proj_q), _ptr(proj_k), float(scale), int(topk),
                                    _ptr(idx), _ptr(sc), _stream(stream)))
    return idx, sc


def sparse_attn_fwd(Q, K, V, block_idx, block: int, tail: str, stats: dict, scale: float, *,
                    alpha=None, out=None, lse=None, stream=None) -> torch.Tensor:
    """Sparse prefill forward; returns O with the shape and dtype of Q.  With
    ``lse`` (float32 [B,H,N]) the rows' log2 log-sum-exp is written there
    (sa_sparse_attn_fwd_lse)."""
    lib = load()
    Bsz, H, N, d = Q.shape
    O = out if out is not None else torch.empty_like(Q)
    topk = block_idx.shape[-1] if block_idx is not None else 0
    cst = _stats_struct(stats or {})
    if lse is not None:
        _check("sa_sparse_attn_fwd_lse",
               lib.sa_sparse_attn_fwd_lse(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(Q), Shape(Bsz, H, N, d, block),
                                          _ptr(block_idx) if topk > 0 else None, int(topk), TAIL[tail],
                                          ctypes.byref(cst), float(scale), _ptr(O), _ptr(lse), _stream(stream)))
        return O
    _check("sa_sparse_attn_fwd",
           lib.sa_sparse_attn_fwd(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(Q),
                                  Shape(Bsz, H, N, d, block),
                                  _ptr(block_idx) if topk > 0 else None, int(topk), TAIL[tail],
                                  _ptr(alpha), ctypes.byref(cst), float(scale), _ptr(O),
                                  _stream(stream)))
    return O


def decode_stats_bf16(stats: dict) -> dict:
    """The view of block statistics that makes sa_decode_fwd read the bf16
    copies (kmean_bf16, kvar_bf16, vmean_bf16; kmean left NULL), plus sexp."""
    return {n: stats[n] for n in ("kmean_bf16", "kvar_bf16", "vmean_bf16", "sexp") if n in stats}


def decode_workspace_size(B: int, Hq: int, Hkv: int, N: int, d: int, block: int, topk: int) -> int:
    return int(load().sa_decode_workspace_size(DecodeShape(B, Hq, Hkv, N, d, block), int(topk)))


def decode_fwd(q, Kcache, Vcache, stats: dict, block: int, topk: int, scale: float, *,
               tail: str = "zero_order", workspace=None, want_route: bool = True, out=None,
               stream=None):
    """GQA decode; returns (o [B,Hq,d], block_idx [B,Hkv,topk] or None, scores [B,Hkv,nb] or None)."""
    lib = load()
    Bsz, Hq, d = q.shape
    Hkv, N = Kcache.shape[1], Kcache.shape[2]
    nb = N // block
    dev = q.device
    ws_bytes = decode_workspace_size(Bsz, Hq, Hkv, N, d, block, topk)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 256), device=dev, dtype=torch.uint8)
    o = out if out is not None else torch.empty_like(q)
    idx = torch.empty(Bsz, Hkv, topk, device=dev, dtype=torch.int32) if want_route else None
    sc = torch.empty(Bsz, Hkv, nb, device=dev, dtype=torch.float32) if want_route else None
    cst = _stats_struct(stats)
    _check("sa_decode_fwd",
           lib.sa_decode_fwd(_ptr(q), _ptr(Kcache), _ptr(Vcache), _dtype_code(q),
                             DecodeShape(Bsz, Hq, Hkv, N, d, block), ctypes.byref(cst), int(topk),
                             float(scale), TAIL[tail], _ptr(idx), _ptr(sc), _ptr(o),
                             _ptr(workspace), workspace.numel(), _stream(stream)))
    return o, idx, sc


def decode_fwd_static(q, Kcache, Vcache, stats: dict, block: int, topk: int, scale: float, *,
                      tail: str = "zero_order", out=None, stream=None):
    """decode_fwd with the library's static scratch instead of a workspace
    (see sa_decode_fwd_static); returns (o, block_idx, scores)."""
    lib = load()
    Bsz, Hq, d = q.shape
    Hkv, N = Kcache.shape[1], Kcache.shape[2]
    nb = N // block
    dev = q.device
    o = out if out is not None else torch.empty_like(q)
    idx = torch.empty(Bsz, Hkv, topk, device=dev, dtype=torch.int32)
    sc = torch.empty(Bsz, Hkv, nb, device=dev, dtype=torch.float32)
    cst = _stats_struct(stats)
    _check("sa_decode_fwd_static",
           lib.sa_decode_fwd_static(_ptr(q), _ptr(Kcache), _ptr(Vcache), _dtype_code(q),
                                    DecodeShape(Bsz, Hq, Hkv, N, d, block), ctypes.byref(cst), int(topk),
                                    float(scale), TAIL[tail], _ptr(idx), _ptr(sc), _ptr(o),
                                    _stream(stream)))
    return o, idx, sc


def quantize_e4m3(X: torch.Tensor, block: int = 128, *, want_max: bool = False, stream=None):
    """Per-block e4m3 codes of a bf16 tensor [B,H,N,d]: returns (codes uint8
    [B,H,N,d], scales float32 [B,H,ceil(N/block)], scale_max [B,H] or None)."""
    lib = load()
    Bsz, H, N, d = X.shape
    nblk = (N + block - 1) // block
    codes = torch.empty(X.shape, device=X.device, dtype=torch.uint8)
    scales = torch.empty(Bsz, H, nblk, device=X.device, dtype=torch.float32)
    smax = torch.empty(Bsz, H, device=X.device, dtype=torch.float32) if want_max else None
    _check("sa_quantize_e4m3", lib.sa_quantize_e4m3(_ptr(X), Bsz * H, N, d, block, _ptr(codes), _ptr(scales),
                                                    _ptr(smax), _stream(stream)))
    return codes, scales, smax


def fp8_operands(Q, K, V, stats: dict, block: int = 128, stream=None) -> dict:
    """Quantises Q, K, V and (if present) the bf16 centroid tiles of ``stats``."""
    q, qs, _ = quantize_e4m3(Q, block, stream=stream)
    k, ks, _ = quantize_e4m3(K, block, stream=stream)
    v, vs, vmax = quantize_e4m3(V, block, want_max=True, stream=stream)
    ops = {"q": q, "k": k, "v": v, "q_scale": qs, "k_scale": ks, "v_scale": vs, "v_scale_max": vmax}
    if stats.get("kmean_bf16") is not None:
        ops["kbar"], ops["kbar_scale"], _ = quantize_e4m3(stats["kmean_bf16"].view(torch.bfloat16), 128,
                                                          stream=stream)
        ops["vbar"], ops["vbar_scale"], _ = quantize_e4m3(stats["vmean_bf16"].view(torch.bfloat16), 128,
                                                          stream=stream)
    return ops


def sparse_attn_fwd_fp8(ops: dict, shape, block_idx, tail: str, scale: float, *, out=None, stream=None):
    """e4m3 sparse prefill; ``ops`` from fp8_operands; returns bf16 O [B,H,N,d]."""
    lib = load()
    Bsz, H, N, d, block = shape
    O = out if out is not None else torch.empty(Bsz, H, N, d, device=ops["q"].device, dtype=torch.bfloat16)
    topk = block_idx.shape[-1] if block_idx is not None else 0
    cops = Fp8Operands(*[_ptr(ops.get(n)) for n in _FP8_FIELDS])
    _check("sa_sparse_attn_fwd_fp8",
           lib.sa_sparse_attn_fwd_fp8(ctypes.byref(cops), Shape(Bsz, H, N, d, block),
                                      _ptr(block_idx) if topk > 0 else None, int(topk), TAIL[tail],
                                      float(scale), _ptr(O), _stream(stream)))
    return O


def sfa_encode(X: torch.Tensor, kf: int, *, want_dense: bool = True, stream=None):
    """Sparse feature codes of a bf16 tensor [..., d]: returns (vals bf16 [..., kf],
    idx uint8 [..., kf], dense bf16 [..., d] zero-filled rows or None)."""
    lib = load()
    d = X.shape[-1]
    rows = X.numel() // d
    vals = torch.empty(X.shape[:-1] + (kf,), device=X.device, dtype=torch.bfloat16)
    idx = torch.empty(X.shape[:-1] + (kf,), device=X.device, dtype=torch.uint8)
    dense = torch.empty_like(X) if want_dense else None
    _check("sa_sfa_encode", lib.sa_sfa_encode(_ptr(X), rows, d, int(kf), _ptr(vals), _ptr(idx), _ptr(dense),
                                              _stream(stream)))
    return vals, idx, dense


def sfa_densify(vals: torch.Tensor, idx: torch.Tensor, d: int, *, stream=None) -> torch.Tensor:
    """Zero-filled rows [..., d] bf16 from sparse feature codes."""
    lib = load()
    kf = vals.shape[-1]
    rows = vals.numel() // kf
    dense = torch.empty(vals.shape[:-1] + (d,), device=vals.device, dtype=torch.bfloat16)
    _check("sa_sfa_densify", lib.sa_sfa_densify(_ptr(vals), _ptr(idx), rows, int(d), int(kf), _ptr(dense),
                                                _stream(stream)))
    return dense


def sfa_attn_fwd(Qs, Ks, V, block: int, scale: float, *, workspace=None, out=None, stream=None) -> torch.Tensor:
    """Sparse feature attention on zero-filled sparse Q, K [B,H,N,d] and dense V."""
    lib = load()
    Bsz, H, N, d = Qs.shape
    shape = Shape(Bsz, H, N, d, block)
    ws = int(lib.sa_sfa_workspace_size(shape))
    if workspace is None:
        workspace = torch.empty(max(ws, 256), device=Qs.device, dtype=torch.uint8)
    O = out if out is not None else torch.empty_like(Qs)
    _check("sa_sfa_attn_fwd", lib.sa_sfa_attn_fwd(_ptr(Qs), _ptr(Ks), _ptr(V), _dtype_code(Qs), shape, float(scale),
                                                  _ptr(O), _ptr(workspace), workspace.numel(), _stream(stream)))
    return O


def sparse_attn_bwd(Q, K, V, O, dO, block_idx, block: int, tail: str, stats: dict, scale: float, *,
                    lse=None, workspace=None, stream=None):
    """Backward of sparse_attn_fwd (drop, zero_order): returns float32 (dQ, dK, dV).
    ``lse``: the forward's log-sum-exp (sparse_attn_fwd(..., lse=...)), which
    sa_sparse_attn_bwd_lse uses instead of recomputing it."""
    lib = load()
    Bsz, H, N, d = Q.shape
    topk = block_idx.shape[-1] if block_idx is not None else 0
    shape = Shape(Bsz, H, N, d, block)
    ws = int(lib.sa_sparse_attn_bwd_workspace_size(shape, int(topk)))
    if workspace is None:
        workspace = torch.empty(max(ws, 256), device=Q.device, dtype=torch.uint8)
    f = dict(device=Q.device, dtype=torch.float32)
    dQ, dK, dV = torch.empty(Q.shape, **f), torch.empty(K.shape, **f), torch.empty(V.shape, **f)
    cst = _stats_struct(stats or {})
    if lse is not None:
        _check("sa_sparse_attn_bwd_lse",
               lib.sa_sparse_attn_bwd_lse(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(lse), _dtype_code(Q),
                                          shape, _ptr(block_idx) if topk > 0 else None, int(topk), TAIL[tail],
                                          ctypes.byref(cst), float(scale), _ptr(dQ), _ptr(dK), _ptr(dV),
                                          _ptr(workspace), workspace.numel(), _stream(stream)))
        return dQ, dK, dV
    _check("sa_sparse_attn_bwd",
           lib.sa_sparse_attn_bwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _dtype_code(Q), shape,
                                  _ptr(block_idx) if topk > 0 else None, int(topk), TAIL[tail], ctypes.byref(cst),
                                  float(scale), _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(workspace), workspace.numel(),
                                  _stream(stream)))
    return dQ, dK, dV


def sparse_attn_bwd_linear_mix(Q, K, V, O, dO, block_idx, block: int, alpha, stats: dict, scale: float, *,
                               workspace=None, stream=None):
    """Backward of sparse_attn_fwd(..., "linear_mix", alpha=alpha): returns float32 (dQ, dK, dV)."""
    lib = load()
    Bsz, H, N, d = Q.shape
    topk = block_idx.shape[-1] if block_idx is not None else 0
    shape = Shape(Bsz, H, N, d, block)
    ws = int(lib.sa_sparse_attn_bwd_linear_mix_workspace_size(shape, int(topk)))
    if workspace is None:
        workspace = torch.empty(max(ws, 256), device=Q.device, dtype=torch.uint8)
    f = dict(device=Q.device, dtype=torch.float32)
    dQ, dK, dV = torch.empty(Q.shape, **f), torch.empty(K.shape, **f), torch.empty(V.shape, **f)
    cst = _stats_struct(stats or {})
    _check("sa_sparse_attn_bwd_linear_mix",
           lib.sa_sparse_attn_bwd_linear_mix(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _dtype_code(Q), shape,
                                             _ptr(block_idx) if topk > 0 else None, int(topk), _ptr(alpha),
                                             ctypes.byref(cst), float(scale), _ptr(dQ), _ptr(dK), _ptr(dV),
                                             _ptr(workspace), workspace.numel(), _stream(stream)))
    return dQ, dK, dV


# ---------------------------------------------------------------- paged KV cache
# A serving step makes these calls with a few microseconds of GPU work each,
# so the checks are kept to one attribute comparison apiece.

_I32, _I64, _U8 = torch.int32, torch.int64, torch.uint8
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _paged_ptr(t: torch.Tensor, i: int, dtype, name: str, dense: bool = True) -> int:
    """Pointer of a tensor that must live on CUDA device ``i`` with ``dtype`` (and be contiguous)."""
    if t.get_device() != i or t.dtype != dtype or (dense and not t.is_contiguous()):
        if t.get_device() != i or i < 0:
            raise ValueError(f"{name} must live on the call's CUDA device")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _paged_rows(t: torch.Tensor, name: str) -> int:
    """The row stride (elements) of packed rows [T, heads, d] whose rows are dense."""
    T, H, d = t.shape
    s0, s1, s2 = t.stride()
    if (s2 != 1 or (s1 != d and H > 1)) and t.numel():
        raise ValueError(f"{name}: the heads of a row must be contiguous (only the row stride is free)")
    return s0 if T > 1 else H * d


# A field of PagedShape would cut a size that leaves 32 bits without a word.
# Checked are those that tensors of this card's memory (or plain numbers) can
# have.
_TOO_LARGE = "paged cache: every size must be below 2^31"


def _paged_call(i: int, stream, fn: str, f, *args):
    """Calls the C entry point ``f`` with device ``i`` current, on ``stream`` (default: the device's current stream)."""
    if i < 0:
        raise ValueError(f"{fn}: tensors must live on a CUDA device")
    if stream is not None:
        s = stream.cuda_stream
    elif _raw_stream is not None:
        s = _raw_stream(i)
    else:
        s = torch.cuda.current_stream(i).cuda_stream
    if i == torch.cuda.current_device():
        status = f(*args, s)
    else:
        with torch.cuda.device(i):
            status = f(*args, s)
    if status != SA_OK:
        _check(fn, status)


def _paged_empty(like: torch.Tensor, shape, dtype, stream):
    """An empty tensor on ``like``'s device and the stream that will use it, so that the caching allocator's
    reuse stays ordered with it."""
    if not like.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def paged_plan(ctx_len: torch.Tensor, new_len: torch.Tensor, held: torch.Tensor, table: torch.Tensor,
               free_pages: torch.Tensor, free_state: torch.Tensor, tokens: int, page: int, *, q_start=None,
               kv_len=None, slots=None, stream=None):
    """Pages and places of a serving step's new tokens, from the requests'
    lengths (int32 [S]): updates held [S], table [S,max_pages], free_pages [P]
    and free_state [2] (all int32) in place and returns (q_start int32 [S+1],
    kv_len int32 [S], slots int64 [tokens]).  ``tokens``: rows of the step's
    packed arrays, padding included.  None of the arrays that are written may
    overlap another (SparseAttnError): the lengths are the caller's own
    tensors.  See sa_paged_plan for refused requests."""
    (S,), (P,), (rows, width) = ctx_len.shape, free_pages.shape, table.shape
    if rows != S or new_len.shape != (S,) or held.shape != (S,) or free_state.shape != (2,):
        raise ValueError("new_len and held must be [S], table [S, max_pages], free_state [2]")
    if (S | tokens | page | P | width) >> 31 > 0:
        raise ValueError(_TOO_LARGE)
    i = ctx_len.get_device()
    if q_start is None:
        q_start = _paged_empty(ctx_len, S + 1, _I32, stream)
    if kv_len is None:
        kv_len = _paged_empty(ctx_len, S, _I32, stream)
    if slots is None:
        slots = _paged_empty(ctx_len, tokens, _I64, stream)
    if q_start.shape != (S + 1,) or kv_len.shape != (S,) or slots.shape != (tokens,):
        raise ValueError("q_start must be [S + 1], kv_len [S], slots [tokens]")
    ptr = _paged_ptr
    _paged_call(i, stream, "sa_paged_plan", load().sa_paged_plan, ptr(ctx_len, i, _I32, "ctx_len"),
                ptr(new_len, i, _I32, "new_len"), PagedShape(S, tokens, 1, 1, 64, page, P, width),
                ptr(held, i, _I32, "held"), ptr(table, i, _I32, "table"), ptr(free_pages, i, _I32, "free_pages"),
                ptr(free_state, i, _I32, "free_state"), ptr(q_start, i, _I32, "q_start"),
                ptr(kv_len, i, _I32, "kv_len"), ptr(slots, i, _I64, "slots"))
    return q_start, kv_len, slots


def paged_append(K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, Kcache: torch.Tensor, Vcache: torch.Tensor, *,
                 stream=None) -> None:
    """Writes the rows K, V [T,Hkv,d] (views with a row stride serve) to their
    slots (int64 [T], negative: skipped) in the pools [P,Hkv,page,d]."""
    P, Hkv, page, d = Kcache.shape
    rows = K.shape
    T = rows[0]
    if rows != (T, Hkv, d) or V.shape != rows or Vcache.shape != Kcache.shape or slots.shape != (T,):
        raise ValueError("K and V must be [T,Hkv,d], slots [T], the caches [P,Hkv,page,d]")
    if T >> 31:
        raise ValueError(_TOO_LARGE)
    i, dt, ptr = Kcache.get_device(), Kcache.dtype, _paged_ptr
    _paged_call(i, stream, "sa_paged_append", load().sa_paged_append, ptr(K, i, dt, "K", False),
                ptr(V, i, dt, "V", False), _paged_rows(K, "K"), _paged_rows(V, "V"), _dtype_code(Kcache),
                PagedShape(0, T, Hkv, Hkv, d, page, P, 0), ptr(slots, i, _I64, "slots"), ptr(Kcache, i, dt, "Kcache"),
                ptr(Vcache, i, dt, "Vcache"))


def paged_attn_workspace_size(S: int, T: int, Hq: int, Hkv: int, d: int, page: int, P: int, max_pages: int) -> int:
    if max(S, T, Hq, Hkv, d, page, P, max_pages) >> 31 > 0:
        raise ValueError(_TOO_LARGE)
    return int(load().sa_paged_attn_workspace_size(PagedShape(S, T, Hq, Hkv, d, page, P, max_pages)))


def paged_attn_fwd(Q: torch.Tensor, Kcache: torch.Tensor, Vcache: torch.Tensor, table: torch.Tensor,
                   q_start: torch.Tensor, kv_len: torch.Tensor, scale: float, *, window: int = 0, out=None,
                   workspace=None, stream=None) -> torch.Tensor:
    """Causal (and, with ``window`` > 0, sliding-window) attention of the packed
    rows Q [T,Hq,d] over their requests' pages; returns O [T,Hq,d], in which
    the rows from q_start[S] on are not written.  Chunks of prompts and
    single decoded tokens may share a call."""
    T, Hq, d = Q.shape
    P, Hkv, page, dc = Kcache.shape
    (S,), (rows, width) = kv_len.shape, table.shape
    if Vcache.shape != Kcache.shape or dc != d:
        raise ValueError("the caches must be [P,Hkv,page,d] with Q's d")
    if rows != S or q_start.shape != (S + 1,):
        raise ValueError("q_start must be [S + 1], kv_len [S], table [S, max_pages]")
    if not 0 <= window < 1 << 31:
        raise ValueError("window must be 0 (none) or a number of keys below 2^31")
    if (T | width) >> 31:
        raise ValueError(_TOO_LARGE)
    i, dt, ptr, lib = Q.get_device(), Q.dtype, _paged_ptr, load()
    if out is None:
        out = _paged_empty(Q, (T, Hq, d), dt, stream)
    elif out.shape != Q.shape:
        raise ValueError("out must have Q's shape")
    shape = PagedShape(S, T, Hq, Hkv, d, page, P, width)
    if workspace is None:
        workspace = _paged_empty(Q, max(lib.sa_paged_attn_workspace_size(shape), 256), _U8, stream)
    _paged_call(i, stream, "sa_paged_attn_fwd", lib.sa_paged_attn_fwd, ptr(Q, i, dt, "Q", False), _paged_rows(Q, "Q"),
                ptr(Kcache, i, dt, "Kcache"), ptr(Vcache, i, dt, "Vcache"), _dtype_code(Q), shape,
                ptr(q_start, i, _I32, "q_start"), ptr(kv_len, i, _I32, "kv_len"), ptr(table, i, _I32, "table"),
                window, scale, ptr(out, i, dt, "out"), ptr(workspace, i, _U8, "workspace"), workspace.numel())
    return out
