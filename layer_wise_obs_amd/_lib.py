"""ctypes binding of libthanos (include/thanos.h): argument marshalling only.

Every step of the pruning path runs in the HIP library. Tensors provide device
memory and the current stream; nothing here computes on the CPU. If the library
has not been built, loading raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libthanos.so")

TH_OK, TH_ERR_INVALID_ARG, TH_ERR_NOT_SPD, TH_ERR_NONFINITE, TH_ERR_WORKSPACE, TH_ERR_HIP = range(6)
TH_F32, TH_BF16 = 0, 1
TH_UNSTRUCTURED, TH_NM = 0, 1
TH_SCORE_OBS, TH_SCORE_WANDA = 0, 1
TH_BASE_MAGNITUDE, TH_BASE_WANDA = 0, 1
TH_ACT_NONE, TH_ACT_RELU, TH_ACT_SILU, TH_ACT_GELU = range(4)
TH_ROTARY_HALF, TH_ROTARY_INTERLEAVED = 0, 1
TH_MX_E4M3, TH_MX_E2M1 = 0, 1
STATUS_NAMES = {0: "TH_OK", 1: "TH_ERR_INVALID_ARG", 2: "TH_ERR_NOT_SPD", 3: "TH_ERR_NONFINITE",
                4: "TH_ERR_WORKSPACE", 5: "TH_ERR_HIP"}


class ThanosError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class Pattern(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("n", ctypes.c_int32), ("m", ctypes.c_int32)]


class PruneParams(ctypes.Structure):
    _fields_ = [("sparsity", ctypes.c_double), ("pattern", Pattern), ("block", ctypes.c_int64),
                ("lam", ctypes.c_double), ("lambda_is_relative", ctypes.c_int32),
                ("score", ctypes.c_int32)]


class Stats(ctypes.Structure):
    _fields_ = [("lambda_used", ctypes.c_double), ("total_pruned", ctypes.c_int64),
                ("nblocks", ctypes.c_int64)]


class Heads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("norm", ctypes.c_void_p),
                ("heads", ctypes.c_int64), ("x_token", ctypes.c_int64), ("x_head", ctypes.c_int64),
                ("y_token", ctypes.c_int64), ("y_head", ctypes.c_int64)]


class RotaryScaling(ctypes.Structure):
    _fields_ = [("base", ctypes.c_double), ("divide", ctypes.c_double),
                ("original_length", ctypes.c_double), ("slow_turns", ctypes.c_double),
                ("fast_turns", ctypes.c_double), ("by_bands", ctypes.c_int32)]


class AttentionParams(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in (
        "nq", "nk", "hq", "hk", "d", "q_token", "q_head", "k_token", "k_head", "v_token", "v_head",
        "o_token", "o_head", "nseq")] + [("causal", ctypes.c_int32), ("scale", ctypes.c_double)]


class Mx(ctypes.Structure):
    _fields_ = [("elements", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("lds", ctypes.c_int64), ("type", ctypes.c_int32)]


class PagedCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p)] + [(x, ctypes.c_int64) for x in (
        "npages", "page_tokens", "hk", "d", "k_page", "k_token", "k_head", "v_page", "v_token",
        "v_head")] + [("pages", ctypes.c_void_p), ("k_len", ctypes.c_void_p)] + [
        (x, ctypes.c_int64) for x in ("nseq", "width", "pages_row")]


class PagedParams(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in ("nq", "hq", "q_token", "q_head", "o_token", "o_head")] + [
        ("causal", ctypes.c_int32), ("even", ctypes.c_int32), ("scale", ctypes.c_double)]


_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SIG = {
    "th_hessian_accumulate": [_P, _P, _I32, _I64, _I64, _I64, _P, ctypes.c_size_t, _P],
    "th_hessian_workspace_size": [_I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "th_hessian_finalize": [_P, _I64, ctypes.c_double, _I32, ctypes.POINTER(ctypes.c_double), _P],
    "th_prune_layer": [_P, _I32, _I64, _I64, _P, _I32, _I64, _P, ctypes.POINTER(PruneParams), _P,
                       _P, _P, ctypes.c_size_t, ctypes.POINTER(Stats), ctypes.POINTER(_I64), _P],
    "th_prune_layer_workspace_size": [_I64, _I64, _I64, _I32, ctypes.POINTER(PruneParams),
                                      ctypes.POINTER(ctypes.c_size_t)],
    "th_prune_layer_noalloc": [_P, _I32, _I64, _I64, _P, _I32, _I64, _P,
                               ctypes.POINTER(PruneParams), _P, _P, ctypes.POINTER(Stats),
                               ctypes.POINTER(_I64), _P],
    "th_factor": [_P, _I32, _I64, _P, _I64, ctypes.c_double, _I32, _P,
                  ctypes.POINTER(ctypes.c_double), _P, ctypes.c_size_t, _P],
    "th_factor_workspace_size": [_I64, _I64, _I32, ctypes.POINTER(ctypes.c_size_t)],
    "th_prune_layer_factored": [_P, _I32, _I64, _I64, _P, ctypes.POINTER(PruneParams), _P, _P, _P,
                                ctypes.c_size_t, ctypes.POINTER(Stats), ctypes.POINTER(_I64), _P],
    "th_prune_layer_factored_workspace_size": [_I64, _I64, ctypes.POINTER(PruneParams),
                                               ctypes.POINTER(ctypes.c_size_t)],
    "th_prune_layer_alpha": [_P, _I32, _I64, _I64, _P, _I32, _I64, _P, ctypes.POINTER(PruneParams),
                             ctypes.c_double, _P, _P, _P, _P, ctypes.c_size_t, ctypes.POINTER(Stats),
                             ctypes.POINTER(_I64), _P],
    "th_prune_layer_alpha_workspace_size": [_I64, _I64, _I64, _I32, ctypes.POINTER(PruneParams),
                                            ctypes.c_double, ctypes.POINTER(ctypes.c_size_t)],
    "th_gated_ffn_input": [_P, _P, _P, _I32, _I64, _I64, _I64, _P, _P],
    "th_linear_workspace_size": [_I64, _I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "th_linear": [_P, _I64, _P, _I32, _I64, _I64, _I64, _P, _I32, _P, _I64, _P, _I32, _I64, _P,
                  ctypes.c_size_t, _P],
    "th_rms_norm": [_P, _I32, _I64, _I64, _I64, _P, ctypes.c_double, _P, _I32, _I64, _P],
    "th_rotary": [ctypes.POINTER(Heads), ctypes.POINTER(Heads), _I32, _I64, _I64, _I64, _I32, _P,
                  _P, ctypes.c_double, ctypes.c_double, _P],
    "th_rotary_freqs": [_I64, ctypes.POINTER(RotaryScaling), ctypes.POINTER(ctypes.c_double)],
    "th_attention_workspace_size": [ctypes.POINTER(AttentionParams),
                                    ctypes.POINTER(ctypes.c_size_t)],
    "th_attention": [_P, _P, _P, _I32, _P, _P, ctypes.POINTER(AttentionParams), _P, _P,
                     ctypes.c_size_t, _P],
    "th_mx_quantize": [_P, _I32, _I64, _I64, _I64, ctypes.POINTER(Mx), _P],
    "th_mx_dequantize": [ctypes.POINTER(Mx), _I64, _I64, _P, _I32, _I64, _P],
    "th_mx_linear_workspace_size": [_I32, _I64, _I64, _I64, _I32, ctypes.POINTER(ctypes.c_size_t)],
    "th_debug_mx_linear_plan": [_I32, _I64, _I64, _I64, _I32, _I32] + [ctypes.POINTER(_I32)] * 3,
    "th_mx_linear": [ctypes.POINTER(Mx), ctypes.POINTER(Mx), _I64, _I64, _I64, _P, _I32, _P, _I64, _P,
                     _I32, _I64, _P, ctypes.c_size_t, _P],
    "th_add_rms_norm": [_P, _I64, _P, _I64, _I32, _I64, _I64, _P, ctypes.c_double, _P, _I64, _P, _I32,
                        _I64, ctypes.POINTER(Mx), _P],
    "th_cache_store": [_P, _I64, _I64, _P, _I64, _I64, _I32, _I64, _P, ctypes.POINTER(PagedCache),
                       _P],
    "th_paged_attention_workspace_size": [ctypes.POINTER(PagedCache), ctypes.POINTER(PagedParams),
                                          ctypes.POINTER(ctypes.c_size_t)],
    "th_paged_attention": [_P, _I32, _P, ctypes.POINTER(PagedCache), ctypes.POINTER(PagedParams), _P,
                           _P, ctypes.c_size_t, _P],
    "th_prune_sparsegpt": [_P, _I32, _I64, _I64, _P, _I32, _I64, _P, ctypes.POINTER(PruneParams),
                           _P, _P, _P, ctypes.c_size_t, ctypes.POINTER(Stats),
                           ctypes.POINTER(_I64), _P],
    "th_prune_sparsegpt_workspace_size": [_I64, _I64, _I64, _I32, ctypes.POINTER(PruneParams),
                                          ctypes.POINTER(ctypes.c_size_t)],
    "th_reconstruction_error": [_P, _P, _I32, _I64, _I64, _P, _I32, _I64, _P, _P, ctypes.c_size_t,
                                ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
                                _P],
    "th_reconstruction_error_workspace_size": [_I64, _I64, _I32, ctypes.POINTER(ctypes.c_size_t)],
    "th_debug_select_nm": [_P, _I64, _I64, _I32, _I32, _P, _P],
    "th_debug_select_global": [_P, _I64, _I64, _I64, _I64, _I64, _I64, _P, _P, _P,
                               ctypes.c_size_t, _P],
    "th_debug_factor": [_P, _I64, _P, _P, ctypes.c_size_t, _P],
    "th_debug_syrk_rect": [_P, _P, _I64, _I64, _I64, _I32, _I32, _P, ctypes.c_size_t, _P],
    "th_debug_far_update": [_P, _I64, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P,
                            ctypes.c_size_t, _P],
    "th_column_sq_norms_workspace_size": [_I64, _I64, ctypes.POINTER(ctypes.c_size_t)],
    "th_column_sq_norms": [_P, _I32, _I64, _I64, _I64, _P, _P, ctypes.c_size_t, _P],
    "th_prune_baseline": [_P, _I32, _I64, _I64, _I32, _P, ctypes.POINTER(PruneParams), _P, _P],
}

_lib = None


def lib() -> ctypes.CDLL:
    """Load libthanos.so from the package directory (raises if it is missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run `python -m layer_wise_obs_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIG.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.th_last_error.argtypes = []
        L.th_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(status: int):
    if status != TH_OK:
        raise ThanosError(status, lib().th_last_error().decode())


# ------------------------------------------------------------------ helpers

def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return TH_BF16
    if t.dtype == torch.float32:
        return TH_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(device=None):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must live on the GPU")
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _device_index(t) -> int:
    """GPU that the forward steps' call runs on: the one its first tensor lives on."""
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must live on the GPU")
    return index


def _require(index, name, t, shape, dtype):
    """Strides of a tensor of the forward steps: on GPU index, of this shape and dtype, its last
    dimension contiguous (any outer strides)."""
    strides = t.stride()
    if (t.get_device() == index and t.shape == shape and t.dtype == dtype
            and (strides[-1] == 1 or shape[-1] <= 1)):
        return strides
    if t.get_device() != index:
        raise ValueError(f"{name} must live on GPU {index}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    raise ValueError(f"the last dimension of {name} must be contiguous")


def _fresh(torch, t, dtype=None):
    """A new dense tensor of t's shape, dtype (or this one) and GPU; less host time than
    torch.empty with a shape."""
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _row_pitch(strides, n, dense):
    """Row stride of a tensor [n, dense]; a single row's, which no access uses, is given as the
    dense one."""
    return strides[0] if n > 1 else dense


def _addr(t):
    return None if t is None else t.data_ptr()


def _call_on(index, fn, *args):
    """Call fn with GPU index current, on that GPU's current stream (its last argument)."""
    torch = _torch()
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _check(fn(*args, torch.cuda.current_stream(index).cuda_stream))
    _check(fn(*args, torch._C._cuda_getCurrentRawStream(index)))


def _workspace_on(index, ws):
    """(address, bytes) of a caller's workspace tensor."""
    if ws.get_device() != index:
        raise ValueError(f"ws must live on GPU {index}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def make_params(sparsity=0.5, pattern=None, block=128, lam=0.01, relative=True,
                score="obs") -> PruneParams:
    p = PruneParams()
    p.sparsity = float(sparsity)
    if pattern is None:
        p.pattern = Pattern(TH_UNSTRUCTURED, 0, 0)
    else:
        p.pattern = Pattern(TH_NM, int(pattern[0]), int(pattern[1]))
    p.block = int(block)
    p.lam = float(lam)
    p.lambda_is_relative = 1 if relative else 0
    p.score = {"obs": TH_SCORE_OBS, "wanda": TH_SCORE_WANDA}[score]
    return p


def workspace(nbytes: int, device):
    torch = _torch()
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- entry points

def hessian_workspace_size(t: int, b: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().th_hessian_workspace_size(t, b, ctypes.byref(out)))
    return out.value


def hessian_accumulate(H, X, ws=None):
    """H (b x b fp32, lower) += 2 X^T X for token-major X [t, b]."""
    _require_cuda(H, X)
    t, b = X.shape
    _check(lib().th_hessian_accumulate(_ptr(H), _ptr(X), _dtype_code(X), t, b, X.stride(0),
                                       _ptr(ws), 0 if ws is None else ws.numel(),
                                       _stream(X.device)))


def hessian_finalize(H, lam=0.01, relative=True) -> float:
    _require_cuda(H)
    out = ctypes.c_double(0.0)
    _check(lib().th_hessian_finalize(_ptr(H), H.shape[0], float(lam), 1 if relative else 0,
                                     ctypes.byref(out), _stream(H.device)))
    return out.value


def prune_layer_workspace_size(c, b, n, have_x, params: PruneParams) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().th_prune_layer_workspace_size(c, b, n, 1 if have_x else 0, ctypes.byref(params),
                                               ctypes.byref(out)))
    return out.value


def _layer_call(entry, size_entry, W, X, H, params, W_out, mask_out, ws) -> dict:
    _require_cuda(W, X, H, W_out, mask_out)
    if params is None:
        params = make_params()
    c, b = W.shape
    n = X.shape[0] if X is not None else 0
    if ws is None:
        out = ctypes.c_size_t(0)
        _check(size_entry(c, b, n, 1 if X is not None else 0, ctypes.byref(params),
                          ctypes.byref(out)))
        ws = workspace(out.value, W.device)
    stats = Stats()
    nblk = -(-b // params.block)
    counts = (_I64 * nblk)()
    _check(entry(_ptr(W), _dtype_code(W), c, b, _ptr(X), _dtype_code(X) if X is not None else 0,
                 n, _ptr(H), ctypes.byref(params), _ptr(W_out), _ptr(mask_out), _ptr(ws),
                 ws.numel(), ctypes.byref(stats), counts, _stream(W.device)))
    return {"lambda": stats.lambda_used, "pruned": stats.total_pruned, "nblocks": stats.nblocks,
            "counts": list(counts)}


def prune_layer(W, X=None, H=None, params: PruneParams | None = None, W_out=None, mask_out=None,
                ws=None) -> dict:
    """Prune W (c x b, bf16/fp32) in place; returns stats and per-block counts."""
    return _layer_call(lib().th_prune_layer, lib().th_prune_layer_workspace_size, W, X, H,
                       params, W_out, mask_out, ws)


NOALLOC_SCRATCH_BYTES = 64 << 20  # TH_NOALLOC_SCRATCH_BYTES in include/thanos.h


def prune_layer_noalloc(W, X=None, H=None, params: PruneParams | None = None, W_out=None,
                        mask_out=None) -> dict:
    """th_prune_layer_noalloc: the layer step in the library's fixed scratch array
    (no workspace, nothing allocated); same results as prune_layer."""
    _require_cuda(W, X, H, W_out, mask_out)
    if params is None:
        params = make_params()
    c, b = W.shape
    n = X.shape[0] if X is not None else 0
    stats = Stats()
    counts = (_I64 * (-(-b // params.block)))()
    _check(lib().th_prune_layer_noalloc(
        _ptr(W), _dtype_code(W), c, b, _ptr(X), _dtype_code(X) if X is not None else 0, n,
        _ptr(H), ctypes.byref(params), _ptr(W_out), _ptr(mask_out), ctypes.byref(stats), counts,
        _stream(W.device)))
    return {"lambda": stats.lambda_used, "pruned": stats.total_pruned, "nblocks": stats.nblocks,
            "counts": list(counts)}


def factor(X=None, H=None, lam=0.01, relative=True, U=None, ws=None):
    """U (b x b fp32, upper) with H^-1 = U^T U from X [n, b] or a damped H; returns (U, lambda)."""
    torch = _torch()
    _require_cuda(X, H, U)
    b = X.shape[1] if X is not None else H.shape[0]
    dev = (X if X is not None else H).device
    n = X.shape[0] if X is not None else 0
    if U is None:
        U = torch.empty((b, b), dtype=torch.float32, device=dev)
    if ws is None:
        out = ctypes.c_size_t(0)
        _check(lib().th_factor_workspace_size(b, n, 1 if X is not None else 0, ctypes.byref(out)))
        ws = workspace(out.value, dev)
    lam_out = ctypes.c_double(0.0)
    _check(lib().th_factor(_ptr(X), _dtype_code(X) if X is not None else 0, n, _ptr(H), b,
                           float(lam), 1 if relative else 0, _ptr(U), ctypes.byref(lam_out),
                           _ptr(ws), ws.numel(), _stream(dev)))
    return U, lam_out.value


def prune_layer_factored(W, U, params: PruneParams | None = None, W_out=None, mask_out=None,
                         ws=None) -> dict:
    """prune_layer from a factor U that layers sharing one input reuse."""
    _require_cuda(W, U, W_out, mask_out)
    if params is None:
        params = make_params()
    c, b = W.shape
    if ws is None:
        out = ctypes.c_size_t(0)
        _check(lib().th_prune_layer_factored_workspace_size(c, b, ctypes.byref(params),
                                                            ctypes.byref(out)))
        ws = workspace(out.value, W.device)
    stats = Stats()
    counts = (_I64 * (-(-b // params.block)))()
    _check(lib().th_prune_layer_factored(_ptr(W), _dtype_code(W), c, b, _ptr(U),
                                         ctypes.byref(params), _ptr(W_out), _ptr(mask_out),
                                         _ptr(ws), ws.numel(), ctypes.byref(stats), counts,
                                         _stream(W.device)))
    return {"lambda": stats.lambda_used, "pruned": stats.total_pruned, "nblocks": stats.nblocks,
            "counts": list(counts)}


def prune_layer_alpha(W, alpha: float, X=None, H=None, params: PruneParams | None = None,
                      W_out=None, mask_out=None, dense_out=None, ws=None) -> dict:
    """prune_layer with round(alpha c) rows of largest output energy kept dense."""
    _require_cuda(W, X, H, W_out, mask_out, dense_out)
    if params is None:
        params = make_params()
    c, b = W.shape
    n = X.shape[0] if X is not None else 0
    if ws is None:
        out = ctypes.c_size_t(0)
        _check(lib().th_prune_layer_alpha_workspace_size(c, b, n, 1 if X is not None else 0,
                                                         ctypes.byref(params), float(alpha),
                                                         ctypes.byref(out)))
        ws = workspace(out.value, W.device)
    stats = Stats()
    counts = (_I64 * (-(-b // params.block)))()
    _check(lib().th_prune_layer_alpha(_ptr(W), _dtype_code(W), c, b, _ptr(X),
                                      _dtype_code(X) if X is not None else 0, n, _ptr(H),
                                      ctypes.byref(params), float(alpha), _ptr(W_out),
                                      _ptr(mask_out), _ptr(dense_out), _ptr(ws), ws.numel(),
                                      ctypes.byref(stats), counts, _stream(W.device)))
    return {"lambda": stats.lambda_used, "pruned": stats.total_pruned, "nblocks": stats.nblocks,
            "counts": list(counts)}


def gated_ffn_input(X, W_gate, W_up, Y=None):
    """Y = silu(X W_gate^T) * (X W_up^T) in bf16 for X [n, d], W [f, d] (bf16)."""
    torch = _torch()
    _require_cuda(X, W_gate, W_up, Y)
    n, d = X.shape
    f = W_gate.shape[0]
    if Y is None:
        Y = torch.empty((n, f), dtype=torch.bfloat16, device=X.device)
    _check(lib().th_gated_ffn_input(_ptr(X), _ptr(W_gate), _ptr(W_up), _dtype_code(X), n, d, f,
                                    _ptr(Y), _stream(X.device)))
    return Y


def linear_workspace_size(n: int, b: int, c: int) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().th_linear_workspace_size(n, b, c, ctypes.byref(out)))
    return out.value


_ACTIVATIONS = {"none": TH_ACT_NONE, "relu": TH_ACT_RELU, "silu": TH_ACT_SILU,
                "gelu": TH_ACT_GELU}


def linear(X, W, bias=None, act="none", residual=None, Y=None, out_dtype=None, ws=None):
    """Y = act(X W^T + bias) + residual for X [n, b], W [c, b] and bias [c] (bf16); residual and
    Y [n, c] in out_dtype (bf16 or fp32, default the residual's or X's). Y may be the residual.
    Forward only, like the steps below: Y carries no gradient, whatever X and W require."""
    torch = _torch()
    index = _device_index(X)
    n, b = X.shape
    c = W.shape[0]
    if out_dtype is None:
        out_dtype = next((t.dtype for t in (Y, residual) if t is not None), X.dtype)
    ldx = _row_pitch(_require(index, "X", X, (n, b), X.dtype), n, b)
    _require(index, "W", W, (c, b), X.dtype)
    if not W.is_contiguous():
        raise ValueError("W must be contiguous")
    if bias is not None:
        _require(index, "bias", bias, (c,), X.dtype)
    ldr = ldy = c
    if residual is not None:
        ldr = _row_pitch(_require(index, "residual", residual, (n, c), out_dtype), n, c)
    if Y is None:
        Y = (torch.empty((n, c), dtype=out_dtype, device=X.device) if residual is None
             else _fresh(torch, residual))
    else:
        ldy = _row_pitch(_require(index, "Y", Y, (n, c), out_dtype), n, c)
    if ws is None:
        nbytes = linear_workspace_size(n, b, c)
        ws = workspace(nbytes, X.device) if nbytes else None
    at, nbytes = (None, 0) if ws is None else _workspace_on(index, ws)
    _call_on(index, lib().th_linear, X.data_ptr(), ldx, W.data_ptr(), _dtype_code(X), n, b, c,
             _addr(bias), _ACTIVATIONS[act], _addr(residual), ldr, Y.data_ptr(), _dtype_code(Y),
             ldy, at, nbytes)
    return Y


def rms_norm(X, weight, eps=1e-5, Y=None, out_dtype=None):
    """Y = X / sqrt(mean(X^2) + eps) * weight by rows, X [n, b]; Y in out_dtype (default X's).
    Y may be X. Forward only: Y carries no gradient."""
    torch = _torch()
    index = _device_index(X)
    n, b = X.shape
    ldx = _row_pitch(_require(index, "X", X, (n, b), X.dtype), n, b)
    _require(index, "weight", weight, (b,), X.dtype)
    ldy = b
    if Y is None:
        Y = _fresh(torch, X, out_dtype)
    else:
        ldy = _row_pitch(_require(index, "Y", Y, (n, b), out_dtype or Y.dtype), n, b)
    _call_on(index, lib().th_rms_norm, X.data_ptr(), _dtype_code(X), n, b, ldx, weight.data_ptr(),
             float(eps), Y.data_ptr(), _dtype_code(Y), ldy)
    return Y


_MX_TYPES = {"e4m3": TH_MX_E4M3, "e2m1": TH_MX_E2M1}


class MxMatrix:
    """A microscaled matrix [n, b]: its type ("e4m3" or "e2m1"), elements (uint8 [n, b], or
    [n, b / 2] with element 2i in the low half of byte i) and scales (uint8 [n, b / 32]); a value is
    its element times 2^(scale - 127) of its 32. The scales' rows are a multiple of 16 bytes apart
    where mx_linear is to read them, and their memory holds the last (or only) row up to the next
    multiple of 16 too."""
    __slots__ = ("type", "_elements", "_scales", "_new", "_host")

    def __init__(self, type, elements, scales):
        if type not in _MX_TYPES:
            raise ValueError(f"type must be one of {sorted(_MX_TYPES)}, not {type!r}")
        self.type, self._elements, self._scales = type, elements, scales
        self._new = self._host = None

    @classmethod
    def empty(cls, n, b, type, device):
        """A new one, both parts in one allocation, with its host struct; the tensors are made when
        they are asked for (2 us less on the way to a kernel)."""
        torch = _torch()
        if type not in _MX_TYPES:
            raise ValueError(f"type must be one of {sorted(_MX_TYPES)}, not {type!r}")
        if b % 32:
            raise ValueError(f"b must be a multiple of 32, not {b}")
        width = b if type == "e4m3" else b // 2
        pitch = -(-b // 512) * 16
        m = cls.__new__(cls)
        m.type, m._elements, m._scales = type, None, None
        buf = torch.empty(n * (width + pitch), dtype=torch.uint8, device=device)
        m._new, at = (buf, n, b, width, pitch), buf.data_ptr()
        # its scales begin 16-byte aligned: rows of 16 bytes and more before them
        m._host = Mx(at, at + n * width, width, pitch, _MX_TYPES[type])
        return m

    @property
    def elements(self):
        if self._elements is None:
            buf, n, _, width, _ = self._new
            self._elements = buf.as_strided((n, width), (width, 1))
        return self._elements

    @property
    def scales(self):
        if self._scales is None:
            buf, n, b, width, pitch = self._new
            self._scales = buf.as_strided((n, b // 32), (pitch, 1), n * width)
        return self._scales

    @property
    def shape(self):
        if self._new is not None:
            return self._new[1:3]
        n, width = self._elements.shape
        return n, width if self.type == "e4m3" else 2 * width

    @property
    def device(self):
        return (self._elements if self._new is None else self._new[0]).device


def _mx_index(m) -> int:
    return _device_index(m._elements if m._new is None else m._new[0])


def _mx(index, name, m, product=False):
    """(n, b, host struct) of a microscaled matrix on GPU index; a product reads its rows of scales
    up to the next multiple of 16 bytes, the last one's too."""
    if m._new is not None:
        buf, n, b, _, _ = m._new
        if buf.get_device() != index:
            raise ValueError(f"{name} must live on GPU {index}")
        return n, b, m._host
    torch = _torch()
    n, width = m._elements.shape
    b = width if m.type == "e4m3" else 2 * width
    e = _require(index, name + ".elements", m._elements, m._elements.shape, torch.uint8)[0]
    s = _require(index, name + ".scales", m._scales, (n, b // 32), torch.uint8)[0]
    if n == 1:  # a single row's pitches, which no access uses: multiples of 16 that hold it
        e, s = -(-width // 16) * 16, -(-b // 512) * 16
    if product and b % 512 and n:
        t, row = m._scales, -(-b // 512) * 16
        if t.storage_offset() + (n - 1) * t.stride(0) + row > t.untyped_storage().nbytes():
            raise ValueError(f"{name}.scales must have memory for {row} bytes of the last row")
    return n, b, Mx(m._elements.data_ptr(), m._scales.data_ptr(), e, s, _MX_TYPES[m.type])


def mx_quantize(X, type="e2m1", out=None):
    """X [n, b] (bf16 or fp32, b a multiple of 32) as a new microscaled matrix, or in out: a block's
    scale is the smallest power at which none of its elements passes the type's largest number;
    elements rounded to nearest even. A block with a NaN or an infinity holds no numbers."""
    index = _device_index(X)
    n, b = X.shape
    ldx = _row_pitch(_require(index, "X", X, (n, b), X.dtype), n, b)
    if out is None:
        out = MxMatrix.empty(n, b, type, X.device)
    no, bo, y = _mx(index, "out", out)
    if (no, bo) != (n, b):
        raise ValueError(f"out must have shape {(n, b)}, not {(no, bo)}")
    _call_on(index, lib().th_mx_quantize, X.data_ptr(), _dtype_code(X), n, b, ldx, y)
    return out


def mx_dequantize(X, Y=None, out_dtype=None):
    """The values of a microscaled matrix, Y [n, b] in out_dtype (default bf16)."""
    torch = _torch()
    index = _mx_index(X)
    n, b, x = _mx(index, "X", X)
    ldy = b
    if Y is None:
        Y = torch.empty((n, b), dtype=out_dtype or torch.bfloat16, device=X.device)
    else:
        ldy = _row_pitch(_require(index, "Y", Y, (n, b), out_dtype or Y.dtype), n, b)
    _call_on(index, lib().th_mx_dequantize, x, n, b, Y.data_ptr(), _dtype_code(Y), ldy)
    return Y


@functools.lru_cache(maxsize=1024)
def mx_linear_workspace_size(type: str, n: int, b: int, c: int, out_dtype) -> int:
    """Kept by its sizes, of which it is a function."""
    torch = _torch()
    out = ctypes.c_size_t(0)
    _check(lib().th_mx_linear_workspace_size(_MX_TYPES[type], n, b, c,
                                             TH_F32 if out_dtype == torch.float32 else TH_BF16,
                                             ctypes.byref(out)))
    return out.value


def debug_mx_linear_plan(type: str, n: int, b: int, c: int, out_dtype, ws=True):
    """(tokens, channels, pieces): the tile of a workgroup and the pieces of the contraction that a
    product of these sizes runs on, with a workspace or without one."""
    out = [_I32(0) for _ in range(3)]
    _check(lib().th_debug_mx_linear_plan(_MX_TYPES[type], n, b, c,
                                         TH_F32 if out_dtype == _torch().float32 else TH_BF16,
                                         1 if ws else 0, *(ctypes.byref(v) for v in out)))
    return tuple(v.value for v in out)


def mx_linear(X, W, bias=None, act="none", residual=None, Y=None, out_dtype=None, ws=None):
    """Y = act(X W^T + bias) + residual for microscaled X [n, b] (either type) and W [c, b]
    ("e2m1"), bias [c] bf16; residual and Y [n, c] in out_dtype (bf16 or fp32, default the
    residual's or bf16). Y may be the residual. Forward only."""
    torch = _torch()
    index = _mx_index(X)
    n, b, x = _mx(index, "X", X, True)
    c, bw, w = _mx(index, "W", W, True)
    if bw != b:
        raise ValueError(f"W must have {b} columns, not {bw}")
    if out_dtype is None:
        out_dtype = next((t.dtype for t in (Y, residual) if t is not None), torch.bfloat16)
    if bias is not None:
        _require(index, "bias", bias, (c,), torch.bfloat16)
    ldr = ldy = c
    if residual is not None:
        ldr = _row_pitch(_require(index, "residual", residual, (n, c), out_dtype), n, c)
    if Y is None:
        Y = (torch.empty((n, c), dtype=out_dtype, device=X.device) if residual is None
             else _fresh(torch, residual))
    else:
        ldy = _row_pitch(_require(index, "Y", Y, (n, c), out_dtype), n, c)
    if ws is None:
        nbytes = mx_linear_workspace_size(X.type, n, b, c, out_dtype)
        ws = workspace(nbytes, X.device) if nbytes else None
    at, nbytes = (None, 0) if ws is None else _workspace_on(index, ws)
    _call_on(index, lib().th_mx_linear, x, w, n, b, c, _addr(bias), _ACTIVATIONS[act],
             _addr(residual), ldr, Y.data_ptr(), _dtype_code(Y), ldy, at, nbytes)
    return Y


def add_rms_norm(X, weight, residual=None, eps=1e-5, out=None, sum_out=None):
    """(h, Y): h = X + residual in X's dtype (a new tensor, or sum_out, which may be X or the
    residual; X itself without a residual) and Y = h / sqrt(mean(h^2) + eps) * weight by rows.
    out: "e4m3", "e2m1" or a MxMatrix for a microscaled Y; a dtype or a tensor for a plain one
    (default X's dtype). Forward only."""
    torch = _torch()
    index = _device_index(X)
    n, b = X.shape
    dtype = X.dtype
    ldx = _row_pitch(_require(index, "X", X, (n, b), dtype), n, b)
    _require(index, "weight", weight, (b,), dtype)
    ldr = ldsum = ldy = b
    h = X
    if residual is not None:
        ldr = _row_pitch(_require(index, "residual", residual, (n, b), dtype), n, b)
        if sum_out is None:
            h = _fresh(torch, X)
        else:
            h = sum_out
            ldsum = _row_pitch(_require(index, "sum_out", h, (n, b), dtype), n, b)
    elif sum_out is not None:
        raise ValueError("sum_out goes with residual")
    Y, y, mx, code = None, None, None, TH_BF16
    if isinstance(out, str):
        out = MxMatrix.empty(n, b, out, X.device)
    if isinstance(out, MxMatrix):
        Y = out
        no, bo, mx = _mx(index, "out", out)
        if (no, bo) != (n, b):
            raise ValueError(f"out must have shape {(n, b)}, not {(no, bo)}")
    else:
        if out is None or isinstance(out, torch.dtype):
            Y = _fresh(torch, X, out)
        else:
            Y = out
            ldy = _row_pitch(_require(index, "out", Y, (n, b), Y.dtype), n, b)
        y, code = Y.data_ptr(), _dtype_code(Y)
    _call_on(index, lib().th_add_rms_norm, X.data_ptr(), ldx, _addr(residual), ldr, _dtype_code(X), n,
             b, weight.data_ptr(), float(eps), None if residual is None else h.data_ptr(), ldsum, y,
             code, ldy, mx)
    return h, Y


def rotary_freqs(rot: int, base=10000.0, divide=1.0, bands=None, device=None):
    """Frequencies of the rot/2 pairs (float64, rot/2 values, on device) for rotary().

    divide: every frequency is divided by it; with bands = (original_length, slow_turns,
    fast_turns) only those of pairs that turn slowly over the original length are."""
    torch = _torch()
    length, slow, fast = bands if bands is not None else (0.0, 0.0, 0.0)
    g = RotaryScaling(float(base), float(divide), float(length), float(slow), float(fast),
                      0 if bands is None else 1)
    out = (ctypes.c_double * max(rot // 2, 1))()
    _check(lib().th_rotary_freqs(rot, ctypes.byref(g), out))
    return torch.tensor(out[:rot // 2], dtype=torch.float64, device=device)


_ROTARY_LAYOUTS = {"half": TH_ROTARY_HALF, "interleaved": TH_ROTARY_INTERLEAVED}


def _pitches(strides, n, h, d):
    """Token and head strides of a tensor [n, h, d]; those of a dimension of one element, which
    no access uses, are given as the dense ones."""
    return strides[0] if n > 1 else h * d, strides[1] if h > 1 else d


def rotary(q, k, freqs, positions=None, layout="half", amplitude=1.0, q_norm=None, k_norm=None,
           eps=1e-6, q_out=None, k_out=None):
    """Heads q [n, hq, d] and k [n, hk, d] (or None) normed where a weight is given, then their
    first 2 * len(freqs) elements turned by positions * freqs (positions: int32 [n], default
    0 .. n-1). Returns (q_out, k_out), which may be q and k themselves. Forward only: they carry
    no gradient."""
    torch = _torch()
    index = _device_index(q)
    n, _, d = q.shape
    dtype = q.dtype

    def heads(name, x, out, norm):
        h = x.shape[1]
        strides = _require(index, name, x, (n, h, d), dtype)
        if norm is not None:
            _require(index, name + "_norm", norm, (d,), dtype)
        if out is None:
            out = _fresh(torch, x)
            out_pitches = h * d, d
        else:
            out_pitches = _pitches(_require(index, name + "_out", out, (n, h, d), dtype), n, h, d)
        return out, Heads(x.data_ptr(), out.data_ptr(), _addr(norm), h,
                          *_pitches(strides, n, h, d), *out_pitches)

    pairs = freqs.shape[0]
    _require(index, "freqs", freqs, (pairs,), torch.float64)
    if positions is not None:
        _require(index, "positions", positions, (n,), torch.int32)
    q_out, qh = heads("q", q, q_out, q_norm)
    kh = None
    if k is not None:
        k_out, kh = heads("k", k, k_out, k_norm)
    elif k_out is not None or k_norm is not None:
        raise ValueError("k_out and k_norm go with k")
    _call_on(index, lib().th_rotary, qh, kh, _dtype_code(q), n, d, 2 * pairs,
             _ROTARY_LAYOUTS[layout], _addr(positions), freqs.data_ptr(), float(amplitude),
             float(eps))
    return q_out, k_out


def attention_workspace_size(params: AttentionParams) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().th_attention_workspace_size(ctypes.byref(params), ctypes.byref(out)))
    return out.value


def attention(Q, K, V, q_start=None, k_start=None, causal=True, scale=None, O=None, ws=None):
    """O = softmax(scale Q K^T) V for Q [nq, hq, d], K and V [nk, hk, d] (bf16) of sequences packed
    along the rows: q_start and k_start int32 [nseq + 1] on the GPU (k_start defaults to q_start;
    without q_start all rows are one sequence). scale defaults to 1 / sqrt(d). Rows of O that
    belong to no sequence are not written (in a new O they hold anything). Forward only: O carries
    no gradient."""
    torch = _torch()
    index = _device_index(Q)
    nq, hq, d = Q.shape
    nk, hk, _ = K.shape
    dtype = Q.dtype
    q_s = _pitches(_require(index, "Q", Q, (nq, hq, d), dtype), nq, hq, d)
    k_s = _pitches(_require(index, "K", K, (nk, hk, d), dtype), nk, hk, d)
    v_s = _pitches(_require(index, "V", V, (nk, hk, d), dtype), nk, hk, d)
    if O is None:  # rows that belong to no sequence are not written
        O = _fresh(torch, Q)
        o_s = hq * d, d
    else:
        o_s = _pitches(_require(index, "O", O, (nq, hq, d), dtype), nq, hq, d)
    nseq = 1
    if q_start is not None:
        nseq = q_start.shape[0] - 1
        _require(index, "q_start", q_start, (nseq + 1,), torch.int32)
        if k_start is not None:
            _require(index, "k_start", k_start, (nseq + 1,), torch.int32)
    elif k_start is not None:
        raise ValueError("k_start goes with q_start")
    p = AttentionParams(nq, nk, hq, hk, d, *q_s, *k_s, *v_s, *o_s, nseq, 1 if causal else 0,
                        d ** -0.5 if scale is None else float(scale))
    if ws is None:
        nbytes = attention_workspace_size(p)
        ws = workspace(nbytes, Q.device) if nbytes else None
    at, nbytes = (None, 0) if ws is None else _workspace_on(index, ws)
    _call_on(index, lib().th_attention, Q.data_ptr(), K.data_ptr(), V.data_ptr(), _dtype_code(Q),
             _addr(q_start), _addr(k_start), p, O.data_ptr(), at, nbytes)
    return O


def _paged_cache(index, k_cache, v_cache, pages, k_len):
    """Host struct of a paged cache on GPU index."""
    torch = _torch()
    shape = k_cache.shape
    npages, page, hk, d = shape
    dtype = k_cache.dtype
    kp, kt, kh, _ = _require(index, "k_cache", k_cache, shape, dtype)
    vp, vt, vh, _ = _require(index, "v_cache", v_cache, shape, dtype)
    if npages <= 1:  # strides of a dimension of one element, which no access uses: the dense ones
        kp = vp = page * hk * d
    if hk <= 1:
        kh = vh = d
    nseq, width = pages.shape
    row = _row_pitch(_require(index, "pages", pages, (nseq, width), torch.int32), nseq, width)
    _require(index, "k_len", k_len, (nseq,), torch.int32)
    return PagedCache(k_cache.data_ptr(), v_cache.data_ptr(), npages, page, hk, d, kp, kt, kh, vp, vt,
                      vh, pages.data_ptr(), k_len.data_ptr(), nseq, width, row)


def cache_store(K, V, k_cache, v_cache, pages, k_len, q_start=None):
    """New keys and values K and V [nq, hk, d] (bf16) into the pages of k_cache and v_cache
    [pages, page_tokens, hk, d] (any strides of whole heads): rows q_start[s] .. q_start[s+1]-1 are the
    last keys of sequence s, whose key x is row x % page_tokens of page pages[s, x // page_tokens];
    pages int32 [nseq, width], k_len int32 [nseq] with the new ones counted, q_start int32
    [nseq + 1] (default: nq / nseq rows each). Rows whose key or page is out of range are not
    stored."""
    torch = _torch()
    index = _device_index(K)
    nq, hk, d = K.shape
    dtype = K.dtype
    k_s = _pitches(_require(index, "K", K, (nq, hk, d), dtype), nq, hk, d)
    v_s = _pitches(_require(index, "V", V, (nq, hk, d), dtype), nq, hk, d)
    cache = _paged_cache(index, k_cache, v_cache, pages, k_len)
    if (cache.hk, cache.d) != (hk, d) or k_cache.dtype != dtype:
        raise ValueError("K, V and the cache must have the same heads and dtype")
    if q_start is not None:
        _require(index, "q_start", q_start, (cache.nseq + 1,), torch.int32)
    _call_on(index, lib().th_cache_store, K.data_ptr(), *k_s, V.data_ptr(), *v_s, _dtype_code(K), nq,
             _addr(q_start), cache)


def paged_attention_workspace_size(cache: PagedCache, params: PagedParams) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().th_paged_attention_workspace_size(ctypes.byref(cache), ctypes.byref(params),
                                                   ctypes.byref(out)))
    return out.value


_paged_sizes = {}  # workspace sizes by all sizes that they follow from


def _paged_workspace(cache, p) -> int:
    key = (p.nq, p.hq, p.even, cache.hk, cache.d, cache.nseq, cache.width, cache.page_tokens)
    nbytes = _paged_sizes.get(key)
    if nbytes is None:
        nbytes = paged_attention_workspace_size(cache, p)
        if len(_paged_sizes) >= 1024:
            _paged_sizes.clear()
        _paged_sizes[key] = nbytes
    return nbytes


def paged_attention(Q, k_cache, v_cache, pages, k_len, q_start=None, causal=True, scale=None, O=None,
                    ws=None):
    """attention() of new tokens Q [nq, hq, d] (bf16) over a paged cache that holds their keys (see
    cache_store): rows q_start[s] .. q_start[s+1]-1 (default nq / nseq each) over the k_len[s] keys of
    sequence s, causal to its last key. The lengths stay on the GPU; a narrower view of pages than the
    longest sequence cuts it off. Rows of O that belong to no sequence are not written (in a new O
    they hold anything). Forward only."""
    torch = _torch()
    index = _device_index(Q)
    nq, hq, d = Q.shape
    dtype = Q.dtype
    q_s = _pitches(_require(index, "Q", Q, (nq, hq, d), dtype), nq, hq, d)
    cache = _paged_cache(index, k_cache, v_cache, pages, k_len)
    if cache.d != d or k_cache.dtype != dtype:
        raise ValueError("Q and the cache must have the same elements per head and dtype")
    if O is None:  # rows that belong to no sequence are not written
        O = _fresh(torch, Q)
        o_s = hq * d, d
    else:
        o_s = _pitches(_require(index, "O", O, (nq, hq, d), dtype), nq, hq, d)
    if q_start is not None:
        _require(index, "q_start", q_start, (cache.nseq + 1,), torch.int32)
    p = PagedParams(nq, hq, *q_s, *o_s, 1 if causal else 0, 1 if q_start is None else 0,
                    d ** -0.5 if scale is None else float(scale))
    if ws is None:
        nbytes = _paged_workspace(cache, p)
        ws = workspace(nbytes, Q.device) if nbytes else None
    at, nbytes = (None, 0) if ws is None else _workspace_on(index, ws)
    _call_on(index, lib().th_paged_attention, Q.data_ptr(), _dtype_code(Q), _addr(q_start), cache, p,
             O.data_ptr(), at, nbytes)
    return O


def prune_sparsegpt_workspace_size(c, b, n, have_x, params: PruneParams) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().th_prune_sparsegpt_workspace_size(c, b, n, 1 if have_x else 0,
                                                   ctypes.byref(params), ctypes.byref(out)))
    return out.value


def prune_sparsegpt(W, X=None, H=None, params: PruneParams | None = None, W_out=None,
                    mask_out=None, ws=None) -> dict:
    """The column-sequential comparator on W (c x b) in place; same arguments as prune_layer."""
    return _layer_call(lib().th_prune_sparsegpt, lib().th_prune_sparsegpt_workspace_size, W, X,
                       H, params, W_out, mask_out, ws)


def reconstruction_error(W, W_hat, X=None, G=None, ws=None):
    _require_cuda(W, W_hat, X, G)
    c, b = W.shape
    if ws is None:
        out = ctypes.c_size_t(0)
        _check(lib().th_reconstruction_error_workspace_size(c, b, 1 if X is not None else 0,
                                                            ctypes.byref(out)))
        ws = workspace(out.value, W.device)
    e = ctypes.c_double(0.0)
    r = ctypes.c_double(0.0)
    _check(lib().th_reconstruction_error(_ptr(W), _ptr(W_hat), _dtype_code(W), c, b, _ptr(X),
                                         _dtype_code(X) if X is not None else 0,
                                         X.shape[0] if X is not None else 0, _ptr(G), _ptr(ws),
                                         ws.numel(), ctypes.byref(e), ctypes.byref(r),
                                         _stream(W.device)))
    return e.value, r.value


def debug_select_nm(scores, n: int, m: int):
    torch = _torch()
    _require_cuda(scores)
    c, blk = scores.shape
    mask = torch.empty((c, blk), dtype=torch.uint8, device=scores.device)
    _check(lib().th_debug_select_nm(_ptr(scores), c, blk, n, m, _ptr(mask), _stream(scores.device)))
    return mask


def debug_select_global(scores, b_full: int, j0: int, blk: int, r: int):
    torch = _torch()
    _require_cuda(scores)
    c, f = scores.shape
    mask = torch.empty((c, blk), dtype=torch.uint8, device=scores.device)
    s_k = torch.empty((c,), dtype=torch.int32, device=scores.device)
    ws = workspace(1 << 16, scores.device)
    _check(lib().th_debug_select_global(_ptr(scores), c, f, b_full, j0, blk, r, _ptr(mask),
                                        _ptr(s_k), _ptr(ws), ws.numel(), _stream(scores.device)))
    return mask, s_k


def debug_syrk_rect(H, X, P, m=0):
    """H (b x b fp32, lower) += 2 X^T X through the rectangles: whole tiles in rounds
    of P workgroups, the rest cut into m pieces each (m = 0: chosen)."""
    _require_cuda(H, X)
    t, b = X.shape
    tiles = -(-b // 384) * -(-b // 256)  # bounds the cut tiles
    ws = workspace(tiles * max(m, 16) * 98304 * 4 + 4 * tiles, H.device)
    _check(lib().th_debug_syrk_rect(_ptr(H), _ptr(X), t, b, X.stride(0), P, m, _ptr(ws),
                                    ws.numel(), _stream(X.device)))


def debug_far_update(W, Z, R, r0, K, col0, col_end):
    """W[:, col0:col_end] -= Z[:, :K] R[r0:r0+K, col0:col_end] (split-bf16 planes, 256 tiles)."""
    _require_cuda(W, Z, R)
    c, b = W.shape
    kp = -(-K // 64) * 64
    ybytes = 3 * kp * (-(-c // 256) + -(-(col_end - col0) // 256)) * 256 * 2
    nbytes = -(-ybytes // 256) * 256 + 256 * 256 * 256 * 4  # planes, then 256 piece slots
    ws = workspace(nbytes, W.device)
    _check(lib().th_debug_far_update(_ptr(W), c, b, _ptr(Z), Z.stride(0), _ptr(R), r0, K, col0,
                                     col_end, _ptr(ws), ws.numel(), _stream(W.device)))
    return ws


def debug_factor(H):
    torch = _torch()
    _require_cuda(H)
    b = H.shape[0]
    U = torch.empty_like(H)
    # b*b fp32, two panel buffers, two split panels (3 planes of 256 x ceil(b/256)*256 bf16)
    nbytes = (4 * b * b + 2 * 4 * (-(-b // 128)) * 128 * 256
              + 2 * 2 * 3 * 256 * (-(-b // 256)) * 256 + (1 << 16))
    ws = workspace(nbytes, H.device)
    _check(lib().th_debug_factor(_ptr(H), b, _ptr(U), _ptr(ws), ws.numel(), _stream(H.device)))
    return U


def column_sq_norms(X):
    """G_qq = sum_t X_tq^2 (fp32, b values) for token-major X [n, b]."""
    torch = _torch()
    _require_cuda(X)
    n, b = X.shape
    out = ctypes.c_size_t(0)
    _check(lib().th_column_sq_norms_workspace_size(n, b, ctypes.byref(out)))
    ws = workspace(out.value, X.device)
    g = torch.empty((b,), dtype=torch.float32, device=X.device)
    _check(lib().th_column_sq_norms(_ptr(X), _dtype_code(X), n, b, X.stride(0), _ptr(g), _ptr(ws),
                                    ws.numel(), _stream(X.device)))
    return g


def prune_baseline(W, method: str, gdiag=None, params: PruneParams | None = None, mask_out=None):
    """Magnitude or Wanda pruning of W (c x b, bf16/fp32) in place, no compensation."""
    _require_cuda(W, gdiag, mask_out)
    if params is None:
        params = make_params()
    c, b = W.shape
    code = {"magnitude": TH_BASE_MAGNITUDE, "wanda": TH_BASE_WANDA}[method]
    _check(lib().th_prune_baseline(_ptr(W), _dtype_code(W), c, b, code, _ptr(gdiag),
                                   ctypes.byref(params), _ptr(mask_out), _stream(W.device)))
