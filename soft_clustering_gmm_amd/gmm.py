"""Thin ctypes binding of libgmm_mi355x.so (argument marshalling only).

Every function takes torch tensors that already live on the GPU, passes their
device pointers and torch's current HIP stream to the C-ABI, and returns
tensors the library wrote. All computation happens in the HIP kernels; there
is no CPU path. The library must have been built (``build.py``); importing
this module on a machine without it raises immediately.
"""
from __future__ import annotations

import array
import ctypes
import functools
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgmm_mi355x.so")

GMM_F32, GMM_F16, GMM_BF16 = 0, 1, 2
REGIME_AUTO, REGIME_SINGLE, REGIME_TWOPASS, REGIME_SMALLK = 0, 1, 2, 3
ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU = 0, 1, 2, 3
WORKSPACE_NONE = 256  # what gmm_linear_workspace_bytes reports for a call that needs no workspace
STATS_FP32, STATS_SPLIT_BF16, STATS_AUTO = 0, 1, 2  # STATS_AUTO is the default

EXPORTS = (
    "gmm_version", "gmm_error_string", "gmm_workspace_bytes", "gmm_estep_stats",
    "gmm_estep_stats_regime", "gmm_estep_resp", "gmm_mstep", "gmm_em_iterate", "gmm_assign_top2",
    "gmm_set_timing_events", "gmm_set_stats_precision", "gmm_estep_stats_chunked", "gmm_workspace_bytes_chunked",
    "gmm_border_lists", "gmm_border_lists_workspace_bytes",
    "gmm_kmeans_assign", "gmm_kmeans_update", "gmm_kmeans_iterate", "gmm_kmeans_workspace_bytes",
    "gmm_plan_info", "gmm_estep_stats_static",
    "gmm_linear", "gmm_linear_backward", "gmm_linear_workspace_bytes",
    "gmm_expert_layer", "gmm_expert_rows", "gmm_expert_workspace_bytes",
    "gmm_layer_norm", "gmm_layer_norm_backward", "gmm_layer_norm_workspace_bytes",
    "gmm_cross_entropy", "gmm_cross_entropy_gradients", "gmm_cross_entropy_workspace_bytes",
    "gmm_adamw_step", "gmm_adamw_state_elements",
    "gmm_peak_mfma", "gmm_peak_mfma_flops", "gmm_peak_hbm_read", "gmm_peak_coissue",
)
PEAK_FP32, PEAK_FP64 = 0, 1


class GmmError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {code} ({error_string(code)})")
        self.code = code


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with soft_clustering_gmm_amd/build.py "
                           "(or __graft_entry__.build()); there is no fallback path")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    F64 = ctypes.c_double
    L.gmm_version.restype = ctypes.c_int
    L.gmm_version.argtypes = []
    L.gmm_error_string.restype = ctypes.c_char_p
    L.gmm_error_string.argtypes = [ctypes.c_int]
    L.gmm_workspace_bytes.restype = SZ
    L.gmm_workspace_bytes.argtypes = [I64, I32, I32]
    L.gmm_estep_stats.restype = ctypes.c_int
    L.gmm_estep_stats.argtypes = [P, I32, I64, I32, P, P, P, I32, P, P, P, P, P, P, SZ, P]
    L.gmm_estep_stats_regime.restype = ctypes.c_int
    L.gmm_estep_stats_regime.argtypes = [P, I32, I64, I32, P, P, P, I32, P, P, P, P, P, P, SZ, I32, P]
    L.gmm_estep_resp.restype = ctypes.c_int
    L.gmm_estep_resp.argtypes = [P, I32, I64, I32, P, P, P, I32, P, P, P, SZ, I32, P]
    L.gmm_mstep.restype = ctypes.c_int
    L.gmm_mstep.argtypes = [P, P, P, I64, I32, I32, F32, P, P, P, P]
    L.gmm_em_iterate.restype = ctypes.c_int
    L.gmm_em_iterate.argtypes = [P, I32, I64, I32, I32, I32, F32, P, P, P, P, P, SZ, P]
    L.gmm_assign_top2.restype = ctypes.c_int
    L.gmm_assign_top2.argtypes = [P, I32, I64, I32, P, P, P, I32, P, P, P, SZ, P]
    L.gmm_set_timing_events.restype = ctypes.c_int
    L.gmm_set_timing_events.argtypes = [P, P]
    L.gmm_set_stats_precision.restype = ctypes.c_int
    L.gmm_set_stats_precision.argtypes = [ctypes.c_int32]
    L.gmm_estep_stats_chunked.restype = ctypes.c_int
    L.gmm_estep_stats_chunked.argtypes = [P, I32, I64, I32, P, P, P, I32, P, P, P, P, P, I64, P, SZ, P]
    L.gmm_workspace_bytes_chunked.restype = SZ
    L.gmm_workspace_bytes_chunked.argtypes = [I64, I32, I32, I64, I32]
    L.gmm_border_lists.restype = ctypes.c_int
    L.gmm_border_lists.argtypes = [P, P, I64, I32, F32, P, P, I64, P, SZ, P]
    L.gmm_border_lists_workspace_bytes.restype = SZ
    L.gmm_border_lists_workspace_bytes.argtypes = [I64, I32]
    L.gmm_kmeans_assign.restype = ctypes.c_int
    L.gmm_kmeans_assign.argtypes = [P, I32, I64, I32, P, I32, P, P, P, P, SZ, P]
    L.gmm_kmeans_update.restype = ctypes.c_int
    L.gmm_kmeans_update.argtypes = [P, I32, I64, I32, P, I32, P, P, P, SZ, P]
    L.gmm_kmeans_iterate.restype = ctypes.c_int
    L.gmm_kmeans_iterate.argtypes = [P, I32, I64, I32, I32, I32, P, P, P, SZ, P]
    L.gmm_kmeans_workspace_bytes.restype = SZ
    L.gmm_kmeans_workspace_bytes.argtypes = [I64, I32, I32]
    L.gmm_plan_info.restype = ctypes.c_int
    L.gmm_plan_info.argtypes = [I64, I32, I32, I32, P]
    L.gmm_peak_mfma.restype = ctypes.c_int
    L.gmm_peak_mfma.argtypes = [I32, I64, I32, P, P]
    L.gmm_peak_mfma_flops.restype = ctypes.c_double
    L.gmm_peak_mfma_flops.argtypes = [I32, I64, I32]
    L.gmm_peak_hbm_read.restype = ctypes.c_int
    L.gmm_peak_hbm_read.argtypes = [P, SZ, I32, P, P]
    L.gmm_peak_coissue.restype = ctypes.c_int
    L.gmm_peak_coissue.argtypes = [I32, I64, I32, P, P]
    L.gmm_estep_stats_static.restype = ctypes.c_int
    L.gmm_estep_stats_static.argtypes = [P, I32, I64, I32, P, P, P, I32, P, P, P, P, P, P]
    L.gmm_linear.restype = ctypes.c_int
    L.gmm_linear.argtypes = [P, I32, I64, I32, P, I32, P, I32, P, P, I32, P, P, SZ, P]
    L.gmm_linear_backward.restype = ctypes.c_int
    L.gmm_linear_backward.argtypes = [P, I32, P, I32, I64, I32, P, I32, P, I32, P, P, P, P, SZ, P]
    L.gmm_linear_workspace_bytes.restype = SZ
    L.gmm_linear_workspace_bytes.argtypes = [I64, I32, I32, I32, I32]
    L.gmm_expert_layer.restype = ctypes.c_int
    L.gmm_expert_layer.argtypes = [P, I32, I64, I32, P, I32, P, P, P, I32, I32, F32, I32, P, P, P, P, I32, I32, I32, P,
                                   P, P, P, P, SZ, P]
    L.gmm_expert_rows.restype = ctypes.c_int
    L.gmm_expert_rows.argtypes = [P, I32, I64, I32, P, P, I32, I32, P, P, P, P, I32, I32, I32, P, P, P, SZ, P]
    L.gmm_expert_workspace_bytes.restype = SZ
    L.gmm_expert_workspace_bytes.argtypes = [I64, I32, I32, I32, I32, I32, I32]
    L.gmm_layer_norm.restype = ctypes.c_int
    L.gmm_layer_norm.argtypes = [P, I32, I64, I32, P, P, I32, F32, P, I32, P, P]
    L.gmm_layer_norm_backward.restype = ctypes.c_int
    L.gmm_layer_norm_backward.argtypes = [P, I32, P, I32, I64, I32, P, P, I32, P, P, P, P, SZ, P]
    L.gmm_layer_norm_workspace_bytes.restype = SZ
    L.gmm_layer_norm_workspace_bytes.argtypes = [I64, I32, I32]
    L.gmm_cross_entropy.restype = ctypes.c_int
    L.gmm_cross_entropy.argtypes = [P, I32, I64, I32, P, I32, P, P, P, I32, P, P, P, SZ, P]
    L.gmm_cross_entropy_gradients.restype = ctypes.c_int
    L.gmm_cross_entropy_gradients.argtypes = [P, P, I32, I64, I32, P, I32, P, P, P, I32, P, P, P, P, P, P, SZ, P]
    L.gmm_cross_entropy_workspace_bytes.restype = SZ
    L.gmm_cross_entropy_workspace_bytes.argtypes = [I64, I32, I32, I32, I32]
    L.gmm_adamw_step.restype = ctypes.c_int
    L.gmm_adamw_step.argtypes = [I32, P, P, I32, P, I32, P, P, P, I32, P, P, P, F64, F64, F64, F64, F64, P, P, P]
    L.gmm_adamw_state_elements.restype = I64
    L.gmm_adamw_state_elements.argtypes = [I32, P]
    return L


_LIB = None


def lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def error_string(code: int) -> str:
    return lib().gmm_error_string(code).decode()


def _check(fn: str, code: int) -> None:
    if code != 0:
        raise GmmError(fn, code)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _xtype(X: torch.Tensor) -> int:
    if X.dtype == torch.float32:
        return GMM_F32
    if X.dtype == torch.float16:
        return GMM_F16
    if X.dtype == torch.bfloat16:
        return GMM_BF16
    raise ValueError(f"X must be float32, float16 or bfloat16, got {X.dtype}")


_DTYPES = {torch.float32: GMM_F32, torch.float16: GMM_F16, torch.bfloat16: GMM_BF16}


def _need(t: torch.Tensor, name: str, dtype, shape, device):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _params(X, mu, var, logw):
    if X.dim() != 2:
        raise ValueError("X must be N x d")
    N, d = X.shape
    K = mu.shape[0]
    dev = X.device
    if dev.type != "cuda":
        raise ValueError("X must be on the GPU")
    _xtype(X)
    if not X.is_contiguous():
        raise ValueError("X must be contiguous")
    _need(mu, "mu", torch.float32, (K, d), dev)
    _need(var, "var", torch.float32, (K, d), dev)
    _need(logw, "logw", torch.float32, (K,), dev)
    return N, d, K, dev


def plan_info(N: int, d: int, K: int, regime: int = REGIME_AUTO) -> dict:
    """The launch shape gmm_estep_stats_regime takes for (N, d, K, regime) (host only)."""
    buf = (ctypes.c_int64 * 7)()
    _check("gmm_plan_info", lib().gmm_plan_info(N, d, K, regime, buf))
    keys = ("regime", "waves", "kslabs", "rows_per_chunk", "chunks", "tiles", "scratch_bytes")
    return dict(zip(keys, (int(v) for v in buf)))


def workspace_bytes(N: int, d: int, K: int) -> int:
    return int(lib().gmm_workspace_bytes(N, d, K))


def workspace(N: int, d: int, K: int, device) -> torch.Tensor:
    """A device workspace large enough for every entry point at (N, d, K)."""
    nb = workspace_bytes(N, d, K)
    if nb == 0:
        raise ValueError(f"unsupported shape N={N} d={d} K={K}")
    return torch.empty(nb, dtype=torch.uint8, device=device)


def _ws(ws, N, d, K, dev):
    if ws is None:
        ws = workspace(N, d, K, dev)
    return ws


def estep_stats(X, mu, var, logw, *, regime: int = REGIME_AUTO, want_point_loglik: bool = False, ws=None):
    """Fused E-step: returns (Nk[K], Sx[K,d], Sxx[K,d], L (0-d float64), l_n[N] or None)."""
    N, d, K, dev = _params(X, mu, var, logw)
    Nk = torch.empty(K, dtype=torch.float32, device=dev)
    Sx = torch.empty(K, d, dtype=torch.float32, device=dev)
    Sxx = torch.empty(K, d, dtype=torch.float32, device=dev)
    L = torch.empty((), dtype=torch.float64, device=dev)
    lp = torch.empty(N, dtype=torch.float32, device=dev) if want_point_loglik else None
    ws = _ws(ws, N, d, K, dev)
    _check("gmm_estep_stats_regime", lib().gmm_estep_stats_regime(
        _ptr(X), _xtype(X), N, d, _ptr(mu), _ptr(var), _ptr(logw), K, _ptr(Nk), _ptr(Sx), _ptr(Sxx),
        _ptr(L), _ptr(lp), _ptr(ws), ws.numel(), regime, _stream(dev)))
    return Nk, Sx, Sxx, L, lp


def estep_stats_static(X, mu, var, logw, *, want_point_loglik: bool = False):
    """Allocation-free fused E-step (the library's static per-GPU scratch, no
    workspace): returns the estep_stats outputs. Calls on one GPU must not overlap."""
    N, d, K, dev = _params(X, mu, var, logw)
    Nk = torch.empty(K, dtype=torch.float32, device=dev)
    Sx = torch.empty(K, d, dtype=torch.float32, device=dev)
    Sxx = torch.empty(K, d, dtype=torch.float32, device=dev)
    L = torch.empty((), dtype=torch.float64, device=dev)
    lp = torch.empty(N, dtype=torch.float32, device=dev) if want_point_loglik else None
    _check("gmm_estep_stats_static", lib().gmm_estep_stats_static(
        _ptr(X), _xtype(X), N, d, _ptr(mu), _ptr(var), _ptr(logw), K, _ptr(Nk), _ptr(Sx), _ptr(Sxx),
        _ptr(L), _ptr(lp), _stream(dev)))
    return Nk, Sx, Sxx, L, lp


def workspace_chunked(N: int, d: int, K: int, chunk_rows: int, x_dtype: int, device) -> torch.Tensor:
    """A device workspace for estep_stats_chunked."""
    nb = int(lib().gmm_workspace_bytes_chunked(N, d, K, chunk_rows, x_dtype))
    if nb == 0:
        raise ValueError(f"unsupported shape N={N} d={d} K={K} chunk_rows={chunk_rows}")
    return torch.empty(nb, dtype=torch.uint8, device=device)


def estep_stats_chunked(X_host, mu, var, logw, chunk_rows: int, *, want_point_loglik: bool = False, ws=None):
    """E-step over X in host memory (a CPU tensor, ideally pinned), streamed to the
    device chunk_rows rows at a time; returns the estep_stats outputs (on mu's device)."""
    if X_host.device.type != "cpu" or X_host.dim() != 2 or not X_host.is_contiguous():
        raise ValueError("X_host must be a contiguous 2-d CPU tensor")
    N, d = X_host.shape
    K = mu.shape[0]
    dev = mu.device
    xt = _xtype(X_host)
    _need(mu, "mu", torch.float32, (K, d), dev)
    _need(var, "var", torch.float32, (K, d), dev)
    _need(logw, "logw", torch.float32, (K,), dev)
    Nk = torch.empty(K, dtype=torch.float32, device=dev)
    Sx = torch.empty(K, d, dtype=torch.float32, device=dev)
    Sxx = torch.empty(K, d, dtype=torch.float32, device=dev)
    L = torch.empty((), dtype=torch.float64, device=dev)
    lp = torch.empty(N, dtype=torch.float32, device=dev) if want_point_loglik else None
    if ws is None:
        ws = workspace_chunked(N, d, K, chunk_rows, xt, dev)
    _check("gmm_estep_stats_chunked", lib().gmm_estep_stats_chunked(
        _ptr(X_host), xt, N, d, _ptr(mu), _ptr(var), _ptr(logw), K, _ptr(Nk), _ptr(Sx), _ptr(Sxx), _ptr(L),
        _ptr(lp), chunk_rows, _ptr(ws), ws.numel(), _stream(dev)))
    return Nk, Sx, Sxx, L, lp


def estep_resp(X, mu, var, logw, *, regime: int = REGIME_AUTO, ws=None):
    """Testing aid: the responsibilities R[N,K] and l_n[N] from the same kernels."""
    N, d, K, dev = _params(X, mu, var, logw)
    R = torch.empty(N, K, dtype=torch.float32, device=dev)
    lp = torch.empty(N, dtype=torch.float32, device=dev)
    ws = _ws(ws, N, d, K, dev)
    _check("gmm_estep_resp", lib().gmm_estep_resp(
        _ptr(X), _xtype(X), N, d, _ptr(mu), _ptr(var), _ptr(logw), K, _ptr(R), _ptr(lp), _ptr(ws),
        ws.numel(), regime, _stream(dev)))
    return R, lp


def mstep(Nk, Sx, Sxx, N: int, var_floor: float, mu, var, logw):
    """In-place M-step on (mu, var, logw) from the statistics."""
    K, d = mu.shape
    dev = mu.device
    _need(Nk, "Nk", torch.float32, (K,), dev)
    _need(Sx, "Sx", torch.float32, (K, d), dev)
    _need(Sxx, "Sxx", torch.float32, (K, d), dev)
    _need(var, "var", torch.float32, (K, d), dev)
    _need(logw, "logw", torch.float32, (K,), dev)
    _check("gmm_mstep", lib().gmm_mstep(_ptr(Nk), _ptr(Sx), _ptr(Sxx), N, d, K, float(var_floor),
                                        _ptr(mu), _ptr(var), _ptr(logw), _stream(dev)))


def em_iterate(X, mu, var, logw, iters: int, var_floor: float, *, ws=None):
    """`iters` EM iterations in place; returns the log-likelihood history (device float64)."""
    N, d, K, dev = _params(X, mu, var, logw)
    hist = torch.empty(max(iters, 1), dtype=torch.float64, device=dev)
    ws = _ws(ws, N, d, K, dev)
    _check("gmm_em_iterate", lib().gmm_em_iterate(
        _ptr(X), _xtype(X), N, d, K, iters, float(var_floor), _ptr(mu), _ptr(var), _ptr(logw),
        _ptr(hist), _ptr(ws), ws.numel(), _stream(dev)))
    return hist[:iters]


def set_timing_events(start, stop) -> None:
    """One-shot: the next E-step on this thread records these torch.cuda.Events
    (already created, e.g. by one record()) around its fused kernel(s)."""
    _check("gmm_set_timing_events", lib().gmm_set_timing_events(
        None if start is None else ctypes.c_void_p(start.cuda_event),
        None if stop is None else ctypes.c_void_p(stop.cuda_event)))


def set_stats_precision(mode: int) -> None:
    """Statistics contraction of the fused E-step kernels, process-wide:
    STATS_AUTO (default: fp32 products, exact fp16 splits in the second pass over half-precision X),
    STATS_FP32 or STATS_SPLIT_BF16 (split-bf16 products)."""
    _check("gmm_set_stats_precision", lib().gmm_set_stats_precision(int(mode)))


def assign_top2(X, mu, var, logw, *, ws=None):
    """Top-2 components per point: (idx[N,2] int32, resp[N,2] float32)."""
    N, d, K, dev = _params(X, mu, var, logw)
    idx = torch.empty(N, 2, dtype=torch.int32, device=dev)
    resp = torch.empty(N, 2, dtype=torch.float32, device=dev)
    ws = _ws(ws, N, d, K, dev)
    _check("gmm_assign_top2", lib().gmm_assign_top2(
        _ptr(X), _xtype(X), N, d, _ptr(mu), _ptr(var), _ptr(logw), K, _ptr(idx), _ptr(resp),
        _ptr(ws), ws.numel(), _stream(dev)))
    return idx, resp


def border_lists(idx, resp, K: int, threshold: float, *, ws=None, members=None):
    """Inverted lists with border vectors from a top-2 assignment (idx N x 2 int32,
    resp N x 2 float32, on the GPU): returns (offsets[K+1] int64, members int32
    of capacity 2N; the lists are members[:offsets[K]])."""
    N = idx.shape[0]
    dev = idx.device
    _need(idx, "idx", torch.int32, (N, 2), dev)
    _need(resp, "resp", torch.float32, (N, 2), dev)
    offsets = torch.empty(K + 1, dtype=torch.int64, device=dev)
    if members is None:
        members = torch.empty(max(2 * N, 1), dtype=torch.int32, device=dev)
    if ws is None:
        nb = int(lib().gmm_border_lists_workspace_bytes(N, K))
        if nb == 0:
            raise ValueError(f"unsupported N={N} K={K}")
        ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    _check("gmm_border_lists", lib().gmm_border_lists(
        _ptr(idx), _ptr(resp), N, K, float(threshold), _ptr(offsets), _ptr(members), members.numel(),
        _ptr(ws), ws.numel(), _stream(dev)))
    return offsets, members


def kmeans_workspace(N: int, d: int, K: int, device) -> torch.Tensor:
    nb = int(lib().gmm_kmeans_workspace_bytes(N, d, K))
    if nb == 0:
        raise ValueError(f"unsupported shape N={N} d={d} K={K}")
    return torch.empty(nb, dtype=torch.uint8, device=device)


def _kmeans_args(X, C):
    if X.dim() != 2 or not X.is_contiguous() or X.device.type != "cuda":
        raise ValueError("X must be a contiguous N x d GPU tensor")
    N, d = X.shape
    K = C.shape[0]
    _need(C, "C", torch.float32, (K, d), X.device)
    return N, d, K, X.device


def kmeans_assign(X, C, *, ws=None):
    """Nearest centres: (assign[N] int32, dist2[N] float32, inertia 0-d float64)."""
    N, d, K, dev = _kmeans_args(X, C)
    assign = torch.empty(N, dtype=torch.int32, device=dev)
    dist2 = torch.empty(N, dtype=torch.float32, device=dev)
    inertia = torch.empty((), dtype=torch.float64, device=dev)
    ws = kmeans_workspace(N, d, K, dev) if ws is None else ws
    _check("gmm_kmeans_assign", lib().gmm_kmeans_assign(
        _ptr(X), _xtype(X), N, d, _ptr(C), K, _ptr(assign), _ptr(dist2), _ptr(inertia), _ptr(ws), ws.numel(),
        _stream(dev)))
    return assign, dist2, inertia


def kmeans_update(X, assign, C, *, ws=None):
    """In-place centre update from a hard assignment; returns the counts (int64 K)."""
    N, d, K, dev = _kmeans_args(X, C)
    _need(assign, "assign", torch.int32, (N,), dev)
    counts = torch.empty(K, dtype=torch.int64, device=dev)
    ws = kmeans_workspace(N, d, K, dev) if ws is None else ws
    _check("gmm_kmeans_update", lib().gmm_kmeans_update(
        _ptr(X), _xtype(X), N, d, _ptr(assign), K, _ptr(C), _ptr(counts), _ptr(ws), ws.numel(), _stream(dev)))
    return counts


def kmeans_iterate(X, C, iters: int, *, ws=None):
    """`iters` Lloyd iterations in place on C; returns the inertia history (device float64)."""
    N, d, K, dev = _kmeans_args(X, C)
    hist = torch.empty(max(iters, 1), dtype=torch.float64, device=dev)
    ws = kmeans_workspace(N, d, K, dev) if ws is None else ws
    _check("gmm_kmeans_iterate", lib().gmm_kmeans_iterate(
        _ptr(X), _xtype(X), N, d, K, iters, _ptr(C), _ptr(hist), _ptr(ws), ws.numel(), _stream(dev)))
    return hist[:iters]


# A layer's call is often shorter than its launch: sizes are looked up once, and the stream is torch's raw handle (its
# tensors are on a GPU, so torch's part of it is initialised).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _at(t):
    return None if t is None else t.data_ptr()


def _matrix(t, name):
    if t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-d GPU tensor")
    return t.shape


def _optional(t, name, dtype, shape, device):
    if t is not None:
        _need(t, name, dtype, shape, device)


_grad_mode = torch.is_grad_enabled


def _tracked(*tensors):
    """Whether torch would record a graph for these inputs."""
    if _grad_mode():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


class _Linear(torch.autograd.Function):
    """linear in torch's graph: its backward pass is linear_backward."""

    @staticmethod
    def forward(ctx, X, W, bias, residual, act, out_dtype, want_pre, ws):
        need = act != ACT_NONE and any(ctx.needs_input_grad[:3])
        Y, pre = linear(X, W, bias=bias, act=act, residual=residual, out_dtype=out_dtype, want_pre=want_pre or need,
                        ws=ws)
        ctx.act = act
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(X, W, pre if need else None)
        if not want_pre:
            return Y, None
        ctx.mark_non_differentiable(pre)
        return Y, pre

    @staticmethod
    def backward(ctx, dY, _):
        if torch.is_grad_enabled():  # create_graph: the gradients would count as constants
            raise NotImplementedError("gmm.linear has no second derivatives")
        need = ctx.needs_input_grad
        grads = (None, None, None)
        if dY is not None and any(need[:3]):
            X, W, pre = ctx.saved_tensors
            grads = linear_backward(dY.contiguous(), X, W, pre=pre, act=ctx.act, want_dx=need[0], want_dw=need[1],
                                    want_db=need[2])
        return (*grads, dY if need[3] else None, None, None, None, None)


class _ForwardOnly(torch.autograd.Function):
    """A call without a backward pass in torch's graph: it says so there, rather than leave its inputs out."""

    @staticmethod
    def forward(ctx, name, call, *tensors):
        ctx.name = name
        ctx.set_materialize_grads(False)
        return call()

    @staticmethod
    def backward(ctx, *grads):
        raise NotImplementedError(f"gmm.{ctx.name} has no backward pass: call it on detached tensors or under "
                                  "torch.no_grad()")


@functools.lru_cache(maxsize=4096)
def _linear_bytes(N, d_in, d_out, x_dtype, backward):
    return int(lib().gmm_linear_workspace_bytes(N, d_in, d_out, x_dtype, backward))


@functools.lru_cache(maxsize=4096)
def _expert_bytes(N, D, K, F, d, top, x_dtype):
    return int(lib().gmm_expert_workspace_bytes(N, D, K, F, d, top, x_dtype))


def _scratch(nbytes, device, what):
    if nbytes == 0:
        raise ValueError(f"unsupported {what}")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _space(ws, device):
    """(address, bytes) of a caller's workspace."""
    if ws is None:
        return None, 0
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous tensor on {device}, got {tuple(ws.stride())} on {ws.device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def linear_workspace(N: int, d_in: int, d_out: int, dtype, device, *, backward: bool = False) -> torch.Tensor:
    """A device workspace for linear (or linear_backward) with operands of this torch dtype."""
    return _scratch(_linear_bytes(N, d_in, d_out, _DTYPES[dtype], int(backward)), device,
                    f"N={N} d_in={d_in} d_out={d_out}")


def linear(X, W, *, bias=None, act: int = ACT_NONE, residual=None, out_dtype=None, want_pre: bool = False, ws=None):
    """Y = act(X W^T + bias) + residual; returns (Y, pre), pre = X W^T + bias or None.

    X N x d_in, W d_out x d_in and bias d_out share one type; Y, residual and pre are N x d_out of out_dtype
    (X's type, the default, or float32). Y carries gradients to X, W, bias and residual that require them (first
    derivatives; pre carries none). A captured step calls linear_backward itself, under torch.no_grad()."""
    # as _tracked, written out: a one-row call is as long as its host time
    if _grad_mode() and (X.requires_grad or W.requires_grad or bias is not None and bias.requires_grad
                         or residual is not None and residual.requires_grad):
        return _Linear.apply(X, W, bias, residual, act, out_dtype, want_pre, ws)
    N, d_in = _matrix(X, "X")
    dev, t = X.device, X.dtype
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return linear(X, W, bias=bias, act=act, residual=residual, out_dtype=out_dtype, want_pre=want_pre, ws=ws)
    xt = _xtype(X)
    d_out = W.shape[0]
    _need(W, "W", t, (d_out, d_in), dev)
    _optional(bias, "bias", t, (d_out,), dev)
    if out_dtype is None:
        out_dtype = t
    elif out_dtype != t and out_dtype != torch.float32:
        raise ValueError(f"out_dtype must be {t} or float32, got {out_dtype}")
    _optional(residual, "residual", out_dtype, (N, d_out), dev)
    Y = torch.empty(N, d_out, dtype=out_dtype, device=dev)
    pre = torch.empty(N, d_out, dtype=out_dtype, device=dev) if want_pre else None
    if ws is None and _linear_bytes(N, d_in, d_out, xt, 0) != WORKSPACE_NONE:
        ws = linear_workspace(N, d_in, d_out, t, dev)
    _check("gmm_linear", lib().gmm_linear(
        X.data_ptr(), xt, N, d_in, W.data_ptr(), d_out, _at(bias), act, _at(residual), Y.data_ptr(),
        _DTYPES[out_dtype], _at(pre), *_space(ws, dev), _raw_stream(dev.index)))
    return Y, pre


def linear_backward(dY, X, W, *, pre=None, act: int = ACT_NONE, want_dx: bool = True, want_dw: bool = True,
                    want_db: bool = True, ws=None):
    """Gradients of linear: (dX, dW, db) in X's type, None for what is not wanted. pre is linear's second result
    (not needed with ACT_NONE). The residual's gradient is dY."""
    N, d_in = _matrix(X, "X")
    dev, t = X.device, X.dtype
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return linear_backward(dY, X, W, pre=pre, act=act, want_dx=want_dx, want_dw=want_dw, want_db=want_db,
                                   ws=ws)
    xt = _xtype(X)
    d_out = W.shape[0]
    _need(W, "W", t, (d_out, d_in), dev)
    yt = dY.dtype
    if yt != t and yt != torch.float32:
        raise ValueError(f"dY must be {t} or float32, got {yt}")
    _need(dY, "dY", yt, (N, d_out), dev)
    if pre is None and act != ACT_NONE:
        raise ValueError("pre is needed with an activation")
    _optional(pre, "pre", yt, (N, d_out), dev)
    dX = torch.empty_like(X) if want_dx else None
    dW = torch.empty_like(W) if want_dw else None
    db = torch.empty(d_out, dtype=t, device=dev) if want_db else None
    if ws is None:
        ws = linear_workspace(N, d_in, d_out, t, dev, backward=True)
    _check("gmm_linear_backward", lib().gmm_linear_backward(
        dY.data_ptr(), _DTYPES[yt], X.data_ptr(), xt, N, d_in, W.data_ptr(), d_out, _at(pre), act, _at(dX), _at(dW),
        _at(db), *_space(ws, dev), _raw_stream(dev.index)))
    return dX, dW, db


def expert_workspace(N: int, D: int, K: int, F: int, d: int, top: int, dtype, device) -> torch.Tensor:
    """A device workspace for expert_layer (d >= 1 features) or expert_rows (d = 0)."""
    return _scratch(_expert_bytes(N, D, K, F, d, top, _DTYPES[dtype]), device,
                    f"N={N} D={D} K={K} F={F} d={d} top={top}")


def _experts_args(X, W1, W2, b1, b2, glu, residual):
    N, D = _matrix(X, "X")
    dev, t = X.device, X.dtype
    if W2.dim() != 3:
        raise ValueError("W2 must be K x D x F")
    K, _, F = W2.shape
    up = 2 * F if glu else F
    _need(W1, "W1", t, (K, up, D), dev)
    _need(W2, "W2", t, (K, D, F), dev)
    _optional(b1, "b1", t, (K, up), dev)
    _optional(b2, "b2", t, (K, D), dev)
    _optional(residual, "residual", t, (N, D), dev)
    return N, D, K, F, dev, _xtype(X)


def expert_layer(X, P, mu, var, logw, W1, W2, *, b1=None, b2=None, act: int = ACT_SILU, glu: bool = True,
                 top: int = 2, border_threshold: float = 0.0, renorm: bool = False, residual=None, ws=None):
    """Layer of experts gated by the mixture's posterior at P x, for at most 128 rows: returns
    (Y[N,D], idx[N,top] int32, resp[N,top] float32). It has no backward pass."""
    if _tracked(X, P, mu, var, logw, W1, W2, b1, b2, residual):
        return _ForwardOnly.apply("expert_layer", lambda: expert_layer(
            X, P, mu, var, logw, W1, W2, b1=b1, b2=b2, act=act, glu=glu, top=top, border_threshold=border_threshold,
            renorm=renorm, residual=residual, ws=ws), X, P, mu, var, logw, W1, W2, b1, b2, residual)
    N, D, K, F, dev, xt = _experts_args(X, W1, W2, b1, b2, glu, residual)
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return expert_layer(X, P, mu, var, logw, W1, W2, b1=b1, b2=b2, act=act, glu=glu, top=top,
                                border_threshold=border_threshold, renorm=renorm, residual=residual, ws=ws)
    d = P.shape[0]
    _need(P, "P", X.dtype, (d, D), dev)
    _need(mu, "mu", torch.float32, (K, d), dev)
    _need(var, "var", torch.float32, (K, d), dev)
    _need(logw, "logw", torch.float32, (K,), dev)
    if ws is None:
        ws = expert_workspace(N, D, K, F, d, top, X.dtype, dev)
    Y = torch.empty(N, D, dtype=X.dtype, device=dev)
    idx = torch.empty(N, top, dtype=torch.int32, device=dev)
    resp = torch.empty(N, top, dtype=torch.float32, device=dev)
    _check("gmm_expert_layer", lib().gmm_expert_layer(
        X.data_ptr(), xt, N, D, P.data_ptr(), d, mu.data_ptr(), var.data_ptr(), logw.data_ptr(), K, top,
        border_threshold, renorm, W1.data_ptr(), _at(b1), W2.data_ptr(), _at(b2), F, act, glu, _at(residual),
        Y.data_ptr(), idx.data_ptr(), resp.data_ptr(), *_space(ws, dev), _raw_stream(dev.index)))
    return Y, idx, resp


def expert_rows(X, idx, wts, W1, W2, *, b1=None, b2=None, act: int = ACT_SILU, glu: bool = True, residual=None,
                ws=None):
    """The experts of expert_layer for given picks (idx N x top int32, wts N x top float32, for instance those of
    assign_top2): returns Y[N,D]. A pick outside [0, K) is skipped. It has no backward pass."""
    if _tracked(X, wts, W1, W2, b1, b2, residual):
        return _ForwardOnly.apply("expert_rows", lambda: expert_rows(
            X, idx, wts, W1, W2, b1=b1, b2=b2, act=act, glu=glu, residual=residual, ws=ws), X, wts, W1, W2, b1, b2,
            residual)
    N, D, K, F, dev, xt = _experts_args(X, W1, W2, b1, b2, glu, residual)
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return expert_rows(X, idx, wts, W1, W2, b1=b1, b2=b2, act=act, glu=glu, residual=residual, ws=ws)
    if idx.dim() != 2:
        raise ValueError("idx must be N x top")
    top = idx.shape[1]
    _need(idx, "idx", torch.int32, (N, top), dev)
    _need(wts, "wts", torch.float32, (N, top), dev)
    if ws is None:
        ws = expert_workspace(N, D, K, F, 0, top, X.dtype, dev)
    Y = torch.empty(N, D, dtype=X.dtype, device=dev)
    _check("gmm_expert_rows", lib().gmm_expert_rows(
        X.data_ptr(), xt, N, D, idx.data_ptr(), wts.data_ptr(), top, K, W1.data_ptr(), _at(b1), W2.data_ptr(),
        _at(b2), F, act, glu, _at(residual), Y.data_ptr(), *_space(ws, dev), _raw_stream(dev.index)))
    return Y


class _LayerNorm(torch.autograd.Function):
    """layer_norm in torch's graph: its backward pass is layer_norm_backward."""

    @staticmethod
    def forward(ctx, X, gamma, beta, eps, out_dtype, want_stats):
        Y, stats = layer_norm(X, gamma, beta, eps=eps, out_dtype=out_dtype, want_stats=True)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(X, gamma, stats)
        ctx.weights = next((t.dtype for t in (gamma, beta) if t is not None), None)
        if not want_stats:
            return Y, None
        ctx.mark_non_differentiable(stats)
        return Y, stats

    @staticmethod
    def backward(ctx, dY, _):
        if torch.is_grad_enabled():  # create_graph: the gradients would count as constants
            raise NotImplementedError("gmm.layer_norm has no second derivatives")
        grads = (None, None, None)
        if dY is not None:
            X, gamma, stats = ctx.saved_tensors
            need = ctx.needs_input_grad
            grads = layer_norm_backward(dY.contiguous(), X, stats, gamma, want_dx=need[0], want_dgamma=need[1],
                                        want_dbeta=need[2], param_dtype=ctx.weights)
        return (*grads, None, None, None)


def layer_norm(X, gamma=None, beta=None, *, eps: float = 1e-5, out_dtype=None, want_stats: bool = False):
    """Y = (x - mean) / sqrt(var + eps) gamma + beta over the rows of X; returns (Y, stats), stats N x 2 float32 (mean
    and 1 / sqrt(var + eps)) or None.

    X and Y are N x D, Y of out_dtype (X's type, the default, or any where X is float32); gamma and beta (1 and 0 where
    None) share a type, Y's or float32. Y carries gradients to X, gamma and beta (first derivatives). A captured step
    calls layer_norm_backward itself, under torch.no_grad()."""
    if _tracked(X, gamma, beta):
        return _LayerNorm.apply(X, gamma, beta, eps, out_dtype, want_stats)
    N, D = _matrix(X, "X")
    dev = X.device
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return layer_norm(X, gamma, beta, eps=eps, out_dtype=out_dtype, want_stats=want_stats)
    xt = _xtype(X)
    if out_dtype is None:
        out_dtype = X.dtype
    elif out_dtype != X.dtype and (xt != GMM_F32 or out_dtype not in _DTYPES):
        raise ValueError(f"out_dtype must be {X.dtype}{'' if xt else ', float16 or bfloat16'}, got {out_dtype}")
    wt = _norm_weights(gamma, beta, out_dtype, D, dev)
    Y = torch.empty(N, D, dtype=out_dtype, device=dev)
    stats = torch.empty(N, 2, dtype=torch.float32, device=dev) if want_stats else None
    _check("gmm_layer_norm", lib().gmm_layer_norm(
        X.data_ptr(), xt, N, D, _at(gamma), _at(beta), wt, eps, Y.data_ptr(), _DTYPES[out_dtype], _at(stats),
        _raw_stream(dev.index)))
    return Y, stats


def _norm_weights(gamma, beta, y_dtype, D, dev, dtype=None):
    """The type of a layer norm's weights, which are checked."""
    if dtype is None:
        dtype = gamma.dtype if gamma is not None else beta.dtype if beta is not None else y_dtype
    if dtype != y_dtype and dtype != torch.float32:
        raise ValueError(f"gamma and beta must be {y_dtype} or float32, got {dtype}")
    _optional(gamma, "gamma", dtype, (D,), dev)
    _optional(beta, "beta", dtype, (D,), dev)
    return _DTYPES[dtype]


@functools.lru_cache(maxsize=4096)
def _norm_bytes(N, D, x_dtype):
    return int(lib().gmm_layer_norm_workspace_bytes(N, D, x_dtype))


def layer_norm_workspace(N: int, D: int, dtype, device) -> torch.Tensor:
    """A device workspace for layer_norm_backward with X of this torch dtype."""
    return _scratch(_norm_bytes(N, D, _DTYPES[dtype]), device, f"N={N} D={D}")


def layer_norm_backward(dY, X, stats, gamma=None, *, want_dx: bool = True, want_dgamma: bool = True,
                        want_dbeta: bool = True, param_dtype=None, ws=None):
    """Gradients of layer_norm: (dX, dgamma, dbeta), None for what is not wanted. stats is layer_norm's second result.
    dX has X's type, dgamma and dbeta that of gamma (param_dtype, or dY's type, where gamma is None)."""
    N, D = _matrix(X, "X")
    dev = X.device
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return layer_norm_backward(dY, X, stats, gamma, want_dx=want_dx, want_dgamma=want_dgamma,
                                       want_dbeta=want_dbeta, param_dtype=param_dtype, ws=ws)
    xt = _xtype(X)
    if dY.dtype != X.dtype and (xt != GMM_F32 or dY.dtype not in _DTYPES):
        raise ValueError(f"dY must be {X.dtype}{'' if xt else ', float16 or bfloat16'}, got {dY.dtype}")
    _need(dY, "dY", dY.dtype, (N, D), dev)
    _need(stats, "stats", torch.float32, (N, 2), dev)
    if gamma is not None:
        param_dtype = gamma.dtype
    elif param_dtype is None:
        param_dtype = dY.dtype
    wt = _norm_weights(gamma, None, dY.dtype, D, dev, param_dtype)
    dX = torch.empty_like(X) if want_dx else None
    dgamma = torch.empty(D, dtype=param_dtype, device=dev) if want_dgamma else None
    dbeta = torch.empty(D, dtype=param_dtype, device=dev) if want_dbeta else None
    if ws is None and (want_dgamma or want_dbeta):
        ws = layer_norm_workspace(N, D, X.dtype, dev)
    _check("gmm_layer_norm_backward", lib().gmm_layer_norm_backward(
        dY.data_ptr(), _DTYPES[dY.dtype], X.data_ptr(), xt, N, D, stats.data_ptr(), _at(gamma), wt, _at(dX),
        _at(dgamma), _at(dbeta), *_space(ws, dev), _raw_stream(dev.index)))
    return dX, dgamma, dbeta


class _CrossEntropy(torch.autograd.Function):
    """cross_entropy in torch's graph: its backward pass is cross_entropy_gradients."""

    @staticmethod
    def forward(ctx, X, W, bias, idx, wts, ws):
        loss, lse = cross_entropy(X, W, idx, wts=wts, bias=bias, ws=ws)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(X, W, bias, idx, wts)
        ctx.mark_non_differentiable(lse)
        return loss, lse

    @staticmethod
    def backward(ctx, dloss, _):
        if torch.is_grad_enabled():  # create_graph: the gradients would count as constants
            raise NotImplementedError("gmm.cross_entropy has no second derivatives")
        need = ctx.needs_input_grad
        if need[4]:
            raise NotImplementedError("gmm.cross_entropy has no gradient of wts")
        if dloss is None:
            return None, None, None, None, None, None
        X, W, bias, idx, wts = ctx.saved_tensors
        _, _, dX, dW, db = cross_entropy_gradients(X, W, idx, dloss=dloss.contiguous(), wts=wts, bias=bias,
                                                   want_dx=need[0], want_dw=need[1], want_db=need[2])
        return dX, dW, db, None, None, None


@functools.lru_cache(maxsize=4096)
def _entropy_bytes(N, d_in, V, x_dtype, gradients):
    return int(lib().gmm_cross_entropy_workspace_bytes(N, d_in, V, x_dtype, gradients))


def cross_entropy_workspace(N: int, d_in: int, V: int, dtype, device, *, gradients: bool = False) -> torch.Tensor:
    """A device workspace for cross_entropy (or cross_entropy_gradients) with operands of this torch dtype."""
    return _scratch(_entropy_bytes(N, d_in, V, _DTYPES[dtype], int(gradients)), device, f"N={N} d_in={d_in} V={V}")


def _entropy_args(X, W, bias, idx, wts):
    N, d_in = _matrix(X, "X")
    dev, t = X.device, X.dtype
    xt = _xtype(X)
    V = W.shape[0]
    _need(W, "W", t, (V, d_in), dev)
    _optional(bias, "bias", t, (V,), dev)
    if idx.dim() not in (1, 2):
        raise ValueError("idx must be N or N x top")
    top = 1 if idx.dim() == 1 else idx.shape[1]
    _need(idx, "idx", torch.int32, (N,) if idx.dim() == 1 else (N, top), dev)
    _optional(wts, "wts", torch.float32, tuple(idx.shape), dev)
    return N, d_in, V, top, dev, xt


def cross_entropy(X, W, idx, *, wts=None, bias=None, ws=None):
    """Cross entropy of the head X W^T + bias against each row's picks; returns (loss[N], lse[N]) float32, with
    loss = sum_j wts_j (lse - z[idx_j]) and lse the log-sum-exp of a row's logits.

    X N x d_in, W V x d_in and bias V share one type. idx (N or N x top int32) and wts (the same shape, float32, 1 where
    None) are those of assign_top2 or kmeans_assign, or any other labels; a pick outside [0, V) counts for nothing. loss
    carries gradients to X, W and bias (first derivatives; lse carries none), for which the logits are computed again. A
    training step that knows its loss's gradients beforehand (a mean over the rows) calls cross_entropy_gradients, under
    torch.no_grad(), and saves that; so does a captured step."""
    if _tracked(X, W, bias, wts):
        return _CrossEntropy.apply(X, W, bias, idx, wts, ws)
    N, d_in, V, top, dev, xt = _entropy_args(X, W, bias, idx, wts)
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return cross_entropy(X, W, idx, wts=wts, bias=bias, ws=ws)
    loss = torch.empty(N, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    if ws is None:
        ws = cross_entropy_workspace(N, d_in, V, X.dtype, dev)
    _check("gmm_cross_entropy", lib().gmm_cross_entropy(
        X.data_ptr(), xt, N, d_in, W.data_ptr(), V, _at(bias), idx.data_ptr(), _at(wts), top, loss.data_ptr(),
        lse.data_ptr(), *_space(ws, dev), _raw_stream(dev.index)))
    return loss, lse


def cross_entropy_gradients(X, W, idx, *, dloss=None, wts=None, bias=None, want_dx: bool = True, want_dw: bool = True,
                            want_db: bool = True, ws=None):
    """cross_entropy with the gradients of sum_n dloss_n loss_n (dloss N float32, 1 where None) in one call: returns
    (loss, lse, dX, dW, db), the gradients in X's type, None for what is not wanted. A row of no picks, or whose dloss is
    0, has no part in them."""
    N, d_in, V, top, dev, xt = _entropy_args(X, W, bias, idx, wts)
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return cross_entropy_gradients(X, W, idx, dloss=dloss, wts=wts, bias=bias, want_dx=want_dx, want_dw=want_dw,
                                           want_db=want_db, ws=ws)
    _optional(dloss, "dloss", torch.float32, (N,), dev)
    loss = torch.empty(N, dtype=torch.float32, device=dev)
    lse = torch.empty(N, dtype=torch.float32, device=dev)
    dX = torch.empty_like(X) if want_dx else None
    dW = torch.empty_like(W) if want_dw else None
    db = torch.empty(V, dtype=X.dtype, device=dev) if want_db else None
    if ws is None:
        ws = cross_entropy_workspace(N, d_in, V, X.dtype, dev, gradients=True)
    _check("gmm_cross_entropy_gradients", lib().gmm_cross_entropy_gradients(
        _at(dloss), X.data_ptr(), xt, N, d_in, W.data_ptr(), V, _at(bias), idx.data_ptr(), _at(wts), top,
        loss.data_ptr(), lse.data_ptr(), _at(dX), _at(dW), _at(db), *_space(ws, dev), _raw_stream(dev.index)))
    return loss, lse, dX, dW, db


ADAMW_BLOCK = 256  # elements of adamw_step's state that share a scale; each tensor's part starts at a multiple


# Over hundreds of tensors a step is as long as its host time: what is asked of each goes through these.
_ptr_of, _numel_of, _size_of = torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.size
_contiguous, _index_of, _dtype_of = torch.Tensor.is_contiguous, torch.Tensor.get_device, torch.Tensor.dtype.__get__


def _state_elements(sizes):
    return sum([-(-n // ADAMW_BLOCK) for n in sizes]) * ADAMW_BLOCK


def _need_all(tensors, dtype, index, what):
    """Every one contiguous, of this type and on this GPU."""
    if not (set(map(_dtype_of, tensors)) <= {dtype} and set(map(_index_of, tensors)) <= {index}
            and all(map(_contiguous, tensors))):
        raise ValueError(f"{what}: expected contiguous {dtype} on cuda:{index}, got "
                         f"{[(t.dtype, tuple(t.shape), tuple(t.stride()), str(t.device)) for t in tensors][:8]}")


def adamw_state(params, *, bits: int = 32, master: bool = False) -> dict:
    """A fresh state of adamw_step for these parameters, as the keyword arguments that it takes: m, v, step, for 8 bits
    m_scale and v_scale, and with `master` float32 copies of the parameters. A tensor's part of m, v and master starts
    at the next multiple of 256 elements."""
    params = list(params)
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits}")
    if not params:
        raise ValueError("no parameters")
    dev, total = params[0].device, _state_elements([p.numel() for p in params])
    state = {k: torch.zeros(total, dtype=torch.float32 if bits == 32 else torch.uint8, device=dev) for k in ("m", "v")}
    state["step"] = torch.zeros(2, dtype=torch.int64, device=dev)
    if bits == 8:
        state = {k: t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t for k, t in state.items()}
        for k in ("m_scale", "v_scale"):
            state[k] = torch.zeros(total // ADAMW_BLOCK, dtype=torch.float32, device=dev)
    if master:
        state["master"] = torch.zeros(total, dtype=torch.float32, device=dev)
        at = 0
        for p in params:
            state["master"][at:at + p.numel()] = p.detach().reshape(-1)
            at += -(-p.numel() // ADAMW_BLOCK) * ADAMW_BLOCK
    return state


def _device_factor(t, name, device):
    if t is not None and (t.dtype != torch.float32 or t.numel() != 1 or t.device != device):
        raise ValueError(f"{name}: expected one float32 on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return _at(t)


def adamw_step(params, grads, m, v, step, *, m_scale=None, v_scale=None, master=None, lr: float = 1e-3,
               beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01,
               lr_factor=None, grad_factor=None) -> None:
    """One AdamW step in place over many parameters of one type (contiguous, on one GPU), whose gradients (None: left as
    it is) have their type or float32. m, v, step, m_scale, v_scale and master are those of adamw_state; m and v are
    float32, or float8_e4m3fn with scales for each 256 elements. With master the float32 copies are updated and the
    parameters receive their rounding. lr_factor and grad_factor (one float32 each, on the GPU) multiply lr and the
    gradients and may change between the replays of a captured step, as step does."""
    n = len(params)
    if len(grads) != n:
        raise ValueError(f"{n} parameters and {len(grads)} gradients")
    dev = m.device
    if dev.type != "cuda":
        raise ValueError("the state must be on the GPU")
    if dev.index != _current_device():
        with torch.cuda.device(dev):
            return adamw_step(params, grads, m, v, step, m_scale=m_scale, v_scale=v_scale, master=master, lr=lr,
                              beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay, lr_factor=lr_factor,
                              grad_factor=grad_factor)
    given, stepped = grads, params
    if any([g is None for g in grads]):
        given = [g for g in grads if g is not None]
        stepped = [p for p, g in zip(params, grads) if g is not None]
    pt = params[0].dtype if n else torch.float32
    gt = given[0].dtype if given else pt
    if pt not in _DTYPES or gt != pt and gt != torch.float32:
        raise ValueError(f"parameters must be float32, float16 or bfloat16 and gradients theirs or float32, got {pt}, {gt}")
    _need_all(params, pt, dev.index, "parameters")
    _need_all(given, gt, dev.index, "gradients")
    if list(map(_size_of, stepped)) != list(map(_size_of, given)):
        raise ValueError("a gradient has another shape than its parameter")
    sizes, at = list(map(_numel_of, params)), list(map(_ptr_of, params))
    # none overlap: in order, none starts before the last one's end
    ends = sorted([a + k * pt.itemsize for a, k in zip(at, sizes) if k])
    if not all(map(operator.le, ends, sorted([a for a, k in zip(at, sizes) if k])[1:])):
        raise ValueError("two parameters share memory")
    total = _state_elements(sizes)
    st = m.dtype
    if st != torch.float32 and st != torch.float8_e4m3fn:
        raise ValueError(f"m must be float32 or float8_e4m3fn, got {st}")
    _need(m, "m", st, (total,), dev)
    _need(v, "v", st, (total,), dev)
    _need(step, "step", torch.int64, (2,), dev)
    if st != torch.float32:
        if m_scale is None or v_scale is None:
            raise ValueError("states of 8 bits need m_scale and v_scale")
        _need(m_scale, "m_scale", torch.float32, (total // ADAMW_BLOCK,), dev)
        _need(v_scale, "v_scale", torch.float32, (total // ADAMW_BLOCK,), dev)
    _optional(master, "master", torch.float32, (total,), dev)
    if master is not None and pt == torch.float32:
        raise ValueError("float32 parameters have no master copies")
    of = list(map(_ptr_of, grads)) if given is grads else [0 if g is None else g.data_ptr() for g in grads]
    sizes, at, of = array.array("q", sizes), array.array("Q", at), array.array("Q", of)
    _check("gmm_adamw_step", lib().gmm_adamw_step(
        n, sizes.buffer_info()[0], at.buffer_info()[0], _DTYPES[pt], of.buffer_info()[0], _DTYPES[gt], _at(master),
        m.data_ptr(), v.data_ptr(), 32 if st == torch.float32 else 8, _at(m_scale), _at(v_scale), step.data_ptr(), lr,
        beta1, beta2, eps, weight_decay, _device_factor(lr_factor, "lr_factor", dev),
        _device_factor(grad_factor, "grad_factor", dev), _raw_stream(dev.index)))
    # a graph that has saved a parameter says so when it comes to it
    torch.autograd.graph.increment_version(stepped)


def peak_mfma(precision: int, trips: int, blocks: int, out: torch.Tensor) -> float:
    """Enqueues the matrix-core issue loop on the current stream; returns the flops it executes."""
    _check("gmm_peak_mfma", lib().gmm_peak_mfma(precision, trips, blocks, _ptr(out), _stream(out.device)))
    return float(lib().gmm_peak_mfma_flops(precision, trips, blocks))


def peak_hbm_read(buf: torch.Tensor, blocks: int, out: torch.Tensor) -> int:
    """Enqueues the HBM read stream over buf on the current stream; returns the bytes it reads."""
    nbytes = buf.numel() * buf.element_size() // 16 * 16
    _check("gmm_peak_hbm_read", lib().gmm_peak_hbm_read(_ptr(buf), nbytes, blocks, _ptr(out), _stream(buf.device)))
    return nbytes


def peak_coissue(mode: int, trips: int, blocks: int, out: torch.Tensor) -> None:
    """Enqueues the co-issue probe (0 matrix only, 1 vector only, 2 both per wave, 3 split waves)."""
    _check("gmm_peak_coissue", lib().gmm_peak_coissue(mode, trips, blocks, _ptr(out), _stream(out.device)))
