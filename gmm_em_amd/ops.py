"""Python binding of libgmm_em.so (argument marshalling only).

Every step of the EM path runs in the HIP library; this module only checks
tensor shapes, dtypes and devices, allocates the workspace with PyTorch and
passes raw device pointers and the current HIP stream through the C ABI
declared in ``include/gmm_em.h``. Importing it fails loudly when the library
has not been built; there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgmm_em.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is not built: run `python -m gmm_em_amd.build`")
lib = ctypes.CDLL(_LIB_PATH)

_vp, _i64, _i32, _f32, _f64, _sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                    ctypes.c_float, ctypes.c_double, ctypes.c_size_t)
lib.gmm_workspace_bytes.argtypes = [_i32, _i32]
lib.gmm_workspace_bytes.restype = _sz
lib.gmm_em_step.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _vp, _vp, _i32, _f32, _vp, _vp, _sz, _vp]
lib.gmm_fit.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _vp, _vp, _i32, _f32, _i32, _f64, _vp,
                        ctypes.POINTER(_i32), _vp, _sz, _vp]
lib.gmm_loglik.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _sz, _vp]
lib.gmm_assign_topm.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _vp, _vp, _i32, _i32, _vp, _vp,
                                _vp, _sz, _vp]
lib.gmm_kmeans_step.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _i32, _vp, _vp, _vp, _sz, _vp]
lib.gmm_kmeans_fit.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _i32, _i32, _f64, _vp,
                               ctypes.POINTER(_i32), _vp, _sz, _vp]
lib.gmm_ivf_workspace_bytes.argtypes = [_i64, _i32, _i32]
lib.gmm_ivf_workspace_bytes.restype = _sz
lib.gmm_ivf_build.argtypes = [_vp, _vp, _i64, _i32, _i32, _f32, _vp, _vp, _vp, _vp, _sz, _vp]
lib.gmm_logits_score_workspace_bytes.argtypes = [_i64, _i32, _i32]
lib.gmm_logits_score_workspace_bytes.restype = _sz
lib.gmm_logits_score.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _i32, _f32, _vp, _vp, _vp, _vp,
                                 _vp, _vp, _sz, _vp]
lib.gmm_logits_score_backward.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _vp, _vp, _vp, _vp,
                                          _f32, _vp, _i64, _vp]
lib.gmm_head_score_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32, _i32]
lib.gmm_head_score_workspace_bytes.restype = _sz
lib.gmm_head_score.argtypes = [_vp, _i64, _i32, _i64, _vp, _i32, _i64, _i32, _vp, _i32, _f32, _vp,
                               _vp, _vp, _vp, _vp, _vp, _sz, _vp]
lib.gmm_head_score_backward_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32]
lib.gmm_head_score_backward_workspace_bytes.restype = _sz
lib.gmm_head_score_backward.argtypes = [_vp, _i64, _i32, _i64, _vp, _i32, _i64, _i32, _vp, _vp, _vp,
                                        _vp, _vp, _f32, _vp, _i64, _vp, _i64, _vp, _sz, _vp]
lib.gmm_moe_layer_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32, _i32, _i32]
lib.gmm_moe_layer_workspace_bytes.restype = _sz
lib.gmm_moe_layer.argtypes = [_vp, _i64, _i32, _i64, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _vp,
                              _vp, _vp, _i64, _vp, _sz, _vp]
lib.gmm_embed.argtypes = [_vp, _i32, _i32, _i64, _i32, _vp, _i64, _f32, _vp, _i64, _vp]
lib.gmm_embed_backward_workspace_bytes.argtypes = [_i64, _i32, _i32]
lib.gmm_embed_backward_workspace_bytes.restype = _sz
lib.gmm_embed_backward.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _i32, _f32, _vp, _i64, _vp, _sz, _vp]
lib.gmm_quantize_rows.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _i64, _vp, _vp]
lib.gmm_quantized_product_workspace_bytes.argtypes = [_i64, _i32, _i32]
lib.gmm_quantized_product_workspace_bytes.restype = _sz
lib.gmm_quantized_product_call_workspace_bytes.argtypes = [_vp, _i64, _i32, _i64, _vp, _i32, _i64]
lib.gmm_quantized_product_call_workspace_bytes.restype = _sz
lib.gmm_quantized_product.argtypes = [_vp, _i64, _i32, _i64, _vp, _vp, _i32, _i64, _vp, _vp, _i64, _i32,
                                      _vp, _sz, _vp]
lib.gmm_beam_step_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32]
lib.gmm_beam_step_workspace_bytes.restype = _sz
lib.gmm_beam_step.argtypes = [_vp, _i64, _i32, _i32, _i64, _i32, _vp, _vp, _i32, _i32, _f32, _vp, _vp, _vp,
                              _vp, _sz, _vp]
lib.gmm_beam_reorder.argtypes = [_vp, _i64, _i64, _i64, _i32, _i64, _i64, _vp, _i32, _vp, _i64, _i64, _vp]
lib.gmm_balance_loss_workspace_bytes.argtypes = [_i64, _i32, _i32]
lib.gmm_balance_loss_workspace_bytes.restype = _sz
lib.gmm_balance_loss.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                 _vp]
lib.gmm_balance_loss_backward.argtypes = [_vp, _i64, _i32, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _i64, _vp]
lib.gmm_device_status.argtypes = [_vp, _vp]
lib.gmm_estep_arithmetic.argtypes = [_vp, _vp]
lib.gmm_estep_arithmetic.restype = ctypes.c_int
lib.gmm_status_string.argtypes = [ctypes.c_int]
lib.gmm_status_string.restype = ctypes.c_char_p
lib.gmm_version.restype = _i32
lib.gmm_profile_begin.argtypes = [_i32]
lib.gmm_profile_end.argtypes = [ctypes.POINTER(_f64), ctypes.POINTER(_i32), ctypes.POINTER(_f64),
                                ctypes.POINTER(_i32)]
for _f in (lib.gmm_em_step, lib.gmm_fit, lib.gmm_loglik, lib.gmm_assign_topm, lib.gmm_kmeans_step,
           lib.gmm_kmeans_fit, lib.gmm_ivf_build, lib.gmm_logits_score, lib.gmm_logits_score_backward,
           lib.gmm_head_score, lib.gmm_head_score_backward, lib.gmm_moe_layer, lib.gmm_embed, lib.gmm_embed_backward,
           lib.gmm_quantize_rows, lib.gmm_quantized_product, lib.gmm_beam_step, lib.gmm_beam_reorder,
           lib.gmm_balance_loss, lib.gmm_balance_loss_backward, lib.gmm_device_status, lib.gmm_profile_begin, lib.gmm_profile_end):
    _f.restype = ctypes.c_int

(GMM_OK, GMM_E_INVALID, GMM_E_DTYPE, GMM_E_WORKSPACE, GMM_E_PARAMS, GMM_E_HIP,
 GMM_E_UNSUPPORTED) = range(7)
GMM_F32, GMM_BF16 = 0, 1  # gmm_dtype


class GmmError(RuntimeError):
    def __init__(self, code: int):
        self.code = code
        super().__init__(f"gmm_em: {lib.gmm_status_string(code).decode()} (status {code})")


def _check(rc: int) -> None:
    if rc != GMM_OK:
        raise GmmError(rc)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def workspace_bytes(d: int, k: int) -> int:
    return int(lib.gmm_workspace_bytes(d, k))


def workspace(d: int, k: int, device="cuda") -> torch.Tensor:
    """A workspace buffer for data of dimension d with k components."""
    nb = workspace_bytes(d, k)
    if nb == 0:
        raise GmmError(GMM_E_UNSUPPORTED)
    return torch.empty(nb, dtype=torch.uint8, device=device)


def _data(x: torch.Tensor):
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit stride along columns")
    if x.dtype == torch.float32:
        dt = GMM_F32
    elif x.dtype == torch.bfloat16:
        dt = GMM_BF16
    else:
        raise TypeError("x must be float32 or bfloat16")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    return dt, max(x.stride(0), x.shape[1])


def _params(x, w, mu, var):
    k, d = mu.shape
    for t, shape in ((w, (k,)), (mu, (k, d)), (var, (k, d))):
        if t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != shape:
            raise ValueError("parameters must be contiguous float32: weights (K,), means/variances (K, D)")
        if t.device != x.device:
            raise ValueError("parameters must be on the device of x")
    if x.shape[1] != d:
        raise ValueError("x and means disagree on D")
    return k, d


def _ws(ws, d, k, device):
    return workspace(d, k, device) if ws is None else ws


def em_step(x, weights, means, variances, var_floor: float = 1e-6, ws=None, loglik=None):
    """One EM iteration in place; returns the 0-d float64 device tensor L(input params)."""
    dt, ldx = _data(x)
    k, d = _params(x, weights, means, variances)
    ws = _ws(ws, d, k, x.device)
    out = torch.empty((), dtype=torch.float64, device=x.device) if loglik is None else loglik
    _check(lib.gmm_em_step(_ptr(x), x.shape[0], d, ldx, dt, _ptr(weights), _ptr(means),
                           _ptr(variances), k, var_floor, _ptr(out), _ptr(ws), ws.numel(),
                           _stream(x.device)))
    return out


def fit(x, weights, means, variances, var_floor: float = 1e-6, max_iter: int = 10,
        tol: float = 0.0, ws=None):
    """EM iterations in place; returns (history float64 tensor of L(theta_t), iterations)."""
    dt, ldx = _data(x)
    k, d = _params(x, weights, means, variances)
    ws = _ws(ws, d, k, x.device)
    hist = torch.full((max(max_iter, 1),), float("nan"), dtype=torch.float64, device=x.device)
    done = _i32(0)
    _check(lib.gmm_fit(_ptr(x), x.shape[0], d, ldx, dt, _ptr(weights), _ptr(means), _ptr(variances),
                       k, var_floor, max_iter, tol, _ptr(hist), ctypes.byref(done), _ptr(ws),
                       ws.numel(), _stream(x.device)))
    return hist[: done.value], done.value


def loglik(x, weights, means, variances, per_row: bool = False, ws=None):
    """Total log-likelihood (0-d float64 device tensor) and optionally per-row values."""
    dt, ldx = _data(x)
    k, d = _params(x, weights, means, variances)
    ws = _ws(ws, d, k, x.device)
    total = torch.empty((), dtype=torch.float64, device=x.device)
    rows = torch.empty(x.shape[0], dtype=torch.float64, device=x.device) if per_row else None
    _check(lib.gmm_loglik(_ptr(x), x.shape[0], d, ldx, dt, _ptr(weights), _ptr(means),
                          _ptr(variances), k, _ptr(total), _ptr(rows), _ptr(ws), ws.numel(),
                          _stream(x.device)))
    return (total, rows) if per_row else total


def assign_topm(x, weights, means, variances, m: int = 2, ws=None):
    """Top-m components per row by responsibility: (idx int32 (N, m), resp float32 (N, m))."""
    dt, ldx = _data(x)
    k, d = _params(x, weights, means, variances)
    ws = _ws(ws, d, k, x.device)
    idx = torch.empty((x.shape[0], m), dtype=torch.int32, device=x.device)
    resp = torch.empty((x.shape[0], m), dtype=torch.float32, device=x.device)
    _check(lib.gmm_assign_topm(_ptr(x), x.shape[0], d, ldx, dt, _ptr(weights), _ptr(means),
                               _ptr(variances), k, m, _ptr(idx), _ptr(resp), _ptr(ws), ws.numel(),
                               _stream(x.device)))
    return idx, resp


def kmeans_step(x, centroids, ws=None, assign: bool = True):
    """One Lloyd step in place on centroids (K, D) float32.

    Returns (inertia 0-d float64 device tensor for the input centroids,
    assignment int32 (N,) or None).
    """
    dt, ldx = _data(x)
    if centroids.dtype != torch.float32 or not centroids.is_contiguous() or centroids.dim() != 2:
        raise ValueError("centroids must be a contiguous float32 (K, D) tensor")
    if centroids.device != x.device or centroids.shape[1] != x.shape[1]:
        raise ValueError("centroids must be on the device of x and match its D")
    k, d = centroids.shape
    ws = _ws(ws, d, k, x.device)
    inertia = torch.empty((), dtype=torch.float64, device=x.device)
    z = torch.empty(x.shape[0], dtype=torch.int32, device=x.device) if assign else None
    _check(lib.gmm_kmeans_step(_ptr(x), x.shape[0], d, ldx, dt, _ptr(centroids), k, _ptr(z),
                               _ptr(inertia), _ptr(ws), ws.numel(), _stream(x.device)))
    return inertia, z


def kmeans_fit(x, centroids, max_iter: int = 10, tol: float = 0.0, ws=None):
    """Lloyd steps in place; returns (inertia history float64 tensor, steps taken)."""
    dt, ldx = _data(x)
    if centroids.dtype != torch.float32 or not centroids.is_contiguous() or centroids.dim() != 2:
        raise ValueError("centroids must be a contiguous float32 (K, D) tensor")
    if centroids.device != x.device or centroids.shape[1] != x.shape[1]:
        raise ValueError("centroids must be on the device of x and match its D")
    k, d = centroids.shape
    ws = _ws(ws, d, k, x.device)
    hist = torch.full((max(max_iter, 1),), float("nan"), dtype=torch.float64, device=x.device)
    done = _i32(0)
    _check(lib.gmm_kmeans_fit(_ptr(x), x.shape[0], d, ldx, dt, _ptr(centroids), k, max_iter, tol,
                              _ptr(hist), ctypes.byref(done), _ptr(ws), ws.numel(),
                              _stream(x.device)))
    return hist[: done.value], done.value


def ivf_build(idx, resp, k: int, min_resp: float = 0.0, values: bool = True):
    """Inverted lists from top-m assignments idx (N, m) int32 / resp (N, m) float32.

    Returns (offsets int64 (k+1,), rows int32 (entries,), values float32 or
    None); list c is rows[offsets[c]:offsets[c+1]]. Synchronises once to
    size the outputs to the entries stored.
    """
    if idx.dtype != torch.int32 or idx.dim() != 2 or not idx.is_contiguous() or not idx.is_cuda:
        raise ValueError("idx must be a contiguous int32 (N, m) device tensor")
    if resp is not None and (resp.dtype != torch.float32 or tuple(resp.shape) != tuple(idx.shape)
                             or not resp.is_contiguous() or resp.device != idx.device):
        raise ValueError("resp must be a contiguous float32 tensor shaped like idx")
    n, m = idx.shape
    nb = int(lib.gmm_ivf_workspace_bytes(n, m, k))
    if nb == 0:
        raise GmmError(GMM_E_UNSUPPORTED)
    dev = idx.device
    ws = torch.empty(nb, dtype=torch.uint8, device=dev)
    offsets = torch.empty(k + 1, dtype=torch.int64, device=dev)
    rows = torch.empty(max(n * m, 1), dtype=torch.int32, device=dev)
    vals = torch.empty(max(n * m, 1), dtype=torch.float32, device=dev) if values else None
    _check(lib.gmm_ivf_build(_ptr(idx), _ptr(resp), n, m, k, min_resp, _ptr(offsets), _ptr(rows),
                             _ptr(vals), _ptr(ws), nb, _stream(dev)))
    total = int(offsets[k].item())
    return offsets, rows[:total], (vals[:total] if values else None)


TOP_MAX = 16  # GMM_TOP_MAX


class Scores(NamedTuple):
    """What :func:`logits_score` and :func:`head_score` return."""

    logprob: Optional[torch.Tensor]  # (N,) float32, None without targets
    entropy: torch.Tensor            # (N,) float32
    norm: torch.Tensor               # (N, 2) float32: max l and log sum exp(l - max l)
    top_idx: Optional[torch.Tensor]  # (N, m) int32, None when m == 0
    top_logprob: Optional[torch.Tensor]  # (N, m) float32


_DTYPES = {torch.float32: GMM_F32, torch.bfloat16: GMM_BF16}


def _rows2(t, name):
    """(dtype code, leading dimension) of a 2-D row-major device tensor."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor with unit stride along columns")
    (n, d), (step, unit) = t.shape, t.stride()
    if unit != 1 and d > 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit stride along columns")
    if n > 1 and step < d:
        raise ValueError(f"the rows of {name} must not overlap")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be float32 or bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return dt, step if step > d else d


def _int32(*sizes):
    """Refuses sizes that the int32 arguments of the C ABI would cut to their low bits."""
    for s in sizes:
        if not 0 <= s <= 0x7fffffff:
            raise GmmError(GMM_E_INVALID)


def _addr(t):
    return None if t is None else t.data_ptr()


def _row(t, n, name, dtype, device):
    """Address of a contiguous per-row vector, or None."""
    if t is None:
        return None
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous ({n},) tensor of {dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on the device of the rows")
    return t.data_ptr()


def _norm(norm, n, device):
    if norm.dtype != torch.float32 or tuple(norm.shape) != (n, 2) or not norm.is_contiguous() \
            or norm.device != device:
        raise ValueError("norm must be the (N, 2) float32 tensor of the forward call")


def _scratch(need, ws, device):
    """(tensor, bytes) of a workspace: the caller's, or a new one."""
    if need == 0:
        raise GmmError(GMM_E_INVALID)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    elif not ws.is_cuda or ws.device != device:
        raise ValueError("ws must be on the device of the rows")
    return ws, ws.numel() * ws.element_size()


class _On:
    """Makes ``device`` current for a call, where it is not; gives the stream's handle."""

    __slots__ = ("device", "guard")

    def __init__(self, device):
        self.device = device

    def __enter__(self):
        index = self.device.index
        self.guard = None
        if torch._C._cuda_getDevice() != index:
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        return torch._C._cuda_getCurrentRawStream(index)

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _score_outputs(n, m, targets, device):
    new = torch.empty
    f32 = torch.float32
    return Scores(None if targets is None else new(n, dtype=f32, device=device),
                  new(n, dtype=f32, device=device), new((n, 2), dtype=f32, device=device),
                  new((n, m), dtype=torch.int32, device=device) if m > 0 else None,
                  new((n, m), dtype=f32, device=device) if m > 0 else None)


def logits_score(logits, targets=None, m: int = 0, scale: float = 1.0, ws=None) -> Scores:
    """Log-probabilities of given codes, entropy and top-m alternatives from logits (N, V).

    logits: float32 or bfloat16 with unit column stride; targets: int32 (N,),
    negative where there is none. See gmm_logits_score in ``include/gmm_em.h``.
    """
    dt, ldl = _rows2(logits, "logits")
    n, v = logits.shape
    _int32(v, m)
    dev = logits.device
    t = _row(targets, n, "targets", torch.int32, dev)
    ws, nb = _scratch(lib.gmm_logits_score_workspace_bytes(n, v, m), ws, dev)
    out = _score_outputs(n, m, targets, dev)
    with _On(dev) as stream:
        _check(lib.gmm_logits_score(logits.data_ptr(), n, v, ldl, dt, t, m, scale, _addr(out[0]),
                                    _addr(out[1]), _addr(out[2]), _addr(out[3]), _addr(out[4]),
                                    ws.data_ptr(), nb, stream))
    return out


def logits_score_backward(logits, targets, norm, entropy=None, g_logprob=None, g_entropy=None,
                          scale: float = 1.0, out=None):
    """Gradient of :func:`logits_score` with respect to the logits, in their type.

    norm and entropy are what the forward call returned; g_logprob and
    g_entropy float32 (N,), each None for 0. out may be the logits themselves.
    """
    dt, ldl = _rows2(logits, "logits")
    n, v = logits.shape
    _int32(v)
    dev = logits.device
    _norm(norm, n, dev)
    if out is None:
        out = torch.empty((n, v), dtype=logits.dtype, device=dev)
    dt2, ldo = _rows2(out, "out")
    if dt2 != dt or out.shape != logits.shape or out.device != dev:
        raise ValueError("out must have the shape, type and device of logits")
    f32 = torch.float32
    t, h, gl, gh = (_row(a, n, nm, ty, dev) for a, nm, ty in (
        (targets, "targets", torch.int32), (entropy, "entropy", f32),
        (g_logprob, "g_logprob", f32), (g_entropy, "g_entropy", f32)))
    with _On(dev) as stream:
        _check(lib.gmm_logits_score_backward(logits.data_ptr(), n, v, ldl, dt, t, norm.data_ptr(), h,
                                             gl, gh, scale, out.data_ptr(), ldo, stream))
    return out


def _head(hidden, weight):
    dt, ldh = _rows2(hidden, "hidden")
    dt2, ldw = _rows2(weight, "weight")
    if dt != dt2 or hidden.shape[1] != weight.shape[1] or hidden.device != weight.device:
        raise ValueError("hidden (N, D) and weight (V, D) must agree in D, type and device")
    _int32(*weight.shape)
    return dt, ldh, ldw, hidden.shape[0], hidden.shape[1], weight.shape[0], hidden.device


def head_score(hidden, weight, targets=None, m: int = 0, scale: float = 1.0, ws=None) -> Scores:
    """:func:`logits_score` of hidden (N, D) @ weight (V, D).T, without the (N, V) logits.

    float32 or bfloat16, both the same, rows of any stride. See gmm_head_score
    in ``include/gmm_em.h``.
    """
    dt, ldh, ldw, n, d, v, dev = _head(hidden, weight)
    _int32(m)
    t = _row(targets, n, "targets", torch.int32, dev)
    ws, nb = _scratch(lib.gmm_head_score_workspace_bytes(n, d, v, dt, m), ws, dev)
    out = _score_outputs(n, m, targets, dev)
    with _On(dev) as stream:
        _check(lib.gmm_head_score(hidden.data_ptr(), n, d, ldh, weight.data_ptr(), v, ldw, dt, t, m,
                                  scale, _addr(out[0]), _addr(out[1]), _addr(out[2]), _addr(out[3]),
                                  _addr(out[4]), ws.data_ptr(), nb, stream))
    return out


def head_score_backward(hidden, weight, targets, norm, entropy=None, g_logprob=None, g_entropy=None,
                        scale: float = 1.0, ws=None):
    """Gradients (d_hidden, d_weight) of :func:`head_score`, in the operands' type.

    norm and entropy are what the forward call returned; g_logprob and
    g_entropy float32 (N,), each None for 0.
    """
    dt, ldh, ldw, n, d, v, dev = _head(hidden, weight)
    _norm(norm, n, dev)
    f32 = torch.float32
    t, h, gl, gh = (_row(a, n, nm, ty, dev) for a, nm, ty in (
        (targets, "targets", torch.int32), (entropy, "entropy", f32),
        (g_logprob, "g_logprob", f32), (g_entropy, "g_entropy", f32)))
    ws, nb = _scratch(lib.gmm_head_score_backward_workspace_bytes(n, d, v, dt), ws, dev)
    dh = torch.empty((n, d), dtype=hidden.dtype, device=dev)
    dw = torch.empty((v, d), dtype=weight.dtype, device=dev)
    with _On(dev) as stream:
        _check(lib.gmm_head_score_backward(hidden.data_ptr(), n, d, ldh, weight.data_ptr(), v, ldw, dt,
                                           t, norm.data_ptr(), h, gl, gh, scale, dh.data_ptr(), d,
                                           dw.data_ptr(), d, ws.data_ptr(), nb, stream))
    return dh, dw


def moe_layer(x, w_in, w_out, gate=None, m: int = 2, share_all: bool = False, idx=None, resp=None,
              ws=None):
    """Mixture-of-experts layer of x (N, D): (y (N, D), idx int32 (N, m), resp float32 (N, m)).

    w_in (E, 2F, D) and w_out (E, D, F), contiguous, in x's type (float32 or
    bfloat16). With gate (E, D) the m experts of largest gate logit are picked
    and weighted by a softmax over them (over all experts with share_all);
    without, idx and resp (N, m) give the picks and their weights, as
    :func:`assign_topm` returns them. See gmm_moe_layer in ``include/gmm_em.h``.
    """
    dt, ldx = _rows2(x, "x")
    n, d = x.shape
    dev = x.device
    e = w_in.shape[0]
    f = w_out.shape[-1]
    for t, nm, shape in ((w_in, "w_in", (e, 2 * f, d)), (w_out, "w_out", (e, d, f)),
                         (gate, "gate", (e, d))):
        if t is not None and (tuple(t.shape) != shape or t.dtype != x.dtype or t.device != dev
                              or not t.is_contiguous()):
            raise ValueError(f"{nm} must be a contiguous tensor {shape} of x's type and device")
    if (gate is None) != (idx is not None) or (idx is None) != (resp is None):
        raise ValueError("give either gate, or idx and resp")
    if gate is None:
        m = idx.shape[1] if idx.dim() == 2 else -1
        for t, nm, ty in ((idx, "idx", torch.int32), (resp, "resp", torch.float32)):
            if t.dtype != ty or tuple(t.shape) != (n, m) or not t.is_contiguous() or t.device != dev:
                raise ValueError(f"{nm} must be a contiguous (N, m) tensor of {ty} on x's device")
    _int32(d, f, e, m)
    ws, nb = _scratch(lib.gmm_moe_layer_workspace_bytes(n, d, f, e, dt, m), ws, dev)
    if gate is not None:
        idx = torch.empty((n, m), dtype=torch.int32, device=dev)
        resp = torch.empty((n, m), dtype=torch.float32, device=dev)
    y = torch.empty((n, d), dtype=x.dtype, device=dev)
    with _On(dev) as stream:
        _check(lib.gmm_moe_layer(x.data_ptr(), n, d, ldx, _addr(gate), e, w_in.data_ptr(),
                                 w_out.data_ptr(), f, dt, m, int(share_all), idx.data_ptr(),
                                 resp.data_ptr(), y.data_ptr(), d, ws.data_ptr(), nb, stream))
    return y, idx, resp


def _call(fn, device, *args):
    """An entry point on ``device``'s current stream, with the device made current."""
    index = device.index
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != GMM_OK:
        raise GmmError(rc)


_UNUSED = {}  # a buffer for each device that no kernel touches


def _scratch_or_none(need, ws, device):
    """:func:`_scratch` for entry points that need 256 bytes where they use none of them."""
    if need == 256 and ws is None:
        ws = _UNUSED.get(device)
        if ws is None:
            ws = _UNUSED[device] = torch.empty(256, dtype=torch.uint8, device=device)
        return ws, 256
    return _scratch(need, ws, device)


def _new_like_rows(out, n, d, x, name="out"):
    """(tensor, leading dimension) of an (n, d) result in x's type: the caller's, or a new one."""
    if out is None:
        return x.new_empty((n, d)), d
    if tuple(out.shape) != (n, d) or out.dtype != x.dtype or out.device != x.device:
        raise ValueError(f"{name} must be an ({n}, {d}) tensor of the operand's type and device")
    return out, _rows2(out, name)[1]


def embed(table, codes, scale: float = 1.0, out=None):
    """Rows scale * table[codes] (N, D), in the table's type.

    table (V, D) float32 or bfloat16, rows of any stride; codes int32 (N,): a negative
    one gives a row of 0, one of V or more a row of NaN. See gmm_embed in ``include/gmm_em.h``.
    """
    dt, ldt = _rows2(table, "table")
    v, d = table.shape
    _int32(v, d)
    dev = table.device
    n = codes.numel()
    c = _row(codes, n, "codes", torch.int32, dev)
    out, ldo = _new_like_rows(out, n, d, table)
    _call(lib.gmm_embed, dev, table.data_ptr(), v, d, ldt, dt, c, n, scale, out.data_ptr(), ldo)
    return out


def embed_backward(grad, codes, v: int, scale: float = 1.0, out=None, ws=None):
    """Gradient (V, D) of :func:`embed` with respect to its table, in the type of grad (N, D).

    Sums in float32 in a fixed order. See gmm_embed_backward in ``include/gmm_em.h``.
    """
    dt, ldg = _rows2(grad, "grad")
    n, d = grad.shape
    _int32(d, v)
    dev = grad.device
    c = _row(codes, n, "codes", torch.int32, dev)
    ws, nb = _scratch_or_none(lib.gmm_embed_backward_workspace_bytes(n, d, v), ws, dev)
    out, ldt = _new_like_rows(out, v, d, grad)
    _call(lib.gmm_embed_backward, dev, grad.data_ptr(), n, d, ldg, dt, c, v, scale, out.data_ptr(), ldt,
          ws.data_ptr(), nb)
    return out


def _bytes2(t, name):
    """Leading dimension of a 2-D row-major int8 device tensor."""
    if t.dtype != torch.int8:
        raise TypeError(f"{name} must be int8")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor with unit stride along columns")
    (n, d), (step, unit) = t.shape, t.stride()
    if unit != 1 and d > 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit stride along columns")
    if n > 1 and step < d:
        raise ValueError(f"the rows of {name} must not overlap")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return step if step > d else d


def quantize_rows(x):
    """Rows in 8-bit integers: (q int8 (N, D), scale float32 (N,)) with x close to q * scale[:, None].

    scale = max |x| / 127 of the row. See gmm_quantize_rows in ``include/gmm_em.h``.
    """
    dt, ldx = _rows2(x, "x")
    n, d = x.shape
    _int32(d)
    q = torch.empty((n, d), dtype=torch.int8, device=x.device)
    scale = torch.empty(n, dtype=torch.float32, device=x.device)
    _call(lib.gmm_quantize_rows, x.device, x.data_ptr(), n, d, ldx, dt, q.data_ptr(), d, scale.data_ptr())
    return q, scale


def quantized_product(q, q_scale, weight, weight_scale, dtype=torch.bfloat16, out=None, ws=None):
    """(q * q_scale[:, None]) @ (weight * weight_scale[:, None]).T (N, V) of int8 rows, in ``dtype``.

    q (N, D) and weight (V, D) int8, rows of any stride, with float32 scales of their rows, as
    :func:`quantize_rows` returns them. Sums are exact. See gmm_quantized_product in
    ``include/gmm_em.h``.
    """
    ldq, ldw = _bytes2(q, "q"), _bytes2(weight, "weight")
    n, d = q.shape
    v = weight.shape[0]
    if weight.shape[1] != d or weight.device != q.device:
        raise ValueError("q (N, D) and weight (V, D) must agree in D and device")
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError("dtype must be float32 or bfloat16")
    _int32(d, v)
    dev = q.device
    qs = _row(q_scale, n, "q_scale", torch.float32, dev)
    wsc = _row(weight_scale, v, "weight_scale", torch.float32, dev)
    need = lib.gmm_quantized_product_call_workspace_bytes(q.data_ptr(), n, d, ldq, weight.data_ptr(), v, ldw)
    ws, nb = _scratch_or_none(need, ws, dev)
    if out is None:
        out, ldy = torch.empty((n, v), dtype=dtype, device=dev), v
    elif tuple(out.shape) != (n, v) or out.dtype != dtype or out.device != dev:
        raise ValueError(f"out must be an ({n}, {v}) tensor of dtype on q's device")
    else:
        ldy = _rows2(out, "out")[1]
    _call(lib.gmm_quantized_product, dev, q.data_ptr(), n, d, ldq, qs, weight.data_ptr(), v, ldw, wsc,
          out.data_ptr(), ldy, dt, ws.data_ptr(), nb)
    return out


class Beams(NamedTuple):
    """What :func:`beam_step` returns, best beam first; places without a beam hold -1, -1 and -inf."""

    parent: torch.Tensor  # (B, m) int32: the beam that is continued
    code: torch.Tensor    # (B, m) int32: its next code
    score: torch.Tensor   # (B, m) float32


def _grid2(t, shape, name, dtype, device):
    """Address of a contiguous 2-D tensor of a given shape."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {shape} tensor of {dtype} on the operand's device")
    return t.data_ptr()


def beam_step(logits, scores, last=None, end: int = -1, m: Optional[int] = None, scale: float = 1.0,
              ws=None) -> Beams:
    """The m best continuations of each search's beams (m = W unless given).

    logits (B * W, V) float32 or bfloat16; scores float32 (B, W), the beams' log-probabilities so
    far (not finite: no beam); last int32 (B, W), their last codes: a beam whose last code is
    ``end`` (not negative) goes on as itself. See gmm_beam_step in ``include/gmm_em.h``.
    """
    dt, ldl = _rows2(logits, "logits")
    dev = logits.device
    if scores.dim() != 2:
        raise ValueError("scores must be a (B, W) tensor")
    b, w = scores.shape
    m = w if m is None else m
    n, v = logits.shape
    if n != b * w:
        raise ValueError("logits must have B * W rows")
    _int32(v, w, m)
    if not -0x80000000 <= end <= 0x7fffffff:
        raise GmmError(GMM_E_INVALID)
    sc = _grid2(scores, (b, w), "scores", torch.float32, dev)
    la = None if last is None else _grid2(last, (b, w), "last", torch.int32, dev)
    ws, nb = _scratch(lib.gmm_beam_step_workspace_bytes(b, w, v, m), ws, dev)
    parent = torch.empty((b, m), dtype=torch.int32, device=dev)
    out = Beams(parent, torch.empty_like(parent), scores.new_empty((b, m)))
    _call(lib.gmm_beam_step, dev, logits.data_ptr(), b, w, v, ldl, dt, sc, la, end, m, scale,
          out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), ws.data_ptr(), nb)
    return out


def _state(t, dim, name):
    """(outer, outer stride, row stride, row bytes) of a tensor as rows along ``dim``, in bytes."""
    if t.is_contiguous():
        row = t.element_size()
        for k in t.shape[dim + 1:]:
            row *= k
        step = row * t.shape[dim]
        return t.numel() * t.element_size() // step, step, row, row
    size, stride, es = list(t.shape), list(t.stride()), t.element_size()
    inner = 1
    for k in range(t.dim() - 1, dim, -1):
        if size[k] != 1:
            if stride[k] != inner:
                raise ValueError(f"the dims of {name} behind dim must be contiguous")
            inner *= size[k]
    outer, step = 1, 0
    for k in range(dim - 1, -1, -1):
        if size[k] != 1:
            if outer == 1:
                step = stride[k]
            elif stride[k] != step * outer:
                raise ValueError(f"the dims of {name} before dim must form one")
            outer *= size[k]
    return outer, step * es, stride[dim] * es if size[dim] > 1 else inner * es, inner * es


def beam_reorder(state, parent, w: int, dim: int = 0, out=None):
    """The states of the beams that :func:`beam_step` chose, for states of any type.

    state's dim ``dim`` holds the B * w beams before the step (as one row of logits each), the
    result's the B * m after it; parent int32 (B, m). A place without a parent gets 0. out may be
    the state itself (m = w): rows that stay are then not touched. See gmm_beam_reorder in
    ``include/gmm_em.h``.
    """
    if not state.is_cuda:
        raise ValueError("state must be a device tensor")
    # (a view that stands for the negated values of its memory is none: bytes are moved)
    if state.is_complex() or state.is_quantized or state.layout is not torch.strided or state.is_neg():
        raise TypeError("state must be a plain strided tensor")
    dims = state.dim()
    if not -dims <= dim < dims:
        raise ValueError("dim must be a dim of state")
    if dim < 0:
        dim += dims
    if parent.dim() != 2:
        raise ValueError("parent must be a (B, m) tensor")
    dev = state.device
    b, m = parent.shape
    pa = _grid2(parent, (b, m), "parent", torch.int32, dev)
    shape = list(state.shape)
    if shape[dim] != b * w:
        raise ValueError("state must have B * w rows along dim")
    _int32(w, m)
    if w == 0:
        raise GmmError(GMM_E_INVALID)
    shape[dim] = b * m
    new = out is None
    if new:
        out = state.new_empty(shape)
    elif list(out.shape) != shape or out.dtype != state.dtype or out.device != dev or out.is_neg():
        raise ValueError("out must have state's shape with B * m rows, its type and device")
    if out.numel() == 0:
        return out
    outer, so, sr, nb = _state(state, dim, "state")
    oo, orow = (b * m * nb, nb) if new else _state(out, dim, "out")[1:3]
    _call(lib.gmm_beam_reorder, dev, state.data_ptr(), outer, so, b, w, sr, nb, pa, m, out.data_ptr(), oo, orow)
    return out


class Balance(NamedTuple):
    """What :func:`balance_loss` returns."""

    loss: torch.Tensor    # () float32
    counts: torch.Tensor  # (E,) int32: picks of each expert
    totals: torch.Tensor  # (2,) int64: rows with a pick, picks
    prob: torch.Tensor    # (E,) float32: mean probability over those rows
    norm: torch.Tensor    # (N, 2) float32, for the gradient


def balance_loss(logits, idx, ws=None) -> Balance:
    """Balance loss E * sum(share of the picks * mean probability) of a router, and what it is made of.

    logits (N, E) float32 or bfloat16; idx int32 (N, m), the picks, as :func:`moe_layer` and
    :func:`assign_topm` return them; those outside [0, E) are none and a row without any is left
    out. See gmm_balance_loss in ``include/gmm_em.h``.
    """
    dt, ldz = _rows2(logits, "logits")
    n, e = logits.shape
    dev = logits.device
    if idx.dim() != 2:
        raise ValueError("idx must be an (N, m) tensor")
    m = idx.shape[1]
    ix = _grid2(idx, (n, m), "idx", torch.int32, dev)
    _int32(e, m)
    ws, nb = _scratch(lib.gmm_balance_loss_workspace_bytes(n, e, m), ws, dev)
    f32 = torch.float32
    out = Balance(torch.empty((), dtype=f32, device=dev), torch.empty(e, dtype=torch.int32, device=dev),
                  torch.empty(2, dtype=torch.int64, device=dev), torch.empty(e, dtype=f32, device=dev),
                  torch.empty((n, 2), dtype=f32, device=dev))
    _call(lib.gmm_balance_loss, dev, logits.data_ptr(), n, e, ldz, dt, ix, m, out[0].data_ptr(),
          out[1].data_ptr(), out[2].data_ptr(), out[3].data_ptr(), out[4].data_ptr(),
          ws.data_ptr(), nb)
    return out


def balance_loss_backward(logits, counts, totals, norm, g_loss=None, out=None):
    """Gradient of :func:`balance_loss`'s loss with respect to the logits, in their type.

    counts, totals and norm are what the forward call returned; g_loss a float32 device tensor
    of one value, None for 1. out may be the logits themselves.
    """
    dt, ldz = _rows2(logits, "logits")
    n, e = logits.shape
    dev = logits.device
    _int32(e)
    _norm(norm, n, dev)
    c = _row(counts, e, "counts", torch.int32, dev)
    t = _row(totals, 2, "totals", torch.int64, dev)
    if g_loss is not None and (g_loss.dtype != torch.float32 or g_loss.numel() != 1 or g_loss.device != dev):
        raise ValueError("g_loss must be a float32 tensor of one value on the device of the logits")
    out, ldo = _new_like_rows(out, n, e, logits)
    _call(lib.gmm_balance_loss_backward, dev, logits.data_ptr(), n, e, ldz, dt, c, t, norm.data_ptr(),
          _addr(g_loss), out.data_ptr(), ldo)
    return out


def device_status(ws, device="cuda") -> int:
    """Synchronise and return the status of the last call that used ``ws``."""
    return int(lib.gmm_device_status(_ptr(ws), _stream(torch.device(device))))


(GMM_ESTEP_FP64, GMM_ESTEP_INT8_SLICES, GMM_ESTEP_INT8_SLICES_BOTH, GMM_ESTEP_INT8_SLICES_MSTEP,
 GMM_ESTEP_BF16_SPLIT) = 0, 1, 2, 3, 4


def estep_arithmetic(ws, device="cuda") -> int:
    """Synchronise; the gmm_estep_kind of the last EM step / log-likelihood /
    k-means / top-m assignment call on ``ws``: GMM_ESTEP_FP64, GMM_ESTEP_INT8_SLICES (normaliser pass on exact
    int8 slices), GMM_ESTEP_INT8_SLICES_BOTH (both passes) or
    GMM_ESTEP_INT8_SLICES_MSTEP (both passes, and the M-step too) or
    GMM_ESTEP_BF16_SPLIT (bf16 data: both passes on split bf16)."""
    return int(lib.gmm_estep_arithmetic(_ptr(ws), _stream(torch.device(device))))


def profile_begin(max_launches: int = 4096) -> None:
    """Record HIP events around every pass-1/pass-2 launch until profile_end()."""
    _check(lib.gmm_profile_begin(max_launches))


def profile_end():
    """Returns {"pass1": (total_ms, launches), "pass2": (total_ms, launches)}."""
    a, b, na, nb = _f64(0), _f64(0), _i32(0), _i32(0)
    _check(lib.gmm_profile_end(ctypes.byref(a), ctypes.byref(na), ctypes.byref(b), ctypes.byref(nb)))
    return {"pass1": (a.value, na.value), "pass2": (b.value, nb.value)}
