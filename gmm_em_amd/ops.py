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
           lib.gmm_head_score, lib.gmm_head_score_backward, lib.gmm_moe_layer, lib.gmm_device_status, lib.gmm_profile_begin, lib.gmm_profile_end):
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


def _rows2(t, name):
    """(dtype code, leading dimension) of a 2-D row-major device tensor."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be a 2-D tensor with unit stride along columns")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"the rows of {name} must not overlap")
    if t.dtype == torch.float32:
        dt = GMM_F32
    elif t.dtype == torch.bfloat16:
        dt = GMM_BF16
    else:
        raise TypeError(f"{name} must be float32 or bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return dt, max(t.stride(0), t.shape[1])


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
        if torch.cuda.current_device() != index:
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
