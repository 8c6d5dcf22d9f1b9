"""MI355X-native fused EM for Gaussian mixture models.

Python names mirror the C ABI of include/gmm.h.  They take torch tensors that
live on the GPU, fill the descriptor structs and call libgmm.so on the current
torch stream; every step of the computation runs in the HIP kernels.

  gmm_workspace_bytes(X, K, cov, op)          -> int
  gmm_estep_stats(X, w, mu, cv, stats, accumulate=False, ws=None)
  gmm_mstep(stats, n_total, w, mu, cv, reg_covar=1e-6, comp_status=None)
  gmm_fit_step(X, w, mu, cv, reg_covar=1e-6, mean_loglik=None, comp_status=None, ws=None)
  gmm_fit(X, w, mu, cv, cov, n_iter, reg_covar=1e-6, mean_loglik=None, comp_status=None, ws=None)
  gmm_fit_step_noalloc(X, w, mu, cv, cov, reg_covar=1e-6, mean_loglik=None, comp_status=None)
  gmm_fit_step_streamed(X_host, w, mu, cv, cov, chunk_rows, reg_covar=1e-6, mean_loglik=None,
                        comp_status=None, ws=None, copy_stream=None)   (rows stay in host memory)
  gmm_predict_proba_topm(X, w, mu, cv, m, threshold, idx, resp, count=None, logp=None, ws=None)
  gmm_ivf_lists(idx, K, resp=None, offsets=None, rows=None, list_resp=None, ws=None)
  gmm_kmeans_workspace_bytes(X, K)            -> int
  gmm_kmeans_step(X, centroids, labels=None, counts=None, inertia=None, ws=None)
  gmm_fisher_vector(X, w, mu, var, power=True, l2=True, fv=None, ws=None)
  gmm_topk_fit_step(X, w, mu, cv, cov, topk, reg_covar=1e-6, mean_loglik=None, comp_status=None, ws=None)
  gmm_kde_score(Y, ref, bandwidth, out=None, ws=None)
  gmm_softmax_xent(X, W, labels, bias=None, loss=None, lse=None, ws=None)             -> (loss, lse)
  gmm_softmax_xent_grad(X, W, labels, lse, gloss=None, bias=None, dX=None, dW=None, dbias=None,
                        accumulate=False, ws=None)                                    -> (dX, dW, dbias)
  gmm_codebook_lookup(table, idx, weights=None, scale=1.0, out=None)                  -> rows
  gmm_codebook_lookup_grad(dout, idx, K, table=None, weights=None, scale=1.0, dtable=None, dweights=None,
                           accumulate=False, ws=None)                                 -> (dtable, dweights)
  gmm_clip_grad_norm(grads, max_norm, out=None, norm=None, ws=None)                   -> norm
  gmm_check_components(comp_status)          -> (status, first index or -1); synchronises

The estimator calls (score_samples, predict, score, aic, bic, fit with
restarts) are in soft_clustering_em_amd.estimator.

X is (N, D) or (B, N, D) with unit stride along D; w (B,K), mu (B,K,D) and the
covariance parameters are float32 and are updated in place by the M-step.
"""
from __future__ import annotations

import ctypes
from array import array

from . import _abi
from ._abi import (COV_CODES, GmmError, GmmData, GmmHead, GmmOptions, GmmParams, GmmStats, OP_ESTEP, OP_FIT,
                   OP_TOPM)

__all__ = ["gmm_workspace_bytes", "gmm_estep_stats", "gmm_mstep", "gmm_fit_step",
           "gmm_predict_proba_topm", "gmm_ivf_workspace_bytes", "gmm_ivf_lists", "gmm_kmeans_workspace_bytes",
           "gmm_kmeans_step", "gmm_fisher_vector_workspace_bytes", "gmm_fisher_vector",
           "gmm_topk_fit_workspace_bytes", "gmm_topk_fit_step", "gmm_softmax_xent", "gmm_softmax_xent_grad",
           "gmm_codebook_lookup", "gmm_codebook_lookup_grad", "gmm_clip_grad_norm", "new_stats", "GmmError",
           "cov_shape"]


def _torch():
    import torch
    return torch


def _dtype_code(t):
    torch = _torch()
    return {torch.float32: _abi.DT_F32, torch.bfloat16: _abi.DT_BF16, torch.float16: _abi.DT_F16}[t.dtype]


def _data(X) -> GmmData:
    if X.dim() == 2:
        B, (N, D) = 1, X.shape
        ld, sb = X.stride(0), N * X.stride(0)
    elif X.dim() == 3:
        B, N, D = X.shape
        ld, sb = X.stride(1), X.stride(0)
    else:
        raise ValueError("X must be (N, D) or (B, N, D)")
    if D > 0 and N > 0 and X.stride(-1) != 1:
        raise ValueError("X needs unit stride along D")
    return GmmData(ctypes.c_void_p(X.data_ptr()), _dtype_code(X), B, N, D, ld, sb)


def _cov_code(cov):
    return COV_CODES[cov] if isinstance(cov, str) else int(cov)


def cov_shape(cov, B, K, D):
    return {"spherical": (B, K), "diag": (B, K, D), "tied": (B, D, D), "full": (B, K, D, D)}[cov]


def _params(w, mu, cv, cov) -> GmmParams:
    for t in (w, mu, cv):
        if not t.is_contiguous():
            raise ValueError("parameter tensors must be contiguous")
    K = w.shape[-1]
    return GmmParams(K, _cov_code(cov), ctypes.c_void_p(w.data_ptr()), ctypes.c_void_p(mu.data_ptr()),
                     ctypes.c_void_p(cv.data_ptr()))


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def gmm_workspace_bytes(X, K, cov, op=OP_FIT, m=0) -> int:
    d = _data(X)
    return int(_abi.lib().gmm_workspace_bytes(ctypes.byref(d), int(K), _cov_code(cov), int(op), int(m)))


def _workspace(X, K, cov, op, m, ws):
    if ws is not None:
        return ws
    torch = _torch()
    n = gmm_workspace_bytes(X, K, cov, op, m)
    if n == 0:
        # let the compute call report the precise reason
        return torch.empty(256, dtype=torch.uint8, device=X.device)
    return torch.empty(n, dtype=torch.uint8, device=X.device)


def new_stats(B, K, D, cov, device):
    """Zeroed float64 statistics buffers (nk, sx, sxx, loglik) for gmm_estep_stats."""
    torch = _torch()
    return dict(nk=torch.zeros(B, K, dtype=torch.float64, device=device),
                sx=torch.zeros(B, K, D, dtype=torch.float64, device=device),
                sxx=torch.zeros(cov_shape(cov, B, K, D), dtype=torch.float64, device=device),
                loglik=torch.zeros(B, dtype=torch.float64, device=device))


def gmm_estep_stats(X, w, mu, cv, cov, stats, accumulate=False, ws=None, stream=None):
    d = _data(X)
    p = _params(w, mu, cv, cov)
    st = GmmStats(_ptr(stats["nk"]), _ptr(stats["sx"]), _ptr(stats["sxx"]), _ptr(stats["loglik"]))
    ws = _workspace(X, p.K, cov, OP_ESTEP, 0, ws)
    _abi.check(_abi.lib().gmm_estep_stats(ctypes.byref(d), ctypes.byref(p), ctypes.byref(st),
                                          int(bool(accumulate)), _ptr(ws), ws.numel(), _stream(stream)))
    return stats


def gmm_mstep(stats, n_total, w, mu, cv, cov, reg_covar=1e-6, comp_status=None, stream=None):
    B, K, D = stats["sx"].shape
    p = _params(w, mu, cv, cov)
    st = GmmStats(_ptr(stats["nk"]), _ptr(stats["sx"]), _ptr(stats["sxx"]), _ptr(stats["loglik"]))
    o = GmmOptions(float(reg_covar), 0, None, None)
    _abi.check(_abi.lib().gmm_mstep(B, D, ctypes.byref(st), int(n_total), ctypes.byref(p), ctypes.byref(o),
                                    _ptr(comp_status), _stream(stream)))


def gmm_fit_step(X, w, mu, cv, cov, reg_covar=1e-6, mean_loglik=None, comp_status=None, ws=None,
                 stream=None, events=None):
    """One EM iteration in place.  events: optional (begin, end) torch.cuda.Event
    pair recorded around the fused E-step kernel."""
    d = _data(X)
    p = _params(w, mu, cv, cov)
    eb = ee = None
    if events is not None:
        eb, ee = (ctypes.c_void_p(e.cuda_event) for e in events)
    o = GmmOptions(float(reg_covar), 0, eb, ee)
    ws = _workspace(X, p.K, cov, OP_FIT, 0, ws)
    _abi.check(_abi.lib().gmm_fit_step(ctypes.byref(d), ctypes.byref(p), ctypes.byref(o), _ptr(mean_loglik),
                                       _ptr(comp_status), _ptr(ws), ws.numel(), _stream(stream)))


def gmm_fit(X, w, mu, cv, cov, n_iter, reg_covar=1e-6, mean_loglik=None, comp_status=None, ws=None, stream=None,
            events=None):
    """n_iter EM iterations in place, the results of n_iter gmm_fit_step calls.
    mean_loglik: optional (n_iter, B) float64 device tensor, row t the mean
    log-likelihood entering iteration t.  events: optional (begin, end) pair
    recorded around the last iteration's E-step."""
    d = _data(X)
    p = _params(w, mu, cv, cov)
    if mean_loglik is not None:
        import torch
        if (mean_loglik.dtype != torch.float64 or not mean_loglik.is_cuda or not mean_loglik.is_contiguous()
                or mean_loglik.numel() < int(n_iter) * int(d.B)):
            raise ValueError("mean_loglik must be a contiguous float64 device tensor of n_iter * B elements")
    eb = ee = None
    if events is not None:
        eb, ee = (ctypes.c_void_p(e.cuda_event) for e in events)
    o = GmmOptions(float(reg_covar), 0, eb, ee)
    ws = _workspace(X, p.K, cov, OP_FIT, 0, ws)
    _abi.check(_abi.lib().gmm_fit(ctypes.byref(d), ctypes.byref(p), ctypes.byref(o), int(n_iter),
                                  _ptr(mean_loglik), _ptr(comp_status), _ptr(ws), ws.numel(), _stream(stream)))


def gmm_fit_step_noalloc(X, w, mu, cv, cov, reg_covar=1e-6, mean_loglik=None, comp_status=None, stream=None):
    """One EM iteration in place, with the library's static scratch array
    instead of a workspace (nothing is allocated on the device)."""
    d = _data(X)
    p = _params(w, mu, cv, cov)
    o = GmmOptions(float(reg_covar), 0, None, None)
    _abi.check(_abi.lib().gmm_fit_step_noalloc(ctypes.byref(d), ctypes.byref(p), ctypes.byref(o),
                                               _ptr(mean_loglik), _ptr(comp_status), _stream(stream)))


def gmm_fit_step_streamed_workspace_bytes(X_host, K, cov, chunk_rows) -> int:
    d = _data(X_host)
    return int(_abi.lib().gmm_fit_step_streamed_workspace_bytes(ctypes.byref(d), int(K), _cov_code(cov),
                                                                int(chunk_rows)))


def gmm_fit_step_streamed(X_host, w, mu, cv, cov, chunk_rows, reg_covar=1e-6, mean_loglik=None, comp_status=None,
                          ws=None, stream=None, copy_stream=None):
    """One EM iteration in place over rows in host memory (X_host: a CPU
    tensor, pinned for overlapped copies), streamed through two device chunk
    buffers of chunk_rows rows; copy_stream: a torch.cuda.Stream for the
    copies (None: the compute stream)."""
    torch = _torch()
    if X_host.is_cuda:
        raise ValueError("gmm_fit_step_streamed takes rows in host memory")
    d = _data(X_host)
    p = _params(w, mu, cv, cov)
    o = GmmOptions(float(reg_covar), 0, None, None)
    if ws is None:
        n = gmm_fit_step_streamed_workspace_bytes(X_host, p.K, cov, chunk_rows)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=w.device)
    cs = None if copy_stream is None else ctypes.c_void_p(copy_stream.cuda_stream)
    _abi.check(_abi.lib().gmm_fit_step_streamed(ctypes.byref(d), ctypes.byref(p), ctypes.byref(o), int(chunk_rows),
                                                _ptr(mean_loglik), _ptr(comp_status), _ptr(ws), ws.numel(),
                                                _stream(stream), cs))


def gmm_predict_proba_topm(X, w, mu, cv, cov, m, threshold, idx, resp, count=None, logp=None, ws=None,
                           stream=None):
    d = _data(X)
    p = _params(w, mu, cv, cov)
    ws = _workspace(X, p.K, cov, OP_TOPM, m, ws)
    _abi.check(_abi.lib().gmm_predict_proba_topm(ctypes.byref(d), ctypes.byref(p), int(m), float(threshold),
                                                 _ptr(idx), _ptr(resp), _ptr(count), _ptr(logp), _ptr(ws),
                                                 ws.numel(), _stream(stream)))


def gmm_ivf_workspace_bytes(B, N, m, K) -> int:
    return int(_abi.lib().gmm_ivf_workspace_bytes(int(B), int(N), int(m), int(K)))


def gmm_ivf_lists(idx, K, resp=None, offsets=None, rows=None, list_resp=None, ws=None, stream=None):
    """Posting lists of a multi-assignment idx ((N, m) or (B, N, m) int32 on the GPU).

    Returns (offsets (B, K+1) int64, rows (B, N*m) int32, list_resp (B, N*m) float32 or None);
    outputs not given are allocated here (rows and list_resp past offsets[b, K] are left as
    allocated)."""
    torch = _torch()
    if idx.dim() == 2:
        idx = idx.unsqueeze(0)
        resp = resp.unsqueeze(0) if resp is not None else None
    if not idx.is_contiguous() or idx.dtype != torch.int32:
        raise ValueError("idx must be a contiguous int32 tensor")
    if resp is not None and (not resp.is_contiguous() or resp.dtype != torch.float32 or resp.shape != idx.shape):
        raise ValueError("resp must be a contiguous float32 tensor shaped like idx")
    B, N, m = idx.shape
    dev = idx.device
    if offsets is None:
        offsets = torch.empty(B, K + 1, dtype=torch.int64, device=dev)
    if rows is None:
        rows = torch.empty(B, N * m, dtype=torch.int32, device=dev)
    if list_resp is None and resp is not None:
        list_resp = torch.empty(B, N * m, dtype=torch.float32, device=dev)
    if ws is None:
        n = gmm_ivf_workspace_bytes(B, N, m, K)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    _abi.check(_abi.lib().gmm_ivf_lists(int(B), int(N), int(m), int(K), _ptr(idx), _ptr(resp), _ptr(offsets),
                                        _ptr(rows), _ptr(list_resp), _ptr(ws), ws.numel(), _stream(stream)))
    return offsets, rows, list_resp


def gmm_kmeans_workspace_bytes(X, K) -> int:
    d = _data(X)
    return int(_abi.lib().gmm_kmeans_workspace_bytes(ctypes.byref(d), int(K)))


def gmm_kmeans_step(X, centroids, labels=None, counts=None, inertia=None, ws=None, stream=None):
    """One k-means (Lloyd) iteration; centroids ((K, D) or (B, K, D) float32)
    are replaced by the cluster means.  Returns (labels (B, N) int32 under the
    entering centroids, counts (B, K) int64, inertia (B,) float64); outputs
    not given are allocated here."""
    torch = _torch()
    d = _data(X)
    B, N = int(d.B), int(d.N)
    K = centroids.shape[-2]
    if centroids.dtype != torch.float32 or not centroids.is_contiguous() or centroids.numel() != B * K * d.D:
        raise ValueError("centroids must be a contiguous float32 tensor of B*K*D elements")
    dev = centroids.device
    if labels is None:
        labels = torch.empty(B, N, dtype=torch.int32, device=dev)
    if counts is None:
        counts = torch.empty(B, K, dtype=torch.int64, device=dev)
    if inertia is None:
        inertia = torch.empty(B, dtype=torch.float64, device=dev)
    if ws is None:
        n = gmm_kmeans_workspace_bytes(X, K)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    _abi.check(_abi.lib().gmm_kmeans_step(ctypes.byref(d), int(K), _ptr(centroids), _ptr(labels), _ptr(counts),
                                          _ptr(inertia), _ptr(ws), ws.numel(), _stream(stream)))
    return labels, counts, inertia


def gmm_fisher_vector_workspace_bytes(X, K) -> int:
    d = _data(X)
    return int(_abi.lib().gmm_fisher_vector_workspace_bytes(ctypes.byref(d), int(K)))


def gmm_fisher_vector(X, w, mu, var, power=True, l2=True, fv=None, ws=None, stream=None):
    """Fisher vectors of the sets X ((N, D) or (B, N, D) float32) under one
    diagonal model (w (K,), mu (K, D), var (K, D) float32): (B, 2 K D)
    float32, [G_mu, G_sigma] per set, optionally with the signed square root
    (power) and L2 normalisation."""
    torch = _torch()
    d = _data(X)
    B, K, D = int(d.B), int(w.shape[-1]), int(d.D)
    if mu.numel() != K * D or var.numel() != K * D:
        raise ValueError("the model is one diagonal GMM: w (K,), mu and var (K, D)")
    p = GmmParams(K, COV_CODES["diag"], ctypes.c_void_p(w.data_ptr()), ctypes.c_void_p(mu.data_ptr()),
                  ctypes.c_void_p(var.data_ptr()))
    if fv is None:
        fv = torch.empty(B, 2 * K * D, dtype=torch.float32, device=w.device)
    if ws is None:
        n = gmm_fisher_vector_workspace_bytes(X, K)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=w.device)
    flags = (1 if power else 0) | (2 if l2 else 0)
    _abi.check(_abi.lib().gmm_fisher_vector(ctypes.byref(d), ctypes.byref(p), flags, _ptr(fv), _ptr(ws), ws.numel(),
                                            _stream(stream)))
    return fv


def gmm_topk_fit_workspace_bytes(X, K, cov, topk) -> int:
    d = _data(X)
    return int(_abi.lib().gmm_topk_fit_workspace_bytes(ctypes.byref(d), int(K), _cov_code(cov), int(topk)))


def gmm_kde_workspace_bytes(Y, M) -> int:
    d = _data(Y)
    return int(_abi.lib().gmm_kde_workspace_bytes(ctypes.byref(d), int(M)))


def gmm_kde_score(Y, ref, bandwidth, out=None, ws=None, stream=None):
    """Log of the Gaussian kernel density estimate with bandwidth h over the
    reference rows ref ((M, D) float32) at the query rows Y ((N, D) or
    (B, N, D) float32): float32 of Y's leading shape."""
    torch = _torch()
    d = _data(Y)
    if ref.dim() != 2 or ref.shape[1] != d.D or ref.dtype != torch.float32:
        raise ValueError("ref must be (M, D) float32 with the queries' D")
    if ref.shape[0] > 0 and ref.stride(1) != 1:
        raise ValueError("ref needs unit stride along D")
    M = int(ref.shape[0])
    if out is None:
        out = torch.empty(Y.shape[:-1], dtype=torch.float32, device=Y.device)
    if ws is None:
        n = gmm_kde_workspace_bytes(Y, M)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=Y.device)
    _abi.check(_abi.lib().gmm_kde_score(ctypes.byref(d), _ptr(ref), M, int(ref.stride(0)), float(bandwidth), _ptr(out),
                                        _ptr(ws), ws.numel(), _stream(stream)))
    return out


def gmm_topk_fit_step(X, w, mu, cv, cov, topk, reg_covar=1e-6, mean_loglik=None, comp_status=None, ws=None,
                      stream=None):
    """One approximate top-k EM iteration in place (each row keeps its topk
    best components and normalises over them)."""
    torch = _torch()
    d = _data(X)
    p = _params(w, mu, cv, cov)
    o = GmmOptions(float(reg_covar), 0, None, None)
    if ws is None:
        n = gmm_topk_fit_workspace_bytes(X, p.K, cov, topk)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=X.device)
    _abi.check(_abi.lib().gmm_topk_fit_step(ctypes.byref(d), ctypes.byref(p), int(topk), ctypes.byref(o),
                                            _ptr(mean_loglik), _ptr(comp_status), _ptr(ws), ws.numel(),
                                            _stream(stream)))


class _on:
    """The device of a call's tensors as the current one, and the stream that
    the call runs on as the current stream (the caller's own, or the device's
    current one), so that a workspace allocated inside belongs to it."""

    __slots__ = ("guards", "stream")

    def __init__(self, stream, *tensors):
        torch = _torch()
        index = tensors[0].get_device()  # -1: not on a GPU
        for t in tensors:
            if t is not None and (index < 0 or t.get_device() != index):
                raise ValueError(f"every tensor must be on one GPU (got {t.device} and {tensors[0].device})")
        if stream is not None and stream.device.index != index:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {tensors[0].device}")
        # a guard costs microseconds: none where the call changes nothing
        self.guards = [torch.cuda.device(index)] if torch.cuda.current_device() != index else []
        if stream is not None:
            self.guards.append(torch.cuda.stream(stream))
            for t in tensors:  # memory freed by its owner while this stream still reads it
                if t is not None:
                    t.record_stream(stream)
        self.stream = stream if stream is not None else torch.cuda.current_stream(index)

    def __enter__(self):
        for c in self.guards:
            c.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        for c in reversed(self.guards):
            c.__exit__(*exc)


def _expect(name, t, dtype, shape):
    """t as the library takes it: a contiguous tensor of one type and shape."""
    if t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"(got {t.dtype}, {tuple(t.shape)})")


def _check_ws(ws):
    """A caller's workspace is one block of ws.numel() elements: an expanded or
    strided view covers less, or more, than it counts."""
    if ws is not None and not ws.is_contiguous():
        raise ValueError("ws must be a contiguous tensor")


def _rows(name, t):
    """The gmm_data of rows at any strides that keep D contiguous and rows apart."""
    torch = _torch()
    if t.dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise ValueError(f"{name} must be float32, bfloat16 or float16 (got {t.dtype})")
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be (N, D) or (B, N, D)")
    D = int(t.shape[-1])
    if D < 1 or (t.dim() == 3 and t.shape[0] < 1):
        raise ValueError(f"{name} needs B >= 1 and D >= 1")
    if D > 1 and t.numel() > 0 and t.stride(-1) != 1:
        raise ValueError(f"{name} needs unit stride along D")
    # strides along an axis of one element mean nothing
    N = int(t.shape[-2])
    ld = int(t.stride(-2)) if N > 1 else D
    if t.dim() == 2:
        return GmmData(ctypes.c_void_p(t.data_ptr()), _dtype_code(t), 1, N, D, max(ld, D) if N <= 1 else ld, N * ld)
    B = int(t.shape[0])
    sb = int(t.stride(0)) if B > 1 else N * ld
    return GmmData(ctypes.c_void_p(t.data_ptr()), _dtype_code(t), B, N, D, ld, max(sb, N * ld) if N == 0 else sb)


def _head(X, W, bias):
    torch = _torch()
    h = _rows("W", W)
    if W.dim() != 2 or W.shape[1] != X.shape[-1] or W.dtype != X.dtype:
        raise ValueError("W must be (V, D) of the rows' D and type")
    if bias is not None:
        _expect("bias", bias, torch.float32, (W.shape[0],))
    return GmmHead(h.x, h.dtype, h.N, h.ld_x, _ptr(bias))


def gmm_softmax_xent(X, W, labels, bias=None, loss=None, lse=None, ws=None, stream=None):
    """Softmax cross entropy of the rows X ((N, D) or (B, N, D) float32,
    bfloat16 or float16) under the linear head W (V, D) of their type, with
    labels (X's leading shape, int32; negative: the row is left out).
    Returns (loss, lse), float32 of X's leading shape; lse is what
    gmm_softmax_xent_grad takes."""
    torch = _torch()
    d, h = _rows("X", X), _head(X, W, bias)
    lead = X.shape[:-1]
    _expect("labels", labels, torch.int32, lead)
    _check_ws(ws)
    with _on(stream, X, W, labels, bias, loss, lse, ws) as s:
        loss = torch.empty(lead, dtype=torch.float32, device=X.device) if loss is None else loss
        lse = torch.empty(lead, dtype=torch.float32, device=X.device) if lse is None else lse
        _expect("loss", loss, torch.float32, lead)
        _expect("lse", lse, torch.float32, lead)
        if ws is None:
            n = int(_abi.lib().gmm_softmax_xent_workspace_bytes(ctypes.byref(d), ctypes.byref(h)))
            ws = torch.empty(max(n, 256), dtype=torch.uint8, device=X.device)
        _abi.check(_abi.lib().gmm_softmax_xent(ctypes.byref(d), ctypes.byref(h), _ptr(labels), _ptr(loss), _ptr(lse),
                                               _ptr(ws), ws.numel() * ws.element_size(), s))
    return loss, lse


def _wanted(given, like, shape, dtype):
    """A gradient's buffer: the caller's, none (False), or a new one (None)."""
    torch = _torch()
    if given is False:
        return None
    return torch.empty(shape, dtype=dtype, device=like.device) if given is None else given


def gmm_softmax_xent_grad(X, W, labels, lse, gloss=None, bias=None, dX=None, dW=None, dbias=None, accumulate=False,
                          ws=None, stream=None):
    """Gradients of sum_i gloss_i loss_i (gloss: float32 of X's leading shape,
    None: ones) with the lse of gmm_softmax_xent: (dX, dW, dbias), dX (X's
    shape) and dW (V, D) in the rows' type, dbias (V,) float32 (None without a
    bias).  Buffers not given are allocated; False leaves one out.
    accumulate=True adds to the buffers, all of which are then given."""
    torch = _torch()
    d, h = _rows("X", X), _head(X, W, bias)
    lead = X.shape[:-1]
    _expect("labels", labels, torch.int32, lead)
    _expect("lse", lse, torch.float32, lead)
    _check_ws(ws)
    if gloss is not None:
        _expect("gloss", gloss, torch.float32, lead)
    if bias is None and dbias is None:
        dbias = False
    if accumulate and any(t is None for t in (dX, dW, dbias)):
        raise ValueError("accumulate=True adds to given buffers (False leaves a gradient out)")
    given = [t for t in (dX, dW, dbias) if t is not None and t is not False]
    with _on(stream, X, W, labels, lse, gloss, bias, ws, *given) as s:
        dX, dW = _wanted(dX, X, X.shape, X.dtype), _wanted(dW, W, W.shape, W.dtype)
        dbias = _wanted(dbias, W, (W.shape[0],), torch.float32)
        for name, t, like in (("dX", dX, X), ("dW", dW, W)):
            if t is not None:
                _expect(name, t, like.dtype, like.shape)
        if dbias is not None:
            _expect("dbias", dbias, torch.float32, (W.shape[0],))
        if ws is None:
            want = (dX is not None) + 2 * (dW is not None) + 4 * (dbias is not None)
            n = int(_abi.lib().gmm_softmax_xent_grad_workspace_bytes(ctypes.byref(d), ctypes.byref(h), want))
            ws = torch.empty(max(n, 256), dtype=torch.uint8, device=X.device)
        _abi.check(_abi.lib().gmm_softmax_xent_grad(ctypes.byref(d), ctypes.byref(h), _ptr(labels), _ptr(lse),
                                                    _ptr(gloss), _ptr(dX), _ptr(dW), _ptr(dbias),
                                                    int(bool(accumulate)), _ptr(ws), ws.numel() * ws.element_size(),
                                                    s))
    return dX, dW, dbias


def _code_shape(rows_dim, idx, weights):
    """(B, N, m) of codes of rows with rows_dim axes: (N,) or (N, m), with a
    leading B where the rows have one; m = 1 codes may leave their axis out."""
    torch = _torch()
    if idx.dtype != torch.int32 or not idx.is_contiguous():
        raise ValueError("idx must be a contiguous int32 tensor")
    if idx.dim() not in (rows_dim - 1, rows_dim):
        raise ValueError(f"idx must have {rows_dim - 1} or {rows_dim} axes beside rows of {rows_dim}")
    if weights is not None:
        _expect("weights", weights, torch.float32, idx.shape)
    lead = idx.shape if idx.dim() == rows_dim - 1 else idx.shape[:-1]
    m = 1 if idx.dim() == rows_dim - 1 else int(idx.shape[-1])
    return (int(lead[0]) if rows_dim == 3 else 1), int(lead[-1]), m, tuple(lead)


def gmm_codebook_lookup(table, idx, weights=None, scale=1.0, out=None, stream=None):
    """Rows rebuilt from codes: out_i = scale * sum_j weights_ij table[idx_ij]
    over a row's leading codes in [0, K).  table (K, D) or (B, K, D) float32,
    bfloat16 or float16; idx (N,), (N, m) (a leading B beside a table with
    one) int32; weights of idx's shape, float32 (None: 1).  Returns
    idx's leading shape + (D,), in the table's type."""
    torch = _torch()
    d = _rows("table", table)
    B, N, m, lead = _code_shape(table.dim(), idx, weights)
    if B != d.B:
        raise ValueError("idx and table differ in B")
    shape = lead + (int(d.D),)
    with _on(stream, table, idx, weights, out) as s:
        out = torch.empty(shape, dtype=table.dtype, device=table.device) if out is None else out
        _expect("out", out, table.dtype, shape)
        _abi.check(_abi.lib().gmm_codebook_lookup(ctypes.byref(d), N, m, _ptr(idx), _ptr(weights), float(scale),
                                                  _ptr(out), s))
    return out


def gmm_codebook_lookup_grad(dout, idx, K, table=None, weights=None, scale=1.0, dtable=None, dweights=None,
                             accumulate=False, ws=None, stream=None):
    """Gradients of gmm_codebook_lookup for the rows' gradient dout ((N, D) or
    (B, N, D)): (dtable, dweights), dtable (K, D) or (B, K, D) in dout's type,
    dweights of idx's shape, float32 (None without weights or a table).
    Buffers not given are allocated; False leaves one out.  accumulate=True
    adds to the given dtable."""
    torch = _torch()
    d = _rows("dout", dout)
    B, N, m, lead = _code_shape(dout.dim(), idx, weights)
    if (B, N) != (d.B, d.N):
        raise ValueError("idx and dout differ in their rows")
    _check_ws(ws)
    t = None
    if table is not None:
        if table.dtype != dout.dtype or table.dim() != dout.dim() or table.shape[-1] != dout.shape[-1] \
                or table.shape[-2] != K or (dout.dim() == 3 and table.shape[0] != dout.shape[0]):
            raise ValueError("table must be (K, D) or (B, K, D) of dout's type, B and D")
        t = _rows("table", table)
    if dweights is None and (table is None or weights is None):
        dweights = False
    if dweights is not False and table is None:
        raise ValueError("dweights needs the table")
    if accumulate and dtable is None:
        raise ValueError("accumulate=True adds to a given dtable")
    K = int(K)
    shape = (K, int(d.D)) if dout.dim() == 2 else (B, K, int(d.D))
    given = [x for x in (dtable, dweights) if x is not None and x is not False]
    with _on(stream, dout, idx, table, weights, ws, *given) as s:
        dtable = _wanted(dtable, dout, shape, dout.dtype)
        dweights = _wanted(dweights, dout, idx.shape, torch.float32)
        if dtable is not None:
            _expect("dtable", dtable, dout.dtype, shape)
        if dweights is not None:
            _expect("dweights", dweights, torch.float32, idx.shape)
        if ws is None:
            n = 0
            if dtable is not None:
                n = int(_abi.lib().gmm_codebook_lookup_grad_workspace_bytes(ctypes.byref(d), K, m))
            ws = torch.empty(max(n, 256), dtype=torch.uint8, device=dout.device)
        _abi.check(_abi.lib().gmm_codebook_lookup_grad(
            ctypes.byref(d), K, m, _ptr(idx), _ptr(weights), float(scale),
            ctypes.byref(t) if t is not None else None, _ptr(dtable), _ptr(dweights), int(bool(accumulate)), _ptr(ws),
            ws.numel() * ws.element_size(), s))
    return dtable, dweights


def gmm_clip_grad_norm(grads, max_norm, out=None, norm=None, ws=None, stream=None):
    """The 2-norm over all the gradients (a list of contiguous float32,
    bfloat16 or float16 tensors), which are scaled by min(1, max_norm /
    (norm + 1e-6)) in place, or into the tensors of out (same shapes and
    types).  Returns the norm before the scaling, (1,) float32."""
    torch = _torch()
    grads = list(grads)
    outs = grads if out is None else list(out)
    if not grads:
        raise ValueError("need one gradient or more")
    if len(outs) != len(grads):
        raise ValueError("out must hold one tensor per gradient")
    _check_ws(ws)
    codes = {torch.float32: _abi.DT_F32, torch.bfloat16: _abi.DT_BF16, torch.float16: _abi.DT_F16}
    desc = array("q")  # a gmm_tensor is four 8-byte words: src, dst, n, dtype
    for i, (g, o) in enumerate(zip(grads, outs)):
        code = codes.get(g.dtype)
        if code is None or not g.is_contiguous():
            raise ValueError(f"gradient {i} must be a contiguous float32, bfloat16 or float16 tensor")
        if o is not g:
            if o.dtype != g.dtype or o.shape != g.shape or not o.is_contiguous():
                _expect(f"out[{i}]", o, g.dtype, g.shape)
        desc.extend((g.data_ptr(), o.data_ptr(), g.numel(), code))
    with _on(stream, *grads, *(() if outs is grads else outs), norm, ws) as s:
        norm = torch.empty(1, dtype=torch.float32, device=grads[0].device) if norm is None else norm
        _expect("norm", norm, torch.float32, (1,))
        if ws is None:
            n = int(_abi.lib().gmm_clip_grad_norm_workspace_bytes(len(grads)))
            ws = torch.empty(n, dtype=torch.uint8, device=grads[0].device)
        _abi.check(_abi.lib().gmm_clip_grad_norm(desc.buffer_info()[0], len(grads), float(max_norm), _ptr(norm), _ptr(ws),
                                                 ws.numel() * ws.element_size(), s))
    return norm


def gmm_check_components(comp_status):
    """Copy comp_status (B, K) to the host (a synchronisation) and summarise it
    with the library's gmm_check_components: (GMM_ERR_NOT_PD, index of the
    first component whose input or updated covariance was not positive
    definite) or (GMM_OK, -1)."""
    import numpy as np
    host = np.ascontiguousarray(comp_status.detach().to("cpu").numpy(), dtype=np.int32).reshape(-1)
    first = ctypes.c_int64(-1)
    st = _abi.lib().gmm_check_components(host.ctypes.data, host.size, ctypes.byref(first))
    if st not in (_abi.GMM_OK, _abi.GMM_ERR_NOT_PD):
        _abi.check(st)
    return st, first.value
