"""Estimator-level calls over the C ABI: per-row log-likelihood, hard
assignment, mean log-likelihood, information criteria, and a fit loop with
restarts -- the estimator surface the GMMXX README lists under "Highlights"
(fit, predict, score, score_samples, aic, bic; restarts as in its estimator).

Every per-row and per-component number comes from the HIP library:
score_samples and predict from gmm_predict_proba_topm (m = 1: the best
component and log p(x_i)), score from gmm_estep_stats (sum_i log p(x_i)),
fit from gmm_fit_step (or gmm_topk_fit_step, the approximate top-k mode of
the GMMXX README), KernelDensity.score_samples from gmm_kde_score, the rows
that reconstruct rebuilds from gmm_codebook_lookup, SoftmaxHead's losses and
gradients from gmm_softmax_xent, gmm_softmax_xent_grad, gmm_clip_grad_norm and
gmm_layer_norm with its gradient, its AdamW steps from gmm_adamw_step, its
routing and its draws from gmm_route_topm and gmm_sample.  What runs here is
argument handling, the stopping rule, the AIC/BIC arithmetic on B returned
scalars, SoftmaxHead's momentum update and the library product of its logits.

  n_parameters(cov, K, D)                       -> int
  score_samples(X, w, mu, cv, cov)              -> (B, N) float32 log p(x_i)
  predict(X, w, mu, cv, cov)                    -> (B, N) int32 argmax_k r_ik
  score(X, w, mu, cv, cov)                      -> (B,) float64 mean log p(x_i)
  information_criteria(mean_ll, N, p)           -> (aic, bic), numpy
  aic(...), bic(...)                            -> (B,) float64
  fit(X, K, cov, ...)                           -> FitResult (the restart with the best mean LL)
  GaussianMixture(n_components, covariance_type, ...)  the same calls as a scikit-learn style class
  KMeans(n_clusters, ...)                       Lloyd iterations over gmm_kmeans_step (the hard limit)
  KernelDensity(bandwidth)                      Gaussian kernel density estimate over gmm_kde_score
  SoftmaxHead(n_classes, ...)                   linear softmax classifier (the discriminative posterior)
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np

from . import (gmm_adamw_step, gmm_clip_grad_norm, gmm_codebook_lookup, gmm_estep_stats, gmm_fit, gmm_fit_step,
               gmm_kde_score, gmm_kmeans_step, gmm_layer_norm, gmm_layer_norm_grad, gmm_predict_proba_topm,
               gmm_route_topm, gmm_sample, gmm_softmax_xent, gmm_softmax_xent_grad, gmm_topk_fit_step,
               gmm_topk_fit_workspace_bytes, new_adamw_state, new_stats)


def _torch():
    import torch
    return torch


def _batched(X):
    return X if X.dim() == 3 else X.unsqueeze(0)


def n_parameters(cov: str, K: int, D: int) -> int:
    """Free parameters of a K-component mixture in D dimensions: K - 1 weights,
    K D means, and the covariance parameters (spherical K, diag K D, tied
    D (D + 1) / 2, full K D (D + 1) / 2)."""
    covp = {"spherical": K, "diag": K * D, "tied": D * (D + 1) // 2, "full": K * D * (D + 1) // 2}[cov]
    return (K - 1) + K * D + covp


def information_criteria(mean_ll, N: int, p: int):
    """AIC = -2 N mean_ll + 2 p and BIC = -2 N mean_ll + p log N (Akaike;
    Schwarz), per problem."""
    total = -2.0 * np.asarray(mean_ll, dtype=np.float64) * N
    return total + 2.0 * p, total + p * math.log(N)


def _topm1(X, w, mu, cv, cov):
    torch = _torch()
    Xb = _batched(X)
    B, N = Xb.shape[0], Xb.shape[1]
    idx = torch.empty(B, N, 1, dtype=torch.int32, device=X.device)
    resp = torch.empty(B, N, 1, dtype=torch.float32, device=X.device)
    logp = torch.empty(B, N, dtype=torch.float32, device=X.device)
    gmm_predict_proba_topm(X, w, mu, cv, cov, 1, 0.0, idx, resp, logp=logp)
    return idx[..., 0], logp


def score_samples(X, w, mu, cv, cov):
    """log p(x_i) (natural log) of every row, (B, N) float32."""
    return _topm1(X, w, mu, cv, cov)[1]


def predict(X, w, mu, cv, cov):
    """The component of largest responsibility of every row (ties: lower
    index), (B, N) int32."""
    return _topm1(X, w, mu, cv, cov)[0]


def score(X, w, mu, cv, cov):
    """(1/N) sum_i log p(x_i) per problem, (B,) float64 on the host."""
    Xb = _batched(X)
    B, N, D = Xb.shape
    st = new_stats(B, w.shape[-1], D, cov, X.device)
    gmm_estep_stats(X, w, mu, cv, cov, st)
    return (st["loglik"] / N).cpu().numpy()


def aic(X, w, mu, cv, cov):
    Xb = _batched(X)
    return information_criteria(score(X, w, mu, cv, cov), Xb.shape[1], n_parameters(cov, w.shape[-1], Xb.shape[2]))[0]


def bic(X, w, mu, cv, cov):
    Xb = _batched(X)
    return information_criteria(score(X, w, mu, cv, cov), Xb.shape[1], n_parameters(cov, w.shape[-1], Xb.shape[2]))[1]


@dataclass
class FitResult:
    weights: object        # (B, K) float32, device
    means: object          # (B, K, D) float32, device
    covars: object         # covariance parameters, device
    mean_ll: np.ndarray    # (B,) mean log-likelihood of the returned parameters' last E-step
    n_iter: int
    converged: bool
    restart: int           # which restart was kept
    history: list          # per restart: list of per-iteration mean LL (problem-averaged)


def random_init(X, K, cov, generator):
    """K distinct rows of each problem as means, equal weights, and the
    problem's sample variance (spherical: its mean over dimensions; diag: per
    dimension; tied/full: the sample covariance) as every component's."""
    torch = _torch()
    Xb = _batched(X).float()
    B, N, D = Xb.shape
    if K > N:
        raise ValueError("K exceeds the number of rows")
    sel = torch.stack([torch.randperm(N, generator=generator, device="cpu")[:K] for _ in range(B)]).to(X.device)
    mu = torch.gather(Xb, 1, sel[..., None].expand(B, K, D)).contiguous()
    w = torch.full((B, K), 1.0 / K, dtype=torch.float32, device=X.device)
    xm = Xb.mean(dim=1, keepdim=True)
    var = ((Xb - xm) ** 2).mean(dim=1)  # (B, D)
    if cov == "spherical":
        cv = var.mean(dim=1, keepdim=True).expand(B, K).contiguous()
    elif cov == "diag":
        cv = var[:, None, :].expand(B, K, D).contiguous()
    else:
        Xc = (Xb - xm).contiguous()
        C = torch.bmm(Xc.transpose(1, 2).contiguous(), Xc) / N
        cv = C.contiguous() if cov == "tied" else C[:, None].expand(B, K, D, D).contiguous()
    if X.dim() == 2:
        w, mu, cv = w[0].contiguous(), mu[0].contiguous(), cv[0].contiguous()
    return w, mu, cv


def fit(X, K, cov, n_iter=100, tol=1e-3, n_init=1, reg_covar=1e-6, seed=0, init=None, topk=None, check_every=1):
    """EM from n_init starts (random_init with a seeded generator, or the
    given init = (w, mu, cv) for the first start); each runs until the change
    of the problem-averaged mean log-likelihood falls below tol or n_iter
    iterations.  Keeps the start whose last mean log-likelihood is highest.
    check_every: iterations per gmm_fit call between two reads of the
    log-likelihoods on the host (1: the test after every iteration, as above;
    c > 1: one synchronisation per c iterations, and up to c - 1 iterations
    past the one where the test first holds, which EM only improves; the
    history and n_iter still end at that iteration).
    topk: run approximate top-k EM steps instead (each row keeps its topk best
    components; spherical and diagonal covariance); the history then holds
    the top-k steps' log-likelihoods, the final score the full mixture's."""
    torch = _torch()
    tws = None
    if topk is not None:
        n = gmm_topk_fit_workspace_bytes(X, K, cov, int(topk))
        tws = torch.empty(max(n, 256), dtype=torch.uint8, device=X.device)
    gen = torch.Generator(device="cpu").manual_seed(seed)
    Xb = _batched(X)
    B = Xb.shape[0]
    best, history = None, []
    for r in range(n_init):
        if r == 0 and init is not None:
            w, mu, cv = (t.clone().contiguous() for t in init)
        else:
            w, mu, cv = random_init(X, K, cov, gen)
        hist, prev, converged, it = [], None, False, 0
        if topk is None and check_every > 1:
            # blocks of check_every iterations in one call each, their
            # log-likelihoods read once per block
            mlls = torch.zeros((int(check_every), B), dtype=torch.float64, device=X.device)
            done = 0
            while done < n_iter and not converged:
                c = min(int(check_every), n_iter - done)
                gmm_fit(X, w, mu, cv, cov, c, reg_covar=reg_covar, mean_loglik=mlls)
                for cur in mlls[:c].mean(dim=1).tolist():  # the LL entering each iteration
                    it += 1
                    hist.append(cur)
                    if prev is not None and abs(cur - prev) < tol:
                        converged = True
                        break
                    prev = cur
                done += c
        else:
            mll = torch.zeros(B, dtype=torch.float64, device=X.device)
            for it in range(1, n_iter + 1):
                if topk is None:
                    gmm_fit_step(X, w, mu, cv, cov, reg_covar=reg_covar, mean_loglik=mll)
                else:
                    gmm_topk_fit_step(X, w, mu, cv, cov, int(topk), reg_covar=reg_covar, mean_loglik=mll, ws=tws)
                cur = float(mll.mean().item())  # the LL of the parameters that entered this step
                hist.append(cur)
                if prev is not None and abs(cur - prev) < tol:
                    converged = True
                    break
                prev = cur
        history.append(hist)
        final = score(X, w, mu, cv, cov)
        if best is None or final.mean() > best.mean_ll.mean():
            best = FitResult(w, mu, cv, final, it, converged, r, history)
    best.history = history
    return best


class GaussianMixture:
    """The estimator in the scikit-learn style of the GMMXX README (its Python
    usage example): fit / predict / predict_proba_topm / score_samples /
    score / aic / bic, with the fitted state in means_, weights_,
    covariances_ (spherical (K,) variances, diag (K, D), tied (D, D), full
    (K, D, D)), lower_bound_ (the last E-step's mean log-likelihood),
    lower_bound_history_ (per iteration, kept restart), n_iter_ and
    converged_.  X is one problem, (N, D), on the GPU; the state stays on
    the GPU as float32 tensors.  Every computation runs in the HIP library."""

    def __init__(self, n_components, covariance_type="full", max_iter=100, tol=1e-3, reg_covar=1e-6, n_init=1,
                 random_state=0, weights_init=None, means_init=None, covariances_init=None, init_params="random",
                 topk=None, check_every=1):
        if covariance_type not in ("spherical", "diag", "tied", "full"):
            raise ValueError(f"unknown covariance_type {covariance_type!r}")
        if init_params not in ("random", "kmeans"):
            raise ValueError(f"unknown init_params {init_params!r}")
        self.init_params = init_params
        self.topk = None if topk is None else int(topk)
        self.check_every = max(1, int(check_every))  # iterations per host read of the log-likelihood
        self.n_components = int(n_components)
        self.covariance_type = covariance_type
        self.max_iter = int(max_iter)
        self.tol = float(tol)
        self.reg_covar = float(reg_covar)
        self.n_init = int(n_init)
        self.random_state = random_state
        self.weights_init, self.means_init, self.covariances_init = weights_init, means_init, covariances_init

    def _init(self, X):
        given = (self.weights_init, self.means_init, self.covariances_init)
        if all(t is None for t in given):
            return self._kmeans_init(X) if self.init_params == "kmeans" else None
        if any(t is None for t in given):
            raise ValueError("weights_init, means_init and covariances_init are given together")
        torch = _torch()
        return tuple(torch.as_tensor(t, dtype=torch.float32, device=X.device).contiguous() for t in given)

    def _kmeans_init(self, X):
        """Means from Lloyd iterations (KMeans with this seed), weights from the
        cluster sizes (at least one row each), and the covariance of
        random_init (the data's variance) for every component."""
        torch = _torch()
        km = KMeans(self.n_components, max_iter=20, random_state=self.random_state).fit(X)
        gen = torch.Generator(device="cpu").manual_seed(int(self.random_state or 0))
        _, _, cv = random_init(X, self.n_components, self.covariance_type, gen)
        cnt = km.counts_.to(torch.float64).clamp_min(1.0)
        w = (cnt / cnt.sum()).to(torch.float32).contiguous()
        return w, km.cluster_centers_.clone().contiguous(), cv

    def fit(self, X):
        if X.dim() != 2:
            raise ValueError("X is (N, D)")
        res = fit(X, self.n_components, self.covariance_type, n_iter=self.max_iter, tol=self.tol,
                  n_init=self.n_init, reg_covar=self.reg_covar, seed=self.random_state or 0, init=self._init(X),
                  topk=self.topk, check_every=self.check_every)
        self.weights_, self.means_, self.covariances_ = res.weights, res.means, res.covars
        self.lower_bound_ = float(res.mean_ll[0])
        self.lower_bound_history_ = list(res.history[res.restart])
        self.n_iter_, self.converged_ = res.n_iter, res.converged
        self.n_features_in_ = int(X.shape[1])
        return self

    def _theta(self):
        if not hasattr(self, "means_"):
            raise RuntimeError("call fit first")
        return self.weights_, self.means_, self.covariances_, self.covariance_type

    def fit_predict(self, X):
        return self.fit(X).predict(X)

    def predict(self, X):
        return predict(X, *self._theta())[0]

    def score_samples(self, X):
        return score_samples(X, *self._theta())[0]

    def score(self, X):
        return float(score(X, *self._theta())[0])

    def aic(self, X):
        return float(aic(X, *self._theta())[0])

    def bic(self, X):
        return float(bic(X, *self._theta())[0])

    def predict_proba_topm(self, X, m=4, threshold=0.1):
        """Soft multi-assignment: per row the components of the m largest
        responsibilities that reach threshold (the largest always kept),
        in descending order with ties to the lower index.  Returns idx (N, m)
        int32 (-1 past count), resp (N, m) float32, count (N,) int32."""
        torch = _torch()
        N = X.shape[0]
        idx = torch.empty(N, m, dtype=torch.int32, device=X.device)
        resp = torch.empty(N, m, dtype=torch.float32, device=X.device)
        count = torch.empty(N, dtype=torch.int32, device=X.device)
        gmm_predict_proba_topm(X, *self._theta(), m, threshold, idx, resp, count=count)
        return idx, resp, count

    def reconstruct(self, X, m=4, threshold=0.1):
        """The rows rebuilt from their soft multi-assignment: sum_j r_ij
        mu_{idx_ij} over the components that predict_proba_topm keeps, (N, D)
        float32 (with every component kept, the posterior mean of the row's
        component mean)."""
        idx, resp, _ = self.predict_proba_topm(X, m, threshold)
        return gmm_codebook_lookup(self.means_, idx, weights=resp)


class KMeans:
    """k-means by Lloyd iterations, each one gmm_kmeans_step (nearest
    centroid on float64 distances, cluster means summed in float64): the
    hard-assignment, shared-variance-to-zero limit of the GMM, and the usual
    IVF coarse quantizer the GMM replaces.  X is one problem, (N, D) float32
    or bfloat16, on the GPU.  Starts from K distinct rows drawn with the seed
    (or init, (K, D)); stops when the inertia falls by less than tol of
    itself, or after max_iter steps.  Fitted state (scikit-learn names):
    cluster_centers_ (K, D) float32, labels_ (N,) int32 and inertia_ under
    the final centres, counts_ (K,) int64, n_iter_, inertia_history_ (the
    inertia under the centres entering each step)."""

    def __init__(self, n_clusters, max_iter=100, tol=1e-4, random_state=0, init=None):
        self.n_clusters = int(n_clusters)
        self.max_iter = int(max_iter)
        self.tol = float(tol)
        self.random_state = random_state
        self.init = init

    def _start(self, X):
        torch = _torch()
        N, K = X.shape[0], self.n_clusters
        if self.init is not None:
            return torch.as_tensor(self.init, dtype=torch.float32, device=X.device).clone().contiguous()
        if K > N:
            raise ValueError("n_clusters exceeds the number of rows")
        gen = torch.Generator(device="cpu").manual_seed(int(self.random_state or 0))
        sel = torch.randperm(N, generator=gen)[:K].to(X.device)
        return X.index_select(0, sel).float().contiguous()

    def fit(self, X):
        if X.dim() != 2:
            raise ValueError("X is (N, D)")
        C = self._start(X)
        hist, it = [], 0
        for it in range(1, self.max_iter + 1):
            _, counts, inertia = gmm_kmeans_step(X, C)
            cur = float(inertia[0].item())
            hist.append(cur)
            if len(hist) > 1 and hist[-2] - cur <= self.tol * hist[-2]:
                break
        self.cluster_centers_ = C
        self.n_iter_ = it
        self.inertia_history_ = hist
        self.labels_, self.counts_, self.inertia_ = self._assign(X)
        return self

    def _assign(self, X):
        if not hasattr(self, "cluster_centers_"):
            raise RuntimeError("call fit first")
        labels, counts, inertia = gmm_kmeans_step(X, self.cluster_centers_.clone())
        return labels[0], counts[0], float(inertia[0].item())

    def predict(self, X):
        """The nearest centre of every row (ties: lower index), (N,) int32."""
        return self._assign(X)[0]

    def fit_predict(self, X):
        return self.fit(X).labels_

    def reconstruct(self, labels):
        """The centres of labels ((N,) int32, as predict returns them), (N, D)
        float32; a label outside [0, n_clusters) gives a row of zeros."""
        if not hasattr(self, "cluster_centers_"):
            raise RuntimeError("call fit first")
        return gmm_codebook_lookup(self.cluster_centers_, labels)


class KernelDensity:
    """Gaussian kernel density estimate in the scikit-learn style
    (KernelDensity(kernel="gaussian")): fit(X) keeps the reference rows (M, D)
    float32 on the GPU; score_samples(Y) is log p(y) per query row from
    gmm_kde_score; score(Y) their sum."""

    def __init__(self, bandwidth=1.0):
        if not (float(bandwidth) > 0.0):
            raise ValueError("bandwidth must be > 0")
        self.bandwidth = float(bandwidth)

    def fit(self, X):
        torch = _torch()
        if X.dim() != 2:
            raise ValueError("X is (M, D)")
        self.reference_ = X.to(torch.float32).contiguous()
        self.n_features_in_ = int(X.shape[1])
        return self

    def score_samples(self, Y):
        if not hasattr(self, "reference_"):
            raise RuntimeError("call fit first")
        return gmm_kde_score(Y.contiguous(), self.reference_, self.bandwidth)

    def score(self, Y):
        return float(self.score_samples(Y).double().sum().item())


class SoftmaxHead:
    """A linear softmax classifier over n_classes, p(k | x) = softmax(W x + b)_k:
    the posterior of a mixture with one shared spherical variance
    (W_k = mu_k / s^2, b_k = log pi_k - |mu_k|^2 / (2 s^2)), trained on labels
    instead of on the rows' density -- a router over the lists of a coarse
    quantizer (route: at most 1024 of them), for example, from the labels of KMeans
    or GaussianMixture.

    fit(X, y) runs full-batch gradient descent on the mean cross entropy of the
    labelled rows (y (N,) int32; a negative label leaves a row out), each step one
    gmm_softmax_xent, one gmm_softmax_xent_grad and, with max_grad_norm, one
    gmm_clip_grad_norm over the gradients, until the loss changes by less than tol.
    optimizer "momentum", or "adamw": gmm_adamw_step with weight_decay on coef_
    alone and its states in state_bits (32 or 8).  layer_norm=True normalises the
    rows first (gmm_layer_norm, with a scale and a shift that are trained too).  X is
    (N, D) float32, bfloat16 or float16 on the GPU; float16 rows are taken as
    float32 (a copy of them), because a head and its gradients leave half's range:
    coefficients past 65504, mean gradients over many classes or confident rows
    below 6e-8.  Fitted state: coef_ (K, D) and intercept_ (K,) float32, with
    layer_norm norm_weight_ and norm_bias_ (D,) float32, loss_ (the mean loss
    entering the last step), loss_history_, grad_norm_ (the last step's norm before
    clipping, None without it), n_iter_."""

    def __init__(self, n_classes, learning_rate=1.0, momentum=0.9, max_iter=100, tol=1e-6, max_grad_norm=None,
                 optimizer="momentum", betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, state_bits=32, layer_norm=False,
                 random_state=0):
        if int(n_classes) < 1:
            raise ValueError("n_classes must be >= 1")
        if int(max_iter) < 1:
            raise ValueError("max_iter must be >= 1")
        if max_grad_norm is not None and not float(max_grad_norm) > 0.0:
            raise ValueError("max_grad_norm must be > 0")
        if optimizer not in ("momentum", "adamw"):
            raise ValueError("optimizer must be 'momentum' or 'adamw'")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        if float(weight_decay) != 0.0 and optimizer != "adamw":
            raise ValueError("weight_decay goes with optimizer='adamw'")
        self.n_classes = int(n_classes)
        self.learning_rate, self.momentum = float(learning_rate), float(momentum)
        self.max_iter, self.tol = int(max_iter), float(tol)
        self.max_grad_norm = None if max_grad_norm is None else float(max_grad_norm)
        self.optimizer, self.betas, self.eps = optimizer, tuple(map(float, betas)), float(eps)
        self.weight_decay, self.state_bits, self.layer_norm = float(weight_decay), state_bits, bool(layer_norm)
        self.random_state = random_state

    @classmethod
    def from_mixture(cls, mixture, variance=None, **kwargs):
        """The head that is the posterior of a fitted spherical GaussianMixture
        with its variances replaced by one (None: their mean under the
        weights)."""
        if mixture.covariance_type != "spherical":
            raise ValueError("the mixture must be spherical")
        w, mu, cv, _ = mixture._theta()
        head = cls(mixture.n_components, **kwargs)
        s2 = (w * cv).sum() / w.sum() if variance is None else float(variance)
        return head._set(mu / s2, w.log() - (mu * mu).sum(1) / (2 * s2))

    def _set(self, coef, intercept):
        self.coef_, self.intercept_ = coef.float().contiguous(), intercept.float().contiguous()
        return self

    def _check(self, X, y):
        torch = _torch()
        if X.dim() != 2:
            raise ValueError("X is (N, D)")
        if y.dtype != torch.int32 or y.shape != X.shape[:1]:
            raise ValueError("y is (N,) int32")
        return X.float() if X.dtype == torch.float16 else X

    def _ready(self):
        if not hasattr(self, "coef_"):
            raise RuntimeError("call fit first")
        if self.layer_norm and not hasattr(self, "norm_weight_"):
            self._set_norm(self.coef_.shape[1], self.coef_.device)

    def _set_norm(self, D, device):
        torch = _torch()
        self.norm_weight_, self.norm_bias_ = torch.ones(D, device=device), torch.zeros(D, device=device)

    def _parameters(self):
        return [self.coef_, self.intercept_] + ([self.norm_weight_, self.norm_bias_] if self.layer_norm else [])

    def loss_and_gradients(self, X, y):
        """(mean loss, its gradients for coef_ and intercept_, with layer_norm for
        norm_weight_ and norm_bias_ too): a 0-dimensional and float32 tensors on the
        GPU."""
        X = self._check(X, y)
        self._ready()
        y = y.contiguous()
        rows = X
        if self.layer_norm:
            rows, mean, rstd = gmm_layer_norm(X, self.norm_weight_, self.norm_bias_)
        W = self.coef_.to(X.dtype)
        loss, lse = gmm_softmax_xent(rows, W, y, bias=self.intercept_)
        n = (y >= 0).sum().clamp_min(1).float()
        gloss = (1.0 / n).expand(y.shape).contiguous()
        dX, dW, db = gmm_softmax_xent_grad(rows, W, y, lse, gloss=gloss, bias=self.intercept_,
                                           dX=None if self.layer_norm else False)
        if not self.layer_norm:
            return loss.sum() / n, dW.float(), db
        _, dg, ds = gmm_layer_norm_grad(dX, X, mean, rstd, gamma=self.norm_weight_, dX=False)
        return loss.sum() / n, dW.float(), db, dg, ds

    def fit(self, X, y):
        torch = _torch()
        X = self._check(X, y)
        if not hasattr(self, "coef_"):
            self._set(torch.zeros(self.n_classes, X.shape[1], device=X.device),
                      torch.zeros(self.n_classes, device=X.device))
        self._ready()
        params = self._parameters()
        adamw = self.optimizer == "adamw"
        if adamw:
            state = new_adamw_state(params, self.state_bits)
            decay = [self.weight_decay] + [0.0] * (len(params) - 1)
        else:
            step = [torch.zeros_like(p) for p in params]
        self.loss_history_, self.grad_norm_ = [], None
        for self.n_iter_ in range(1, self.max_iter + 1):
            loss, *grads = self.loss_and_gradients(X, y)
            if self.max_grad_norm is not None:
                # AdamW scales the gradients on its way: the norm alone
                self.grad_norm_ = gmm_clip_grad_norm(grads, float("inf") if adamw else self.max_grad_norm)
            if adamw:
                gmm_adamw_step(params, grads, step=self.n_iter_, lr=self.learning_rate, betas=self.betas, eps=self.eps,
                               weight_decay=decay, norm=self.grad_norm_, max_norm=self.max_grad_norm,
                               seed=int(self.random_state or 0), **state)
            else:
                for p, v, g in zip(params, step, grads):
                    v.mul_(self.momentum).add_(g)
                    p.sub_(v, alpha=self.learning_rate)
            self.loss_history_.append(float(loss))
            if len(self.loss_history_) > 1 and abs(self.loss_history_[-2] - self.loss_history_[-1]) < self.tol:
                break
        self.loss_ = self.loss_history_[-1]
        return self

    def _rows(self, X):
        return gmm_layer_norm(X, self.norm_weight_, self.norm_bias_)[0] if self.layer_norm else X

    def logits(self, X):
        """W x + b of every row (normalised first with layer_norm), (N, n_classes)
        float32, W rounded to the rows' type as fit and log_proba have it: a library
        product in float32, for the calls that choose among classes."""
        torch = _torch()
        if X.dim() != 2:
            raise ValueError("X is (N, D)")
        self._ready()
        X = X.float() if X.dtype == torch.float16 else X
        return torch.addmm(self.intercept_, self._rows(X).float(), self.coef_.to(X.dtype).float().t())

    def route(self, X, m=4, **how):
        """The m best classes of every row and their weights, as an assignment that
        gmm_codebook_lookup and gmm_ivf_lists read: (idx (N, m) int32, weights (N, m)
        float32).  At most 1024 classes.  Keyword arguments are gmm_route_topm's (bias,
        score, groups, keep_groups, group_top, renormalize, scale)."""
        return gmm_route_topm(self.logits(X), m, **how)

    def sample(self, X, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, u=None):
        """A class drawn for every row from its posterior, cut by top_k, top_p and
        min_p (gmm_sample): (classes (N,) int32, log of their share (N,) float32).  u:
        uniform numbers (N,) float32 in [0, 1); None: drawn from random_state, the same
        ones at every call."""
        torch = _torch()
        logits = self.logits(X)
        if u is None:
            gen = torch.Generator(device=logits.device).manual_seed(int(self.random_state or 0))
            u = torch.rand(logits.shape[0], generator=gen, device=logits.device)
        return gmm_sample(logits, u, temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)

    def log_proba(self, X, y):
        """log p(y_i | x_i) of every row (0 where the label is negative), (N,) float32."""
        X = self._check(X, y)
        self._ready()
        return -gmm_softmax_xent(self._rows(X), self.coef_.to(X.dtype), y.contiguous(), bias=self.intercept_)[0]

    def score(self, X, y):
        """The mean log p(y_i | x_i) of the labelled rows, on the host."""
        lp = self.log_proba(X, y)
        return float(lp.double().sum() / (y >= 0).sum().clamp_min(1))
