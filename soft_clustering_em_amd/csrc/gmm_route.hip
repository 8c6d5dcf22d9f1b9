// gmm_route.hip -- scores of E experts turned into the m best codes of a row
// and their weights, and the gradient of the scores.
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),  t_e = s_e + bias_e
//   groups of E / groups experts: the keep_groups with the largest sum of their
//   group_top best t;  the m largest t in them, ties to the lower index
//   w_j = scale s_j / sum_selected s
// Orders are decided in float64; without a bias the order of the scores is that
// of the logits, which are exact.
#include "gmm_device.h"

#include <hip/hip_runtime.h>

#include <float.h>

namespace gmm {

namespace {

// LDS written by some lanes of a wave, read by others of the same wave
__device__ inline void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// s_e of the code `e` that this lane holds (e < 0: none), over the sum of the
// row's codes (renorm), or over `total`: the largest logit among the codes
// stands for the row's, so that their sum cannot vanish.
__device__ inline double selected(const RouteArgs& A, int64_t base, int e, float mx, double total) {
  const float l = e >= 0 ? fminf(x_value(A.l, A.dtype, base + e), FLT_MAX) : -INFINITY;
  double q = 0.0;
  if (A.sigmoid) {
    if (e >= 0) q = 1.0 / (1.0 + exp(-(double)l));
  } else {
    const float top = A.renorm ? rows4_max(row16_max(l)) : mx;
    if (e >= 0) q = exp((double)l - (double)top);
    if (!A.renorm && e >= 0) q /= total;
  }
  if (A.renorm) {
    const double sum = wave_sum(q);
    q = sum > 0.0 ? q / sum : 0.0;
  }
  return q;
}

// One wave a row: EPL experts a lane, e = lane + 64 k.
template <int EPL>
__global__ void __launch_bounds__(256) route_kernel(RouteArgs A) {
  extern __shared__ double lds[];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t r = (int64_t)blockIdx.x * 4 + w;
  if (r >= A.R) return;
  const int64_t b = A.stride_b ? (uint32_t)r / (uint32_t)A.N : 0;
  const int64_t base = b * A.stride_b + (r - b * A.N) * A.ld;
  float l[EPL];
  double t[EPL], s[EPL];
  float mx = -INFINITY;
#pragma unroll
  for (int k = 0; k < EPL; ++k) {
    const int e = lane + 64 * k;
    l[k] = -INFINITY;
    if (e < A.E) {
      const float v = x_value(A.l, A.dtype, base + e);
      if (v > -INFINITY) l[k] = fminf(v, FLT_MAX);
    }
    mx = fmaxf(mx, l[k]);
  }
  mx = rows4_max(row16_max(mx));
  double total = 1.0;
  if (A.sigmoid) {
#pragma unroll
    for (int k = 0; k < EPL; ++k) s[k] = l[k] > -INFINITY ? 1.0 / (1.0 + exp(-(double)l[k])) : 0.0;
  } else {
    total = 0.0;
#pragma unroll
    for (int k = 0; k < EPL; ++k) {
      s[k] = l[k] > -INFINITY ? exp((double)l[k] - (double)mx) : 0.0;
      total += s[k];
    }
    total = wave_sum(total);
#pragma unroll
    for (int k = 0; k < EPL; ++k) s[k] = l[k] > -INFINITY ? s[k] / total : 0.0;
  }
  const bool by_score = A.bias != nullptr;
#pragma unroll
  for (int k = 0; k < EPL; ++k) {
    const int e = lane + 64 * k;
    t[k] = l[k] > -INFINITY ? (by_score ? s[k] + (double)A.bias[e] : (double)l[k]) : -INFINITY;
  }
  if (A.groups > 1 && A.keep < A.groups) {
    double* row = lds + (size_t)w * A.E;
    const int gs = A.E / A.groups;
#pragma unroll
    for (int k = 0; k < EPL; ++k) {
      const int e = lane + 64 * k;
      if (e < A.E) row[e] = !by_score && A.top == 2 && l[k] > -INFINITY ? s[k] : t[k];
    }
    wave_lds();
    double score = -INFINITY;
    if (lane < A.groups) {
      double best = -INFINITY, next = -INFINITY;
      for (int i = 0; i < gs; ++i) {
        const double v = row[lane * gs + i];
        if (v > best) {
          next = best;
          best = v;
        } else if (v > next) {
          next = v;
        }
      }
      score = A.top == 2 && next > -INFINITY ? best + next : best;
    }
    uint64_t kept = 0;
    for (int i = 0; i < A.keep; ++i) {
      double v = score;
      int g = lane;
      wave_best(v, g);
      kept |= (uint64_t)1 << g;
      if (lane == g) score = -INFINITY;
      if (v == -INFINITY) break;
    }
#pragma unroll
    for (int k = 0; k < EPL; ++k) {
      const int e = lane + 64 * k;
      if (e < A.E && !((kept >> (e / gs)) & 1)) t[k] = -INFINITY;
    }
  }
  int mine = -1;
  for (int j = 0; j < A.m; ++j) {
    double v = -INFINITY;
    int at = 1 << 30;
#pragma unroll
    for (int k = 0; k < EPL; ++k)
      if (t[k] > v) {
        v = t[k];
        at = lane + 64 * k;
      }
    wave_best(v, at);
    if (v == -INFINITY) break;
    if (lane == j) mine = at;
#pragma unroll
    for (int k = 0; k < EPL; ++k)
      if (at == lane + 64 * k) t[k] = -INFINITY;
  }
  const double q = selected(A, base, mine, mx, total);
  if (lane < A.m) {
    A.idx[r * A.m + lane] = mine;
    A.weights[r * A.m + lane] = (float)((double)A.scale * q);
  }
}

// One wave a row.  With u_j = scale dw_j and q_j = s_j / sum_selected s:
//   softmax: dl_e = s_e (ds_e - sum_f ds_f s_f);  sigmoid: dl_e = s_e (1 - s_e) ds_e
// where ds_e = dscores_e, and without renormalising + u_j of the code e; renormalised
// the codes' part is q_j (u_j - sum u q), times 1 - s_j for the sigmoid.
template <int EPL>
__global__ void __launch_bounds__(256) route_grad_kernel(RouteArgs A) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t r = (int64_t)blockIdx.x * 4 + w;
  if (r >= A.R) return;
  const int64_t b = A.stride_b ? (uint32_t)r / (uint32_t)A.N : 0;
  const int64_t base = b * A.stride_b + (r - b * A.N) * A.ld;
  float l[EPL], s[EPL], rest[EPL], ds[EPL], dl[EPL];
  float mx = -INFINITY;
#pragma unroll
  for (int k = 0; k < EPL; ++k) {
    const int e = lane + 64 * k;
    l[k] = -INFINITY;
    ds[k] = dl[k] = 0.f;
    if (e < A.E) {
      const float v = x_value(A.l, A.dtype, base + e);
      if (v > -INFINITY) l[k] = fminf(v, FLT_MAX);
      if (A.dscores) ds[k] = A.dscores[e];
    }
    mx = fmaxf(mx, l[k]);
  }
  mx = rows4_max(row16_max(mx));
  float total = 0.f;
#pragma unroll
  for (int k = 0; k < EPL; ++k) {
    const bool on = l[k] > -INFINITY;
    if (A.sigmoid) {
      const float z = expf(-fabsf(l[k])), hi = 1.f / (1.f + z), lo = z / (1.f + z);
      s[k] = on ? (l[k] >= 0.f ? hi : lo) : 0.f;
      rest[k] = l[k] >= 0.f ? lo : hi;
    } else {
      s[k] = on ? expf(l[k] - mx) : 0.f;
      rest[k] = 1.f;
      total += s[k];
    }
  }
  if (!A.sigmoid) {
    total = rows4_sum(row16_sum(total));
    const float inv = total > 0.f ? 1.f / total : 0.f;
#pragma unroll
    for (int k = 0; k < EPL; ++k) s[k] *= inv;
  }
  if (A.dweights) {
    int mine = lane < A.m ? A.idx[r * A.m + lane] : -1;
    // the row's leading codes in [0, E)
    const uint64_t bad = __ballot(mine < 0 || mine >= A.E);
    const int n = __builtin_ctzll(bad | ((uint64_t)1 << 63));
    if (lane >= n) mine = -1;
    float u = mine >= 0 ? A.scale * A.dweights[r * A.m + lane] : 0.f;
    if (A.renorm) {
      const float q = (float)selected(A, base, mine, mx, 1.0);
      u = q * (u - rows4_sum(row16_sum(q * u)));
    }
    for (int j = 0; j < n; ++j) {
      const int e = __shfl(mine, j);
      const float v = __shfl(u, j);
#pragma unroll
      for (int k = 0; k < EPL; ++k)
        if (e == lane + 64 * k) {
          if (A.renorm) dl[k] += v * rest[k];
          else ds[k] += v;
        }
    }
  }
  float c = 0.f;
  if (!A.sigmoid) {
#pragma unroll
    for (int k = 0; k < EPL; ++k) c += s[k] > 0.f ? ds[k] * s[k] : 0.f;
    c = rows4_sum(row16_sum(c));
  }
#pragma unroll
  for (int k = 0; k < EPL; ++k) {
    const int e = lane + 64 * k;
    if (e >= A.E) break;
    const float d = l[k] > -INFINITY ? dl[k] + s[k] * rest[k] * (ds[k] - c) : 0.f;
    const int64_t o = r * A.E + e;
    if (A.dtype == 0) static_cast<float*>(A.dlogits)[o] = d;
    else if (A.dtype == 1) static_cast<__bf16*>(A.dlogits)[o] = (__bf16)d;
    else static_cast<_Float16*>(A.dlogits)[o] = (_Float16)d;
  }
}

}  // namespace

hipError_t launch_route(const RouteArgs& A, bool grad, hipStream_t s) {
  const dim3 grid((unsigned)((A.R + 3) / 4)), block(256);
  const size_t lds = A.groups > 1 ? sizeof(double) * 4 * (size_t)A.E : 0;
  const int per = (A.E + 63) / 64;
#define GMM_ROUTE(EPL)                                                                      \
  if (per <= EPL) {                                                                         \
    if (grad) hipLaunchKernelGGL(route_grad_kernel<EPL>, grid, block, 0, s, A);             \
    else hipLaunchKernelGGL(route_kernel<EPL>, grid, block, lds, s, A);                     \
    return hipGetLastError();                                                               \
  }
  GMM_ROUTE(1)
  GMM_ROUTE(2)
  GMM_ROUTE(4)
  GMM_ROUTE(8)
  GMM_ROUTE(16)
#undef GMM_ROUTE
  return hipErrorInvalidValue;
}

}  // namespace gmm
