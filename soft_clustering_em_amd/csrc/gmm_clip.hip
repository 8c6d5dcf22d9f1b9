// gmm_clip.hip -- the 2-norm over all elements of many gradients, and the
// gradients scaled so that it is at most max_norm.
//   n = sqrt(sum_t sum_i g_ti^2),  c = min(1, max_norm / (n + 1e-6)),  out = c g
// Squares and sums are float64 (a float32 gradient of 1e20 does not overflow
// its square), in a fixed order: per workgroup over its pieces, then over the
// workgroups.  A piece is 2^15 bytes or less of one tensor; the tensors'
// descriptions travel in the kernel arguments, kClipTensors a launch, so the
// calls can be captured into a graph.  Bound by memory: the gradients are
// read twice and written once (in place with c = 1: nothing is written).
// 340M elements, 0.85 GB: norm 137 us (6.2 TB/s, part of it from the caches),
// scale 267 (6.4 TB/s read and written).
#include "gmm_internal.h"

#include <hip/hip_runtime.h>

#include <algorithm>

namespace gmm {

namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
__device__ inline double squares(const T* p, int64_t n) {
  constexpr int E = 16 / (int)sizeof(T);
  double s = 0.0;
  const int64_t nv = n / E;
  for (int64_t t = threadIdx.x; t < nv; t += 256) {
    T v[E];
    __builtin_memcpy(v, p + t * E, 16);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const double x = (double)(float)v[e];
      s += x * x;
    }
  }
  if ((int)threadIdx.x < n - nv * E) {
    const double x = (double)(float)p[nv * E + threadIdx.x];
    s += x * x;
  }
  return s;
}

template <typename T, typename C>
__device__ inline void scaled(const T* p, T* q, int64_t n, C c) {
  constexpr int E = 16 / (int)sizeof(T);
  const int64_t nv = n / E;
  const bool aligned = (uintptr_t)q % 16 == 0;  // stored past the caches: nobody reads it back soon
#pragma unroll 4
  for (int64_t t = threadIdx.x; t < nv; t += 256) {
    T v[E];
    __builtin_memcpy(v, p + t * E, 16);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = (T)(float)(c * (C)(float)v[e]);
    if (aligned) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(q + t * E));
    else __builtin_memcpy(q + t * E, v, 16);
  }
  if ((int)threadIdx.x < n - nv * E) {
    const int64_t i = nv * E + threadIdx.x;
    q[i] = (T)(float)(c * (C)(float)p[i]);
  }
}

__device__ inline int tensor_of(const ClipArgs& A, int64_t piece) {
  int lo = 0, hi = A.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (A.t[mid].piece0 <= piece) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(256) norm_kernel(ClipArgs A) {
  __shared__ double red[4];
  double s = 0.0;
  for (int64_t p = blockIdx.x; p < A.pieces; p += gridDim.x) {
    const ClipTensor& t = A.t[tensor_of(A, p)];
    const int64_t i0 = (p - t.piece0) * kClipPiece, n = min(kClipPiece, t.n - i0);
    if (t.dtype == 0) s += squares(static_cast<const float*>(t.src) + i0, n);
    else if (t.dtype == 1) s += squares(static_cast<const __bf16*>(t.src) + i0, n);
    else s += squares(static_cast<const _Float16*>(t.src) + i0, n);
  }
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) A.part[blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

__global__ void __launch_bounds__(256) coefficient_kernel(const double* part, int n, double max_norm, float* norm,
                                                          double* coef) {
  __shared__ double red[4];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) s += part[i];
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  const double v = sqrt((red[0] + red[1]) + (red[2] + red[3]));
  const double c = max_norm == INFINITY ? 1.0 : max_norm / (v + 1e-6);  // no limit: a copy, also under an infinite norm
  if (norm) *norm = (float)v;
  *coef = c < 1.0 || c != c ? c : 1.0;  // a NaN norm gives NaN gradients
}

template <typename C>
__device__ inline void scale_pieces(const ClipArgs& A, C c) {
  // from the last piece to the first: the norm's pass left the last ones in the caches
  for (int64_t p = A.pieces - 1 - blockIdx.x; p >= 0; p -= gridDim.x) {
    const ClipTensor& t = A.t[tensor_of(A, p)];
    if (c == C(1) && t.src == t.dst) continue;
    const int64_t i0 = (p - t.piece0) * kClipPiece, n = min(kClipPiece, t.n - i0);
    if (t.dtype == 0) scaled(static_cast<const float*>(t.src) + i0, static_cast<float*>(t.dst) + i0, n, c);
    else if (t.dtype == 1) scaled(static_cast<const __bf16*>(t.src) + i0, static_cast<__bf16*>(t.dst) + i0, n, c);
    else scaled(static_cast<const _Float16*>(t.src) + i0, static_cast<_Float16*>(t.dst) + i0, n, c);
  }
}

// The products are float32, float64 where the coefficient has fewer bits in
// float32 than its 24 (gradients of 1e25 and more under a small limit).
__global__ void __launch_bounds__(256) scale_kernel(ClipArgs A, const double* coef) {
  const double c = *coef;
  if (c > 0.0 && c < 0x1p-100) scale_pieces(A, c);
  else scale_pieces(A, (float)c);
}

}  // namespace

hipError_t launch_clip(const ClipTensor* t, int count, double max_norm, float* norm, double* part, double* coef,
                       hipStream_t s) {
  int nparts = 0;
  for (int phase = 0; phase < 2; ++phase) {
    for (int i0 = 0; i0 < count; i0 += kClipTensors) {
      ClipArgs A{};
      A.count = std::min(kClipTensors, count - i0);
      for (int i = 0; i < A.count; ++i) {
        A.t[i] = t[i0 + i];
        A.t[i].piece0 = A.pieces;
        A.pieces += (A.t[i].n + kClipPiece - 1) / kClipPiece;
      }
      if (A.pieces == 0) continue;
      if (phase == 0) {
        const unsigned grid = (unsigned)std::min<int64_t>(A.pieces, kClipParts);
        A.part = part + nparts;
        hipLaunchKernelGGL(norm_kernel, dim3(grid), dim3(256), 0, s, A);
        nparts += (int)grid;
      } else {
        hipLaunchKernelGGL(scale_kernel, dim3((unsigned)std::min<int64_t>(A.pieces, 1 << 16)), dim3(256), 0, s, A, coef);
      }
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (phase == 0) {
      hipLaunchKernelGGL(coefficient_kernel, dim3(1), dim3(256), 0, s, part, nparts, max_norm, norm, coef);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

}  // namespace gmm
