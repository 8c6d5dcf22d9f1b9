// gmm_adamw.hip -- one AdamW step over many tensors.
//   g' = c g,  m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2
//   p' = p (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
// with c the clipping coefficient of a given norm.  Every operation is float32,
// rounded by itself (no contraction), so that the states do not depend on how
// the compiler pairs them; the factors that all elements share are formed in
// float64.  8-bit states: e4m3 values under one float32 scale for 256 elements,
// the second moment as its root (whose ratio of largest to smallest is half as
// wide in bits).  They are rounded up with the probability of their remainder,
// from a hash of (seed, step, tensor, element): a state that moves by less than
// half a step of its 3 bits a call, as the second moment under b2 = 0.999 does,
// would never move under rounding to nearest.  A root that is not zero is not
// rounded to zero: m' over the next root would be too large a step.
// Bound by memory: every tensor read once and written once.  110M float32 values,
// bf16 gradients: with float32 states and bf16 copies 615 us (28 bytes a value, 5.0
// TB/s), with 8-bit states 321 us (14 bytes, 4.8 TB/s, beside 101 instructions a
// value, which fill the vector units' issue).
#include "gmm_device.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

namespace gmm {

namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
constexpr int kEach = 8;  // elements a thread: a state block of 256 is half a wave

__device__ inline uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x9E3779B1u;
  x = (x ^ (x >> 15)) * 0x6A09E667u;
  return x ^ (x >> 16);
}

template <typename T>
__device__ inline void load_each(float (&f)[kEach], const T* p, int n) {
  T v[kEach];
  if (n >= kEach) {
    __builtin_memcpy(v, p, sizeof(v));
  } else {
#pragma unroll
    for (int e = 0; e < kEach; ++e) v[e] = e < n ? p[e] : (T)0.f;
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) f[e] = (float)v[e];
}

template <typename T>
__device__ inline void store_each(T* p, const float (&f)[kEach], int n) {
  T v[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) v[e] = (T)f[e];
  if (n >= kEach) {
    constexpr int Q = (int)sizeof(v) / 16;
    u32x4 q[Q];
    __builtin_memcpy(q, v, sizeof(v));
    if ((uintptr_t)p % 16 == 0) {
#pragma unroll
      for (int k = 0; k < Q; ++k) __builtin_nontemporal_store(q[k], reinterpret_cast<u32x4*>(p) + k);
    } else {
      __builtin_memcpy(p, v, sizeof(v));
    }
  } else {
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (e < n) p[e] = v[e];
  }
}

__device__ inline void load_codes(float (&f)[kEach], const uint8_t* p, int n, float scale) {
#pragma clang fp contract(off)
  uint32_t w[2] = {0, 0};
  if (n >= kEach) {
    __builtin_memcpy(w, p, 8);
  } else {
    uint8_t b[8];
#pragma unroll
    for (int e = 0; e < kEach; ++e) b[e] = e < n ? p[e] : 0;
    __builtin_memcpy(w, b, 8);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f[4 * h] = __builtin_amdgcn_cvt_f32_fp8(w[h], 0) * scale;
    f[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8(w[h], 1) * scale;
    f[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8(w[h], 2) * scale;
    f[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8(w[h], 3) * scale;
  }
}

// the largest of 32 lanes' values; NaN if a lane is `bad`
__device__ inline float half_wave_max(float v, bool bad) {
  v = row16_max(v);
  auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint64_t any = __ballot(bad);
  const uint32_t mine = (threadIdx.x & 32) ? (uint32_t)(any >> 32) : (uint32_t)any;
  return mine ? __builtin_nanf("") : v;
}

// f (8 elements a lane, 256 a half wave) as e4m3 values and their scale: the
// value below or above, by the 16 bits d of each element.
template <bool ROOT>
__device__ inline void store_codes(uint8_t* p, float* scale, const float (&f)[kEach], const uint32_t (&h)[kEach], int n) {
#pragma clang fp contract(off)
  float top = 0.f, zero = 0.f;  // elements behind the last one are 0
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    top = fmaxf(top, fabsf(f[e]));
    zero = fmaf(f[e], 0.f, zero);  // NaN from NaN and infinities
  }
  top = half_wave_max(top, zero != zero);
  const bool none = top < 0x1p-100f;  // 1 / top times 448 would leave float32
  const float s = none ? 0.f : top * (1.f / 448.f), inv = none ? 0.f : 1.f / top * 448.f;
  uint32_t c[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const float x = f[e] * inv, a = fminf(fabsf(x), 448.f);
    const uint32_t d = ROOT ? h[e] & 0xffff : h[e] >> 16;
    // from 2^-6 on 3 of the 23 mantissa bits stay; below, steps of 2^-9, which few
    // waves have any of
    c[e] = ((__float_as_uint(a) + (d << 4)) >> 20) - (120u << 3);
    if (__ballot(a < 0x1p-6f)) {
      asm volatile("");  // a branch, not work for every wave
      c[e] = a < 0x1p-6f ? (uint32_t)(a * 512.f + (float)d * 0x1p-16f) : c[e];
    }
    if (ROOT) c[e] = max(c[e], min(__float_as_uint(a), 1u));
    else c[e] |= c[e] ? __float_as_uint(x) >> 24 & 0x80 : 0;
  }
  uint8_t b[kEach];
  const bool bad = top != top;
#pragma unroll
  for (int e = 0; e < kEach; ++e) b[e] = bad ? 0x7f : (uint8_t)c[e];
  if (n >= kEach) {
    __builtin_memcpy(p, b, 8);
  } else {
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (e < n) p[e] = b[e];
  }
  if ((threadIdx.x & 31) == 0 && n > 0) *scale = s;
}

struct Factors {
  float c, decay, alpha, root, b1, c1, b2, c2, eps;
  int c_exp;  // the clipping coefficient is c 2^c_exp, c below 1 where c_exp is not 0
  uint32_t key;
};

template <typename P, typename G, bool BITS8>
__device__ inline void adam_piece(const AdamTensor& t, int64_t i0, int64_t n, const Factors& F) {
#pragma clang fp contract(off)
  // every lane of a wave takes part in the blocks' maxima
  static_assert(kAdamRound == 256 * kEach, "a round of the workgroup");
  for (int64_t k = 0; k < n; k += kAdamRound) {
    const int64_t at = k + (int64_t)threadIdx.x * kEach, i = i0 + at;
    const int have = n - at >= kEach ? kEach : n - at > 0 ? (int)(n - at) : 0;
    if (!BITS8 && have == 0) return;
    float p[kEach], g[kEach], m[kEach], v[kEach];
    load_each<P>(p, static_cast<const P*>(t.p) + i, have);
    load_each<G>(g, static_cast<const G*>(t.g) + i, have);
    const int64_t block = i / kAdamBlock;
    if constexpr (BITS8) {
      load_codes(m, static_cast<const uint8_t*>(t.m) + i, have, have ? t.ms[block] : 0.f);
      load_codes(v, static_cast<const uint8_t*>(t.v) + i, have, have ? t.vs[block] : 0.f);
    } else {
      load_each<float>(m, static_cast<const float*>(t.m) + i, have);
      load_each<float>(v, static_cast<const float*>(t.v) + i, have);
    }
    float before[kEach], r[kEach], most = 0.f;  // 8 bits: the roots
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const float d = g[e] = ldexpf(F.c * g[e], F.c_exp);
      before[e] = v[e];
      if constexpr (BITS8) v[e] = v[e] * v[e];
      m[e] = F.b1 * m[e] + F.c1 * d;
      v[e] = F.b2 * v[e] + F.c2 * (d * d);
      r[e] = sqrtf(v[e]);
      most = fmaxf(most, v[e]);
    }
    if constexpr (BITS8) {
      // squares past 1.8e19 leave float32, their root does not; a NaN would take the
      // whole block with it
      if (__ballot(most == INFINITY)) {
        asm volatile("");  // a branch, not work for every wave
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const float x = before[e] * 0x1p-64f, y = g[e] * 0x1p-64f;
          r[e] = r[e] == INFINITY ? sqrtf(F.b2 * (x * x) + F.c2 * (y * y)) * 0x1p64f : r[e];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      p[e] = p[e] * F.decay - F.alpha * (m[e] / (r[e] * F.root + F.eps));
      if constexpr (BITS8) v[e] = r[e];
    }
    store_each<P>(static_cast<P*>(t.p) + i, p, have);
    if (t.copy && have) {
      if (t.copy_dtype == 1) store_each<__bf16>(static_cast<__bf16*>(t.copy) + i, p, have);
      else if (t.copy_dtype == 2) store_each<_Float16>(static_cast<_Float16*>(t.copy) + i, p, have);
      else store_each<float>(static_cast<float*>(t.copy) + i, p, have);
    }
    if constexpr (BITS8) {
      const uint32_t kb = mix32(F.key + (uint32_t)block) + (uint32_t)(i % kAdamBlock) * 0x9E3779B1u;
      uint32_t h[kEach];
#pragma unroll
      for (int e = 0; e < kEach; ++e) h[e] = mix32(kb + (uint32_t)e * 0x9E3779B1u);
      store_codes<false>(static_cast<uint8_t*>(t.m) + i, t.ms + block, m, h, have);
      store_codes<true>(static_cast<uint8_t*>(t.v) + i, t.vs + block, v, h, have);
    } else {
      store_each<float>(static_cast<float*>(t.m) + i, m, have);
      store_each<float>(static_cast<float*>(t.v) + i, v, have);
    }
  }
}

template <typename P, typename G>
__device__ inline void adam_bits(const AdamTensor& t, int64_t i0, int64_t n, const Factors& F) {
  if (t.ms) adam_piece<P, G, true>(t, i0, n, F);
  else adam_piece<P, G, false>(t, i0, n, F);
}

template <typename P>
__device__ inline void adam_grad(const AdamTensor& t, int64_t i0, int64_t n, const Factors& F) {
  if (t.grad_dtype == 0) adam_bits<P, float>(t, i0, n, F);
  else if (t.grad_dtype == 1) adam_bits<P, __bf16>(t, i0, n, F);
  else adam_bits<P, _Float16>(t, i0, n, F);
}

__global__ void __launch_bounds__(256) adamw_kernel(AdamArgs A) {
  __shared__ Factors shared;
  __shared__ double lr;
  if (threadIdx.x == 0) {
    const int64_t step = A.step_dev ? (*A.step_dev > 1 ? *A.step_dev : 1) : A.step;
    lr = A.lr_dev ? (double)*A.lr_dev : A.lr;
    double c = 1.0;
    if (A.norm && A.max_norm != INFINITY) {
      const double q = A.max_norm / ((double)*A.norm + 1e-6);
      c = q < 1.0 || q != q ? q : 1.0;
    }
    Factors f;
    // float32 holds few bits, or none, of a coefficient below 2^-126 (gradients of 1e25
    // and more under a small limit): its power of two goes on the product then
    f.c_exp = c > 0.0 && c < 0x1p-100 ? ilogb(c) + 1 : 0;
    f.c = (float)ldexp(c, -f.c_exp);
    f.alpha = (float)(lr / -expm1((double)step * A.log_b1));
    f.root = (float)(1.0 / sqrt(-expm1((double)step * A.log_b2)));
    f.b1 = (float)A.b1;
    f.c1 = (float)(1.0 - A.b1);
    f.b2 = (float)A.b2;
    f.c2 = (float)(1.0 - A.b2);
    f.eps = (float)A.eps;
    f.decay = 0.f;
    f.key = mix32(A.seed + 0x9E3779B1u * (uint32_t)step);
    shared = f;
  }
  __syncthreads();
  for (int64_t q = blockIdx.x; q < A.pieces; q += gridDim.x) {
    int lo = 0, hi = A.count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (A.t[mid].piece0 <= q) lo = mid;
      else hi = mid - 1;
    }
    const AdamTensor& t = A.t[lo];
    const int64_t i0 = (q - t.piece0) * A.piece, n = min(A.piece, t.n - i0);
    Factors F = shared;
    F.decay = (float)(1.0 - lr * t.weight_decay);
    F.key = mix32(F.key ^ (uint32_t)(A.first + lo));
    if (t.dtype == 0) adam_grad<float>(t, i0, n, F);
    else if (t.dtype == 1) adam_grad<__bf16>(t, i0, n, F);
    else adam_grad<_Float16>(t, i0, n, F);
  }
}

}  // namespace

hipError_t launch_adamw(const AdamTensor* t, int count, AdamArgs A, hipStream_t s) {
  for (int i0 = 0; i0 < count; i0 += kAdamTensors) {
    A.first = i0;
    A.count = std::min(kAdamTensors, count - i0);
    A.pieces = 0;
    // a workgroup's round is 2048 elements: one a piece as long as that fills the
    // card, then four, with a quarter of the look-ups (float32 states, 40000 values 4.9
    // us with one and 7.4 with four, 2M 11.7 and 13.5, 4M 21.7 and 22.5; 8-bit states,
    // 4M 20.4 and 22.1, 8M 35.9 and 33.3, 110M 376 and 362)
    int64_t total = 0;
    for (int i = 0; i < A.count; ++i) total += t[i0 + i].n;
    A.piece = total <= 2048 * kAdamRound ? kAdamRound : 4 * kAdamRound;
    for (int i = 0; i < A.count; ++i) {
      A.t[i] = t[i0 + i];
      A.t[i].piece0 = A.pieces;
      A.pieces += (A.t[i].n + A.piece - 1) / A.piece;
    }
    if (A.pieces == 0) continue;
    hipLaunchKernelGGL(adamw_kernel, dim3((unsigned)std::min<int64_t>(A.pieces, 1 << 13)), dim3(256), 0, s, A);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gmm
