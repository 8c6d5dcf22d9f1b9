// gmm_xent_few.hip -- softmax cross entropy of wide float32 rows under a head
// of at most 128 classes: the two products that read the rows.
//
// With few classes the rows' bytes are everything: a product does 2 V flops for
// the 4 bytes of an element, so the rows are read where they lie, once a
// product for every 64 classes (twice above 64), and become their three bf16
// planes in registers (kPairs); copies with their planes side by side and their
// transposes, which a product over many classes repays, would be most of the
// traffic here.
//   logits  X W^T, parts of k side by side in float32 slabs
//   dW      G^T X, parts of the rows side by side in float32 slabs
// 83230 x 2800 rows, 22 classes: the logits 293 us (3.2 TB/s: rows in pieces of
// 256 bytes), dW 402 (2.3 TB/s, two waves a SIMD), loss and gradients 1.32 ms;
// through packed planes and 128 x 128 tiles 600 and 1013 us, 3.4 ms.
// 65536 x 512, 10 classes: logits 32 us (4.2 TB/s), dW 33 (4.0); 64 classes 69
// and 73 (1.9 TB/s; from 33 classes on dW's registers leave one wave a SIMD);
// 128 classes 131 and 137.
#include "gmm_internal.h"
#include "gmm_xent.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

namespace gmm {

namespace {

// 8 consecutive k of a lane -> its fragment of every plane
__device__ inline void split8(f32x4 lo, f32x4 hi, u32x4* f) {
  u32x2 a[3], b[3];
  split4(lo, a);
  split4(hi, b);
#pragma unroll
  for (int l = 0; l < 3; ++l) f[l] = u32x4{a[l][0], a[l][1], b[l][0], b[l][1]};
}

__device__ inline int64_t few_row(const FewArgs& P, int64_t r) {
  return P.flat ? (P.rows.r0 + r) * P.rows.ld : row_offset(P.rows, P.rows.r0 + r);
}

// A wave: 32 rows (two blocks of 16) against NB blocks of 16 classes, whose
// planes come from the caches; k-steps of 32 elements, U of them at a time.
template <int NB>
__global__ void __launch_bounds__(256) few_logits_kernel(FewArgs P) {
  constexpr int U = NB == 4 ? 1 : 2;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, lr = lane & 15, lq = lane >> 4;
  const int64_t m0 = ((int64_t)blockIdx.x * 4 + wv) * 32;
  const int z = blockIdx.y, D = P.rows.D, cb = blockIdx.z * 64;  // first class
  const char* x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    x[i] = P.rows.x + 4 * few_row(P, min(m0 + 16 * i + lr, P.rows.nr - 1)) + 32 * lq;  // rows past the last are not stored
  const char* w[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) w[j] = P.b + (int64_t)min(cb + 16 * j + lr, P.V - 1) * P.ldb + 16 * lq;
  f32x4 acc[2][NB];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const f32x4 (*v)[2], const u32x4 (*b)[3]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u32x4 a[3];
      split8(v[i][0], v[i][1], a);
#pragma unroll
      for (int q = 5; q >= 0; --q)  // the small products first
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mma<__bf16>(b[j][kPairs[q][1]], a[kPairs[q][0]], acc[i][j]);
    }
  };
  const int steps = (D + 31) / 32;
  const int s0 = (int)((int64_t)steps * z / P.splits), s1 = (int)((int64_t)steps * (z + 1) / P.splits);
  const int whole = min(s1, D / 32);
  // the rows of the next U steps (whole 128-byte lines side by side) are on
  // their way while U steps are multiplied; the classes' planes, in the caches,
  // are asked for first, so that waiting for them does not wait for the rows
  auto load = [&](int s, f32x4 (*v)[2][2]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i) __builtin_memcpy(v[u][i], x[i] + (int64_t)min(s + u, whole - 1) * 128, 32);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](int s, const f32x4 (*v)[2][2], f32x4 (*next)[2][2]) {
    u32x4 b[U][NB][3];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int l = 0; l < 3; ++l) b[u][j][l] = *reinterpret_cast<const u32x4*>(w[j] + l * P.pb + (int64_t)(s + u) * 64);
    __builtin_amdgcn_sched_barrier(0);
    load(s + U, next);
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(v[u], b[u]);
  };
  int s = s0;
  if (s + U <= whole) {
    f32x4 v0[U][2][2], v1[U][2][2];
    load(s, v0);
    while (true) {
      step(s, v0, v1);
      s += U;
      if (s + U > whole) break;
      step(s, v1, v0);
      s += U;
      if (s + U > whole) break;
    }
  }
  for (; s < s1; ++s) {  // steps that may end inside
    const int left = D - 32 * s - 8 * lq;  // elements from this lane's first on
    f32x4 v[2][2];
    u32x4 b[NB][3];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[i][h] = __builtin_bit_cast(f32x4, chunk_at<float>(x[i] + (int64_t)s * 128, 16 * h, 4 * left));
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int l = 0; l < 3; ++l)  // the planes' rows are whole chunks
        b[j][l] = left > 0 ? *reinterpret_cast<const u32x4*>(w[j] + l * P.pb + (int64_t)s * 64) : u32x4{0u, 0u, 0u, 0u};
    multiply(v, b);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + 16 * i + lr;
    if (m >= P.rows.nr) continue;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int n = cb + 16 * j + 4 * lq;
      if (n < P.V) *reinterpret_cast<f32x4*>(P.slab + z * P.slab_stride + m * P.lds + n) = acc[i][j];
    }
  }
}

// A wave: 64 columns (a lane 4 neighbouring ones, each of them a product of its
// own) of NB blocks of 16 classes; k-steps of 32 rows, 8 a lane, so that a
// lane's loads of a column over 8 rows are its fragment and nothing is
// transposed.  Rows with live = 0 enter as zeros.
template <int NB>
__global__ void __launch_bounds__(256) few_dw_kernel(FewArgs P) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, lr = lane & 15, lq = lane >> 4;
  const int d0 = (blockIdx.x * 4 + wv) * 64 + 4 * lr;
  if (d0 - 4 * lr >= P.rows.D) return;
  const int z = blockIdx.y, cb = blockIdx.z * 64;
  const int64_t nr = P.rows.nr;
  const char* g[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) g[j] = P.b + (int64_t)min(cb + 16 * j + lr, P.V - 1) * P.ldb + 16 * lq;
  f32x4 acc[NB][4];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[j][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t steps = (nr + 31) / 32;
  const int64_t s0 = steps * z / P.splits, s1 = steps * (z + 1) / P.splits;
  auto load = [&](int64_t s, f32x4* v, float* live, auto whole) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t r = 32 * s + 8 * lq + k, rc = min(r, nr - 1);
      const char* row = P.rows.x + 4 * few_row(P, rc);
      if (whole.value) __builtin_memcpy(&v[k], row + 4 * d0, 16);
      else v[k] = __builtin_bit_cast(f32x4, chunk_at<float>(row, 4 * d0, 4 * P.rows.D));
      const float t = P.live[rc];
      live[k] = r < nr ? t : 0.f;
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto planes_of = [&](int64_t s, u32x4 (*b)[3]) {
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int l = 0; l < 3; ++l) b[j][l] = *reinterpret_cast<const u32x4*>(g[j] + l * P.pb + s * 64);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](const f32x4* v, const float* live, const u32x4 (*b)[3]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = live[k] != 0.f ? v[k][c] : 0.f;
      u32x4 a[3];
      split8(f32x4{t[0], t[1], t[2], t[3]}, f32x4{t[4], t[5], t[6], t[7]}, a);
#pragma unroll
      for (int q = 5; q >= 0; --q)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[j][c] = mma<__bf16>(b[j][kPairs[q][1]], a[kPairs[q][0]], acc[j][c]);
    }
  };
  auto run = [&](auto whole) {  // a step's loads are on their way while the step before is multiplied
    if (s0 >= s1) return;
    f32x4 v0[8], v1[8];
    float l0[8], l1[8];
    u32x4 b[NB][3];
    load(s0, v0, l0, whole);
    int64_t s = s0;
    for (; s + 2 <= s1; s += 2) {
      planes_of(s, b);
      load(s + 1, v1, l1, whole);
      multiply(v0, l0, b);
      planes_of(s + 1, b);
      load(min(s + 2, s1 - 1), v0, l0, whole);
      multiply(v1, l1, b);
    }
    if (s < s1) {
      planes_of(s, b);
      multiply(v0, l0, b);
    }
  };
  if (d0 - 4 * lr + 64 <= P.rows.D) run(std::true_type{});
  else run(std::false_type{});
  if (d0 >= P.rows.D) return;
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = cb + 16 * j + 4 * lq + e;
      if (n >= P.V) continue;
      float* p = P.slab + z * P.slab_stride + n * P.lds + d0;  // rows of D rounded up to 4
      f32x4 t = {acc[j][0][e], acc[j][1][e], acc[j][2][e], acc[j][3][e]};
      if (P.add) t += *reinterpret_cast<const f32x4*>(p);
      *reinterpret_cast<f32x4*>(p) = t;
    }
}

}  // namespace

// parts that bring four workgroups to every compute unit, each 64 of k or longer
int xent_few_splits(int64_t workgroups, int64_t k) {
  const int64_t want = (4 * kNumCU + workgroups - 1) / workgroups;
  return (int)std::max<int64_t>(1, std::min({want, k / 64, (int64_t)256}));
}

hipError_t launch_xent_few_logits(const FewArgs& P, hipStream_t s) {
  const dim3 grid((unsigned)((P.rows.nr + 127) / 128), (unsigned)P.splits, (unsigned)((P.V + 63) / 64));
  if (P.V <= 16) hipLaunchKernelGGL(few_logits_kernel<1>, grid, dim3(256), 0, s, P);
  else if (P.V <= 32) hipLaunchKernelGGL(few_logits_kernel<2>, grid, dim3(256), 0, s, P);
  else hipLaunchKernelGGL(few_logits_kernel<4>, grid, dim3(256), 0, s, P);
  return hipGetLastError();
}

hipError_t launch_xent_few_dw(const FewArgs& P, hipStream_t s) {
  const dim3 grid((unsigned)((P.rows.D + 255) / 256), (unsigned)P.splits, (unsigned)((P.V + 63) / 64));
  if (P.V <= 16) hipLaunchKernelGGL(few_dw_kernel<1>, grid, dim3(256), 0, s, P);
  else if (P.V <= 32) hipLaunchKernelGGL(few_dw_kernel<2>, grid, dim3(256), 0, s, P);
  else hipLaunchKernelGGL(few_dw_kernel<4>, grid, dim3(256), 0, s, P);
  return hipGetLastError();
}

}  // namespace gmm
