// gmm_norm.hip -- layer norm of rows and its gradients.
//   mean = sum_d x_d / D,  r = 1 / sqrt(sum_d (x_d - mean)^2 / D + eps)
//   y_d  = (x_d - mean) r gamma_d + beta_d
//   dx_d = r (q_d - sum q / D - xh_d sum (q xh) / D),  q = dy gamma, xh = (x - mean) r
//   dgamma_d = sum_rows dy xh,  dbeta_d = sum_rows dy
// A row's values stay in registers from the one read to the one write: TPR
// threads a row, C pieces of 16 bytes a thread.  The mean is corrected by the
// mean of the differences from its first value, and the variance is that of the
// corrected differences, so rows far from zero keep their digits; the gradients
// take the mean as it was stored, rounded to float32.  Sums are
// float32: per thread, then in a fixed order over the row's threads.  The
// gradients of gamma and beta: a thread owns its columns over all the rows that
// its workgroup walks, then the workgroups' sums are added in a fixed order.
// Bound by memory: 32768 x 2048 bf16 forward 50 to 56 us (4.8 TB/s and more), gradients 98 us (4.1
// TB/s) and 7 for the join; 1M x 64 float32 102 and 162 us (5.0 and 4.7 TB/s); one
// row of 4096 3.4 us, latency.
#include "gmm_device.h"

#include <hip/hip_runtime.h>

#include <algorithm>

namespace gmm {

namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int kPer = 16 / (int)sizeof(T);  // elements of a 16-byte piece

// Element e of a piece.  Pieces stay packed in registers, 4 for 8 values of 16
// bits, and are opened where they are used.
template <typename T>
__device__ inline float element(u32x4 v, int e) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(v[e]);
  } else {
    const unsigned short h = (unsigned short)(v[e / 2] >> (16 * (e & 1)));
    return (float)__builtin_bit_cast(T, h);
  }
}
// The compiler keeps no opened copies of v beyond this point.
__device__ inline void packed(u32x4& v) { asm volatile("" : "+v"(v)); }

template <typename T>
__device__ inline u32x4 load_piece(const T* row, int64_t c0, int64_t D) {
  T v[kPer<T>];
  if (c0 + kPer<T> <= D) {
    __builtin_memcpy(v, row + c0, 16);
  } else {
#pragma unroll
    for (int e = 0; e < kPer<T>; ++e) v[e] = c0 + e < D ? row[c0 + e] : (T)0.f;
  }
  return __builtin_bit_cast(u32x4, v);
}

// v shifted down by k elements, zeros behind them
template <typename T>
__device__ inline u32x4 shifted(u32x4 v, int k) {
  uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
  const int s = k * 8 * (int)sizeof(T);  // 16 to 112
  if (s >= 64) {
    lo = hi >> (s - 64);
    hi = 0;
  } else {
    lo = lo >> s | hi << (64 - s);
    hi >>= s;
  }
  return u32x4{(unsigned)lo, (unsigned)(lo >> 32), (unsigned)hi, (unsigned)(hi >> 32)};
}

// A thread's C pieces of a row (zeros past D, and everywhere if not `live`).
// The loads come first and without a branch, so that they are in flight
// together: a piece that reaches past D is the row's last 16 bytes, shifted.
template <typename T, int TPR, int C>
__device__ inline void load_row(u32x4 (&v)[C], const T* row, int t, int64_t D, bool live) {
  constexpr int E = kPer<T>;
  if (D < E) {
#pragma unroll
    for (int j = 0; j < C; ++j) v[j] = load_piece<T>(row, ((int64_t)j * TPR + t) * E, live ? D : 0);
    return;
  }
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int64_t c0 = ((int64_t)j * TPR + t) * E;
    __builtin_memcpy(&v[j], row + (c0 + E <= D ? c0 : D - E), 16);
  }
  if (D == (int64_t)TPR * C * E && live) return;  // every piece lies in the row
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int64_t c0 = ((int64_t)j * TPR + t) * E;
    if (!live || c0 >= D) v[j] = u32x4{0, 0, 0, 0};
    else if (c0 + E > D) v[j] = shifted<T>(v[j], (int)(c0 + E - D));
  }
}

// stream: past the caches
template <typename T>
__device__ inline void store_piece(T* row, const T (&v)[kPer<T>], int64_t c0, int64_t D, bool stream) {
  if (c0 + kPer<T> <= D) {
    if (stream && (uintptr_t)(row + c0) % 16 == 0)
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4*>(row + c0));
    else __builtin_memcpy(row + c0, v, 16);
  } else {
#pragma unroll
    for (int e = 0; e < kPer<T>; ++e)
      if (c0 + e < D) row[c0 + e] = v[e];
  }
}

// E values of gamma or beta as float32 (is_t: stored in the rows' type), `none` past D or without a tensor
template <typename T>
__device__ inline void load_affine(float (&v)[kPer<T>], const void* p, bool is_t, int64_t c0, int64_t D, float none) {
  constexpr int E = kPer<T>;
  if (!p || c0 >= D) {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = none;
  } else if (is_t) {
    const u32x4 t = load_piece<T>(static_cast<const T*>(p), c0, D);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = element<T>(t, e);
  } else {
    const float* f = static_cast<const float*>(p) + c0;
    if (c0 + E <= D) {
      __builtin_memcpy(v, f, sizeof(v));
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = c0 + e < D ? f[e] : none;
    }
  }
}

// over groups of L neighbouring lanes, in every one of them
template <int L>
__device__ inline float lanes_sum(float v) {
  v += dpp_mov<0xB1>(v);
  v += dpp_mov<0x4E>(v);
  if constexpr (L >= 8) v += dpp_mov<0x141>(v);
  if constexpr (L >= 16) v += dpp_mov<0x140>(v);
  if constexpr (L == 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (L == 64) v = rows4_sum(v);
  return v;
}

// The sums of a and b over the TPR threads of a row, in every one of them.
// Rows of more than a wave meet in LDS; `red` alternates between two halves,
// so that one barrier a call is enough.
template <int TPR>
__device__ inline void row_sum2(float& a, float& b, float2 (*red)[TPR > 64 ? TPR / 64 : 1], int& turn) {
  a = lanes_sum<TPR < 64 ? TPR : 64>(a);
  b = lanes_sum<TPR < 64 ? TPR : 64>(b);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 v = red[turn][w];
      a += v.x;
      b += v.y;
    }
    turn ^= 1;
  }
}

__device__ inline int64_t row_at(int64_t r, int64_t N, int64_t ld, int64_t stride_b) {
  if (stride_b == 0) return r * ld;
  const uint32_t b = (uint32_t)r / (uint32_t)N;
  return (int64_t)b * stride_b + (r - (int64_t)b * N) * ld;
}

template <typename T, int TPR, int C>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) norm_kernel(NormArgs A) {
  constexpr int E = kPer<T>, RPB = TPR > 256 ? 1 : 256 / TPR;
  __shared__ float2 red[2][TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x % TPR;
  const int64_t r = A.r0 + (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = r < A.R;  // rows of more than a wave: the whole workgroup agrees
  if (TPR > 64 && !live) return;
  const T* x = static_cast<const T*>(A.x) + (live ? row_at(r, A.N, A.ld, A.stride_b) : 0);
  const float inv = 1.f / (float)A.D;
  u32x4 v[C];
  float s = 0.f, s1 = 0.f, s2 = 0.f, none = 0.f;
  int turn = 0;
  load_row<T, TPR, C>(v, x, t, A.D, live);
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) s += element<T>(v[j], e);
  row_sum2<TPR>(s, none, red, turn);
  const float m1 = s * inv;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    packed(v[j]);
    const int64_t c0 = ((int64_t)j * TPR + t) * E;
    if (c0 >= A.D) break;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float d = c0 + e < A.D ? element<T>(v[j], e) - m1 : 0.f;
      s1 += d;
      s2 += d * d;
    }
  }
  row_sum2<TPR>(s1, s2, red, turn);
  const float m2 = s1 * inv, mean = m1 + m2;
  const float var = fmaxf(0.f, (s2 - s1 * m2) * inv), rstd = 1.f / sqrtf(var + A.eps);
  // NaN in a row stays NaN: fmaxf would drop it
  const float rs = s2 != s2 ? s2 : rstd;
  if (!live) return;
  if (t == 0) {
    if (A.mean) A.mean[r] = mean;
    if (A.rstd) A.rstd[r] = rs;
  }
  T* out = static_cast<T*>(A.out) + r * A.D;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int64_t c0 = ((int64_t)j * TPR + t) * E;
    if (c0 >= A.D) break;
    packed(v[j]);
    float g[E], b[E];
    load_affine<T>(g, A.gamma, A.affine_t, c0, A.D, 1.f);
    load_affine<T>(b, A.beta, A.affine_t, c0, A.D, 0.f);
    T o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = (T)(((element<T>(v[j], e) - m1) - m2) * rs * g[e] + b[e]);
    store_piece<T>(out, o, c0, A.D, A.stream);
  }
}

// The gradients of rows, and (ACC) this workgroup's share of gamma's and
// beta's: sums over the rows blockIdx.x * RPB + k gridDim.x * RPB.  The next
// row's loads are under way while a row is summed, where there are registers.
template <typename T, int TPR, int C, bool ACC>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) norm_grad_kernel(NormArgs A) {
  constexpr int E = kPer<T>, RPB = TPR > 256 ? 1 : 256 / TPR, W = (TPR > 256 ? TPR : 256) / 64;
  constexpr bool AHEAD = TPR <= 256;
  __shared__ float2 red[2][TPR > 64 ? TPR / 64 : 1];
  const int t = threadIdx.x % TPR;
  const float inv = 1.f / (float)A.D;
  u32x4 g[C], nx[C], ny[C];
  float dg[ACC ? C : 1][E], db[ACC ? C : 1][E], next_mean, next_rstd;
  int turn = 0;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    // gamma in the rows' type where it is stored so; opened like them
    if (A.affine_t && A.gamma) g[j] = load_piece<T>(static_cast<const T*>(A.gamma), ((int64_t)j * TPR + t) * E, A.D);
    if constexpr (ACC) {
#pragma unroll
      for (int e = 0; e < E; ++e) dg[j][e] = db[j][e] = 0.f;
    }
  }
  const bool stored = A.affine_t && A.gamma;
  const auto gamma = [&](int j, float (&f)[E]) {
    if (stored) {
      packed(g[j]);
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = element<T>(g[j], e);
    } else {
      load_affine<T>(f, A.gamma, false, ((int64_t)j * TPR + t) * E, A.D, 1.f);
    }
  };
  const auto fetch = [&](int64_t r) {
    const bool live = r < A.R;
    const int64_t at = live ? r : 0;
    load_row<T, TPR, C>(nx, static_cast<const T*>(A.x) + row_at(at, A.N, A.ld, A.stride_b), t, A.D, live);
    load_row<T, TPR, C>(ny, static_cast<const T*>(A.dy) + row_at(at, A.N, A.ld_dy, A.stride_dy), t, A.D, live);
    next_mean = live ? A.mean[r] : 0.f;
    next_rstd = live ? A.rstd[r] : 0.f;
  };
  int64_t r0 = (int64_t)blockIdx.x * RPB;
  if (AHEAD && r0 < A.R) fetch(r0 + threadIdx.x / TPR);
  while (r0 < A.R) {
    const int64_t r = r0 + threadIdx.x / TPR;
    if (!AHEAD) fetch(r);
    const bool live = r < A.R;
    const float mean = next_mean, rstd = next_rstd;
    u32x4 vx[C], vy[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
      vx[j] = nx[j];
      vy[j] = ny[j];
    }
    r0 += (int64_t)gridDim.x * RPB;
    if (AHEAD && r0 < A.R) fetch(r0 + threadIdx.x / TPR);
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int64_t c0 = ((int64_t)j * TPR + t) * E;
      if (c0 >= A.D) break;
      float f[E];
      gamma(j, f);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        // past D the row's gradient is 0, but xh is not: a column of no row
        const float xh = (element<T>(vx[j], e) - mean) * rstd, y = element<T>(vy[j], e), q = y * f[e];
        const bool in = c0 + e < A.D;
        a += q;
        b += in ? q * xh : 0.f;
        if constexpr (ACC) {
          dg[j][e] += in ? y * xh : 0.f;
          db[j][e] += y;
        }
      }
      packed(vx[j]);
      packed(vy[j]);
    }
    if (!A.dx) continue;
    row_sum2<TPR>(a, b, red, turn);
    if (!live) continue;
    T* dx = static_cast<T*>(A.dx) + r * A.D;
    const float ma = a * inv, mb = b * inv;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int64_t c0 = ((int64_t)j * TPR + t) * E;
      if (c0 >= A.D) break;
      float f[E];
      gamma(j, f);
      T o[E];
      if (A.accumulate) {
        const u32x4 old = load_piece<T>(dx, c0, A.D);
        __builtin_memcpy(o, &old, 16);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float xh = (element<T>(vx[j], e) - mean) * rstd;
        const float d = rstd * (element<T>(vy[j], e) * f[e] - ma - xh * mb);
        o[e] = (T)(A.accumulate ? (float)o[e] + d : d);
      }
      store_piece<T>(dx, o, c0, A.D, A.stream);
    }
  }
  if constexpr (ACC) {
    if constexpr (TPR < 64) {  // the rows of a wave
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int o = TPR; o < 64; o *= 2) {
            dg[j][e] += __shfl_xor(dg[j][e], o);
            db[j][e] += __shfl_xor(db[j][e], o);
          }
    }
    constexpr int L = TPR < 64 ? TPR : 64, S = TPR < 64 ? W : RPB;  // lanes with columns of their own, waves to join
    float* part = A.part + (int64_t)blockIdx.x * 2 * A.D;
    if constexpr (S > 1) {
      __shared__ float join[S][2 * E][L];
      const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        __syncthreads();
        if (lane < L) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            join[w][e][lane] = dg[j][e];
            join[w][E + e][lane] = db[j][e];
          }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * E * L; i += W * 64) {
          const int l = i / (2 * E), e = i % (2 * E);
          float v = 0.f;
#pragma unroll
          for (int k = 0; k < S; ++k) v += join[k][e][l];
          const int64_t c = ((int64_t)j * TPR + l) * E + e % E;
          if (c < A.D) part[(e / E) * A.D + c] = v;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int64_t c = ((int64_t)j * TPR + t) * E + e;
          if (c < A.D) {
            part[c] = dg[j][e];
            part[A.D + c] = db[j][e];
          }
        }
    }
  }
}

// gamma's and beta's share of rows too wide for a thread to own its columns
// beside the row: a workgroup takes 256 columns of a slab of rows.
template <typename T>
__global__ void __launch_bounds__(256) norm_columns_kernel(NormArgs A, int64_t rows) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= A.D) return;
  const int64_t r0 = (int64_t)blockIdx.y * rows, r1 = r0 + rows < A.R ? r0 + rows : A.R;
  float dg = 0.f, db = 0.f;
  for (int64_t r = r0; r < r1; ++r) {
    const float x = (float)static_cast<const T*>(A.x)[row_at(r, A.N, A.ld, A.stride_b) + c];
    const float y = (float)static_cast<const T*>(A.dy)[row_at(r, A.N, A.ld_dy, A.stride_dy) + c];
    dg += y * ((x - A.mean[r]) * A.rstd[r]);
    db += y;
  }
  float* part = A.part + (int64_t)blockIdx.y * 2 * A.D;
  part[c] = dg;
  part[A.D + c] = db;
}

// dgamma and dbeta from `parts` rows of 2 D sums: 64 columns a workgroup, the
// parts shared among 16 waves.
__global__ void __launch_bounds__(1024) norm_join_kernel(const float* part, int parts, int64_t D, float* dgamma, float* dbeta,
                                                         int accumulate) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float v = 0.f;
  if (c < 2 * D) {
#pragma unroll 8
    for (int p = w; p < parts; p += 16) v += part[(int64_t)p * 2 * D + c];
  }
  red[w][lane] = v;
  __syncthreads();
  if (w != 0 || c >= 2 * D) return;
  v = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) v += red[k][lane];
  float* o = c < D ? dgamma : dbeta;
  if (!o) return;
  const int64_t i = c < D ? c : c - D;
  o[i] = accumulate ? o[i] + v : v;
}

template <typename F>
hipError_t by_type(int dtype, F f) {
  if (dtype == 0) return f((float)0);
  if (dtype == 1) return f((__bf16)0.f);
  return f((_Float16)0.f);
}

template <typename T, int TPR, int C>
hipError_t run_norm(NormArgs A, hipStream_t s) {
  constexpr int RPB = TPR > 256 ? 1 : 256 / TPR;
  // a launch has fewer than 2^32 threads
  for (const int64_t step = kLaunchThreads / TPR; A.r0 < A.R; A.r0 += step) {
    const int64_t rows = std::min(step, A.R - A.r0);
    hipLaunchKernelGGL((norm_kernel<T, TPR, C>), dim3((unsigned)((rows + RPB - 1) / RPB)), dim3(TPR > 256 ? TPR : 256), 0, s, A);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int TPR, int C, bool ACC>
hipError_t run_grad(const NormArgs& A, unsigned grid, hipStream_t s) {
  hipLaunchKernelGGL((norm_grad_kernel<T, TPR, C, ACC>), dim3(grid), dim3(TPR > 256 ? TPR : 256), 0, s, A);
  return hipGetLastError();
}

}  // namespace

// Threads a row and pieces a thread for rows of `pieces` 16-byte pieces: the
// fewest threads, a power of two, that hold one piece each up to a wave, then up to
// `most` a thread.  bf16 forward: 1M x 24 by 4 lanes 32 us, by 16 93; 65536 x 1024 by
// a wave with 2 pieces 56 us, by 256 threads 123; 32768 x 2048 with 4 pieces 50
// against 68.
static void norm_shape(int64_t pieces, int most, int* tpr, int* c) {
  *tpr = 4;
  while (*tpr < 64 && *tpr < pieces) *tpr *= 2;
  if (pieces > 64 * most) *tpr = pieces <= 256 * most ? 256 : pieces <= 512 * most ? 512 : 1024;
  const int64_t per = (pieces + *tpr - 1) / *tpr;
  *c = per <= 1 ? 1 : per <= 2 ? 2 : per <= 4 ? 4 : 8;
}

// Rows beyond the 32 MB of the eight L2 caches are stored past them: 32768 x 2048
// bf16 forward 80 -> 55 us, with the gradients 168 -> 147.  Fewer stay for the next
// reader.
static bool norm_streams(const NormArgs& A) { return A.R * A.D * (A.dtype == 0 ? 4 : 2) > (int64_t)32 << 20; }

hipError_t launch_norm(NormArgs A, hipStream_t s) {
  A.stream = norm_streams(A);
  return by_type(A.dtype, [&](auto zero) {
    using T = decltype(zero);
    int tpr, c;
    norm_shape((A.D + kPer<T> - 1) / kPer<T>, 4, &tpr, &c);
    switch (tpr * 16 + c) {
      case 4 * 16 + 1: return run_norm<T, 4, 1>(A, s);
      case 8 * 16 + 1: return run_norm<T, 8, 1>(A, s);
      case 16 * 16 + 1: return run_norm<T, 16, 1>(A, s);
      case 32 * 16 + 1: return run_norm<T, 32, 1>(A, s);
      case 64 * 16 + 1: return run_norm<T, 64, 1>(A, s);
      case 64 * 16 + 2: return run_norm<T, 64, 2>(A, s);
      case 64 * 16 + 4: return run_norm<T, 64, 4>(A, s);
      case 256 * 16 + 2: return run_norm<T, 256, 2>(A, s);
      case 256 * 16 + 4: return run_norm<T, 256, 4>(A, s);
      case 512 * 16 + 4: return run_norm<T, 512, 4>(A, s);
      case 1024 * 16 + 4: return run_norm<T, 1024, 4>(A, s);
      default: break;
    }
    if constexpr (sizeof(T) == 4) return run_norm<T, 1024, 8>(A, s);
    return hipErrorInvalidValue;  // D <= 32768
  });
}

NormPlan norm_plan(int64_t R, int64_t D, int dtype, bool want_sums) {
  NormPlan p{};
  const int e = dtype == 0 ? 4 : 8;
  norm_shape((D + e - 1) / e, 2, &p.tpr, &p.c);  // more pieces, fewer waves: their sums beside the row take registers
  // more sums than registers: 2 pieces fit float32 rows (120 of 128) and spill 38 for
  // 16-bit ones; without their sums 4 pieces spill 42 and 75, 8 spill 240
  p.wide = p.c > 2;
  const int64_t rpb = p.tpr >= 256 ? 1 : 256 / p.tpr, groups = (R + rpb - 1) / rpb;
  // sums: enough workgroups to fill the card, each with sums to write and to join
  // (32768 x 2048 bf16, forward and gradients: 512 of them 177 us, 1024 146, 4096 179)
  p.grid = want_sums && !p.wide ? std::min<int64_t>(groups, 1024) : std::min<int64_t>(groups, 1 << 16);
  p.parts = p.wide ? std::min<int64_t>(64, std::max<int64_t>(1, R)) : p.grid;
  p.bytes = want_sums ? sizeof(float) * 2 * (size_t)D * (size_t)p.parts : 0;
  return p;
}

hipError_t launch_norm_grad(NormArgs A, const NormPlan& p, float* dgamma, float* dbeta, hipStream_t s) {
  const bool sums = dgamma || dbeta, acc = sums && !p.wide;
  A.stream = norm_streams(A);
  if (A.dx || acc) {
    const hipError_t e = by_type(A.dtype, [&](auto zero) {
      using T = decltype(zero);
      const unsigned g = (unsigned)p.grid;
      switch ((p.tpr * 16 + p.c) * 2 + acc) {
#define GMM_NORM_GRAD(TPR, C)                                                    \
  case (TPR * 16 + C) * 2: return run_grad<T, TPR, C, false>(A, g, s);           \
  case (TPR * 16 + C) * 2 + 1: return run_grad<T, TPR, C, true>(A, g, s);
        GMM_NORM_GRAD(4, 1)
        GMM_NORM_GRAD(8, 1)
        GMM_NORM_GRAD(16, 1)
        GMM_NORM_GRAD(32, 1)
        GMM_NORM_GRAD(64, 1)
        GMM_NORM_GRAD(64, 2)
        GMM_NORM_GRAD(256, 1)
        GMM_NORM_GRAD(256, 2)
        GMM_NORM_GRAD(512, 2)
        GMM_NORM_GRAD(1024, 2)
#undef GMM_NORM_GRAD
        case (1024 * 16 + 4) * 2: return run_grad<T, 1024, 4, false>(A, g, s);
        default: break;
      }
      if constexpr (sizeof(T) == 4) return run_grad<T, 1024, 8, false>(A, g, s);
      return hipErrorInvalidValue;  // D <= 32768
    });
    if (e != hipSuccess) return e;
  }
  if (!sums) return hipSuccess;
  if (p.wide) {
    const hipError_t e = by_type(A.dtype, [&](auto zero) {
      using T = decltype(zero);
      hipLaunchKernelGGL(norm_columns_kernel<T>, dim3((unsigned)((A.D + 255) / 256), (unsigned)p.parts), dim3(256), 0, s, A,
                         (A.R + p.parts - 1) / p.parts);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_join_kernel, dim3((unsigned)((2 * A.D + 63) / 64)), dim3(1024), 0, s, A.part, (int)p.parts, A.D,
                     dgamma, dbeta, A.accumulate);
  return hipGetLastError();
}

}  // namespace gmm
