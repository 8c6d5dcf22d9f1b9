// gmm_sample.hip -- one token a row from logits, with temperature, min-p, top-k
// and top-p, from one given number u of [0, 1).
//   w_i = exp((l_i - max l) / T);  in descending order of l (ties: lower index)
//   the kept ones are the first k, of those the shortest prefix whose sum
//   reaches top_p of theirs, of those the ones with w >= min_p;
//   the token is the first kept i, by index, with sum_{kept j <= i} w_j > u sum_kept w
// Weights are formed in float64 and held as 64-bit integers, w 2^S rounded, with
// S as large as V such weights leave room for (45 bits at V = 131072): sums do not
// depend on how a row is cut, nor on the order of atomics, and are off by
// 2^-(S+1) a weight.
//
// A row is cut where k elements, or top_p of the mass, are reached by bins of
// its distance to the maximum (1 / 32 of a temperature's unit each): one pass
// finds the maximum, one fills the bins (counts under top-k, sums of weights
// under top-p, by integer atomics in LDS), one collects the elements of the bin
// that the cut falls into and those above it; few enough, they are sorted and
// the row ends there.  Long rows run these as four launches over parts of rows,
// so that one row fills the card too, short rows (kFused) as one.
// 256 rows of 131072, bf16, top-p 0.9: maximum 14 us (4.8 TB/s), bins 40, collecting
// 22, the token 15.  The bins are bound by their arithmetic, 32 instructions an
// element, most of them float64, and by LDS, a table read and an atomic of 8 bytes
// each.  Short rows pay for all 2048 bins too: 1M x 256 float32 under top-p 19 ms.
// One row of 131072, top-k 50: 3.3, 4.6, 6.1 and 8.9 us, latency.
#include "gmm_device.h"

#include <hip/hip_runtime.h>

#include <float.h>

#include <algorithm>

namespace gmm {

namespace {

typedef unsigned long long u64;
constexpr int kBins = 2048, kSegs = 256, kList = 2048;
constexpr int kFewKept = 256;  // top-p: so few elements down to the cut are sorted, more are passed over once more
constexpr double kBinsPerUnit = 32.0;

// Logits in the order of their values, from 1 up.
__device__ inline uint32_t key_of(float l) {
  l += 0.f;  // -0 is 0
  const uint32_t u = __float_as_uint(l);
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ inline float logit_of(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key); }

template <typename T>
struct Row {
  const T* p;
  int64_t V;
  float mx;
  uint32_t first;  // the lowest index of the maximum
  double scale, S; // kBinsPerUnit / temperature, 2^S
  double least;    // min-p
  double u;        // the row's number, in [0, 1)
  float bins;      // scale; NaN where float32 distances would leave its range
  // The distance to the maximum in bins, y >= 0.  exp((l - max) / T) = exp(-b / 32)
  // exp(-t / 32) with b = y rounded and |t| <= 1/2: the first factor is one of
  // kBins values, 0 from there on (2^-92 is below half of any 2^-S), the second
  // its series to t^6 (off by 2^-54).  Descending logits have ascending bins.  A
  // logit's weight is formed again by every pass and each of them has to find the
  // same bits (a token is the element at which sums of two passes meet), so the
  // distance is rounded before b is taken off it, wherever that is compiled.
  __device__ double distance(float l) const {
#pragma clang fp contract(off)
    return ((double)mx - (double)l) * scale;
  }
  __device__ int bin(float l) const { return (int)fmin(rint(distance(l)), (double)(kBins - 1)); }
  static __device__ double near(double y, double b) {
#pragma clang fp contract(off)
    const double t = (y - b) * (-1.0 / kBinsPerUnit);
    double q = 1.0 / 720.0;
    q = fma(q, t, 1.0 / 120.0);
    q = fma(q, t, 1.0 / 24.0);
    q = fma(q, t, 1.0 / 6.0);
    q = fma(q, t, 0.5);
    q = fma(q, t, 1.0);
    return fma(q, t, 1.0);
  }
  static __device__ double far(double b) { return exp_neg(b * (-1.0 / kBinsPerUnit)); }
  __device__ double share(float l) const {
    const double y = distance(l), b = rint(y);
    return b < (double)kBins ? far(b) * near(y, b) : 0.0;
  }
  // e 2^S rounded to an integer: at most 2^52, the low bits of its sum with 2^52
  __device__ u64 fixed(double e) const {
    return (u64)__double_as_longlong(e * S + 0x1p52) - (u64)__double_as_longlong(0x1p52);
  }
  __device__ u64 weight(float l) const { return fixed(share(l)); }
  __device__ u64 weight_min_p(float l) const {
    const double e = share(l);
    return e >= least ? fixed(e) : 0;
  }
};

// U pieces of 16 bytes, `step` elements apart from i on, without a branch: those
// that do not lie whole in [0, i1) are read from its last whole piece (i1 >= E).
template <typename T, int U>
__device__ inline void load_pieces(T (&v)[U][16 / sizeof(T)], const T* p, int64_t i, int64_t step, int64_t i1) {
  constexpr int E = 16 / (int)sizeof(T);
#pragma unroll
  for (int u = 0; u < U; ++u) __builtin_memcpy(v[u], p + min(i + u * step, i1 - E), 16);
}

// f(index, logit) for the live elements of [i0, i1), i0 a multiple of the
// piece, by `threads` threads, U pieces in flight each
template <int U, typename T, typename F>
__device__ inline void each(const Row<T>& R, int64_t i0, int64_t i1, int thread, int threads, F f) {
  constexpr int E = 16 / (int)sizeof(T);
  const auto one = [&](int64_t i, T v) {
    const float l = fminf((float)v, FLT_MAX);
    if ((float)v > -INFINITY) f(i, l);
  };
  const int64_t step = (int64_t)threads * E, whole = i0 + (i1 - i0) / E * E;
  for (int64_t i = i0 + (int64_t)thread * E; i < whole; i += U * step) {
    T v[U][E];
    load_pieces<T, U>(v, R.p, i, step, whole);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u && i + u * step >= whole) break;
#pragma unroll
      for (int e = 0; e < E; ++e) one(i + u * step + e, v[u][e]);
    }
  }
  if (i1 - whole > thread && thread < E) one(whole + thread, R.p[whole + thread]);
}
// 64-bit integers between lanes by DPP: lanes without a source get 0
template <int CTRL, int ROWS = 0xF>
__device__ inline u64 dpp_u64(u64 v) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xF, false);
  return (u64)hi << 32 | lo;
}
// the two halves of 16-lane rows' pairs, and of the wave, as v_permlane*_swap has them
__device__ inline void pair16_u64(u64 v, u64& a, u64& b) {
  const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
  a = (u64)hi[0] << 32 | lo[0];
  b = (u64)hi[1] << 32 | lo[1];
}
__device__ inline void pair32_u64(u64 v, u64& a, u64& b) {
  const auto lo = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
  const auto hi = __builtin_amdgcn_permlane32_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
  a = (u64)hi[0] << 32 | lo[0];
  b = (u64)hi[1] << 32 | lo[1];
}
__device__ inline u64 wave_sum_u64(u64 v) {
  u64 a, b;
  v += dpp_u64<0xB1>(v);
  v += dpp_u64<0x4E>(v);
  v += dpp_u64<0x141>(v);
  v += dpp_u64<0x140>(v);
  pair16_u64(v, a, b);
  pair32_u64(a + b, a, b);
  return a + b;
}
__device__ inline u64 wave_max_u64(u64 v) {
  u64 a, b;
  v = max(v, dpp_u64<0xB1>(v));
  v = max(v, dpp_u64<0x4E>(v));
  v = max(v, dpp_u64<0x141>(v));
  v = max(v, dpp_u64<0x140>(v));
  pair16_u64(v, a, b);
  pair32_u64(max(a, b), a, b);
  return max(a, b);
}
__device__ inline u64 wave_scan_u64(u64 v) {  // inclusive
  v += dpp_u64<0x111>(v);  // from 1, 2, 4 and 8 lanes before in the row
  v += dpp_u64<0x112>(v);
  v += dpp_u64<0x114>(v);
  v += dpp_u64<0x118>(v);
  v += dpp_u64<0x142, 0xA>(v);  // the last lane of the row before, in rows 1 and 3
  v += dpp_u64<0x143, 0xC>(v);  // of the wave's first half, in its second
  return v;
}
template <int TH>
__device__ inline u64 block_sum(u64 v, u64* red) {
  v = wave_sum_u64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int k = 0; k < TH / 64; ++k) v += red[k];
  return v;
}
template <int TH>
__device__ inline u64 block_max(u64 v, u64* red) {
  v = wave_max_u64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int k = 0; k < TH / 64; ++k) v = max(v, red[k]);
  return v;
}
// inclusive over the workgroup
template <int TH>
__device__ inline u64 block_scan(u64 v, u64* red) {
  v = wave_scan_u64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) red[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < TH / 64 - 1; ++k) v += k < (int)(threadIdx.x >> 6) ? red[k] : 0;
  return v;
}

// What is kept: logits above l, and of those equal to it the first `ties` by
// index.  {-INFINITY, 0}: every live element.
struct Cut {
  float l;
  u64 ties;
};

enum Mode { kNone, kGreedy, kOpen, kCount, kMass };
struct Settings {
  Mode mode;
  int64_t k;
  double top_p;
};

struct Cutting {
  u64 red[16], above, edge;
  u64 list[kList];
  int at, na, nb;
};
struct Shared : Cutting {
  u64 bin[kBins], sum[kList], seg[kSegs];
  uint32_t tie[kSegs];
};

// A row's settings, its own before those of the call.
__device__ inline SampleSettings settings_of(const SampleArgs& A, int64_t r) {
  SampleSettings s;
  s.temperature = A.row_temperature ? (double)A.row_temperature[r] : A.temperature;
  s.top_p = A.row_top_p ? (double)A.row_top_p[r] : A.top_p;
  s.min_p = A.row_min_p ? (double)A.row_min_p[r] : A.min_p;
  s.top_k = A.row_top_k ? A.row_top_k[r] : A.top_k;
  s.u = fminf(fmaxf(A.u[r], 0.f), 0x1.fffffep-1f);
  return s;
}

// The row's elements, and what `best` (its largest key, and ~ its lowest index)
// and the settings make of it.
template <typename T>
__device__ inline void place_of(const SampleArgs& A, int64_t r, Row<T>& R) {
  const int64_t b = A.stride_b ? r / A.N : 0;
  R.p = static_cast<const T*>(A.l) + b * A.stride_b + (r - b * A.N) * A.ld;
  R.V = A.V;
  R.S = A.scale;
}
template <typename T>
__device__ inline Settings row_of(const SampleArgs& A, int64_t r, const SampleSettings& s, u64 best, Row<T>& R) {
  place_of(A, r, R);
  R.mx = best ? logit_of((uint32_t)(best >> 32)) : 0.f;
  R.first = ~(uint32_t)best;
  const double t = s.temperature;
  Settings q;
  q.k = s.top_k;
  q.top_p = s.top_p;
  q.mode = !best ? kNone : !(t > 0.0) || q.k == 1 ? kGreedy : q.k > 0 && q.k < A.V ? kCount : q.top_p < 1.0 ? kMass : kOpen;
  R.u = (double)s.u;
  R.scale = t > 0.0 ? fmin(kBinsPerUnit / t, 1e300) : 1.0;
  R.least = s.min_p > 0.0 ? fmin(s.min_p, 1.0) : 0.0;
  // below 2^-100 a difference past float32's largest value may lie in any bin, above
  // 2^100 one among float32's smallest values may
  R.bins = R.scale >= 0x1p-100 && R.scale <= 0x1p100 ? (float)R.scale : __builtin_nanf("");
  return q;
}

// a share of the row: its largest key with ~ its lowest index.  A thread notes
// the piece that its maximum came with, and looks into it at the end.
template <typename T>
__device__ inline u64 best_of(const Row<T>& R, int64_t i0, int64_t i1, int thread, int threads) {
  constexpr int E = 16 / (int)sizeof(T), U = 8;
  const T* p = R.p;
  const int64_t step = (int64_t)threads * E, whole = i0 + (i1 - i0) / E * E;
  float top = -INFINITY;
  int64_t at = -1;
  for (int64_t i = i0 + (int64_t)thread * E; i < whole; i += U * step) {
    T v[U][E];
    load_pieces<T, U>(v, p, i, step, whole);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u && i + u * step >= whole) break;
      float m = -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) m = fmaxf(m, (float)v[u][e]);  // NaN is passed over
      m = fminf(m, FLT_MAX);
      at = m > top ? i + u * step : at;
      top = fmaxf(m, top);
    }
  }
  uint32_t index = 0;
  if (at >= 0) {
#pragma unroll
    for (int e = E - 1; e >= 0; --e) {
      // top is at most FLT_MAX, which +inf counts as; NaN is not above anything
      const float l = (float)p[at + e];
      if (l >= top) index = (uint32_t)(at + e);
    }
  }
  if (i1 - whole > thread && thread < E) {
    const float l = (float)p[whole + thread];
    if (l > -INFINITY && fminf(l, FLT_MAX) > top) {
      top = fminf(l, FLT_MAX);
      index = (uint32_t)(whole + thread);
    }
  }
  return top > -INFINITY ? (u64)key_of(top) << 32 | (uint32_t)~index : 0;
}
// The bins' counts or weights; of an open row the sum of what it keeps, in this
// thread, instead.  factor: exp(-b / 32) of every bin.
template <typename T>
__device__ inline u64 fill_bins(const Row<T>& R, Mode mode, int64_t i0, int64_t i1, int thread, int threads, u64* bin,
                                const double* factor) {
  u64 sum = 0;
  if (mode == kCount) {
    each<2>(R, i0, i1, thread, threads, [&](int64_t, float l) { atomicAdd(&bin[R.bin(l)], (u64)1); });
    return 0;
  }
  const auto share = [&](float l, int& at) {
    const double y = R.distance(l), b = rint(y);
    at = (int)fmin(b, (double)(kBins - 1));
    return b < (double)kBins ? factor[at] * R.near(y, b) : 0.0;
  };
  int at;
  if (mode == kMass) {
    each<2>(R, i0, i1, thread, threads, [&](int64_t, float l) {
      const double e = share(l, at);
      atomicAdd(&bin[at], R.fixed(e));
    });
  } else {
    each<1>(R, i0, i1, thread, threads, [&](int64_t, float l) {
      const double e = share(l, at);
      sum += e >= R.least ? R.fixed(e) : 0;
    });
  }
  return sum;
}
template <typename T>
__device__ inline void fill_factors(const Row<T>& R, int thread, int threads, double* factor) {
#pragma unroll 1
  for (int b = thread; b < kBins; b += threads) factor[b] = R.far((double)b);
}

// sh.at: the bin at which the count or the mass reaches its target (the last one
// that holds anything where it does not), sh.above: what lies before it.  Returns
// the whole.
template <int TH>
__device__ inline u64 cut_bin(const Settings& q, Cutting& sh, const u64* bin) {
  constexpr int EACH = kBins / TH;
  u64 n[EACH], mine = 0;
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    n[e] = bin[threadIdx.x * EACH + e];
    mine += n[e];
  }
  const u64 to = block_scan<TH>(mine, sh.red);
  u64 total = 0;
  __syncthreads();
  if (threadIdx.x == TH - 1) sh.above = to;
  __syncthreads();
  total = sh.above;
  __syncthreads();
  const double target = q.mode == kCount ? fmin((double)q.k, (double)total) : q.top_p * (double)total;
  u64 before = to - mine;
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const u64 after = before + n[e];
    if (n[e] && (double)after >= target && ((double)before < target || before == 0)) {
      sh.at = threadIdx.x * EACH + e;
      sh.above = before;
    }
    before = after;
  }
  __syncthreads();
  return total;
}

// Elements of the bins before sh.at, and of the bin itself, as key << 32 |
// ~index from the two ends of sh.list; counters that pass its half say so.
// Most elements lie below: a thread marks the others of the pieces that it has
// in flight by a comparison with either end (all below where the bin is the last
// one, which has no lower end), and looks at the marked ones after.  Once the
// first list is full, the elements before the bin are passed over.
template <typename T>
__device__ inline void collect(const Row<T>& R, Cutting& sh, int64_t i0, int64_t i1, int thread, int threads) {
  constexpr int E = 16 / (int)sizeof(T), U = 4;
  const int at = sh.at;
  // the float32 distance is off by less than 2^-22 of itself; where it is NaN (no
  // distance in float32, or a NaN logit) the element is looked at
  const float end = at == kBins - 1 ? __builtin_nanf("") : ((float)at + 0.5f) * (1.f + 0x1p-20f);
  const float begin = ((float)at - 0.5f) * (1.f - 0x1p-20f);
  volatile int* filled = &sh.na;
  const auto add = [&](int64_t i, float v) {
    if (!(v > -INFINITY)) return;
    const float l = fminf(v, FLT_MAX);
    const int b = R.bin(l);
    if (b > at) return;
    const u64 entry = (u64)key_of(l) << 32 | (uint32_t)~(uint32_t)i;
    const int slot = atomicAdd(b < at ? &sh.na : &sh.nb, 1);
    if (slot < kList / 2) sh.list[b < at ? slot : kList - 1 - slot] = entry;
  };
  const int64_t step = (int64_t)threads * E, whole = i0 + (i1 - i0) / E * E;
  for (int64_t i = i0 + (int64_t)thread * E; i < whole; i += U * step) {
    T v[U][E];
    load_pieces<T, U>(v, R.p, i, step, whole);
    const float from = *filled > kList / 2 ? begin : -INFINITY;
    uint32_t marked = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float y = (R.mx - (float)v[u][e]) * R.bins;
        m |= !(y >= end) && !(y < from) ? 1u << e : 0u;
      }
      if (i + u * step < whole) marked |= m << (u * E);
    }
    while (marked) {
      const int k = __builtin_ctz(marked);
      marked &= marked - 1;
      const int64_t j = i + k / E * step + k % E;
      add(j, (float)R.p[j]);
    }
  }
  if (i1 - whole > thread && thread < E) add(whole + thread, (float)R.p[whole + thread]);
  __syncthreads();
}

// sh.list[0, n) in descending order
template <int TH>
__device__ inline void sort_list(Shared& sh, int n) {
  int size = 64;
  while (size < n) size *= 2;
  for (int i = n + threadIdx.x; i < size; i += TH) sh.list[i] = 0;
  __syncthreads();
  for (int k = 2; k <= size; k *= 2)
    for (int j = k / 2; j; j /= 2) {
      for (int t = threadIdx.x; t < size / 2; t += TH) {
        const int a = 2 * t - (t & (j - 1)), b = a + j;
        const u64 x = sh.list[a], y = sh.list[b];
        if ((x < y) == ((a & k) == 0)) {
          sh.list[a] = y;
          sh.list[b] = x;
        }
      }
      __syncthreads();
    }
}

// sh.sum[i]: the sum of f(0 .. i), i < n <= kList
template <int TH, typename F>
__device__ inline void scan_list(Shared& sh, int n, F f) {
  u64 base = 0;
  for (int i0 = 0; i0 < n; i0 += TH) {
    const int i = i0 + threadIdx.x;
    const u64 to = base + block_scan<TH>(i < n ? f(i) : 0, sh.red);
    if (i < n) sh.sum[i] = to;
    __syncthreads();
    base = sh.sum[min(i0 + TH, n) - 1];
  }
}

__device__ inline float list_logit(u64 v) { return logit_of((uint32_t)(v >> 32)); }
template <typename T>
__device__ inline void answer(const SampleArgs& A, const Row<T>& R, int64_t r, float l, int64_t i, u64 total) {
#pragma clang fp contract(off)
  A.tokens[r] = (int32_t)i;
  if (A.logp) A.logp[r] = (float)(-R.distance(l) / kBinsPerUnit - log((double)total / R.S));
}
template <typename T>
__device__ inline double aim(const Row<T>& R, u64 total) {
  return R.u * (double)total;
}

template <int TH>
__device__ inline u64 group_sum(u64 v, u64* red) {
  if constexpr (TH == 64) return wave_sum_u64(v);
  else return block_sum<TH>(v, red);
}
template <int TH>
__device__ inline void group_sync() {
  if constexpr (TH == 64) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  } else {
    __syncthreads();
  }
}

// finish_list for n <= kFewKept: places and sums by comparing each element with
// every other one, G threads an element (one wave, without barriers, for n <= 64).
template <int TH, typename T>
__device__ __forceinline__ void finish_few(const SampleArgs& A, const Row<T>& R, const Settings& q, int64_t r, Shared& sh, int n,
                                           u64 mass) {
  constexpr int G = TH / kFewKept > 0 ? TH / kFewKept : 1;
  const int i = threadIdx.x / G, g = threadIdx.x % G;
  const bool own = i < n && g == 0;
  const u64 mine = i < n ? sh.list[i] : 0;
  const double e = i < n ? R.share(list_logit(mine)) : 0.0;
  const u64 w = i < n ? R.fixed(e) : 0;
  if (own) sh.sum[i] = w;
  group_sync<TH>();
  int place = 0;
  u64 before = 0;
  const int others = (threadIdx.x & ~63) / G < n ? n : 0;  // waves without an element have nothing to compare
#pragma unroll 8
  for (int j = g; j < others; j += G) {
    const bool ahead = sh.list[j] > mine;
    place += ahead;
    before += ahead ? sh.sum[j] : 0;
  }
#pragma unroll
  for (int o = 1; o < G; o *= 2) {
    place += __shfl_xor(place, o);
    before += __shfl_xor(before, o);
  }
  const bool first = q.mode != kCount || place < q.k;
  if (q.mode == kCount && q.top_p < 1.0) mass = group_sum<TH>(own && first ? w : 0, sh.red);
  const bool in = own && (place == 0 || (first && (!(q.top_p < 1.0) || (double)before < q.top_p * (double)mass) && e >= R.least));
  const u64 total = group_sum<TH>(in ? w : 0, sh.red);
  const double goal = aim(R, total);
  group_sync<TH>();
  if (own) sh.sum[i] = in ? w : 0;
  group_sync<TH>();
  u64 to = 0;
#pragma unroll 8
  for (int j = g; j < others; j += G) to += (uint32_t)sh.list[j] >= (uint32_t)mine ? sh.sum[j] : 0;  // ~index: descending
#pragma unroll
  for (int o = 1; o < G; o *= 2) to += __shfl_xor(to, o);
  if (in && (double)to > goal && !((double)(to - w) > goal)) answer(A, R, r, list_logit(mine), ~(uint32_t)mine, total);
}

// The row ends with a list of its n largest elements, among which the cut lies.
// mass: of the row (top-p without top-k).
template <int TH, typename T>
__device__ __forceinline__ void finish_list(const SampleArgs& A, const Row<T>& R, const Settings& q, int64_t r, Shared& sh, int n, u64 mass) {
  if (n <= 64) {
    if (threadIdx.x < 64) finish_few<64>(A, R, q, r, sh, n, mass);
    return;
  }
  if (n <= kFewKept) {
    finish_few<TH>(A, R, q, r, sh, n, mass);
    return;
  }
  sort_list<TH>(sh, n);
  if (q.mode == kCount) n = (int)min((int64_t)n, q.k);
  scan_list<TH>(sh, n, [&](int i) { return R.weight(list_logit(sh.list[i])); });
  // the kept ones are a prefix: count them
  const double target = q.top_p * (double)(q.mode == kCount ? sh.sum[n - 1] : mass);
  u64 mine = 0;
  for (int i = threadIdx.x; i < n; i += TH) {
    const bool in = i == 0 || ((!(q.top_p < 1.0) || (double)sh.sum[i - 1] < target) &&
                               (R.least == 0.0 || R.share(list_logit(sh.list[i])) >= R.least));
    mine += in;
  }
  const int kept = (int)block_sum<TH>(mine, sh.red);
  const u64 total = sh.sum[kept - 1];
  __syncthreads();
  // by index: ~index << 32 | place, largest first, with the weights' differences
  for (int i = threadIdx.x; i < kept; i += TH) sh.list[i] = (sh.list[i] << 32) | (uint32_t)i;
  __syncthreads();
  // weights from the sums before these are overwritten
  u64 w[kList / TH];
  sort_list<TH>(sh, kept);
#pragma unroll
  for (int e = 0; e < kList / TH; ++e) {
    const int i = e * TH + threadIdx.x;
    if (i < kept) {
      const uint32_t at = (uint32_t)sh.list[i];
      w[e] = sh.sum[at] - (at ? sh.sum[at - 1] : 0);
    }
  }
  __syncthreads();
  u64 base = 0;
  const double goal = aim(R, total);
#pragma unroll
  for (int e = 0; e < kList / TH; ++e) {
    if (e * TH >= kept) break;
    const int i = e * TH + threadIdx.x;
    const u64 mine_w = i < kept ? w[e] : 0, to = base + block_scan<TH>(mine_w, sh.red);
    if (i < kept && (double)to > goal && !((double)(to - mine_w) > goal)) {
      const uint32_t index = ~(uint32_t)(sh.list[i] >> 32);
      answer(A, R, r, fminf((float)R.p[index], FLT_MAX), index, total);
    }
    __syncthreads();
    if (threadIdx.x == TH - 1) sh.above = to;
    __syncthreads();
    base = sh.above;
  }
}

// One wave: the place at which sums over lanes pass the goal.  n and ties are
// this lane's, wt the weight of a tie, of which `left` are kept; before is what
// lies before lane 0.  Afterwards `before` and `left` are those of the lane
// returned (the last one with anything if none passes).
__device__ inline int pass_at(u64 n, u64 ties, u64 wt, double goal, u64& before, u64& left) {
  const u64 ties_to = wave_scan_u64(ties), ties_from = ties_to - ties;
  n += (min(ties_to, left) - min(ties_from, left)) * wt;
  const u64 to = before + wave_scan_u64(n);
  const u64 hit = __ballot((double)to > goal), any = __ballot(n != 0);
  const int lane = hit ? __builtin_ctzll(hit) : any ? 63 - __builtin_clzll(any) : 0;
  before = __shfl(to - n, lane);
  left -= min(__shfl(ties_from, lane), left);
  return lane;
}

// One wave: the entry of sh.seg (and sh.tie), PER a lane, at which the sum
// passes the goal, as pass_at has it.
template <int PER>
__device__ inline int pass_list(const Shared& sh, u64 wt, double goal, u64& before, u64& left) {
  const int lane = threadIdx.x & 63;
  u64 n = 0, ties = 0;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    n += sh.seg[lane * PER + e];
    ties += sh.tie[lane * PER + e];
  }
  int s = pass_at(n, ties, wt, goal, before, left) * PER;
  for (int e = 0; e < PER - 1; ++e, ++s) {
    const u64 t = min((u64)sh.tie[s], left), m = sh.seg[s] + t * wt;
    if ((double)(before + m) > goal) break;
    before += m;
    left -= t;
  }
  return s;
}
// the whole of sh.seg and sh.tie, by one wave
template <int PER>
__device__ inline u64 whole_list(const Shared& sh, u64 wt, u64 left) {
  const int lane = threadIdx.x & 63;
  u64 n = 0, ties = 0;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    n += sh.seg[lane * PER + e];
    ties += sh.tie[lane * PER + e];
  }
  return wave_sum_u64(n) + min(wave_sum_u64(ties), left) * wt;
}

// The least logit that a cut may keep.
__device__ inline float least_kept(const Cut& cut) { return cut.ties ? cut.l : nextafterf(cut.l, INFINITY); }

// Bit e: element e of the piece at i may be kept; pieces that are not whole below
// b are looked at one by one.
template <typename T>
__device__ inline uint32_t marks(const T (&v)[16 / sizeof(T)], float least) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 16 / (int)sizeof(T); ++e) m |= (float)v[e] >= least ? 1u << e : 0u;
  return m;
}

// Kept weights and elements equal to the cut of the segments of `len` elements;
// a wave reads two of them at once, and opens the marked elements after.
template <int TH, typename T>
__device__ inline void segments(const Row<T>& R, const Cut& cut, int64_t i0, int64_t i1, int64_t len, Shared& sh) {
  constexpr int E = 16 / (int)sizeof(T), U = 2;
  const int lane = threadIdx.x & 63;
  const float least = least_kept(cut);
  const int64_t whole = i0 + (i1 - i0) / E * E;
  const int used = (int)((i1 - i0 + len - 1) / len);
  for (int s = used + threadIdx.x; s < kSegs; s += TH) {
    sh.seg[s] = 0;
    sh.tie[s] = 0;
  }
  for (int s = (threadIdx.x >> 6) * U; s < used; s += TH / 64 * U) {
    u64 mass0 = 0, mass1 = 0;
    uint32_t ties0 = 0, ties1 = 0;
    const auto one = [&](bool second, float v) {
      if (!(v >= least)) return;
      const float l = fminf(v, FLT_MAX);
      const u64 w = l > cut.l ? R.weight_min_p(l) : 0;
      const uint32_t t = l == cut.l;
      (second ? mass1 : mass0) += w;
      (second ? ties1 : ties0) += t;
    };
    for (int64_t t = 0; t < len && i0 + s * len + t < whole; t += 64 * E) {
      const int64_t i = i0 + s * len + t + lane * E;
      T v[U][E];
      load_pieces<T, U>(v, R.p, i, len, whole);
      uint32_t marked = i < whole ? marks<T>(v[0], least) : 0;
      if (i + len < whole) marked |= marks<T>(v[1], least) << E;
#pragma unroll 1
      while (marked) {
        const int k = __builtin_ctz(marked);
        marked &= marked - 1;
        one(k >= E, (float)R.p[i + k / E * len + k % E]);
      }
    }
    // the last elements, less than a piece, belong to the segment that they lie in
    const int64_t a = i0 + s * len;
    if (whole + lane < i1 && lane < E && whole >= a && whole < a + U * len)
      one(whole >= a + len, (float)R.p[whole + lane]);
    mass0 = wave_sum_u64(mass0);
    mass1 = wave_sum_u64(mass1);
    const u64 ties = wave_sum_u64((u64)ties1 << 32 | ties0);
    if (lane == 0) {
      sh.seg[s] = mass0;
      sh.tie[s] = (uint32_t)ties;
      if (s + 1 < used) {
        sh.seg[s + 1] = mass1;
        sh.tie[s + 1] = (uint32_t)(ties >> 32);
      }
    }
  }
}

// The row's (or a part's) segments of whole tiles: their kept weights and their
// elements equal to the cut; then, in one wave, the segment, the tile and the
// element at which the sum passes the goal.  goal < 0: that of the whole.
template <int TH, typename T>
__device__ __forceinline__ void choose(const SampleArgs& A, const Row<T>& R, const Cut& cut, int64_t r, int64_t i0, int64_t i1, u64 before, u64 total,
                       double goal, Shared& sh) {
  constexpr int E = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 63;
  const int64_t tile = 64 * E, tiles = (i1 - i0 + tile - 1) / tile, len = (tiles + kSegs - 1) / kSegs * tile;
  __syncthreads();
  segments<TH>(R, cut, i0, i1, len, sh);
  __syncthreads();
  if (threadIdx.x >= 64) return;
  const u64 wt = cut.ties ? R.weight_min_p(cut.l) : 0;
  if (goal < 0.0) {
    total = whole_list<kSegs / 64>(sh, wt, cut.ties);
    goal = aim(R, total);
  }
  u64 left = cut.ties;
  const int s = pass_list<kSegs / 64>(sh, wt, goal, before, left);
  const float least = least_kept(cut);
  for (int64_t a = i0 + s * len, end = min(a + len, i1); a < end; a += tile) {
    const int64_t i = a + (int64_t)lane * E;
    uint32_t marked = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (i + e < end && (float)R.p[i + e] >= least) marked |= 1u << e;
    // twice over the lane's kept elements: their sum, then the one that passes
    u64 mass = 0, tied = 0, rank = 0, sum = 0;
    bool last = false;
    for (;;) {
#pragma unroll 1
      for (uint32_t m = marked; m; m &= m - 1) {
        const int64_t at = i + __builtin_ctz(m);
        const float l = fminf((float)R.p[at], FLT_MAX);
        const bool tie = l == cut.l;
        if (!last) {
          tied += tie;
          if (!tie) mass += R.weight_min_p(l);
        } else {
          if (!tie) sum += R.weight_min_p(l);
          else if (rank++ < left) sum += wt;
          if ((double)sum > goal) {
            answer(A, R, r, l, at, total);
            return;
          }
        }
      }
      if (last) return;
      const u64 tied_to = wave_scan_u64(tied), tied_from = tied_to - tied;
      mass += (min(tied_to, left) - min(tied_from, left)) * wt;
      const u64 to = before + wave_scan_u64(mass);
      const u64 hit = __ballot((double)to > goal);
      if (!hit) {
        before = __shfl(to, 63);
        left -= min(__shfl(tied_to, 63), left);
        break;
      }
      if (lane != __builtin_ctzll(hit)) return;
      last = true;
      sum = to - mass;
      rank = tied_from;
    }
  }
}

// The prefix of the kept elements, by descending key, at which the count (by
// mass: the sum of the weights) first reaches `target`: bins of the keys'
// range, then of the bin that it is reached in, until one key is left.  For
// rows whose cut lies among more equal or nearly equal logits than a list holds.
template <int TH, bool MASS, typename T>
__device__ __forceinline__ Cut reach(const Row<T>& R, Shared& sh, Cut kept, double target) {
  const uint32_t cut = kept.ties ? key_of(kept.l) : 0;
  uint32_t lo = cut ? cut : 1, hi = key_of(R.mx);
  u64 above = 0;
  const u64 tied = kept.ties * (MASS && cut ? R.weight(kept.l) : 1);
  for (;;) {
    int shift = 0;
    while (((hi - lo) >> shift) >= kBins) ++shift;
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += TH) sh.bin[i] = 0;
    __syncthreads();
    each<1>(R, 0, R.V, threadIdx.x, TH, [&](int64_t, float l) {
      const uint32_t key = key_of(l);
      if (key >= lo && key <= hi && key != cut) atomicAdd(&sh.bin[(hi - key) >> shift], MASS ? R.weight(l) : (u64)1);
    });
    __syncthreads();
    if (threadIdx.x == 0) {
      if (cut >= lo && cut <= hi) sh.bin[(hi - cut) >> shift] += tied;
      sh.at = -1;
    }
    __syncthreads();
    constexpr int EACH = kBins / TH;
    u64 n[EACH], mine = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      n[e] = sh.bin[threadIdx.x * EACH + e];
      mine += n[e];
    }
    u64 before = above + block_scan<TH>(mine, sh.red) - mine;
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      const u64 after = before + n[e];
      if (n[e] && (double)after >= target && ((double)before < target || before == 0)) {
        sh.at = threadIdx.x * EACH + e;
        sh.above = before;
      }
      before = after;
    }
    __syncthreads();
    const int at = sh.at;
    if (at < 0) return kept;
    above = sh.above;
    const u64 in = sh.bin[at];
    hi -= (uint32_t)at << shift;
    const uint32_t last = hi - (((uint32_t)1 << shift) - 1);
    lo = last > lo && last <= hi ? last : lo;
    if (shift != 0) continue;
    const u64 w = MASS ? R.weight(logit_of(hi)) : 1, have = in / w;
    u64 ties = target > (double)above ? (u64)((target - (double)above) / (double)w) : 1;
    ties = ties < 1 ? 1 : ties > have ? have : ties;
    while (ties > 1 && (double)(above + (ties - 1) * w) >= target) --ties;
    while (ties < have && (double)(above + ties * w) < target) ++ties;
    return Cut{logit_of(hi), ties};
  }
}

template <int TH, typename T>
__device__ __forceinline__ Cut cut_by_reach(const Row<T>& R, const Settings& q, Shared& sh) {
  Cut cut{-INFINITY, 0};
  if (q.mode == kCount) cut = reach<TH, false>(R, sh, cut, (double)q.k);
  if (q.top_p < 1.0) {
    u64 mass = 0;
    each<1>(R, 0, R.V, threadIdx.x, TH, [&](int64_t, float l) {
      if (l > cut.l) mass += R.weight(l);
    });
    mass = block_sum<TH>(mass, sh.red) + (cut.ties ? cut.ties * R.weight(cut.l) : 0);
    cut = reach<TH, true>(R, sh, cut, q.top_p * (double)mass);
  }
  return cut;
}

// The cut of a row whose mass is `whole`, among the nb elements of its bin in
// sh.list (sh.above: the mass before them); sh.edge: its last element.
template <int TH, typename T>
__device__ __forceinline__ Cut cut_of_bin(const Row<T>& R, const Settings& q, Shared& sh, u64 whole, int nb) {
  const u64 above = sh.above;
  const double target = q.top_p * (double)whole;
  if (nb <= kFewKept) {
    constexpr int G = TH / kFewKept;
    const int i = threadIdx.x / G, g = threadIdx.x % G;
    const u64 mine = i < nb ? sh.list[i] : 0, w = i < nb ? R.weight(list_logit(mine)) : 0;
    if (i < nb && g == 0) sh.sum[i] = w;
    __syncthreads();
    u64 before = 0;
    int place = 0;
    const int others = (threadIdx.x & ~63) / G < nb ? nb : 0;
#pragma unroll 8
    for (int j = g; j < others; j += G) {
      const bool ahead = sh.list[j] > mine;
      before += ahead ? sh.sum[j] : 0;
      place += ahead;
    }
#pragma unroll
    for (int o = 1; o < G; o *= 2) {
      before += __shfl_xor(before, o);
      place += __shfl_xor(place, o);
    }
    before += above;
    if (i < nb && g == 0 && (double)(before + w) >= target && (place == 0 || (double)before < target)) sh.edge = mine;
    __syncthreads();
    const u64 edge = sh.edge;
    const bool tie = i < nb && g == 0 && mine >= edge && mine >> 32 == edge >> 32;
    return Cut{list_logit(edge), block_sum<TH>(tie, sh.red)};
  }
  sort_list<TH>(sh, nb);
  scan_list<TH>(sh, nb, [&](int i) { return R.weight(list_logit(sh.list[i])); });
  for (int i = threadIdx.x; i < nb; i += TH)
    if ((double)(above + sh.sum[i]) >= target && (i == 0 || (double)(above + sh.sum[i - 1]) < target)) sh.edge = sh.list[i];
  __syncthreads();
  const u64 edge = sh.edge;
  u64 same = 0;
  for (int i = threadIdx.x; i < nb; i += TH) same += sh.list[i] >= edge && sh.list[i] >> 32 == edge >> 32;
  return Cut{list_logit(edge), block_sum<TH>(same, sh.red)};
}

template <typename T>
__device__ inline bool plain_answer(const SampleArgs& A, const Row<T>& R, const Settings& q, int64_t r) {
  if (q.mode != kNone && q.mode != kGreedy) return false;
  if (threadIdx.x == 0) {
    A.tokens[r] = q.mode == kNone ? -1 : (int32_t)R.first;
    if (A.logp) A.logp[r] = q.mode == kNone ? -INFINITY : 0.f;
  }
  return true;
}

// A row by one workgroup.
template <typename T, int TH>
__global__ void __launch_bounds__(TH) sample_row_kernel(SampleArgs A) {
  __shared__ Shared sh;
  const int64_t r = (int64_t)blockIdx.x + A.r0;
  Row<T> R;
  const SampleSettings own = settings_of(A, r);
  place_of(A, r, R);
  const Settings q = row_of(A, r, own, block_max<TH>(best_of(R, 0, R.V, threadIdx.x, TH), sh.red), R);
  if (plain_answer(A, R, q, r)) return;
  Cut cut{-INFINITY, 0};
  int64_t i0 = 0, i1 = R.V;
  u64 before = 0, total = 0;
  double goal = -1.0, *factor = reinterpret_cast<double*>(sh.sum);
  if (q.mode == kOpen) {
    // a wave sums a share of the row, whole tiles; the token lies in one of them
    const int64_t len = ((R.V + TH / 64 - 1) / (TH / 64) + 511) / 512 * 512;
    const int wave = threadIdx.x >> 6;
    fill_factors(R, threadIdx.x, TH, factor);
    for (int i = threadIdx.x; i < kSegs; i += TH) {
      sh.seg[i] = 0;
      sh.tie[i] = 0;
    }
    __syncthreads();
    const u64 mass = wave_sum_u64(fill_bins(R, kOpen, min(wave * len, R.V), min((wave + 1) * len, R.V), threadIdx.x & 63, 64,
                                            sh.bin, factor));
    if ((threadIdx.x & 63) == 0) sh.seg[wave] = mass;
    __syncthreads();
    // every wave
    total = whole_list<kSegs / 64>(sh, 0, 0);
    goal = aim(R, total);
    u64 left = 0;
    i0 = pass_list<kSegs / 64>(sh, 0, goal, before, left) * len;
    i1 = min(i0 + len, R.V);
  } else {
    for (int i = threadIdx.x; i < kBins; i += TH) sh.bin[i] = 0;
    if (threadIdx.x == 0) sh.na = sh.nb = 0;
    if (q.mode == kMass) fill_factors(R, threadIdx.x, TH, factor);
    __syncthreads();
    fill_bins(R, q.mode, 0, R.V, threadIdx.x, TH, sh.bin, factor);
    __syncthreads();
    const u64 whole = cut_bin<TH>(q, sh, sh.bin);
    collect(R, sh, 0, R.V, threadIdx.x, TH);
    const int na = sh.na, nb = sh.nb;
    const bool list = na <= kList / 2 && nb <= kList / 2 && (q.mode == kCount || na + nb <= kFewKept);
    if (!list && (q.mode == kCount || nb > kList / 2)) {
      cut = cut_by_reach<TH>(R, q, sh);
    } else {
      // the bin's elements from the list's end to its front, behind those above it
      const int to = list ? na : 0;
      u64 v[kList / 2 / TH];
#pragma unroll
      for (int e = 0; e < kList / 2 / TH; ++e) {
        const int i = e * TH + threadIdx.x;
        if (i < nb) v[e] = sh.list[kList - 1 - i];
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kList / 2 / TH; ++e) {
        const int i = e * TH + threadIdx.x;
        if (i < nb) sh.list[to + i] = v[e];
      }
      __syncthreads();
      if (list) {
        finish_list<TH>(A, R, q, r, sh, na + nb, whole);
        return;
      }
      cut = cut_of_bin<TH>(R, q, sh, whole, nb);
    }
  }
  choose<TH>(A, R, cut, r, i0, i1, before, total, goal, sh);
}

// Long rows: parts of a row in workgroups of their own, whose waves have a
// quarter each where what is kept is summed.
constexpr int kQuarters = 4;
__device__ inline void part_of(const SampleArgs& A, int64_t& i0, int64_t& i1) {
  i0 = (int64_t)blockIdx.x * A.part;
  i1 = min(i0 + A.part, A.V);
}
__device__ inline void quarter_of(const SampleArgs& A, int64_t& q0, int64_t& q1) {
  const int64_t quarter = A.part / kQuarters;
  q0 = min((int64_t)blockIdx.x * A.part + (threadIdx.x >> 6) * quarter, A.V);
  q1 = min(q0 + quarter, A.V);
}
// every wave looks at all parts
__device__ inline u64 best_part(const SampleRow& w, int parts) {
  const int lane = threadIdx.x & 63;
  return wave_max_u64(lane < parts ? (u64)w.best[lane] : 0);
}

template <typename T>
__global__ void __launch_bounds__(256) sample_best_kernel(SampleArgs A) {
  constexpr int TH = 256;
  __shared__ u64 red[TH / 64];
  const int64_t r = (int64_t)blockIdx.y + A.r0;
  SampleRow& w = A.rows[blockIdx.y];
  Row<T> R;
  place_of(A, r, R);
  int64_t i0, i1;
  part_of(A, i0, i1);
  const u64 best = block_max<TH>(best_of(R, i0, i1, threadIdx.x, TH), red);
  if (threadIdx.x == 0) {
    w.best[blockIdx.x] = best;
    if (blockIdx.x == 0) {
      w.na = w.nb = 0;
      w.settings = settings_of(A, r);
    }
  }
  for (int i = blockIdx.x * TH + threadIdx.x; i < kBins; i += gridDim.x * TH) w.bin[i] = 0;
}

template <typename T>
__global__ void __launch_bounds__(256) sample_bins_kernel(SampleArgs A) {
  constexpr int TH = 256;
  __shared__ u64 bin[kBins];
  __shared__ double factor[kBins];
  const int64_t r = (int64_t)blockIdx.y + A.r0;
  SampleRow& w = A.rows[blockIdx.y];
  Row<T> R;
  for (int i = threadIdx.x; i < kBins; i += TH) bin[i] = 0;
  const Settings q = row_of(A, r, w.settings, best_part(w, gridDim.x), R);
  if (q.mode == kNone || q.mode == kGreedy) return;
  int64_t i0, i1;
  part_of(A, i0, i1);
  if (q.mode != kCount) fill_factors(R, threadIdx.x, TH, factor);
  __syncthreads();
  const bool open = q.mode == kOpen;  // its waves take a quarter each
  if (open) quarter_of(A, i0, i1);
  const u64 mass = wave_sum_u64(
      fill_bins(R, q.mode, i0, i1, open ? threadIdx.x & 63 : threadIdx.x, open ? 64 : TH, bin, factor));
  if (open) {
    if ((threadIdx.x & 63) == 0) w.mass[blockIdx.x * kQuarters + (threadIdx.x >> 6)] = mass;
    return;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += TH)
    if (bin[i]) atomicAdd((u64*)&w.bin[i], bin[i]);
}

template <typename T>
__global__ void __launch_bounds__(256) sample_collect_kernel(SampleArgs A) {
  constexpr int TH = 256;
  __shared__ Cutting sh;
  const int64_t r = (int64_t)blockIdx.y + A.r0;
  SampleRow& w = A.rows[blockIdx.y];
  Row<T> R;
  const Settings q = row_of(A, r, w.settings, best_part(w, gridDim.x), R);
  if (q.mode != kCount && q.mode != kMass) return;
  const u64 whole = cut_bin<TH>(q, sh, (const u64*)w.bin);
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) {
      w.whole = whole;
      w.above = sh.above;
      w.at = sh.at;
    }
    sh.na = sh.nb = 0;
  }
  __syncthreads();
  int64_t i0, i1, q0, q1;
  part_of(A, i0, i1);
  quarter_of(A, q0, q1);
  collect(R, sh, i0, i1, threadIdx.x, TH);
  // a place in the row's list for all of them; too many here are too many there
  const int na = sh.na, nb = sh.nb;
  __shared__ int base[2];
  if (threadIdx.x == 0) {
    base[0] = na ? atomicAdd(&w.na, na > kList / 2 ? kSampleList + 1 : na) : 0;
    base[1] = nb ? atomicAdd(&w.nb, nb > kList / 2 ? kSampleList + 1 : nb) : 0;
  }
  __syncthreads();
  if (na <= kList / 2)
    for (int i = threadIdx.x; i < na; i += TH)
      if (base[0] + i < kSampleList) w.list[base[0] + i] = sh.list[i];
  if (nb <= kList / 2)
    for (int i = threadIdx.x; i < nb; i += TH)
      if (base[1] + i < kSampleList) w.list[2 * kSampleList - 1 - base[1] - i] = sh.list[kList - 1 - i];
  if (q.mode == kMass) {  // what the part keeps for sure
    if (na <= kList / 2) {
      if (threadIdx.x < kQuarters) sh.red[threadIdx.x] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < na; i += TH)
        atomicAdd(&sh.red[(~(uint32_t)sh.list[i] - (uint32_t)i0) >> (A.part_bits - 2)], R.weight_min_p(list_logit(sh.list[i])));
      __syncthreads();
      if (threadIdx.x < kQuarters) w.mass[blockIdx.x * kQuarters + threadIdx.x] = sh.red[threadIdx.x];
    } else {
      // many: by the bins' factors, in the list's place
      static_assert(kList >= kBins, "a factor an entry");
      double* factor = reinterpret_cast<double*>(sh.list);
      __syncthreads();
      fill_factors(R, threadIdx.x, TH, factor);
      __syncthreads();
      const double at = (double)sh.at;
      u64 mass = 0;
      each<1>(R, q0, q1, threadIdx.x & 63, 64, [&](int64_t, float l) {
        const double y = R.distance(l), b = rint(y);
        if (b < at) {
          const double e = factor[(int)b] * R.near(y, b);
          mass += e >= R.least ? R.fixed(e) : 0;
        }
      });
      mass = wave_sum_u64(mass);
      if ((threadIdx.x & 63) == 0) w.mass[blockIdx.x * kQuarters + (threadIdx.x >> 6)] = mass;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(1024) sample_finish_kernel(SampleArgs A, int parts) {
  constexpr int TH = 1024;
  __shared__ Shared sh;
  const int64_t r = (int64_t)blockIdx.x + A.r0;
  SampleRow& w = A.rows[blockIdx.x];
  // what the row may need, on its way while its maximum is found
  const SampleSettings own = w.settings;
  const int na = w.na, nb = w.nb;
  const u64 whole = w.whole, above = w.above, mass = threadIdx.x < parts * kQuarters ? w.mass[threadIdx.x] : 0;
  const u64 front = w.list[threadIdx.x], back = w.list[2 * kSampleList - 1 - threadIdx.x];
  Row<T> R;
  const Settings q = row_of(A, r, own, best_part(w, parts), R);
  if (plain_answer(A, R, q, r)) return;
  Cut cut{-INFINITY, 0};
  int64_t i0 = 0, i1 = A.V;
  u64 before = 0, total = 0;
  double goal = -1.0;
  const bool list = na <= kSampleList && nb <= kSampleList && na + nb <= (q.mode == kCount ? kList : kFewKept);
  if (q.mode != kOpen && !list && (q.mode == kCount || nb > kList)) {
    cut = cut_by_reach<TH>(R, q, sh);
  } else {
    static_assert(kSegs >= kSampleParts * kQuarters && TH >= kSegs, "a segment a quarter, a thread a segment");
    const int s = threadIdx.x;
    const int64_t quarter = A.part / kQuarters;
    if (s < kSegs) {
      sh.seg[s] = mass;
      sh.tie[s] = 0;
    }
    u64 wt = 0;
    if (q.mode != kOpen) {
      const int to = list ? na : 0;
      for (int i = threadIdx.x; i < to; i += TH) sh.list[i] = i < TH ? front : w.list[i];
      for (int i = threadIdx.x; i < nb; i += TH) sh.list[to + i] = i < TH ? back : w.list[2 * kSampleList - 1 - i];
      if (threadIdx.x == 0) sh.above = above;
      __syncthreads();
      if (list) {
        finish_list<TH>(A, R, q, r, sh, na + nb, whole);
        return;
      }
      cut = cut_of_bin<TH>(R, q, sh, whole, nb);
      // what the quarters keep of the bin: all above the cut, and the ties by index
      for (int i = threadIdx.x; i < nb; i += TH) {
        if (sh.list[i] < sh.edge) continue;
        const float l = list_logit(sh.list[i]);
        const int k = (int)(~(uint32_t)sh.list[i] >> (A.part_bits - 2));  // its quarter
        if (l > cut.l) atomicAdd(&sh.seg[k], R.weight_min_p(l));
        else atomicAdd(&sh.tie[k], 1u);
      }
      wt = R.weight_min_p(cut.l);
    }
    __syncthreads();
    // every wave
    total = whole_list<kSegs / 64>(sh, wt, cut.ties);
    goal = aim(R, total);
    u64 left = cut.ties;
    const int k = pass_list<kSegs / 64>(sh, wt, goal, before, left);
    cut.ties = left;
    i0 = (k / kQuarters) * A.part + (k % kQuarters) * quarter;
    i1 = min(i0 + quarter, A.V);
  }
  choose<TH>(A, R, cut, r, i0, i1, before, total, goal, sh);
}

// The longest row that one workgroup takes.  One workgroup and row against parts
// in four launches, bf16, top-p 0.9: 256 x 8192 24 against 38 us, 256 x 32768 37
// against 49; past it top-p alone costs a single row more than four launches do
// (50001: 39 against 31), and flat rows do from here (one row, top-p 0.99 at
// temperature 1.3: 70 against 45).
constexpr int64_t kFused = 32768;
// Rows up to one a compute unit take 1024 threads each, more of them 256, of
// which three workgroups fit a unit: 8192 values, top-p 0.9, 256 rows 24 against
// 42 us; 512 rows with top-k 50 32 against 18.
constexpr int64_t kUnits = 256;
constexpr int64_t kPartLeast = 4096;  // a workgroup's least share of a long row

}  // namespace

// Rows in flight: what a call holds of the workspace at once.
static int64_t sample_rows(int64_t R, int64_t V) { return V <= kFused ? 0 : std::min<int64_t>(R, 1024); }
size_t sample_bytes(int64_t R, int64_t V) { return sizeof(SampleRow) * (size_t)sample_rows(R, V); }

template <typename T>
static hipError_t run_sample(SampleArgs A, void* ws, hipStream_t s) {
  const int64_t step = sample_rows(A.R, A.V);
  if (step == 0) {
    for (A.r0 = 0; A.r0 < A.R; A.r0 += 1 << 21) {
      const dim3 grid((unsigned)std::min<int64_t>(A.R - A.r0, 1 << 21));
      if (A.R <= kUnits) hipLaunchKernelGGL((sample_row_kernel<T, 1024>), grid, dim3(1024), 0, s, A);
      else hipLaunchKernelGGL((sample_row_kernel<T, 256>), grid, dim3(256), 0, s, A);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  A.rows = static_cast<SampleRow*>(ws);
  for (A.r0 = 0; A.r0 < A.R; A.r0 += step) {
    const unsigned n = (unsigned)std::min(step, A.R - A.r0);
    // four workgroups a compute unit or more, where the rows are long enough; the
    // parts are powers of two.  256 x 131072 bf16, top-p 0.9: 89 us, with two workgroups
    // and parts of 8192 at least 139, with eight and 2048 93; 64 rows 47, 48 and 53
    const int64_t want = std::min<int64_t>(std::max<int64_t>(1, 1024 / n), (A.V + kPartLeast - 1) / kPartLeast);
    A.part_bits = 12;
    static_assert(kPartLeast == 1 << 12, "the least part");
    while (((int64_t)1 << A.part_bits) * want * 2 <= A.V || ((int64_t)kSampleParts << A.part_bits) < A.V) ++A.part_bits;
    A.part = (int64_t)1 << A.part_bits;
    const unsigned parts = (unsigned)((A.V + A.part - 1) / A.part);
    hipLaunchKernelGGL(sample_best_kernel<T>, dim3(parts, n), dim3(256), 0, s, A);
    hipLaunchKernelGGL(sample_bins_kernel<T>, dim3(parts, n), dim3(256), 0, s, A);
    hipLaunchKernelGGL(sample_collect_kernel<T>, dim3(parts, n), dim3(256), 0, s, A);
    hipLaunchKernelGGL(sample_finish_kernel<T>, dim3(n), dim3(1024), 0, s, A, (int)parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_sample(const SampleArgs& A, int dtype, void* ws, hipStream_t s) {
  if (dtype == 0) return run_sample<float>(A, ws, s);
  if (dtype == 1) return run_sample<__bf16>(A, ws, s);
  return run_sample<_Float16>(A, ws, s);
}

}  // namespace gmm
