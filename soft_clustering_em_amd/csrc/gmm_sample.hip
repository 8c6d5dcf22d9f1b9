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
// its distance to the maximum (1 / 64 of a temperature's unit each): one pass
// finds the maximum, one fills the bins (counts under top-k, sums of weights
// under top-p, by integer atomics in LDS), one collects the elements of the bin
// that the cut falls into and those above it; few enough, they are sorted and
// the row ends there.  Long rows run these as four launches over parts of rows,
// so that one row fills the card too, short rows (kFused) as one.
// Bound by the float64 exponential of every element under top-p, by memory else.
#include "gmm_device.h"

#include <hip/hip_runtime.h>

#include <float.h>

#include <algorithm>

namespace gmm {

namespace {

typedef unsigned long long u64;
constexpr int kBins = 2048, kSegs = 128, kList = 2048;
constexpr float kBinsPerUnit = 64.f;

// Live logits in the order of their values, from 1 up; 0 for NaN and -inf.
__device__ inline uint32_t key_of(float l) {
  if (!(l > -INFINITY)) return 0;
  l = fminf(l, FLT_MAX) + 0.f;  // -0 is 0
  const uint32_t u = __float_as_uint(l);
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ inline float logit_of(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key); }

// exp(z) for z <= 0: 2^n exp(r), |r| <= ln 2 / 2, by its series to r^13 / 13!
// (what is left out is below 2^-57), 0 below -745.
__device__ inline double exp_neg(double z) {
  z = fmax(z, -800.0);
  const double n = rint(z * 1.4426950408889634);
  const double r = fma(n, -2.3190468138462996e-17, fma(n, -0.6931471805599453, z));  // ln 2 in two parts
  double p = 1.0 / 6227020800.0;
  p = fma(p, r, 1.0 / 479001600.0);
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return ldexp(p, (int)n);
}

struct Row {
  const void* l;
  int64_t V, at;   // elements, first element
  int dtype;
  float mx;
  uint32_t first;  // the lowest index of the maximum
  double inv, S;   // 1 / temperature, 2^S
  double least;    // min-p
  float bins;      // bins a unit of logits
  __device__ double z(uint32_t key) const { return ((double)logit_of(key) - (double)mx) * inv; }
  __device__ double share(uint32_t key) const { return exp_neg(z(key)); }
  // e 2^S rounded to an integer: at most 2^52, the low bits of its sum with 2^52
  __device__ u64 fixed(double e) const {
    return (u64)__double_as_longlong(e * S + 0x1p52) - (u64)__double_as_longlong(0x1p52);
  }
  __device__ u64 weight(uint32_t key) const { return fixed(share(key)); }
  __device__ u64 weight_min_p(uint32_t key) const {
    const double e = share(key);
    return e >= least ? fixed(e) : 0;
  }
  // descending logits have ascending bins
  __device__ int bin(uint32_t key) const { return (int)fminf((mx - logit_of(key)) * bins, (float)(kBins - 1)); }
};

// f(index, key) for the live elements of [i0, i1), i0 a multiple of the piece, by `threads` threads
template <typename T, typename F>
__device__ inline void pieces(const Row& R, int64_t i0, int64_t i1, int thread, int threads, F f) {
  constexpr int E = 16 / (int)sizeof(T);
  const T* p = static_cast<const T*>(R.l) + R.at;
  for (int64_t i = i0 + (int64_t)thread * E; i < i1; i += (int64_t)threads * E) {
    T v[E];
    if (i + E <= i1) {
      __builtin_memcpy(v, p + i, 16);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = i + e < i1 ? p[i + e] : (T)-INFINITY;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t key = key_of((float)v[e]);
      if (key) f(i + e, key);
    }
  }
}
template <typename F>
__device__ inline void each(const Row& R, int64_t i0, int64_t i1, int thread, int threads, F f) {
  if (R.dtype == 0) pieces<float>(R, i0, i1, thread, threads, f);
  else if (R.dtype == 1) pieces<__bf16>(R, i0, i1, thread, threads, f);
  else pieces<_Float16>(R, i0, i1, thread, threads, f);
}

__device__ inline u64 wave_sum_u64(u64 v) {
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ inline u64 wave_max_u64(u64 v) {
  for (int o = 32; o; o >>= 1) v = max(v, (u64)__shfl_xor(v, o));
  return v;
}
__device__ inline u64 wave_scan_u64(u64 v) {  // inclusive
  const int lane = threadIdx.x & 63;
  for (int o = 1; o < 64; o <<= 1) {
    const u64 x = __shfl_up(v, o);
    if (lane >= o) v += x;
  }
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
  for (int k = 0; k < (int)(threadIdx.x >> 6); ++k) v += red[k];
  return v;
}

// What is kept: keys above `key`, and of the keys equal to it the first `ties`
// by index.  {0, 0}: every live element.
struct Cut {
  uint32_t key;
  u64 ties;
};

enum Mode { kNone, kGreedy, kOpen, kCount, kMass };
struct Settings {
  Mode mode;
  int64_t k;
  double top_p;
};

struct Cutting {
  u64 red[16], above;
  u64 list[kList];
  int at, na, nb;
};
struct Shared : Cutting {
  u64 bin[kBins], sum[kList], seg[kSegs];
  uint32_t tie[kSegs];
};

// The row's elements, and what `best` (its largest key, and ~ its lowest index)
// and the settings make of it.
__device__ inline Settings row_of(const SampleArgs& A, int64_t r, u64 best, Row& R) {
  R.l = A.l;
  R.V = A.V;
  R.dtype = A.dtype;
  const int64_t b = A.stride_b ? r / A.N : 0;
  R.at = b * A.stride_b + (r - b * A.N) * A.ld;
  R.S = A.scale;
  R.mx = best ? logit_of((uint32_t)(best >> 32)) : 0.f;
  R.first = ~(uint32_t)best;
  const double T = A.row_temperature ? (double)A.row_temperature[r] : A.temperature;
  const double min_p = A.row_min_p ? (double)A.row_min_p[r] : A.min_p;
  Settings q;
  q.k = A.row_top_k ? A.row_top_k[r] : A.top_k;
  q.top_p = A.row_top_p ? (double)A.row_top_p[r] : A.top_p;
  q.mode = !best ? kNone : !(T > 0.0) || q.k == 1 ? kGreedy : q.k > 0 && q.k < A.V ? kCount : q.top_p < 1.0 ? kMass : kOpen;
  R.inv = T > 0.0 ? 1.0 / T : 1.0;
  R.least = min_p > 0.0 ? fmin(min_p, 1.0) : 0.0;
  R.bins = (float)fmin((double)kBinsPerUnit * R.inv, (double)FLT_MAX);
  return q;
}

// a share of the row: its largest key with ~ its lowest index
__device__ inline u64 best_of(const Row& R, int64_t i0, int64_t i1, int thread, int threads) {
  uint32_t top = 0, at = 0;
  each(R, i0, i1, thread, threads, [&](int64_t i, uint32_t key) {
    if (key > top) {
      top = key;
      at = (uint32_t)i;
    }
  });
  return top ? (u64)top << 32 | (uint32_t)~at : 0;
}

__device__ inline void fill_bins(const Row& R, Mode mode, int64_t i0, int64_t i1, int thread, int threads, u64* bin) {
  if (mode == kCount)
    each(R, i0, i1, thread, threads, [&](int64_t, uint32_t key) { atomicAdd(&bin[R.bin(key)], (u64)1); });
  else
    each(R, i0, i1, thread, threads, [&](int64_t, uint32_t key) { atomicAdd(&bin[R.bin(key)], R.weight(key)); });
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
__device__ inline void collect(const Row& R, Cutting& sh, int64_t i0, int64_t i1, int thread, int threads) {
  const int at = sh.at;
  each(R, i0, i1, thread, threads, [&](int64_t i, uint32_t key) {
    const int b = R.bin(key);
    if (b > at) return;
    const u64 v = (u64)key << 32 | (uint32_t)~(uint32_t)i;
    const int slot = atomicAdd(b < at ? &sh.na : &sh.nb, 1);
    if (slot < kList / 2) sh.list[b < at ? slot : kList - 1 - slot] = v;
  });
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

__device__ inline void answer(const SampleArgs& A, const Row& R, int64_t r, uint32_t key, int64_t i, u64 total) {
  A.tokens[r] = (int32_t)i;
  if (A.logp) A.logp[r] = (float)(R.z(key) - log((double)total / R.S));
}
__device__ inline double aim(const SampleArgs& A, int64_t r, u64 total) {
  return (double)fminf(fmaxf(A.u[r], 0.f), 0x1.fffffep-1f) * (double)total;
}

// The row ends with a list of its n largest elements, among which the cut lies.
// mass: of the row (top-p without top-k).
template <int TH>
__device__ void finish_list(const SampleArgs& A, const Row& R, const Settings& q, int64_t r, Shared& sh, int n, u64 mass) {
  sort_list<TH>(sh, n);
  if (q.mode == kCount) n = (int)min((int64_t)n, q.k);
  scan_list<TH>(sh, n, [&](int i) { return R.weight((uint32_t)(sh.list[i] >> 32)); });
  // the kept ones are a prefix: count them
  const double target = q.top_p * (double)(q.mode == kCount ? sh.sum[n - 1] : mass);
  u64 mine = 0;
  for (int i = threadIdx.x; i < n; i += TH) {
    const bool in = i == 0 || ((!(q.top_p < 1.0) || (double)sh.sum[i - 1] < target) &&
                               (R.least == 0.0 || R.share((uint32_t)(sh.list[i] >> 32)) >= R.least));
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
  const double goal = aim(A, r, total);
#pragma unroll
  for (int e = 0; e < kList / TH; ++e) {
    if (e * TH >= kept) break;
    const int i = e * TH + threadIdx.x;
    const u64 mine_w = i < kept ? w[e] : 0, to = base + block_scan<TH>(mine_w, sh.red);
    if (i < kept && (double)to > goal && !((double)(to - mine_w) > goal)) {
      const uint32_t index = ~(uint32_t)(sh.list[i] >> 32);
      answer(A, R, r, key_of(x_value(R.l, R.dtype, R.at + index)), index, total);
    }
    __syncthreads();
    if (threadIdx.x == TH - 1) sh.above = to;
    __syncthreads();
    base = sh.above;
  }
}

// Segments of [i0, i1): their kept weights, and their elements equal to the cut.
template <int TH>
__device__ inline int64_t segments(const Row& R, const Cut& cut, int64_t i0, int64_t i1, Shared& sh) {
  const int E = R.dtype == 0 ? 4 : 8, lane = threadIdx.x & 63;
  const int64_t tile = 64 * E, tiles = (i1 - i0 + tile - 1) / tile, len = (tiles + kSegs - 1) / kSegs * tile;
  for (int s = threadIdx.x >> 6; s < kSegs; s += TH / 64) {
    const int64_t a = i0 + s * len, b = min(a + len, i1);
    u64 mass = 0, ties = 0;
    if (a < i1)
      each(R, a, b, lane, 64, [&](int64_t, uint32_t key) {
        if (key > cut.key) mass += R.weight_min_p(key);
        else if (key == cut.key) ++ties;
      });
    mass = wave_sum_u64(mass);
    ties = wave_sum_u64(ties);
    if (lane == 0) {
      sh.seg[s] = mass;
      sh.tie[s] = (uint32_t)ties;
    }
  }
  __syncthreads();
  return len;
}

// The token: the segment in which the sum passes the goal, then its tiles.  One wave.
__device__ inline void choose(const SampleArgs& A, const Row& R, const Cut& cut, int64_t r, int64_t i0, int64_t i1, int64_t len,
                              u64 before, u64 total, double goal, Shared& sh) {
  const int E = R.dtype == 0 ? 4 : 8, lane = threadIdx.x & 63;
  const int64_t tile = 64 * E;
  const u64 wt = cut.key ? R.weight_min_p(cut.key) : 0;
  u64 ties = 0;
  int s = 0;
  for (; s < kSegs - 1; ++s) {
    const u64 t = min((u64)sh.tie[s], cut.ties - ties), n = sh.seg[s] + t * wt;
    if ((double)(before + n) > goal) break;
    before += n;
    ties += t;
  }
  for (int64_t a = i0 + s * len, end = min(a + len, i1); a < end; a += tile) {
    const int64_t b = min(a + tile, end);
    u64 mass = 0, tied = 0;
    each(R, a, b, lane, 64, [&](int64_t, uint32_t key) {
      if (key > cut.key) mass += R.weight_min_p(key);
      else if (key == cut.key) ++tied;
    });
    const u64 tied_to = ties + wave_scan_u64(tied), tied_from = tied_to - tied;
    mass += (min(tied_to, cut.ties) - min(tied_from, cut.ties)) * wt;
    const u64 to = before + wave_scan_u64(mass);
    const u64 hit = __ballot((double)to > goal);
    if (hit) {
      if (lane == __builtin_ctzll(hit)) {
        u64 sum = to - mass, rank = tied_from;
        bool found = false;
        each(R, a + (int64_t)lane * E, min(a + (int64_t)(lane + 1) * E, b), 0, 64, [&](int64_t i, uint32_t key) {
          if (found) return;
          if (key > cut.key) sum += R.weight_min_p(key);
          else if (key == cut.key && rank++ < cut.ties) sum += wt;
          if ((double)sum > goal) {
            found = true;
            answer(A, R, r, key, i, total);
          }
        });
      }
      return;
    }
    before = __shfl(to, 63);
    ties = __shfl(tied_to, 63);
  }
}

template <int TH>
__device__ void finish_cut(const SampleArgs& A, const Row& R, const Cut& cut, int64_t r, Shared& sh) {
  __syncthreads();
  const int64_t len = segments<TH>(R, cut, 0, R.V, sh);
  if (threadIdx.x >= 64) return;
  const u64 wt = cut.key ? R.weight_min_p(cut.key) : 0;
  u64 total = 0, ties = 0;
  for (int s = 0; s < kSegs; ++s) {
    const u64 t = min((u64)sh.tie[s], cut.ties - ties);
    total += sh.seg[s] + t * wt;
    ties += t;
  }
  choose(A, R, cut, r, 0, R.V, len, 0, total, aim(A, r, total), sh);
}

// The prefix of the kept elements, by descending key, at which the count (by
// mass: the sum of the weights) first reaches `target`: bins of the keys'
// range, then of the bin that it is reached in, until one key is left.  For
// rows whose cut lies among more equal or nearly equal logits than a list holds.
template <int TH, bool MASS>
__device__ Cut reach(const Row& R, Shared& sh, Cut kept, uint32_t hi, double target) {
  uint32_t lo = kept.key ? kept.key : 1;
  u64 above = 0;
  const u64 tied = kept.key ? kept.ties * (MASS ? R.weight(kept.key) : 1) : 0;
  for (;;) {
    int shift = 0;
    while (((hi - lo) >> shift) >= kBins) ++shift;
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += TH) sh.bin[i] = 0;
    __syncthreads();
    each(R, 0, R.V, threadIdx.x, TH, [&](int64_t, uint32_t key) {
      if (key >= lo && key <= hi && key != kept.key) atomicAdd(&sh.bin[(hi - key) >> shift], MASS ? R.weight(key) : (u64)1);
    });
    __syncthreads();
    if (threadIdx.x == 0) {
      if (kept.key >= lo && kept.key <= hi && kept.key) sh.bin[(hi - kept.key) >> shift] += tied;
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
    const u64 w = MASS ? R.weight(hi) : 1, have = in / w;
    u64 ties = target > (double)above ? (u64)((target - (double)above) / (double)w) : 1;
    ties = ties < 1 ? 1 : ties > have ? have : ties;
    while (ties > 1 && (double)(above + (ties - 1) * w) >= target) --ties;
    while (ties < have && (double)(above + ties * w) < target) ++ties;
    return Cut{hi, ties};
  }
}

template <int TH>
__device__ void finish_reach(const SampleArgs& A, const Row& R, const Settings& q, int64_t r, Shared& sh) {
  const uint32_t top = key_of(R.mx);
  Cut cut{0, 0};
  if (q.mode == kCount) cut = reach<TH, false>(R, sh, cut, top, (double)q.k);
  if (q.top_p < 1.0) {
    u64 mass = 0;
    each(R, 0, R.V, threadIdx.x, TH, [&](int64_t, uint32_t key) {
      if (key > cut.key) mass += R.weight(key);
    });
    mass = block_sum<TH>(mass, sh.red) + (cut.key ? cut.ties * R.weight(cut.key) : 0);
    cut = reach<TH, true>(R, sh, cut, top, q.top_p * (double)mass);
  }
  finish_cut<TH>(A, R, cut, r, sh);
}

// The row from its bins' cut (sh.at, sh.above), the `nb` elements of that bin and
// the `na` above it, which `copy` brings into sh.list.
template <int TH, typename F>
__device__ void finish(const SampleArgs& A, const Row& R, const Settings& q, int64_t r, Shared& sh, u64 whole, int na, int nb,
                       int cap, F copy) {
  if (na <= cap && nb <= cap && na + nb <= kList) {
    copy(0, na, nb);
    __syncthreads();
    finish_list<TH>(A, R, q, r, sh, na + nb, whole);
  } else if (q.mode == kMass && nb <= min(cap, kList)) {
    // the cut inside its bin, then the row by index
    const u64 above = sh.above;
    copy(0, 0, nb);
    __syncthreads();
    sort_list<TH>(sh, nb);
    scan_list<TH>(sh, nb, [&](int i) { return R.weight((uint32_t)(sh.list[i] >> 32)); });
    const double target = q.top_p * (double)whole;
    for (int i = threadIdx.x; i < nb; i += TH)
      if ((double)(above + sh.sum[i]) >= target && (i == 0 || (double)(above + sh.sum[i - 1]) < target)) sh.at = i;
    __syncthreads();
    const int at = sh.at;
    const uint32_t key = (uint32_t)(sh.list[at] >> 32);
    u64 same = 0;
    for (int i = threadIdx.x; i <= at; i += TH) same += (uint32_t)(sh.list[i] >> 32) == key;
    finish_cut<TH>(A, R, Cut{key, block_sum<TH>(same, sh.red)}, r, sh);
  } else {
    finish_reach<TH>(A, R, q, r, sh);
  }
}

__device__ inline bool plain_answer(const SampleArgs& A, const Row& R, const Settings& q, int64_t r) {
  if (q.mode != kNone && q.mode != kGreedy) return false;
  if (threadIdx.x == 0) {
    A.tokens[r] = q.mode == kNone ? -1 : (int32_t)R.first;
    if (A.logp) A.logp[r] = q.mode == kNone ? -INFINITY : 0.f;
  }
  return true;
}

// A short row by one workgroup.
__global__ void __launch_bounds__(256) sample_row_kernel(SampleArgs A) {
  constexpr int TH = 256;
  __shared__ Shared sh;
  const int64_t r = (int64_t)blockIdx.x + A.r0;
  Row R;
  row_of(A, r, 0, R);
  const Settings q = row_of(A, r, block_max<TH>(best_of(R, 0, R.V, threadIdx.x, TH), sh.red), R);
  if (plain_answer(A, R, q, r)) return;
  if (q.mode == kOpen) {
    finish_cut<TH>(A, R, Cut{0, 0}, r, sh);
    return;
  }
  for (int i = threadIdx.x; i < kBins; i += TH) sh.bin[i] = 0;
  if (threadIdx.x == 0) sh.na = sh.nb = 0;
  __syncthreads();
  fill_bins(R, q.mode, 0, R.V, threadIdx.x, TH, sh.bin);
  __syncthreads();
  const u64 whole = cut_bin<TH>(q, sh, sh.bin);
  collect(R, sh, 0, R.V, threadIdx.x, TH);
  const int na = sh.na, nb = sh.nb;
  // from the list's two ends to its front
  finish<TH>(A, R, q, r, sh, whole, na, nb, kList / 2, [&](int to, int a, int b) {
    u64 v[kList / 2 / TH];
#pragma unroll
    for (int e = 0; e < kList / 2 / TH; ++e) {
      const int i = e * TH + threadIdx.x;
      if (i < b) v[e] = sh.list[kList - 1 - i];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kList / 2 / TH; ++e) {
      const int i = e * TH + threadIdx.x;
      if (i < b) sh.list[to + a + i] = v[e];
    }
  });
}

// Long rows: parts of a row in workgroups of their own.
__device__ inline void part_of(const SampleArgs& A, int64_t& i0, int64_t& i1) {
  i0 = (int64_t)blockIdx.x * A.part;
  i1 = min(i0 + A.part, A.V);
}
__device__ inline u64 best_part(const SampleRow& w, int parts) {
  u64 v = 0;
  for (int k = 0; k < parts; ++k) v = max(v, (u64)w.best[k]);
  return v;
}

__global__ void __launch_bounds__(256) sample_best_kernel(SampleArgs A) {
  constexpr int TH = 256;
  __shared__ u64 red[TH / 64];
  const int64_t r = (int64_t)blockIdx.y + A.r0;
  SampleRow& w = A.rows[blockIdx.y];
  Row R;
  row_of(A, r, 0, R);
  int64_t i0, i1;
  part_of(A, i0, i1);
  const u64 best = block_max<TH>(best_of(R, i0, i1, threadIdx.x, TH), red);
  if (threadIdx.x == 0) {
    w.best[blockIdx.x] = best;
    if (blockIdx.x == 0) w.na = w.nb = 0;
  }
  for (int i = blockIdx.x * TH + threadIdx.x; i < kBins; i += gridDim.x * TH) w.bin[i] = 0;
}

__global__ void __launch_bounds__(256) sample_bins_kernel(SampleArgs A) {
  constexpr int TH = 256;
  __shared__ u64 bin[kBins];
  __shared__ u64 red[TH / 64];
  const int64_t r = (int64_t)blockIdx.y + A.r0;
  SampleRow& w = A.rows[blockIdx.y];
  Row R;
  const Settings q = row_of(A, r, best_part(w, gridDim.x), R);
  if (q.mode == kNone || q.mode == kGreedy) return;
  int64_t i0, i1;
  part_of(A, i0, i1);
  if (q.mode == kOpen) {
    u64 mass = 0;
    each(R, i0, i1, threadIdx.x, TH, [&](int64_t, uint32_t key) { mass += R.weight_min_p(key); });
    mass = block_sum<TH>(mass, red);
    if (threadIdx.x == 0) w.mass[blockIdx.x] = mass;
    return;
  }
  for (int i = threadIdx.x; i < kBins; i += TH) bin[i] = 0;
  __syncthreads();
  fill_bins(R, q.mode, i0, i1, threadIdx.x, TH, bin);
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += TH)
    if (bin[i]) atomicAdd((u64*)&w.bin[i], bin[i]);
}

__global__ void __launch_bounds__(256) sample_collect_kernel(SampleArgs A) {
  constexpr int TH = 256;
  __shared__ Cutting sh;
  const int64_t r = (int64_t)blockIdx.y + A.r0;
  SampleRow& w = A.rows[blockIdx.y];
  Row R;
  const Settings q = row_of(A, r, best_part(w, gridDim.x), R);
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
  int64_t i0, i1;
  part_of(A, i0, i1);
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
}

__global__ void __launch_bounds__(1024) sample_finish_kernel(SampleArgs A, int parts) {
  constexpr int TH = 1024;
  __shared__ Shared sh;
  const int64_t r = (int64_t)blockIdx.x + A.r0;
  SampleRow& w = A.rows[blockIdx.x];
  Row R;
  const Settings q = row_of(A, r, best_part(w, parts), R);
  if (plain_answer(A, R, q, r)) return;
  if (q.mode == kOpen) {
    u64 total = 0, before = 0;
    for (int k = 0; k < parts; ++k) total += w.mass[k];
    const double goal = aim(A, r, total);
    int k = 0;
    for (; k < parts - 1 && !((double)(before + w.mass[k]) > goal); ++k) before += w.mass[k];
    const int64_t i0 = k * A.part, i1 = min(i0 + A.part, A.V), len = segments<TH>(R, Cut{0, 0}, i0, i1, sh);
    if (threadIdx.x < 64) choose(A, R, Cut{0, 0}, r, i0, i1, len, before, total, goal, sh);
    return;
  }
  if (threadIdx.x == 0) {
    sh.at = w.at;
    sh.above = w.above;
  }
  __syncthreads();
  finish<TH>(A, R, q, r, sh, w.whole, w.na, w.nb, kSampleList, [&](int to, int a, int b) {
    for (int i = threadIdx.x; i < a; i += TH) sh.list[to + i] = w.list[i];
    for (int i = threadIdx.x; i < b; i += TH) sh.list[to + a + i] = w.list[2 * kSampleList - 1 - i];
  });
}

constexpr int64_t kFused = 8192;     // longest row that one workgroup takes
constexpr int64_t kPartLeast = 4096; // a workgroup's least share of a long row

}  // namespace

// Rows in flight: what a call holds of the workspace at once.
static int64_t sample_rows(int64_t R, int64_t V) { return V <= kFused ? 0 : std::min<int64_t>(R, 1024); }
size_t sample_bytes(int64_t R, int64_t V) { return sizeof(SampleRow) * (size_t)sample_rows(R, V); }

hipError_t launch_sample(SampleArgs A, void* ws, hipStream_t s) {
  const int64_t step = sample_rows(A.R, A.V);
  if (step == 0) {
    for (A.r0 = 0; A.r0 < A.R; A.r0 += 1 << 22) {
      hipLaunchKernelGGL(sample_row_kernel, dim3((unsigned)std::min<int64_t>(A.R - A.r0, 1 << 22)), dim3(256), 0, s, A);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  A.rows = static_cast<SampleRow*>(ws);
  for (A.r0 = 0; A.r0 < A.R; A.r0 += step) {
    const unsigned n = (unsigned)std::min(step, A.R - A.r0);
    // about four workgroups a compute unit, of whole pieces
    const int64_t want = std::min<int64_t>(std::max<int64_t>(1, 1024 / n), (A.V + kPartLeast - 1) / kPartLeast);
    const int64_t most = std::min<int64_t>(want, kSampleParts);
    A.part = ((A.V + most - 1) / most + 7) / 8 * 8;
    const unsigned parts = (unsigned)((A.V + A.part - 1) / A.part);
    hipLaunchKernelGGL(sample_best_kernel, dim3(parts, n), dim3(256), 0, s, A);
    hipLaunchKernelGGL(sample_bins_kernel, dim3(parts, n), dim3(256), 0, s, A);
    hipLaunchKernelGGL(sample_collect_kernel, dim3(parts, n), dim3(256), 0, s, A);
    hipLaunchKernelGGL(sample_finish_kernel, dim3(n), dim3(1024), 0, s, A, (int)parts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace gmm
