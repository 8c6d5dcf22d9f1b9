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
#include "gmm_device.h"

#include <hip/hip_runtime.h>

#include <float.h>

#include <algorithm>

namespace gmm {

namespace {

typedef unsigned long long u64;
constexpr int kThreads = 1024, kWaves = kThreads / 64, kBins = 2048, kSegs = 128;

// Live logits in the order of their values, from 1 up; 0 for NaN and -inf.
__device__ inline uint32_t key_of(float l) {
  if (!(l > -INFINITY)) return 0;
  l = fminf(l, FLT_MAX) + 0.f;  // -0 is 0
  const uint32_t u = __float_as_uint(l);
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ inline float logit_of(uint32_t key) { return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key); }

struct Row {
  const void* l;
  int64_t V, at;   // elements, first element
  int dtype;
  float mx;
  double T, S;     // temperature, 2^S
  __device__ u64 weight(uint32_t key) const { return (u64)__double2ll_rn(exp(((double)logit_of(key) - (double)mx) / T) * S); }
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
__device__ inline u64 wave_scan_u64(u64 v) {  // inclusive
  const int lane = threadIdx.x & 63;
  for (int o = 1; o < 64; o <<= 1) {
    const u64 x = __shfl_up(v, o);
    if (lane >= o) v += x;
  }
  return v;
}
__device__ inline u64 block_sum(u64 v, u64* red) {
  v = wave_sum_u64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
  for (int k = 0; k < kWaves; ++k) v += red[k];
  return v;
}
__device__ inline uint32_t block_max(uint32_t v, u64* red) {
  for (int o = 32; o; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
  for (int k = 0; k < kWaves; ++k) v = max(v, (uint32_t)red[k]);
  return v;
}

// What is kept: keys above `key`, and of the keys equal to it the first `ties`
// by index.  {0, 0}: every live element.
struct Cut {
  uint32_t key;
  u64 ties;
};

struct Shared {
  u64 bin[kBins];
  u64 red[kWaves], seg[kSegs];
  uint32_t tie[kSegs];
  u64 above, ties;
  int at;
};

// The prefix of the kept elements, by descending key, at which the count (by
// mass: the sum of the weights) first reaches `target`: bins of the keys'
// range, then of the bin that it is reached in, until one key is left.
template <bool MASS>
__device__ Cut reach(const Row& R, Shared& sh, Cut kept, uint32_t hi, double target) {
  uint32_t lo = kept.key ? kept.key : 1;
  u64 above = 0;
  const u64 tied = kept.key ? kept.ties * (MASS ? R.weight(kept.key) : 1) : 0;
  for (;;) {
    int shift = 0;
    while (((hi - lo) >> shift) >= kBins) ++shift;
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.bin[i] = 0;
    __syncthreads();
    each(R, 0, R.V, threadIdx.x, kThreads, [&](int64_t, uint32_t key) {
      if (key >= lo && key <= hi && key != kept.key) atomicAdd(&sh.bin[(hi - key) >> shift], MASS ? R.weight(key) : (u64)1);
    });
    __syncthreads();
    if (threadIdx.x == 0 && kept.key >= lo && kept.key <= hi && kept.key) sh.bin[(hi - kept.key) >> shift] += tied;
    __syncthreads();
    // two bins a thread, scanned over the workgroup
    const u64 a = sh.bin[2 * threadIdx.x], b = sh.bin[2 * threadIdx.x + 1];
    const u64 in = wave_scan_u64(a + b);
    if ((threadIdx.x & 63) == 63) sh.red[threadIdx.x >> 6] = in;
    if (threadIdx.x == 0) sh.at = -1;
    __syncthreads();
    u64 before = above + in - (a + b);
    for (int k = 0; k < (int)(threadIdx.x >> 6); ++k) before += sh.red[k];
    auto crosses = [&](u64 from, u64 n, bool first) {
      return n && (double)(from + n) >= target && ((double)from < target || (first && from == 0));
    };
    if (crosses(before, a, true)) {
      sh.at = 2 * threadIdx.x;
      sh.above = before;
    } else if (crosses(before + a, b, true)) {
      sh.at = 2 * threadIdx.x + 1;
      sh.above = before + a;
    }
    __syncthreads();
    const int at = sh.at;
    above = sh.above;
    const u64 n = at >= 0 ? sh.bin[at] : 0;
    __syncthreads();
    if (at < 0) return kept;
    hi -= (uint32_t)at << shift;
    const uint32_t last = hi - (((uint32_t)1 << shift) - 1);
    lo = last > lo && last <= hi ? last : lo;
    if (shift != 0) continue;
    const u64 w = MASS ? R.weight(hi) : 1, have = n / w;
    u64 ties = target > (double)above ? (u64)((target - (double)above) / (double)w) : 1;
    ties = ties < 1 ? 1 : ties > have ? have : ties;
    while (ties > 1 && (double)(above + (ties - 1) * w) >= target) --ties;
    while (ties < have && (double)(above + ties * w) < target) ++ties;
    return Cut{hi, ties};
  }
}

__global__ void __launch_bounds__(kThreads) sample_kernel(SampleArgs A) {
  __shared__ Shared sh;
  const int64_t r = blockIdx.x;
  Row R;
  R.l = A.l;
  R.V = A.V;
  R.dtype = A.dtype;
  const int64_t b = A.stride_b ? r / A.N : 0;
  R.at = b * A.stride_b + (r - b * A.N) * A.ld;
  R.S = A.scale;
  const double T = A.row_temperature ? (double)A.row_temperature[r] : A.temperature;
  const int64_t k = A.row_top_k ? A.row_top_k[r] : A.top_k;
  const double top_p = A.row_top_p ? (double)A.row_top_p[r] : A.top_p, min_p = A.row_min_p ? (double)A.row_min_p[r] : A.min_p;
  uint32_t top = 0;
  u64 live = 0;
  each(R, 0, R.V, threadIdx.x, kThreads, [&](int64_t, uint32_t key) {
    top = max(top, key);
    ++live;
  });
  top = block_max(top, sh.red);
  live = block_sum(live, sh.red);
  if (top == 0) {
    if (threadIdx.x == 0) {
      A.tokens[r] = -1;
      if (A.logp) A.logp[r] = -INFINITY;
    }
    return;
  }
  const bool greedy = !(T > 0.0);
  R.mx = logit_of(top);
  R.T = greedy ? 1.0 : T;
  Cut cut{0, 0};
  if (greedy) cut = Cut{top, 1};
  else if (k > 0 && k < (int64_t)live) cut = reach<false>(R, sh, cut, top, (double)k);
  if (!greedy && top_p < 1.0) {
    u64 mass = 0;
    each(R, 0, R.V, threadIdx.x, kThreads, [&](int64_t, uint32_t key) {
      if (key > cut.key) mass += R.weight(key);
    });
    mass = block_sum(mass, sh.red) + (cut.key ? cut.ties * R.weight(cut.key) : 0);
    cut = reach<true>(R, sh, cut, top, top_p * (double)mass);
  }
  // segments of whole waves' pieces, their kept weights and ties
  const int E = A.dtype == 0 ? 4 : 8;
  const int64_t tile = 64 * E, tiles = (R.V + tile - 1) / tile, len = (tiles + kSegs - 1) / kSegs * tile;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const double least = greedy || !(min_p > 0.0) ? 0.0 : fmin(min_p, 1.0);
  const auto weight = [&](uint32_t key) -> u64 {
    const double e = exp(((double)logit_of(key) - (double)R.mx) / R.T);
    return e >= least ? (u64)__double2ll_rn(e * R.S) : 0;
  };
  const u64 wt = cut.key ? weight(cut.key) : 0;
  for (int s = w; s < kSegs; s += kWaves) {
    const int64_t i0 = s * len, i1 = std::min(i0 + len, R.V);
    u64 mass = 0, ties = 0;
    if (i0 < R.V)
      each(R, i0, i1, lane, 64, [&](int64_t, uint32_t key) {
        if (key > cut.key) mass += weight(key);
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
  if (w != 0) return;
  u64 total = 0, ties = 0;
  for (int s = 0; s < kSegs; ++s) {
    const u64 t = std::min<u64>(sh.tie[s], cut.ties - ties);
    total += sh.seg[s] + t * wt;
    ties += t;
  }
  const float u = fminf(fmaxf(A.u[r], 0.f), 0x1.fffffep-1f);
  const double target = (double)u * (double)total;
  u64 before = 0;
  ties = 0;
  int s = 0;
  for (; s < kSegs - 1; ++s) {
    const u64 t = std::min<u64>(sh.tie[s], cut.ties - ties), n = sh.seg[s] + t * wt;
    if ((double)(before + n) > target) break;
    before += n;
    ties += t;
  }
  for (int64_t i0 = s * len, end = std::min(i0 + len, R.V); i0 < end; i0 += tile) {
    const int64_t i1 = std::min(i0 + tile, end);
    u64 mass = 0, tied = 0;
    each(R, i0, i1, lane, 64, [&](int64_t, uint32_t key) {
      if (key > cut.key) mass += weight(key);
      else if (key == cut.key) ++tied;
    });
    const u64 tied_to = ties + wave_scan_u64(tied), tied_from = tied_to - tied;
    const u64 counted = std::min(tied_to, cut.ties) - std::min(tied_from, cut.ties);
    mass += counted * wt;
    const u64 to = before + wave_scan_u64(mass);
    const u64 hit = __ballot((double)to > target);
    if (hit) {
      if (lane == __builtin_ctzll(hit)) {
        u64 sum = to - mass, rank = tied_from;
        bool found = false;
        each(R, i0 + (int64_t)lane * E, std::min(i0 + (int64_t)(lane + 1) * E, i1), 0, 64, [&](int64_t i, uint32_t key) {
          if (found) return;
          if (key > cut.key) sum += weight(key);
          else if (key == cut.key && rank++ < cut.ties) sum += wt;
          if ((double)sum > target) {
            found = true;
            A.tokens[r] = (int32_t)i;
            if (A.logp)
              A.logp[r] = (float)(((double)logit_of(key) - (double)R.mx) / R.T - log((double)total / R.S));
          }
        });
      }
      return;
    }
    before = __shfl(to, 63);
    ties = __shfl(tied_to, 63);
  }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& A, hipStream_t s) {
  hipLaunchKernelGGL(sample_kernel, dim3((unsigned)A.R), dim3(kThreads), 0, s, A);
  return hipGetLastError();
}

}  // namespace gmm
