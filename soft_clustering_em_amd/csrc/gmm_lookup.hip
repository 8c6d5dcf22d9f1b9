// gmm_lookup.hip -- rows rebuilt from codes (a codebook or embedding lookup
// with weights and a scale), and the gradients of that lookup.
//
// What it computes.  Row i of a problem has up to m codes idx_i0 .. idx_i,m-1
// (its leading values in [0, K); the first value outside ends the row) with
// weights w_ij (1 where none are given), as the multi-assignment writes them:
//   out_i = s sum_j w_ij T[idx_ij]
//   dT_k  = s sum over the entries (i, j) with idx_ij = k of w_ij dout_i
//   dw_ij = s <dout_i, T[idx_ij]>
// Sums are float32, rounded once to the rows' type.
//
// How.
//   lookup   a thread per 16 bytes of a row; the row's codes are read by every
//            thread of the row (one address, the L1 serves it).
//   dw       a group of up to 64 lanes per row, the dot products over it.
//   dT       deterministic, no global atomics: the entries are sorted by code
//            (up to 8192 entries by ranks in one launch; above by a stable
//            radix sort of at most 10 bits a pass, three launches each: block
//            histograms, their prefixes, ranks by ballot; entries that take no
//            part go along under a key past every code's), then summed
//            in that order in chunks of entries.  A run of one code inside a
//            chunk is written at once; a run that crosses a chunk's ends leaves
//            partial sums, which a last kernel joins, so that a code with most
//            of the entries is summed by as many workgroups as many codes are.
// Bound by memory: every dout row is read once per entry, every dT row
// written once.  1M x 128, 4 codes a row of 4096, float32: lookup 114 us (4.8
// TB/s).  262144 x 128, 4 codes of 4096, float32: dw 54 us, sort 57, sums 65
// (8.3 TB/s out of the caches), joins 13.  32768 x 2048 into 65536 codes, bf16:
// sort and zeros 64 us, sums 61 (rows in random order), joins 11.
#include "gmm_internal.h"

#include <hip/hip_runtime.h>

#include <algorithm>

namespace gmm {

namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes at any alignment of their element
template <typename T>
struct Vec {
  static constexpr int E = 16 / (int)sizeof(T);
  float v[E];
  __device__ void load(const T* p, int n) {  // n: elements that exist (E or more: all)
    if (n >= E) {
      T t[E];
      __builtin_memcpy(t, p, 16);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = (float)t[e];
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = e < n ? (float)p[e] : 0.f;
    }
  }
  // rows that nobody reads back soon pass by the caches where they are aligned
  __device__ void store(T* p, int n, bool stream = false) const {
    if (n >= E) {
      T t[E];
#pragma unroll
      for (int e = 0; e < E; ++e) t[e] = (T)v[e];
      if (stream) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, t), reinterpret_cast<u32x4*>(p));
      else __builtin_memcpy(p, t, 16);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e < n) p[e] = (T)v[e];
    }
  }
};

// lanes per row: a power of two, 2^lg
struct RowSplit {
  int lg, slabs;
};

template <typename T>
__device__ inline void lookup_row(const LookupArgs& A, int64_t row, int64_t d, int n) {
  constexpr int E = Vec<T>::E;
  const int64_t b = A.B == 1 ? 0 : row / A.N;
  const T* t = reinterpret_cast<const T*>(A.table) + b * A.stride_b + d;
  const int32_t* ix = A.idx + row * A.m;
  const float* w = A.weights ? A.weights + row * A.m : nullptr;
  Vec<T> acc;
#pragma unroll
  for (int e = 0; e < E; ++e) acc.v[e] = 0.f;
  constexpr int U = 4;  // rows of the table in flight
  for (int j0 = 0; j0 < A.m; j0 += U) {
    int k[U];
    float wj[U];
    bool live = true;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u] = j0 + u < A.m ? ix[j0 + u] : -1;
      live = live && k[u] >= 0 && k[u] < A.K;
      if (!live) k[u] = -1;
      wj[u] = w && j0 + u < A.m ? w[j0 + u] : 1.f;
    }
    Vec<T> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k[u] >= 0) r[u].load(t + k[u] * A.ld, n);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k[u] >= 0)
#pragma unroll
        for (int e = 0; e < E; ++e) acc.v[e] = fmaf(wj[u], r[u].v[e], acc.v[e]);
    if (!live) break;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) acc.v[e] *= A.scale;
  acc.store(reinterpret_cast<T*>(A.out) + row * A.D + d, n, A.stream);
}

template <typename T>
__global__ void __launch_bounds__(256) lookup_kernel(LookupArgs A, RowSplit S) {
  constexpr int E = Vec<T>::E;
  const int64_t d = ((int64_t)blockIdx.y << S.lg | (threadIdx.x & ((1 << S.lg) - 1))) * E;
  if (d >= A.D) return;
  const int n = (int)min((int64_t)E, A.D - d);
  for (int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> S.lg; row < A.B * A.N;  // over all problems
       row += (int64_t)gridDim.x * 256 >> S.lg)
    lookup_row<T>(A, row, d, n);
}

template <typename T>
__global__ void __launch_bounds__(256) dweights_kernel(LookupArgs A, int lg) {
  constexpr int E = Vec<T>::E;
  const int lane = threadIdx.x & ((1 << lg) - 1);
  for (int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> lg; row < A.B * A.N;  // whole groups of lanes
       row += (int64_t)gridDim.x * 256 >> lg) {
    const int64_t b = A.B == 1 ? 0 : row / A.N, i = row - b * A.N;
    const T* t = reinterpret_cast<const T*>(A.table) + b * A.stride_b;
    const T* g = reinterpret_cast<const T*>(A.dout) + b * A.stride_g + i * A.ld_g;
    const int32_t* ix = A.idx + row * A.m;
    float* out = A.dweights + row * A.m;
    bool live = true;
    constexpr int U = 4;  // codes at a time: their loads and their sums overlap
    for (int j0 = 0; j0 < A.m; j0 += U) {
      int k[U];
      float s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) k[u] = ix[min(j0 + u, A.m - 1)];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        live = live && j0 + u < A.m && k[u] >= 0 && k[u] < A.K;
        k[u] = live ? k[u] : -1;
        s[u] = 0.f;
      }
      for (int64_t d = (int64_t)lane * E; d < A.D; d += (int64_t)E << lg) {
        const int n = (int)min((int64_t)E, A.D - d);
        Vec<T> a, r[U];
        a.load(g + d, n);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (k[u] >= 0) r[u].load(t + k[u] * A.ld + d, n);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (k[u] >= 0)
#pragma unroll
            for (int e = 0; e < E; ++e) s[u] = fmaf(a.v[e], r[u].v[e], s[u]);
      }
      for (int o = 1; o < 1 << lg; o <<= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] += __shfl_xor(s[u], o);
      if (lane == 0)
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (j0 + u < A.m) out[j0 + u] = k[u] >= 0 ? A.scale * s[u] : 0.f;
    }
  }
}

// ---- entries sorted by code.  An entry is e = row * m + slot over all
// problems, its key b * K + code; entries that take no part get key B K.
__device__ inline uint32_t key_of(const LookupArgs& A, int64_t e, uint32_t none) {
  const int64_t row = e / A.m;
  const int j = (int)(e - row * A.m);
  const int32_t* ix = A.idx + row * A.m;
  int k = 0;
  if (A.len) {
    if (j >= A.len[row]) return none;
    return (uint32_t)((A.B == 1 ? 0 : row / A.N) * A.K + ix[j]);
  }
  for (int q = 0; q <= j; ++q) {
    k = ix[q];
    if (k < 0 || k >= A.K) return none;
  }
  return (uint32_t)((A.B == 1 ? 0 : row / A.N) * A.K + k);
}

// Rows of more than kScanCodes codes: their lengths, 16 lanes a row, so that an
// entry does not look at every code before it.
constexpr int kScanCodes = 16;
__global__ void __launch_bounds__(256) length_kernel(LookupArgs A, int32_t* len) {
  const int l = threadIdx.x & 15;
  for (int64_t row = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); row < A.B * A.N; row += (int64_t)gridDim.x * 16) {
    const int32_t* ix = A.idx + row * A.m;
    int n = A.m;
    for (int j0 = 0; j0 < n; j0 += 16) {
      int at = A.m;  // the first code outside among these 16
      if (j0 + l < A.m) {
        const int k = ix[j0 + l];
        if (k < 0 || k >= A.K) at = j0 + l;
      }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) at = min(at, __shfl_xor(at, o));
      n = min(n, at);
    }
    if (l == 0) len[row] = n;
  }
}

// any bytes <- 0 (a kernel: memory operations in a captured graph are avoided)
__global__ void __launch_bounds__(256) zero_kernel(char* p, int64_t bytes) {
  const int64_t n = bytes / 16;
  const u32x4 z = {0u, 0u, 0u, 0u};
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n; t += (int64_t)gridDim.x * 256)
    __builtin_memcpy(p + t * 16, &z, 16);
  if (blockIdx.x == 0 && threadIdx.x < bytes % 16) p[n * 16 + threadIdx.x] = 0;
}

// The sort's kernels wait for latencies on a few workgroups; the workgroups
// past theirs clear a share of dT meanwhile.
__device__ inline bool cleared(const SortPass& P, unsigned own) {
  if (blockIdx.x < own) return false;
  const u32x4 z = {0u, 0u, 0u, 0u};
  const int64_t n = P.zbytes / 16, step = (int64_t)(gridDim.x - own) * 256;
  for (int64_t t = (int64_t)(blockIdx.x - own) * 256 + threadIdx.x; t < n; t += step) __builtin_memcpy(P.zero + t * 16, &z, 16);
  if (blockIdx.x == own && threadIdx.x < P.zbytes % 16) P.zero[n * 16 + threadIdx.x] = 0;
  return true;
}

// The whole sort of up to kRankEntries entries in one kernel: an entry's place
// is the number of smaller keys and of equal ones before it, counted by 8 lanes
// over every key in LDS.
__global__ void __launch_bounds__(256) sort_rank_kernel(LookupArgs A, SortPass P) {
  if (cleared(P, (unsigned)P.nblk)) return;
  __shared__ __attribute__((aligned(16))) uint32_t keys[kRankEntries];
  const int S = (int)P.S, S4 = (S + 3) / 4;
  for (int e = threadIdx.x; e < 4 * S4; e += 256) keys[e] = e < S ? key_of(A, e, P.none) : 0xffffffffu;
  __syncthreads();
  const int e = blockIdx.x * 32 + (threadIdx.x >> 3), p = threadIdx.x & 7;
  const uint32_t mine = keys[min(e, S - 1)];
  uint32_t place = 0;
  for (int c = p; c < S4; c += 8) {
    const u32x4 k = *reinterpret_cast<const u32x4*>(keys + 4 * c);
#pragma unroll
    for (int u = 0; u < 4; ++u) place += k[u] < mine + (4 * c + u < e ? 1u : 0u);
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) place += __shfl_xor(place, o);
  if (p == 0 && e < S) {
    P.kout[place] = mine;
    P.sout[place] = (uint32_t)e;
  }
}

// digit counts of a block of 256 PER entries
template <int PER>
__global__ void __launch_bounds__(256) sort_count_kernel(LookupArgs A, SortPass P) {
  if (cleared(P, (unsigned)P.nblk)) return;
  extern __shared__ uint32_t cnt[];
  const int64_t e0 = (int64_t)blockIdx.x * (256 * PER) + threadIdx.x;
  uint32_t key[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int64_t e = e0 + u * 256;
    key[u] = e < P.S ? (P.kin ? P.kin[e] : key_of(A, e, P.none)) : 0;
  }
  for (int d = threadIdx.x; d < P.bins; d += 256) cnt[d] = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PER; ++u)
    if (e0 + u * 256 < P.S) atomicAdd(&cnt[(key[u] >> P.shift) & (P.bins - 1)], 1u);  // in LDS; a count has no order
  __syncthreads();
  for (int d = threadIdx.x; d < P.bins; d += 256) P.hist[(int64_t)blockIdx.x * P.bins + d] = cnt[d];
}

// counts [block][digit] -> the digit's entries in earlier blocks, and their
// total; 16 digits a workgroup, 16 threads a digit
__global__ void __launch_bounds__(256) sort_scan_kernel(SortPass P) {
  if (cleared(P, (P.bins + 15) / 16)) return;
  __shared__ uint32_t tot[16][16];
  const int c = threadIdx.x & 15, sl = threadIdx.x >> 4, d = blockIdx.x * 16 + c;
  const int64_t per = (P.nblk + 15) / 16, b0 = min(P.nblk, sl * per), b1 = min(P.nblk, b0 + per);
  uint32_t s = 0;
  if (d < P.bins)
#pragma unroll 8
    for (int64_t b = b0; b < b1; ++b) s += P.hist[b * P.bins + d];
  tot[sl][c] = s;
  __syncthreads();
  s = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) s += k < sl ? tot[k][c] : 0;
  if (d >= P.bins) return;
  constexpr int U = 8;
  for (int64_t b = b0; b < b1; b += U) {
    uint32_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = b + u < b1 ? P.hist[(b + u) * P.bins + d] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (b + u < b1) {
        P.hist[(b + u) * P.bins + d] = s;
        s += v[u];
      }
  }
  if (sl == 15) P.base[d] = s;
}

// places a block's entries; equal digits keep their order
template <int PER>
__global__ void __launch_bounds__(256) sort_scatter_kernel(LookupArgs A, SortPass P) {
  if (cleared(P, (unsigned)P.nblk)) return;
  extern __shared__ uint32_t next[];  // [4 waves][bins]: the wave's next position of a digit
  __shared__ uint32_t part[256];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int64_t e0 = ((int64_t)blockIdx.x * 4 + wv) * (64 * PER);  // consecutive entries of a wave
  uint32_t key[PER], src[PER];
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int64_t e = e0 + u * 64 + lane;
    key[u] = e < P.S ? (P.kin ? P.kin[e] : key_of(A, e, P.none)) : 0;
    src[u] = e < P.S ? (P.sin ? P.sin[e] : (uint32_t)e) : 0;
  }
  // the digits' totals -> where each digit's entries begin
  uint32_t sum = 0;
  const int dper = (P.bins + 255) / 256, d0 = threadIdx.x * dper;
  for (int d = d0; d < min(P.bins, d0 + dper); ++d) sum += P.base[d];
  part[threadIdx.x] = sum;
  for (int d = threadIdx.x; d < 4 * P.bins; d += 256) next[d] = 0;
  __syncthreads();
  for (int o = 1; o < 256; o <<= 1) {
    const uint32_t v = (int)threadIdx.x >= o ? part[threadIdx.x - o] : 0;
    __syncthreads();
    part[threadIdx.x] += v;
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < PER; ++u)
    if (e0 + u * 64 + lane < P.S) atomicAdd(&next[wv * P.bins + ((key[u] >> P.shift) & (P.bins - 1))], 1u);
  __syncthreads();
  uint32_t first = part[threadIdx.x] - sum;
  for (int d = d0; d < min(P.bins, d0 + dper); ++d) {
    uint32_t at = first + P.hist[(int64_t)blockIdx.x * P.bins + d];
    first += P.base[d];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t c = next[w * P.bins + d];
      next[w * P.bins + d] = at;
      at += c;
    }
  }
  __syncthreads();
  volatile uint32_t* mine = next + wv * P.bins;
  const uint64_t below = lane == 0 ? 0ull : ~0ull >> (64 - lane);
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const bool in = e0 + u * 64 + lane < P.S;
    const uint32_t d = (key[u] >> P.shift) & (P.bins - 1);
    uint64_t same = __builtin_amdgcn_ballot_w64(in);
    for (int bit = 0; bit < P.bits; ++bit) {
      const uint64_t set = __builtin_amdgcn_ballot_w64((d >> bit) & 1);
      same &= (d >> bit) & 1 ? set : ~set;
    }
    if (in) {
      const uint32_t at = mine[d] + __builtin_popcountll(same & below);
      P.kout[at] = key[u];
      P.sout[at] = src[u];
    }
    __builtin_amdgcn_wave_barrier();  // every lane has read its digit's position
    if (in && (same >> lane) == 1ull) mine[d] += __builtin_popcountll(same);  // the digit's last lane
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename T>
__device__ inline void put(const LookupArgs& A, uint32_t key, int64_t d, int n, Vec<T>& acc) {
  T* p = reinterpret_cast<T*>(A.dtable) + (int64_t)key * A.D + d;
#pragma unroll
  for (int e = 0; e < Vec<T>::E; ++e) acc.v[e] *= A.scale;
  if (A.accumulate) {
    Vec<T> old;
    old.load(p, n);
#pragma unroll
    for (int e = 0; e < Vec<T>::E; ++e) acc.v[e] += old.v[e];
  }
  acc.store(p, n);
}

// Sums the entries of a chunk, in sorted order; a group of 2^lg lanes holds
// 16 bytes of columns a lane.  The rows of the next U entries are on their way
// while the U before them are added.
template <typename T>
__global__ void __launch_bounds__(256) sum_kernel(LookupArgs A, SumArgs P, RowSplit S) {
  constexpr int E = Vec<T>::E, U = 4;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> S.lg;
  const int64_t d = ((int64_t)blockIdx.y << S.lg | (threadIdx.x & ((1 << S.lg) - 1))) * E;
  if (c >= P.chunks || d >= A.D) return;
  const int n = (int)min((int64_t)E, A.D - d);
  const int64_t s0 = c * P.C, s1 = min(P.S, s0 + P.C);
  const uint32_t before = s0 > 0 ? P.key[s0 - 1] : 0xffffffffu, after = s1 < P.S ? P.key[s1] : 0xffffffffu;
  Vec<T> acc;
#pragma unroll
  for (int e = 0; e < E; ++e) acc.v[e] = 0.f;
  uint32_t cur = P.key[s0];
  if (cur >= P.none) return;  // entries behind the last code
  bool first = true;  // the run reaches the chunk's start
  auto partial = [&](int slot) {
    float* p = P.part + ((c * 2 + slot) * P.Dp + d);
#pragma unroll
    for (int e = 0; e < E; ++e) p[e] = acc.v[e];  // Dp: D rounded up to whole chunks
  };
  struct Batch {
    uint32_t k[U];
    float w[U];
    Vec<T> r[U];
  };
  const bool whole = n == E;
  auto load = [&](int64_t s, Batch& t) {
    uint32_t e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = s + u < s1;
      t.k[u] = in ? P.key[s + u] : P.none;
      e[u] = in ? P.src[s + u] : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t.k[u] >= P.none) e[u] = 0;  // entry 0 always exists
      const int64_t row = A.m == 1 ? e[u] : e[u] / (uint32_t)A.m;
      const int64_t b = A.B == 1 ? 0 : row / A.N;
      t.w[u] = A.weights ? A.weights[e[u]] : 1.f;
      const T* p = reinterpret_cast<const T*>(A.dout) + b * A.stride_g + (row - b * A.N) * A.ld_g + d;
      if (whole) t.r[u].load(p, E);
      else t.r[u].load(p, n);
    }
  };
  auto add = [&](const Batch& t) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t.k[u] >= P.none) continue;
      if (t.k[u] != cur) {
        if (first && before == cur) partial(0);
        else put<T>(A, cur, d, n, acc);
        first = false;
        cur = t.k[u];
#pragma unroll
        for (int e = 0; e < E; ++e) acc.v[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) acc.v[e] = fmaf(t.w[u], t.r[u].v[e], acc.v[e]);
    }
  };
  Batch x, y;
  load(s0, x);
  for (int64_t s = s0; s < s1; s += 2 * U) {
    load(s + U, y);
    add(x);
    load(s + 2 * U, x);
    add(y);
  }
  if (first && before == cur) partial(0);
  else if (after == cur) partial(1);
  else put<T>(A, cur, d, n, acc);
}

// Joins the runs that cross chunks: the workgroup of the chunk where such a
// run starts adds its tail and the heads of the chunks that it goes on into,
// 8 groups of 32 lanes over the chunks, 16 bytes of float32 columns a lane.
template <typename T>
__global__ void __launch_bounds__(256) join_runs_kernel(LookupArgs A, SumArgs P) {
  __shared__ float4 red[8][32];
  const int64_t c = blockIdx.x;
  const int64_t s1 = (c + 1) * P.C;
  if (s1 >= P.S) return;
  const uint32_t key = P.key[s1 - 1];
  if (key >= P.none || P.key[s1] != key) return;                                 // no run crosses this end
  if (c > 0 && P.key[c * P.C] == key && P.key[c * P.C - 1] == key) return;       // it started earlier
  // the last chunk whose first entry has the key
  int64_t lo = c + 1, hi = P.chunks - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) / 2;
    if (P.key[mid * P.C] == key) lo = mid;
    else hi = mid - 1;
  }
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  for (int64_t d0 = (int64_t)blockIdx.y * 128; d0 < A.D; d0 += (int64_t)gridDim.y * 128) {
    const int64_t d = d0 + 4 * lane;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (d < A.D) {
      if (g == 0) a = *reinterpret_cast<const float4*>(P.part + (c * 2 + 1) * P.Dp + d);
#pragma unroll 4
      for (int64_t q = c + 1 + g; q <= lo; q += 8) {
        const float4 v = *reinterpret_cast<const float4*>(P.part + q * 2 * P.Dp + d);
        a.x += v.x;
        a.y += v.y;
        a.z += v.z;
        a.w += v.w;
      }
    }
    __syncthreads();
    red[g][lane] = a;
    __syncthreads();
    if (g != 0 || d >= A.D) continue;
    for (int q = 1; q < 8; ++q) {
      const float4 v = red[q][lane];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    const float v[4] = {a.x, a.y, a.z, a.w};
    T* p = reinterpret_cast<T*>(A.dtable) + (int64_t)key * A.D + d;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (d + e < A.D) p[e] = (T)(A.scale * v[e] + (A.accumulate ? (float)p[e] : 0.f));
  }
}

constexpr int64_t kLookupGrid = 8192;
constexpr int64_t kMaxGrid = 1 << 22;  // workgroups along x: a launch has fewer than 2^32 threads an axis

RowSplit row_split(int64_t D, int E) {
  const int64_t ch = (D + E - 1) / E;
  RowSplit s{0, 1};
  while (s.lg < 8 && (1 << s.lg) < ch) ++s.lg;
  s.slabs = (int)((ch + (1 << s.lg) - 1) >> s.lg);
  return s;
}

#define GMM_TRY(call)             \
  do {                            \
    const hipError_t e_ = (call); \
    if (e_ != hipSuccess) return e_; \
  } while (0)

template <typename T>
hipError_t lookup(LookupArgs a, hipStream_t s) {
  a.stream = ((uintptr_t)a.out | (uintptr_t)(a.D * (int64_t)sizeof(T))) % 16 == 0;
  const RowSplit sp = row_split(a.D, Vec<T>::E);
  const int64_t rows = a.B * a.N, per = 256 >> sp.lg;
  const dim3 grid((unsigned)std::min<int64_t>((rows + per - 1) / per, kLookupGrid), (unsigned)sp.slabs);
  hipLaunchKernelGGL((lookup_kernel<T>), grid, dim3(256), 0, s, a, sp);
  return hipGetLastError();
}

template <typename T>
hipError_t lookup_grad(LookupArgs a, const LookupPlan& p, char* ws, hipStream_t s) {
  const int64_t rows = a.B * a.N;
  if (a.dweights && rows > 0) {
    int lg = row_split(a.D, Vec<T>::E).lg;
    lg = std::min(lg, 6);
    const int64_t per = 256 >> lg;
    hipLaunchKernelGGL((dweights_kernel<T>), dim3((unsigned)std::min<int64_t>((rows + per - 1) / per, kMaxGrid)), dim3(256), 0, s, a,
                       lg);
    GMM_TRY(hipGetLastError());
  }
  if (!a.dtable) return hipSuccess;
  const int64_t bytes = a.accumulate ? 0 : a.B * a.K * a.D * (int64_t)sizeof(T);
  if (rows == 0) return launch_zero(a.dtable, bytes, s);
  if (p.lengths) {
    int32_t* len = reinterpret_cast<int32_t*>(ws + p.off_len);
    hipLaunchKernelGGL(length_kernel, dim3((unsigned)std::min<int64_t>((rows + 15) / 16, kLookupGrid)), dim3(256), 0, s, a, len);
    GMM_TRY(hipGetLastError());
    a.len = len;
  }
  uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(ws + p.off_key[0]), reinterpret_cast<uint32_t*>(ws + p.off_key[1])};
  uint32_t* srcs[2] = {reinterpret_cast<uint32_t*>(ws + p.off_src[0]), reinterpret_cast<uint32_t*>(ws + p.off_src[1])};
  SortPass P{};
  P.S = p.S;
  P.nblk = p.nblk;
  P.none = p.none;
  P.hist = reinterpret_cast<uint32_t*>(ws + p.off_hist);
  P.base = reinterpret_cast<uint32_t*>(ws + p.off_base);
  P.bits = p.bits;
  P.bins = 1 << p.bits;
  // dT is cleared in equal shares beside the sort's 3 kernels a pass
  const int64_t share = p.passes ? bytes / (3 * p.passes) / 16 * 16 : bytes;
  P.zbytes = share;
  P.zero = static_cast<char*>(a.dtable);
  const unsigned zgrid = bytes ? (unsigned)std::min<int64_t>(2048, share / 4096 + 1) : 0;
  if (p.passes == 0) {
    P.kout = keys[0];
    P.sout = srcs[0];
    hipLaunchKernelGGL(sort_rank_kernel, dim3((unsigned)p.nblk + zgrid), dim3(256), 0, s, a, P);
    GMM_TRY(hipGetLastError());
  }
  for (int q = 0; q < p.passes; ++q) {
    P.shift = q * p.bits;
    P.kin = q ? keys[(q + 1) & 1] : nullptr;
    P.sin = q ? srcs[(q + 1) & 1] : nullptr;
    P.kout = keys[q & 1];
    P.sout = srcs[q & 1];
    const dim3 grid((unsigned)p.nblk + zgrid), scan((P.bins + 15) / 16 + zgrid);
    if (p.per == kSortSmall) hipLaunchKernelGGL(sort_count_kernel<kSortSmall>, grid, dim3(256), P.bins * 4, s, a, P);
    else hipLaunchKernelGGL(sort_count_kernel<kSortLarge>, grid, dim3(256), P.bins * 4, s, a, P);
    GMM_TRY(hipGetLastError());
    P.zero += share;
    hipLaunchKernelGGL(sort_scan_kernel, scan, dim3(256), 0, s, P);
    GMM_TRY(hipGetLastError());
    P.zero += share;
    if (q == p.passes - 1) P.zbytes = bytes - (3 * p.passes - 1) * share;
    if (p.per == kSortSmall) hipLaunchKernelGGL(sort_scatter_kernel<kSortSmall>, grid, dim3(256), P.bins * 16, s, a, P);
    else hipLaunchKernelGGL(sort_scatter_kernel<kSortLarge>, grid, dim3(256), P.bins * 16, s, a, P);
    GMM_TRY(hipGetLastError());
    P.zero += share;
  }
  SumArgs Q{};
  Q.S = p.S;
  Q.C = p.C;
  Q.chunks = p.chunks;
  Q.Dp = p.Dp;
  Q.none = p.none;
  Q.key = keys[p.passes ? (p.passes - 1) & 1 : 0];
  Q.src = srcs[p.passes ? (p.passes - 1) & 1 : 0];
  Q.part = reinterpret_cast<float*>(ws + p.off_part);
  const RowSplit sp = row_split(a.D, Vec<T>::E);
  const int64_t per = 256 >> sp.lg;
  hipLaunchKernelGGL((sum_kernel<T>), dim3((unsigned)((p.chunks + per - 1) / per), (unsigned)sp.slabs), dim3(256), 0, s, a, Q,
                     sp);
  GMM_TRY(hipGetLastError());
  if (p.chunks > 1) {
    hipLaunchKernelGGL((join_runs_kernel<T>), dim3((unsigned)(p.chunks - 1), (unsigned)std::min<int64_t>(4, (a.D + 127) / 128)), dim3(256),
                       0, s, a, Q);
    GMM_TRY(hipGetLastError());
  }
  return hipSuccess;
}

size_t upz(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

}  // namespace

hipError_t launch_zero(void* p, int64_t bytes, hipStream_t s) {
  if (bytes <= 0) return hipSuccess;
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(8192, (bytes / 16 + 255) / 256));
  hipLaunchKernelGGL(zero_kernel, dim3(grid), dim3(256), 0, s, (char*)p, bytes);
  return hipGetLastError();
}

LookupPlan lookup_plan(int64_t B, int64_t N, int64_t m, int64_t K, int64_t D, int dtype, bool want_table) {
  LookupPlan p{};
  if (!want_table || B * N == 0) return p;
  p.S = B * N * m;
  p.none = (uint32_t)(B * K);
  if (p.S <= kRankEntries) {  // passes 0: one kernel ranks them
    p.nblk = (p.S + 31) / 32;
  } else {
    int total = 0;
    while (((int64_t)1 << total) <= B * K) ++total;  // bits of the key B K
    p.passes = (total + 9) / 10;
    p.bits = (total + p.passes - 1) / p.passes;
    p.per = p.S <= 1 << 20 ? kSortSmall : kSortLarge;
    p.nblk = (p.S + 256 * p.per - 1) / (256 * p.per);
  }
  // entries of a chunk: as few as fill the card with threads (a thread per 16
  // bytes of a chunk), 8 at least, and at most 2^13 chunks up to 2^23 entries
  const RowSplit sp = row_split(D, dtype == 0 ? 4 : 8);
  const int64_t lanes = (int64_t)sp.slabs << sp.lg;
  p.C = 8;
  while (p.C < 1024 && (p.S / p.C * lanes > 1 << 18 || p.S / p.C > 1 << 13)) p.C *= 2;
  p.chunks = (p.S + p.C - 1) / p.C;
  p.Dp = (D + 7) / 8 * 8;
  size_t o = 0;
  for (int i = 0; i < 2; ++i) {
    p.off_key[i] = o; o = upz(o + sizeof(uint32_t) * (size_t)p.S);
    p.off_src[i] = o; o = upz(o + sizeof(uint32_t) * (size_t)p.S);
  }
  p.off_hist = o; o = upz(o + sizeof(uint32_t) * ((size_t)p.nblk << p.bits));
  p.off_base = o; o = upz(o + sizeof(uint32_t) * ((size_t)1 << p.bits));
  p.off_part = o; o = upz(o + sizeof(float) * (size_t)(2 * p.chunks * p.Dp));
  p.lengths = m > kScanCodes;
  if (p.lengths) { p.off_len = o; o = upz(o + sizeof(int32_t) * (size_t)(B * N)); }
  p.bytes = o;
  return p;
}

hipError_t launch_lookup(const LookupArgs& a, hipStream_t s) {
  if (a.dtype == 1) return lookup<__bf16>(a, s);
  if (a.dtype == 2) return lookup<_Float16>(a, s);
  return lookup<float>(a, s);
}

hipError_t launch_lookup_grad(const LookupArgs& a, const LookupPlan& p, char* ws, hipStream_t s) {
  if (a.dtype == 1) return lookup_grad<__bf16>(a, p, ws, s);
  if (a.dtype == 2) return lookup_grad<_Float16>(a, p, ws, s);
  return lookup_grad<float>(a, p, ws, s);
}

}  // namespace gmm
