// gmm_xent_small.hip -- softmax cross entropy and its gradients for rows of at
// most 128 features (the width of the mixtures' rows), without G in memory.
//
// With few features the products are cheap and what costs is everything per
// element of the N x V matrix: its exponential and, were G written, its bytes.
// So nothing of it leaves the registers.  A wave keeps the rows of one side
// (the owner: 16 RB rows, features as matrix-core fragments), the other side
// streams through LDS in tiles of 64 rows, and each 16 x 16 block of logits
// becomes in turn
//   LSE  owner rows, streamed classes: a running maximum and sum per lane
//   DX   owner rows, streamed classes: p - [v = y], rounded to the rows' type,
//        the second operand of dX^T += W^T G^T right from the registers
//   DW   owner classes, streamed rows: the same with c (p - [v = y]) and X
// The logits are formed as stream x owner^T, so that a lane holds 4 consecutive
// streamed rows of one owner row: the k order that the second product's
// fragment wants (two blocks for the 32 of an instruction), and its other
// operand, the streamed tile with its rows along k, comes out of LDS through
// the transposing read.  The bias enters as the accumulator's start.
// Three exponentials an element (LSE, DX, DW) and 10 N V D flops take the place
// of G's traffic, 8 bytes an element.
//
// Bound by the matrix cores and the exponentials together, at the 1.9 GHz that
// the card holds under them: 262144 x 128 rows, 4096 classes, bf16: LSE 0.32 ms,
// DX 0.58, DW 0.68 (0.84, 0.95 and 0.81 PFLOP/s with the logits' share); 1M x 64,
// 256 classes, float32: 0.26, 0.47, 0.43.  Two waves a SIMD: with three the
// fragments spill (DX 0.80, DW 1.55 ms); LSE of 128 features in 16 bits spills
// 8 of its 256 registers with two.
//
// LDS: a tile's rows are RBytes = D_padded * size apart, a row's 16-byte chunk c
// in slot c ^ f(row); f makes the reads of 16 rows touch all 64 banks.
//
// float32 rows run on the bf16 matrix cores too, as three planes (kPairs): six
// products at 16 times the rate of the float32 instruction, what they leave out
// below 2^-23 of |x| |w|, the size of the roundings of the sum.
//
// Rounding: as in gmm_xent.hip.  DX rounds p - [v = y] itself and multiplies
// by the row's coefficient in float32 at the end; half: p is scaled by 2^15
// (in the exponent).
#include "gmm_internal.h"
#include "gmm_xent.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <type_traits>

namespace gmm {

namespace {

enum Pass { LSE = 0, DX = 1, DW = 2 };

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

// exp(l - z) is exp2 of one fma, k l - k z, with k = log2(e).  Where |z| is so
// large that k z could leave float32, two float32 values apart are 2^99 apart or
// more, and exp(l - z) is 0 or 1 whatever k: there k = 1.  Over k = log2(e) for
// every row, which overflows there, that takes 0.8% more of the loss and gradients
// of 262144 x 128 bf16 rows, 4096 classes; the subtraction first everywhere 3.7%;
// a branch between the two inside the loop 5%, between two bodies of a tile
// spills (DW 562 -> 1684 us).
constexpr float kFar = 1e38f;
__device__ inline float factor_of(float z) { return fabsf(z) > kFar ? 1.f : kLog2e; }

// streamed rows per tile
constexpr int tile_rows(int es, int dp) { return es == 4 && dp == 128 ? 32 : 64; }

// rows of any layout -> [3][nr][Dp] bf16 planes, zeros past D; a thread per 4 elements
__global__ void __launch_bounds__(256) split_kernel(RowsArgs R, char* dst, int Dp) {
  const int q = Dp / 4;
  const int64_t n = R.nr * q, plane = R.nr * Dp * 2;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n; t += (int64_t)gridDim.x * 256) {
    const int64_t r = t / q;
    const int c = (int)(t - r * q) * 16;
    u32x2 p[3];
    split4(__builtin_bit_cast(f32x4, chunk_at<float>(R.x + row_offset(R, R.r0 + r) * 4, c, R.D * 4)), p);
#pragma unroll
    for (int k = 0; k < 3; ++k) *reinterpret_cast<u32x2*>(dst + k * plane + t * 8) = p[k];
  }
}

template <typename T>
__device__ inline float dot16(u32x4 a, u32x4 b) {
  T x[16 / sizeof(T)], y[16 / sizeof(T)];
  __builtin_memcpy(x, &a, 16);
  __builtin_memcpy(y, &b, 16);
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 16 / (int)sizeof(T); ++e) s = fmaf((float)x[e], (float)y[e], s);
  return s;
}

// waves per SIMD: DX at 32 features takes a few registers more than three waves
// leave it (262144 x 24 half rows, 4096 classes: 217 us with two, 205 so)
constexpr int min_waves(int es, int dp, int pass) { return es == 2 && dp == 32 && pass == DX ? 3 : 2; }

// S: the rows' type; its matrix-core form is itself, or bf16 planes
template <typename S, int DP, int RB, int PASS>
__global__ void __launch_bounds__(256, min_waves(sizeof(S), DP, PASS)) small_kernel(SmallArgs P) {
  using T = std::conditional_t<sizeof(S) == 4, __bf16, S>;
  constexpr int PL = planes(sizeof(S)), NP = PL == 1 ? 1 : 6, kTile = tile_rows(sizeof(S), DP);
  constexpr int RBytes = DP * 2, KC = RBytes / 16, KS = KC / 4;
  constexpr int kPlane = kTile * RBytes, kBytes = PL * kPlane, JS = kPlane / 4096;  // 16-byte loads of a thread per plane
  constexpr int RPB = RBytes >= 256 ? 1 : 256 / RBytes, FM = (KC < 16 ? KC : 16) - 1;
  constexpr int NB = kTile / 16, ND = DP / 16;
  // f(row), on the rows that share 256 bytes as one (g): a fragment read's 16
  // lanes at a time are rows 0-3 and 12-15 of one chunk and rows 4-11 of the
  // next, so the first eight's places have to be whole pairs; a transposing
  // read takes pairs of chunks of 8 rows, so those have to be of 8 pairs
  auto swizzle = [](int row) {
    const int g = (row / RPB) & FM, H = (FM + 1) / 2;
    return g < H ? 2 * g : 2 * ((g - H) ^ (H / 2)) + 1;
  };
  constexpr float kTop = __is_same(S, _Float16) ? 32768.f : 1.f;  // DX: scale of p
  __shared__ __attribute__((aligned(1024))) char st0[kBytes];
  __shared__ __attribute__((aligned(1024))) char st1[kBytes];
  __shared__ __attribute__((aligned(16))) float sp0[PASS == DW ? 4 * kTile : kTile];
  __shared__ __attribute__((aligned(16))) float sp1[PASS == DW ? 4 * kTile : kTile];

  // workgroups of one split of the stream on one XCD (they go round the 8)
  const unsigned total = gridDim.x, id = blockIdx.x, q8 = total / 8, r8 = total % 8, xc = id % 8;
  const unsigned pid = xc * q8 + (xc < r8 ? xc : r8) + id / 8;
  const int split = pid / P.tiles_own, tile_own = pid % P.tiles_own;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int64_t o0 = ((int64_t)tile_own * 4 + wv) * (16 * RB);  // the wave's first owner row

  const int ntiles = (int)((P.count + kTile - 1) / kTile);
  const int t0 = (int)((int64_t)ntiles * split / P.splits), t1 = (int)((int64_t)ntiles * (split + 1) / P.splits);
  // rows of a tile; those of tiles from t1 on belong to others or to nobody and
  // load as zeros that weigh nothing, so that a part may run one tile past its end
  auto rows_of = [&](int t) { return t < t1 ? (int)min((int64_t)kTile, P.count - (int64_t)t * kTile) : 0; };

  // ---- the owner's rows and what goes with each
  u32x4 own[RB][PL][KS];
  float oa[RB];  // DX: -k lse (+ log2 kTop);  DW: the class's bias
  float ok[RB];  // DX: k
  float oc[RB];  // DX: the row's coefficient
  int oy[RB];    // LSE: label;  DX: label within the piece;  DW: the class
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int64_t o = o0 + 16 * i + lr;
    bool live = o < P.own.nr;
    oa[i] = oc[i] = 0.f;
    oy[i] = -1;
    if (PASS == LSE && live) oy[i] = P.labels[o];
    if (PASS == DX && live) {
      oc[i] = P.coef[o];
      live = oc[i] != 0.f;  // a row that takes no part is read as zeros
    }
    if (PASS == DX) {
      const float z = live ? P.lse[o] : 0.f;
      ok[i] = factor_of(z);
      // k = 1: kTop has no room beside z, the row goes without it
      oa[i] = live ? fmaf(-z, ok[i], ok[i] == 1.f ? 0.f : __builtin_log2f(kTop)) : -INFINITY;
      if (live) oy[i] = P.labels[o] - (int)P.v0;  // a class of this piece, or none
    }
    if (PASS == DW) {
      oy[i] = (int)o;
      oa[i] = live ? (P.bias ? P.bias[o] : 0.f) : -INFINITY;
    }
    const char* row = P.own.x + (live ? row_offset(P.own, o) : 0) * (int64_t)sizeof(S);
    const int bytes = live ? P.own.D * (int)sizeof(S) : 0;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      if constexpr (PL == 1) {
        own[i][0][k] = chunk_at<S>(row, (k * 4 + lq) * 16, bytes);
      } else {
        u32x2 p[2][3];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          split4(__builtin_bit_cast(f32x4, chunk_at<S>(row, (k * 4 + lq) * 32 + 16 * u, bytes)), p[u]);
#pragma unroll
        for (int l = 0; l < PL; ++l) own[i][l][k] = u32x4{p[0][l][0], p[0][l][1], p[1][l][0], p[1][l][1]};
      }
    }
  }

  // ---- streamed tiles.  Load j of a thread: row row0 + j RPJ of the tile, one
  // 16-byte chunk, the same of every row (rows a multiple of 16 apart have the same f)
  constexpr int RPJ = 4096 / RBytes;
  const int kpad = (P.own.D * 2 + 15) & ~15;  // the stream's rows hold zeros from D to whole chunks
  const int row0 = (wv * 1024 + lane * 16) / RBytes;
  const int ch0 = ((wv * 1024 + lane * 16) % RBytes / 16) ^ swizzle(row0);
  const unsigned last = (unsigned)P.count - 1;
  float flag[JS];  // DW: the coefficients of the rows that are issued next
  auto flags = [&](int t) {
    if constexpr (PASS == DW) {  // rows past the last read the last one's; issue() leaves them out
#pragma unroll
      for (int j = 0; j < JS; ++j) flag[j] = P.coef[min((unsigned)(t * kTile + row0 + j * RPJ), last)];
    }
  };
  auto issue = [&](char* st, int t) {
    const int n = rows_of(t);
#pragma unroll
    for (int l = 0; l < PL; ++l) {
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<char*>(P.stream) + l * P.plane + (n > 0 ? (int64_t)t * kTile * P.ld_stream : 0), 0,
          n > 0 ? (unsigned)((n - 1) * P.ld_stream + kpad) : 0u, 0x00020000);
#pragma unroll
      for (int j = 0; j < JS; ++j) {
        bool in = row0 + j * RPJ < n && ch0 * 16 < kpad;
        if (PASS == DW) in = in && flag[j] != 0.f;  // rows that take no part arrive as zeros
        const unsigned o = in ? (unsigned)((row0 + j * RPJ) * (int)P.ld_stream + ch0 * 16) : kOutside;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (__attribute__((address_space(3))) void*)(st + l * kPlane + (j * 4 + wv) * 1024), 16, o, 0, 0, 0);
      }
    }
  };
  // what goes with each streamed row: LSE, DX: bias;  DW: -k lse, c, label, k
  float pa = 0.f, pb = 0.f;
  int py = -1;
  const float mult = PASS == DW && P.scal ? P.scal[0] : 1.f;
  auto fetch = [&](int t) {
    const unsigned r = min((unsigned)(t * kTile) + lane, last);
    if constexpr (PASS == DW) {
      pa = P.lse[r];
      pb = P.coef[r];
      py = P.labels[r];
    } else {
      pa = P.bias ? P.bias[P.v0 + r] : 0.f;
    }
  };
  auto put = [&](float* sp, int t) {
    if (wv != 0 || lane >= kTile) return;  // every wave fetches, the first puts
    const bool in = lane < rows_of(t);
    if constexpr (PASS == DW) {
      const bool live = in && pb != 0.f;
      const float k = factor_of(pa);
      sp[lane] = live ? pa * -k : -INFINITY;
      sp[3 * kTile + lane] = k;
      sp[kTile + lane] = live ? pb * mult : 0.f;
      sp[2 * kTile + lane] = __builtin_bit_cast(float, live ? py : -1);
    } else {
      sp[lane] = in ? pa : -INFINITY;
    }
  };

  constexpr int NA = PASS == LSE ? 1 : RB;
  f32x4 acc[NA][ND];  // DX, DW: element e of acc[i][d]: feature 16 d + 4 lq + e of owner row 16 i + lr
#pragma unroll
  for (int i = 0; i < NA; ++i)
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[i][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  float mx[RB], sm[RB];  // LSE: maximum and sum;  DW: mx is the bias gradient
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    mx[i] = PASS == LSE ? -FLT_MAX : 0.f;  // finite: -inf logits stay below it
    sm[i] = 0.f;
  }

  // logits of streamed block jb (16 rows) against owner block i
  const int fr = swizzle(lr);
  auto logits = [&](const char* st, const float* sp, int jb, f32x4* s) {
    if constexpr (PASS == DW) {
#pragma unroll
      for (int i = 0; i < RB; ++i) s[i] = f32x4{oa[i], oa[i], oa[i], oa[i]};
    } else {
      const f32x4 b = *reinterpret_cast<const f32x4*>(sp + 16 * jb + 4 * lq);
#pragma unroll
      for (int i = 0; i < RB; ++i) s[i] = b;
    }
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      u32x4 a[PL];
#pragma unroll
      for (int l = 0; l < PL; ++l)
        a[l] = *reinterpret_cast<const u32x4*>(st + l * kPlane + (16 * jb + lr) * RBytes + (((k * 4 + lq) ^ fr) * 16));
#pragma unroll
      for (int p = NP - 1; p >= 0; --p)  // the small products first
#pragma unroll
        for (int i = 0; i < RB; ++i) s[i] = mma<T>(a[kPairs[p][0]], own[i][kPairs[p][1]][k], s[i]);
    }
  };
  auto top_of = [](float k) { return kTop == 1.f || k == 1.f ? 1.f : kTop; };
  // G of a block, in place
  // (a block holds few labels: the lanes vote before they look for theirs)
  auto gradient = [&](const float* sp, int jb, int t, f32x4* s) {
    if constexpr (PASS == DX) {
#pragma unroll
      for (int i = 0; i < RB; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = __builtin_amdgcn_exp2f(fmaf(s[i][e], ok[i], oa[i]));
        const int y = oy[i] - t * kTile - 16 * jb;  // outside 0 .. 15 where the block has not got the label
        if (__builtin_amdgcn_ballot_w64((unsigned)y < 16u))
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] -= y == 4 * lq + e ? top_of(ok[i]) : 0.f;
      }
    } else {
      const f32x4 nl = *reinterpret_cast<const f32x4*>(sp + 16 * jb + 4 * lq);
      const f32x4 c = *reinterpret_cast<const f32x4*>(sp + kTile + 16 * jb + 4 * lq);
      const f32x4 k = *reinterpret_cast<const f32x4*>(sp + 3 * kTile + 16 * jb + 4 * lq);
      const i32x4 y = *reinterpret_cast<const i32x4*>(sp + 2 * kTile + 16 * jb + 4 * lq);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = c[e] * __builtin_amdgcn_exp2f(fmaf(s[i][e], k[e], nl[e]));
        if (__builtin_amdgcn_ballot_w64(y[0] == oy[i] || y[1] == oy[i] || y[2] == oy[i] || y[3] == oy[i]))
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] -= y[e] == oy[i] ? c[e] : 0.f;
        mx[i] += (s[i][0] + s[i][1]) + (s[i][2] + s[i][3]);
        asm volatile("" : "+v"(mx[i]));  // summed here: left alone, every G would stay in a register until the loop's end
      }
    }
  };

  auto compute = [&](const char* st, const float* sp, int t) {
    if constexpr (PASS == LSE) {
      f32x4 s[NB][RB];
#pragma unroll
      for (int jb = 0; jb < NB; ++jb) logits(st, sp, jb, s[jb]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        float m = mx[i];
#pragma unroll
        for (int jb = 0; jb < NB; ++jb)
#pragma unroll
          for (int e = 0; e < 4; ++e) m = fmaxf(m, s[jb][i][e]);
        const float k = factor_of(m), nm = -m * k;
        float a = sm[i] * __builtin_amdgcn_exp2f((mx[i] - m) * kLog2e);  // exactly 1 where nothing changed
#pragma unroll
        for (int jb = 0; jb < NB; ++jb)
#pragma unroll
          for (int e = 0; e < 4; ++e) a += __builtin_amdgcn_exp2f(fmaf(s[jb][i][e], k, nm));
        sm[i] = a;
        mx[i] = m;
      }
    } else {
#pragma unroll
      for (int h = 0; h < NB / 2; ++h) {
        f32x4 s[2][RB];
        u32x2 g[RB][2][PL];
#pragma unroll
        for (int u = 0; u < 2; ++u) logits(st, sp, 2 * h + u, s[u]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          gradient(sp, 2 * h + u, t, s[u]);
#pragma unroll
          for (int i = 0; i < RB; ++i) {
            if constexpr (PL == 1) {
              const T v[4] = {(T)s[u][i][0], (T)s[u][i][1], (T)s[u][i][2], (T)s[u][i][3]};
              g[i][u][0] = __builtin_bit_cast(u32x2, v);
            } else {
              split4(s[u][i], g[i][u]);
            }
          }
        }
        // lane 16 a + b reads feature 16 d + b of streamed rows 4 a .. 4 a + 3 of either block
        const int rr = lane >> 2, fx = swizzle(rr);
        const char* src = st + (32 * h + rr) * RBytes + 8 * (lane & 1);
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          const int slot = ((2 * d + ((lane & 3) >> 1)) ^ fx) * 16;
          u32x4 a[PL];
#pragma unroll
          for (int l = 0; l < PL; ++l) {
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(src + l * kPlane + slot));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(src + l * kPlane + 16 * RBytes + slot));
            a[l] = __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
          }
#pragma unroll
          for (int p = NP - 1; p >= 0; --p)
#pragma unroll
            for (int i = 0; i < RB; ++i) {
              const u32x2 *g0 = &g[i][0][kPairs[p][1]], *g1 = &g[i][1][kPairs[p][1]];
              acc[i][d] = mma<T>(a[kPairs[p][0]], u32x4{(*g0)[0], (*g0)[1], (*g1)[0], (*g1)[1]}, acc[i][d]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // loads of a tile run while the tile before it is computed
  auto step = [&](char* cur, float* pcur, char* nxt, float* pnxt, int t) {
    __builtin_amdgcn_s_waitcnt(kVm0);
    __syncthreads();
    issue(nxt, t + 1);
    fetch(t + 1);
    flags(t + 2);
    compute(cur, pcur, t);
    put(pnxt, t + 1);
  };
  flags(t0);
  issue(st0, t0);
  fetch(t0);
  put(sp0, t0);
  flags(t0 + 1);
  for (int t = t0; t < t1; t += 2) {
    step(st0, sp0, st1, sp1, t);
    step(st1, sp1, st0, sp0, t + 1);
  }
  __builtin_amdgcn_s_waitcnt(kVm0);  // nothing of the last loads is in flight at the end

  // ---- results
  if constexpr (PASS == LSE) {
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int64_t o = o0 + 16 * i + lr;
      const bool in = o < P.own.nr;
      // the label's logit: the row against the label's row of the head
      const bool lab = oy[i] >= 0 && oy[i] < P.V;
      float l = 0.f;
      const int bytes = P.own.D * (int)sizeof(S);
      const char* wr = P.w + (lab ? oy[i] * P.ld_w * (int64_t)sizeof(S) : 0);
      const char* xr = P.own.x + (lab ? row_offset(P.own, o) : 0) * (int64_t)sizeof(S);
      if (lab)
        for (int c = lq * 16; c < bytes; c += 64) l += dot16<S>(chunk_at<S>(xr, c, bytes), chunk_at<S>(wr, c, bytes));
      float m = mx[i], s = sm[i];
#pragma unroll
      for (int off = 16; off < 64; off <<= 1) {
        l += __shfl_xor(l, off);
        const float m2 = __shfl_xor(m, off), s2 = __shfl_xor(s, off), top = fmaxf(m, m2);
        s = s * __builtin_amdgcn_exp2f((m - top) * kLog2e) + s2 * __builtin_amdgcn_exp2f((m2 - top) * kLog2e);
        m = top;
      }
      if (lab && P.bias) l += P.bias[oy[i]];
      if (!in || lq != 0) continue;
      if (P.part) {
        P.part[split * P.own.nr + o] = make_float2(m, s);
        if (split == 0) P.lab[o] = l;
      } else {
        const float z = m + logf(s);
        P.lse_out[o] = z;
        P.loss[o] = oy[i] < 0 ? 0.f : lab ? z - l : NAN;
      }
    }
  } else {
    const float back = PASS == DW && P.scal ? P.scal[1] : 1.f;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int64_t o = o0 + 16 * i + lr;
      const bool in = o < P.own.nr;
      if (PASS == DW && P.dbp) {
        float v = mx[i] * back;
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
        if (in && lq == 0) P.dbp[split * P.own.nr + o] = v;
      }
      if (!in) continue;
      const float c = PASS == DX ? oc[i] / top_of(ok[i]) : back;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const int64_t f = 16 * d + 4 * lq;
        if (f >= P.own.D) continue;
        f32x4 v = acc[i][d] * c;
        if (PASS == DX && oc[i] == 0.f) v = f32x4{0.f, 0.f, 0.f, 0.f};
        if (P.slab) {
          float* p = P.slab + split * P.slab_stride + o * P.lds + f;
          if (P.add) v += *reinterpret_cast<const f32x4*>(p);
          *reinterpret_cast<f32x4*>(p) = v;
          continue;
        }
        S* p = reinterpret_cast<S*>(P.out) + o * P.own.D + f;
        if (f + 4 <= P.own.D && !P.accumulate) {
          store4<S>(p, v);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (f + e < P.own.D) p[e] = (S)(v[e] + (P.accumulate ? to_f32(p[e]) : 0.f));
        }
      }
    }
  }
}

// 16-row blocks of a wave: as many as the registers hold
constexpr int owner_blocks(int es, int dp, int pass) {
  if (es == 2) return pass == LSE || dp <= 64 ? 4 : 2;
  if (pass == LSE) return dp >= 64 ? 2 : 4;
  return dp == 128 ? 1 : 2;
}

template <typename T, int DP, int PASS>
hipError_t launch_p(const SmallArgs& P, hipStream_t s) {
  constexpr int RB = owner_blocks(sizeof(T), DP, PASS);
  const dim3 grid((unsigned)((int64_t)P.tiles_own * P.splits));
  hipLaunchKernelGGL((small_kernel<T, DP, RB, PASS>), grid, dim3(256), 0, s, P);
  return hipGetLastError();
}
template <typename T, int DP>
hipError_t launch(const SmallArgs& P, int pass, hipStream_t s) {
  if (pass == LSE) return launch_p<T, DP, LSE>(P, s);
  if (pass == DX) return launch_p<T, DP, DX>(P, s);
  return launch_p<T, DP, DW>(P, s);
}

template <typename T>
hipError_t launch_t(const SmallArgs& P, int pass, hipStream_t s) {
  if (P.own.D <= 32) return launch<T, 32>(P, pass, s);
  if (P.own.D <= 64) return launch<T, 64>(P, pass, s);
  return launch<T, 128>(P, pass, s);
}

}  // namespace

int xent_small_rows(int dtype, int64_t D, int pass) {
  return 64 * owner_blocks(dtype == 0 ? 4 : 2, D <= 32 ? 32 : D <= 64 ? 64 : 128, pass);
}

int xent_small_splits(int64_t owners, int64_t streamed, int dtype, int64_t D, int pass) {
  const int rows = xent_small_rows(dtype, D, pass);
  const int64_t t = (owners + rows - 1) / rows, tiles = (streamed + 63) / 64;
  const int64_t want = t >= 2 * kNumCU ? 1 : (2 * kNumCU) / t;
  return (int)std::max<int64_t>(1, std::min(want, tiles / 4));
}

hipError_t launch_xent_split(const RowsArgs& r, char* dst, int64_t Dp, hipStream_t s) {
  const int64_t n = r.nr * Dp / 4;
  hipLaunchKernelGGL(split_kernel, dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, 1 << 16))),
                     dim3(256), 0, s, r, dst, (int)Dp);
  return hipGetLastError();
}

hipError_t launch_xent_small(SmallArgs P, int dtype, int pass, hipStream_t s) {
  const int rows = xent_small_rows(dtype, P.own.D, pass);
  P.tiles_own = (int)((P.own.nr + rows - 1) / rows);
  if (dtype == 1) return launch_t<__bf16>(P, pass, s);
  if (dtype == 2) return launch_t<_Float16>(P, pass, s);
  return launch_t<float>(P, pass, s);
}

}  // namespace gmm
