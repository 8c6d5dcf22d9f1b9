// gmm_xent.hip -- softmax cross entropy of rows under a linear head of V
// classes, and its gradient, without the N x V logits ever being kept.
//
// What it computes.  For row x_i with label y_i, head rows W_v and bias b_v:
//   l_iv   = W_v . x_i + b_v
//   lse_i  = log sum_v exp(l_iv)
//   loss_i = lse_i - l_{i, y_i}
//   G_iv   = g_i (exp(l_iv - lse_i) - [v = y_i])       (g_i: the loss's gradient)
//   dX = G W,   dW = G^T X,   db = sum_i G_i
// (the log-sum-exp and the responsibility-weighted sums of the mixture's
// E-step, with a head's weights in the place of means and variances).
//
// How.  Everything is one matrix-core kernel, C[m][n] = sum_k A[m][k] B[n][k]
// with both operands contiguous along k, under three epilogues:
//   LSE   rows x classes: each tile leaves one (max, sum of exponentials) per
//         row, and the label's logit; a small kernel joins the tiles;
//   GRAD  rows x classes of one piece: the logits again, turned into G in the
//         accumulators; G and its transpose are written in the rows' type;
//   OUT   the products G W and G^T X over such a piece;
// few tiles over a long k run as OUT too, in parts of k side by side, and two
// small kernels do the other epilogues from the parts' sum (logit_parts).
// A piece is at most 2^27 (float32: 2^26) elements of G, whatever N and V.
// The gradients form the logits again, a third more arithmetic (4096 x 4096
// rows, 65536 classes, bf16: 1.8 ms), and no N V floats are allocated; kept in
// float32, chunk by chunk, they would cost 8 N V bytes written and read (0.4 ms
// there) and a call that takes the loss and its gradients together.  W and X
// enter the OUT products transposed, so that one main loop serves all three: a
// copy of a piece of W and one of a chunk's rows, a few percent of the time over
// many rows (0.24 of 7.4 ms), but most of W's traffic where the rows are few.
//
// The tile's operands go from global memory straight into LDS with 16-byte
// buffer loads, two buffers, one barrier per k-tile of 128 bytes.  The loads
// carry their own bounds: a row or k-chunk outside the operand has an offset
// past the resource's end and arrives as zeros.  A row's 16-byte chunk c sits
// in slot c ^ f(row) of its LDS row, so the fragment reads of 16 rows touch
// all 64 banks.  Each quarter of a k-tile is multiplied from registers that the
// quarter before it read.  Bound by the matrix cores: 4096 x 4096 rows, 65536
// classes, bf16: LSE 1.76 ms (1.25 PFLOP/s), GRAD 2.14 (1.03; its epilogue adds
// 0.2), G W and G^T X 1.85 each (1.19).
//
// float32 rows enter as three bf16 planes (kPairs), packed on the way in: six
// products of planes follow each other along k, the smallest first.  4096 x 4096
// rows, 16384 classes: loss 2.53 ms, loss and gradients 10.6 (the float32
// instruction: 3.79 and 15.3).
//
// Rounding.  Accumulators, maxima, sums, G and the bias gradient are float32;
// G is rounded once to the rows' type to enter the matrix cores (2^-9 of each
// element for bf16, the size of the rounding of the outputs themselves), after
// it was divided by max |g_i| (scal_kernel says why).
#include "gmm_internal.h"
#include "gmm_xent.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

namespace gmm {

namespace {

enum Mode { LSE = 0, GRAD = 1, OUT = 2 };

struct GemmArgs {
  const char* A;       // [M][K], row stride lda bytes
  const char* B;       // [N][K], row stride ldb bytes
  int64_t lda, ldb;
  int64_t M, N;
  int64_t pa, pb;      // float32: bytes from one bf16 plane of an operand to the next
  int kbytes;          // valid bytes of a row (of one plane), a multiple of 16
  int ktiles, splits;  // 128-byte k-tiles (over all pairs of planes), shared among splits
  int tm, tn;          // tiles
  // LSE and GRAD: classes v0 .. v0 + N of the head
  const float* bias;   // (V) or null
  const int32_t* labels;
  int64_t v0;
  float2* part;        // LSE: [tile n][M]
  float* lab;          // LSE: the label's logit
  const float* lse;    // GRAD
  const float* coef;   // GRAD: g_i (0: the row takes no part)
  const float* scal;   // {multiplier of G, its inverse}; null: 1
  char* G;             // GRAD: [M][ldg] 16-bit, [3] of them for float32
  char* GT;            // GRAD: [N][ldgt] likewise, null: not wanted
  int64_t ldg, ldgt;   // elements, whole k-tiles
  int64_t gcols;       // columns of G from this launch's first on, whole k-tiles
  int64_t gp, tp;      // float32: elements from one plane of G, of its transpose, to the next
  float* dbp;          // GRAD: [tile m][N] column sums, null: not wanted
  // OUT
  float* slab;         // [splits][M][lds] float32, null: straight to out
  int64_t lds, slab_stride;
  int add;             // slabs: add to what is there
  char* out;           // [M][N] rows' type
  int accumulate;      // out: add to what is there
  const float* rowlive;  // rows with 0 here get zeros (null: none)
};

// tile of the workgroup: consecutive tiles of a group of 8 tile rows on one
// XCD (workgroups go round the 8 XCDs), so that an XCD's L2 holds what they share
__device__ inline void tile_of(const GemmArgs& P, int& tm, int& tn, int& z) {
  const unsigned total = gridDim.x, id = blockIdx.x;
  const unsigned q = total / 8, r = total % 8, x = id % 8, i = id / 8;
  const unsigned pid = x * q + (x < r ? x : r) + i;
  const unsigned per = (unsigned)P.tm * P.tn;
  z = pid / per;
  const unsigned t = pid % per, width = 8u * P.tn, first = t / width * 8;
  const unsigned rows = min((unsigned)P.tm - first, 8u);
  tm = first + (t % width) % rows;
  tn = (t % width) / rows;
}

// row m's label, counted from class n of the piece (-1: not among the next 2^20)
__device__ inline int label_at(const GemmArgs& P, int64_t m, int64_t n) {
  if (m >= P.M) return -1;
  const int64_t y = (int64_t)P.labels[m] - P.v0 - n;
  return y < 0 || y >= (1 << 20) ? -1 : (int)y;
}

// this wave's loads into LDS have landed and its LDS reads are done; then the
// other waves' too
__device__ inline void next_tile() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// S: the rows' type; its matrix-core form is itself, or bf16 planes
template <typename S, int BM, int BN, int WM, int WN, int MODE>
__global__ void __launch_bounds__(WM* WN * 64, 2) gemm_kernel(GemmArgs P) {
  using T = std::conditional_t<sizeof(S) == 4, __bf16, S>;
  constexpr int PL = planes(sizeof(S)), NP = PL == 1 ? 1 : 6;
  constexpr int NT = WM * WN * 64;          // threads
  constexpr int MT = BM / WM / 16, NN = BN / WN / 16;  // 16 x 16 tiles of a wave
  constexpr int JA = BM * 8 / NT, JB = BN * 8 / NT;    // 16-byte loads of a thread per k-tile
  constexpr int kStage = (BM + BN) * 128;
  // two objects, so that the reads of one do not wait for the loads into the other
  __shared__ __attribute__((aligned(1024))) char st0[kStage];
  __shared__ __attribute__((aligned(1024))) char st1[kStage];

  int tm, tn, z;
  tile_of(P, tm, tn, z);
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv / WN, wn = wv % WN;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int mrows = (int)min((int64_t)BM, P.M - m0), nrows = (int)min((int64_t)BN, P.N - n0);

  const int kt0 = (int)((int64_t)P.ktiles * z / P.splits), kt1 = (int)((int64_t)P.ktiles * (z + 1) / P.splits);
  // load j of lane l: LDS row 8 (j * waves + wave) + l / 8, slot l % 8, which
  // holds the same chunk c for every j.  Rows past the operand's last have
  // offsets past the resource's end by themselves.
  static_assert((NT / 64) % 2 == 0, "rows of a thread's loads are a multiple of 16 apart");
  const int row0 = 8 * wv + (lane >> 3), c16 = ((lane & 7) ^ ((row0 >> 1) & 7)) * 16;
  const unsigned oa = (unsigned)(row0 * P.lda) + c16, ob = (unsigned)(row0 * P.ldb) + c16;
  const unsigned sa = (unsigned)(8 * (NT / 64) * P.lda), sb = (unsigned)(8 * (NT / 64) * P.ldb);
  // k-tiles are issued in order; the pairs of planes follow each other, the
  // small products first
  const int per = P.ktiles / NP;
  int pair = NP - 1 - kt0 / per, kk = kt0 % per;
  auto issue = [&](lds_char* st, int kt) {
    const char *A = P.A + m0 * P.lda, *B = P.B + n0 * P.ldb;
    if (PL > 1) {
      A += kPairs[max(pair, 0)][0] * P.pa;
      B += kPairs[max(pair, 0)][1] * P.pb;
    }
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(A), 0, (unsigned)((mrows - 1) * P.lda + P.kbytes), 0x00020000);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(B), 0, (unsigned)((nrows - 1) * P.ldb + P.kbytes), 0x00020000);
    const unsigned kb = kk * 128;
    // past the last k the offset's top bit is set (added, not selected: a
    // select becomes branches around the loads)
    const unsigned out = kt < kt1 && (int)kb + c16 < P.kbytes ? 0u : kOutside;
    const unsigned xa = oa + out, xb = ob + out;
#pragma unroll
    for (int j = 0; j < JA; ++j)
      load_lds16(ra, st + (j * (NT / 64) + wv) * 1024, xa + (kb + j * sa));
#pragma unroll
    for (int j = 0; j < JB; ++j)
      load_lds16(rb, st + BM * 128 + (j * (NT / 64) + wv) * 1024, xb + (kb + j * sb));
    if (++kk == per) {
      kk = 0;
      --pair;
    }
  };

  f32x4 acc[MT][NN];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int lr = lane & 15, lq = lane >> 4;
  constexpr int MH = MT / 2;
  auto read_a = [&](const char* st, int half, int g, u32x4* f) {
    const int slot = ((half * 4 + lq) ^ ((lr >> 1) & 7)) * 16;
#pragma unroll
    for (int i = 0; i < MH; ++i)
      f[i] = *reinterpret_cast<const u32x4*>(st + ((wm * MT + g * MH + i) * 16 + lr) * 128 + slot);
  };
  auto read_b = [&](const char* st, int half, u32x4* f) {
    const int slot = ((half * 4 + lq) ^ ((lr >> 1) & 7)) * 16;
#pragma unroll
    for (int j = 0; j < NN; ++j)
      f[j] = *reinterpret_cast<const u32x4*>(st + BM * 128 + ((wn * NN + j) * 16 + lr) * 128 + slot);
  };
  auto multiply = [&](const u32x4* fb, const u32x4* fa, int g) {
    __builtin_amdgcn_sched_barrier(0);  // the reads and loads before it first: they have the longest way
#pragma unroll
    for (int i = 0; i < MH; ++i)
#pragma unroll
      for (int j = 0; j < NN; ++j) acc[g * MH + i][j] = mma<T>(fb[j], fa[i], acc[g * MH + i][j]);
    __builtin_amdgcn_sched_barrier(0);
  };

  // A k-tile is multiplied in four steps (two halves of k, two of the wave's
  // rows), each from registers that the step before it read from LDS, so that
  // no product waits for LDS.  A tile's buffer is free once the last step's
  // operands are in registers: the tile after next starts into it there, and
  // has until the same point of the next tile to land.
  u32x4 b0[NN], b1[NN], a0[MH], a1[MH];
  auto tile = [&](char* cur, const char* nxt, int k) {
    read_a(cur, 0, 1, a1);
    multiply(b0, a0, 0);
    read_b(cur, 1, b1);
    read_a(cur, 1, 0, a0);
    multiply(b0, a1, 1);
    read_a(cur, 1, 1, a1);
    multiply(b1, a0, 0);
    next_tile();  // tile k + 1 has landed, tile k is read out
    issue((lds_char*)cur, k + 2);
    read_b(nxt, 0, b0);
    read_a(nxt, 0, 0, a0);
    multiply(b1, a1, 1);
  };
  issue((lds_char*)st0, kt0);
  next_tile();
  issue((lds_char*)st1, kt0 + 1);
  read_b(st0, 0, b0);
  read_a(st0, 0, 0, a0);
  int kt = kt0;
  for (; kt + 2 <= kt1; kt += 2) {
    tile(st0, st1, kt);
    tile(st1, st0, kt + 1);
  }
  if (kt < kt1) tile(st0, st1, kt);

  // accumulator element e of acc[i][j]: row m = 16 (wm MT + i) + lr of the
  // tile, column n = 16 (wn NN + j) + 4 lq + e
  const int mw = wm * MT * 16 + lr, nw = wn * NN * 16 + 4 * lq;

  if constexpr (MODE == OUT) {
    const bool vec = (P.N % 4) == 0;  // rows of out start 4 elements apart
    const float sc = P.scal ? P.scal[1] : 1.f;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int64_t m = m0 + mw + 16 * i;
      if (m >= P.M) continue;
      const bool dead = P.rowlive && P.rowlive[m] == 0.f;
#pragma unroll
      for (int j = 0; j < NN; ++j) {
        const int64_t n = n0 + nw + 16 * j;
        if (n >= P.N) continue;
        f32x4 v = acc[i][j];
        if (P.slab) {
          float* p = P.slab + z * P.slab_stride + m * P.lds + n;  // lds: N rounded up to 4
          if (P.add) v += *reinterpret_cast<const f32x4*>(p);
          *reinterpret_cast<f32x4*>(p) = v;
          continue;
        }
        v = dead ? f32x4{0.f, 0.f, 0.f, 0.f} : v * sc;
        S* p = reinterpret_cast<S*>(P.out) + m * P.N + n;
        if (vec && !P.accumulate) {
          store4<S>(p, v);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < P.N) p[e] = (S)(v[e] + (P.accumulate ? to_f32(p[e]) : 0.f));
        }
      }
    }
    return;
  } else {
    // logits: the bias, and -inf past the last class
    f32x4 bv[NN];
#pragma unroll
    for (int j = 0; j < NN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t n = n0 + nw + 16 * j + e;
        bv[j][e] = n < P.N ? (P.bias ? P.bias[P.v0 + n] : 0.f) : -INFINITY;
      }
    __builtin_amdgcn_s_waitcnt(kVm0);
    __syncthreads();  // no load is on its way, the last k-tile is read out: LDS is free

    if constexpr (MODE == LSE) {
      float2* red = reinterpret_cast<float2*>(st0);  // [WN][BM]
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + mw + 16 * i;
        const int y = label_at(P, m, n0 + nw);
        float mx = -INFINITY, lab = 0.f;
#pragma unroll
        for (int j = 0; j < NN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[i][j][e] += bv[j][e];
            mx = fmaxf(mx, acc[i][j][e]);
            lab = y == 16 * j + e ? acc[i][j][e] : lab;
          }
        if (y >= 0 && y < 16 * NN && (y & 15) < 4) P.lab[m] = lab;  // this lane holds the label's column
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float base = mx == -INFINITY ? 0.f : mx;  // nothing but -inf: a sum of 0
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < NN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s += __builtin_amdgcn_exp2f((acc[i][j][e] - base) * kLog2e);
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if (lq == 0) red[wn * BM + mw + 16 * i] = make_float2(mx, s);
        __builtin_amdgcn_sched_barrier(0);  // one row block's temporaries at a time
      }
      __syncthreads();
      for (int r = tid; r < mrows; r += NT) {
        float mx = -INFINITY, s = 0.f;
#pragma unroll
        for (int w = 0; w < WN; ++w) mx = fmaxf(mx, red[w * BM + r].x);
        const float base = mx == -INFINITY ? 0.f : mx;  // a wave of -inf alone has sum 0
#pragma unroll
        for (int w = 0; w < WN; ++w) {
          const float2 t = red[w * BM + r];
          s += t.y * __builtin_amdgcn_exp2f((t.x - base) * kLog2e);
        }
        P.part[(int64_t)tn * P.M + m0 + r] = make_float2(mx, s);
      }
    } else {
      constexpr int kRegion = 16384;                       // bytes of LDS per wave
      constexpr int kSub = kRegion / (PL * NN * 16 * 16 * 2);
      constexpr int SUB = kSub < MT ? kSub : MT;           // row blocks transposed at a time
      constexpr int EPC = 8;                               // elements of a 16-byte chunk
      constexpr int CR = SUB * 16 / EPC, CL = 16 / EPC;    // chunks of a transposed row; of 16 elements
      constexpr int kGPlane = NN * 16 * SUB * 16;          // elements of a plane in the region
      static_assert(MT % SUB == 0, "transposing in whole sub-tiles");
      static_assert(WM * WN * kRegion <= 2 * kStage, "the waves' regions fill the two stages");
      T* reg = reinterpret_cast<T*>((wv < WM * WN / 2 ? st0 : st1) + (wv % (WM * WN / 2)) * kRegion);
      const float mult = P.scal ? P.scal[0] : 1.f;
      const unsigned pick = lane & 1 ? 0x03020706u : 0x05040100u;  // this lane's column of a pair
      float cs[NN][4];
#pragma unroll
      for (int j = 0; j < NN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) cs[j][e] = 0.f;
#pragma unroll
      for (int i0 = 0; i0 < MT; i0 += SUB) {
#pragma unroll
        for (int ii = 0; ii < SUB; ++ii) {
          const int i = i0 + ii;
          const int64_t m = m0 + mw + 16 * i;
          const float c = m < P.M ? P.coef[m] : 0.f;
          const float ls = m < P.M ? P.lse[m] : 0.f;
          const int y = label_at(P, m, n0 + nw);
          const float cm = c * mult;
#pragma unroll
          for (int j = 0; j < NN; ++j) {
            f32x4 g;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = __builtin_amdgcn_exp2f((acc[i][j][e] + bv[j][e] - ls) * kLog2e);
              const bool live = c != 0.f && n0 + nw + 16 * j + e < P.N;  // NaN is live
              g[e] = live ? cm * (p - (y == 16 * j + e ? 1.f : 0.f)) : 0.f;
              cs[j][e] += g[e];
            }
            const int64_t n = n0 + nw + 16 * j;
            const int ml = 16 * ii + lr, nl = 16 * j + 4 * lq;
            u32x2 w[3];
            if constexpr (PL == 1) {
              const T t[4] = {(T)g[0], (T)g[1], (T)g[2], (T)g[3]};
              w[0] = __builtin_bit_cast(u32x2, t);
            } else {
              split4(g, w);
            }
#pragma unroll
            for (int l = 0; l < PL; ++l) {
              if (m < P.M && n < P.gcols) *reinterpret_cast<u32x2*>(reinterpret_cast<T*>(P.G) + l * P.gp + m * P.ldg + n) = w[l];
              if (P.GT) {
                // a dword holds two columns of one row; neighbouring rows' lanes
                // trade, so that each writes two rows of one column
                const int mp = ml & ~1, ch = (mp / EPC) ^ ((CL * lq) & (CR - 1));  // rows 4 apart would share banks
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const unsigned o = __builtin_amdgcn_mov_dpp(w[l][u], 0xB1, 0xF, 0xF, true);  // quad_perm 1 0 3 2
                  const unsigned v = __builtin_amdgcn_perm(o, w[l][u], pick);
                  *reinterpret_cast<unsigned*>(reg + l * kGPlane + (nl + 2 * u + (lane & 1)) * (SUB * 16) + ch * EPC +
                                               mp % EPC) = v;
                }
              }
            }
            __builtin_amdgcn_sched_barrier(0);  // one 16 x 16 tile's temporaries at a time
          }
        }
        if (P.GT) {
          __syncthreads();
#pragma unroll
          for (int l = 0; l < PL; ++l)
#pragma unroll
            for (int t = 0; t < NN * 16 * CR / 64; ++t) {
              const int idx = t * 64 + lane, nl = idx / CR, ch = idx % CR;
              const u32x4 v = *reinterpret_cast<const u32x4*>(reg + l * kGPlane + nl * (SUB * 16) +
                                                              (ch ^ ((CL * ((nl >> 2) & 3)) & (CR - 1))) * EPC);
              const int64_t n = n0 + wn * NN * 16 + nl, m = m0 + wm * MT * 16 + i0 * 16 + ch * EPC;
              if (n < P.N && m < P.ldgt) *reinterpret_cast<u32x4*>(reinterpret_cast<T*>(P.GT) + l * P.tp + n * P.ldgt + m) = v;
            }
          __syncthreads();
        }
      }
      if (P.dbp) {
        float* red = reinterpret_cast<float*>(st0);  // [WM][BN]
#pragma unroll
        for (int j = 0; j < NN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = cs[j][e];
            v += __shfl_xor(v, 1);
            v += __shfl_xor(v, 2);
            v += __shfl_xor(v, 4);
            v += __shfl_xor(v, 8);
            if (lr == 0) red[wm * BN + nw + 16 * j + e] = v;
          }
        __syncthreads();
        for (int c = tid; c < nrows; c += NT) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < WM; ++w) v += red[w * BN + c];
          P.dbp[(int64_t)tm * P.N + n0 + c] = v;
        }
      }
    }
  }
}

// Scoring of a few rows (serving): at most 16 MT rows against the whole head,
// bound by reading W once.  A wave owns 16 classes and walks their rows of W
// from global memory into MFMA fragments (no LDS: nothing is shared); the
// rows' fragments come from the L1.  One (max, sum) per row and 64 classes.
// 1 x 2048 under 32768 classes, bf16: 24.8 us, 5.4 TB/s of W.
template <typename T, int MT>
__global__ void __launch_bounds__(256) skinny_kernel(GemmArgs P, RowsArgs R) {
  constexpr int U = 8;  // k-steps of 64 bytes in flight
  __shared__ float2 red[4][16 * MT];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, lr = lane & 15, lq = lane >> 4;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + wv) * 16;
  const int64_t nr = min(n0 + lr, P.N - 1);  // classes past the last read its row and are masked
  const char* w = P.B + nr * P.ldb;
  const char* x[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
    x[i] = R.x + row_offset(R, min((int64_t)(16 * i + lr), P.M - 1)) * (int64_t)sizeof(T);
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k0 = lq * 16; k0 < P.kbytes + lq * 16; k0 += 64 * U) {
    u32x4 b[U], a[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + 64 * u;
      b[u] = chunk_at<T>(w, k, P.kbytes);
#pragma unroll
      for (int i = 0; i < MT; ++i) a[u][i] = chunk_at<T>(x[i], k, P.kbytes);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] = mma<T>(b[u], a[u][i], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = 16 * i + lr;
    const int64_t y = m < P.M ? (int64_t)P.labels[m] - n0 - 4 * lq : -1;
    float mx = -INFINITY;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t n = n0 + 4 * lq + e;
      acc[i][e] = n < P.N ? acc[i][e] + (P.bias ? P.bias[n] : 0.f) : -INFINITY;
      mx = fmaxf(mx, acc[i][e]);
      if (y == e && n < P.N) P.lab[m] = acc[i][e];
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float base = mx == -INFINITY ? 0.f : mx;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) s += __builtin_amdgcn_exp2f((acc[i][e] - base) * kLog2e);
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lq == 0) red[wv][16 * i + lr] = make_float2(mx, s);
  }
  __syncthreads();
  const int r = threadIdx.x;
  if (r < 16 * MT && r < P.M) {
    float mx = -INFINITY, s = 0.f;
#pragma unroll
    for (int w2 = 0; w2 < 4; ++w2) mx = fmaxf(mx, red[w2][r].x);
    const float base = mx == -INFINITY ? 0.f : mx;
#pragma unroll
    for (int w2 = 0; w2 < 4; ++w2) s += red[w2][r].y * __builtin_amdgcn_exp2f((red[w2][r].x - base) * kLog2e);
    P.part[(int64_t)blockIdx.x * P.M + r] = make_float2(mx, s);
  }
}

// Joins the tiles' (max, sum): RB rows per workgroup, 256 / RB threads a row,
// so that few rows with many tiles wait for few loads (latency: 3.9 to 5.5 us).
template <int RB>
__global__ void __launch_bounds__(256) join_kernel(const float2* part, int64_t ntiles, int64_t M, const int32_t* labels,
                                                   int64_t V, const float* lab, float* loss, float* lse) {
  constexpr int SL = 256 / RB;
  __shared__ float2 red[SL][RB];
  const int r = threadIdx.x % RB, sl = threadIdx.x / RB;
  const int64_t m = (int64_t)blockIdx.x * RB + r;
  float mx = -INFINITY, s = 0.f;
  if (m < M) {
    constexpr int U = 8;  // loads in flight
    for (int64_t t0 = sl; t0 < ntiles; t0 += SL * U) {
      float2 v[U];
      float nm = mx;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t t = t0 + (int64_t)u * SL;
        v[u] = t < ntiles ? part[t * M + m] : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) nm = fmaxf(nm, v[u].x);
      const float base = nm == -INFINITY ? 0.f : nm;
      s *= __builtin_amdgcn_exp2f((mx - base) * kLog2e);
#pragma unroll
      for (int u = 0; u < U; ++u) s += v[u].y * __builtin_amdgcn_exp2f((v[u].x - base) * kLog2e);
      mx = nm;
    }
  }
  red[sl][r] = make_float2(mx, s);
  // halves of the slices, one into the other
#pragma unroll
  for (int h = SL / 2; h > 0; h /= 2) {
    __syncthreads();
    if (sl < h) {
      const float2 t = red[sl + h][r];
      const float top = fmaxf(mx, t.x), base = top == -INFINITY ? 0.f : top;
      s = s * __builtin_amdgcn_exp2f((mx - base) * kLog2e) + t.y * __builtin_amdgcn_exp2f((t.x - base) * kLog2e);
      mx = top;
      red[sl][r] = make_float2(mx, s);
    }
  }
  if (sl != 0 || m >= M) return;
  const float top = mx, tot = s;
  const float z = top + logf(tot);
  const int32_t y = labels[m];
  lse[m] = z;
  loss[m] = y < 0 ? 0.f : y >= V ? NAN : z - lab[m];
}

// coef_i: the loss's gradient of a labelled row, 0 where the label is
// negative, NaN past the last class; block maxima of |coef|.
__global__ void __launch_bounds__(256) coef_kernel(const int32_t* labels, const float* gloss, int64_t M, int64_t V,
                                                   float* coef, float* bmax) {
  __shared__ float red[4];
  float mx = 0.f;
  for (int64_t m = (int64_t)blockIdx.x * 256 + threadIdx.x; m < M; m += (int64_t)gridDim.x * 256) {
    const int32_t y = labels[m];
    const float c = y < 0 ? 0.f : y >= V ? NAN : (gloss ? gloss[m] : 1.f);
    coef[m] = c;
    mx = fmaxf(mx, fabsf(c));
  }
  for (int o = 32; o; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
  __syncthreads();
  if (threadIdx.x == 0) bmax[blockIdx.x] = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

// scal: what G is multiplied by before it is rounded, and the inverse that its
// products are multiplied by.  1 / max |coef|: the rows of a mean loss then have
// label entries p - 1 next to -1, which round to nearly nothing off, where
// coef (p - 1) would round every row's the same way; `top` further on for half
// rows, so that small probabilities stay in range.
__global__ void __launch_bounds__(64) scal_kernel(const float* bmax, int n, float top, float* scal) {
  float mx = 0.f;
  for (int i = threadIdx.x; i < n; i += 64) mx = fmaxf(mx, bmax[i]);
  for (int o = 32; o; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
  if (threadIdx.x == 0) {
    if (!(mx > 0.f)) mx = 1.f;  // no row takes part
    mx = fminf(fmaxf(mx, 0x1p-100f), 0x1p100f);
    scal[0] = top / mx;
    scal[1] = mx / top;
  }
}

// rows of any layout -> [nr][Dp], zeros past D; a thread per 16 bytes.  Only
// for rows that the GEMM's 16-byte loads cannot take (10007 x 515 half: 5.8 us).
template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(RowsArgs R, T* dst, int Dp) {
  constexpr int E = 16 / (int)sizeof(T);
  const int CR = Dp / E;  // Dp: whole chunks
  const int64_t n = R.nr * CR;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n; t += (int64_t)gridDim.x * 256) {
    const int64_t r = t / CR;
    const int c = (int)(t - r * CR) * 16;
    const u32x4 v = chunk_at<T>(R.x + row_offset(R, R.r0 + r) * (int64_t)sizeof(T), c, R.D * (int)sizeof(T));
    *reinterpret_cast<u32x4*>(reinterpret_cast<char*>(dst) + t * 16) = v;
  }
}

// rows of any layout -> [D][ldo] 16-bit (float32: [3] planes of it), zeros past
// nr; rows with live = 0 become zeros.  64 x 64 tiles, 16 bytes a thread in and
// out; bound by memory (32768 x 4096 bf16 twice read and written in 219 us, 4.9 TB/s).
template <typename S>
__global__ void __launch_bounds__(256) transpose_kernel(RowsArgs R, const float* live, char* dst, int64_t ldo) {
  constexpr int E = 16 / (int)sizeof(S), CR = 64 / E;  // elements of a chunk, chunks of a tile row
  __shared__ __attribute__((aligned(16))) S tile[64][64 + E];
  const int64_t r0 = (int64_t)blockIdx.x * 64;
  const int d0 = blockIdx.y * 64;
#pragma unroll
  for (int u = 0; u < 64 * CR / 256; ++u) {
    const int i = threadIdx.x + 256 * u, rr = i / CR, c = i % CR;
    const int64_t r = r0 + rr;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (r < R.nr && !(live && live[r] == 0.f))
      v = chunk_at<S>(R.x + row_offset(R, R.r0 + r) * (int64_t)sizeof(S), (d0 + c * E) * (int)sizeof(S),
                      R.D * (int)sizeof(S));
    *reinterpret_cast<u32x4*>(&tile[rr][c * E]) = v;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = threadIdx.x + 256 * u, d = i / 8, c = i % 8;
    if (d0 + d >= R.D || r0 + c * 8 >= ldo) continue;  // ldo: whole k-tiles
    char* p = dst + ((int64_t)(d0 + d) * ldo + r0 + c * 8) * 2;
    if constexpr (sizeof(S) == 2) {
      S v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = tile[c * 8 + e][d];
      __builtin_memcpy(p, v, 16);
    } else {
      u32x2 w[2][3];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        split4(f32x4{tile[c * 8 + 4 * h][d], tile[c * 8 + 4 * h + 1][d], tile[c * 8 + 4 * h + 2][d], tile[c * 8 + 4 * h + 3][d]},
               w[h]);
#pragma unroll
      for (int l = 0; l < 3; ++l)
        *reinterpret_cast<u32x4*>(p + l * R.D * ldo * 2) = u32x4{w[0][l][0], w[0][l][1], w[1][l][0], w[1][l][1]};
    }
  }
}

// out[r][c] = scale sum_z slab[z][r][c]  (+ out); SL threads share a sum over z
template <typename T, int SL>
__global__ void __launch_bounds__(256) finish_kernel(const float* slab, int splits, int64_t stride, int64_t lds, int64_t M,
                                                     int64_t N, const float* scal, const float* live, T* out,
                                                     int accumulate) {
  constexpr int W = 256 / SL;
  __shared__ f32x4 red[SL == 1 ? 1 : 256];
  const int64_t q = lds / 4, n = M * q;
  const float sc = scal ? scal[1] : 1.f;
  const int sl = threadIdx.x / W;
  for (int64_t t0 = (int64_t)blockIdx.x * W; t0 < n; t0 += (int64_t)gridDim.x * W) {
    const int64_t t = t0 + threadIdx.x % W;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (t < n)  // lds / 4 groups a row: element 4 t of the slab
#pragma unroll 8
      for (int z = sl; z < splits; z += SL) v += *reinterpret_cast<const f32x4*>(slab + z * stride + 4 * t);
    if constexpr (SL > 1) {
      __syncthreads();
      red[threadIdx.x] = v;
      __syncthreads();
      if (sl == 0)
#pragma unroll
        for (int k = 1; k < SL; ++k) v += red[k * W + threadIdx.x];
    }
    if (sl != 0 || t >= n) continue;
    const int64_t r = t / q, c = t % q * 4;
    v = live && live[r] == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : v * sc;
    T* p = out + r * N + c;
    if (N % 4 == 0 && !accumulate) {
      store4<T>(p, v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < N) p[e] = (T)(v[e] + (accumulate ? to_f32(p[e]) : 0.f));
    }
  }
}

// out[n] = scale sum over tile rows of the column sums (+ before[n], the chunks'
// before this one) (+ out[n]); 16 threads a sum
__global__ void __launch_bounds__(256) dbias_kernel(const float* dbp, int tm, int64_t N, const float* scal,
                                                    const float* before, float* out, int add) {
  __shared__ float red[16][16];
  const int c = threadIdx.x & 15, sl = threadIdx.x >> 4;
  const int64_t n = (int64_t)blockIdx.x * 16 + c;
  float v = 0.f;
  if (n < N)
#pragma unroll 8
    for (int t = sl; t < tm; t += 16) v += dbp[(int64_t)t * N + n];
  red[sl][c] = v;
  __syncthreads();
  if (sl == 0 && n < N) {
#pragma unroll
    for (int k = 1; k < 16; ++k) v += red[k][c];
    v *= scal ? scal[1] : 1.f;
    if (before) v += before[n];
    out[n] = add ? out[n] + v : v;
  }
}

// Few tiles over a long k (its parts side by side in float32 slabs, as the OUT
// products write them): what the LSE and GRAD epilogues do, from the slabs.
// Bound by the slabs' bytes and the launch.

// the slabs' sum of 4 logits and their biases, -inf past the last class
__device__ inline f32x4 logits_at(const GemmArgs& P, int64_t m, int64_t n) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  const float* p = P.slab + m * P.lds + n;
#pragma unroll 4
  for (int z = 0; z < P.splits; ++z) v += *reinterpret_cast<const f32x4*>(p + z * P.slab_stride);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = n + e < P.N ? v[e] + (P.bias ? P.bias[P.v0 + n + e] : 0.f) : -INFINITY;
  return v;
}

// L lanes per row and 4 L U classes: their (max, sum), and the label's logit
template <int L, int U>
__global__ void __launch_bounds__(256) slab_lse_kernel(GemmArgs P) {
  const int lane = threadIdx.x % L;
  const int64_t m = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  if (m >= P.M) return;
  const int64_t n0 = (int64_t)blockIdx.y * (4 * L * U);
  const int y = label_at(P, m, n0);
  f32x4 v[U];
  float mx = -INFINITY;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = 4 * (L * u + lane);
    v[u] = n0 + c < P.N ? logits_at(P, m, n0 + c) : f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      mx = fmaxf(mx, v[u][e]);
      if (y == c + e && n0 + c + e < P.N) P.lab[m] = v[u][e];
    }
  }
#pragma unroll
  for (int d = 1; d < L; d *= 2) mx = fmaxf(mx, __shfl_xor(mx, d));
  const float base = mx == -INFINITY ? 0.f : mx;
  float t = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) t += __builtin_amdgcn_exp2f((v[u][e] - base) * kLog2e);
#pragma unroll
  for (int d = 1; d < L; d *= 2) t += __shfl_xor(t, d);
  if (lane == 0) P.part[(int64_t)blockIdx.y * P.M + m] = make_float2(mx, t);
}

// G and its transpose, 128 rows x 64 classes a workgroup (the column sums' row
// tiles), 64 x 64 at a time; a thread holds 4 classes of every 16th row
template <typename S>
__global__ void __launch_bounds__(256) slab_grad_kernel(GemmArgs P) {
  using T = std::conditional_t<sizeof(S) == 4, __bf16, S>;
  constexpr int PL = planes(sizeof(S)), kRow = 72;  // elements of a transposed row in LDS: 64 and 16 bytes
  __shared__ __attribute__((aligned(16))) T tile[PL][64][kRow];
  __shared__ float red[16][64];
  const int tid = threadIdx.x, c = (tid & 15) * 4, r = tid >> 4;
  const int64_t n0 = (int64_t)blockIdx.y * 64;
  const float mult = P.scal ? P.scal[0] : 1.f;
  f32x4 cs = {0.f, 0.f, 0.f, 0.f};
  for (int h = 0; h < 2; ++h) {
    const int64_t m0 = (int64_t)blockIdx.x * 128 + 64 * h;
    if (m0 >= P.M) break;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int ml = 16 * u + r;
      const int64_t m = m0 + ml, n = n0 + c;
      f32x4 g = {0.f, 0.f, 0.f, 0.f};
      const float co = m < P.M ? P.coef[m] : 0.f;
      if (co != 0.f && n < P.N) {  // NaN is live
        const float ls = P.lse[m], cm = co * mult;
        const int y = label_at(P, m, n);
        const f32x4 v = logits_at(P, m, n);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          g[e] = n + e < P.N ? cm * (__builtin_amdgcn_exp2f((v[e] - ls) * kLog2e) - (y == e ? 1.f : 0.f)) : 0.f;
      }
      cs += g;
      u32x2 w[3];
      if constexpr (PL == 1) {
        const T t[4] = {(T)g[0], (T)g[1], (T)g[2], (T)g[3]};
        w[0] = __builtin_bit_cast(u32x2, t);
      } else {
        split4(g, w);
      }
#pragma unroll
      for (int l = 0; l < PL; ++l) {
        if (m < P.M) *reinterpret_cast<u32x2*>(reinterpret_cast<T*>(P.G) + l * P.gp + m * P.ldg + n) = w[l];
        T t[4];
        __builtin_memcpy(t, &w[l], 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) tile[l][c + e][ml] = t[e];
      }
    }
    __syncthreads();
    if (P.GT) {
#pragma unroll
      for (int l = 0; l < PL; ++l)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = tid + 256 * u, nl = i / 8, ch = i % 8;
          if (n0 + nl < P.N)
            *reinterpret_cast<u32x4*>(reinterpret_cast<T*>(P.GT) + l * P.tp + (n0 + nl) * P.ldgt + m0 + ch * 8) =
                *reinterpret_cast<const u32x4*>(&tile[l][nl][ch * 8]);
        }
    }
    __syncthreads();
  }
  if (P.dbp) {
#pragma unroll
    for (int e = 0; e < 4; ++e) red[r][c + e] = cs[e];
    __syncthreads();
    if (tid < 64 && n0 + tid < P.N) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) v += red[k][tid];
      P.dbp[(int64_t)blockIdx.x * P.N + n0 + tid] = v;
    }
  }
}

template <typename T, int MODE>
hipError_t launch_gemm(GemmArgs& P, bool big, hipStream_t s) {
  const int bt = big ? 256 : 128;
  P.tm = (int)((P.M + bt - 1) / bt);
  P.tn = (int)((P.N + bt - 1) / bt);
  const dim3 grid((unsigned)((int64_t)P.tm * P.tn * P.splits));
  if (big) hipLaunchKernelGGL((gemm_kernel<T, 256, 256, 2, 4, MODE>), grid, dim3(512), 0, s, P);
  else hipLaunchKernelGGL((gemm_kernel<T, 128, 128, 2, 2, MODE>), grid, dim3(256), 0, s, P);
  return hipGetLastError();
}

int64_t tiles(int64_t M, int64_t N, int bt) { return ((M + bt - 1) / bt) * ((N + bt - 1) / bt); }
// Tile size and parts of the k axis for a product, by what they would cost in
// multiply-adds of one compute unit: a unit runs one 256 x 256 workgroup at
// full rate, two 128 x 128 at 0.95 of it, one alone at half; a workgroup's start
// and end cost about 256 (512) of k; a part's float32 slab about 4 a value
// (written and read at the memory's rate), a launch for the parts' sum `apart`.
// Parts are 8 k-tiles or longer.
// Measured: 4096 x 1024 over 98304 (float32, six pairs of planes), 256
// workgroups of 128 x 128 1475 us, 64 of 256 x 256 in 4 parts 647; 1000 x 50001
// over 1024, 3128 tiles of 128 x 128 158 us, 784 of 256 x 256 138.
struct Tiling {
  bool big;
  int splits;
  double cost;
};
Tiling tiling(int64_t M, int64_t N, int64_t ktiles, bool parts, double apart = 0.0) {
  Tiling best{true, 1, 1e300};
  for (int big = 1; big >= 0; --big) {
    const int64_t t = tiles(M, N, big ? 256 : 128);
    for (int64_t s = 1; s == 1 || (parts && s <= ktiles / 8 && s <= 32); ++s) {
      const int64_t wg = t * s;
      const double k = 64.0 * (double)((ktiles + s - 1) / s) + (big ? 256.0 : 512.0);
      const double rounds = big ? (double)((wg + kNumCU - 1) / kNumCU) * 65536.0
                            : wg <= kNumCU ? 16384.0 / 0.5
                                           : (double)((wg + 2 * kNumCU - 1) / (2 * kNumCU)) * 2 * 16384.0 / 0.95;
      const double cost = rounds * k + (s > 1 ? apart + 4.0 * (double)s * (double)M * (double)N : 0.0);
      if (cost < best.cost) best = Tiling{big != 0, (int)s, cost};
    }
  }
  return best;
}
unsigned blocks(int64_t n, int64_t cap = 4096) { return (unsigned)std::max<int64_t>(1, std::min((n + 255) / 256, cap)); }

}  // namespace

static int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }
static size_t upz(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// Classes of the logits' first launch: where the 256 x 256 tiles' last round of
// the compute units is nearly empty, the whole rounds', the rest in a launch of
// its own (of smaller tiles mostly).  1000 rows, 50001 classes, 784 tiles over
// D = 1000, half: 146 us at once, 132 so; over D = 4096, bf16, 438 and 362.
// Loss and gradients, both passes so: 5634 x 1456, 5845 classes, float32, 2685
// and 2543 us; 2000 x 1000, 20000 classes, float32, 2244 and 2110.
static int64_t whole_rounds(int64_t M, int64_t V, int64_t ktiles) {
  const int64_t tm = (M + 255) / 256, rounds = tiles(M, V, 256) / kNumCU;
  const int64_t first = rounds * kNumCU / tm * 256;
  if (rounds < 1 || first >= V) return V;
  const double apart = tiling(M, first, ktiles, false).cost + tiling(M, V - first, ktiles, false).cost + 1e7;
  return apart < tiling(M, V, ktiles, false).cost ? first : V;
}

// the logits' parts: G or the (max, sum) pairs from slabs take a launch of about
// 4 us more, at 4.9e6 multiply-adds of a compute unit a us.
// Measured, loss and gradients: 871 x 2563 rows, 517 classes, float32, 35 tiles
// of 128 x 128 whole 571 us, in parts 204; 500 x 4096, 1000 classes, bf16, 138
// and 107; loss of 300 x 4000, 10 classes, float32, 226 and 39.
static void plan_logits(const XentArgs& a, XentPlan& p, int64_t mc, int64_t vcc, size_t& o) {
  p.ldl = up(vcc, 4);
  if (p.few) {
    p.split_l = xent_few_splits((mc + 127) / 128 * ((vcc + 63) / 64), a.D);
    p.slab_l = true;
  } else {
    const Tiling t = tiling(mc, vcc, (p.kbytes + 127) / 128 * (a.es == 4 ? 6 : 1), true, 2e7);
    p.split_l = t.splits;
    p.big_l = t.big;
    p.slab_l = t.splits > 1;
  }
  if (p.slab_l) { p.off_sl = o; o = upz(o + sizeof(float) * (size_t)(p.split_l * mc * p.ldl)); }
}

// what a call does and where its parts of the workspace lie
XentPlan xent_plan(const XentArgs& a, bool grad, bool want_dx, bool want_dw, bool want_db) {
  XentPlan p{};
  const int64_t es = a.es, kt = 64;
  const int64_t pl = es == 4 ? 3 : 1;  // 16-bit planes of an element
  p.kbytes = (int)up(a.D * 2, 16);
  const bool aligned_x = ((uintptr_t)a.x | (uintptr_t)(a.ld * es)) % 16 == 0 && (a.D * es) % 16 == 0 &&
                         a.ld * es * 256 < ((int64_t)1 << 31) && (a.B == 1 || a.stride_b == a.N * a.ld);
  const bool aligned_w = ((uintptr_t)a.w | (uintptr_t)(a.ld_w * es)) % 16 == 0 && (a.D * es) % 16 == 0 &&
                         a.ld_w * es * 256 < ((int64_t)1 << 31);
  p.pack_x = !aligned_x || es == 4;
  p.pack_w = !aligned_w || es == 4;
  p.Dp = up(a.D, 8);
  const int64_t R = std::max<int64_t>(a.B * a.N, 1), V = a.V;
  size_t o = 0;
  p.small = a.D <= 128 && R > 64;
  p.skinny = !grad && !p.small && R <= 64;
  p.few = es == 4 && V <= kFewClasses && !p.small && !p.skinny;
  if (p.few) p.pack_x = false;
  if (p.small) {
    // rows stream past in chunks only where they are copied to aligned rows
    // first (float32: as planes), classes likewise
    p.pack_x = p.pack_x && grad && (want_dw || want_db);
    p.pack_w = p.pack_w && (!grad || want_dx);
    p.nc = p.pack_x ? std::min<int64_t>(R, 1 << 20) : R;
    p.vc = p.pack_w ? std::min<int64_t>(V, 1 << 18) : V;
    p.np_r = (R + p.nc - 1) / p.nc;
    p.np_v = (V + p.vc - 1) / p.vc;
    p.lds = up(a.D, 4);
    if (!grad) {
      p.split_x = xent_small_splits(R, p.vc, a.dtype, a.D, 0);
      if (p.split_x * p.np_v > 1) {
        p.off_part = o; o = upz(o + sizeof(float2) * (size_t)(p.split_x * p.np_v * R));
        p.off_lab = o;  o = upz(o + sizeof(float) * (size_t)R);
      }
    } else {
      p.off_coef = o; o = upz(o + sizeof(float) * (size_t)R);
      p.off_bmax = o; o = upz(o + sizeof(float) * 1024);
      p.off_scal = o; o = upz(o + sizeof(float) * 2);
      if (want_dx) {
        p.split_x = xent_small_splits(R, p.vc, a.dtype, a.D, 1);
        p.slab_x = p.split_x > 1 || p.np_v > 1;
        if (p.slab_x) { p.off_sx = o; o = upz(o + sizeof(float) * (size_t)(p.split_x * R * p.lds)); }
      }
      if (want_dw || want_db) {
        p.split_w = xent_small_splits(V, p.nc, a.dtype, a.D, 2);
        p.slab_w = p.split_w > 1 || p.np_r > 1 || !want_dw;
        if (p.slab_w) { p.off_sw = o; o = upz(o + sizeof(float) * (size_t)(p.split_w * V * p.lds)); }
        if (want_db) { p.off_dbp = o; o = upz(o + sizeof(float) * (size_t)(p.split_w * V)); }
        if (want_db && p.np_r > 1) { p.off_dbr = o; o = upz(o + sizeof(float) * (size_t)V); }
      }
    }
  } else if (!grad) {
    if (p.skinny) p.pack_x = p.pack_w = false;  // it takes any alignment
    // rows of a chunk: at most 2^24 (max, sum) pairs; classes of a piece: all,
    // or 2^15 where they are copied to aligned rows first
    const int64_t per = p.skinny ? 64 : 128;
    p.vc = p.pack_w ? std::min<int64_t>(V, 1 << 15) : V;
    const int64_t nt = (V + per - 1) / per + V / p.vc + 1;
    p.nc = std::min<int64_t>(R, std::max<int64_t>(256, ((int64_t)1 << 24) / nt / 256 * 256));
    if (p.few) p.nc = std::min<int64_t>(p.nc, 1 << 20);
    else if (!p.skinny && p.vc == V) p.vc = whole_rounds(p.nc, V, (p.kbytes + 127) / 128 * (pl == 1 ? 1 : 6));
    p.off_part = o; o = upz(o + sizeof(float2) * (size_t)(nt * p.nc));
    if (!p.skinny) plan_logits(a, p, std::min(p.nc, R), std::min(p.vc, V), o);
    p.off_lab = o;  o = upz(o + sizeof(float) * (size_t)p.nc);
  } else {
    const int64_t cap = (int64_t)1 << (es == 2 ? 27 : 26);
    const int64_t side = 1 << 15;
    const int64_t Rp = up(R, kt), Vp = up(V, kt);
    if (R <= V) {
      p.nc = std::min(Rp, side);
      p.vc = std::min(Vp, std::max<int64_t>(256, cap / p.nc / 256 * 256));
    } else {
      p.vc = std::min(Vp, side);
      p.nc = std::min(Rp, std::max<int64_t>(256, cap / p.vc / 256 * 256));
    }
    p.ldg = up(std::min(p.vc, Vp), kt);
    p.ldgt = up(std::min(p.nc, Rp), kt);
    const int64_t mc = std::min(p.nc, R), vcc = std::min(p.vc, V);
    p.np_v = (V + p.vc - 1) / p.vc;
    p.np_r = (R + p.nc - 1) / p.nc;
    p.lds = up(a.D, 4);
    p.off_coef = o; o = upz(o + sizeof(float) * (size_t)R);
    p.off_bmax = o; o = upz(o + sizeof(float) * 1024);
    p.off_scal = o; o = upz(o + sizeof(float) * 2);
    p.off_G = o;    o = upz(o + (size_t)(mc * p.ldg * 2 * pl));
    plan_logits(a, p, mc, vcc, o);
    if (want_db) { p.off_dbp = o; o = upz(o + sizeof(float) * (size_t)(((mc + 127) / 128) * vcc)); }
    // chunks of rows and pieces of classes both: the larger side in the outer
    // loop finishes its gradients one by one, the smaller side's stay in one
    // float32 slab until the end.  No parts of k beside that slab: a chunk or
    // piece of that side has 2^15 rows, tiles enough.  Against slabs of every row
    // times every part: 200000 x 256 bf16, 50000 classes, 37.5 and 37.2 ms; 60000 x
    // 256, 70000 classes, 14.2 and 14.5; 50000 x 256 float32, 40000 classes, 33.9
    // and 32.7.
    const bool both = p.np_r > 1 && p.np_v > 1;
    p.rows_out = both && R > V;
    p.keep_x = both && !p.rows_out;
    p.keep_w = p.rows_out;
    if (want_db && p.np_r > 1) { p.off_dbr = o; o = upz(o + sizeof(float) * (size_t)(p.rows_out ? V : vcc)); }
    if (want_dx) {
      p.off_WT = o; o = upz(o + (size_t)(a.D * p.ldg * 2 * pl));
      const Tiling t = tiling(mc, a.D, p.ldg / kt * (pl == 1 ? 1 : 6), !p.keep_x);
      p.split_x = t.splits;
      p.big_x = t.big;
      p.slab_x = p.split_x > 1 || p.np_v > 1;
      if (p.slab_x) { p.off_sx = o; o = upz(o + sizeof(float) * (size_t)(p.split_x * (p.keep_x ? R : mc) * p.lds)); }
    }
    if (want_dw) {
      p.off_GT = o; o = upz(o + (size_t)(vcc * p.ldgt * 2 * pl));
      if (!p.few) { p.off_XT = o; o = upz(o + (size_t)(a.D * p.ldgt * 2 * pl)); }
      const Tiling t = tiling(vcc, a.D, p.ldgt / kt * (pl == 1 ? 1 : 6), !p.keep_w);
      p.split_w = t.splits;
      p.big_w = t.big;
      if (p.few) p.split_w = xent_few_splits((a.D + 255) / 256 * ((vcc + 63) / 64), mc);
      p.slab_w = p.few || p.split_w > 1 || p.np_r > 1;
      if (p.slab_w) { p.off_sw = o; o = upz(o + sizeof(float) * (size_t)(p.split_w * (p.keep_w ? V : vcc) * p.lds)); }
    }
  }
  if (p.pack_x) { p.off_px = o; o = upz(o + (size_t)(std::min(p.nc, R) * p.Dp * 2 * pl)); }
  if (p.pack_w) { p.off_pw = o; o = upz(o + (size_t)(std::min(p.vc, V) * p.Dp * 2 * pl)); }
  p.bytes = o;
  return p;
}

namespace {

#define GMM_TRY(call)                                  \
  do {                                                 \
    const hipError_t e_ = (call);                      \
    if (e_ != hipSuccess) return e_;                   \
  } while (0)

template <typename T>
hipError_t finish(const float* slab, int splits, int64_t stride, int64_t lds, int64_t M, int64_t N, const float* scal,
                  const float* live, char* out, int accumulate, hipStream_t s) {
  const int64_t n = M * lds / 4;
  // 16 threads a sum where one would walk 16 slabs or more
  if (splits >= 16)
    hipLaunchKernelGGL((finish_kernel<T, 16>), dim3(blocks(n * 16)), dim3(256), 0, s, slab, splits, stride, lds, M, N, scal,
                       live, reinterpret_cast<T*>(out), accumulate);
  else
    hipLaunchKernelGGL((finish_kernel<T, 1>), dim3(blocks(n)), dim3(256), 0, s, slab, splits, stride, lds, M, N, scal, live,
                       reinterpret_cast<T*>(out), accumulate);
  return hipGetLastError();
}
// rows copied to aligned ones of Dp 16-bit elements (float32: as planes)
template <typename T>
hipError_t pack(const RowsArgs& r, char* dst, int64_t Dp, hipStream_t s) {
  if constexpr (sizeof(T) == 4) return launch_xent_split(r, dst, Dp, s);
  hipLaunchKernelGGL((pack_kernel<T>), dim3(blocks(r.nr * Dp * (int64_t)sizeof(T) / 16, 1 << 16)), dim3(256), 0, s, r,
                     reinterpret_cast<T*>(dst), (int)Dp);
  return hipGetLastError();
}
template <typename T>
hipError_t transpose(const RowsArgs& r, const float* live, char* dst, int64_t ldo, hipStream_t s) {
  const dim3 grid((unsigned)((ldo + 63) / 64), (unsigned)((r.D + 63) / 64));
  hipLaunchKernelGGL((transpose_kernel<T>), grid, dim3(256), 0, s, r, live, dst, ldo);
  return hipGetLastError();
}

// the operands of a chunk of rows against a piece of the head
template <typename T>
hipError_t logit_operands(const XentArgs& a, const XentPlan& p, int64_t r0, int64_t nr, int64_t v0, int64_t nv,
                          char* ws, bool new_rows, bool new_classes, GemmArgs& P, hipStream_t s) {
  const int64_t es = sizeof(T);
  if (p.pack_x) {
    if (new_rows) {
      RowsArgs r{(const char*)a.x, a.N, a.ld, a.stride_b, r0, nr, (int)a.D};
      GMM_TRY(pack<T>(r, ws + p.off_px, p.Dp, s));
    }
    P.A = ws + p.off_px;
    P.lda = p.Dp * 2;
    P.pa = nr * p.Dp * 2;
  } else {
    P.A = (const char*)a.x + r0 * a.ld * es;
    P.lda = a.ld * es;
  }
  if (p.pack_w) {
    if (new_classes) {
      RowsArgs r{(const char*)a.w, a.V, a.ld_w, 0, v0, nv, (int)a.D};
      GMM_TRY(pack<T>(r, ws + p.off_pw, p.Dp, s));
    }
    P.B = ws + p.off_pw;
    P.ldb = p.Dp * 2;
    P.pb = nv * p.Dp * 2;
  } else {
    P.B = (const char*)a.w + v0 * a.ld_w * es;
    P.ldb = a.ld_w * es;
  }
  P.M = nr;
  P.N = nv;
  P.kbytes = p.kbytes;
  P.ktiles = (p.kbytes + 127) / 128 * (sizeof(T) == 4 ? 6 : 1);
  P.splits = 1;
  P.bias = a.bias;
  P.labels = a.labels + r0;
  P.v0 = v0;
  return hipSuccess;
}

FewArgs few_args(const XentArgs& a, int64_t r0, int64_t nr) {
  FewArgs F{};
  F.rows = RowsArgs{(const char*)a.x, a.N, a.ld, a.stride_b, r0, nr, (int)a.D};
  F.flat = a.B == 1 || a.stride_b == a.N * a.ld;
  F.V = (int)a.V;
  return F;
}

// the logits' product in parts, side by side in slabs
template <typename T>
hipError_t logit_slabs(const XentArgs& a, const XentPlan& p, int64_t r0, char* ws, GemmArgs& P, hipStream_t s) {
  P.splits = p.split_l;
  P.slab = reinterpret_cast<float*>(ws + p.off_sl);
  P.lds = p.ldl;
  P.slab_stride = P.M * p.ldl;
  if (!p.few) return launch_gemm<T, OUT>(P, p.big_l, s);
  FewArgs F = few_args(a, r0, P.M);
  F.b = P.B;
  F.ldb = P.ldb;
  F.pb = P.pb;
  F.splits = P.splits;
  F.slab = P.slab;
  F.lds = P.lds;
  F.slab_stride = P.slab_stride;
  return launch_xent_few_logits(F, s);
}

// The bias gradients of a chunk of rows.  The chunks' sum stays in `run` until
// the last of them: what a caller accumulates into is added to once, as dX and
// dW are, and not rounded with every chunk.
hipError_t dbias(const float* dbp, int tm, int64_t N, const float* scal, float* run, float* db, bool first, bool last,
                 int accumulate, hipStream_t s) {
  hipLaunchKernelGGL(dbias_kernel, dim3((unsigned)((N + 15) / 16)), dim3(256), 0, s, dbp, tm, N, scal,
                     first ? (const float*)nullptr : run, last ? db : run, last && accumulate);
  return hipGetLastError();
}

// ---- rows of at most 128 features (gmm_xent_small.hip)
template <typename T>
hipError_t copy_stream(const RowsArgs& r, char* dst, int64_t Dp, SmallArgs& P, hipStream_t s) {
  GMM_TRY(pack<T>(r, dst, Dp, s));
  P.stream = dst;
  P.ld_stream = Dp * 2;
  P.plane = r.nr * Dp * 2;
  return hipSuccess;
}

template <typename T>
hipError_t stream_classes(const XentArgs& a, const XentPlan& p, int64_t v0, int64_t nv, char* ws, SmallArgs& P,
                          hipStream_t s) {
  const int64_t es = sizeof(T);
  P.own = RowsArgs{(const char*)a.x, a.N, a.ld, a.stride_b, 0, a.B * a.N, (int)a.D};
  P.stream = (const char*)a.w + v0 * a.ld_w * es;
  P.ld_stream = a.ld_w * es;
  if (p.pack_w) {
    const RowsArgs r{(const char*)a.w, a.V, a.ld_w, 0, v0, nv, (int)a.D};
    GMM_TRY(copy_stream<T>(r, ws + p.off_pw, p.Dp, P, s));
  }
  P.count = nv;
  P.v0 = v0;
  P.V = a.V;
  P.splits = p.split_x;
  P.bias = a.bias;
  P.labels = a.labels;
  P.w = (const char*)a.w;
  P.ld_w = a.ld_w;
  return hipSuccess;
}

hipError_t join(const float2* part, int64_t nt, int64_t nr, const int32_t* labels, int64_t V, const float* lab,
                float* loss, float* lse, hipStream_t s) {
  if (nr == 1)
    hipLaunchKernelGGL(join_kernel<1>, dim3(1), dim3(256), 0, s, part, nt, nr, labels, V, lab, loss, lse);
  else if (nr <= 4096)
    hipLaunchKernelGGL(join_kernel<16>, dim3((unsigned)((nr + 15) / 16)), dim3(256), 0, s, part, nt, nr, labels, V, lab,
                       loss, lse);
  else
    hipLaunchKernelGGL(join_kernel<64>, dim3((unsigned)((nr + 63) / 64)), dim3(256), 0, s, part, nt, nr, labels, V, lab,
                       loss, lse);
  return hipGetLastError();
}

template <typename T>
hipError_t small_forward(const XentArgs& a, const XentPlan& p, float* loss, float* lse, char* ws, hipStream_t s) {
  const int64_t R = a.B * a.N;
  const bool joined = p.split_x * p.np_v > 1;
  float2* part = reinterpret_cast<float2*>(ws + p.off_part);
  float* lab = reinterpret_cast<float*>(ws + p.off_lab);
  int64_t nt = 0;
  for (int64_t v0 = 0; v0 < a.V; v0 += p.vc) {
    SmallArgs P{};
    GMM_TRY(stream_classes<T>(a, p, v0, std::min(p.vc, a.V - v0), ws, P, s));
    P.part = joined ? part + nt * R : nullptr;
    P.lab = lab;
    P.loss = loss;
    P.lse_out = lse;
    GMM_TRY(launch_xent_small(P, a.dtype, 0, s));
    nt += p.split_x;
  }
  return joined ? join(part, nt, R, a.labels, a.V, lab, loss, lse, s) : hipSuccess;
}

template <typename T>
hipError_t small_backward(const XentArgs& a, const XentPlan& p, const float* lse, const float* coef, const float* scal,
                          char* dx, char* dw, float* db, int accumulate, char* ws, hipStream_t s) {
  const int64_t R = a.B * a.N, es = sizeof(T);
  if (dx) {
    float* slab = p.slab_x ? reinterpret_cast<float*>(ws + p.off_sx) : nullptr;
    for (int64_t v0 = 0; v0 < a.V; v0 += p.vc) {
      SmallArgs P{};
      GMM_TRY(stream_classes<T>(a, p, v0, std::min(p.vc, a.V - v0), ws, P, s));
      P.lse = lse;
      P.coef = coef;
      P.slab = slab;
      P.lds = p.lds;
      P.slab_stride = R * p.lds;
      P.add = v0 > 0;
      P.out = dx;
      P.accumulate = accumulate;
      GMM_TRY(launch_xent_small(P, a.dtype, 1, s));
    }
    if (slab) {
      GMM_TRY(finish<T>(slab, p.split_x, R * p.lds, p.lds, R, a.D, nullptr, coef, dx, accumulate, s));
    }
  }
  if (!dw && !db) return hipSuccess;
  float* slab = p.slab_w ? reinterpret_cast<float*>(ws + p.off_sw) : nullptr;
  for (int64_t r0 = 0; r0 < R; r0 += p.nc) {
    const int64_t nr = std::min(p.nc, R - r0);
    SmallArgs P{};
    P.own = RowsArgs{(const char*)a.w, a.V, a.ld_w, 0, 0, a.V, (int)a.D};
    P.stream = (const char*)a.x;
    P.ld_stream = a.ld * es;
    if (p.pack_x) {
      const RowsArgs r{(const char*)a.x, a.N, a.ld, a.stride_b, r0, nr, (int)a.D};
      GMM_TRY(copy_stream<T>(r, ws + p.off_px, p.Dp, P, s));
    }
    P.count = nr;
    P.V = a.V;
    P.splits = p.split_w;
    P.bias = a.bias;
    P.labels = a.labels + r0;
    P.lse = lse + r0;
    P.coef = coef + r0;
    P.scal = scal;
    P.slab = slab;
    P.lds = p.lds;
    P.slab_stride = a.V * p.lds;
    P.add = r0 > 0;
    P.out = dw;
    P.accumulate = accumulate;
    P.dbp = db ? reinterpret_cast<float*>(ws + p.off_dbp) : nullptr;
    GMM_TRY(launch_xent_small(P, a.dtype, 2, s));
    if (db)  // the column sums were multiplied back already
      GMM_TRY(dbias(P.dbp, p.split_w, a.V, nullptr, accumulate ? reinterpret_cast<float*>(ws + p.off_dbr) : db, db, r0 == 0,
                    r0 + nr >= R, accumulate, s));
  }
  if (slab && dw) {
    GMM_TRY(finish<T>(slab, p.split_w, a.V * p.lds, p.lds, a.V, a.D, nullptr, nullptr, dw, accumulate, s));
  }
  return hipSuccess;
}

template <typename T>
hipError_t forward(const XentArgs& a, const XentPlan& p, float* loss, float* lse, char* ws, hipStream_t s) {
  if (p.small) return small_forward<T>(a, p, loss, lse, ws, s);
  const int64_t R = a.B * a.N;
  float2* part = reinterpret_cast<float2*>(ws + p.off_part);
  float* lab = reinterpret_cast<float*>(ws + p.off_lab);
  for (int64_t r0 = 0; r0 < R; r0 += p.nc) {
    const int64_t nr = std::min(p.nc, R - r0);
    int64_t nt = 0;
    for (int64_t v0 = 0; v0 < a.V; v0 += p.vc) {
      const int64_t nv = std::min(p.vc, a.V - v0);
      GemmArgs P{};
      GMM_TRY(logit_operands<T>(a, p, r0, nr, v0, nv, ws, v0 == 0, p.vc < a.V || r0 == 0, P, s));
      P.part = part + nt * nr;
      P.lab = lab;
      if (p.skinny) {
        P.kbytes = (int)(a.D * (int64_t)sizeof(T));
        P.B = (const char*)a.w;
        P.ldb = a.ld_w * (int64_t)sizeof(T);
        const RowsArgs x{(const char*)a.x, a.N, a.ld, a.stride_b, 0, nr, (int)a.D};
        const dim3 grid((unsigned)((nv + 63) / 64));
        if (nr <= 16) hipLaunchKernelGGL((skinny_kernel<T, 1>), grid, dim3(256), 0, s, P, x);
        else if (nr <= 32) hipLaunchKernelGGL((skinny_kernel<T, 2>), grid, dim3(256), 0, s, P, x);
        else hipLaunchKernelGGL((skinny_kernel<T, 4>), grid, dim3(256), 0, s, P, x);
        GMM_TRY(hipGetLastError());
        nt += grid.x;
      } else if (p.slab_l) {
        GMM_TRY(logit_slabs<T>(a, p, r0, ws, P, s));
        const int L = nv <= 64 ? 16 : 64, span = nv <= 64 ? 64 : 512;
        const dim3 grid((unsigned)((nr + 256 / L - 1) / (256 / L)), (unsigned)((nv + span - 1) / span));
        if (L == 16) hipLaunchKernelGGL((slab_lse_kernel<16, 1>), grid, dim3(256), 0, s, P);
        else hipLaunchKernelGGL((slab_lse_kernel<64, 2>), grid, dim3(256), 0, s, P);
        GMM_TRY(hipGetLastError());
        nt += grid.y;
      } else {
        GMM_TRY((launch_gemm<T, LSE>(P, tiling(nr, nv, P.ktiles, false).big, s)));
        nt += P.tn;
      }
    }
    GMM_TRY(join(part, nt, nr, a.labels + r0, a.V, lab, loss + r0, lse + r0, s));
  }
  return hipSuccess;
}

template <typename T>
hipError_t backward(const XentArgs& a, const XentPlan& p, const float* lse, const float* gloss, char* dx, char* dw,
                    float* db, int accumulate, char* ws, hipStream_t s) {
  const int64_t R = a.B * a.N, es = sizeof(T), kt = 64;
  const int pairs = es == 4 ? 6 : 1;
  float* coef = reinterpret_cast<float*>(ws + p.off_coef);
  float* bmax = reinterpret_cast<float*>(ws + p.off_bmax);
  float* scal = nullptr;
  const unsigned cb = blocks(R, 1024);
  hipLaunchKernelGGL(coef_kernel, dim3(cb), dim3(256), 0, s, a.labels, gloss, R, a.V, coef, bmax);
  GMM_TRY(hipGetLastError());
  if (es == 2) {
    scal = reinterpret_cast<float*>(ws + p.off_scal);
    hipLaunchKernelGGL(scal_kernel, dim3(1), dim3(64), 0, s, bmax, (int)cb, a.dtype == 2 ? 32768.f : 1.f, scal);
    GMM_TRY(hipGetLastError());
  }
  if (p.small) return small_backward<T>(a, p, lse, coef, scal, dx, dw, db, accumulate, ws, s);
  // a chunk of rows against a piece of the classes
  auto part = [&](int64_t r0, int64_t v0) -> hipError_t {
    const int64_t nr = std::min(p.nc, R - r0), nv = std::min(p.vc, a.V - v0);
    const bool new_rows = p.rows_out ? v0 == 0 : p.np_r > 1 || v0 == 0, new_classes = p.rows_out || r0 == 0;
    if (dx && new_classes) {
      RowsArgs r{(const char*)a.w, a.V, a.ld_w, 0, v0, nv, (int)a.D};
      GMM_TRY(transpose<T>(r, nullptr, ws + p.off_WT, up(nv, kt), s));
    }
    GemmArgs P{};
    GMM_TRY(logit_operands<T>(a, p, r0, nr, v0, nv, ws, new_rows, new_classes, P, s));
    P.lse = lse + r0;
    P.coef = coef + r0;
    P.scal = scal;
    P.G = ws + p.off_G;
    P.ldg = P.gcols = up(nv, kt);
    P.GT = dw ? ws + p.off_GT : nullptr;
    P.ldgt = up(nr, kt);
    P.gp = nr * P.ldg;
    P.tp = nv * P.ldgt;
    P.dbp = db ? reinterpret_cast<float*>(ws + p.off_dbp) : nullptr;
    // classes c0 .. c0 + cn of the piece
    auto columns = [&](int64_t c0, int64_t cn) -> hipError_t {
      GemmArgs S = P;
      S.B += c0 * S.ldb;
      S.v0 += c0;
      S.N = cn;
      S.G += c0 * 2;
      S.gcols -= c0;
      if (S.GT) S.GT += c0 * S.ldgt * 2;
      if (S.dbp) S.dbp += (nr + 127) / 128 * c0;
      if (p.slab_l) {
        GMM_TRY(logit_slabs<T>(a, p, r0, ws, S, s));
        const dim3 grid((unsigned)((nr + 127) / 128), (unsigned)(S.gcols / 64));
        hipLaunchKernelGGL(slab_grad_kernel<T>, grid, dim3(256), 0, s, S);
        GMM_TRY(hipGetLastError());
        S.tm = (int)grid.x;
      } else {
        GMM_TRY((launch_gemm<T, GRAD>(S, tiling(nr, cn, S.ktiles, false).big, s)));
      }
      if (db) {
        float *out = db + v0 + c0, *run = reinterpret_cast<float*>(ws + p.off_dbr) + (p.rows_out ? v0 : 0) + c0;
        GMM_TRY(dbias(S.dbp, S.tm, cn, scal, accumulate ? run : out, out, r0 == 0, r0 + nr >= R, accumulate, s));
      }
      return hipSuccess;
    };
    const int64_t first = p.slab_l ? nv : whole_rounds(nr, nv, P.ktiles);
    GMM_TRY(columns(0, first));
    if (first < nv) GMM_TRY(columns(first, nv - first));
    if (dx) {  // dX of the chunk += G W of the piece
      GemmArgs Q{};
      Q.A = P.G;
      Q.lda = P.ldg * 2;
      Q.pa = nr * P.ldg * 2;
      Q.B = ws + p.off_WT;
      Q.ldb = P.ldg * 2;
      Q.pb = a.D * P.ldg * 2;
      Q.M = nr;
      Q.N = a.D;
      Q.kbytes = (int)(P.ldg * 2);
      Q.ktiles = (int)(P.ldg / kt) * pairs;
      Q.splits = std::min<int>(p.split_x, Q.ktiles);
      Q.scal = scal;
      Q.rowlive = coef + r0;
      Q.out = dx + r0 * a.D * es;
      Q.accumulate = accumulate;
      if (p.slab_x) {
        Q.splits = p.split_x;  // every slab is written by the first piece; empty k ranges add zeros
        Q.slab = reinterpret_cast<float*>(ws + p.off_sx) + (p.keep_x ? r0 * p.lds : 0);
        Q.lds = p.lds;
        Q.slab_stride = nr * p.lds;
        Q.add = v0 > 0;
      }
      GMM_TRY((launch_gemm<T, OUT>(Q, p.big_x, s)));
      if (p.slab_x && v0 + nv >= a.V) {
        GMM_TRY(finish<T>(Q.slab, Q.splits, Q.slab_stride, p.lds, nr, a.D, scal, coef + r0, Q.out, accumulate, s));
      }
    }
    if (dw) {  // dW of the piece += G^T X of the chunk
      RowsArgs r{(const char*)a.x, a.N, a.ld, a.stride_b, r0, nr, (int)a.D};
      if (!p.few && new_rows) GMM_TRY(transpose<T>(r, coef + r0, ws + p.off_XT, P.ldgt, s));
      GemmArgs Q{};
      Q.A = P.GT;
      Q.lda = P.ldgt * 2;
      Q.pa = nv * P.ldgt * 2;
      Q.B = ws + p.off_XT;
      Q.ldb = P.ldgt * 2;
      Q.pb = a.D * P.ldgt * 2;
      Q.M = nv;
      Q.N = a.D;
      Q.kbytes = (int)(P.ldgt * 2);
      Q.ktiles = (int)(P.ldgt / kt) * pairs;
      Q.splits = p.split_w;
      Q.scal = scal;
      Q.out = dw + v0 * a.D * es;
      Q.accumulate = accumulate;
      if (p.slab_w) {
        Q.slab = reinterpret_cast<float*>(ws + p.off_sw) + (p.keep_w ? v0 * p.lds : 0);
        Q.lds = p.lds;
        Q.slab_stride = std::min(p.vc, a.V) * p.lds;
        Q.add = r0 > 0;
      }
      if (p.few) {
        FewArgs F = few_args(a, r0, nr);
        F.b = Q.A;
        F.ldb = Q.lda;
        F.pb = Q.pa;
        F.splits = Q.splits;
        F.slab = Q.slab;
        F.lds = Q.lds;
        F.slab_stride = Q.slab_stride;
        F.add = Q.add;
        F.live = coef + r0;
        GMM_TRY(launch_xent_few_dw(F, s));
      } else {
        GMM_TRY((launch_gemm<T, OUT>(Q, p.big_w, s)));
      }
      if (p.slab_w && r0 + nr >= R) {
        GMM_TRY(finish<T>(Q.slab, Q.splits, Q.slab_stride, p.lds, nv, a.D, scal, nullptr, Q.out, accumulate, s));
      }
    }
    return hipSuccess;
  };
  if (p.rows_out) {
    for (int64_t r0 = 0; r0 < R; r0 += p.nc)
      for (int64_t v0 = 0; v0 < a.V; v0 += p.vc) GMM_TRY(part(r0, v0));
  } else {
    for (int64_t v0 = 0; v0 < a.V; v0 += p.vc)
      for (int64_t r0 = 0; r0 < R; r0 += p.nc) GMM_TRY(part(r0, v0));
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_xent(const XentArgs& a, const XentPlan& p, float* loss, float* lse, char* ws, hipStream_t s) {
  if (a.dtype == 1) return forward<__bf16>(a, p, loss, lse, ws, s);
  if (a.dtype == 2) return forward<_Float16>(a, p, loss, lse, ws, s);
  return forward<float>(a, p, loss, lse, ws, s);
}

hipError_t launch_xent_grad(const XentArgs& a, const XentPlan& p, const float* lse, const float* gloss, void* dx, void* dw,
                            float* db, int accumulate, char* ws, hipStream_t s) {
  char *x = (char*)dx, *w = (char*)dw;
  if (a.dtype == 1) return backward<__bf16>(a, p, lse, gloss, x, w, db, accumulate, ws, s);
  if (a.dtype == 2) return backward<_Float16>(a, p, lse, gloss, x, w, db, accumulate, ws, s);
  return backward<float>(a, p, lse, gloss, x, w, db, accumulate, ws, s);
}

}  // namespace gmm
