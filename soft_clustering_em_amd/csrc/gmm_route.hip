// gmm_route.hip -- scores of E experts turned into the m best codes of a row
// and their weights, and the gradient of the scores.
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),  t_e = s_e + bias_e
//   groups of E / groups experts: the keep_groups with the largest sum of their
//   group_top best t;  the m largest t in them, ties to the lower index
//   w_j = scale s_j / sum_selected s
// Orders are decided in float64; without a bias the order of the scores is that
// of the logits, which are exact.
// L lanes take a row (16 up to 256 experts: four rows a wave).  float32 scores,
// off by at most kOff(t), leave the few candidates that may be among the m
// largest: those not below the m-th largest of the lanes' maxima.  These alone
// are scored in float64, a lane each, and placed by comparing each with every
// other one.  Rows whose groups are too close to tell in float32, or with more
// candidates than places, go through the float64 scores of every expert.
// 65536 x 256 sigmoid in groups, float32, m = 8: 50 us where the bytes take 14 (235 if
// every row takes the float64 scores of all experts); bound
// by instructions, with registers for five waves a SIMD (six 58 us, eight 87:
// spills).  One row: 9 us, latency.
// The gradient forms the scores again from the logits: 100000 x 60 softmax, bf16,
// m = 4: 20 us forward and 20 us gradient.
#include "gmm_device.h"

#include <hip/hip_runtime.h>

#include <float.h>

namespace gmm {

namespace {

// float32 scores and sums with a bias: exp's argument (at most |x| e^x 2^-23 <
// 2^-24), 2^-21 for exp, sum and quotient, the sum's rounding 2^-24 |t|
__device__ inline float kOff(float t) { return 0x1p-20f + 0x1p-23f * fabsf(t); }

template <typename T>
__device__ inline float logit(const RouteArgs& A, int64_t i) {
  return (float)static_cast<const T*>(A.l)[i];
}

__device__ inline int64_t row_base(const RouteArgs& A, int64_t r) {
  const int64_t b = A.stride_b ? (uint32_t)r / (uint32_t)A.N : 0;
  return b * A.stride_b + (r - b * A.N) * A.ld;
}

// 1 / x for x in [1, 2^60]: two Newton steps leave about 1 unit in the last place
__device__ inline double reciprocal(double x) {
  double y = __builtin_amdgcn_rcp(x);
  y = fma(fma(-x, y, 1.0), y, y);
  return fma(fma(-x, y, 1.0), y, y);
}
__device__ inline double sigmoid_f64(double l) {
  const double z = exp_neg(-fabs(l)), y = reciprocal(1.0 + z);
  return l >= 0.0 ? y : z * y;
}

template <int L>
__device__ inline float lanes_max(float v) {
  v = row16_max(v);
  return L == 64 ? rows4_max(v) : v;
}
template <int L>
__device__ inline float lanes_sum(float v) {
  v = row16_sum(v);
  return L == 64 ? rows4_sum(v) : v;
}
template <int L>
__device__ inline double lanes_sum_f64(double v) {
  v = row16_sum_f64(v);
  return L == 64 ? rows4_sum_f64(v) : v;
}

// LDS written by some lanes of a wave, read by others of the same wave
__device__ inline void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// s_e of the code `e` that this lane holds (e < 0: none), over the sum of the
// row's codes (renorm), or over `total`: the largest logit among the codes
// stands for the row's, so that their sum cannot vanish.
template <typename T, int L>
__device__ inline double selected(const RouteArgs& A, int64_t base, int e, float mx, double total) {
  // a NaN, which only a caller's own code can lead to, is switched off like -inf
  const float l = e >= 0 ? fminf(fmaxf(logit<T>(A, base + e), -INFINITY), FLT_MAX) : -INFINITY;
  double q = 0.0;
  if (A.sigmoid) {
    if (e >= 0) q = sigmoid_f64((double)l);
  } else {
    const float top = A.renorm ? lanes_max<L>(l) : mx;
    if (e >= 0) q = exp_neg((double)l - (double)top);
    if (!A.renorm && e >= 0) q /= total;
  }
  if (A.renorm) {
    const double sum = lanes_sum_f64<L>(q);
    q = sum > 0.0 ? q / sum : 0.0;
  }
  return q;
}

// Row r by a whole wave, every score in float64: EPL experts a lane, e = lane +
// 64 k.  row: E doubles of LDS.
template <typename T, int EPL>
__device__ void route_exact(const RouteArgs& A, int64_t r, double* row) {
  const int lane = threadIdx.x & 63;
  const int64_t base = row_base(A, r);
  float l[EPL];
  double t[EPL], s[EPL];
  float mx = -INFINITY;
#pragma unroll
  for (int k = 0; k < EPL; ++k) {
    const int e = lane + 64 * k;
    l[k] = -INFINITY;
    if (e < A.E) {
      const float v = logit<T>(A, base + e);
      if (v > -INFINITY) l[k] = fminf(v, FLT_MAX);
    }
    mx = fmaxf(mx, l[k]);
  }
  mx = rows4_max(row16_max(mx));
  double total = 1.0;
  if (A.sigmoid) {
#pragma unroll
    for (int k = 0; k < EPL; ++k) s[k] = l[k] > -INFINITY ? sigmoid_f64((double)l[k]) : 0.0;
  } else {
    total = 0.0;
#pragma unroll
    for (int k = 0; k < EPL; ++k) {
      s[k] = l[k] > -INFINITY ? exp_neg((double)l[k] - (double)mx) : 0.0;
      total += s[k];
    }
    total = wave_sum(total);
#pragma unroll
    for (int k = 0; k < EPL; ++k) s[k] = l[k] > -INFINITY ? s[k] / total : 0.0;
  }
  const bool by_score = A.bias != nullptr;
#pragma unroll
  for (int k = 0; k < EPL; ++k) {
    const int e = lane + 64 * k;
    t[k] = l[k] > -INFINITY ? (by_score ? fmax(s[k] + (double)A.bias[e], -INFINITY) : (double)l[k]) : -INFINITY;
  }
  if (A.groups > 1 && A.keep < A.groups) {
    const int gs = A.E / A.groups;
#pragma unroll
    for (int k = 0; k < EPL; ++k) {
      const int e = lane + 64 * k;
      if (e < A.E) row[e] = !by_score && A.top == 2 && l[k] > -INFINITY ? s[k] : t[k];
    }
    wave_lds();
    double score = -INFINITY;
    if (lane < A.groups) {
      double best = -INFINITY, next = -INFINITY;
      for (int i = 0; i < gs; ++i) {
        const double v = row[lane * gs + i];
        if (v > best) {
          next = best;
          best = v;
        } else if (v > next) {
          next = v;
        }
      }
      score = A.top == 2 && next > -INFINITY ? best + next : best;
    }
    uint64_t kept = 0;
    for (int i = 0; i < A.keep; ++i) {
      double v = score;
      int g = lane;
      wave_best(v, g);
      kept |= (uint64_t)1 << g;
      if (lane == g) score = -INFINITY;
      if (v == -INFINITY) break;
    }
#pragma unroll
    for (int k = 0; k < EPL; ++k) {
      const int e = lane + 64 * k;
      if (e < A.E && !((kept >> (e / gs)) & 1)) t[k] = -INFINITY;
    }
  }
  int mine = -1;
  for (int j = 0; j < A.m; ++j) {
    double v = -INFINITY;
    int at = 1 << 30;
#pragma unroll
    for (int k = 0; k < EPL; ++k)
      if (t[k] > v) {
        v = t[k];
        at = lane + 64 * k;
      }
    wave_best(v, at);
    if (v == -INFINITY) break;
    if (lane == j) mine = at;
#pragma unroll
    for (int k = 0; k < EPL; ++k)
      if (at == lane + 64 * k) t[k] = -INFINITY;
  }
  const double q = selected<T, 64>(A, base, mine, mx, total);
  if (lane < A.m) {
    A.idx[r * A.m + lane] = mine;
    A.weights[r * A.m + lane] = (float)((double)A.scale * q);
  }
}

constexpr int kPlaces = 64;  // candidates of a row at most

// doubles of LDS a row: its scores, the groups' and what those are off by
// (float32; float64 scores in route_exact, which has a wave's share), or its
// candidates and codes
__host__ __device__ inline int route_room(int E, int groups, int lanes) {
  const int f32 = (E + E / 32 + 1 + 2 * groups + 1) / 2, list = kPlaces * 2 + kRouteMaxM / 2;
  const int scores = groups == 1 ? 0 : lanes == 64 && E > f32 ? E : f32;
  return ((scores > list ? scores : list) + 1) / 2 * 2;
}

// The row's logits, expert sub + L k in l[k]: -inf past E, where there is no row
// and for NaN, at most FLT_MAX.  The loads are made without a branch.
template <typename T, int L, int EPL>
__device__ inline void load_logits(float (&l)[EPL], const T* row, int sub, int E, bool in) {
  T v[EPL];
  if (E == L * EPL) {
#pragma unroll
    for (int k = 0; k < EPL; ++k) v[k] = row[sub + L * k];
  } else {
#pragma unroll
    for (int k = 0; k < EPL; ++k) v[k] = row[min(sub + L * k, E - 1)];
  }
#pragma unroll
  for (int k = 0; k < EPL; ++k) {
    l[k] = fminf(fmaxf((float)v[k], -INFINITY), FLT_MAX);  // NaN gives way to -inf
    if (E != L * EPL && sub + L * k >= E) l[k] = -INFINITY;
    if (!in) l[k] = -INFINITY;
  }
}

// how many of a 16-lane row's lanes hold an `a` that is not below this lane's v
__device__ inline int row_not_below(float a, float v) {
  int n = a >= v;
#define GMM_ROTATED(R) n += dpp_mov<0x120 + R>(a) >= v;
  GMM_ROTATED(1) GMM_ROTATED(2) GMM_ROTATED(3) GMM_ROTATED(4) GMM_ROTATED(5) GMM_ROTATED(6) GMM_ROTATED(7) GMM_ROTATED(8)
  GMM_ROTATED(9) GMM_ROTATED(10) GMM_ROTATED(11) GMM_ROTATED(12) GMM_ROTATED(13) GMM_ROTATED(14) GMM_ROTATED(15)
#undef GMM_ROTATED
  return n;
}
// of the L lanes that take a row
template <int L>
__device__ inline int not_below(float a, float v) {
  if constexpr (L == 16) return row_not_below(a, v);
  // each of the wave's four 16-lane rows to all of them
  int n = 0;
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(a), false, false);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto q = __builtin_amdgcn_permlane32_swap(p[i], p[i], false, false);
    n += row_not_below(__uint_as_float(q[0]), v) + row_not_below(__uint_as_float(q[1]), v);
  }
  return n;
}

// TWO: m is more than half of L.  Registers for as many waves a SIMD as leave the
// least spills: EPL = 16 five, 8 seven (131072 x 128 54 us; six 58), below eight
// (262144 x 64 83 us; seven 86).
template <typename T, int L, int EPL, bool TWO>
__global__ void __launch_bounds__(256, L == 16 ? (EPL == 16 ? 5 : EPL == 8 ? 7 : 8) : 1) route_kernel(RouteArgs A) {
  constexpr int RPW = 64 / L, EXACT = L * EPL > 64 ? L * EPL / 64 : 1;
  extern __shared__ double lds[];  // a wave: RPW rows of `room` doubles
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, sub = lane % L, row = lane / L;
  const int room = route_room(A.E, A.groups, L);
  double* mine_lds = lds + (size_t)(w * RPW + row) * room;
  const int64_t r = A.r0 + ((int64_t)blockIdx.x * 4 + w) * RPW + row;
  const bool in = r < A.R;
  const int64_t base = in ? row_base(A, r) : 0;
  const bool grouped = A.groups > 1 && A.keep < A.groups, by_score = A.bias != nullptr;
  float l[EPL], t[EPL];
  float mx = -INFINITY;
  load_logits<T, L, EPL>(l, static_cast<const T*>(A.l) + base, sub, A.E, in);
  // scores in float32, where the order is not that of the logits; the softmax's
  // sum in float64, where a score itself is asked for
  double total = 1.0;
  const bool need_s = by_score || (grouped && A.top == 2);
  if (!A.sigmoid && (need_s || !A.renorm)) {
#pragma unroll
    for (int k = 0; k < EPL; ++k) mx = fmaxf(mx, l[k]);
    mx = lanes_max<L>(mx);
    total = 0.0;
#pragma unroll
    for (int k = 0; k < EPL; ++k) total += l[k] > -INFINITY ? exp_neg((double)l[k] - (double)mx) : 0.0;
    total = lanes_sum_f64<L>(total);
  }
  const float inv = total > 0.0 ? (float)(1.0 / total) : 0.f;
  const auto score = [&](int k) {
    if (A.sigmoid) return __builtin_amdgcn_rcpf(1.f + __expf(-l[k]));
    return __expf(l[k] - mx) * inv;
  };
#pragma unroll
  for (int k = 0; k < EPL; ++k) t[k] = l[k];
  if (by_score) {
#pragma unroll
    for (int k = 0; k < EPL; ++k) {
      const float v = score(k) + A.bias[min(sub + L * k, A.E - 1)];
      t[k] = l[k] > -INFINITY ? v : -INFINITY;  // NaN, from a NaN bias, is passed over below
    }
  }
  bool unsure = false;
  if (grouped) {
    // the groups' scores from LDS: P lanes a group, each over a run of it.  One
    // place in 33 stays empty, so that runs 32 apart start in other banks.
    float* row_t = reinterpret_cast<float*>(mine_lds);
    const auto at = [](int e) { return e + (e >> 5); };
    float* group_t = row_t + at(A.E);
    float* group_off = group_t + A.groups;
#pragma unroll
    for (int k = 0; k < EPL; ++k) {
      const int e = sub + L * k;
      if (e < A.E) row_t[at(e)] = !by_score && A.top == 2 && l[k] > -INFINITY ? score(k) : t[k];
    }
    wave_lds();
    const int gs = A.E / A.groups;
    int P = 1;
    while (2 * P * A.groups <= L) P *= 2;
    const int run = (gs + P - 1) / P;
    for (int g0 = 0; g0 < A.groups; g0 += L / P) {
      const int g = g0 + sub / P, first = g * gs + sub % P * run;
      const int n = g < A.groups ? min(run, (g + 1) * gs - first) : 0;
      float best = -INFINITY, next = -INFINITY;
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const float v = row_t[at(first + i)];
        next = __builtin_amdgcn_fmed3f(best, next, v);  // of a NaN and two numbers the lower one
        best = fmaxf(best, v);
      }
      for (int o = 1; o < P; o *= 2) {
        const float b = __shfl_xor(best, o), x = __shfl_xor(next, o);
        next = fmaxf(fmaxf(next, x), fminf(best, b));
        best = fmaxf(best, b);
      }
      // a sum is off by what its terms are (biases of either sign may leave it far
      // smaller than they are), and its rounding
      const bool two = A.top == 2 && next > -INFINITY;
      const float v = two ? best + next : best;
      if (g < A.groups) {
        group_t[g] = v;
        group_off[g] = need_s && v > -INFINITY ? kOff(best) + (two ? kOff(next) : 0.f) + 0x1p-22f * fabsf(v) : 0.f;
      }
    }
    wave_lds();
    // the least that a group kept may score and the most that another one may
    float least = INFINITY, most = -INFINITY;
    for (int g0 = 0; g0 < A.groups; g0 += L / P) {
      const int g = g0 + sub / P, first = g * gs + sub % P * run;
      if (g >= A.groups) continue;
      const float v = group_t[g], off = group_off[g];
      int place = 0;
      for (int j = 0; j < A.groups; ++j) {
        const float o = group_t[j];
        place += o > v || (o == v && j < g);
      }
      if (place < A.keep) {
        least = v - off < least ? v - off : v < INFINITY ? least : -INFINITY;
      } else {
        most = fmaxf(most, v + off);
        const int n = min(run, (g + 1) * gs - first);
#pragma unroll 4
        for (int i = 0; i < n; ++i) row_t[at(first + i)] = -INFINITY;
      }
    }
    least = -lanes_max<L>(-least);
    most = lanes_max<L>(most);
    if (need_s) unsure = most > -INFINITY && !(least > most);
    wave_lds();
#pragma unroll
    for (int k = 0; k < EPL; ++k) {
      const int e = sub + L * k;
      if (e < A.E && row_t[at(e)] == -INFINITY) t[k] = -INFINITY;
    }
  }
  // at least m experts are not below the m-th largest of the lanes' maxima, or,
  // where m is more than half the lanes, of their two largest each (with one each
  // the bound would be among the smallest maxima, and hold few experts off: 65536 x
  // 256, m = 16 130 -> 56 us)
  float bound = -FLT_MAX;  // EPL = 1: every expert may be placed
  if constexpr (EPL > 1) {
    float top = -INFINITY, next = -INFINITY;
#pragma unroll
    for (int k = 0; k < EPL; ++k) top = fmaxf(top, t[k]);
    int reach = not_below<L>(top, top);
    if constexpr (TWO) {
      float first = -INFINITY;
#pragma unroll
      for (int k = 0; k < EPL; ++k) {
        next = __builtin_amdgcn_fmed3f(first, next, t[k]);
        first = fmaxf(first, t[k]);
      }
      reach += not_below<L>(next, top);
      if (not_below<L>(top, next) + not_below<L>(next, next) < A.m) next = -INFINITY;
    }
    bound = lanes_max<L>(fmaxf(reach >= A.m ? top : -INFINITY, next));
    if (by_score) bound -= 3.f * kOff(bound);
    bound = fmaxf(bound, -FLT_MAX);
  }
  int count = 0;
#pragma unroll
  for (int k = 0; k < EPL; ++k) count += t[k] >= bound;
  int before = count;
#pragma unroll
  for (int o = 1; o < L; o *= 2) {
    const int x = __shfl_up(before, o, L);
    if (sub >= o) before += x;
  }
  const int n = __shfl(before, L - 1, L);
  before -= count;
  unsure |= n > kPlaces;
  double* list_t = mine_lds;                                        // kPlaces float64 scores,
  int* list_e = reinterpret_cast<int*>(mine_lds + kPlaces);         // their experts,
  float* list_l = reinterpret_cast<float*>(list_e + kPlaces);       // and their logits;
  int* placed = reinterpret_cast<int*>(list_l + kPlaces);           // the m codes
  wave_lds();
  if (n <= kPlaces) {
#pragma unroll
    for (int k = 0; k < EPL; ++k)
      if (t[k] >= bound) {
        list_e[before] = sub + L * k;
        list_l[before++] = l[k];
      }
  }
  wave_lds();
  const int rounds = (n <= kPlaces ? n + L - 1 : 0) / L;  // of L candidates
  // float64 scores where a bias takes part
  for (int s = 0; s < rounds; ++s) {
    const int i = s * L + sub;
    if (i < n) {
      double x = (double)list_l[i];
      if (by_score)
        x = (A.sigmoid ? sigmoid_f64(x) : exp_neg(x - (double)mx) / total) + (double)A.bias[list_e[i]];
      list_t[i] = x;
    }
  }
  wave_lds();
  int e_mine = -1;
  for (int s = 0; s < rounds; ++s) {
    const int i = s * L + sub;
    if (i < n) {
      const double t_i = list_t[i];
      const int e_i = list_e[i];
      int place = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const double o = list_t[j];
        place += o > t_i || (o == t_i && list_e[j] < e_i);
      }
      if (place < A.m) placed[place] = e_i;
    }
  }
  wave_lds();
  if (!unsure && sub < A.m && sub < n) e_mine = placed[sub];
  const double q = selected<T, L>(A, base, e_mine, mx, total);
  if (in && !unsure && sub < A.m) {
    A.idx[r * A.m + sub] = e_mine;
    A.weights[r * A.m + sub] = (float)((double)A.scale * q);
  }
  uint64_t again = __ballot(in && unsure && sub == 0);
  while (again) {
    const int at = __builtin_ctzll(again);
    again &= again - 1;
    wave_lds();
    route_exact<T, EXACT>(A, r - row + at / L, lds + (size_t)w * RPW * room);
  }
}

// L lanes a row.  With u_j = scale dw_j and q_j = s_j / sum_selected s:
//   softmax: dl_e = s_e (ds_e - sum_f ds_f s_f);  sigmoid: dl_e = s_e (1 - s_e) ds_e
// where ds_e = dscores_e, and without renormalising + u_j of the code e; renormalised
// the codes' part is q_j (u_j - sum u q), times 1 - s_j for the sigmoid.
template <typename T, int L, int EPL>
__global__ void __launch_bounds__(256) route_grad_kernel(RouteArgs A) {
  constexpr int RPW = 64 / L;
  const int lane = threadIdx.x & 63, sub = lane % L, row = lane / L;
  const int64_t r = A.r0 + ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * RPW + row;
  const bool in = r < A.R;
  const int64_t base = in ? row_base(A, r) : 0;
  float l[EPL], s[EPL], rest[EPL], ds[EPL], dl[EPL];
  float mx = -INFINITY;
  int mine = in && A.dweights && sub < A.m ? A.idx[r * A.m + sub] : -1;
  float u = mine >= 0 ? A.scale * A.dweights[r * A.m + sub] : 0.f;
  load_logits<T, L, EPL>(l, static_cast<const T*>(A.l) + base, sub, A.E, in);
#pragma unroll
  for (int k = 0; k < EPL; ++k) {
    ds[k] = A.dscores ? A.dscores[min(sub + L * k, A.E - 1)] : 0.f;
    dl[k] = 0.f;
    mx = fmaxf(mx, l[k]);
  }
  mx = lanes_max<L>(mx);
  // a renormalised row without dscores needs no softmax of its own
  const bool need_s = A.dscores || !A.renorm;
  float total = 0.f;
#pragma unroll
  for (int k = 0; k < EPL; ++k) {
    const bool on = l[k] > -INFINITY;
    s[k] = 0.f;
    rest[k] = 1.f;
    if (A.sigmoid) {
      const float z = expf(-fabsf(l[k])), hi = 1.f / (1.f + z), lo = z * hi;
      s[k] = on ? (l[k] >= 0.f ? hi : lo) : 0.f;
      rest[k] = l[k] >= 0.f ? lo : hi;
    } else if (need_s) {
      s[k] = on ? expf(l[k] - mx) : 0.f;
      total += s[k];
    }
  }
  if (!A.sigmoid && need_s) {
    total = lanes_sum<L>(total);
    const float inv = total > 0.f ? 1.f / total : 0.f;
#pragma unroll
    for (int k = 0; k < EPL; ++k) s[k] *= inv;
  }
  if (A.dweights) {
    // the row's leading codes in [0, E)
    const uint64_t bad = __ballot(mine < 0 || mine >= A.E) >> (row * L);
    const int n = __builtin_ctzll(bad | (uint64_t)1 << kRouteMaxM);
    if (sub >= n) mine = -1;
    if (mine < 0) u = 0.f;
    if (A.renorm) {
      const float q = (float)selected<T, L>(A, base, mine, mx, 1.0);
      u = q * (u - lanes_sum<L>(q * u));
    }
#pragma unroll 1
    for (int j = 0; j < A.m; ++j) {
      const int e = __shfl(mine, j, L) - sub;
      const float v = __shfl(u, j, L);
#pragma unroll
      for (int k = 0; k < EPL; ++k) dl[k] += e == L * k ? v : 0.f;
    }
#pragma unroll
    for (int k = 0; k < EPL; ++k) {
      if (!A.renorm) ds[k] += dl[k];
      dl[k] = A.renorm ? dl[k] * rest[k] : 0.f;
    }
  }
  float c = 0.f;
  if (!A.sigmoid && need_s) {
#pragma unroll
    for (int k = 0; k < EPL; ++k) c += s[k] > 0.f ? ds[k] * s[k] : 0.f;
    c = lanes_sum<L>(c);
  }
  if (!in) return;
#pragma unroll
  for (int k = 0; k < EPL; ++k) {
    const int e = sub + L * k;
    if (e >= A.E) break;
    const float d = l[k] > -INFINITY ? dl[k] + s[k] * rest[k] * (ds[k] - c) : 0.f;
    static_cast<T*>(A.dlogits)[r * A.E + e] = (T)d;
  }
}

}  // namespace

template <typename T, int L, int EPL>
static hipError_t run_route(RouteArgs A, bool grad, hipStream_t s) {
  constexpr int rows = 4 * (64 / L);
  constexpr bool two = L == 16 && EPL > 1;
  const size_t lds = sizeof(double) * rows * route_room(A.E, A.groups, L);
  for (const int64_t step = kLaunchThreads / L; A.r0 < A.R; A.r0 += step) {
    const int64_t n = A.R - A.r0 < step ? A.R - A.r0 : step;
    const dim3 grid((unsigned)((n + rows - 1) / rows)), block(256);
    if (grad) hipLaunchKernelGGL((route_grad_kernel<T, L, EPL>), grid, block, 0, s, A);
    else if (two && A.m > L / 2) hipLaunchKernelGGL((route_kernel<T, L, EPL, two>), grid, block, lds, s, A);
    else hipLaunchKernelGGL((route_kernel<T, L, EPL, false>), grid, block, lds, s, A);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Sixteen lanes a row where they hold it, 16 experts each, a wave else (by a wave:
// 65536 x 256 134 us against 52 to 56, 131072 x 128 143 against 41, 100000 x 60 153
// against 19).
template <typename T>
static hipError_t run_routes(const RouteArgs& A, bool grad, hipStream_t s) {
  if (A.E <= 16) return run_route<T, 16, 1>(A, grad, s);
  if (A.E <= 32) return run_route<T, 16, 2>(A, grad, s);
  if (A.E <= 64) return run_route<T, 16, 4>(A, grad, s);
  if (A.E <= 128) return run_route<T, 16, 8>(A, grad, s);
  if (A.E <= 256) return run_route<T, 16, 16>(A, grad, s);
  if (A.E <= 512) return run_route<T, 64, 8>(A, grad, s);
  return run_route<T, 64, 16>(A, grad, s);
}

hipError_t launch_route(const RouteArgs& A, int dtype, bool grad, hipStream_t s) {
  if (dtype == 0) return run_routes<float>(A, grad, s);
  if (dtype == 1) return run_routes<__bf16>(A, grad, s);
  return run_routes<_Float16>(A, grad, s);
}

}  // namespace gmm
