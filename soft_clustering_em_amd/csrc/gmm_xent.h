// gmm_xent.h -- device pieces shared by the softmax cross entropy kernels:
// 16-byte fragments into the matrix cores, rows of any layout.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gmm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr unsigned kOutside = 0x80000000u;  // an offset past every resource's end

constexpr int kVm0 = 0x0f70;  // s_waitcnt vmcnt(0): the loads into LDS too

typedef __attribute__((address_space(3))) char lds_char;
// 16 bytes per lane from a buffer straight to LDS: lane l to at + 16 l; an
// offset past the resource's end brings zeros
__device__ inline void load_lds16(__amdgpu_buffer_rsrc_t r, lds_char* at, unsigned offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)at, 16, offset, 0, 0, 0);
}

template <typename T>
__device__ inline float to_f32(T v) {
  return (float)v;
}

// one 16-byte chunk per lane of both operands: acc[n][m] += B[n][:] A[m][:]
template <typename T>
__device__ inline f32x4 mma(u32x4 b, u32x4 a, f32x4 c);
template <>
__device__ inline f32x4 mma<__bf16>(u32x4 b, u32x4 a, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0,
                                                 0);
}
template <>
__device__ inline f32x4 mma<_Float16>(u32x4 b, u32x4 a, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, b), __builtin_bit_cast(f16x8, a), c, 0, 0, 0);
}
template <>
__device__ inline f32x4 mma<float>(u32x4 b, u32x4 a, f32x4 c) {
  // element j of every lane's chunk: k = 4 (lane / 16) + j, the same order in both operands
  const f32x4 bf = __builtin_bit_cast(f32x4, b), af = __builtin_bit_cast(f32x4, a);
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(bf[j], af[j], c, 0, 0, 0);
  return c;
}

// float32 rows enter the matrix cores as three bf16 planes, x = h + m + l, each
// the rounding of what the ones before it leave; of the nine products of two
// such sums the six down to 2^-16 of the largest are taken
constexpr int kPairs[6][2] = {{0, 0}, {0, 1}, {1, 0}, {1, 1}, {0, 2}, {2, 0}};
constexpr int planes(int es) { return es == 4 ? 3 : 1; }

// 4 float32 -> 4 bf16 of each plane
__device__ inline void split4(f32x4 v, u32x2* p) {
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const __bf16 t[4] = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    p[k] = __builtin_bit_cast(u32x2, t);
    if (k < 2)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float r = v[e] - (float)t[e];
        v[e] = __builtin_isfinite(v[e]) ? r : 0.f;  // an infinity or NaN stays in the first plane
      }
  }
}

template <typename T>
__device__ inline void store4(T* p, f32x4 v) {
  T t[4] = {(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
  __builtin_memcpy(p, t, 4 * sizeof(T));  // any alignment of the elements
}

struct RowsArgs {
  const char* x;            // element (b, i, d) at x + es (b stride_b + i ld + d)
  int64_t N, ld, stride_b;  // rows per problem
  int64_t r0, nr;           // rows of this chunk, over all problems
  int D;
};
__device__ inline int64_t row_offset(const RowsArgs& R, int64_t r) {
  return (r / R.N) * R.stride_b + (r % R.N) * R.ld;
}

// chunk k / 16 of a row of `bytes` bytes, zeros past them; any alignment of the elements
template <typename T>
__device__ inline u32x4 chunk_at(const char* row, int k, int bytes) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (k + 16 <= bytes) {
    __builtin_memcpy(&v, row + k, 16);  // any alignment of the elements
  } else if (k < bytes) {
    T t[16 / sizeof(T)];
#pragma unroll
    for (int e = 0; e < 16 / (int)sizeof(T); ++e)
      t[e] = k + e * (int)sizeof(T) < bytes ? reinterpret_cast<const T*>(row + k)[e] : T(0);
    v = __builtin_bit_cast(u32x4, t);
  }
  return v;
}

// Arguments of the kernels for rows of D <= 128 (gmm_xent_small.hip): one
// side's rows stay in registers (the owner's), the other side's stream past.
struct SmallArgs {
  RowsArgs own;            // LSE, DX: the rows; DW: the classes
  const char* stream;      // LSE, DX: classes v0 .. v0 + count of the head; DW: the chunk's rows
  int64_t ld_stream;       // bytes, a multiple of 16
  int64_t plane;           // float32: bytes from one bf16 plane of the stream to the next
  int64_t count;           // streamed rows
  int64_t v0;              // first class of the piece
  int64_t V;
  int tiles_own, splits;
  const float* bias;       // (V) or null
  const int32_t* labels;   // of the rows (of the owner, or streamed)
  const float* lse;
  const float* coef;       // 0: the row takes no part
  const float* scal;       // DW: multiplier of G and its inverse; null: 1
  // LSE
  const char* w;           // the whole head, any alignment
  int64_t ld_w;            // elements
  float2* part;            // [split][rows], null: one split, loss and lse straight
  float* lab;
  float *loss, *lse_out;
  // DX, DW
  float* slab;             // [split][owners][lds] float32, null: straight to out
  int64_t lds, slab_stride;
  int add;
  char* out;
  int accumulate;
  float* dbp;              // DW: [split][owners] column sums of G, null: not wanted
};

// float32 rows -> three bf16 planes [3][nr][Dp]
hipError_t launch_xent_split(const RowsArgs& r, char* dst, int64_t Dp, hipStream_t s);
// passes of launch_xent_small: 0 LSE, 1 DX, 2 DW
hipError_t launch_xent_small(SmallArgs P, int dtype, int pass, hipStream_t s);
int xent_small_rows(int dtype, int64_t D, int pass);  // owner rows of a workgroup
// parts of the streamed side that bring two workgroups to every compute unit,
// each part 4 tiles of 64 rows or longer
int xent_small_splits(int64_t owners, int64_t streamed, int dtype, int64_t D, int pass);

// Arguments of the kernels for wide float32 rows and at most 128 classes
// (gmm_xent_few.hip), 64 a workgroup: above 64 the rows are read twice.  The
// border goes by the classes alone; near it the two ways are within a few percent.
// Loss and gradients here and through tiles of 128 x 128: 65536 x 512, 64
// classes, 332 and 633 us; 20000 x 2000, 64 classes, 414 and 617; 65536 x 512, 128
// classes, 547 and 675; 57491 x 2410, 128 classes, 2453 and 2493; 2000 x 700, 100
// classes, 112 and 109.
constexpr int kFewClasses = 128;
struct FewArgs {
  RowsArgs rows;
  int flat;                // rows of all problems evenly apart: row r at r ld
  const char* b;           // bf16 planes [3][V][..]: logits the head's, dW the transpose of G
  int64_t ldb, pb;         // bytes of a row, of a plane
  int V, splits;           // classes; parts of k (logits: features, dW: rows)
  float* slab;             // logits [split][rows][lds], dW [split][V][lds]
  int64_t lds, slab_stride;
  int add;                 // dW: add to what is there
  const float* live;       // dW: rows with 0 take no part
};
hipError_t launch_xent_few_logits(const FewArgs& P, hipStream_t s);
hipError_t launch_xent_few_dw(const FewArgs& P, hipStream_t s);
int xent_few_splits(int64_t workgroups, int64_t k);

}  // namespace gmm
