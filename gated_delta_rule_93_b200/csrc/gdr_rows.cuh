// Helpers of the row-wise kernels (output norm, prologue): vectors of
// elements, sums over the lanes that share a row, sums of partial rows.
#pragma once

#include "gdr_internal.cuh"

namespace gdr {

constexpr int kSMs = 148;
constexpr int kRowThreads = 256;

// Rows of G groups (heads) each, spread over `slots` slots of lanes; a slot
// keeps its group for all its rows, which are `step` apart.
struct RowPlan {
  int blocks, slots;
  long long step;  // rows between a slot's groups
};

inline RowPlan row_plan(long long rows, int G, int per_block, int max_blocks) {
  const long long want = (rows * G + per_block - 1) / per_block;
  const long long least = ((long long)G + per_block - 1) / per_block;  // every group once
  long long blocks = want < max_blocks ? want : max_blocks;
  if (blocks < least) blocks = least;
  if (blocks < 1) blocks = 1;
  RowPlan p;
  p.blocks = (int)blocks;
  p.step = blocks * per_block / G;
  p.slots = (int)(p.step * G);
  return p;
}

// VEC consecutive elements of type T: one access of `Raw`, unpacked to floats
// where they are used (a row waits in half the registers as bf16).
template <int BYTES>
struct Bits;
template <> struct Bits<2> { using T = unsigned short; };
template <> struct Bits<4> { using T = unsigned int; };
template <> struct Bits<8> { using T = uint2; };
template <> struct Bits<16> { using T = uint4; };
template <typename T, int VEC>
using Raw = typename Bits<sizeof(T) * VEC>::T;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float &d, float x) { d = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16 &d, float x) { d = __float2bfloat16_rn(x); }

// A load of data that is read once (it need not stay in L1).
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T *p) {
  return __ldcs(reinterpret_cast<const Raw<T, VEC> *>(p));
}

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Raw<T, VEC> &raw, float *x) {
  union {
    Raw<T, VEC> b;
    T t[VEC];
  } u;
  u.b = raw;
#pragma unroll
  for (int e = 0; e < VEC; ++e) x[e] = to_f(u.t[e]);
}

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float *x) {
  unpack<T, VEC>(load_raw<T, VEC>(p), x);
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float *x) {
  union {
    Raw<T, VEC> b;
    T t[VEC];
  } u;
#pragma unroll
  for (int e = 0; e < VEC; ++e) from_f(u.t[e], x[e]);
  *reinterpret_cast<Raw<T, VEC> *>(p) = u.b;
}

// The sum over the L lanes (a power of two) that share a row, in all of them.
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int m = L / 2; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }
// The same from the fast exponential and reciprocal: relative error below (4 + |x|) 2^-23,
// a few instructions instead of about thirty.
__device__ __forceinline__ float fast_sigmoid(float x) {
  return __fdividef(1.f, 1.f + __expf(-x));
}
// log(1 + e^x), with no branch that overflows.
__device__ __forceinline__ float softplus(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

// out[c] = sum over k of part[k * cols + c], in a fixed order: a block takes
// 32 columns, its 32 row threads every 32nd row each, then one thread a column.
__device__ __forceinline__ void sum_columns(const float *part, int rows, int cols, float *out,
                                            int block) {
  __shared__ float s[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = block * 32 + x;
  float v = 0.f;
  if (c < cols)
    for (int k = y; k < rows; k += 32) v += part[(size_t)k * cols + c];
  s[y][x] = v;
  __syncthreads();
  if (y == 0) {
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += s[k][x];
    if (c < cols) out[c] = v;
  }
}

}  // namespace gdr
