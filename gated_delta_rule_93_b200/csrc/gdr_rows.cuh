// Helpers of the row-wise kernels (output norm, prologue): vectors of
// elements, sums over the lanes that share a row, sums of partial rows.
#pragma once

#include "gdr_internal.cuh"

namespace gdr {

constexpr int kSMs = 148;
constexpr int kRowThreads = 256;

// How the rows of G groups (heads) each are spread over a grid: slots of
// lanes take a group each and keep it for all their rows, `step` apart.
//   by slot:  consecutive slots take consecutive groups;
//   by block: the slots of a block share a group (sums over rows then end in
//             one value a block and channel).
struct RowPlan {
  int blocks;
  int slots;  // in use (by slot: a multiple of G)
  int by_block;
  int sum;  // whether partial rows are left for a second launch
  long long step;

  __device__ __forceinline__ int group(int block, int slot_in_block, int per_block, int G) const {
    return by_block ? block % G : (block * per_block + slot_in_block) % G;
  }
  __device__ __forceinline__ long long first_row(int block, int slot_in_block, int per_block,
                                                 int G) const {
    return by_block ? (long long)(block / G) * per_block + slot_in_block
                    : (block * per_block + slot_in_block) / G;
  }
  __device__ __forceinline__ bool used(int block, int slot_in_block, int per_block) const {
    return by_block || block * per_block + slot_in_block < slots;
  }
};

inline RowPlan row_plan(long long rows, int G, int per_block, int max_blocks, bool by_block) {
  const long long least = by_block ? G : ((long long)G + per_block - 1) / per_block;
  long long blocks = by_block ? (rows + per_block - 1) / per_block * G
                              : (rows * G + per_block - 1) / per_block;
  if (blocks > max_blocks) blocks = by_block ? max_blocks / G * G : max_blocks;
  if (blocks < least) blocks = least;  // every group once
  RowPlan p;
  p.blocks = (int)blocks;
  p.by_block = by_block;
  p.sum = 0;
  p.step = by_block ? blocks / G * per_block : blocks * per_block / G;
  p.slots = (int)(by_block ? blocks * per_block : p.step * G);
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

// Fast exponential and reciprocal: relative error below (4 + |x|) 2^-23, a few
// instructions instead of about thirty.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// log(1 + e^x), with no branch that overflows, and 1 / (1 + e^-x) from the same exponential.
__device__ __forceinline__ float softplus(float x, float *sig = nullptr) {
  const float e = __expf(-fabsf(x));
  if (sig) *sig = __fdividef(x >= 0.f ? 1.f : e, 1.f + e);
  return fmaxf(x, 0.f) + log1pf(e);
}

// out[c] = sum over k of part[k * cols + c], in a fixed order.  A block of 1024
// threads takes W columns (a power of two up to 32, fewer where there are
// few columns, so that more threads share one) and adds up in a tree.
__host__ __device__ __forceinline__ int sum_width(int cols) {
  return cols <= 4 ? 4 : cols <= 8 ? 8 : cols <= 16 ? 16 : 32;
}
__device__ __forceinline__ void sum_columns(const float *part, int rows, int cols, float *out,
                                            int block) {
  __shared__ float s[1024];
  const int W = sum_width(cols), Y = 1024 / W;
  const int x = threadIdx.x % W, y = threadIdx.x / W;
  const int c = block * W + x;
  float v[4] = {};
  if (c < cols) {
    int k = y;
    for (; k + 3 * Y < rows; k += 4 * Y)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += part[(size_t)(k + i * Y) * cols + c];
    for (; k < rows; k += Y) v[0] += part[(size_t)k * cols + c];
  }
  s[threadIdx.x] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  for (int n = 512; n >= W; n >>= 1) {
    if ((int)threadIdx.x < n) s[threadIdx.x] += s[threadIdx.x + n];
    __syncthreads();
  }
  if ((int)threadIdx.x < W && c < cols) out[c] = s[threadIdx.x];
}

}  // namespace gdr
