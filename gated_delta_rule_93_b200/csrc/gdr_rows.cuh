// Helpers of the kernels around the mixer (pooled decode, slot map, output
// norm, prologue): vectors and pairs of elements, sums over the lanes that share
// a row, sums of partial rows, launches that overlap the kernel before them.
#pragma once

#include <cooperative_groups.h>

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
  int turns;  // rows of a slot at most

  __device__ __forceinline__ int group(int block, int slot_in_block, int per_block, int G) const {
    return (unsigned)(by_block ? block : block * per_block + slot_in_block) % (unsigned)G;
  }
  __device__ __forceinline__ long long first_row(int block, int slot_in_block, int per_block,
                                                 int G) const {
    const unsigned q = (unsigned)(by_block ? block : block * per_block + slot_in_block) / (unsigned)G;
    return by_block ? (long long)q * per_block + slot_in_block : q;
  }
  __device__ __forceinline__ bool used(int block, int slot_in_block, int per_block) const {
    return by_block || block * per_block + slot_in_block < slots;
  }
  // The rows of a slot: row `first` and those every `step` after it.  (Only the last turn's can
  // lie behind the end.)
  __device__ __forceinline__ int count(bool used, long long first, long long rows) const {
    return used ? turns - (first + (turns - 1) * step >= rows) : 0;
  }
};

// A plan in which a slot takes about `turns` rows, and at least `least_blocks`
// blocks share the work where there is enough of it.
inline RowPlan row_plan(long long rows, int G, int per_block, int turns, int least_blocks,
                        bool by_block) {
  const long long whole = by_block ? (rows + per_block - 1) / per_block * G
                                   : (rows * G + per_block - 1) / per_block;  // a row a slot
  const long long every = by_block ? G : ((long long)G + per_block - 1) / per_block;
  long long blocks = (whole + turns - 1) / turns;
  if (blocks < least_blocks) {
    blocks = whole < least_blocks ? whole : least_blocks;
    if (by_block) blocks = blocks / G * G;  // (not one block more than fit at once)
  } else if (by_block) {
    blocks = (blocks + G - 1) / G * G;
  }
  if (blocks < every) blocks = every;  // every group once
  if (blocks > 1 << 24) blocks = by_block ? (1 << 24) / G * G : 1 << 24;  // (32-bit slots)
  RowPlan p;
  p.blocks = (int)blocks;
  p.by_block = by_block;
  p.sum = 0;
  p.step = by_block ? blocks / G * per_block : blocks * per_block / G;
  p.slots = by_block ? 0 : (int)(p.step * G);
  p.turns = (int)((rows + p.step - 1) / p.step);
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

// NV accesses of a lane as pairs of elements, in order.
template <typename T, int VEC, int NV>
__device__ __forceinline__ void unpack_row(const Raw<T, VEC> (&raw)[NV],
                                           float2 (&x)[VEC * NV / 2]) {
  static_assert(VEC * NV % 2 == 0);
  float v[VEC * NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) unpack<T, VEC>(raw[i], v + i * VEC);
#pragma unroll
  for (int e = 0; e < VEC * NV / 2; ++e) x[e] = make_float2(v[2 * e], v[2 * e + 1]);
}

// Element j of a lane's pairs.
template <int N>
__device__ __forceinline__ float element(const float2 (&x)[N], int j) {
  return j % 2 ? x[j / 2].y : x[j / 2].x;
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

// Access i of a lane's pairs.
template <typename T, int VEC, int N>
__device__ __forceinline__ void store_access(T *p, const float2 (&x)[N], int i) {
  float v[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) v[e] = element(x, i * VEC + e);
  store_vec<T, VEC>(p, v);
}

// A thread's own queue of loads of R (8 or 16 bytes) in shared memory, STAGES
// rows of N accesses: more bytes in flight than registers have room for.  Only
// the thread that asked for them reads them, so nothing waits at a barrier.
template <typename R, int N, int STAGES>
struct Queue {
  R (*buf)[N][kRowThreads];  // [STAGES] in shared memory

  __device__ __forceinline__ void request(int stage, int i, const void *p) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(&buf[stage][i][threadIdx.x]);
    if constexpr (sizeof(R) == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(p) : "memory");
  }
  // Ends a row's requests (also of a row that has none).
  __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // Waits for all rows but the last STAGES - 1 that were asked for.
  __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
  }
  __device__ __forceinline__ R get(int stage, int i) const { return buf[stage][i][threadIdx.x]; }
};

// The sum over the L lanes (a power of two) that share a row, in all of them.
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
  for (int m = L / 2; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// Two fp32 values in one register pair, worked on by one instruction.
__device__ __forceinline__ unsigned long long bits(float2 x) {
  return *reinterpret_cast<unsigned long long *>(&x);
}
__device__ __forceinline__ float2 pair(unsigned long long x) {
  return *reinterpret_cast<float2 *>(&x);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return pair(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair(d);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The sigmoid of the output norm's activations, on the fast exponential and reciprocal: the
// negated argument is scaled to a power of two in one instruction, whose rounding stays:
// relative error below (4 + |x|) 2^-23 (0 below -87.3, where e^x leaves the normal numbers).
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 t = mul2(x, both(-1.4426950408889634f));  // -log2(e)
  float2 e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  e = add2(e, both(1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
  return e;
}

// e^-|x|, for the gates, whose logits lie far out in earnest: t = -|x| log2(e) is rounded to
// fp32, by up to |t| 2^-24, which ex2 would turn into a relative error that grows with |x|.
// What t leaves out, r = -|x| - t ln(2) in two exact-product steps (Cody and Waite's splitting
// of ln(2)), is small and goes back in as 1 + r: relative error below 2.5 2^-23 for
// every x, 0 from |x| = 87.3 on (2^-126); NaN stays.
__device__ __forceinline__ float2 exp_neg_abs2(float2 x) {
  float2 n, e;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(n.x) : "f"(-fabsf(x.x)), "f"(-104.f));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(n.y) : "f"(-fabsf(x.y)), "f"(-104.f));
  const float2 t = mul2(n, both(1.4426950408889634f));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
  constexpr float kLn2 = 0.693147180559945309f;
  constexpr float kLn2Rest = (float)(0.693147180559945309 - (double)kLn2);
  float2 r = fma2(t, both(-kLn2), n);
  r = fma2(t, both(-kLn2Rest), r);
  return fma2(e, r, e);
}

// 1 / (1 + e^-x), for the write strengths: relative error below 4.5 2^-23.
__device__ __forceinline__ float sigmoid(float x) {
  const float e = exp_neg_abs2(both(x)).x;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return (x >= 0.f ? 1.f : e) * r;
}

// log(1 + e^x) = max(x, 0) + log(1 + e) with e = e^-|x| <= 1, and 1 / (1 + e^-x) from the same e.
// log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3; atanh(s) / s is taken as a polynomial in s^2
// of least relative error on [0, 1/9] with 1 in front (own fit, 4.5e-9): relative error below
// 6 2^-23 for every x (the sigmoid's 4.5 2^-23), in place of log1pf's longer way (a per-channel
// prologue of 8192 x 16 x 128: 64 us with log1pf, 48.8 us; 48.4 us where the rounding of t stays).
__device__ __forceinline__ float2 softplus2(float2 x, float2 *sig = nullptr) {
  const float2 e = exp_neg_abs2(x);
  float2 r;
  const float2 d = add2(e, both(2.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  const float2 s = mul2(e, r), t = mul2(s, s);
  float2 p = fma2(t, both(0.14005993f), both(0.14000903f));
  p = fma2(t, p, both(0.20010763f));
  p = fma2(t, p, both(0.33333209f));
  p = fma2(t, p, both(1.f));
  if (sig) {
    const float2 o = add2(e, both(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(o.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(o.y));
    *sig = mul2(r, make_float2(x.x >= 0.f ? 1.f : e.x, x.y >= 0.f ? 1.f : e.y));
  }
  return fma2(add2(s, s), p, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}
__device__ __forceinline__ float softplus(float x, float *sig = nullptr) {
  float2 both_sig;
  const float2 y = softplus2(both(x), sig ? &both_sig : nullptr);
  if (sig) *sig = both_sig.x;
  return y.x;
}

// Launches `kernel` so that its blocks may be set up while the kernel before it
// on the stream ends.  It has to begin, in every thread, with after_previous(),
// which waits until that kernel is done and its writes are seen: nothing is
// read or written earlier, so the order on the stream is the ordinary one.
// let_next() tells that the kernel behind may be set up in turn.
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t config = {};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, P(args)...);
}
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// out[c] = sum over k of part[k * cols + c], in a fixed order.  A block takes
// kSumWidth columns (32 bytes of a row), a thread every kSumRows-th row of one;
// they add up in a tree.  Many rows are shared by a cluster of kSumParts blocks, whose
// first adds up their sums (2048 rows of 128 columns: 3.3 us less than with one block of
// 1024 threads for 8 columns).
constexpr int kSumThreads = 256, kSumWidth = 8, kSumRows = kSumThreads / kSumWidth;
constexpr int kSumParts = 8, kSumManyRows = 4 * kSumRows;

template <int PARTS>
__device__ __forceinline__ void sum_columns(const float *part, int rows, int cols, float *out) {
  __shared__ float s[kSumThreads];
  const int x = threadIdx.x % kSumWidth, y = threadIdx.x / kSumWidth;
  const int rank = blockIdx.x % PARTS, c = blockIdx.x / PARTS * kSumWidth + x;
  const int step = PARTS * kSumRows;
  float v[4] = {};
  if (c < cols) {
    int k = rank * kSumRows + y;
    for (; k + 3 * step < rows; k += 4 * step)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += part[(size_t)(k + i * step) * cols + c];
    for (; k < rows; k += step) v[0] += part[(size_t)k * cols + c];
  }
  s[threadIdx.x] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
#pragma unroll
  for (int n = kSumThreads / 2; n >= kSumWidth; n >>= 1) {
    if ((int)threadIdx.x < n) s[threadIdx.x] += s[threadIdx.x + n];
    __syncthreads();
  }
  if constexpr (PARTS > 1) {
    const auto cluster = cooperative_groups::this_cluster();
    cluster.sync();
    if (rank == 0 && (int)threadIdx.x < kSumWidth && c < cols) {
      float sum = s[x];
#pragma unroll
      for (int r = 1; r < PARTS; ++r) sum += *cluster.map_shared_rank(&s[x], r);
      out[c] = sum;
    }
    cluster.sync();  // (a block's sums stay until they are read)
  } else if ((int)threadIdx.x < kSumWidth && c < cols) {
    out[c] = s[threadIdx.x];
  }
}

// Columns of `a` from the first `rows` partial rows, and of `b`, where there is one, from the
// next `rows` (the second half of the grid's y).
template <int PARTS>
__global__ void __launch_bounds__(kSumThreads) __cluster_dims__(PARTS, 1, 1)
    sum_kernel(const float *part, int rows, int cols, float *a, float *b) {
  after_previous();
  float *out = blockIdx.y ? b : a;
  if (out) sum_columns<PARTS>(part + (blockIdx.y ? (size_t)rows * cols : 0), rows, cols, out);
}

inline cudaError_t launch_sums(const float *part, int rows, int cols, float *a, float *b,
                               cudaStream_t stream) {
  const int blocks = (cols + kSumWidth - 1) / kSumWidth;
  if (rows > kSumManyRows)
    return launch_next(sum_kernel<kSumParts>, dim3(blocks * kSumParts, b ? 2 : 1), kSumThreads, stream,
                       part, rows, cols, a, b);
  return launch_next(sum_kernel<1>, dim3(blocks, b ? 2 : 1), kSumThreads, stream, part, rows, cols, a,
                     b);
}

}  // namespace gdr
