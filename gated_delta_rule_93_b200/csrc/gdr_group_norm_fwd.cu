// Forward of the output norm (see gdr_group_norm.cuh):
//   n = (x - m) rstd,  l = n w + b,  y = act(z) l  (gated)  or  act(l)
#include "gdr_group_norm.cuh"

namespace gdr {
namespace {

// Rows requested at a time (16 bytes of a tensor a lane), and blocks on an SM, for E elements a lane.
constexpr int rows_ahead(int bytes) { return bytes <= 4 ? 4 : bytes <= 8 ? 2 : 1; }
constexpr int blocks_per_sm(int E, int vec) {
  return E <= 8 ? (vec == 1 ? 3 : 4) : E <= 20 ? 2 : 1;
}

constexpr int kTurns = 8;

// y of N pairs in place of x: x are normalised but for rstd.
template <int ACT, bool GATED, int N>
__device__ __forceinline__ void finish(float2 (&x)[N], const float2 (&z)[N], const float2 (&w)[N],
                                       const float2 (&b)[N], float rstd) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float2 l = fma2(mul2(x[e], both(rstd)), w[e], b[e]);
    const float2 u = GATED ? z[e] : l;
    float2 f = u;
    if constexpr (ACT != GDR_ACT_NONE) f = sigmoid2(u);
    if constexpr (ACT == GDR_ACT_SILU) f = mul2(f, u);
    x[e] = GATED ? mul2(f, l) : f;
  }
}

template <typename T, int VEC, int L, int NV>
__global__ void __launch_bounds__(kRowThreads, blocks_per_sm(VEC *NV, VEC))
    group_norm_fwd_kernel(GroupNormArgs a, RowPlan p) {
  constexpr int E = VEC * NV, U = rows_ahead(E * sizeof(T));
  constexpr int N = E / 2;  // pairs of a lane
  constexpr bool kQueue = sizeof(Raw<T, VEC>) == 16 && NV == 1;
  // (single elements and wide rows have no registers for a second one)
  constexpr bool kAhead = !kQueue && VEC > 1 && E <= 16;
  const int lane = threadIdx.x % L;
  constexpr int kPerBlock = kRowThreads / L;
  const int slot = threadIdx.x / L, g = p.group(blockIdx.x, slot, kPerBlock, a.G);
  const float inv_d = 1.f / (float)a.D;
  constexpr bool kKeep = E <= 8;  // wider rows take their weights from L1 each time
  float2 w[N], b[N];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = (i * L + lane) * VEC < a.D;
  const auto affine = [&] {
    const int c = (a.per_channel ? g * a.D : 0) + lane * VEC;
    load_affine<VEC, L, NV>(a.weight, c, in, 1.f, w);
    load_affine<VEC, L, NV>(a.bias, c, in, 0.f, b);
  };
  if constexpr (kKeep) affine();
  // (all lanes of a warp take every turn: the sums shuffle over whole warps)
  const long long last = p.used(blockIdx.x, slot, kPerBlock) ? a.rows : 0;  // rows of this slot end here
  const T *xp = static_cast<const T *>(a.x) + (long long)g * a.D + lane * VEC;
  const T *zp = static_cast<const T *>(a.z) + (long long)g * a.D + lane * VEC;
  T *yp = static_cast<T *>(a.y) + (long long)g * a.D + lane * VEC;
  const long long turns = (a.rows + U * p.step - 1) / (U * p.step);
  long long row = p.first_row(blockIdx.x, slot, kPerBlock, a.G);
  // 16-byte accesses wait in shared memory, 4 rows of them; others a turn ahead in registers.
  constexpr int kStages = 4;
  __shared__ uint4 waiting[kQueue ? kStages : 1][2][kRowThreads];
  Queue<2, kStages> queue{waiting};
  const auto ask = [&](long long at, int stage) {
    if (at < last && in[0]) {
      queue.request(stage, 0, xp + at * a.x_stride);
      if (a.z) queue.request(stage, 1, zp + at * a.z_stride);
    }
    queue.commit();
  };
  Raw<T, VEC> xn[U][NV], zn[U][NV];  // the next turn's rows
  const auto request = [&](long long from) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const long long at = from + u * p.step;
        xn[u][i] = zn[u][i] = Raw<T, VEC>{};
        if (at < last && in[i]) {
          xn[u][i] = load_raw<T, VEC>(xp + at * a.x_stride + i * L * VEC);
          if (a.z) zn[u][i] = load_raw<T, VEC>(zp + at * a.z_stride + i * L * VEC);
        }
      }
  };
  if constexpr (kAhead) request(row);
  if constexpr (kQueue) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) ask(row + i * p.step, i);
  }
  int stage = 0;
  for (long long k = 0; k < turns; ++k) {
    Raw<T, VEC> xr[U][NV], zr[U][NV];
    if constexpr (kQueue) {
      ask(row + (kStages - 1) * p.step, stage == 0 ? kStages - 1 : stage - 1);
      queue.wait();
      const bool live = row < last && in[0];
      const uint4 x16 = live ? queue.get(stage, 0) : uint4{};
      const uint4 z16 = live && a.z ? queue.get(stage, 1) : uint4{};
      xr[0][0] = *reinterpret_cast<const Raw<T, VEC> *>(&x16);
      zr[0][0] = *reinterpret_cast<const Raw<T, VEC> *>(&z16);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    } else {
      if constexpr (!kAhead) request(row);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          xr[u][i] = xn[u][i];
          zr[u][i] = zn[u][i];
        }
      if constexpr (kAhead) request(row + U * p.step);
    }
#pragma unroll
    for (int u = 0; u < U; ++u, row += p.step) {
      float2 x[N], z[N];
      unpack_row<T, VEC, NV>(xr[u], x);
      unpack_row<T, VEC, NV>(zr[u], z);
      const float rstd = normalise<VEC, L, NV>(x, in, a.center, inv_d, a.eps);
      if constexpr (!kKeep) affine();
      if (a.z) {
        if (a.act == GDR_ACT_SILU) finish<GDR_ACT_SILU, true>(x, z, w, b, rstd);
        else if (a.act == GDR_ACT_SIGMOID) finish<GDR_ACT_SIGMOID, true>(x, z, w, b, rstd);
        else finish<GDR_ACT_NONE, true>(x, z, w, b, rstd);
      } else {
        if (a.act == GDR_ACT_SILU) finish<GDR_ACT_SILU, false>(x, z, w, b, rstd);
        else if (a.act == GDR_ACT_SIGMOID) finish<GDR_ACT_SIGMOID, false>(x, z, w, b, rstd);
        else finish<GDR_ACT_NONE, false>(x, z, w, b, rstd);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (row < last && in[i])
          store_access<T, VEC>(yp + row * a.G * a.D + i * L * VEC, x, i);
    }
  }
}

struct Launch {
  const GroupNormArgs &a;
  cudaStream_t stream;
  template <typename T, int VEC, int L, int NV>
  cudaError_t operator()() const {
    const RowPlan p =
        row_plan(a.rows, a.G, kRowThreads / L, kTurns, kSMs * blocks_per_sm(VEC * NV, VEC), false);
    group_norm_fwd_kernel<T, VEC, L, NV><<<p.blocks, kRowThreads, 0, stream>>>(a, p);
    return cudaGetLastError();
  }
};

}  // namespace

cudaError_t launch_group_norm_fwd(const GroupNormArgs &a, cudaStream_t stream) {
  return norm_layout(a, Launch{a, stream});
}

}  // namespace gdr
