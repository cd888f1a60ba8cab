// Forward of the output norm (see gdr_group_norm.cuh):
//   n = (x - m) rstd,  l = n w + b,  y = act(z) l  (gated)  or  act(l)
#include "gdr_group_norm.cuh"

namespace gdr {
namespace {

// Blocks on an SM for E elements a lane in accesses of `vec`.
constexpr int blocks_per_sm(int E, int vec) {
  return E <= 8 ? (vec == 1 ? 3 : 4) : E <= 20 ? 2 : 1;
}
constexpr int kTurns = 8;  // rows of a lane in a block

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
  after_previous();
  let_next();
  constexpr int E = VEC * NV, N = E / 2;  // elements and pairs of a lane
  constexpr int kPerBlock = kRowThreads / L;
  const int lane = threadIdx.x % L;
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
  const long long first = p.first_row(blockIdx.x, slot, kPerBlock, a.G);
  const int mine = p.count(p.used(blockIdx.x, slot, kPerBlock), first, a.rows);
  const long long off = (long long)g * a.D + lane * VEC, dense = (long long)a.G * a.D;
  const T *xp = static_cast<const T *>(a.x) + off + first * a.x_stride;  // the row asked for next
  const T *zp = static_cast<const T *>(a.z) + off + first * a.z_stride;
  T *yp = static_cast<T *>(a.y) + off + first * dense;
  const long long x_step = p.step * a.x_stride, z_step = p.step * a.z_stride;

  constexpr bool kQueue = norm_queue<T, VEC, NV>;
  constexpr int kStages = NV == 1 ? 4 : 3;
  constexpr int kWaiting = kQueue ? 2 * NV : 1;
  __shared__ Raw<T, VEC> waiting[kQueue ? kStages : 1][kWaiting][kRowThreads];
  Queue<Raw<T, VEC>, kWaiting, kStages> queue{waiting};
  const auto ask = [&](int turn, int stage) {
    if (turn < mine) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in[i]) {
          queue.request(stage, i, xp + i * L * VEC);
          if (a.z) queue.request(stage, NV + i, zp + i * L * VEC);
        }
    }
    queue.commit();
    xp += x_step;
    zp += z_step;
  };
  if constexpr (kQueue) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) ask(i, i);
  }
  int stage = 0;
  for (int k = 0; k < p.turns; ++k, yp += p.step * dense) {
    const bool live = k < mine;
    Raw<T, VEC> xr[NV], zr[NV];
    if constexpr (kQueue) {
      ask(k + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
      queue.wait();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xr[i] = zr[i] = Raw<T, VEC>{};
      if (!live || !in[i]) continue;
      if constexpr (kQueue) {
        xr[i] = queue.get(stage, i);
        if (a.z) zr[i] = queue.get(stage, NV + i);
      } else {
        xr[i] = load_raw<T, VEC>(xp + i * L * VEC);
        if (a.z) zr[i] = load_raw<T, VEC>(zp + i * L * VEC);
      }
    }
    if constexpr (kQueue) {
      stage = stage == kStages - 1 ? 0 : stage + 1;
    } else {
      xp += x_step;
      zp += z_step;
    }
    float2 x[N], z[N];
    unpack_row<T, VEC, NV>(xr, x);
    unpack_row<T, VEC, NV>(zr, z);
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
      if (live && in[i]) store_access<T, VEC>(yp + i * L * VEC, x, i);
  }
}

struct Launch {
  const GroupNormArgs &a;
  cudaStream_t stream;
  template <typename T, int VEC, int L, int NV>
  cudaError_t operator()() const {
    const RowPlan p =
        row_plan(a.rows, a.G, kRowThreads / L, kTurns, kSMs * blocks_per_sm(VEC * NV, VEC), false);
    return launch_next(group_norm_fwd_kernel<T, VEC, L, NV>, dim3(p.blocks), kRowThreads, stream, a,
                       p);
  }
};

}  // namespace

cudaError_t launch_group_norm_fwd(const GroupNormArgs &a, cudaStream_t stream) {
  return norm_layout(a, Launch{a, stream});
}

}  // namespace gdr
