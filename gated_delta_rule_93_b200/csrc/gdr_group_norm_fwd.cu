// Forward of the output norm (see gdr_group_norm.cuh):
//   n = (x - m) rstd,  l = n w + b,  y = act(z) l  (gated)  or  act(l)
#include "gdr_group_norm.cuh"

namespace gdr {
namespace {

// Rows requested at a time (16 bytes of a tensor a lane), and blocks on an SM, for E elements a lane.
constexpr int rows_ahead(int bytes) { return bytes <= 4 ? 4 : bytes <= 8 ? 2 : 1; }
constexpr int blocks_per_sm(int E) { return E <= 8 ? 4 : E <= 16 ? 2 : 1; }

__device__ __forceinline__ float act_of(int act, float u) {
  if (act == GDR_ACT_NONE) return u;
  const float s = sigmoid(u);
  return act == GDR_ACT_SILU ? u * s : s;
}

template <typename T, int VEC, int L, int NV>
__global__ void __launch_bounds__(kRowThreads, blocks_per_sm(VEC *NV))
    group_norm_fwd_kernel(GroupNormArgs a, RowPlan p) {
  constexpr int E = VEC * NV, U = rows_ahead(E * sizeof(T));
  constexpr bool kAhead = E <= 16;  // (wider rows have no registers for a second one)
  const int lane = threadIdx.x % L;
  constexpr int kPerBlock = kRowThreads / L;
  const int slot = threadIdx.x / L, g = p.group(blockIdx.x, slot, kPerBlock, a.G);
  const float inv_d = 1.f / (float)a.D;
  float w[E], b[E];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * L + lane) * VEC;
    in[i] = c < a.D;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int at = (a.per_channel ? g * a.D : 0) + c + e;
      w[i * VEC + e] = a.weight && in[i] ? a.weight[at] : 1.f;
      b[i * VEC + e] = a.bias && in[i] ? a.bias[at] : 0.f;
    }
  }
  // (all lanes of a warp take every turn: the sums shuffle over whole warps)
  const long long last = p.used(blockIdx.x, slot, kPerBlock) ? a.rows : 0;  // rows of this slot end here
  const T *xp = static_cast<const T *>(a.x) + (long long)g * a.D + lane * VEC;
  const T *zp = static_cast<const T *>(a.z) + (long long)g * a.D + lane * VEC;
  T *yp = static_cast<T *>(a.y) + (long long)g * a.D + lane * VEC;
  const long long turns = (a.rows + U * p.step - 1) / (U * p.step);
  long long row = p.first_row(blockIdx.x, slot, kPerBlock, a.G);
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
  for (long long k = 0; k < turns; ++k) {
    if constexpr (!kAhead) request(row);
    Raw<T, VEC> xr[U][NV], zr[U][NV];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        xr[u][i] = xn[u][i];
        zr[u][i] = zn[u][i];
      }
    if constexpr (kAhead) request(row + U * p.step);
#pragma unroll
    for (int u = 0; u < U; ++u, row += p.step) {
      float x[E], m = 0.f, ss = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) unpack<T, VEC>(xr[u][i], &x[i * VEC]);
      if (a.center) {
#pragma unroll
        for (int e = 0; e < E; ++e) m += x[e];
        m = lanes_sum<L>(m) * inv_d;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float d = x[i * VEC + e] - m;
          x[i * VEC + e] = d;
          ss += in[i] ? d * d : 0.f;
        }
      const float rstd = rsqrtf(lanes_sum<L>(ss) * inv_d + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (row >= last || !in[i]) continue;
        float z[VEC], y[VEC];
        unpack<T, VEC>(zr[u][i], z);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float l = x[i * VEC + e] * rstd * w[i * VEC + e] + b[i * VEC + e];
          y[e] = a.z ? act_of(a.act, z[e]) * l : act_of(a.act, l);
        }
        store_vec<T, VEC>(yp + row * a.G * a.D + i * L * VEC, y);
      }
    }
  }
}

struct Launch {
  const GroupNormArgs &a;
  cudaStream_t stream;
  template <typename T, int VEC, int L, int NV>
  cudaError_t operator()() const {
    const RowPlan p =
        row_plan(a.rows, a.G, kRowThreads / L, kSMs * blocks_per_sm(VEC * NV), false);
    group_norm_fwd_kernel<T, VEC, L, NV><<<p.blocks, kRowThreads, 0, stream>>>(a, p);
    return cudaGetLastError();
  }
};

}  // namespace

cudaError_t launch_group_norm_fwd(const GroupNormArgs &a, cudaStream_t stream) {
  return norm_layout(a, Launch{a, stream});
}

}  // namespace gdr
