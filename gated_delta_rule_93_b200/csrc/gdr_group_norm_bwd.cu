// Backward of the output norm (see gdr_group_norm.cuh):
//   dl = dy act(z) or dy act'(l),  dz = dy l act'(z),  h = dl w
//   dx = rstd (h - [center] mean(h) - n mean(h n)),  dw = sum dl n,  db = sum dl
//
// The statistics are computed again from x, which is read anyway.  The weight
// gradients add up in registers over a lane's rows; then each block (weights
// shared by the groups) or each row slot (weights per channel) writes one
// partial row, and a second launch adds the partial rows in a fixed order.
#include "gdr_group_norm.cuh"

namespace gdr {
namespace {

// Rows in flight and blocks on an SM for E elements a lane.
constexpr int rows_ahead(int E) { return E <= 8 ? 2 : 1; }
constexpr int blocks_per_sm(int E) { return E <= 8 ? 2 : 1; }

// Value and slope of the activation.
__device__ __forceinline__ void act_both(int act, float u, float &f, float &df) {
  if (act == GDR_ACT_NONE) {
    f = u;
    df = 1.f;
    return;
  }
  const float s = fast_sigmoid(u);
  if (act == GDR_ACT_SILU) {
    f = u * s;
    df = s + f * (1.f - s);
  } else {
    f = s;
    df = s * (1.f - s);
  }
}

template <typename T, int VEC, int L, int NV>
__global__ void __launch_bounds__(kRowThreads, blocks_per_sm(VEC *NV))
    group_norm_bwd_kernel(GroupNormArgs a, RowPlan p) {
  constexpr int E = VEC * NV, U = rows_ahead(E);
  constexpr int kPerBlock = kRowThreads / L;
  const int lane = threadIdx.x % L;
  const int slot = blockIdx.x * kPerBlock + threadIdx.x / L;
  const int g = slot % a.G;
  const float inv_d = 1.f / (float)a.D;
  float w[E], b[E], dw[E], db[E];
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
      dw[i * VEC + e] = db[i * VEC + e] = 0.f;
    }
  }
  const long long last = slot < p.slots ? a.rows : 0;  // rows of this slot end here
  const long long off = (long long)g * a.D + lane * VEC, dense = (long long)a.G * a.D;
  const T *xp = static_cast<const T *>(a.x) + off, *zp = static_cast<const T *>(a.z) + off;
  const T *dyp = static_cast<const T *>(a.dy) + off;
  const long long turns = (a.rows + U * p.step - 1) / (U * p.step);
  long long row = slot / a.G;
  for (long long k = 0; k < turns; ++k) {
    Raw<T, VEC> xr[U][NV], zr[U][NV], dyr[U][NV];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const long long at = row + u * p.step;
        xr[u][i] = zr[u][i] = dyr[u][i] = Raw<T, VEC>{};
        if (at < last && in[i]) {
          xr[u][i] = load_raw<T, VEC>(xp + at * a.x_stride + i * L * VEC);
          dyr[u][i] = load_raw<T, VEC>(dyp + at * dense + i * L * VEC);
          if (a.z) zr[u][i] = load_raw<T, VEC>(zp + at * a.z_stride + i * L * VEC);
        }
      }
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
      float h[E], sh = 0.f, shn = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float z[VEC], dy[VEC], dz[VEC];
        unpack<T, VEC>(zr[u][i], z);
        unpack<T, VEC>(dyr[u][i], dy);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int j = i * VEC + e;
          const float n = x[j] * rstd;
          const float l = n * w[j] + b[j];
          float f, df;
          act_both(a.act, a.z ? z[e] : l, f, df);
          const float dl = dy[e] * (a.z ? f : df);
          dz[e] = dy[e] * l * df;
          // (dy is zero outside the group and the rows: so are all of these)
          dw[j] += dl * n;
          db[j] += dl;
          h[j] = dl * w[j];
          x[j] = n;
          sh += h[j];
          shn += h[j] * n;
        }
        if (a.dz && row < last && in[i])
          store_vec<T, VEC>(static_cast<T *>(a.dz) + off + row * dense + i * L * VEC, dz);
      }
      shn = lanes_sum<L>(shn) * inv_d;
      sh = a.center ? lanes_sum<L>(sh) * inv_d : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (row >= last || !in[i]) continue;
        float d[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          d[e] = rstd * (h[i * VEC + e] - sh - x[i * VEC + e] * shn);
        constexpr int V4 = VEC < 4 ? VEC : 4;
#pragma unroll
        for (int e = 0; e < VEC; e += V4)
          store_vec<float, V4>(a.dx + off + row * dense + i * L * VEC + e, d + e);
      }
    }
  }

  // Partial rows of the weight gradients, db behind dw.
  if (!a.dweight && !a.dbias) return;
  if (a.per_channel) {  // [step][G D]
    if (slot < p.slots) {
      float *pw = a.ws + (long long)slot * a.D;
      float *pb = pw + p.step * a.G * a.D;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (in[i]) {
            pw[(i * L + lane) * VEC + e] = dw[i * VEC + e];
            pb[(i * L + lane) * VEC + e] = db[i * VEC + e];
          }
    }
  } else {  // [blocks][D]
    __shared__ float s[kRowThreads];
    float *pw = a.ws + (long long)blockIdx.x * a.D;
    float *pb = pw + (long long)p.blocks * a.D;
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        __syncthreads();
        s[threadIdx.x] = which ? db[e] : dw[e];
        __syncthreads();
        if (threadIdx.x < L) {
          float v = 0.f;
#pragma unroll
          for (int i = 0; i < kPerBlock; ++i) v += s[i * L + lane];
          const int c = ((e / VEC) * L + lane) * VEC + e % VEC;
          if (c < a.D) (which ? pb : pw)[c] = v;
        }
      }
  }
}

// Columns of dweight, then (second half of the grid's y) of dbias.
__global__ void __launch_bounds__(1024) group_norm_sum_kernel(const float *part, int rows, int cols,
                                                              float *dweight, float *dbias) {
  float *out = blockIdx.y ? dbias : dweight;
  if (out)
    sum_columns(part + (blockIdx.y ? (size_t)rows * cols : 0), rows, cols, out, blockIdx.x);
}

struct Launch {
  const GroupNormArgs &a;
  cudaStream_t stream;
  template <typename T, int VEC, int L, int NV>
  cudaError_t operator()() const {
    const RowPlan p =
        row_plan(a.rows, a.G, kRowThreads / L, kSMs * blocks_per_sm(VEC * NV));
    group_norm_bwd_kernel<T, VEC, L, NV><<<p.blocks, kRowThreads, 0, stream>>>(a, p);
    if (a.dweight || a.dbias) {
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      const int rows = a.per_channel ? (int)p.step : p.blocks;
      const int cols = a.per_channel ? a.G * a.D : a.D;
      group_norm_sum_kernel<<<dim3((cols + 31) / 32, 2), 1024, 0, stream>>>(a.ws, rows, cols,
                                                                           a.dweight, a.dbias);
    }
    return cudaGetLastError();
  }
};

}  // namespace

size_t group_norm_bwd_ws_bytes(long long rows, int G, int D, int, int per_channel) {
  // the widest grid that any layout of these sizes takes (4 to 32 lanes a group)
  size_t most = 0;
  for (int lanes = 4; lanes <= 32; lanes *= 2)
    for (int per_sm = 1; per_sm <= blocks_per_sm(1); ++per_sm) {
      const RowPlan p = row_plan(rows, G, kRowThreads / lanes, kSMs * per_sm);
      const size_t part = per_channel ? (size_t)p.step * G * D : (size_t)p.blocks * D;
      if (part > most) most = part;
    }
  return 2 * most * sizeof(float);
}

cudaError_t launch_group_norm_bwd(const GroupNormArgs &a, cudaStream_t stream) {
  return norm_layout(a, Launch{a, stream});
}

}  // namespace gdr
