// Backward of the output norm (see gdr_group_norm.cuh):
//   dl = dy act(z) or dy act'(l),  dz = dy l act'(z),  h = dl w
//   dx = rstd (h - [center] mean(h) - n mean(h n)),  dw = sum dl n,  db = sum dl
//
// The statistics are computed again from x, which is read anyway.  The weight
// gradients add up in registers over a lane's rows, then over the block (with weights per channel
// a block's slots share a group), and a second launch adds the blocks' partial rows in a fixed
// order; where one block has all rows of its channels, it writes the gradients itself.
#include "gdr_group_norm.cuh"

namespace gdr {
namespace {

// Rows requested at a time (16 bytes of a tensor a lane), and blocks on an SM, for E elements a lane.
constexpr int rows_ahead(int bytes) { return bytes <= 4 ? 4 : bytes <= 8 ? 2 : 1; }
constexpr int blocks_per_sm(int E) { return E <= 8 ? 2 : 1; }

// Value and slope of the activation.
__device__ __forceinline__ void act_both(int act, float u, float &f, float &df) {
  if (act == GDR_ACT_NONE) {
    f = u;
    df = 1.f;
    return;
  }
  const float s = sigmoid(u);
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
  constexpr int E = VEC * NV, U = rows_ahead(E * sizeof(T));
  constexpr bool kAhead = E <= 16;  // (wider rows have no registers for a second one)
  constexpr int kPerBlock = kRowThreads / L;
  const int lane = threadIdx.x % L;
  const int slot = threadIdx.x / L, g = p.group(blockIdx.x, slot, kPerBlock, a.G);
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
  const long long last = p.used(blockIdx.x, slot, kPerBlock) ? a.rows : 0;  // rows of this slot end here
  const long long off = (long long)g * a.D + lane * VEC, dense = (long long)a.G * a.D;
  const T *xp = static_cast<const T *>(a.x) + off, *zp = static_cast<const T *>(a.z) + off;
  const T *dyp = static_cast<const T *>(a.dy) + off;
  const long long turns = (a.rows + U * p.step - 1) / (U * p.step);
  long long row = p.first_row(blockIdx.x, slot, kPerBlock, a.G);
  Raw<T, VEC> xn[U][NV], zn[U][NV], dyn[U][NV];  // the next turn's rows
  const auto request = [&](long long from) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const long long at = from + u * p.step;
        xn[u][i] = zn[u][i] = dyn[u][i] = Raw<T, VEC>{};
        if (at < last && in[i]) {
          xn[u][i] = load_raw<T, VEC>(xp + at * a.x_stride + i * L * VEC);
          dyn[u][i] = load_raw<T, VEC>(dyp + at * dense + i * L * VEC);
          if (a.z) zn[u][i] = load_raw<T, VEC>(zp + at * a.z_stride + i * L * VEC);
        }
      }
  };
  if constexpr (kAhead) request(row);
  for (long long k = 0; k < turns; ++k) {
    if constexpr (!kAhead) request(row);
    Raw<T, VEC> xr[U][NV], zr[U][NV], dyr[U][NV];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        xr[u][i] = xn[u][i];
        zr[u][i] = zn[u][i];
        dyr[u][i] = dyn[u][i];
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

  // Partial rows of the weight gradients, a block's D values each, db behind dw:
  // over the slots of a warp, then over the warps.
  if (!a.dweight && !a.dbias) return;
  __shared__ float s[kRowThreads / 32][L * E];
  const int warp = threadIdx.x / 32, at = threadIdx.x % 32;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float *out = which ? a.dbias : a.dweight;
    if (!out) continue;
    if (p.sum) out = a.ws + ((which ? (long long)p.blocks : 0) + blockIdx.x) * a.D;
    else if (p.by_block) out += (long long)g * a.D;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float v = which ? db[e] : dw[e];
#pragma unroll
      for (int m = L; m < 32; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
      // (element e of a lane is channel ((e / VEC) L + lane) VEC + e % VEC)
      if (at < L) s[warp][((e / VEC) * L + lane) * VEC + e % VEC] = v;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += kRowThreads) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kRowThreads / 32; ++i) v += s[i][c];
      out[c] = v;
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

constexpr int kFewTurns = 4;  // rows a slot takes rather than have a second launch

RowPlan bwd_plan(long long rows, int G, int lanes, int per_sm, int per_channel) {
  const int per_block = kRowThreads / lanes;
  RowPlan p = row_plan(rows, G, per_block, kSMs * per_sm, per_channel);
  // few rows: as few blocks as have every channel once
  if (per_channel ? rows <= kFewTurns * per_block : rows * G <= kFewTurns * per_block)
    p = row_plan(rows, G, per_block, per_channel ? G : 1, per_channel);
  p.sum = p.blocks > (per_channel ? G : 1);
  return p;
}

struct Launch {
  const GroupNormArgs &a;
  cudaStream_t stream;
  template <typename T, int VEC, int L, int NV>
  cudaError_t operator()() const {
    const RowPlan p = bwd_plan(a.rows, a.G, L, blocks_per_sm(VEC * NV), a.per_channel);
    group_norm_bwd_kernel<T, VEC, L, NV><<<p.blocks, kRowThreads, 0, stream>>>(a, p);
    if (p.sum && (a.dweight || a.dbias)) {
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      const int rows = a.per_channel ? p.blocks / a.G : p.blocks;
      const int cols = a.per_channel ? a.G * a.D : a.D;
      const dim3 grid((cols + sum_width(cols) - 1) / sum_width(cols), a.dbias ? 2 : 1);
      group_norm_sum_kernel<<<grid, 1024, 0, stream>>>(a.ws, rows, cols, a.dweight, a.dbias);
    }
    return cudaGetLastError();
  }
};

}  // namespace

size_t group_norm_bwd_ws_bytes(long long rows, int G, int D, int, int per_channel) {
  // the widest grid that any layout of these sizes takes (4 to 32 lanes a group)
  int most = 0;
  for (int lanes = 4; lanes <= 32; lanes *= 2)
    for (int per_sm = 1; per_sm <= blocks_per_sm(1); ++per_sm) {
      const RowPlan p = bwd_plan(rows, G, lanes, per_sm, per_channel);
      if (p.blocks > most) most = p.blocks;
    }
  return 2 * (size_t)most * D * sizeof(float);
}

cudaError_t launch_group_norm_bwd(const GroupNormArgs &a, cudaStream_t stream) {
  return norm_layout(a, Launch{a, stream});
}

}  // namespace gdr
