// The mixer's output norm: group norm, channels last, with an activation,
// forward and backward.
//
//   n = (x - m) rstd,  l = n w + b,  y = act(z) l  (gated)  or  act(l)
//   dl = dy act(z) or dy act'(l),  dz = dy l act'(z),  h = dl w
//   dx = rstd (h - [center] mean(h) - n mean(h n)),  dw = sum dl n,  db = sum dl
//
// A group (one head of one token) is a few hundred bytes, so L lanes of a
// warp hold it in registers: x (and z, dy) are read once, every sum over the
// group is a shuffle, and the results are written once.  Both directions are
// bound by HBM.
//
// A lane keeps the same group index for all its rows (the number of groups
// in flight is a multiple of G), so weights are loaded once and the weight
// gradients add up in registers.  Each block (weights shared by the groups)
// or each of its row slots (weights per channel) then writes one partial row,
// and a second launch adds the partial rows in a fixed order.
#include "gdr_rows.cuh"

namespace gdr {
namespace {

// Value and slope of the activation.
__device__ __forceinline__ float act_of(int act, float u) {
  if (act == GDR_ACT_NONE) return u;
  const float s = sigmoid(u);
  return act == GDR_ACT_SILU ? u * s : s;
}
__device__ __forceinline__ void act_both(int act, float u, float &f, float &df) {
  if (act == GDR_ACT_NONE) {
    f = u;
    df = 1.f;
    return;
  }
  const float s = sigmoid(u);
  if (act == GDR_ACT_SILU) {
    f = u * s;
    df = s * (1.f + u * (1.f - s));
  } else {
    f = s;
    df = s * (1.f - s);
  }
}

// The groups in flight: `slots` of L lanes each over the grid, `step` rows apart.
struct Plan {
  int blocks, slots;
  long long step;  // rows between a slot's groups
};

Plan make_plan(long long rows, int G, int per_block) {
  const long long want = (rows * G + per_block - 1) / per_block;
  const long long least = ((long long)G + per_block - 1) / per_block;  // every group once
  long long blocks = want < kRowBlocks ? want : kRowBlocks;
  if (blocks < least) blocks = least;
  if (blocks < 1) blocks = 1;
  Plan p;
  p.blocks = (int)blocks;
  p.step = blocks * per_block / G;
  p.slots = (int)(p.step * G);
  return p;
}

template <typename T, int VEC, int L, int NV>
__global__ void __launch_bounds__(kRowThreads) group_norm_fwd_kernel(GroupNormArgs a, Plan p) {
  constexpr int E = VEC * NV;
  const int lane = threadIdx.x % L;
  const int slot = blockIdx.x * (kRowThreads / L) + threadIdx.x / L;
  const bool used = slot < p.slots;
  const int g = slot % a.G;
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
  const long long first = slot / a.G;
  const long long turns = (a.rows + p.step - 1) / p.step;
  for (long long k = 0; k < turns; ++k) {
    const long long row = first + k * p.step;
    const bool live = used && row < a.rows;
    const T *xp = static_cast<const T *>(a.x) + row * a.x_stride + (long long)g * a.D;
    const T *zp = static_cast<const T *>(a.z) + row * a.z_stride + (long long)g * a.D;
    float x[E], z[E];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[i * VEC + e] = z[i * VEC + e] = 0.f;
      if (live && in[i]) {
        load_vec<T, VEC>(xp + (i * L + lane) * VEC, &x[i * VEC]);
        if (a.z) load_vec<T, VEC>(zp + (i * L + lane) * VEC, &z[i * VEC]);
      }
    }
    float m = 0.f, ss = 0.f;
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
    T *yp = static_cast<T *>(a.y) + (row * a.G + g) * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (live && in[i]) {
        float y[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float l = x[i * VEC + e] * rstd * w[i * VEC + e] + b[i * VEC + e];
          y[e] = a.z ? act_of(a.act, z[i * VEC + e]) * l : act_of(a.act, l);
        }
        store_vec<T, VEC>(yp + (i * L + lane) * VEC, y);
      }
    }
  }
}

template <typename T, int VEC, int L, int NV>
__global__ void __launch_bounds__(kRowThreads) group_norm_bwd_kernel(GroupNormArgs a, Plan p) {
  constexpr int E = VEC * NV;
  constexpr int kPerBlock = kRowThreads / L;
  const int lane = threadIdx.x % L;
  const int slot = blockIdx.x * kPerBlock + threadIdx.x / L;
  const bool used = slot < p.slots;
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
  const long long first = slot / a.G;
  const long long turns = (a.rows + p.step - 1) / p.step;
  for (long long k = 0; k < turns; ++k) {
    const long long row = first + k * p.step;
    const bool live = used && row < a.rows;
    const long long dense = (row * a.G + g) * a.D;
    const T *xp = static_cast<const T *>(a.x) + row * a.x_stride + (long long)g * a.D;
    const T *zp = static_cast<const T *>(a.z) + row * a.z_stride + (long long)g * a.D;
    const T *dyp = static_cast<const T *>(a.dy) + dense;
    float x[E], z[E], dy[E];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * L + lane) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[i * VEC + e] = z[i * VEC + e] = dy[i * VEC + e] = 0.f;
      if (live && in[i]) {
        load_vec<T, VEC>(xp + c, &x[i * VEC]);
        load_vec<T, VEC>(dyp + c, &dy[i * VEC]);
        if (a.z) load_vec<T, VEC>(zp + c, &z[i * VEC]);
      }
    }
    float m = 0.f, ss = 0.f;
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
    for (int e = 0; e < E; ++e) {
      const float n = x[e] * rstd;
      const float l = n * w[e] + b[e];
      float f, df, dl;
      if (a.z) {
        act_both(a.act, z[e], f, df);
        dl = dy[e] * f;
        z[e] = dy[e] * l * df;  // dz
      } else {
        act_both(a.act, l, f, df);
        dl = dy[e] * df;
      }
      // (dy is zero outside the group and the rows: so are all of these)
      dw[e] += dl * n;
      db[e] += dl;
      h[e] = dl * w[e];
      x[e] = n;
      sh += h[e];
      shn += h[e] * n;
    }
    shn = lanes_sum<L>(shn) * inv_d;
    sh = a.center ? lanes_sum<L>(sh) * inv_d : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * L + lane) * VEC;
      if (live && in[i]) {
        float d[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          d[e] = rstd * (h[i * VEC + e] - sh - x[i * VEC + e] * shn);
        constexpr int V4 = VEC < 4 ? VEC : 4;
#pragma unroll
        for (int e = 0; e < VEC; e += V4) store_vec<float, V4>(a.dx + dense + c + e, d + e);
        if (a.dz) store_vec<T, VEC>(static_cast<T *>(a.dz) + dense + c, &z[i * VEC]);
      }
    }
  }

  // Partial rows of the weight gradients, db behind dw.
  if (!a.dweight && !a.dbias) return;
  if (a.per_channel) {  // [step][G D]
    if (used) {
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

bool multiple(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Elements per access: 16 bytes where every row and group starts on 16.
int vector_width(const GroupNormArgs &a) {
  const int vec = a.bf16 ? 8 : 4;
  const bool ok = a.D % vec == 0 && a.x_stride % vec == 0 && (!a.z || a.z_stride % vec == 0) &&
                  multiple(a.x, 16) && multiple(a.z, 16) && multiple(a.dy, 16) &&
                  multiple(a.y, 16) && multiple(a.dx, 16) && multiple(a.dz, 16);
  return ok ? vec : 1;
}

template <bool BWD, typename T, int VEC, int L, int NV>
cudaError_t launch_one(const GroupNormArgs &a, cudaStream_t stream) {
  const Plan p = make_plan(a.rows, a.G, kRowThreads / L);
  if constexpr (!BWD) {
    group_norm_fwd_kernel<T, VEC, L, NV><<<p.blocks, kRowThreads, 0, stream>>>(a, p);
  } else {
    group_norm_bwd_kernel<T, VEC, L, NV><<<p.blocks, kRowThreads, 0, stream>>>(a, p);
    if (a.dweight || a.dbias) {
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
      const int rows = a.per_channel ? (int)p.step : p.blocks;
      const int cols = a.per_channel ? a.G * a.D : a.D;
      group_norm_sum_kernel<<<dim3((cols + 31) / 32, 2), 1024, 0, stream>>>(a.ws, rows, cols,
                                                                           a.dweight, a.dbias);
    }
  }
  return cudaGetLastError();
}

template <bool BWD, typename T, int VEC>
cudaError_t launch_vec(const GroupNormArgs &a, cudaStream_t stream) {
  const int n = (a.D + VEC - 1) / VEC;  // vectors of a group
  if (n <= 4) return launch_one<BWD, T, VEC, 4, 1>(a, stream);
  if (n <= 8) return launch_one<BWD, T, VEC, 8, 1>(a, stream);
  if (n <= 16) return launch_one<BWD, T, VEC, 16, 1>(a, stream);
  if (n <= 32) return launch_one<BWD, T, VEC, 32, 1>(a, stream);
  if (n <= 64) return launch_one<BWD, T, VEC, 32, 2>(a, stream);
  if (n <= 128) return launch_one<BWD, T, VEC, 32, 4>(a, stream);
  if constexpr (VEC <= 4) {
    if (n <= 256) return launch_one<BWD, T, VEC, 32, 8>(a, stream);
  }
  if constexpr (VEC == 1) {
    if (n <= 512) return launch_one<BWD, T, VEC, 32, 16>(a, stream);
    if (n <= 1024) return launch_one<BWD, T, VEC, 32, 32>(a, stream);
  }
  return cudaErrorInvalidValue;
}

template <bool BWD>
cudaError_t launch_any(const GroupNormArgs &a, cudaStream_t stream) {
  const int vec = vector_width(a);
  if (a.bf16)
    return vec == 8 ? launch_vec<BWD, __nv_bfloat16, 8>(a, stream)
                    : launch_vec<BWD, __nv_bfloat16, 1>(a, stream);
  return vec == 4 ? launch_vec<BWD, float, 4>(a, stream) : launch_vec<BWD, float, 1>(a, stream);
}

}  // namespace

size_t group_norm_bwd_ws_bytes(long long rows, int G, int D, int bf16, int per_channel) {
  // the widest grid any layout of these sizes takes (4 to 32 lanes a group)
  size_t most = 0;
  for (int lanes = 4; lanes <= 32; lanes *= 2) {
    const Plan p = make_plan(rows, G, kRowThreads / lanes);
    const size_t part = per_channel ? (size_t)p.step * G * D : (size_t)p.blocks * D;
    if (part > most) most = part;
  }
  (void)bf16;
  return 2 * most * sizeof(float);
}

cudaError_t launch_group_norm_fwd(const GroupNormArgs &a, cudaStream_t stream) {
  return launch_any<false>(a, stream);
}

cudaError_t launch_group_norm_bwd(const GroupNormArgs &a, cudaStream_t stream) {
  return launch_any<true>(a, stream);
}

}  // namespace gdr
