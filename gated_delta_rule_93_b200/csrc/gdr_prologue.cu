// The prologue as a map of its own, and its gradient.
//
//   q^ = q r with r = 1 / sqrt(|q|^2 + 1e-6), repeated for the value heads
//   that share the key head (k likewise);  g = -s_h softplus(a),
//   beta = sigmoid(b)
//   dq = r (G - q^ (q^ . G)),  G = the sum of dq^ over the sharing heads
//   da = -s_h sigmoid(a) dg,  db = beta (1 - beta) dbeta,
//   ds_h = -sum dg softplus(a)
//
// L lanes hold one key head of one token in registers (16-byte accesses), so
// every tensor is read once and written once: bound by HBM, with the loads of
// U tokens of q and k requested before the first is used.  The gates are the work
// of other blocks of the same launch: a thread for a (token, head) with a
// scalar gate, dk / 4 lanes with a per-channel one.  Every slot keeps its head
// for all its tokens (no division in the loops), so ds adds up in registers;
// a second launch adds the slots' sums in a fixed order.
#include "gdr_rows.cuh"

namespace gdr {
namespace {

constexpr float kNormEps = 1e-6f;
constexpr int kMaxBlocks = 4 * kSMs;  // of each kind of work

struct Split {
  RowPlan norm, gate;
};

Split make_split(const PrologueArgs &a, int L) {
  const int lanes = a.per_channel ? a.d / 4 : 1;
  return {row_plan(a.tokens, a.Hk, kRowThreads / L, kMaxBlocks),
          row_plan(a.tokens, a.H, kRowThreads / lanes, kMaxBlocks)};
}

// g and beta of one block's gate slots.
__device__ __forceinline__ void gates_fwd(const PrologueArgs &a, const RowPlan &p, int block) {
  const int thread = block * kRowThreads + threadIdx.x;
  const int quads = a.per_channel ? a.d / 4 : 1, slot = thread / quads, lane = thread % quads;
  if (slot >= p.slots) return;
  const int h = slot % a.H;
  const float s = -a.gate_scale[h];
  for (long long t = slot / a.H; t < a.tokens; t += p.step) {
    const long long th = t * a.H + h;
    if (lane == 0) a.beta[th] = sigmoid(a.b[th]);
    if (!a.per_channel) {
      a.g[th] = s * softplus(a.a[th]);
    } else {
      float x[4];
      load_vec<float, 4>(a.a + th * a.d + 4 * lane, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = s * softplus(x[e]);
      store_vec<float, 4>(a.g + th * a.d + 4 * lane, x);
    }
  }
}

// da, db and the slot's part of ds.
__device__ __forceinline__ void gates_bwd(const PrologueArgs &a, const RowPlan &p, int block) {
  const int thread = block * kRowThreads + threadIdx.x;
  const int quads = a.per_channel ? a.d / 4 : 1, slot = thread / quads, lane = thread % quads;
  const bool used = slot < p.slots;
  const int h = slot % a.H;
  const float s = a.gate_scale[h];
  float ds = 0.f;
  if (used)
    for (long long t = slot / a.H; t < a.tokens; t += p.step) {
      const long long th = t * a.H + h;
      if (lane == 0) {
        const float beta = sigmoid(a.b[th]);
        a.db[th] = beta * (1.f - beta) * a.dbeta[th];
      }
      if (!a.per_channel) {
        const float x = a.a[th], dg = a.dg[th];
        a.da[th] = -s * sigmoid(x) * dg;
        ds -= dg * softplus(x);
      } else {
        float x[4], dg[4];
        load_vec<float, 4>(a.a + th * a.d + 4 * lane, x);
        load_vec<float, 4>(a.dg + th * a.d + 4 * lane, dg);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ds -= dg[e] * softplus(x[e]);
          x[e] = -s * sigmoid(x[e]) * dg[e];
        }
        store_vec<float, 4>(a.da + th * a.d + 4 * lane, x);
      }
    }
  for (int m = quads / 2; m; m >>= 1) ds += __shfl_xor_sync(0xffffffffu, ds, m);
  if (used && lane == 0) a.ws[slot] = ds;
}

template <typename T, int VEC, int L>
__global__ void __launch_bounds__(kRowThreads, 4) prologue_fwd_kernel(PrologueArgs a, Split p) {
  if ((int)blockIdx.x >= p.norm.blocks) {
    gates_fwd(a, p.gate, blockIdx.x - p.norm.blocks);
    return;
  }
  constexpr int U = 2;
  const int lane = threadIdx.x % L;
  const int slot = blockIdx.x * (kRowThreads / L) + threadIdx.x / L;
  const int hk = slot % a.Hk, share = a.H / a.Hk;
  // (all lanes of a warp take every turn: the sums shuffle over whole warps)
  const long long last = slot < p.norm.slots ? a.tokens : 0;
  const T *qp = static_cast<const T *>(a.q) + hk * a.d + lane * VEC;
  const T *kp = static_cast<const T *>(a.k) + hk * a.d + lane * VEC;
  const long long out = (long long)hk * share * a.d + lane * VEC;
  const long long turns = (a.tokens + U * p.norm.step - 1) / (U * p.norm.step);
  long long t = slot / a.Hk;
  for (long long k = 0; k < turns; ++k) {
    Raw<T, VEC> raw[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long at = t + u * p.norm.step;
      raw[u][0] = raw[u][1] = Raw<T, VEC>{};
      if (at < last) {
        raw[u][0] = load_raw<T, VEC>(qp + at * a.q_stride);
        raw[u][1] = load_raw<T, VEC>(kp + at * a.k_stride);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u, t += p.norm.step)
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        float x[VEC];
        unpack<T, VEC>(raw[u][which], x);
        if (a.norm_qk & (which ? GDR_NORM_K : GDR_NORM_Q)) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) ss += x[e] * x[e];
          const float r = rsqrtf(lanes_sum<L>(ss) + kNormEps);
#pragma unroll
          for (int e = 0; e < VEC; ++e) x[e] *= r;
        }
        T *to = static_cast<T *>(which ? a.kn : a.qn) + t * a.H * a.d + out;
        if (t < last)
          for (int s = 0; s < share; ++s) store_vec<T, VEC>(to + s * a.d, x);
      }
  }
}

template <typename T, int VEC, int L>
__global__ void __launch_bounds__(kRowThreads, 3) prologue_bwd_kernel(PrologueArgs a, Split p) {
  if ((int)blockIdx.x >= p.norm.blocks) {
    gates_bwd(a, p.gate, blockIdx.x - p.norm.blocks);
    return;
  }
  const int lane = threadIdx.x % L;
  const int slot = blockIdx.x * (kRowThreads / L) + threadIdx.x / L;
  const int hk = slot % a.Hk, share = a.H / a.Hk;
  const long long last = slot < p.norm.slots ? a.tokens : 0;
  const long long in = (long long)hk * a.d + lane * VEC;
  const long long up = (long long)hk * share * a.d + lane * VEC;
  const long long turns = (a.tokens + p.norm.step - 1) / p.norm.step;
  long long t = slot / a.Hk;
  for (long long k = 0; k < turns; ++k, t += p.norm.step) {
    float d[2][VEC] = {};
    Raw<T, VEC> raw[2] = {};
    if (t < last) {
      raw[0] = load_raw<T, VEC>(static_cast<const T *>(a.q) + t * a.q_stride + in);
      raw[1] = load_raw<T, VEC>(static_cast<const T *>(a.k) + t * a.k_stride + in);
#pragma unroll 2
      for (int s = 0; s < share; ++s) {
        const long long at = (t * a.H + s) * a.d + up;
        float u[2][VEC];
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          load_vec<float, 4>(a.dqn + at + e, &u[0][e]);
          load_vec<float, 4>(a.dkn + at + e, &u[1][e]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          d[0][e] += u[0][e];
          d[1][e] += u[1][e];
        }
      }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      if (a.norm_qk & (which ? GDR_NORM_K : GDR_NORM_Q)) {
        float x[VEC], ss = 0.f, dot = 0.f;
        unpack<T, VEC>(raw[which], x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          ss += x[e] * x[e];
          dot += x[e] * d[which][e];
        }
        const float r = rsqrtf(lanes_sum<L>(ss) + kNormEps);
        dot = lanes_sum<L>(dot) * r;  // q^ . G
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[which][e] = r * (d[which][e] - x[e] * r * dot);
      }
      if (t < last)
        store_vec<T, VEC>(static_cast<T *>(which ? a.dk : a.dq) + t * a.Hk * a.d + in, d[which]);
    }
  }
}

__global__ void __launch_bounds__(1024) prologue_sum_kernel(const float *part, int rows, int cols,
                                                            float *out) {
  sum_columns(part, rows, cols, out, blockIdx.x);
}

template <bool BWD, typename T, int VEC, int L>
cudaError_t launch_one(const PrologueArgs &a, cudaStream_t stream) {
  const Split p = make_split(a, L);
  const int blocks = p.norm.blocks + p.gate.blocks;
  if constexpr (!BWD) {
    prologue_fwd_kernel<T, VEC, L><<<blocks, kRowThreads, 0, stream>>>(a, p);
  } else {
    prologue_bwd_kernel<T, VEC, L><<<blocks, kRowThreads, 0, stream>>>(a, p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    prologue_sum_kernel<<<(a.H + 31) / 32, 1024, 0, stream>>>(a.ws, (int)p.gate.step, a.H,
                                                             a.dgate_scale);
  }
  return cudaGetLastError();
}

template <bool BWD, typename T, int VEC>
cudaError_t launch_d(const PrologueArgs &a, cudaStream_t stream) {
  switch (a.d) {
    case 32: return launch_one<BWD, T, VEC, 32 / VEC>(a, stream);
    case 64: return launch_one<BWD, T, VEC, 64 / VEC>(a, stream);
    case 128: return launch_one<BWD, T, VEC, 128 / VEC>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t prologue_bwd_ws_bytes(long long tokens, int H, int dk, int per_channel) {
  PrologueArgs a{};
  a.tokens = tokens;
  a.Hk = 1;
  a.H = H;
  a.d = dk;
  a.per_channel = per_channel;
  return (size_t)make_split(a, 1).gate.slots * sizeof(float);
}

cudaError_t launch_prologue_fwd(const PrologueArgs &a, cudaStream_t stream) {
  return a.bf16 ? launch_d<false, __nv_bfloat16, 8>(a, stream) : launch_d<false, float, 4>(a, stream);
}

cudaError_t launch_prologue_bwd(const PrologueArgs &a, cudaStream_t stream) {
  return a.bf16 ? launch_d<true, __nv_bfloat16, 8>(a, stream) : launch_d<true, float, 4>(a, stream);
}

}  // namespace gdr
