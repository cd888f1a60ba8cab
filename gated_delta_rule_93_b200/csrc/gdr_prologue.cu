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
// every tensor is read once and written once: bound by HBM.  The gates are
// elementwise work of other blocks of the same launch.  The gate threads of
// the backward keep one head for all their tokens (their number is a multiple of H), so ds adds
// up in registers; a second launch adds their partial sums in a fixed order.
#include "gdr_rows.cuh"

namespace gdr {
namespace {

constexpr float kNormEps = 1e-6f;

// Blocks of the two kinds of work, and the gate slots (backward).
struct Split {
  int norm_blocks, gate_blocks;
  int slots;       // gate slots in use (a multiple of H)
  long long step;  // tokens between a slot's gates
};

int blocks_for(long long items, int per_block) {
  const long long n = (items + per_block - 1) / per_block;
  return (int)(n < 1 ? 1 : n > kRowBlocks ? kRowBlocks : n);
}

// Gate slots: a thread for a (token, head) with a scalar gate, dk / 4 lanes
// with a per-channel one.
Split make_split(long long tokens, int H, int dk, int per_channel) {
  Split s;
  const int per_block = kRowThreads / (per_channel ? dk / 4 : 1);
  s.norm_blocks = 0;
  s.gate_blocks = blocks_for(tokens * H, per_block);
  const int least = (H + per_block - 1) / per_block;  // every head once
  if (s.gate_blocks < least) s.gate_blocks = least;
  s.step = (long long)s.gate_blocks * per_block / H;
  s.slots = (int)(s.step * H);
  return s;
}

template <typename T, int VEC, int L>
__global__ void __launch_bounds__(kRowThreads) prologue_fwd_kernel(PrologueArgs a, Split p) {
  if ((int)blockIdx.x >= p.norm_blocks) {
    const long long step = (long long)p.gate_blocks * kRowThreads;
    const long long first = (long long)(blockIdx.x - p.norm_blocks) * kRowThreads + threadIdx.x;
    for (long long i = first; i < a.tokens * a.H; i += step) {
      a.beta[i] = sigmoid(a.b[i]);
      if (!a.per_channel) a.g[i] = -a.gate_scale[i % a.H] * softplus(a.a[i]);
    }
    if (a.per_channel) {
      const int quads = a.d / 4;
      for (long long i = first; i < a.tokens * a.H * quads; i += step) {
        float x[4];
        load_vec<float, 4>(a.a + 4 * i, x);
        const float s = -a.gate_scale[(i / quads) % a.H];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = s * softplus(x[e]);
        store_vec<float, 4>(a.g + 4 * i, x);
      }
    }
    return;
  }
  const int lane = threadIdx.x % L;
  const int share = a.H / a.Hk;
  const long long groups = a.tokens * a.Hk;
  const long long step = (long long)p.norm_blocks * (kRowThreads / L);
  const long long turns = (groups + step - 1) / step;
  long long f = (long long)blockIdx.x * (kRowThreads / L) + threadIdx.x / L;
  for (long long k = 0; k < turns; ++k, f += step) {
    const bool live = f < groups;
    const long long t = f / a.Hk;
    const int hk = (int)(f % a.Hk);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const T *in = static_cast<const T *>(which ? a.k : a.q) +
                    t * (which ? a.k_stride : a.q_stride) + hk * a.d + lane * VEC;
      float x[VEC] = {};
      if (live) load_vec<T, VEC>(in, x);
      if (a.norm_qk & (which ? GDR_NORM_K : GDR_NORM_Q)) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss += x[e] * x[e];
        const float r = rsqrtf(lanes_sum<L>(ss) + kNormEps);
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[e] *= r;
      }
      T *out = static_cast<T *>(which ? a.kn : a.qn) + (t * a.H + hk * share) * a.d + lane * VEC;
      if (live)
        for (int s = 0; s < share; ++s) store_vec<T, VEC>(out + s * a.d, x);
    }
  }
}

template <typename T, int VEC, int L>
__global__ void __launch_bounds__(kRowThreads) prologue_bwd_kernel(PrologueArgs a, Split p) {
  if ((int)blockIdx.x >= p.norm_blocks) {
    const int thread = (blockIdx.x - p.norm_blocks) * kRowThreads + threadIdx.x;
    float ds = 0.f;
    if (!a.per_channel) {
      if (thread >= p.slots) return;
      const int h = thread % a.H;
      const float s = a.gate_scale[h];
      for (long long t = thread / a.H; t < a.tokens; t += p.step) {
        const long long i = t * a.H + h;
        const float x = a.a[i], dg = a.dg[i], beta = sigmoid(a.b[i]);
        a.da[i] = -s * sigmoid(x) * dg;
        a.db[i] = beta * (1.f - beta) * a.dbeta[i];
        ds -= dg * softplus(x);
      }
      a.ws[thread] = ds;
    } else {
      const int quads = a.d / 4, slot = thread / quads, lane = thread % quads;
      const bool used = slot < p.slots;
      const int h = slot % a.H;
      const float s = a.gate_scale[h];
      if (used)
        for (long long t = slot / a.H; t < a.tokens; t += p.step) {
          const long long th = t * a.H + h, i = th * a.d + 4 * lane;
          float x[4], dg[4];
          load_vec<float, 4>(a.a + i, x);
          load_vec<float, 4>(a.dg + i, dg);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ds -= dg[e] * softplus(x[e]);
            x[e] = -s * sigmoid(x[e]) * dg[e];
          }
          store_vec<float, 4>(a.da + i, x);
          if (lane == 0) {
            const float beta = sigmoid(a.b[th]);
            a.db[th] = beta * (1.f - beta) * a.dbeta[th];
          }
        }
      for (int m = quads / 2; m; m >>= 1) ds += __shfl_xor_sync(0xffffffffu, ds, m);
      if (used && lane == 0) a.ws[slot] = ds;
    }
    return;
  }
  const int lane = threadIdx.x % L;
  const int share = a.H / a.Hk;
  const long long groups = a.tokens * a.Hk;
  const long long step = (long long)p.norm_blocks * (kRowThreads / L);
  const long long turns = (groups + step - 1) / step;
  long long f = (long long)blockIdx.x * (kRowThreads / L) + threadIdx.x / L;
  for (long long k = 0; k < turns; ++k, f += step) {
    const bool live = f < groups;
    const long long t = f / a.Hk;
    const int hk = (int)(f % a.Hk);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float *up = (which ? a.dkn : a.dqn) + (t * a.H + hk * share) * a.d + lane * VEC;
      float d[VEC] = {};
      if (live)
        for (int s = 0; s < share; ++s) {
          float u[VEC];
#pragma unroll
          for (int e = 0; e < VEC; e += 4) load_vec<float, 4>(up + s * a.d + e, u + e);
#pragma unroll
          for (int e = 0; e < VEC; ++e) d[e] += u[e];
        }
      if (a.norm_qk & (which ? GDR_NORM_K : GDR_NORM_Q)) {
        const T *in = static_cast<const T *>(which ? a.k : a.q) +
                      t * (which ? a.k_stride : a.q_stride) + hk * a.d + lane * VEC;
        float x[VEC] = {}, ss = 0.f, dot = 0.f;
        if (live) load_vec<T, VEC>(in, x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          ss += x[e] * x[e];
          dot += x[e] * d[e];
        }
        const float r = rsqrtf(lanes_sum<L>(ss) + kNormEps);
        dot = lanes_sum<L>(dot) * r;  // q^ . G
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[e] = r * (d[e] - x[e] * r * dot);
      }
      T *out = static_cast<T *>(which ? a.dk : a.dq) + f * a.d + lane * VEC;
      if (live) store_vec<T, VEC>(out, d);
    }
  }
}

__global__ void __launch_bounds__(1024) prologue_sum_kernel(const float *part, int rows, int cols,
                                                            float *out) {
  sum_columns(part, rows, cols, out, blockIdx.x);
}

template <bool BWD, typename T, int VEC, int L>
cudaError_t launch_one(const PrologueArgs &a, cudaStream_t stream) {
  Split p = make_split(a.tokens, a.H, a.d, a.per_channel);
  p.norm_blocks = blocks_for(a.tokens * a.Hk, kRowThreads / L);
  const int blocks = p.norm_blocks + p.gate_blocks;
  if constexpr (!BWD) {
    prologue_fwd_kernel<T, VEC, L><<<blocks, kRowThreads, 0, stream>>>(a, p);
  } else {
    prologue_bwd_kernel<T, VEC, L><<<blocks, kRowThreads, 0, stream>>>(a, p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    prologue_sum_kernel<<<(a.H + 31) / 32, 1024, 0, stream>>>(a.ws, (int)p.step, a.H,
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
  return (size_t)make_split(tokens, H, dk, per_channel).slots * sizeof(float);
}

cudaError_t launch_prologue_fwd(const PrologueArgs &a, cudaStream_t stream) {
  return a.bf16 ? launch_d<false, __nv_bfloat16, 8>(a, stream) : launch_d<false, float, 4>(a, stream);
}

cudaError_t launch_prologue_bwd(const PrologueArgs &a, cudaStream_t stream) {
  return a.bf16 ? launch_d<true, __nv_bfloat16, 8>(a, stream) : launch_d<true, float, 4>(a, stream);
}

}  // namespace gdr
