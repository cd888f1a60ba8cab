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
// two tokens of q and k requested before the first is used, and blocks of 4 tokens
// a slot so that the SMs finish together.  The gates are the work of other blocks
// of the same launch: a thread for a (token, head) with a scalar gate, dk / 4
// lanes with a per-channel one.  Every slot keeps its head for all its tokens (no
// division in the loops: 115 us with them, 70 us without, where it is 65 us now), so ds
// adds up in registers and then over the block; a second launch adds the blocks'
// sums in a fixed order, unless one block had all tokens.
//
// 32768 tokens, bf16, scalar gates, 8 key heads of 128 for 16 value heads: forward
// 64.8 us (6347 GB/s; a copy runs at 6456), gradient 128.7 us (6353 GB/s).
// Per-channel gates spend a third of their time on softplus and sigmoid: 8192
// tokens x 16 x 128 forward 48.8 us (5521 GB/s), gradient 82.5 us (5712 GB/s).  The
// gradient takes q, then k, so that 64 registers do and four blocks fit an SM (both
// at once, three blocks: 131.1 and 91.0 us).
#include "gdr_rows.cuh"

namespace gdr {
namespace {

constexpr float kNormEps = 1e-6f;
// Tokens of a slot in a block, or fewer where that leaves less than so many blocks.
constexpr int kNormTurns = 4, kNormBlocks = 4 * kSMs;
constexpr int kGateTurns = 8, kGateBlocks = 4 * kSMs;
constexpr int kMostParts = 4096;  // partial sums of a head at most

// The gates' blocks: `heads` heads of `tokens` tokens at a time; blocks that
// share a tile of heads are `step` tokens apart.
struct GatePlan {
  int blocks, heads, tiles, tokens;
  long long step;
};

struct Split {
  RowPlan norm;
  GatePlan gate;
};

// A thread for a (token, head) with a scalar gate, dk / 4 lanes with a
// per-channel one (a block then has one head).
GatePlan gate_plan(long long tokens, int H, int dk, int per_channel) {
  GatePlan p;
  const int slots = kRowThreads / (per_channel ? dk / 4 : 1);
  p.heads = per_channel ? 1 : H < slots ? H : slots;
  p.tiles = (H + p.heads - 1) / p.heads;
  p.tokens = slots / p.heads;
  const long long passes = (tokens + p.tokens - 1) / p.tokens;
  long long rows = (passes + kGateTurns - 1) / kGateTurns;
  const int least = (kGateBlocks + p.tiles - 1) / p.tiles;
  if (rows < least) rows = passes < least ? passes : least;
  if (rows < 1) rows = 1;
  if (rows > kMostParts) rows = kMostParts;
  p.blocks = (int)(rows * p.tiles);
  p.step = rows * p.tokens;
  return p;
}

// The place of a thread among its block's gates.
struct GatePlace {
  int h, lane;
  long long token;
  bool used;
};
__device__ __forceinline__ GatePlace gate_place(const PrologueArgs &a, const GatePlan &p, int block) {
  const int quads = a.per_channel ? a.d / 4 : 1, slot = threadIdx.x / quads;
  GatePlace g;
  g.lane = threadIdx.x % quads;
  g.h = block % p.tiles * p.heads + slot % p.heads;
  g.token = (long long)(block / p.tiles) * p.tokens + slot / p.heads;
  g.used = g.h < a.H && slot < p.tokens * p.heads;
  return g;
}

// g and beta of one block's gates.
__device__ __forceinline__ void gates_fwd(const PrologueArgs &a, const GatePlan &p, int block) {
  constexpr int U = 4;  // tokens on their way at once
  const GatePlace g = gate_place(a, p, block);
  if (!g.used) return;
  const float s = -a.gate_scale[g.h];
  for (long long t = g.token; t < a.tokens; t += U * p.step) {
    float b[U], x[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long at = t + u * p.step, th = at * a.H + g.h;
      if (at >= a.tokens) continue;
      if (g.lane == 0) b[u] = __ldcs(a.b + th);
      if (!a.per_channel)
        x[u][0] = __ldcs(a.a + th);
      else
        load_vec<float, 4>(a.a + th * a.d + 4 * g.lane, x[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long at = t + u * p.step, th = at * a.H + g.h;
      if (at >= a.tokens) continue;
      if (g.lane == 0) a.beta[th] = sigmoid(b[u]);
      if (!a.per_channel) {
        a.g[th] = s * softplus(x[u][0]);
      } else {
        const float2 lo = mul2(both(s), softplus2(make_float2(x[u][0], x[u][1])));
        const float2 hi = mul2(both(s), softplus2(make_float2(x[u][2], x[u][3])));
        const float y[4] = {lo.x, lo.y, hi.x, hi.y};
        store_vec<float, 4>(a.g + th * a.d + 4 * g.lane, y);
      }
    }
  }
}

// da, db and the block's part of ds: [blocks / tiles][H].
__device__ __forceinline__ void gates_bwd(const PrologueArgs &a, const GatePlan &p, int block) {
  constexpr int U = 2;
  const GatePlace g = gate_place(a, p, block);
  float ds = 0.f;
  if (g.used) {
    const float s = a.gate_scale[g.h];
    for (long long t = g.token; t < a.tokens; t += U * p.step) {
      float b[U], dbeta[U], x[U][4], dg[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long at = t + u * p.step, th = at * a.H + g.h;
        if (at >= a.tokens) continue;
        if (g.lane == 0) {
          b[u] = __ldcs(a.b + th);
          dbeta[u] = __ldcs(a.dbeta + th);
        }
        if (!a.per_channel) {
          x[u][0] = __ldcs(a.a + th);
          dg[u][0] = __ldcs(a.dg + th);
        } else {
          load_vec<float, 4>(a.a + th * a.d + 4 * g.lane, x[u]);
          load_vec<float, 4>(a.dg + th * a.d + 4 * g.lane, dg[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long at = t + u * p.step, th = at * a.H + g.h;
        if (at >= a.tokens) continue;
        if (g.lane == 0) {
          const float beta = sigmoid(b[u]);
          a.db[th] = beta * (1.f - beta) * dbeta[u];
        }
        if (!a.per_channel) {
          float sig;
          ds -= dg[u][0] * softplus(x[u][0], &sig);
          a.da[th] = -s * sig * dg[u][0];
        } else {
          float2 sum = both(0.f), y[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 d = make_float2(dg[u][2 * e], dg[u][2 * e + 1]);
            float2 sig;
            sum = fma2(d, softplus2(make_float2(x[u][2 * e], x[u][2 * e + 1]), &sig), sum);
            y[e] = mul2(mul2(both(-s), sig), d);
          }
          ds -= sum.x + sum.y;
          store_access<float, 4>(a.da + th * a.d + 4 * g.lane, y, 0);
        }
      }
    }
  }
  // over the lanes of a head (a power of two of them, whole warps or less), then over its slots
  const int quads = a.per_channel ? a.d / 4 : 1;
  for (int m = quads / 2; m; m >>= 1) ds += __shfl_xor_sync(0xffffffffu, ds, m);
  __shared__ float part[kRowThreads];
  if (g.lane == 0) part[threadIdx.x / quads] = ds;
  __syncthreads();
  const int mine = threadIdx.x, h = block % p.tiles * p.heads + mine;
  if (mine < p.heads && h < a.H) {
    float v = 0.f;
    for (int i = 0; i < p.tokens; ++i) v += part[i * p.heads + mine];
    const bool all = p.blocks == p.tiles;  // this block had all tokens
    (all ? a.dgate_scale : a.ws + (long long)(block / p.tiles) * a.H)[h] = v;
  }
}

template <typename T, int VEC, int L>
__global__ void __launch_bounds__(kRowThreads, 4) prologue_fwd_kernel(PrologueArgs a, Split p) {
  after_previous();
  let_next();
  const int block = blockIdx.x;
  if (block >= p.norm.blocks) {
    gates_fwd(a, p.gate, block - p.norm.blocks);
    return;
  }
  constexpr int U = 2;
  const int lane = threadIdx.x % L;
  constexpr int kPerBlock = kRowThreads / L;
  const int slot = threadIdx.x / L, hk = p.norm.group(block, slot, kPerBlock, a.Hk);
  const int share = a.H / a.Hk;
  // (all lanes of a warp take every turn: the sums shuffle over whole warps)
  const long long last = p.norm.used(block, slot, kPerBlock) ? a.tokens : 0;
  const T *qp = static_cast<const T *>(a.q) + hk * a.d + lane * VEC;
  const T *kp = static_cast<const T *>(a.k) + hk * a.d + lane * VEC;
  const long long out = (long long)hk * share * a.d + lane * VEC;
  const long long turns = (a.tokens + U * p.norm.step - 1) / (U * p.norm.step);
  long long t = p.norm.first_row(block, slot, kPerBlock, a.Hk);
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
__global__ void __launch_bounds__(kRowThreads, 4) prologue_bwd_kernel(PrologueArgs a, Split p) {
  after_previous();
  let_next();
  const int block = blockIdx.x;
  if (block >= p.norm.blocks) {
    gates_bwd(a, p.gate, block - p.norm.blocks);
    return;
  }
  const int lane = threadIdx.x % L;
  constexpr int kPerBlock = kRowThreads / L;
  const int slot = threadIdx.x / L, hk = p.norm.group(block, slot, kPerBlock, a.Hk);
  const int share = a.H / a.Hk;
  const long long last = p.norm.used(block, slot, kPerBlock) ? a.tokens : 0;
  const long long in = (long long)hk * a.d + lane * VEC;
  const long long up = (long long)hk * share * a.d + lane * VEC;
  const long long turns = (a.tokens + p.norm.step - 1) / p.norm.step;
  long long t = p.norm.first_row(block, slot, kPerBlock, a.Hk);
  for (long long k = 0; k < turns; ++k, t += p.norm.step) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      float d[VEC] = {};
      Raw<T, VEC> raw = {};
      if (t < last) {
        raw = load_raw<T, VEC>(static_cast<const T *>(which ? a.k : a.q) +
                               t * (which ? a.k_stride : a.q_stride) + in);
        const float *from = (which ? a.dkn : a.dqn) + t * a.H * a.d + up;
#pragma unroll 2
        for (int s = 0; s < share; ++s) {
          float u[VEC];
#pragma unroll
          for (int e = 0; e < VEC; e += 4) load_vec<float, 4>(from + s * a.d + e, u + e);
#pragma unroll
          for (int e = 0; e < VEC; ++e) d[e] += u[e];
        }
      }
      if (a.norm_qk & (which ? GDR_NORM_K : GDR_NORM_Q)) {
        float x[VEC], ss = 0.f, dot = 0.f;
        unpack<T, VEC>(raw, x);
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
      if (t < last)
        store_vec<T, VEC>(static_cast<T *>(which ? a.dk : a.dq) + t * a.Hk * a.d + in, d);
    }
  }
}

template <bool BWD, typename T, int VEC, int L>
cudaError_t launch_one(const PrologueArgs &a, cudaStream_t stream) {
  const Split p = {row_plan(a.tokens, a.Hk, kRowThreads / L, kNormTurns, kNormBlocks, false),
                   gate_plan(a.tokens, a.H, a.d, a.per_channel)};
  const int blocks = p.norm.blocks + p.gate.blocks;
  if constexpr (!BWD) {
    return launch_next(prologue_fwd_kernel<T, VEC, L>, dim3(blocks), kRowThreads, stream, a, p);
  } else {
    const cudaError_t e =
        launch_next(prologue_bwd_kernel<T, VEC, L>, dim3(blocks), kRowThreads, stream, a, p);
    if (e == cudaSuccess && p.gate.blocks > p.gate.tiles)
      return launch_sums(a.ws, p.gate.blocks / p.gate.tiles, a.H, a.dgate_scale, nullptr, stream);
    return e;
  }
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
  const GatePlan p = gate_plan(tokens, H, dk, per_channel);
  return (size_t)(p.blocks / p.tiles) * H * sizeof(float);
}

cudaError_t launch_prologue_fwd(const PrologueArgs &a, cudaStream_t stream) {
  return a.bf16 ? launch_d<false, __nv_bfloat16, 8>(a, stream) : launch_d<false, float, 4>(a, stream);
}

cudaError_t launch_prologue_bwd(const PrologueArgs &a, cudaStream_t stream) {
  return a.bf16 ? launch_d<true, __nv_bfloat16, 8>(a, stream) : launch_d<true, float, 4>(a, stream);
}

}  // namespace gdr
