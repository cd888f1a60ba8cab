// The gated delta rule token by token over a pool of state slots.
//
// Source: "Decoding Hybrid Linear Attention Architectures", section 6 (each
// decoded token costs one constant-size update of the state) and section 3
// item 6 (decay, then erase along k, then write).  Per state row i with
// S' = S Diag(alpha):
//     p_i = S'_i . k,  r_i = S'_i . q,  u_i = beta (v_i - p_i)
//     S_i <- S'_i + u_i k^T,  o_i = r_i + u_i (k . q)
// Rows are independent, so a thread block takes 16 RPT rows of one (request,
// value head), reads them once, runs the request's tokens with the rows in
// registers and writes them wherever the request keeps a state.  One token a
// request moves 2 * 4 * dk * dv bytes per (request, head) for 7 dk dv flops:
// bound by HBM.
//
// Layout: 8 lanes share a row, lane l of them holding the float4s at columns
// 32 c + 4 l: a warp's load is four whole 128-byte lines, and a row's two dot
// products need 3 shuffle steps instead of 5.  What all rows of a head share (k, q
// with their norms, the gates, k . q) is prepared once per block, a warp per
// token, in shared memory, while the state's loads are in flight.
#include "gdr_internal.cuh"

namespace gdr {
namespace {

constexpr int kWarps = 4;
constexpr int kTokens = 4;  // tokens prepared at a time, a warp each
constexpr float kNormEps = 1e-6f;

template <int DK, bool PERCH>
struct __align__(16) Prepared {
  float k[kTokens][DK];
  float q[kTokens][DK];
  float al[kTokens][PERCH ? DK : 4];
  float beta[kTokens], kq[kTokens];
  int dst[kTokens];
};

// log(1 + e^x), with no branch that overflows.
__device__ __forceinline__ float softplus(float x) {
  return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// Sum NV per-lane values over groups of 8 lanes, halving the values while the
// lane masks allow it: afterwards a lane holds the sum of value (lane & 7) >> SH,
// NV = 8 >> SH.
template <int NV>
__device__ __forceinline__ float reduce8(float (&x)[NV], int lane) {
  static_assert(NV == 2 || NV == 4 || NV == 8);
  int n = NV;
#pragma unroll
  for (int m = 4; m; m >>= 1) {
    if (n > 1) {
      n >>= 1;
#pragma unroll
      for (int i = 0; i < NV / 2; ++i) {
        if (i < n) {
          const bool hi = lane & m;
          const float send = hi ? x[i] : x[i + n];
          const float keep = hi ? x[i + n] : x[i];
          x[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
      }
    } else {
      x[0] += __shfl_xor_sync(0xffffffffu, x[0], m);
    }
  }
  return x[0];
}

template <int DK, int RPT, bool BF16, bool PERCH>
__global__ void __launch_bounds__(kWarps * 32) gdr_step_slots_kernel(StepSlotsArgs a) {
  constexpr int NC = DK / 32;                                 // float4s of a row per lane
  constexpr int NV = 2 * RPT;                                 // dot products per thread
  constexpr int SH = NV == 8 ? 0 : NV == 4 ? 1 : 2;
  __shared__ Prepared<DK, PERCH> sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks_per_head = a.dv / (kWarps * 4 * RPT);
  const unsigned rh = blockIdx.x / blocks_per_head;
  const int r = rh / a.H, h = rh % a.H;
  const int hk = h / (a.H / a.Hk);
  const int row0 = (blockIdx.x % blocks_per_head) * (kWarps * 4 * RPT) + warp * 4 * RPT +
                   (lane >> 3);  // this thread's rows: row0 + 4 i
  const int col0 = (lane & 7) * 4;

  int t0 = r, t1 = r + 1;
  if (a.cu) {
    t0 = min(max(a.cu[r], 0), a.total);
    t1 = min(max(a.cu[r + 1], t0), a.total);
  }
  const int src = a.src[r];
  if (t0 >= t1 || src == GDR_SLOT_SKIP) return;
  if (src < GDR_SLOT_ZERO || src >= a.slots) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusSlot);
    return;
  }
  const size_t in_slot = ((size_t)h * a.dv + row0) * DK + col0;

  float s[RPT][NC * 4];
  if (src >= 0) {
    const float *p = a.pool + (size_t)src * a.slot_stride + in_slot;
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c)
        *reinterpret_cast<float4 *>(&s[i][4 * c]) =
            __ldcs(reinterpret_cast<const float4 *>(p + (size_t)i * 4 * DK + c * 32));
  } else {
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int c = 0; c < NC * 4; ++c) s[i][c] = 0.f;
  }

  for (int tb = t0; tb < t1; tb += kTokens) {
    const int n = min(kTokens, t1 - tb);
    if (tb != t0) __syncthreads();
    if (warp < n) {  // warp w prepares token tb + w, DK / 32 channels a lane
      const size_t t = tb + warp;
      const size_t th = t * a.H + h;
      float kv[NC], qv[NC], kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        kv[e] = load_in(a.k, t * a.k_stride + (size_t)hk * DK + lane + 32 * e, BF16);
        qv[e] = load_in(a.q, t * a.q_stride + (size_t)hk * DK + lane + 32 * e, BF16);
        kk += kv[e] * kv[e];
        qq += qv[e] * qv[e];
        kq += kv[e] * qv[e];
      }
      float bl = a.beta[th];
      if (a.gate_scale) bl = 1.f / (1.f + expf(-bl));
      const float sc = a.gate_scale ? a.gate_scale[h] : 0.f;
      if constexpr (PERCH) {
#pragma unroll
        for (int e = 0; e < NC; ++e) {
          float g = a.g[th * DK + lane + 32 * e];
          if (a.gate_scale) g = -sc * softplus(g);
          sm.al[warp][lane + 32 * e] = expf(g);
        }
      } else {
        float g = a.g[th];
        if (a.gate_scale) g = -sc * softplus(g);
        if (lane == 0) sm.al[warp][0] = expf(g);
      }
      kq = warp_sum(kq);
      float rk = 1.f, rq = 1.f;
      if (a.norm_qk & GDR_NORM_K) rk = rsqrtf(warp_sum(kk) + kNormEps);
      if (a.norm_qk & GDR_NORM_Q) rq = rsqrtf(warp_sum(qq) + kNormEps);
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        sm.k[warp][lane + 32 * e] = kv[e] * rk;
        sm.q[warp][lane + 32 * e] = qv[e] * rq;
      }
      if (lane == 0) {
        sm.beta[warp] = bl;
        sm.kq[warp] = kq * rk * rq;
        // where the state goes after this token (-1: nowhere)
        int d = a.dst ? a.dst[t] : (tb + warp == t1 - 1 ? src : -1);
        if (d >= a.slots || d < -1) {
          atomicOr(a.status, kStatusSlot);
          d = -1;
        }
        sm.dst[warp] = d;
      }
    }
    __syncthreads();
    for (int j = 0; j < n; ++j) {
      const size_t to = ((size_t)(tb + j) * a.H + h) * a.dv;
      const int idx = (lane & 7) >> SH;   // the dot product this lane ends up with
      const int mine = idx % RPT;         // its row: p for idx < RPT, r after
      const float v = load_in(a.v, (size_t)(tb + j) * a.v_stride + (size_t)h * a.dv + row0 + 4 * mine,
                              BF16);
      float part[NV] = {};
      float al0 = 0.f;
      if constexpr (!PERCH) al0 = sm.al[j][0];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 k4 = *reinterpret_cast<const float4 *>(&sm.k[j][col0 + 32 * c]);
        const float4 q4 = *reinterpret_cast<const float4 *>(&sm.q[j][col0 + 32 * c]);
        float4 a4 = make_float4(al0, al0, al0, al0);
        if constexpr (PERCH) a4 = *reinterpret_cast<const float4 *>(&sm.al[j][col0 + 32 * c]);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          float *x = &s[i][4 * c];
          x[0] *= a4.x; x[1] *= a4.y; x[2] *= a4.z; x[3] *= a4.w;  // decay first
          part[i] += x[0] * k4.x + x[1] * k4.y + x[2] * k4.z + x[3] * k4.w;
          part[RPT + i] += x[0] * q4.x + x[1] * q4.y + x[2] * q4.z + x[3] * q4.w;
        }
      }
      const float red = reduce8<NV>(part, lane);
      const float u_mine = sm.beta[j] * (v - red);  // meaningful where idx < RPT
      float u[RPT], um = 0.f;
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        u[i] = __shfl_sync(0xffffffffu, u_mine, (lane & 24) + (i << SH));
        if (i == mine) um = u[i];
      }
      if (idx >= RPT && (lane & ((1 << SH) - 1)) == 0)
        store_out(a.o, to + row0 + 4 * mine, red + um * sm.kq[j], BF16);
      const int d = sm.dst[j];
      float *out = a.pool + (size_t)max(d, 0) * a.slot_stride + in_slot;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 k4 = *reinterpret_cast<const float4 *>(&sm.k[j][col0 + 32 * c]);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          float *x = &s[i][4 * c];
          x[0] += u[i] * k4.x; x[1] += u[i] * k4.y; x[2] += u[i] * k4.z; x[3] += u[i] * k4.w;
          if (d >= 0)
            __stcs(reinterpret_cast<float4 *>(out + (size_t)i * 4 * DK + c * 32),
                   make_float4(x[0], x[1], x[2], x[3]));
        }
      }
    }
  }
}

template <int DK, int RPT>
cudaError_t launch_rpt(const StepSlotsArgs &a, cudaStream_t stream) {
  const size_t blocks = (size_t)a.R * a.H * (a.dv / (kWarps * 4 * RPT));
  if (blocks > 0x7fffffffu) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(kWarps * 32);
  if (a.bf16) {
    if (a.per_channel)
      gdr_step_slots_kernel<DK, RPT, true, true><<<grid, block, 0, stream>>>(a);
    else
      gdr_step_slots_kernel<DK, RPT, true, false><<<grid, block, 0, stream>>>(a);
  } else {
    if (a.per_channel)
      gdr_step_slots_kernel<DK, RPT, false, true><<<grid, block, 0, stream>>>(a);
    else
      gdr_step_slots_kernel<DK, RPT, false, false><<<grid, block, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_step_slots(const StepSlotsArgs &a, cudaStream_t stream) {
  switch (a.dk) {
    case 32: return launch_rpt<32, 2>(a, stream);
    case 64: return launch_rpt<64, 2>(a, stream);
    case 128: return launch_rpt<128, 2>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace gdr
