// The gated delta rule token by token over a pool of state slots.
//
// Source: "Decoding Hybrid Linear Attention Architectures", section 6 (each
// decoded token costs one constant-size update of the state) and section 3
// item 6 (decay, then erase along k, then write).  Per state row i with
// S' = S Diag(alpha):
//     p_i = S'_i . k,  r_i = S'_i . q,  u_i = beta (v_i - p_i)
//     S_i <- S'_i + u_i k^T,  o_i = r_i + u_i (k . q)
// Rows are independent, so a block takes some rows of one (request, value
// head), reads them once, runs the request's tokens with the rows in registers
// and writes them wherever the request keeps a state.  One token a request moves
// 2 * 4 * dk * dv bytes per (request, head) for 7 dk dv flops: bound by HBM.  Two
// kernels, by whether the call has cu_seqlens (and see launch_dk):
//
// One token a request: a warp for 8 rows that prepares k, q and the gate for
// itself, no shared memory, no barrier.  256 requests x 16 heads of 128 x 128:
// 83.1 us, 6508 GB/s (a copy runs at 6456); with the preparation shared by a block,
// whose warps then load, wait and store in step, 90 to 95 us.
//
// Several tokens: a block of 4 warps takes 64 rows (2 warps, 32 rows, where dv is
// 32), and what all rows of a head share (k, q with their norms, the gates, k . q)
// is prepared once per block in shared memory, 8 tokens at a time, two a warp.
// 8 lanes share a row, lane l of them holding the float4s at columns 32 c + 4 l (a
// warp's load is four whole 128-byte lines), and a lane has 4 rows, so that the
// shared k and q are read once for 4 rows and a row's two dot products cost 7/4
// shuffles.  48 requests of 1 to 5 tokens, 32 heads of 128 x 128, every state kept:
// 65.1 us, 6144 GB/s; 64 requests of 1 to 4 tokens, 16 heads, one state kept: 26.9 us
// (2 rows a lane in blocks of 8 warps: 71.2 and 36.1 us).  Long requests run at about
// 0.6 us a token (8 requests x 16 heads), bound by the instructions and the latency of
// one token after the other: 13.0 us with 16 tokens, where the chunked forward takes 14.2, and
// 22.9 us with 32, where it takes 14.7.
#include "gdr_rows.cuh"

namespace gdr {
namespace {

constexpr int kRpt = 4;             // rows of a lane, 4 apart
constexpr int kWarpRows = 4 * kRpt;  // rows of a warp
constexpr int kTokens = 8;           // tokens prepared at a time
constexpr int rows_of(int warps) { return kWarpRows * warps; }  // of a block

constexpr float kNormEps = 1e-6f;

template <int DK, int WARPS, bool PERCH>
struct __align__(16) Prepared {
  float k[kTokens][DK];
  float q[kTokens][DK];
  float al[kTokens][PERCH ? DK : 4];
  float v[kTokens][rows_of(WARPS)];
  float beta[kTokens], kq[kTokens];
  int dst[kTokens];
};

// VEC consecutive values of a lane: q, k, v or a gate, and the state's (read once).
template <int VEC, bool BF16>
__device__ __forceinline__ void load_lane(const void *p, size_t i, float (&x)[VEC]) {
  if constexpr (!BF16 && VEC == 4) {
    const float4 t = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
  } else if constexpr (!BF16 && VEC == 2) {
    const float2 t = *reinterpret_cast<const float2 *>(static_cast<const float *>(p) + i);
    x[0] = t.x; x[1] = t.y;
  } else if constexpr (BF16 && VEC == 2) {
    const unsigned t = *reinterpret_cast<const unsigned *>(static_cast<const __nv_bfloat16 *>(p) + i);
    x[0] = __uint_as_float(t << 16); x[1] = __uint_as_float(t & 0xffff0000u);
  } else if constexpr (BF16 && VEC == 4) {
    const uint2 t = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + i);
    x[0] = __uint_as_float(t.x << 16); x[1] = __uint_as_float(t.x & 0xffff0000u);
    x[2] = __uint_as_float(t.y << 16); x[3] = __uint_as_float(t.y & 0xffff0000u);
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] = load_in(p, i + e, BF16);
  }
}
template <int VEC>
__device__ __forceinline__ void store_lane(float *p, const float (&x)[VEC]) {
  if constexpr (VEC == 4)
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else if constexpr (VEC == 2)
    *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
  else
    p[0] = x[0];
}
template <int VEC>
__device__ __forceinline__ void load_lane_stream(const float *p, float (&x)[VEC]) {
  if constexpr (VEC == 4) {
    const float4 t = __ldcs(reinterpret_cast<const float4 *>(p));
    x[0] = t.x; x[1] = t.y; x[2] = t.z; x[3] = t.w;
  } else if constexpr (VEC == 2) {
    const float2 t = __ldcs(reinterpret_cast<const float2 *>(p));
    x[0] = t.x; x[1] = t.y;
  } else {
    x[0] = __ldcs(p);
  }
}
template <int VEC>
__device__ __forceinline__ void store_lane_stream(float *p, const float (&x)[VEC]) {
  if constexpr (VEC == 4)
    __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
  else if constexpr (VEC == 2)
    __stcs(reinterpret_cast<float2 *>(p), make_float2(x[0], x[1]));
  else
    __stcs(p, x[0]);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// Sums 8 per-lane values over groups of 8 lanes, halving the values each
// time: lane l ends up with the sum of value l & 7.
__device__ __forceinline__ float reduce8(float (&x)[8], int lane) {
#pragma unroll
  for (int m = 4; m; m >>= 1)
#pragma unroll
    for (int i = 0; i < m; ++i) {
      const bool hi = lane & m;
      const float send = hi ? x[i] : x[i + m];
      const float keep = hi ? x[i + m] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
    }
  return x[0];
}

template <int DK, int WARPS, bool BF16, bool PERCH>
__global__ void __launch_bounds__(WARPS * 32, (DK == 128 ? 16 : DK == 64 ? 24 : 32) / WARPS)
    gdr_step_slots_kernel(StepSlotsArgs a) {
  after_previous();
  let_next();
  constexpr int kRows = rows_of(WARPS);
  constexpr int NC = DK / 32;  // float4s of a row per lane
  __shared__ Prepared<DK, WARPS, PERCH> sm;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks_per_head = a.dv / kRows;
  const unsigned rh = blockIdx.x / blocks_per_head;
  const int r = rh / a.H, h = rh % a.H;
  const int hk = h / (a.H / a.Hk);
  const int block_row = blockIdx.x % blocks_per_head * kRows;
  const int in_block = warp * kWarpRows + (lane >> 3);  // this thread's rows: in_block + 4 i
  const int row0 = block_row + in_block;
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

  float2 s[kRpt][2 * NC];
  if (src >= 0) {
    const float *p = a.pool + (size_t)src * a.slot_stride + in_slot;
#pragma unroll
    for (int i = 0; i < kRpt; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 x = __ldcs(reinterpret_cast<const float4 *>(p + i * 4 * DK + c * 32));
        s[i][2 * c] = make_float2(x.x, x.y);
        s[i][2 * c + 1] = make_float2(x.z, x.w);
      }
  } else {
#pragma unroll
    for (int i = 0; i < kRpt; ++i)
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) s[i][c] = make_float2(0.f, 0.f);
  }

  for (int tb = t0; tb < t1; tb += kTokens) {
    const int n = min(kTokens, t1 - tb);
    if (tb != t0) __syncthreads();
    for (int j = warp; j < n; j += WARPS) {  // a token a warp, DK / 32 channels a lane
      const size_t t = tb + j, th = t * a.H + h;
      float kv[NC], qv[NC], gv[PERCH ? NC : 1];
      load_lane<NC, BF16>(a.k, t * a.k_stride + (size_t)hk * DK + lane * NC, kv);
      load_lane<NC, BF16>(a.q, t * a.q_stride + (size_t)hk * DK + lane * NC, qv);
      if constexpr (PERCH)
        load_lane<NC, false>(a.g, th * DK + lane * NC, gv);
      else
        gv[0] = a.g[th];
      const float bl = a.beta[th];
      // where the state goes after this token (-1: nowhere)
      int d = a.dst ? a.dst[t] : ((int)t == t1 - 1 ? src : -1);
      float vv[kRows / 32];
      load_lane<kRows / 32, BF16>(
          a.v, t * a.v_stride + (size_t)h * a.dv + block_row + lane * (kRows / 32), vv);
      const float scale = a.gate_scale ? a.gate_scale[h] : 0.f;
      float kk = 0.f, qq = 0.f, kq = 0.f, rk = 1.f, rq = 1.f;
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        kk += kv[e] * kv[e];
        qq += qv[e] * qv[e];
        kq += kv[e] * qv[e];
      }
      kq = warp_sum(kq);
      if (a.norm_qk & GDR_NORM_K) rk = rsqrtf(warp_sum(kk) + kNormEps);
      if (a.norm_qk & GDR_NORM_Q) rq = rsqrtf(warp_sum(qq) + kNormEps);
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        kv[e] *= rk;
        qv[e] *= rq;
        if constexpr (PERCH)
          gv[e] = expf(a.gate_scale ? -scale * softplus(gv[e]) : gv[e]);
      }
      store_lane<NC>(&sm.k[j][lane * NC], kv);
      store_lane<NC>(&sm.q[j][lane * NC], qv);
      if constexpr (PERCH) store_lane<NC>(&sm.al[j][lane * NC], gv);
      store_lane<kRows / 32>(&sm.v[j][lane * (kRows / 32)], vv);
      if (lane == 0) {
        if constexpr (!PERCH)
          sm.al[j][0] = expf(a.gate_scale ? -scale * softplus(gv[0]) : gv[0]);
        sm.beta[j] = a.gate_scale ? sigmoid(bl) : bl;
        sm.kq[j] = kq * rk * rq;
        if (d >= a.slots || d < -1) {
          atomicOr(a.status, kStatusSlot);
          d = -1;
        }
        sm.dst[j] = d;
      }
    }
    __syncthreads();
    for (int j = 0; j < n; ++j) {
      const size_t to = ((size_t)(tb + j) * a.H + h) * a.dv;
      // the dot product this lane ends up with: p of row `mine` on lanes 0-3 of 8, r on 4-7
      const int mine = lane & 3;
      const bool is_p = !(lane & 4);
      const float v = sm.v[j][in_block + 4 * mine];
      float2 p2[kRpt] = {}, r2[kRpt] = {}, kr[2 * NC];
      float2 al = both(0.f);
      if constexpr (!PERCH) al = both(sm.al[j][0]);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 k4 = *reinterpret_cast<const float4 *>(&sm.k[j][col0 + 32 * c]);
        const float4 q4 = *reinterpret_cast<const float4 *>(&sm.q[j][col0 + 32 * c]);
        float4 a4;
        if constexpr (PERCH) a4 = *reinterpret_cast<const float4 *>(&sm.al[j][col0 + 32 * c]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float2 k2 = half ? make_float2(k4.z, k4.w) : make_float2(k4.x, k4.y);
          kr[2 * c + half] = k2;
          const float2 q2 = half ? make_float2(q4.z, q4.w) : make_float2(q4.x, q4.y);
          if constexpr (PERCH) al = half ? make_float2(a4.z, a4.w) : make_float2(a4.x, a4.y);
#pragma unroll
          for (int i = 0; i < kRpt; ++i) {
            float2 &x = s[i][2 * c + half];
            x = mul2(x, al);  // decay first
            p2[i] = fma2(x, k2, p2[i]);
            r2[i] = fma2(x, q2, r2[i]);
          }
        }
      }
      float part[2 * kRpt];
#pragma unroll
      for (int i = 0; i < kRpt; ++i) {
        part[i] = p2[i].x + p2[i].y;
        part[kRpt + i] = r2[i].x + r2[i].y;
      }
      const float red = reduce8(part, lane);
      const float u_mine = sm.beta[j] * (v - red);  // meaningful where is_p
      float u[kRpt], um = 0.f;
#pragma unroll
      for (int i = 0; i < kRpt; ++i) {
        u[i] = __shfl_sync(0xffffffffu, u_mine, (lane & 24) + i);
        if (i == mine) um = u[i];
      }
      if (!is_p)
        store_out(a.o, to + row0 + 4 * mine, red + um * sm.kq[j], BF16);
      const int d = sm.dst[j];
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c)
#pragma unroll
        for (int i = 0; i < kRpt; ++i) s[i][c] = fma2(both(u[i]), kr[c], s[i][c]);
      if (d >= 0) {
        float *out = a.pool + (size_t)d * a.slot_stride + in_slot;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int i = 0; i < kRpt; ++i)
            __stcs(reinterpret_cast<float4 *>(out + i * 4 * DK + c * 32),
                   make_float4(s[i][2 * c].x, s[i][2 * c].y, s[i][2 * c + 1].x, s[i][2 * c + 1].y));
      }
    }
  }
}

// One token a request (a decode step): 8 rows a warp, lane l holding channels
// [l DK / 32, (l + 1) DK / 32) of each, so that k, q and the gate are DK / 32
// values a lane and every warp prepares them for itself: nothing is shared and
// nothing waits at a barrier, and a warp's stores leave while others load.
template <int DK, bool BF16, bool PERCH>
__global__ void __launch_bounds__(128, 7) gdr_step_slots_one_kernel(StepSlotsArgs a) {
  after_previous();
  let_next();
  constexpr int VEC = DK / 32, kRows = 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks_per_head = a.dv / (4 * kRows);
  const unsigned rh = blockIdx.x / blocks_per_head;
  const int r = rh / a.H, h = rh % a.H;
  const int hk = h / (a.H / a.Hk);
  const int row0 = (blockIdx.x % blocks_per_head) * 4 * kRows + warp * kRows;
  const int src = a.src[r];
  int dst = a.dst ? a.dst[r] : src;
  const size_t th = rh;
  // (requested before the slot is known)
  float kv[VEC], qv[VEC], al[VEC];
  load_lane<VEC, BF16>(a.k, (size_t)r * a.k_stride + (size_t)hk * DK + lane * VEC, kv);
  load_lane<VEC, BF16>(a.q, (size_t)r * a.q_stride + (size_t)hk * DK + lane * VEC, qv);
  if constexpr (PERCH)
    load_lane<VEC, false>(a.g, th * DK + lane * VEC, al);
  else
    al[0] = a.g[th];
  float beta = a.beta[th];
  // v of row (lane / 2) % 8, as the sums come out below
  const float v = load_in(a.v, (size_t)r * a.v_stride + (size_t)h * a.dv + row0 + ((lane >> 1) & 7), BF16);

  if (src == GDR_SLOT_SKIP) return;
  if (src < GDR_SLOT_ZERO || src >= a.slots) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusSlot);
    return;
  }
  if (a.dst && (dst < -1 || dst >= a.slots)) {
    if (threadIdx.x == 0) atomicOr(a.status, kStatusSlot);
    dst = -1;
  }
  const size_t in_slot = ((size_t)h * a.dv + row0) * DK + lane * VEC;
  float s[kRows][VEC];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (src >= 0) {
      load_lane_stream<VEC>(a.pool + (size_t)src * a.slot_stride + in_slot + i * DK, s[i]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[i][e] = 0.f;
    }
  }

  float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    kk += kv[e] * kv[e];
    qq += qv[e] * qv[e];
    kq += kv[e] * qv[e];
  }
  kq = warp_sum(kq);
  if (a.norm_qk & GDR_NORM_K) {
    const float f = rsqrtf(warp_sum(kk) + kNormEps);
    kq *= f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) kv[e] *= f;
  }
  if (a.norm_qk & GDR_NORM_Q) {
    const float f = rsqrtf(warp_sum(qq) + kNormEps);
    kq *= f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) qv[e] *= f;
  }
  const float scale = a.gate_scale ? a.gate_scale[h] : 0.f;
  if (a.gate_scale) beta = sigmoid(beta);
#pragma unroll
  for (int e = 0; e < (PERCH ? VEC : 1); ++e)
    al[e] = expf(a.gate_scale ? -scale * softplus(al[e]) : al[e]);
  if constexpr (!PERCH) {
#pragma unroll
    for (int e = 1; e < VEC; ++e) al[e] = al[0];
  }

  float part[16];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float p = 0.f, o = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      s[i][e] *= al[e];  // decay first
      p += s[i][e] * kv[e];
      o += s[i][e] * qv[e];
    }
    part[i] = p;
    part[8 + i] = o;
  }
  // Halving sums over the warp: lane l ends up with value l / 2 (p of row l / 2 below 8, else
  // r of row l / 2 - 8).
#pragma unroll
  for (int m = 16, n = 8; n; m >>= 1, n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool hi = lane & m;
      const float send = hi ? part[i] : part[i + n];
      const float keep = hi ? part[i + n] : part[i];
      part[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
    }
  const float red = part[0] + __shfl_xor_sync(0xffffffffu, part[0], 1);
  const float u_mine = beta * (v - red);  // meaningful on lanes < 16
  const float u_row = __shfl_sync(0xffffffffu, u_mine, lane & 15);
  if (lane >= 16 && !(lane & 1))
    store_out(a.o, th * a.dv + row0 + ((lane >> 1) & 7), red + u_row * kq, BF16);
  if (dst < 0) return;
  float *out = a.pool + (size_t)dst * a.slot_stride + in_slot;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float u = __shfl_sync(0xffffffffu, u_mine, 2 * i);
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[i][e] += u * kv[e];
    store_lane_stream<VEC>(out + i * DK, s[i]);
  }
}

template <int DK, int WARPS>
cudaError_t launch_warps(const StepSlotsArgs &a, cudaStream_t stream) {
  const size_t blocks = (size_t)a.R * a.H * (a.dv / rows_of(WARPS));
  if (blocks > 0x7fffffffu) return cudaErrorInvalidValue;
  const auto kernel = a.bf16 ? (a.per_channel ? gdr_step_slots_kernel<DK, WARPS, true, true>
                                              : gdr_step_slots_kernel<DK, WARPS, true, false>)
                             : (a.per_channel ? gdr_step_slots_kernel<DK, WARPS, false, true>
                                              : gdr_step_slots_kernel<DK, WARPS, false, false>);
  return launch_next(kernel, dim3((unsigned)blocks), WARPS * 32, stream, a);
}

template <int DK>
cudaError_t launch_dk(const StepSlotsArgs &a, cudaStream_t stream) {
  // One token a request: a warp for itself, whose lanes load DK / 32 floats at a time.  With
  // DK = 32 that is 4 bytes, and many rows go faster through the block kernel's 16 bytes (1024
  // states of 32 x 32 3.4 against 4.1 us, of 128 x 32 6.5 against 9.2 us; 128 states of
  // 128 x 32, and the launch of fewer, 2.7 against 2.7 us and 2.5 against 2.2 us).
  if (!a.cu && (DK > 32 || (long long)a.R * a.H * a.dv <= 128 * 128)) {
    const size_t blocks = (size_t)a.R * a.H * (a.dv / 32);
    if (blocks > 0x7fffffffu) return cudaErrorInvalidValue;
    const auto kernel = a.bf16 ? (a.per_channel ? gdr_step_slots_one_kernel<DK, true, true>
                                                : gdr_step_slots_one_kernel<DK, true, false>)
                               : (a.per_channel ? gdr_step_slots_one_kernel<DK, false, true>
                                                : gdr_step_slots_one_kernel<DK, false, false>);
    return launch_next(kernel, dim3((unsigned)blocks), 128, stream, a);
  }
  constexpr int kWarps = 4;
  return a.dv == 32 ? launch_warps<DK, 2>(a, stream) : launch_warps<DK, kWarps>(a, stream);
}

}  // namespace

cudaError_t launch_step_slots(const StepSlotsArgs &a, cudaStream_t stream) {
  switch (a.dk) {
    case 32: return launch_dk<32>(a, stream);
    case 64: return launch_dk<64>(a, stream);
    case 128: return launch_dk<128>(a, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace gdr
