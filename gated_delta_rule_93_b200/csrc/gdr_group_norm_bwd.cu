// Backward of the output norm (see gdr_group_norm.cuh):
//   dl = dy act(z) or dy act'(l),  dz = dy l act'(z),  h = dl w
//   dx = rstd (h - [center] mean(h) - n mean(h n)),  dw = sum dl n,  db = sum dl
//
// The statistics are computed again from x, which is read anyway.  The weight
// gradients add up in registers over a lane's rows, then over the block (with
// weights per channel a block's slots share a group), and a second launch, set up
// while the first ends (1.2 us less), adds the blocks' partial rows in a fixed
// order; where one block has all rows of its channels, it writes the gradients
// itself.
#include "gdr_group_norm.cuh"

namespace gdr {
namespace {

// Blocks on an SM for E elements a lane.
constexpr int blocks_per_sm(int E) { return E <= 4 ? 3 : E <= 8 ? 2 : 1; }

// N pairs of a row.  On return x holds n and z dz; h, the running dw and db are
// set, and the lane's part of sum(h n) is returned.  (dy is 0 outside the group and
// behind the last row: so is all that is added up.)
template <int ACT, bool GATED, int N>
__device__ __forceinline__ float gradients(float2 (&x)[N], float2 (&z)[N], const float2 (&dy)[N],
                                           const float2 (&w)[N], const float2 (&b)[N], float rstd,
                                           float2 (&h)[N], float2 (&dw)[N], float2 (&db)[N]) {
  float2 hn = both(0.f);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float2 n = mul2(x[e], both(rstd));
    const float2 l = fma2(n, w[e], b[e]);
    const float2 u = GATED ? z[e] : l;
    float2 f = u, df = both(1.f);  // value and slope of the activation
    if constexpr (ACT != GDR_ACT_NONE) {
      const float2 s = sigmoid2(u), t = fma2(s, both(-1.f), both(1.f));
      if constexpr (ACT == GDR_ACT_SILU) {
        f = mul2(u, s);
        df = fma2(f, t, s);
      } else {
        f = s;
        df = mul2(s, t);
      }
    }
    const float2 dl = mul2(dy[e], GATED ? f : df);
    if constexpr (GATED) z[e] = mul2(mul2(dy[e], l), df);
    dw[e] = fma2(dl, n, dw[e]);
    db[e] = add2(db[e], dl);
    h[e] = mul2(dl, w[e]);
    hn = fma2(h[e], n, hn);
    x[e] = n;
  }
  return hn.x + hn.y;
}

template <typename T, int VEC, int L, int NV>
__global__ void __launch_bounds__(kRowThreads, blocks_per_sm(VEC *NV))
    group_norm_bwd_kernel(GroupNormArgs a, RowPlan p) {
  after_previous();
  let_next();
  constexpr int E = VEC * NV, N = E / 2;  // elements and pairs of a lane
  constexpr int kPerBlock = kRowThreads / L;
  const int lane = threadIdx.x % L;
  const int slot = threadIdx.x / L, g = p.group(blockIdx.x, slot, kPerBlock, a.G);
  const float inv_d = 1.f / (float)a.D;
  float2 w[N], b[N], dw[N], db[N];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) in[i] = (i * L + lane) * VEC < a.D;
  const int channel = (a.per_channel ? g * a.D : 0) + lane * VEC;
  load_affine<VEC, L, NV>(a.weight, channel, in, 1.f, w);
  load_affine<VEC, L, NV>(a.bias, channel, in, 0.f, b);
#pragma unroll
  for (int e = 0; e < N; ++e) dw[e] = db[e] = both(0.f);
  const long long first = p.first_row(blockIdx.x, slot, kPerBlock, a.G);
  const int mine = p.count(p.used(blockIdx.x, slot, kPerBlock), first, a.rows);
  const long long off = (long long)g * a.D + lane * VEC, dense = (long long)a.G * a.D;
  const T *xp = static_cast<const T *>(a.x) + off + first * a.x_stride;  // the row asked for next
  const T *zp = static_cast<const T *>(a.z) + off + first * a.z_stride;
  const T *dyp = static_cast<const T *>(a.dy) + off + first * dense;
  long long out = off + first * dense;  // of dx and dz
  const long long x_step = p.step * a.x_stride, z_step = p.step * a.z_stride;
  const long long step = p.step * dense;

  // The queue's memory takes the sums over the block at the end.
  constexpr bool kQueue = norm_queue<T, VEC, NV>;
  constexpr int kStages = NV == 1 ? 3 : 2;
  constexpr int kWaiting = kQueue ? 3 * NV : 1;
  using Waiting = Raw<T, VEC>[kQueue ? kStages : 1][kWaiting][kRowThreads];
  using Sums = float[kRowThreads / 32][L * E];
  __shared__ __align__(16) unsigned char memory[sizeof(Waiting) > sizeof(Sums) ? sizeof(Waiting)
                                                                              : sizeof(Sums)];
  Queue<Raw<T, VEC>, kWaiting, kStages> queue{*reinterpret_cast<Waiting *>(memory)};
  const auto ask = [&](int turn, int stage) {
    if (turn < mine) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (in[i]) {
          queue.request(stage, i, xp + i * L * VEC);
          queue.request(stage, NV + i, dyp + i * L * VEC);
          if (a.z) queue.request(stage, 2 * NV + i, zp + i * L * VEC);
        }
    }
    queue.commit();
    xp += x_step;
    zp += z_step;
    dyp += step;
  };
  if constexpr (kQueue) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) ask(i, i);
  }
  int stage = 0;
  for (int k = 0; k < p.turns; ++k, out += step) {
    const bool live = k < mine;
    Raw<T, VEC> xr[NV], zr[NV], dyr[NV];
    if constexpr (kQueue) {
      ask(k + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
      queue.wait();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xr[i] = zr[i] = dyr[i] = Raw<T, VEC>{};
      if (!live || !in[i]) continue;
      if constexpr (kQueue) {
        xr[i] = queue.get(stage, i);
        dyr[i] = queue.get(stage, NV + i);
        if (a.z) zr[i] = queue.get(stage, 2 * NV + i);
      } else {
        xr[i] = load_raw<T, VEC>(xp + i * L * VEC);
        dyr[i] = load_raw<T, VEC>(dyp + i * L * VEC);
        if (a.z) zr[i] = load_raw<T, VEC>(zp + i * L * VEC);
      }
    }
    if constexpr (kQueue) {
      stage = stage == kStages - 1 ? 0 : stage + 1;
    } else {
      xp += x_step;
      zp += z_step;
      dyp += step;
    }
    float2 x[N], z[N], dy[N], h[N];
    unpack_row<T, VEC, NV>(xr, x);
    const float rstd = normalise<VEC, L, NV>(x, in, a.center, inv_d, a.eps);
    unpack_row<T, VEC, NV>(zr, z);
    unpack_row<T, VEC, NV>(dyr, dy);
    float hn;
    if (a.z) {
      if (a.act == GDR_ACT_SILU)
        hn = gradients<GDR_ACT_SILU, true>(x, z, dy, w, b, rstd, h, dw, db);
      else if (a.act == GDR_ACT_SIGMOID)
        hn = gradients<GDR_ACT_SIGMOID, true>(x, z, dy, w, b, rstd, h, dw, db);
      else
        hn = gradients<GDR_ACT_NONE, true>(x, z, dy, w, b, rstd, h, dw, db);
    } else {
      if (a.act == GDR_ACT_SILU)
        hn = gradients<GDR_ACT_SILU, false>(x, z, dy, w, b, rstd, h, dw, db);
      else if (a.act == GDR_ACT_SIGMOID)
        hn = gradients<GDR_ACT_SIGMOID, false>(x, z, dy, w, b, rstd, h, dw, db);
      else
        hn = gradients<GDR_ACT_NONE, false>(x, z, dy, w, b, rstd, h, dw, db);
    }
    hn = lanes_sum<L>(hn) * inv_d;
    float mean = 0.f;  // of h
    if (a.center) {
      float2 sum = both(0.f);
#pragma unroll
      for (int e = 0; e < N; ++e) sum = add2(sum, h[e]);
      mean = lanes_sum<L>(sum.x + sum.y) * inv_d;
    }
#pragma unroll
    for (int e = 0; e < N; ++e)  // dx in place of h: rstd h - rstd mean - n (rstd hn)
      h[e] = fma2(h[e], both(rstd), fma2(x[e], both(-rstd * hn), both(-rstd * mean)));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!live || !in[i]) continue;
      const long long at = out + i * L * VEC;
      if (a.dz) store_access<T, VEC>(static_cast<T *>(a.dz) + at, z, i);
      constexpr int V4 = VEC < 4 ? VEC : 4;
#pragma unroll
      for (int e = 0; e < VEC; e += V4) store_access<float, V4>(a.dx + at + e, h, (i * VEC + e) / V4);
    }
  }

  // Partial rows of the weight gradients, a block's D values each, db behind dw:
  // over the slots of a warp, then over the warps.
  if (!a.dweight && !a.dbias) return;
  Sums &s = *reinterpret_cast<Sums *>(memory);  // (no request is left)
  const int warp = threadIdx.x / 32, at = threadIdx.x % 32;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float *to = which ? a.dbias : a.dweight;
    if (!to) continue;
    if (p.sum) to = a.ws + ((which ? (long long)p.blocks : 0) + blockIdx.x) * a.D;
    else if (p.by_block) to += (long long)g * a.D;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float v = element(which ? db : dw, e);
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
      to[c] = v;
    }
  }
}

// Rows of a lane in a block, more where that makes more than kMostBlocks blocks (each
// leaves a partial row to add up).  32768 x 16 x 128 bf16 with 8 and 16: weights shared by the
// heads 130.9 and 131.7 us, per channel (as many columns to add up as G D) with biases 154 and 137 us.
constexpr int kTurns = 8, kChannelTurns = 16;
constexpr int kMostBlocks = 8192;
constexpr int kFewTurns = 4;       // rows a slot takes rather than have a second launch

RowPlan bwd_plan(long long rows, int G, int lanes, int per_sm, int per_channel) {
  const int per_block = kRowThreads / lanes;
  const long long most = rows * G / ((long long)kMostBlocks * per_block);
  const int least = per_channel ? kChannelTurns : kTurns;
  const int turns = most > least ? (int)(most < (1 << 30) ? most : 1 << 30) : least;
  RowPlan p = row_plan(rows, G, per_block, turns, kSMs * per_sm, per_channel);
  // few rows: as few blocks as have every channel once
  if (per_channel ? rows <= kFewTurns * per_block : rows * G <= kFewTurns * per_block)
    p = row_plan(rows, G, per_block, kFewTurns, 1, per_channel);
  p.sum = p.blocks > (per_channel ? G : 1);
  return p;
}

struct Launch {
  const GroupNormArgs &a;
  cudaStream_t stream;
  template <typename T, int VEC, int L, int NV>
  cudaError_t operator()() const {
    const RowPlan p = bwd_plan(a.rows, a.G, L, blocks_per_sm(VEC * NV), a.per_channel);
    const cudaError_t e =
        launch_next(group_norm_bwd_kernel<T, VEC, L, NV>, dim3(p.blocks), kRowThreads, stream, a, p);
    if (e == cudaSuccess && p.sum && (a.dweight || a.dbias)) {
      const int rows = a.per_channel ? p.blocks / a.G : p.blocks;
      const int cols = a.per_channel ? a.G * a.D : a.D;
      return launch_sums(a.ws, rows, cols, a.dweight, a.dbias, stream);
    }
    return e;
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
