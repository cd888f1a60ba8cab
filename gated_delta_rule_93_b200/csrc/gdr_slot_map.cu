// Slot maps of a batch from its request lengths, in one launch.
//
// A block owns 64 or 256 requests.  It adds up every length before them by
// itself (R <= 65536 values out of L2) rather than wait for another block, scans its
// own, checks its requests' slots, and writes the tokens of its requests, a
// thread per token, finding a token's request by bisection of its offsets in
// shared memory.  The entries behind the last token are split over all blocks.  The
// work is a few KB: the launch and two dependent reads from memory bound it (3 us
// for a few requests, where an empty kernel takes 2).
#include "gdr_rows.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;
// Up to here a block owns 64 requests, so that four threads share a request's
// tokens (4096 requests of 0 to 8 tokens: 4.1 us, with 256 a block 5.6 us); beyond,
// 256, since every block reads all lengths.
constexpr int kFewRequests = 8192;
constexpr int kAhead = 8;  // lengths a thread asks for at once

__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

__global__ void __launch_bounds__(kThreads) gdr_slot_map_kernel(SlotMapArgs a, int own) {
  after_previous();
  let_next();
  constexpr int kWarps = kThreads / 32;
  __shared__ long long s_all[kWarps], s_before[kWarps], s_scan[kWarps];
  __shared__ int s_cu[kThreads + 1];
  __shared__ int s_len[kThreads];  // -1: the request is skipped
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = blockIdx.x * own, r = tid < own ? r0 + tid : a.R;  // (a.R: none)

  const int raw = r < a.R ? a.lens[r] : 0;
  const int kept = r < a.R ? a.kept[r] : 0;
  long long all = 0, before = 0;
  for (int i = tid; i < a.R; i += kAhead * kThreads) {
    int n[kAhead];  // (on their way at once)
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      n[u] = i + u * kThreads < a.R ? a.lens[i + u * kThreads] : 0;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      all += max(n[u], 0);
      if (i + u * kThreads < r0) before += max(n[u], 0);
    }
  }
  const int len = max(raw, 0);
  long long incl = len;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, m);
    if (lane >= m) incl += up;
  }
  all = warp_sum(all);
  before = warp_sum(before);
  if (lane == 31) {
    s_all[warp] = all;
    s_before[warp] = before;
    s_scan[warp] = incl;
  }
  __syncthreads();
  all = before = 0;
  long long ahead = 0;
  for (int w = 0; w < kWarps; ++w) {
    all += s_all[w];
    before += s_before[w];
    if (w < warp) ahead += s_scan[w];
  }
  const long long start = before + ahead + incl - len, cap = a.max_tokens;
  const int cu = (int)min(start, cap), end = (int)min(start + len, cap);

  bool bad = raw < 0;
  int src = GDR_SLOT_SKIP;
  const int *row = a.table + (size_t)r * a.table_stride;
  if (r < a.R && len > 0) {
    const int uses = a.keep_all ? len : 1;
    bool run = kept >= 0 && kept <= a.W && uses <= a.W && start + len <= cap;
    if (run) {
      src = GDR_SLOT_ZERO;
      if (kept > 0) {
        src = row[kept - 1];
        run = src >= 0 && src < a.slots;
      }
#pragma unroll 4
      for (int j = 0; j < uses; ++j) {
        const unsigned d = row[j];
        run &= d < (unsigned)a.slots;
      }
    }
    if (!run) {
      src = GDR_SLOT_SKIP;
      bad = true;
    }
  }
  if (bad) atomicOr(a.status, kStatusSlot);
  s_cu[tid] = cu;
  if (tid == kThreads - 1) s_cu[kThreads] = end;
  s_len[tid] = src == GDR_SLOT_SKIP ? -1 : len;
  if (r < a.R) {
    a.cu[r] = cu;
    a.src[r] = src;
    if (r == a.R - 1) a.cu[a.R] = end;
  } else if (a.R == 0 && tid == 0) {
    a.cu[0] = 0;  // no request at all
  }
  __syncthreads();

  // (unsigned: the step behind the last of 2^31 - 1 tokens does not wrap)
  for (unsigned t = s_cu[0] + tid; t < (unsigned)s_cu[own]; t += kThreads) {
    int lo = 0, hi = own;  // s_cu[lo] <= t < s_cu[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((unsigned)s_cu[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const int at = t - s_cu[lo], n = s_len[lo];
    const int *named = a.table + (size_t)(r0 + lo) * a.table_stride;
    int d = -1;
    if (n >= 0) {
      if (a.keep_all)
        d = named[at];
      else if (at == n - 1)
        d = named[0];
    }
    a.request[t] = r0 + lo;
    a.dst[t] = d;
  }
  for (long long t = min(all, cap) + (long long)blockIdx.x * kThreads + tid; t < cap;
       t += (long long)gridDim.x * kThreads) {
    a.request[t] = -1;
    a.dst[t] = -1;
  }
}

}  // namespace

cudaError_t launch_slot_map(const SlotMapArgs &a, cudaStream_t stream) {
  const int own = a.R <= kFewRequests ? kThreads / 4 : kThreads;
  const int blocks = a.R > 0 ? (a.R + own - 1) / own : 1;
  return launch_next(gdr_slot_map_kernel, dim3(blocks), kThreads, stream, a, own);
}

}  // namespace gdr
