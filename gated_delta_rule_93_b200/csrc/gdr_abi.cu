// C ABI of the gated delta-rule library: argument validation, dispatch to
// the kernels, status reporting.  See include/gdr.h for the contract.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "gdr_internal.cuh"
#include "gdr_testing.h"

namespace gdr {
__device__ unsigned int g_device_status = 0;
}

namespace {

thread_local char t_msg[512] = "";
thread_local int t_skip_stage_chunk = -1;  // testing hook, consumed by the next call

gdr_status fail(gdr_status s, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_msg, sizeof t_msg, fmt, ap);
  va_end(ap);
  return s;
}

gdr_status ok() {
  t_msg[0] = '\0';
  return GDR_OK;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool aligned_to(const void *p, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

bool aligned4(const void *p) { return aligned_to(p, 4); }

bool head_dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

gdr_status from_cuda(cudaError_t e, const char *what) {
  if (e == cudaSuccess) return ok();
  return fail(GDR_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

gdr_status check_kinds(gdr_dtype in_dtype, gdr_gate_kind gate, int norm_qk) {
  if (in_dtype != GDR_F32 && in_dtype != GDR_BF16)
    return fail(GDR_ERR_INVALID_ARG, "in_dtype must be GDR_F32 or GDR_BF16");
  if (gate != GDR_GATE_SCALAR && gate != GDR_GATE_PER_CHANNEL)
    return fail(GDR_ERR_INVALID_ARG, "unknown gate kind");
  if (norm_qk < 0 || norm_qk > 3) return fail(GDR_ERR_INVALID_ARG, "norm_qk must be 0..3");
  return GDR_OK;
}

// A distance between rows of `width` elements: no overlap, whole 16-byte units.
gdr_status check_stride(const char *name, long long stride, long long width, long long rows,
                        gdr_dtype dtype) {
  if (rows <= 1) return GDR_OK;  // (never multiplied by more than zero)
  if (stride < width)
    return fail(GDR_ERR_INVALID_ARG, "%s stride %lld is less than a row's %lld elements", name,
                stride, width);
  if (stride % (dtype == GDR_BF16 ? 8 : 4) != 0)
    return fail(GDR_ERR_INVALID_ARG, "%s stride %lld is not a multiple of 16 bytes", name, stride);
  if (stride > (1ll << 40) / rows)
    return fail(GDR_ERR_INVALID_ARG, "%s stride %lld: problem too large", name, stride);
  return GDR_OK;
}

// Number of SMs of the current device (cached per device; 0 if unknown).
int device_sms() {
  static int cache[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  if (!cache[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    cache[dev] = n;
  }
  return cache[dev];
}

// The arguments as the kernels see them (no pointers).
gdr::ChunkArgs chunk_shape(int B, int T, int H, int dk, int dv, gdr_dtype in_dtype,
                           gdr_gate_kind gate) {
  gdr::ChunkArgs a{};
  a.B = B; a.T = T; a.H = H; a.dk = dk; a.dv = dv;
  a.bf16 = in_dtype == GDR_BF16;
  a.per_channel = gate == GDR_GATE_PER_CHANNEL;
  a.skip_stage_chunk = -1;
  a.s0_seg = 0;
  a.s0_identity = 0;
  a.write_o = 1;
  return a;
}

// Segments per sequence for this problem on the current device (1: none).
int segments_for(int B, int T, int H, int dk, int dv, int C, gdr_dtype in_dtype,
                 gdr_gate_kind gate) {
  if (B <= 0 || T <= 0 || H <= 0 || C != 64) return 1;
  if (in_dtype != GDR_F32 && in_dtype != GDR_BF16) return 1;
  if (gate != GDR_GATE_SCALAR && gate != GDR_GATE_PER_CHANNEL) return 1;
  return gdr::chunk_segments(chunk_shape(B, T, H, dk, dv, in_dtype, gate), device_sms());
}

// Device address of the status word on the current device (cached per device).
cudaError_t status_word(unsigned int **out) {
  static unsigned int *cache[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!cache[dev]) {
    void *p = nullptr;
    e = cudaGetSymbolAddress(&p, gdr::g_device_status);
    if (e != cudaSuccess) return e;
    cache[dev] = static_cast<unsigned int *>(p);
  }
  *out = cache[dev];
  return cudaSuccess;
}

}  // namespace

extern "C" {

int gdr_version(void) { return 100; }

const char *gdr_status_string(gdr_status s) {
  switch (s) {
    case GDR_OK: return "GDR_OK";
    case GDR_ERR_INVALID_ARG: return "GDR_ERR_INVALID_ARG";
    case GDR_ERR_UNSUPPORTED: return "GDR_ERR_UNSUPPORTED";
    case GDR_ERR_WORKSPACE: return "GDR_ERR_WORKSPACE";
    case GDR_ERR_CUDA: return "GDR_ERR_CUDA";
    case GDR_ERR_TIMEOUT: return "GDR_ERR_TIMEOUT";
    case GDR_ERR_RANGE: return "GDR_ERR_RANGE";
    case GDR_ERR_SLOT: return "GDR_ERR_SLOT";
  }
  return "GDR_ERR_UNKNOWN";
}

const char *gdr_last_error_message(void) { return t_msg; }

size_t gdr_chunk_fwd_workspace_bytes(int B, int T, int H, int dk, int dv, int C,
                                     gdr_dtype in_dtype, gdr_gate_kind gate) {
  // Only the segment path of long sequences with few (b, h) needs scratch
  // (one fp32 state per segment and head, three sets); every kernel keeps its
  // intermediates on chip.
  const int P = segments_for(B, T, H, dk, dv, C, in_dtype, gate);
  return gdr::chunk_segments_ws_bytes(chunk_shape(B, T, H, dk, dv, in_dtype, gate), P);
}

int gdr_chunk_fwd_kernel_launches(int B, int T, int H, int dk, int dv, int C,
                                  gdr_dtype in_dtype, gdr_gate_kind gate) {
  if (B <= 0 || H <= 0 || T < 0) return 0;
  return segments_for(B, T, H, dk, dv, C, in_dtype, gate) > 1 ? 4 : 1;
}

}  // extern "C"

namespace {

// Checks shared by the chunked-forward entry points (everything but the
// workspace); fills the kernel arguments.  Returns GDR_OK or the error.
// (need_beta = false: beta is not read and may be null)
gdr_status check_chunk(const void *q, const void *k, const void *v, gdr_dtype in_dtype,
                       const float *g, gdr_gate_kind gate, const float *beta, const float *S0,
                       void *o, float *S_T, int B, int T, int H, int dk, int dv, int C,
                       gdr::ChunkArgs *out, bool need_beta = true) {
  if (B < 0 || T < 0 || H < 0) return fail(GDR_ERR_INVALID_ARG, "negative B/T/H");
  if (in_dtype != GDR_F32 && in_dtype != GDR_BF16)
    return fail(GDR_ERR_INVALID_ARG, "in_dtype must be GDR_F32 or GDR_BF16");
  if (gate != GDR_GATE_SCALAR && gate != GDR_GATE_PER_CHANNEL)
    return fail(GDR_ERR_INVALID_ARG, "unknown gate kind");
  if (C != 64) return fail(GDR_ERR_UNSUPPORTED, "chunk size C=%d (only 64 is built)", C);
  if (!head_dim_ok(dk) || !head_dim_ok(dv))
    return fail(GDR_ERR_UNSUPPORTED, "head dims dk=%d dv=%d (need 32, 64 or 128)", dk, dv);
  if ((size_t)B * (size_t)H * (size_t)T > (size_t)1 << 40)
    return fail(GDR_ERR_INVALID_ARG, "problem too large");
  const bool empty_tokens = (size_t)B * H * T == 0;
  if (!empty_tokens) {
    if (!q || !k || !v || !g || (need_beta && !beta) || !o)
      return fail(GDR_ERR_INVALID_ARG, need_beta ? "null q/k/v/g/beta/o" : "null q/k/v/g/o");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) ||
        (need_beta && !aligned16(beta)) || !aligned16(o))
      return fail(GDR_ERR_INVALID_ARG, "q/k/v/g/beta/o must be 16-byte aligned");
  }
  if ((S0 && !aligned16(S0)) || (S_T && !aligned16(S_T)))
    return fail(GDR_ERR_INVALID_ARG, "S0/S_T must be 16-byte aligned");
  gdr::ChunkArgs a = chunk_shape(B, T, H, dk, dv, in_dtype, gate);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S0 = S0; a.o = o; a.S_T = S_T;
  *out = a;
  return ok();
}

}  // namespace

extern "C" {

gdr_status gdr_chunk_fwd(const void *q, const void *k, const void *v, gdr_dtype in_dtype,
                         const float *g, gdr_gate_kind gate, const float *beta,
                         const float *S0, void *o, float *S_T, int B, int T, int H, int dk,
                         int dv, int C, void *workspace, size_t ws_bytes,
                         gdr_stream_t stream) {
  gdr::ChunkArgs a;
  gdr_status st = check_chunk(q, k, v, in_dtype, g, gate, beta, S0, o, S_T, B, T, H, dk, dv, C,
                              &a);
  if (st != GDR_OK) return st;
  const size_t need_ws = gdr_chunk_fwd_workspace_bytes(B, T, H, dk, dv, C, in_dtype, gate);
  if (ws_bytes < need_ws || (need_ws && !workspace))
    return fail(GDR_ERR_WORKSPACE, "workspace %zu B < required %zu B", ws_bytes, need_ws);
  if (need_ws && !aligned16(workspace))
    return fail(GDR_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  if ((size_t)B * H == 0) return ok();
  a.skip_stage_chunk = t_skip_stage_chunk;
  t_skip_stage_chunk = -1;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return from_cuda(e, "gdr_chunk_fwd status word");
  // (an armed load-skip test hook keeps the single-pass kernel)
  const int P = a.skip_stage_chunk >= 0 ? 1 : segments_for(B, T, H, dk, dv, C, in_dtype, gate);
  if (P > 1)
    e = gdr::launch_chunk_segments(a, P, workspace, s);
  else if (gdr::chunk_tc_supports(a))
    e = gdr::launch_chunk_tc(a, s);
  else
    e = gdr::launch_chunk_split(a, s);
  return from_cuda(e, "gdr_chunk_fwd launch");
}

gdr_status gdr_chunk_fwd_segmented(const void *q, const void *k, const void *v,
                                   gdr_dtype in_dtype, const float *g, gdr_gate_kind gate,
                                   const float *beta, const float *S0, void *o, float *S_T,
                                   int B, int T, int H, int dk, int dv, int C, int P,
                                   void *workspace, size_t ws_bytes, gdr_stream_t stream) {
  gdr::ChunkArgs a;
  gdr_status st = check_chunk(q, k, v, in_dtype, g, gate, beta, S0, o, S_T, B, T, H, dk, dv, C,
                              &a);
  if (st != GDR_OK) return st;
  if (in_dtype != GDR_BF16 || dk != 128 || dv != 128)
    return fail(GDR_ERR_UNSUPPORTED, "segments need bf16 inputs and dk = dv = 128");
  if (P < 2 || T <= 0 || T % (64 * P) != 0)
    return fail(GDR_ERR_UNSUPPORTED, "P=%d segments of whole 64-token chunks (T=%d)", P, T);
  if ((size_t)B * P * H > (size_t)1 << 31) return fail(GDR_ERR_INVALID_ARG, "B*P*H too large");
  const size_t need_ws = gdr::chunk_segments_ws_bytes(a, P);
  if (ws_bytes < need_ws || !workspace)
    return fail(GDR_ERR_WORKSPACE, "workspace %zu B < required %zu B", ws_bytes, need_ws);
  if (!aligned16(workspace)) return fail(GDR_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  if ((size_t)B * H == 0) return ok();
  a.skip_stage_chunk = -1;
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return from_cuda(e, "gdr_chunk_fwd_segmented status word");
  return from_cuda(gdr::launch_chunk_segments(a, P, workspace,
                                              reinterpret_cast<cudaStream_t>(stream)),
                   "gdr_chunk_fwd_segmented launch");
}

// The segment path with its scratch in the library's fixed array instead of
// a caller's workspace, for callers that cannot allocate device memory when
// they run the mixer (see gdr.h).  Validation as gdr_chunk_fwd_segmented;
// sizes beyond the array are refused before anything touches the device.
gdr_status gdr_chunk_fwd_segmented_noalloc(const void *q, const void *k, const void *v,
                                           gdr_dtype in_dtype, const float *g,
                                           gdr_gate_kind gate, const float *beta,
                                           const float *S0, void *o, float *S_T, int B, int T,
                                           int H, int dk, int dv, int C, int P,
                                           gdr_stream_t stream) {
  gdr::ChunkArgs a;
  gdr_status st = check_chunk(q, k, v, in_dtype, g, gate, beta, S0, o, S_T, B, T, H, dk, dv, C,
                              &a);
  if (st != GDR_OK) return st;
  if (in_dtype != GDR_BF16 || dk != 128 || dv != 128)
    return fail(GDR_ERR_UNSUPPORTED, "segments need bf16 inputs and dk = dv = 128");
  if (P < 2 || T <= 0 || T % (64 * P) != 0)
    return fail(GDR_ERR_UNSUPPORTED, "P=%d segments of whole 64-token chunks (T=%d)", P, T);
  if ((size_t)B * P * H > (size_t)1 << 31) return fail(GDR_ERR_INVALID_ARG, "B*P*H too large");
  const size_t need = gdr::chunk_segments_ws_bytes(a, P);
  if (need > (size_t)GDR_NOALLOC_SCRATCH_BYTES)
    return fail(GDR_ERR_WORKSPACE,
                "needs %zu B of scratch (B*P*H = %zu segment-heads); the library's fixed array "
                "holds %zu B (B*P*H <= %zu)",
                need, (size_t)B * P * H, (size_t)GDR_NOALLOC_SCRATCH_BYTES,
                (size_t)GDR_NOALLOC_SCRATCH_BYTES / (3 * (size_t)dv * dk * sizeof(float)));
  if ((size_t)B * H == 0) return ok();
  a.skip_stage_chunk = -1;
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return from_cuda(e, "gdr_chunk_fwd_segmented_noalloc status word");
  void *scratch = nullptr;
  e = gdr::noalloc_scratch(&scratch);
  if (e != cudaSuccess) return from_cuda(e, "gdr_chunk_fwd_segmented_noalloc scratch address");
  return from_cuda(gdr::launch_chunk_segments(a, P, scratch,
                                              reinterpret_cast<cudaStream_t>(stream)),
                   "gdr_chunk_fwd_segmented_noalloc launch");
}

gdr_status gdr_chunk_fwd_varlen(const void *q, const void *k, const void *v, gdr_dtype in_dtype,
                                const float *g, gdr_gate_kind gate, const float *beta,
                                const int *cu_seqlens, const float *S0, void *o, float *S_T,
                                int N, int total_T, int H, int dk, int dv, int C,
                                gdr_stream_t stream) {
  if (N < 0) return fail(GDR_ERR_INVALID_ARG, "negative N");
  gdr::ChunkArgs a;
  gdr_status st = check_chunk(q, k, v, in_dtype, g, gate, beta, S0, o, S_T, 1, total_T, H, dk,
                              dv, C, &a);
  if (st != GDR_OK) return st;
  if ((size_t)N * H == 0) return ok();
  if (!cu_seqlens) return fail(GDR_ERR_INVALID_ARG, "null cu_seqlens");
  if ((size_t)N * H > 0x7fffffffu) return fail(GDR_ERR_INVALID_ARG, "N*H too large");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return from_cuda(e, "gdr_chunk_fwd_varlen status word");
  if (total_T == 0) {  // every sequence is empty: S_T = S0 (or 0)
    const size_t bytes = (size_t)N * H * dv * dk * sizeof(float);
    if (S_T && S0 && S_T != S0)
      e = cudaMemcpyAsync(S_T, S0, bytes, cudaMemcpyDeviceToDevice, s);
    else if (S_T && !S0)
      e = cudaMemsetAsync(S_T, 0, bytes, s);
    return from_cuda(e, "gdr_chunk_fwd_varlen copy");
  }
  a.B = N;
  a.cu_seqlens = cu_seqlens;
  return from_cuda(gdr::chunk_tc_supports(a) ? gdr::launch_chunk_tc(a, s)
                                             : gdr::launch_chunk_split(a, s),
                   "gdr_chunk_fwd_varlen launch");
}

gdr_status gdr_chunk_fwd_gla(const void *q, const void *k, const void *v, gdr_dtype in_dtype,
                             const float *g, gdr_gate_kind gate, const float *S0, void *o,
                             float *S_T, int B, int T, int H, int dk, int dv, int C,
                             gdr_stream_t stream) {
  gdr::ChunkArgs a;
  gdr_status st = check_chunk(q, k, v, in_dtype, g, gate, nullptr, S0, o, S_T, B, T, H, dk, dv,
                              C, &a, false);
  if (st != GDR_OK) return st;
  if ((size_t)B * H == 0) return ok();
  if ((size_t)B * H > 0x7fffffffu) return fail(GDR_ERR_INVALID_ARG, "B*H too large");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return from_cuda(e, "gdr_chunk_fwd_gla status word");
  if (T == 0) {  // no tokens: S_T = S0 (or 0)
    const size_t bytes = (size_t)B * H * dv * dk * sizeof(float);
    if (S_T && S0 && S_T != S0)
      e = cudaMemcpyAsync(S_T, S0, bytes, cudaMemcpyDeviceToDevice, s);
    else if (S_T && !S0)
      e = cudaMemsetAsync(S_T, 0, bytes, s);
    return from_cuda(e, "gdr_chunk_fwd_gla copy");
  }
  a.beta = nullptr;
  a.additive = 1;
  return from_cuda(gdr::chunk_tc_supports(a) ? gdr::launch_chunk_tc(a, s)
                                             : gdr::launch_chunk_split(a, s),
                   "gdr_chunk_fwd_gla launch");
}

gdr_status gdr_chunk_fwd_prologue(const void *q, const void *k, const void *v,
                                  gdr_dtype in_dtype, const float *a, gdr_gate_kind gate,
                                  const float *gate_scale, const float *b, const float *S0,
                                  void *o, float *S_T, int B, int T, int H, int dk, int dv, int C,
                                  int norm_qk, gdr_stream_t stream) {
  gdr::ChunkArgs ca;
  gdr_status st = check_chunk(q, k, v, in_dtype, a, gate, b, S0, o, S_T, B, T, H, dk, dv, C,
                              &ca);
  if (st != GDR_OK) return st;
  if (norm_qk < 0 || norm_qk > 3) return fail(GDR_ERR_INVALID_ARG, "norm_qk must be 0..3");
  if ((size_t)B * H == 0) return ok();
  if (!gate_scale) return fail(GDR_ERR_INVALID_ARG, "null gate_scale");
  if ((size_t)B * H > 0x7fffffffu) return fail(GDR_ERR_INVALID_ARG, "B*H too large");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = status_word(&ca.status);
  if (e != cudaSuccess) return from_cuda(e, "gdr_chunk_fwd_prologue status word");
  if (T == 0) {  // no tokens: S_T = S0 (or 0)
    const size_t bytes = (size_t)B * H * dv * dk * sizeof(float);
    if (S_T && S0 && S_T != S0)
      e = cudaMemcpyAsync(S_T, S0, bytes, cudaMemcpyDeviceToDevice, s);
    else if (S_T && !S0)
      e = cudaMemsetAsync(S_T, 0, bytes, s);
    return from_cuda(e, "gdr_chunk_fwd_prologue copy");
  }
  ca.prologue = 1;
  ca.norm_qk = norm_qk;
  ca.gate_scale = gate_scale;
  // the warp-specialised kernel takes bf16, d = 128 with a scalar gate; every
  // other shape and per-channel gates run the split-operand kernel
  const bool tc = gdr::chunk_tc_supports(ca) && gate == GDR_GATE_SCALAR;
  ca.skip_stage_chunk = tc ? t_skip_stage_chunk : -1;
  t_skip_stage_chunk = -1;
  return from_cuda(tc ? gdr::launch_chunk_tc(ca, s) : gdr::launch_chunk_split(ca, s),
                   "gdr_chunk_fwd_prologue launch");
}

gdr_status gdr_dplr_fwd(const void *q, const void *k, const void *v, const void *a,
                        const void *b, gdr_dtype in_dtype, const float *g, gdr_gate_kind gate,
                        const float *S0, void *o, float *S_T, int B, int T, int H, int dk,
                        int dv, gdr_stream_t stream) {
  if (B < 0 || T < 0 || H < 0) return fail(GDR_ERR_INVALID_ARG, "negative B/T/H");
  if (in_dtype != GDR_F32 && in_dtype != GDR_BF16)
    return fail(GDR_ERR_INVALID_ARG, "in_dtype must be GDR_F32 or GDR_BF16");
  if (gate != GDR_GATE_SCALAR && gate != GDR_GATE_PER_CHANNEL)
    return fail(GDR_ERR_INVALID_ARG, "unknown gate kind");
  if (!head_dim_ok(dk) || !head_dim_ok(dv))
    return fail(GDR_ERR_UNSUPPORTED, "DPLR head dims dk=%d dv=%d (need 32, 64 or 128)", dk, dv);
  if ((size_t)B * (size_t)H * (size_t)T > (size_t)1 << 40)
    return fail(GDR_ERR_INVALID_ARG, "problem too large");
  if ((size_t)B * H > 0x7fffffffu) return fail(GDR_ERR_INVALID_ARG, "B*H too large");
  if ((size_t)B * H * T != 0) {
    if (!q || !k || !v || !a || !b || !g || !o)
      return fail(GDR_ERR_INVALID_ARG, "null q/k/v/a/b/g/o");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(a) || !aligned16(b) ||
        !aligned16(g) || !aligned16(o))
      return fail(GDR_ERR_INVALID_ARG, "q/k/v/a/b/g/o must be 16-byte aligned");
  }
  if ((S0 && !aligned16(S0)) || (S_T && !aligned16(S_T)))
    return fail(GDR_ERR_INVALID_ARG, "S0/S_T must be 16-byte aligned");
  if ((size_t)B * H == 0) return ok();
  gdr::DplrChunkArgs p;
  p.q = q; p.k = k; p.v = v; p.a = a; p.b = b; p.g = g; p.S0 = S0; p.o = o; p.S_T = S_T;
  p.B = B; p.T = T; p.H = H; p.dk = dk; p.dv = dv;
  p.bf16 = in_dtype == GDR_BF16;
  p.per_channel = gate == GDR_GATE_PER_CHANNEL;
  cudaError_t e = status_word(&p.status);
  if (e != cudaSuccess) return from_cuda(e, "gdr_dplr_fwd status word");
  return from_cuda(gdr::launch_dplr_chunk(p, reinterpret_cast<cudaStream_t>(stream)),
                   "gdr_dplr_fwd launch");
}

namespace {
// The backward's path for a shape: the tensor-core chunked backward, or the
// per-step recurrence on CUDA cores.
bool bwd_on_tensor_cores(int T, int d, gdr_dtype in_dtype, gdr_gate_kind gate) {
  return T > 0 && gdr::bwd_tc_supports(in_dtype == GDR_BF16, gate == GDR_GATE_PER_CHANNEL, d);
}
}  // namespace

size_t gdr_chunk_bwd_workspace_bytes(int B, int T, int H, int dk, int dv, gdr_dtype in_dtype,
                                     gdr_gate_kind gate) {
  if (dk != dv || (dk != 32 && dk != 64 && dk != 128)) return 0;
  if (bwd_on_tensor_cores(T, dk, in_dtype, gate)) return gdr::bwd_tc_ws_bytes(B, T, H);
  return gdr::bwd_ws_bytes(B, T, H, dk);
}

gdr_status gdr_chunk_bwd(const void *q, const void *k, const void *v, gdr_dtype in_dtype,
                         const float *g, gdr_gate_kind gate, const float *beta, const float *S0,
                         const float *dout, const float *dS_T, float *dq, float *dk, float *dv,
                         float *dg, float *dbeta, float *dS0, int B, int T, int H, int dk_,
                         int dv_, void *workspace, size_t ws_bytes, gdr_stream_t stream) {
  if (B < 0 || T < 0 || H < 0) return fail(GDR_ERR_INVALID_ARG, "negative B/T/H");
  if (in_dtype != GDR_F32 && in_dtype != GDR_BF16)
    return fail(GDR_ERR_INVALID_ARG, "in_dtype must be GDR_F32 or GDR_BF16");
  if (gate != GDR_GATE_SCALAR && gate != GDR_GATE_PER_CHANNEL)
    return fail(GDR_ERR_INVALID_ARG, "unknown gate kind");
  if (dk_ != dv_ || (dk_ != 32 && dk_ != 64 && dk_ != 128))
    return fail(GDR_ERR_UNSUPPORTED, "backward needs dk = dv in {32, 64, 128} (got %d, %d)", dk_,
                dv_);
  if ((size_t)B * (size_t)H * (size_t)T > (size_t)1 << 40)
    return fail(GDR_ERR_INVALID_ARG, "problem too large");
  if ((size_t)B * H > 0x7fffffffu) return fail(GDR_ERR_INVALID_ARG, "B*H too large");
  if ((size_t)B * H * T != 0) {
    if (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta)
      return fail(GDR_ERR_INVALID_ARG, "null input or gradient pointer");
  }
  const size_t need = gdr_chunk_bwd_workspace_bytes(B, T, H, dk_, dv_, in_dtype, gate);
  if ((size_t)B * H != 0 && (ws_bytes < need || !workspace))
    return fail(GDR_ERR_WORKSPACE, "workspace %zu B < required %zu B", ws_bytes, need);
  if (workspace && !aligned16(workspace))
    return fail(GDR_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  if ((size_t)B * H == 0) return ok();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (bwd_on_tensor_cores(T, dk_, in_dtype, gate)) {
    if ((size_t)B * H * ((T + 63) / 64) > 0x7fffffffu)
      return fail(GDR_ERR_INVALID_ARG, "B*H*chunks too large");
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dout))
      return fail(GDR_ERR_INVALID_ARG, "q/k/v/dout must be 16-byte aligned");
    unsigned int *status = nullptr;
    cudaError_t e = status_word(&status);
    if (e != cudaSuccess) return from_cuda(e, "gdr_chunk_bwd status word");
    return from_cuda(gdr::launch_bwd_tc(q, k, v, g, beta, S0, dout, dS_T, dq, dk, dv, dg, dbeta,
                                        dS0, B, T, H, workspace, status, s),
                     "gdr_chunk_bwd launch (tensor cores)");
  }
  return from_cuda(gdr::launch_bwd(q, k, v, in_dtype == GDR_BF16, g, gate == GDR_GATE_PER_CHANNEL,
                                   beta, S0, dout, dS_T, dq, dk, dv, dg, dbeta, dS0, B, T, H,
                                   dk_, workspace, s),
                   "gdr_chunk_bwd launch");
}

gdr_status gdr_step(const void *q, const void *k, const void *v, gdr_dtype in_dtype,
                    const float *g, gdr_gate_kind gate, const float *beta, float *S, void *o,
                    int N, int H, int dk, int dv, gdr_stream_t stream) {
  if (N < 0 || H < 0) return fail(GDR_ERR_INVALID_ARG, "negative N/H");
  if (in_dtype != GDR_F32 && in_dtype != GDR_BF16)
    return fail(GDR_ERR_INVALID_ARG, "in_dtype must be GDR_F32 or GDR_BF16");
  if (gate != GDR_GATE_SCALAR && gate != GDR_GATE_PER_CHANNEL)
    return fail(GDR_ERR_INVALID_ARG, "unknown gate kind");
  if (!head_dim_ok(dk) || !head_dim_ok(dv))
    return fail(GDR_ERR_UNSUPPORTED, "head dims dk=%d dv=%d (need 32, 64 or 128)", dk, dv);
  if ((size_t)N * H == 0) return ok();
  if (!q || !k || !v || !g || !beta || !S || !o)
    return fail(GDR_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
      !aligned16(S) || !aligned16(o))
    return fail(GDR_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  if ((size_t)N * H > (size_t)1 << 31) return fail(GDR_ERR_INVALID_ARG, "N*H too large");
  gdr::StepArgs a;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.S = S; a.o = o;
  a.N = N; a.H = H; a.dk = dk; a.dv = dv;
  a.bf16 = in_dtype == GDR_BF16;
  a.per_channel = gate == GDR_GATE_PER_CHANNEL;
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return from_cuda(e, "gdr_step status word");
  return from_cuda(gdr::launch_step(a, reinterpret_cast<cudaStream_t>(stream)),
                   "gdr_step launch");
}

gdr_status gdr_step_slots(const void *q, const void *k, const void *v, gdr_dtype in_dtype,
                          long long q_stride, long long k_stride, long long v_stride,
                          const float *g, gdr_gate_kind gate, const float *beta,
                          const float *gate_scale, int norm_qk, float *pool, int slots,
                          long long slot_stride, const int *src, const int *dst,
                          const int *cu_seqlens, void *o, int R, int total, int Hk, int H,
                          int dk, int dv, gdr_stream_t stream) {
  if (R < 0 || total < 0 || Hk < 0 || H < 0 || slots < 0)
    return fail(GDR_ERR_INVALID_ARG, "negative R/total/Hk/H/slots");
  gdr_status st = check_kinds(in_dtype, gate, norm_qk);
  if (st != GDR_OK) return st;
  if (!head_dim_ok(dk) || !head_dim_ok(dv))
    return fail(GDR_ERR_UNSUPPORTED, "head dims dk=%d dv=%d (need 32, 64 or 128)", dk, dv);
  if ((size_t)R * H == 0 || total == 0) return ok();
  if (Hk == 0 || H % Hk != 0)
    return fail(GDR_ERR_INVALID_ARG, "H=%d is not a multiple of Hk=%d", H, Hk);
  if (!cu_seqlens && total != R)
    return fail(GDR_ERR_INVALID_ARG, "without cu_seqlens total=%d must be R=%d", total, R);
  if (!q || !k || !v || !g || !beta || !src || !o || (slots && !pool))
    return fail(GDR_ERR_INVALID_ARG, "null q/k/v/g/beta/pool/src/o");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) ||
      !aligned16(gate_scale) || !aligned16(pool) || !aligned16(o))
    return fail(GDR_ERR_INVALID_ARG, "q/k/v/g/beta/gate_scale/pool/o must be 16-byte aligned");
  if (!aligned4(src) || !aligned4(dst) || !aligned4(cu_seqlens))
    return fail(GDR_ERR_INVALID_ARG, "src/dst/cu_seqlens must be 4-byte aligned");
  st = check_stride("q", q_stride, (long long)Hk * dk, total, in_dtype);
  if (st == GDR_OK) st = check_stride("k", k_stride, (long long)Hk * dk, total, in_dtype);
  if (st == GDR_OK) st = check_stride("v", v_stride, (long long)H * dv, total, in_dtype);
  if (st == GDR_OK) st = check_stride("pool", slot_stride, (long long)H * dv * dk, slots, GDR_F32);
  if (st != GDR_OK) return st;
  if ((size_t)R * H > (size_t)1 << 28) return fail(GDR_ERR_INVALID_ARG, "R*H too large");
  gdr::StepSlotsArgs a{};
  a.q = q; a.k = k; a.v = v;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.g = g; a.beta = beta; a.gate_scale = gate_scale; a.norm_qk = norm_qk;
  a.pool = pool; a.slots = slots; a.slot_stride = slot_stride;
  a.src = src; a.dst = dst; a.cu = cu_seqlens; a.o = o;
  a.R = R; a.total = total; a.Hk = Hk; a.H = H; a.dk = dk; a.dv = dv;
  a.bf16 = in_dtype == GDR_BF16;
  a.per_channel = gate == GDR_GATE_PER_CHANNEL;
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return from_cuda(e, "gdr_step_slots status word");
  return from_cuda(gdr::launch_step_slots(a, reinterpret_cast<cudaStream_t>(stream)),
                   "gdr_step_slots launch");
}

gdr_status gdr_slot_map(const int *lens, const int *kept, const int *table,
                        long long table_stride, int R, int W, int slots, int max_tokens,
                        int keep_all, int *cu_seqlens, int *request, int *src, int *dst,
                        gdr_stream_t stream) {
  if (R < 0 || slots < 0 || max_tokens < 0)
    return fail(GDR_ERR_INVALID_ARG, "negative R/slots/max_tokens");
  if (R > 65536) return fail(GDR_ERR_UNSUPPORTED, "R=%d requests (at most 65536)", R);
  if (W < 1) return fail(GDR_ERR_INVALID_ARG, "W=%d slots a request (need at least 1)", W);
  if (keep_all != 0 && keep_all != 1) return fail(GDR_ERR_INVALID_ARG, "keep_all must be 0 or 1");
  if (R > 1 && table_stride < W)
    return fail(GDR_ERR_INVALID_ARG, "table_stride=%lld is less than W=%d", table_stride, W);
  if (!cu_seqlens || (R && (!lens || !kept || !table || !src)) ||
      (max_tokens && (!request || !dst)))
    return fail(GDR_ERR_INVALID_ARG, "null pointer argument");
  if (!aligned4(lens) || !aligned4(kept) || !aligned4(table) || !aligned4(cu_seqlens) ||
      !aligned4(request) || !aligned4(src) || !aligned4(dst))
    return fail(GDR_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  gdr::SlotMapArgs a{};
  a.lens = lens; a.kept = kept; a.table = table; a.table_stride = table_stride;
  a.R = R; a.W = W; a.slots = slots; a.max_tokens = max_tokens; a.keep_all = keep_all;
  a.cu = cu_seqlens; a.request = request; a.src = src; a.dst = dst;
  cudaError_t e = status_word(&a.status);
  if (e != cudaSuccess) return from_cuda(e, "gdr_slot_map status word");
  return from_cuda(gdr::launch_slot_map(a, reinterpret_cast<cudaStream_t>(stream)),
                   "gdr_slot_map launch");
}

}  // extern "C"

namespace {

// Checks shared by both directions of the output norm; fills the arguments.
gdr_status check_group_norm(const void *x, const void *z, gdr_dtype dtype, long long x_stride,
                            long long z_stride, const float *weight, const float *bias,
                            int per_channel, gdr_act act, int center, float eps, long long rows,
                            int G, int D, gdr::GroupNormArgs *out) {
  if (rows < 0 || G < 1 || D < 1) return fail(GDR_ERR_INVALID_ARG, "rows < 0, G < 1 or D < 1");
  if (dtype != GDR_F32 && dtype != GDR_BF16)
    return fail(GDR_ERR_INVALID_ARG, "dtype must be GDR_F32 or GDR_BF16");
  if (act != GDR_ACT_NONE && act != GDR_ACT_SILU && act != GDR_ACT_SIGMOID)
    return fail(GDR_ERR_INVALID_ARG, "unknown activation");
  if (per_channel != 0 && per_channel != 1)
    return fail(GDR_ERR_INVALID_ARG, "per_channel must be 0 or 1");
  if (!(eps > 0.f) || eps > 1e30f) return fail(GDR_ERR_INVALID_ARG, "eps must be positive");
  if (D > 1024 || (long long)G * D > 65536)
    return fail(GDR_ERR_UNSUPPORTED, "G=%d groups of D=%d (D <= 1024, G*D <= 65536)", G, D);
  if (rows > (1ll << 40)) return fail(GDR_ERR_INVALID_ARG, "problem too large");
  const size_t size = dtype == GDR_BF16 ? 2 : 4;
  if (rows && !x) return fail(GDR_ERR_INVALID_ARG, "null x");
  if (!aligned_to(x, size) || !aligned_to(z, size) || !aligned4(weight) || !aligned4(bias))
    return fail(GDR_ERR_INVALID_ARG, "x/z/weight/bias must be aligned to their elements");
  if (rows > 1 && (x_stride < (long long)G * D || (z && z_stride < (long long)G * D)))
    return fail(GDR_ERR_INVALID_ARG, "x_stride/z_stride less than G*D=%lld", (long long)G * D);
  gdr::GroupNormArgs a{};
  a.x = x; a.z = z; a.x_stride = x_stride; a.z_stride = z_stride;
  a.weight = weight; a.bias = bias; a.per_channel = per_channel; a.act = act;
  a.center = center != 0; a.eps = eps; a.rows = rows; a.G = G; a.D = D;
  a.bf16 = dtype == GDR_BF16;
  *out = a;
  return ok();
}

// Checks shared by both directions of the prologue; fills the arguments.
gdr_status check_prologue(const void *q, const void *k, gdr_dtype in_dtype, long long q_stride,
                          long long k_stride, const float *a, gdr_gate_kind gate, const float *b,
                          const float *gate_scale, int norm_qk, long long tokens, int Hk, int H,
                          int dk, gdr::PrologueArgs *out) {
  if (tokens < 0 || Hk < 1 || H < 1) return fail(GDR_ERR_INVALID_ARG, "tokens < 0, Hk < 1 or H < 1");
  gdr_status st = check_kinds(in_dtype, gate, norm_qk);
  if (st != GDR_OK) return st;
  if (!head_dim_ok(dk)) return fail(GDR_ERR_UNSUPPORTED, "head dim dk=%d (need 32, 64 or 128)", dk);
  if (H % Hk != 0) return fail(GDR_ERR_INVALID_ARG, "H=%d is not a multiple of Hk=%d", H, Hk);
  if (H > 65536) return fail(GDR_ERR_UNSUPPORTED, "H=%d heads (at most 65536)", H);
  if (tokens > (1ll << 40) / H) return fail(GDR_ERR_INVALID_ARG, "problem too large");
  if (tokens && (!q || !k || !a || !b || !gate_scale))
    return fail(GDR_ERR_INVALID_ARG, "null q/k/a/b/gate_scale");
  if (!aligned16(q) || !aligned16(k) || !aligned16(a) || !aligned16(b) || !aligned16(gate_scale))
    return fail(GDR_ERR_INVALID_ARG, "q/k/a/b/gate_scale must be 16-byte aligned");
  st = check_stride("q", q_stride, (long long)Hk * dk, tokens, in_dtype);
  if (st == GDR_OK) st = check_stride("k", k_stride, (long long)Hk * dk, tokens, in_dtype);
  if (st != GDR_OK) return st;
  gdr::PrologueArgs p{};
  p.q = q; p.k = k; p.q_stride = q_stride; p.k_stride = k_stride;
  p.a = a; p.b = b; p.gate_scale = gate_scale; p.norm_qk = norm_qk;
  p.tokens = tokens; p.Hk = Hk; p.H = H; p.d = dk;
  p.bf16 = in_dtype == GDR_BF16;
  p.per_channel = gate == GDR_GATE_PER_CHANNEL;
  *out = p;
  return ok();
}

}  // namespace

extern "C" {

gdr_status gdr_group_norm_fwd(const void *x, const void *z, gdr_dtype dtype, long long x_stride,
                              long long z_stride, const float *weight, const float *bias,
                              int per_channel, gdr_act act, int center, float eps, void *y,
                              long long rows, int G, int D, gdr_stream_t stream) {
  gdr::GroupNormArgs a;
  gdr_status st = check_group_norm(x, z, dtype, x_stride, z_stride, weight, bias, per_channel, act,
                                   center, eps, rows, G, D, &a);
  if (st != GDR_OK) return st;
  if (rows == 0) return ok();
  if (!y) return fail(GDR_ERR_INVALID_ARG, "null y");
  if (!aligned_to(y, a.bf16 ? 2 : 4))
    return fail(GDR_ERR_INVALID_ARG, "y must be aligned to its elements");
  a.y = y;
  return from_cuda(gdr::launch_group_norm_fwd(a, reinterpret_cast<cudaStream_t>(stream)),
                   "gdr_group_norm_fwd launch");
}

size_t gdr_group_norm_bwd_workspace_bytes(long long rows, int G, int D, gdr_dtype dtype,
                                          int per_channel) {
  if (rows < 0 || G < 1 || D < 1 || D > 1024 || (long long)G * D > 65536 || rows > (1ll << 40))
    return 0;
  return gdr::group_norm_bwd_ws_bytes(rows, G, D, dtype == GDR_BF16, per_channel);
}

gdr_status gdr_group_norm_bwd(const void *dy, const void *x, const void *z, gdr_dtype dtype,
                              long long x_stride, long long z_stride, const float *weight,
                              const float *bias, int per_channel, gdr_act act, int center,
                              float eps, float *dx, void *dz, float *dweight, float *dbias,
                              long long rows, int G, int D, void *workspace, size_t ws_bytes,
                              gdr_stream_t stream) {
  gdr::GroupNormArgs a;
  gdr_status st = check_group_norm(x, z, dtype, x_stride, z_stride, weight, bias, per_channel, act,
                                   center, eps, rows, G, D, &a);
  if (st != GDR_OK) return st;
  if (dz && !z) return fail(GDR_ERR_INVALID_ARG, "dz without z");
  if (rows && (!dy || !dx)) return fail(GDR_ERR_INVALID_ARG, "null dy/dx");
  const size_t size = a.bf16 ? 2 : 4;
  if (!aligned_to(dy, size) || !aligned_to(dz, size) || !aligned4(dx) || !aligned4(dweight) ||
      !aligned4(dbias))
    return fail(GDR_ERR_INVALID_ARG, "dy/dx/dz/dweight/dbias must be aligned to their elements");
  if (dweight || dbias) {
    const size_t need = gdr_group_norm_bwd_workspace_bytes(rows, G, D, dtype, per_channel);
    if (ws_bytes < need || !workspace)
      return fail(GDR_ERR_WORKSPACE, "workspace %zu B < required %zu B", ws_bytes, need);
    if (!aligned16(workspace))
      return fail(GDR_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  } else if (rows == 0) {
    return ok();
  }
  a.dy = dy; a.dx = dx; a.dz = dz; a.dweight = dweight; a.dbias = dbias;
  a.ws = static_cast<float *>(workspace);
  return from_cuda(gdr::launch_group_norm_bwd(a, reinterpret_cast<cudaStream_t>(stream)),
                   "gdr_group_norm_bwd launch");
}

gdr_status gdr_prologue_fwd(const void *q, const void *k, gdr_dtype in_dtype, long long q_stride,
                            long long k_stride, const float *a, gdr_gate_kind gate,
                            const float *b, const float *gate_scale, int norm_qk, void *qn,
                            void *kn, float *g, float *beta, long long tokens, int Hk, int H,
                            int dk, gdr_stream_t stream) {
  gdr::PrologueArgs p;
  gdr_status st = check_prologue(q, k, in_dtype, q_stride, k_stride, a, gate, b, gate_scale,
                                 norm_qk, tokens, Hk, H, dk, &p);
  if (st != GDR_OK) return st;
  if (tokens == 0) return ok();
  if (!qn || !kn || !g || !beta) return fail(GDR_ERR_INVALID_ARG, "null qn/kn/g/beta");
  if (!aligned16(qn) || !aligned16(kn) || !aligned16(g) || !aligned16(beta))
    return fail(GDR_ERR_INVALID_ARG, "qn/kn/g/beta must be 16-byte aligned");
  p.qn = qn; p.kn = kn; p.g = g; p.beta = beta;
  return from_cuda(gdr::launch_prologue_fwd(p, reinterpret_cast<cudaStream_t>(stream)),
                   "gdr_prologue_fwd launch");
}

size_t gdr_prologue_bwd_workspace_bytes(long long tokens, int H, int dk, gdr_gate_kind gate) {
  if (tokens < 0 || H < 1 || H > 65536 || !head_dim_ok(dk) || tokens > (1ll << 40) / H) return 0;
  return gdr::prologue_bwd_ws_bytes(tokens, H, dk, gate == GDR_GATE_PER_CHANNEL);
}

gdr_status gdr_prologue_bwd(const void *q, const void *k, gdr_dtype in_dtype, long long q_stride,
                            long long k_stride, const float *a, gdr_gate_kind gate,
                            const float *b, const float *gate_scale, int norm_qk,
                            const float *dqn, const float *dkn, const float *dg,
                            const float *dbeta, void *dq, void *dk_, float *da, float *db,
                            float *dgate_scale, long long tokens, int Hk, int H, int dk,
                            void *workspace, size_t ws_bytes, gdr_stream_t stream) {
  gdr::PrologueArgs p;
  gdr_status st = check_prologue(q, k, in_dtype, q_stride, k_stride, a, gate, b, gate_scale,
                                 norm_qk, tokens, Hk, H, dk, &p);
  if (st != GDR_OK) return st;
  if (!dgate_scale || (tokens && (!dqn || !dkn || !dg || !dbeta || !dq || !dk_ || !da || !db)))
    return fail(GDR_ERR_INVALID_ARG, "null gradient pointer");
  if (!aligned16(dqn) || !aligned16(dkn) || !aligned16(dg) || !aligned16(dbeta) ||
      !aligned16(dq) || !aligned16(dk_) || !aligned16(da) || !aligned16(db) ||
      !aligned16(dgate_scale))
    return fail(GDR_ERR_INVALID_ARG, "gradients must be 16-byte aligned");
  const size_t need = gdr_prologue_bwd_workspace_bytes(tokens, H, dk, gate);
  if (ws_bytes < need || !workspace)
    return fail(GDR_ERR_WORKSPACE, "workspace %zu B < required %zu B", ws_bytes, need);
  if (!aligned16(workspace)) return fail(GDR_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (tokens == 0)  // no tokens: the sum over them is zero
    return from_cuda(cudaMemsetAsync(dgate_scale, 0, (size_t)H * sizeof(float), s),
                     "gdr_prologue_bwd clear");
  p.dqn = dqn; p.dkn = dkn; p.dg = dg; p.dbeta = dbeta;
  p.dq = dq; p.dk = dk_; p.da = da; p.db = db; p.dgate_scale = dgate_scale;
  p.ws = static_cast<float *>(workspace);
  return from_cuda(gdr::launch_prologue_bwd(p, s), "gdr_prologue_bwd launch");
}

gdr_status gdr_testing_skip_stage_load(int chunk) {
  if (chunk < 0) return fail(GDR_ERR_INVALID_ARG, "chunk must be >= 0");
  t_skip_stage_chunk = chunk;
  return ok();
}

gdr_status gdr_get_device_status(gdr_stream_t stream) {
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  unsigned int word = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&word, gdr::g_device_status, sizeof word, 0,
                                            cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(gdr::g_device_status, &zero, sizeof zero, 0,
                                cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return from_cuda(e, "gdr_get_device_status");
  if (word & gdr::kStatusTimeout)
    return fail(GDR_ERR_TIMEOUT, "a kernel gave up a bounded wait (status word 0x%x)", word);
  if (word & gdr::kStatusRange)
    return fail(GDR_ERR_RANGE,
                "a per-channel gate decayed beyond the tensor-core path's range (more than "
                "about 83 in log decay over half a chunk); those results are not valid "
                "(status word 0x%x)",
                word);
  if (word & gdr::kStatusSlot)
    return fail(GDR_ERR_SLOT,
                "a request named a state slot, a length or a kept count that does not exist; it "
                "was skipped (status word 0x%x)",
                word);
  return ok();
}

}  // extern "C"
