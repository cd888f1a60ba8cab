// The mixer's output norm: group norm, channels last, with an activation.
// What its two directions share.
//
// A group (one head of one token) is a few hundred bytes, so L lanes of a
// warp hold it in registers: every input is read once, every sum over the
// group is a few shuffles, every output is written once.  Both directions are
// bound by HBM as long as enough bytes are in flight: a lane's next two or three
// rows are on their way to shared memory while it works on one.
//
// A lane keeps the same group index for all its rows (the number of groups
// in flight is a multiple of G), so its weights are loaded once and addresses
// advance by a constant.  A block takes few rows a lane (8, or 16): with
// a grid that fills the SMs once and runs to the end, the slowest SM sets the
// time (forward of 32768 x 16 x 128 bf16: 74.7 us, with 8 rows 62.4 us, with 1 row,
// where blocks spend their time on starting, 121 us).
//
// Arithmetic is in pairs of fp32 and on the fast exponential and reciprocal: a
// gated SiLU takes 23 instructions an element forward and 34 backward (counted), just
// what HBM leaves time for (the forward issues on 78 % of the cycles).
//
// 32768 x 16 x 128 bf16, SiLU gate: forward 62.4 us (6447 GB/s; a copy runs at 6456),
// gradient 130.9 us (6151 GB/s, its second launch included).  Groups that do not start
// on 16 bytes: 32768 x 16 x 100 bf16 (8-byte accesses) forward 62.4 us (5044 GB/s), 31 x 33
// (2-byte accesses, bound by instructions) 66.4 us (3030 GB/s), gradient 169 us.
#pragma once

#include "gdr_rows.cuh"

namespace gdr {

inline bool multiple_of(const void *p, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

// Elements per access: 16 bytes where every row and group starts on 16, for
// bf16 also 8 bytes; else single elements.
inline int norm_vector(const GroupNormArgs &a) {
  const int size = a.bf16 ? 2 : 4;
  for (int vec : {16 / size, 4}) {
    const size_t bytes = (size_t)vec * size;
    if (a.D % vec == 0 && a.x_stride % vec == 0 && (!a.z || a.z_stride % vec == 0) &&
        multiple_of(a.x, bytes) && multiple_of(a.z, bytes) && multiple_of(a.dy, bytes) &&
        multiple_of(a.y, bytes) && multiple_of(a.dz, bytes) && multiple_of(a.dx, 16) &&
        multiple_of(a.weight, 16) && multiple_of(a.bias, 16))
      return vec;
  }
  return 1;
}

// A lane's weights or biases from p + at on (`none` where there are none).
template <int VEC, int L, int NV>
__device__ __forceinline__ void load_affine(const float *p, int at, const bool (&in)[NV], float none,
                                            float2 (&x)[VEC * NV / 2]) {
  float v[VEC * NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float *w = v + i * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] = none;
    if (!p || !in[i]) continue;
    const float *from = p + at + i * L * VEC;
    if constexpr (VEC >= 4) {
#pragma unroll
      for (int e = 0; e < VEC; e += 4) {
        const float4 t = *reinterpret_cast<const float4 *>(from + e);
        w[e] = t.x; w[e + 1] = t.y; w[e + 2] = t.z; w[e + 3] = t.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = from[e];
    }
  }
#pragma unroll
  for (int e = 0; e < VEC * NV / 2; ++e) x[e] = make_float2(v[2 * e], v[2 * e + 1]);
}

// Subtracts the group's mean from x (with center; what lies outside the group
// stays 0) and returns 1 / sqrt(mean square + eps).
template <int VEC, int L, int NV>
__device__ __forceinline__ float normalise(float2 (&x)[VEC * NV / 2], const bool (&in)[NV],
                                           int center, float inv_d, float eps) {
  constexpr int N = VEC * NV / 2;
  if (center) {
    float2 sum = both(0.f);
#pragma unroll
    for (int e = 0; e < N; ++e) sum = add2(sum, x[e]);
    const float m = lanes_sum<L>(sum.x + sum.y) * inv_d;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      x[e].x = in[2 * e / VEC] ? x[e].x - m : 0.f;
      x[e].y = in[(2 * e + 1) / VEC] ? x[e].y - m : 0.f;
    }
  }
  float2 ss = both(0.f);
#pragma unroll
  for (int e = 0; e < N; ++e) ss = fma2(x[e], x[e], ss);
  return rsqrtf(lanes_sum<L>(ss.x + ss.y) * inv_d + eps);
}

// Whether a layout's rows wait in shared memory.
template <typename T, int VEC, int NV>
constexpr bool norm_queue = sizeof(Raw<T, VEC>) >= 8 && NV <= 2;

// Calls f.template operator()<T, VEC, L, NV>() for the layout of these
// arguments: L lanes a group, NV accesses of VEC elements a lane.  16-byte
// accesses: one a lane where they fit, so that most rows are in flight.  Narrower
// ones are bound by instructions, most of them the same for every group of a
// warp: several accesses a lane and fewer lanes a group (33 channels of bf16, 1 M
// groups: 32 lanes of 2 elements 194 us, 8 lanes of 6 elements 66 us).
template <typename T, int VEC, typename F>
cudaError_t norm_layout_vec(int D, F f) {
  const int n = (D + VEC - 1) / VEC;  // accesses of a group
  if constexpr (sizeof(T) * VEC == 16) {
    if (n <= 4) return f.template operator()<T, VEC, 4, 1>();
    if (n <= 8) return f.template operator()<T, VEC, 8, 1>();
    if (n <= 16) return f.template operator()<T, VEC, 16, 1>();
    if (n <= 32) return f.template operator()<T, VEC, 32, 1>();
    if (n <= 64) return f.template operator()<T, VEC, 32, 2>();
    if (n <= 128) return f.template operator()<T, VEC, 32, 4>();
    if constexpr (VEC == 4) {
      if (n <= 256) return f.template operator()<T, VEC, 32, 8>();
    }
  } else if constexpr (VEC == 4) {
    if (n <= 16) return f.template operator()<T, VEC, 8, 2>();
    if (n <= 32) return f.template operator()<T, VEC, 16, 2>();
    if (n <= 64) return f.template operator()<T, VEC, 32, 2>();
    if (n <= 128) return f.template operator()<T, VEC, 32, 4>();
    if (n <= 256) return f.template operator()<T, VEC, 32, 8>();
  } else {
    // (6 or 8 accesses a lane: the fewer, the less of a short group's lanes are idle)
    if (n <= 24) return f.template operator()<T, VEC, 4, 6>();
    if (n <= 32) return f.template operator()<T, VEC, 4, 8>();
    if (n <= 48) return f.template operator()<T, VEC, 8, 6>();
    if (n <= 64) return f.template operator()<T, VEC, 8, 8>();
    if (n <= 96) return f.template operator()<T, VEC, 16, 6>();
    if (n <= 128) return f.template operator()<T, VEC, 16, 8>();
    if (n <= 192) return f.template operator()<T, VEC, 32, 6>();
    if (n <= 256) return f.template operator()<T, VEC, 32, 8>();
    if (n <= 512) return f.template operator()<T, VEC, 32, 16>();
    if (n <= 640) return f.template operator()<T, VEC, 32, 20>();
    if (n <= 1024) return f.template operator()<T, VEC, 32, 32>();
  }
  return cudaErrorInvalidValue;
}

template <typename F>
cudaError_t norm_layout(const GroupNormArgs &a, F f) {
  const int vec = norm_vector(a);
  if (!a.bf16)
    return vec == 4 ? norm_layout_vec<float, 4>(a.D, f) : norm_layout_vec<float, 1>(a.D, f);
  if (vec == 8) return norm_layout_vec<__nv_bfloat16, 8>(a.D, f);
  return vec == 4 ? norm_layout_vec<__nv_bfloat16, 4>(a.D, f)
                  : norm_layout_vec<__nv_bfloat16, 1>(a.D, f);
}

}  // namespace gdr
