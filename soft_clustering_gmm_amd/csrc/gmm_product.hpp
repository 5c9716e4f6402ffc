// Device code shared by the product kernels (the linear layer and the layer
// of experts): element types, matrix instructions, activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/gmm.h"

namespace gmm {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// One 16-byte fragment holds kPer elements. The 64 lanes of a wave hold 16
// rows x 4 groups of kPer consecutive k: lane l has row l % 16, group l / 16.
// mma() multiplies such a fragment of A with one of B over those 4 kPer
// values of k and adds to D: lane l has column l % 16 of B and rows
// 4 (l / 16) + i of A. The single-precision instruction takes one k per lane
// and group, so it runs once per element of the fragment; which k meet in
// which instruction does not matter, as both fragments agree on it.
template <typename T>
struct Frag;

// acc[i][j] += the product of fb[j] and fa[i], for all tiles.
template <typename T, int MI, int NI>
__device__ __forceinline__ void mma_each(const u32x4* fb, const u32x4* fa, f32x4 (*acc)[NI]) {
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = Frag<T>::mma(fb[j], fa[i], acc[i][j]);
}

template <>
struct Frag<float> {
  static constexpr int kPer = 4;
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
    return c;
  }
  // One element at a time over all tiles: the four products of a tile wait for
  // each other.
  template <int MI, int NI>
  static __device__ __forceinline__ void mma_tiles(const u32x4* fb, const u32x4* fa, f32x4 (*acc)[NI]) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(f32x4, fb[j])[q],
                                                           __builtin_bit_cast(f32x4, fa[i])[q], acc[i][j], 0, 0, 0);
  }
};

template <>
struct Frag<_Float16> {
  static constexpr int kPer = 8;
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
  }
  template <int MI, int NI>
  static __device__ __forceinline__ void mma_tiles(const u32x4* fb, const u32x4* fa, f32x4 (*acc)[NI]) {
    mma_each<_Float16, MI, NI>(fb, fa, acc);
  }
};

template <>
struct Frag<__bf16> {
  static constexpr int kPer = 8;
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  }
  template <int MI, int NI>
  static __device__ __forceinline__ void mma_tiles(const u32x4* fb, const u32x4* fa, f32x4 (*acc)[NI]) {
    mma_each<__bf16, MI, NI>(fb, fa, acc);
  }
};

// Activations in single precision. A NaN z stays NaN.
//
// gelu is z Phi(z). The tail of the normal distribution is taken from Abramowitz
// and Stegun, Handbook of Mathematical Functions, 7.1.26:
//   erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2),  t = 1 / (1 + p x),  x >= 0,
// within 1.5e-7, which is 0.75e-7 of Phi: below half a step of single precision
// next to 1. With x = |z| / sqrt 2 the exponential is also the density's, which
// the slope needs. It takes a third of erff's instructions.
struct Normal {
  float cdf, e;  // Phi(z), exp(-z^2 / 2)
};
__device__ __forceinline__ Normal normal_of(float z) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, x, 1.f));
  const float e = __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  const float tail = 0.5f * q * t * e;
  return {z < 0.f ? tail : 1.f - tail, e};
}

// 1 / (1 + exp(-z)): a far negative z gives 1 / inf = 0.
__device__ __forceinline__ float logistic(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * z));
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == GMM_ACT_RELU) return z < 0.f ? 0.f : z;
  if (ACT == GMM_ACT_GELU) return z * normal_of(z).cdf;
  if (ACT == GMM_ACT_SILU) return z * logistic(z);
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == GMM_ACT_RELU) return z > 0.f ? 1.f : z == z ? 0.f : z;
  if (ACT == GMM_ACT_GELU) {
    const Normal n = normal_of(z);
    return fmaf(0.39894228040143268f * z, n.e, n.cdf);
  }
  if (ACT == GMM_ACT_SILU) {
    const float q = logistic(z);
    return q * (1.f + z * (1.f - q));
  }
  return 1.f;
}

// Orders this wave's LDS accesses (all lanes) before its later ones.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 16 bytes from an address of any alignment (the hardware's unaligned loads).
__device__ __forceinline__ u32x4 load16(const void* p) {
  u32x4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// The kPer elements at p[0..], zero from n on (n <= 0: all zero, p not read).
template <typename T>
__device__ __forceinline__ u32x4 load_frag(const T* p, int n) {
  if (n >= Frag<T>::kPer) return load16(p);
  union {
    u32x4 v;
    T e[Frag<T>::kPer];
  } u;
#pragma unroll
  for (int i = 0; i < Frag<T>::kPer; ++i) u.e[i] = i < n ? p[i] : (T)0.f;
  return u.v;
}

// A stream over weights with a few rows beside them: NT * 16 rows of B (at
// brow[j], this lane's row of tile j) times RT * 16 rows of A (at arow[t]), both
// k-contiguous with K elements a row and of any alignment, over the steps of k
// that are this wave's of NW. Every lane holds U steps of 16-byte loads in
// flight; the loads of B come first, as A's addresses may still be on their way.
template <typename T, int NW, int RT, int NT, int U>
__device__ __forceinline__ void stream_rows(const T* const* brow, const T* const* arow, int K, int wave, int g,
                                            f32x4 (*acc)[NT]) {
  constexpr int P = Frag<T>::kPer, kStep = 4 * P;
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int steps = (K + kStep - 1) / kStep, per = (steps + NW - 1) / NW;
  const int s1 = min(steps, (wave + 1) * per), whole = min(s1, K / kStep);  // whole steps, and all of them
  int s = wave * per;
  auto batch = [&](auto steps_in_flight) {
    constexpr int V = decltype(steps_in_flight)::value;
    const int k = s * kStep + g * P;
    u32x4 fb[V][NT], fa[V][RT];
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j) fb[u][j] = load16(brow[j] + k + u * kStep);
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
      for (int t = 0; t < RT; ++t) fa[u][t] = load16(arow[t] + k + u * kStep);
#pragma unroll
    for (int u = 0; u < V; ++u) Frag<T>::template mma_tiles<RT, NT>(fb[u], fa[u], acc);
    s += V;
  };
  while (s + U <= whole) batch(std::integral_constant<int, U>{});
  // what is left in halves: each batch is one round trip to memory
  if (U > 4 && s + 4 <= whole) batch(std::integral_constant<int, 4>{});
  if (U > 2 && s + 2 <= whole) batch(std::integral_constant<int, 2>{});
  if (U > 1 && s < whole) batch(std::integral_constant<int, 1>{});
  if (s < s1) {  // the step at the end of the rows
    const int k = s * kStep + g * P;
    u32x4 fb[NT], fa[RT];
#pragma unroll
    for (int j = 0; j < NT; ++j) fb[j] = load_frag<T>(brow[j] + k, K - k);
#pragma unroll
    for (int t = 0; t < RT; ++t) fa[t] = load_frag<T>(arow[t] + k, K - k);
    Frag<T>::template mma_tiles<RT, NT>(fb, fa, acc);
  }
}

// Block b of `total` in launch order -> its place in an order in which the
// blocks that one XCD runs (every eighth) are neighbours and share its L2.
__device__ __forceinline__ int xcd_place(int b, int total) {
  const int q = total >> 3, r = total & 7, x = b & 7, i = b >> 3;
  return x < r ? x * (q + 1) + i : r * (q + 1) + (x - r) * q + i;
}

}  // namespace gmm
