// Device code shared by the kernels of the layers: element types, loads and
// stores, matrix instructions, activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/gmm.h"
#include "gmm_linear.hpp"

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

// Activations in single precision. A NaN z stays NaN. Float results take the
// FULL forms of gelu and silu (within 2^-20 of the value); results that are
// rounded to 2 bytes are within 2^-16 of it before, a thirty-second of half's
// half step, in fewer instructions. The form is part of the kernel: with both
// behind a branch the bfloat16 product of 8192 x 4096 to 16384 with gelu took
// 965 us against 912. The kernels' ACT is one of gmm_activation or these:
enum { kGeluFull = 4, kSiluFull = 5 };

// gelu is z Phi(z). With x = |z| the lower tail of the normal distribution is
//   Phi(-x) = exp(-x^2 / 2) r(x),  r(x) = erfc(x / sqrt 2) exp(x^2 / 2) / 2,
// where r falls slowly, like 1 / x, and t P(t), t = 1 / (1 + p x), with a
// polynomial P fits it with the smallest largest relative error over x = 0..14,
// beyond which the exponential is 0: of degree 8 with p = 0.2625 within 1.8e-8,
// of degree 6 with p = 0.265 within 6.3e-7. (A small absolute error of erfc is
// not enough: gelu's negative values are the tail itself.) The exponential is
// also the density's, which the slope needs.
struct Normal {
  float cdf, e;  // Phi(z), exp(-z^2 / 2)
};

// 2^(h + lo) for a small lo, the rounding errors of h.
__device__ __forceinline__ float exp2_of(float h, float lo) {
  const float e = __builtin_amdgcn_exp2f(h);
  return fmaf(e, 0.69314718055994531f * lo, e);
}

template <bool FULL>
__device__ __forceinline__ Normal normal_of(float z) {
  float tail, e;
  if (FULL) {
    const float x = fminf(fabsf(z), 16.f);  // from here on the exponential is 0
    const float d = fmaf(0.2625f, x, 1.f), t0 = __builtin_amdgcn_rcpf(d), t = fmaf(fmaf(-d, t0, 1.f), t0, t0);
    // -x^2 / 2 in units of log 2, with what its roundings leave
    constexpr float kHigh = 0.721347511f, kLow = 9.62981495e-9f;
    const float s = x * x, h = -kHigh * s;
    e = exp2_of(h, fmaf(-kHigh, fmaf(x, x, -s), fmaf(-kLow, s, fmaf(-kHigh, s, -h))));
    float q = fmaf(0.0307454728f, t, -0.148810312f);
    q = fmaf(q, t, 0.234761387f);
    q = fmaf(q, t, -0.133391514f);
    q = fmaf(q, t, 0.149138391f);
    q = fmaf(q, t, 0.0558492616f);
    q = fmaf(q, t, 0.102818556f);
    q = fmaf(q, t, 0.104138888f);
    q = fmaf(q, t, 0.104749881f);
    tail = q * t * e;
  } else {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.265f, fabsf(z), 1.f));
    e = __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
    float q = fmaf(-0.0677870363f, t, 0.195273101f);
    q = fmaf(q, t, -0.0663629025f);
    q = fmaf(q, t, 0.142493322f);
    q = fmaf(q, t, 0.0829465911f);
    q = fmaf(q, t, 0.107836783f);
    q = fmaf(q, t, 0.105599836f);
    tail = q * t * e;
  }
  return {z < 0.f ? tail : 1.f - tail, e};
}

// 1 / (1 + exp(-z)) and 1 / (1 + exp(z)).
struct Logistic {
  float q, p;
};
template <bool FULL>
__device__ __forceinline__ Logistic logistic(float z) {
  if (FULL) {
    const float x = fminf(fabsf(z), 128.f);  // from here on the exponential is 0
    constexpr float kHigh = 1.44269502f, kLow = 1.92596299e-8f;
    const float h = -kHigh * x, e = exp2_of(h, fmaf(-kLow, x, fmaf(-kHigh, x, -h)));
    const float near = 1.f / (1.f + e), far = e / (1.f + e);
    return z < 0.f ? Logistic{far, near} : Logistic{near, far};
  }
  // a far negative z gives 1 / inf = 0
  const float q = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * z));
  return {q, 1.f - q};
}

template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == GMM_ACT_RELU) return z < 0.f ? 0.f : z;
  if (ACT == GMM_ACT_GELU || ACT == kGeluFull) return z * normal_of<ACT == kGeluFull>(z).cdf;
  if (ACT == GMM_ACT_SILU || ACT == kSiluFull) return z * logistic<ACT == kSiluFull>(z).q;
  return z;
}

// z held to +-most; a NaN stays one.
__device__ __forceinline__ float within(float z, float most) { return z > most ? most : z < -most ? -most : z; }

// The slopes are constant beyond 16 and 128, where the exponentials are 0. z is
// held to that range because a pre of 2 bytes may be infinite where z was not,
// and infinity times 0 is not the slope's limit.
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == GMM_ACT_RELU) return z > 0.f ? 1.f : z == z ? 0.f : z;
  if (ACT == GMM_ACT_GELU || ACT == kGeluFull) {
    z = within(z, 16.f);
    const Normal n = normal_of<ACT == kGeluFull>(z);
    return fmaf(0.39894228040143268f * z, n.e, n.cdf);
  }
  if (ACT == GMM_ACT_SILU || ACT == kSiluFull) {
    z = within(z, 128.f);
    const Logistic l = logistic<ACT == kSiluFull>(z);
    return l.q * (1.f + z * l.p);
  }
  return 1.f;
}

// f with the activation's form for results of type T, or float where `to_float`
// (only if MIXED).
template <typename T, bool MIXED, typename F>
hipError_t with_act(int act, bool to_float, F&& f) {
  if (act == GMM_ACT_RELU) return f(std::integral_constant<int, GMM_ACT_RELU>{});
  if constexpr (MIXED || sizeof(T) == 4) {
    if (to_float || sizeof(T) == 4) {
      if (act == GMM_ACT_GELU) return f(std::integral_constant<int, kGeluFull>{});
      if (act == GMM_ACT_SILU) return f(std::integral_constant<int, kSiluFull>{});
    }
  }
  if constexpr (sizeof(T) != 4) {
    if (act == GMM_ACT_GELU) return f(std::integral_constant<int, GMM_ACT_GELU>{});
    if (act == GMM_ACT_SILU) return f(std::integral_constant<int, GMM_ACT_SILU>{});
  }
  return f(std::integral_constant<int, GMM_ACT_NONE>{});
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

// W consecutive values of a row, n of them inside it, as floats; whole ones in
// 16-byte accesses of any alignment.
template <typename E, int W>
__device__ __forceinline__ void load_as(const E* q, int n, float* out) {
  constexpr int P = 16 / sizeof(E) < W ? 16 / sizeof(E) : W;
  if (n >= W) {
#pragma unroll
    for (int i = 0; i < W; i += P) {
      E e[P];
      __builtin_memcpy(e, q + i, sizeof(e));
#pragma unroll
      for (int k = 0; k < P; ++k) out[i + k] = (float)e[k];
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) out[i] = i < n ? (float)q[i] : 0.f;
  }
}

// STREAM: past the caches' replacement, for what is too large to be found there.
template <typename E, int W, bool STREAM = false>
__device__ __forceinline__ void store_as(E* q, int n, const float* v) {
  constexpr int P = 16 / sizeof(E) < W ? 16 / sizeof(E) : W;
  if (n >= W) {
#pragma unroll
    for (int i = 0; i < W; i += P) {
      E e[P];
#pragma unroll
      for (int k = 0; k < P; ++k) e[k] = (E)v[i + k];
      if constexpr (STREAM && sizeof(e) == 16) {
        typedef u32x4 any_u32x4 __attribute__((aligned(2)));
        u32x4 w;
        __builtin_memcpy(&w, e, 16);
        __builtin_nontemporal_store(w, reinterpret_cast<any_u32x4*>(q + i));
      } else {
        __builtin_memcpy(q + i, e, sizeof(e));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (i < n) q[i] = (E)v[i];
  }
}

// The same at element `at` of an array of C's type.
template <typename T, int W>
__device__ __forceinline__ void load_row(const void* p, int64_t at, int n, bool is_f32, float* out) {
  if (is_f32)
    load_as<float, W>(static_cast<const float*>(p) + at, n, out);
  else
    load_as<T, W>(static_cast<const T*>(p) + at, n, out);
}

template <typename T, int W, bool STREAM = false>
__device__ __forceinline__ void store_row(void* p, int64_t at, int n, bool is_f32, const float* v) {
  if (is_f32)
    store_as<float, W, STREAM>(static_cast<float*>(p) + at, n, v);
  else
    store_as<T, W, STREAM>(static_cast<T*>(p) + at, n, v);
}

// Sums of K values over the G threads of a row, in every thread and in a fixed
// order. Rows of several waves meet in LDS: `red` has two halves that calls take
// in turn, so one barrier a call is enough (who writes a half again has passed
// the barrier that all pass after reading it).
template <int G, int K>
__device__ __forceinline__ void row_sum(float* v, float (*red)[G > 64 ? G / 64 : 1][2], int& turn) {
#pragma unroll
  for (int o = (G < 64 ? G : 64) / 2; o; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], o);
  if constexpr (G > 64) {
    const int wave = threadIdx.x / 64;
    if (threadIdx.x % 64 == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) red[turn][wave][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.f;
#pragma unroll
      for (int w = 0; w < G / 64; ++w) v[k] += red[turn][w][k];
    }
    turn ^= 1;
  }
}

// exp(x), x <= 0 or so: the error is that of x log2(e) in float, |x| 2^-23.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(1.44269504088896341f * x); }

// A row's pick: a class and its weight, -1 and 0 where there is none.
struct Pick {
  int v;
  float w;
};
__device__ __forceinline__ Pick pick_of(const RowPicks& p, int64_t row, int j, int V) {
  const int64_t at = row * p.top + j;
  const int v = p.idx[at];
  const bool is = v >= 0 && v < V;
  return {is ? v : -1, !is ? 0.f : p.wts ? p.wts[at] : 1.f};
}

// The gradients of W logits of a row, from column `col` of V on; 0 behind the
// last. z are the logits, or (KEPT) numbers that c.up makes their dloss s p. What
// few pieces have, picks and the last column, is behind branches: with
// a comparison for each entry the products that end in this (8192 x 64 to 32768
// classes) took 271 us, so 222.
template <int W, bool KEPT = false>
__device__ __forceinline__ void logit_gradient(const RowCoef& c, const RowPicks& picks, int64_t row, int col, int V,
                                               const float* z, float* g) {
  if (c.d == 0.f) {
#pragma unroll
    for (int i = 0; i < W; ++i) g[i] = 0.f;
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) g[i] = c.up * (KEPT ? z[i] : exp_of(z[i] - c.base));
  if (col + W > V)
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (col + i >= V) g[i] = 0.f;
  if (!c.all) {
    if ((unsigned)(c.v0 - col) < (unsigned)W)
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (col + i == c.v0) g[i] -= c.c0;
    if ((unsigned)(c.v1 - col) < (unsigned)W)
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (col + i == c.v1) g[i] -= c.c1;
    return;
  }
  for (int j = 0; j < picks.top; ++j) {
    const Pick k = pick_of(picks, row, j, V);
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (col + i == k.v) g[i] = fmaf(-c.d, k.w, g[i]);
  }
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
