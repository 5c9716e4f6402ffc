// The AdamW step over many tensors.
#include "gmm_adamw.hpp"

#include <type_traits>

#include "gmm_product.hpp"

namespace gmm {

constexpr int kAdamWaves = 4;
constexpr float kF8Most = 448.f;  // the largest e4m3 value

// 32 bits for an element of the state at a step: what decides how its 8-bit
// states are rounded; the states repeat exactly. A multiply-xorshift hash with the
// shifts and factors that C. Wellons' search for such hashes of least bias
// published ("Prospecting for Hash Functions", 2018); the step's factor is 2^32
// over the golden ratio.
__device__ __forceinline__ uint32_t chance(uint32_t place, uint32_t step) {
  uint32_t x = place ^ (step * 0x9E3779B1u);
  x = (x ^ (x >> 16)) * 0x7FEB352Du;
  x = (x ^ (x >> 15)) * 0x846CA68Bu;
  return x ^ (x >> 16);
}

// x * up as an e4m3 value: of its two neighbours the larger one where `bits`
// (16 of them, as a fraction) and the share that lies beyond the smaller come
// to 1 or more. A moving average moves by less than half a step of 3 bits, and
// would never leave its value were it rounded to the nearest. Not a number stays
// so, infinity becomes it.
__device__ __forceinline__ float to_f8(float x, uint32_t bits) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x), a = u & 0x7fffffffu;
  float q;
  if (a >= 0x3c800000u) {  // 2^-6 and more: 3 bits of the mantissa stay
    q = __builtin_bit_cast(float, (a + (bits << 4)) & 0xfff00000u);
    q = fminf(q, kF8Most);
  } else {  // steps of 2^-9
    q = floorf(fmaf(__builtin_bit_cast(float, a), 512.f, (float)bits * (1.f / 65536.f))) * (1.f / 512.f);
  }
  if (a >= 0x7f800000u) q = __builtin_nanf("");
  return __builtin_copysignf(q, x);
}

__device__ __forceinline__ float wave_most(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// The four e4m3 values of a word.
__device__ __forceinline__ void from_f8(uint32_t c, float* out) {
  out[0] = __builtin_amdgcn_cvt_f32_fp8(c, 0);
  out[1] = __builtin_amdgcn_cvt_f32_fp8(c, 1);
  out[2] = __builtin_amdgcn_cvt_f32_fp8(c, 2);
  out[3] = __builtin_amdgcn_cvt_f32_fp8(c, 3);
}

// A step's numbers that are the same for all elements.
struct AdamStep {
  float beta1, beta2, rest1, rest2, scale_g, shrink, rate, root, eps;
  uint32_t n;
};

// What a lane holds of a block of the state. STREAM: past the caches'
// replacement, for states too large to be found there at the next step.
template <typename TP, typename TG, bool MASTER, bool F8, bool STREAM>
struct AdamLane {
  TG g[4];
  TP p[4];
  float master[4], m[4], v[4], ms, vs;
  uint32_t mc, vc;

  // The first `left` of 4 elements.
  template <typename E>
  static __device__ __forceinline__ void get(const E* q, int left, E* out) {
    if (left == 4) {
      typedef E Four __attribute__((ext_vector_type(4), aligned(sizeof(E))));
      const Four* from = reinterpret_cast<const Four*>(q);
      const Four w = STREAM ? __builtin_nontemporal_load(from) : *from;
      __builtin_memcpy(out, &w, sizeof(w));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) out[k] = k < left ? q[k] : (E)0.f;
    }
  }
  template <typename E>
  static __device__ __forceinline__ void put(E* q, int left, const E* from) {
    if (left == 4) {
      typedef E Four __attribute__((ext_vector_type(4), aligned(sizeof(E))));
      Four w, *to = reinterpret_cast<Four*>(q);
      __builtin_memcpy(&w, from, sizeof(w));
      if (STREAM)
        __builtin_nontemporal_store(w, to);
      else
        *to = w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < left) q[k] = from[k];
    }
  }

  __device__ __forceinline__ void load(const AdamArgs& a, const AdamArgs::Tensor& t, int64_t e, int left) {
    const int64_t at = t.at + e;
    get(static_cast<const TG*>(t.g) + e, left, g);
    if (MASTER)
      get(a.master + at, left, master);
    else
      get(static_cast<const TP*>(t.p) + e, left, p);
    if (F8) {  // whole words: the state's own padding lies behind a tensor's last element
      uint8_t c[2][4];
      get(static_cast<const uint8_t*>(a.m) + at, 4, c[0]);
      get(static_cast<const uint8_t*>(a.v) + at, 4, c[1]);
      __builtin_memcpy(&mc, c[0], 4);
      __builtin_memcpy(&vc, c[1], 4);
      ms = a.m_scale[at / kStateBlock];
      vs = a.v_scale[at / kStateBlock];
    } else {
      get(static_cast<const float*>(a.m) + at, left, m);
      get(static_cast<const float*>(a.v) + at, left, v);
    }
  }

  // In the averages every product and sum is rounded by itself, so that what 8
  // bits hold follows from float arithmetic whatever the compiler fuses.
  __device__ __forceinline__ void step(const AdamStep& s) {
#pragma clang fp contract(off)
    if (F8) {
      from_f8(mc, m);
      from_f8(vc, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        m[k] = m[k] * ms;
        const float r = v[k] * vs;
        v[k] = r * r;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = (float)g[k] * s.scale_g;
      m[k] = s.beta1 * m[k] + s.rest1 * x;
      v[k] = s.beta2 * v[k] + s.rest2 * x * x;
      const float r = sqrtf(v[k]);  // the instruction alone would take a denormal v for 0
      const float old = MASTER ? master[k] : (float)p[k];
      // lr decay stays a small number of its own: in 1 - lr decay it would be a multiple of 2^-24, for all elements alike
      master[k] = old - fmaf(s.shrink, old, s.rate * m[k] * __builtin_amdgcn_rcpf(fmaf(r, s.root, s.eps)));
      p[k] = (TP)master[k];
      if (F8) v[k] = r;
    }
  }

  __device__ __forceinline__ void store(const AdamArgs& a, const AdamArgs::Tensor& t, const AdamStep& s, int64_t e,
                                        int left) {
    const int64_t at = t.at + e;
    if (MASTER) put(a.master + at, left, master);
    put(static_cast<TP*>(t.p) + e, left, p);
    if (!F8) {
      put(static_cast<float*>(a.m) + at, left, m);
      put(static_cast<float*>(a.v) + at, left, v);
      return;
    }
    float mm = 0.f, vm = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < left) {
        const float x = fabsf(m[k]);
        if (x < __builtin_inff()) mm = fmaxf(mm, x);
        if (v[k] < __builtin_inff()) vm = fmaxf(vm, v[k]);
      }
    mm = wave_most(mm);
    vm = wave_most(vm);
    // below 448 / FLT_MAX the factor would be infinite: the block is held as 0
    const float mu = mm > 1e-35f ? 1.f / mm * kF8Most : 0.f, vu = vm > 1e-35f ? 1.f / vm * kF8Most : 0.f;
    float q[4], r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t h = chance((uint32_t)(at + k), s.n);
      q[k] = to_f8(m[k] * mu, h & 0xffff);
      r[k] = to_f8(v[k] * vu, h >> 16);
      if (v[k] > 0.f && vu > 0.f && r[k] < 1.f / 512.f) r[k] = 1.f / 512.f;  // it is divided by
    }
    int w[2] = {0, 0};
    w[0] = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], w[0], false);
    w[0] = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w[0], true);
    w[1] = __builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], w[1], false);
    w[1] = __builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], w[1], true);
    uint8_t b[2][4];
    __builtin_memcpy(b, w, 8);
    put(static_cast<uint8_t*>(a.m) + at, left, b[0]);
    put(static_cast<uint8_t*>(a.v) + at, left, b[1]);
    if ((threadIdx.x & 63) == 0) {
      a.m_scale[at / kStateBlock] = mu > 0.f ? mm * (1.f / kF8Most) : 0.f;
      a.v_scale[at / kStateBlock] = vu > 0.f ? vm * (1.f / kF8Most) : 0.f;
    }
  }
};

// ---------------------------------------------------------------------------
//   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
//   p = p - lr decay p - lr (m / (1 - beta1^n)) / (sqrt(v / (1 - beta2^n)) + eps)
// HBM bounds it: every byte of p, m, v and the float copy moves once each way,
// g once. A wave takes 256 elements (a block of the state) at a time, 4
// consecutive ones a lane, with 4 blocks in flight. The tensors come in the
// kernel's arguments, so that a launch needs no table in memory. 268M bfloat16
// parameters with float copies and states: 1340 us, 5.6 TB/s; with one block in
// flight 1346, through the caches 1435, with 512 blocks of the state a thread
// block 1436. The same with 8 bits: 804 us, 5.3 TB/s, and 841, 847, 869.
// 8 bits: m and sqrt(v) as e4m3 with a scale for each 256 elements, its largest
// finite value / 448; sqrt(v) because its range is half as wide.
// ---------------------------------------------------------------------------
template <typename TP, typename TG, bool MASTER, bool F8, bool STREAM>
__global__ void __launch_bounds__(64 * kAdamWaves) adamw_kernel(const AdamArgs a) {
  const int64_t n = a.step[0] + 1;
  const int block = blockIdx.x;
  if (block < a.first[a.count]) {
    constexpr int U = 4;
    int i = 0;  // the tensor whose blocks hold this one: the last with first <= block
    for (int step = 64; step; step >>= 1)
      if (i + step < a.count && a.first[i + step] <= block) i += step;
    const AdamArgs::Tensor t = a.tensor[i];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const float lr = a.lr * (a.lr_factor ? *a.lr_factor : 1.f);
    const double c1 = -expm1((double)n * a.log_beta1), c2 = -expm1((double)n * a.log_beta2);
    const AdamStep s{a.beta1, a.beta2, a.rest1, a.rest2, a.grad_factor ? *a.grad_factor : 1.f, lr * a.decay,
                     (float)(lr / c1), (float)(1. / sqrt(c2)), a.eps, (uint32_t)n};
    const int64_t blocks = (t.n + kStateBlock - 1) / kStateBlock, b0 = (int64_t)(block - a.first[i]) * a.chunk;
    const int64_t b1 = b0 + a.chunk < blocks ? b0 + a.chunk : blocks;
    const int64_t whole = t.n / kStateBlock < b1 ? t.n / kStateBlock : b1;
    AdamLane<TP, TG, MASTER, F8, STREAM> l[U];
    int64_t b = b0 + wave;
    for (; b + (U - 1) * kAdamWaves < whole; b += U * kAdamWaves) {
#pragma unroll
      for (int u = 0; u < U; ++u) l[u].load(a, t, (b + u * kAdamWaves) * kStateBlock + 4 * lane, 4);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        l[u].step(s);
        l[u].store(a, t, s, (b + u * kAdamWaves) * kStateBlock + 4 * lane, 4);
      }
    }
    for (; b < b1; b += kAdamWaves) {
      const int64_t e = b * kStateBlock + 4 * lane;
      const int left = (int)(t.n - e < 4 ? (t.n > e ? t.n - e : 0) : 4);
      l[0].load(a, t, e, left);
      l[0].step(s);
      l[0].store(a, t, s, e, left);
    }
  }
  // The block that is done last counts the step: all others have read it then (a
  // value that was used has arrived; nothing else passes between blocks, so no
  // fence, which costs a block as much as 60 KB of its work). Earlier launches of
  // the same call are done altogether.
  if (!a.last) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned long long* done = reinterpret_cast<unsigned long long*>(a.step + 1);
    if (__hip_atomic_fetch_add(done, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1 == gridDim.x) {
      a.step[0] = n;
      a.step[1] = 0;
    }
  }
}

template <typename TP, typename TG, bool MASTER>
static hipError_t launch_adamw_types(int bits, const AdamArgs& a, hipStream_t s) {
  const unsigned grid = a.first[a.count] > 0 ? (unsigned)a.first[a.count] : 1u;
  auto go = [&](auto kernel) { kernel<<<grid, 64 * kAdamWaves, 0, s>>>(a); };
  if (bits == 8)
    a.stream ? go(adamw_kernel<TP, TG, MASTER, true, true>) : go(adamw_kernel<TP, TG, MASTER, true, false>);
  else
    a.stream ? go(adamw_kernel<TP, TG, MASTER, false, true>) : go(adamw_kernel<TP, TG, MASTER, false, false>);
  return hipGetLastError();
}

template <typename TP>
static hipError_t launch_adamw_half(int g_dtype, int bits, const AdamArgs& a, hipStream_t s) {
  if (g_dtype == GMM_F32)
    return a.master ? launch_adamw_types<TP, float, true>(bits, a, s) : launch_adamw_types<TP, float, false>(bits, a, s);
  return a.master ? launch_adamw_types<TP, TP, true>(bits, a, s) : launch_adamw_types<TP, TP, false>(bits, a, s);
}

hipError_t launch_adamw(int p_dtype, int g_dtype, int bits, const AdamArgs& a, hipStream_t s) {
  if (p_dtype == GMM_F16) return launch_adamw_half<_Float16>(g_dtype, bits, a, s);
  if (p_dtype == GMM_BF16) return launch_adamw_half<__bf16>(g_dtype, bits, a, s);
  return launch_adamw_types<float, float, false>(bits, a, s);
}

}  // namespace gmm
