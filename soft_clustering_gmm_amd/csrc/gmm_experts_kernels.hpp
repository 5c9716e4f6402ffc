// Kernels of the layer of experts, instantiated once per element type.
#pragma once

#include <climits>
#include <type_traits>

#include "gmm_experts.hpp"
#include "gmm_product.hpp"

namespace gmm {

// ---------------------------------------------------------------------------
// Gate: the mixture's posterior at the row's features, in double precision
// throughout, since a pick is decided by the difference of two scores.
// ---------------------------------------------------------------------------

// f[t][j] = P_j . x_t, one wave per feature and 4 rows.
template <typename T>
__global__ void __launch_bounds__(256) gate_features_kernel(const ExpertArgs p) {
  constexpr int P = Frag<T>::kPer, R = 4;
  const int lane = threadIdx.x & 63, j = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int t0 = blockIdx.y * R;
  if (j >= p.d) return;
  const T* w = static_cast<const T*>(p.proj) + (int64_t)j * p.D;
  const T* x[R];
#pragma unroll
  for (int r = 0; r < R; ++r) x[r] = static_cast<const T*>(p.X) + (int64_t)min(t0 + r, p.T - 1) * p.D;
  double sum[R] = {0., 0., 0., 0.};
  for (int k = lane * P; k < p.D; k += 64 * P) {
    union U {
      u32x4 v;
      T e[P];
    } a, b;
    a.v = load_frag<T>(w + k, p.D - k);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      b.v = load_frag<T>(x[r] + k, p.D - k);
#pragma unroll
      for (int i = 0; i < P; ++i) sum[r] = fma((double)(float)a.e[i], (double)(float)b.e[i], sum[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int o = 32; o; o >>= 1) sum[r] += __shfl_xor(sum[r], o);
    if (lane == 0 && t0 + r < p.T) p.feats[(int64_t)(t0 + r) * p.d + j] = sum[r];
  }
}

struct Best {
  double s;
  int k;
};
__device__ __forceinline__ bool better(double s, int k, const Best& b) { return s > b.s || (s == b.s && k < b.k); }

// Scores of one row against all components, then its picks. One wave scores a
// component at a time, two features per lane; sum_j log var_j is taken as the
// logarithm of the product of the mantissas (at least 2^-128) and the sum of
// the exponents, one logarithm a component.
template <int NW>
__global__ void __launch_bounds__(64 * NW) gate_pick_kernel(const ExpertArgs p) {
  __shared__ Best wave_best[NW];
  __shared__ double wave_sum[NW];
  __shared__ int odd;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x;
  const int j0 = lane, j1 = lane + 64;
  const double* f = p.feats + (int64_t)t * p.d;
  const double f0 = j0 < p.d ? f[j0] : 0., f1 = j1 < p.d ? f[j1] : 0.;
  double* sc = p.scores + (int64_t)t * p.K;
  if (threadIdx.x == 0) odd = 0;
  __syncthreads();
  for (int k = wave; k < p.K; k += NW) {
    const float *mu = p.mu + (int64_t)k * p.d, *var = p.var + (int64_t)k * p.d;
    double q = 0., m = 1.;
    int e = 0;
    if (j0 < p.d) {
      const double v = var[j0], u = f0 - mu[j0];
      q = u * u / v;
      m = frexp(v, &e);
    }
    if (j1 < p.d) {
      const double v = var[j1], u = f1 - mu[j1];
      int e1;
      q += u * u / v;
      m *= frexp(v, &e1);
      e += e1;
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
      q += __shfl_xor(q, o);
      m *= __shfl_xor(m, o);
      e += __shfl_xor(e, o);
    }
    if (lane == 0) {
      const double log2pi = 1.8378770664093454836, ln2 = 0.69314718055994530942;
      const double s = (double)p.logw[k] - 0.5 * (p.d * log2pi + (log(m) + e * ln2) + q);
      sc[k] = s;
      if (!(s < INFINITY)) odd = 1;  // NaN or +inf: the posterior is not a number
    }
  }
  __threadfence_block();
  __syncthreads();

  Best last{INFINITY, -1};
  double lse = 0., kept = 0.;
  double r_of[kMaxTop];
  int k_of[kMaxTop];
  bool bad = odd != 0;
#pragma unroll
  for (int pick = 0; pick < kMaxTop; ++pick) {
    if (pick >= p.top) break;
    Best b{-INFINITY, INT_MAX};
    for (int k = threadIdx.x; k < p.K; k += 64 * NW) {
      const double s = sc[k];
      // after the last pick in the order (score down, index up)
      if ((s < last.s || (s == last.s && k > last.k)) && better(s, k, b)) b = Best{s, k};
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) {
      const double s = __shfl_xor(b.s, o);
      const int k = __shfl_xor(b.k, o);
      if (better(s, k, b)) b = Best{s, k};
    }
    if (lane == 0) wave_best[wave] = b;
    __syncthreads();
    b = wave_best[0];
#pragma unroll
    for (int w = 1; w < NW; ++w)
      if (better(wave_best[w].s, wave_best[w].k, b)) b = wave_best[w];
    if (pick == 0) {  // the normaliser
      double z = 0.;
      for (int k = threadIdx.x; k < p.K; k += 64 * NW) z += exp(sc[k] - b.s);
#pragma unroll
      for (int o = 32; o; o >>= 1) z += __shfl_xor(z, o);
      if (lane == 0) wave_sum[wave] = z;
      __syncthreads();
      z = 0.;
#pragma unroll
      for (int w = 0; w < NW; ++w) z += wave_sum[w];
      bad = bad || !(b.s > -INFINITY);
      lse = b.s + log(z);
    }
    __syncthreads();
    // components of weight zero (score -inf) are no picks
    const bool some = !bad && b.k != INT_MAX && b.s > -INFINITY;
    const double r = some ? exp(b.s - lse) : 0.;
    const bool keep = some && (pick == 0 || r >= (double)p.threshold);
    k_of[pick] = keep ? b.k : -1;
    r_of[pick] = keep ? r : 0.;
    kept += r_of[pick];
    last = b;
  }
  if (threadIdx.x == 0) {
    p.bad[t] = bad;
#pragma unroll
    for (int pick = 0; pick < kMaxTop; ++pick) {
      if (pick >= p.top) break;
      const int at = t * p.top + pick;
      p.idx[at] = k_of[pick];
      p.resp[at] = (float)r_of[pick];
      p.wts[at] = (float)(p.renorm && k_of[pick] >= 0 ? r_of[pick] / kept : r_of[pick]);
    }
  }
}

// ---------------------------------------------------------------------------
// Experts' products. A block takes one expert with picks and 16 rows of its
// weights, reads them once, and multiplies them with all rows of X (or of h)
// picked for that expert, 16 at a time. The waves split the contraction.
// UP: h = act(W1 x + b1), or with GLU act(gate) * up, the block's 16 weight
// rows being 8 gate rows and their 8 up rows. Otherwise: out = W2 h.
// ---------------------------------------------------------------------------
template <typename T, int NW, int RT, bool UP, bool GLU, int ACT>
__device__ __forceinline__ void expert_rows_part(const ExpertArgs& p, const T* B, int K, int e, int place0, int rows,
                                                 float (*red)[RT][16][17]) {
  constexpr int P = Frag<T>::kPer, kStep = 4 * P, U = RT == 1 ? 8 : 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const T* A[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int place = place0 + min(16 * t + r, rows - 1);
    A[t] = (UP ? static_cast<const T*>(p.X) + (int64_t)p.row_of[place] * K
               : static_cast<const T*>(p.h) + (int64_t)place * K) + g * P;
  }
  f32x4 acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int steps = (K + kStep - 1) / kStep, per = (steps + NW - 1) / NW;
  const int s1 = min(steps, (wave + 1) * per);
  int s = wave * per;
  for (; s + U <= s1 && (s + U) * kStep <= K; s += U) {
    u32x4 fb[U], fa[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      fb[u] = load16(B + (s + u) * kStep);
#pragma unroll
      for (int t = 0; t < RT; ++t) fa[u][t] = load16(A[t] + (s + u) * kStep);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[t] = Frag<T>::mma(fb[u], fa[u][t], acc[t]);
  }
  for (; s < s1; ++s) {
    const int left = K - s * kStep - g * P;
    const u32x4 fb = load_frag<T>(B + s * kStep, left);
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = Frag<T>::mma(fb, load_frag<T>(A[t] + s * kStep, left), acc[t]);
  }
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) red[wave][t][r][4 * g + q] = acc[t][q];
  __syncthreads();
  constexpr int kOut = GLU ? 8 : 16;
  const int N = UP ? p.F : p.D, n0 = blockIdx.x * kOut;
  for (int i = threadIdx.x; i < 16 * RT * kOut; i += 64 * NW) {
    const int n = i % kOut, m = i / kOut;
    if (m >= rows || n0 + n >= N) continue;
    float z = 0.f, u = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      z += red[w][m >> 4][m & 15][n];
      if (GLU) u += red[w][m >> 4][m & 15][n + 8];
    }
    const int64_t place = place0 + m;
    if (UP) {
      const T* b1 = static_cast<const T*>(p.b1);
      const int64_t at = (int64_t)e * (GLU ? 2 * p.F : p.F) + n0 + n;
      if (b1) z += (float)b1[at];
      if (GLU && b1) u += (float)b1[at + p.F];
      z = act_value<ACT>(z);
      // rounded to the operands' type: what the second product's matrix instruction takes
      static_cast<T*>(p.h)[place * p.F + n0 + n] = (T)(GLU ? z * u : z);
    } else {
      p.out[place * p.D + n0 + n] = z;
    }
  }
  __syncthreads();
}

template <typename T, int NW, int RT, bool UP, bool GLU, int ACT>
__global__ void __launch_bounds__(64 * NW) expert_kernel(const ExpertArgs p) {
  __shared__ float red[NW * RT * 16 * 17];
  const int a = blockIdx.y;
  if (a >= *p.count) return;
  const int e = p.expert[a], first = p.first[a], rows = p.first[a + 1] - first;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int K = UP ? p.D : p.F, N = UP ? (GLU ? 2 * p.F : p.F) : p.D;
  int brow;
  if (GLU)
    brow = (r < 8 ? 0 : p.F) + min((int)blockIdx.x * 8 + (r & 7), p.F - 1);
  else
    brow = min((int)blockIdx.x * 16 + r, N - 1);
  const T* B = static_cast<const T*>(UP ? p.W1 : p.W2) + ((int64_t)e * N + brow) * K + g * Frag<T>::kPer;
  if (RT == 1 || rows <= 16) {
    for (int i = 0; i < rows; i += 16)
      expert_rows_part<T, NW, 1, UP, GLU, ACT>(p, B, K, e, first + i, min(16, rows - i),
                                               reinterpret_cast<float(*)[1][16][17]>(red));
  } else {
    for (int i = 0; i < rows; i += 16 * RT)
      expert_rows_part<T, NW, RT, UP, GLU, ACT>(p, B, K, e, first + i, min(16 * RT, rows - i),
                                                reinterpret_cast<float(*)[RT][16][17]>(red));
  }
}

// y = residual + sum over the row's picks of w (out + b2), in the picks' order.
template <typename T>
__global__ void __launch_bounds__(256) expert_combine_kernel(const ExpertArgs p) {
  const int c = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
  if (c >= p.D) return;
  const int64_t at = (int64_t)t * p.D + c;
  float y = p.residual ? (float)static_cast<const T*>(p.residual)[at] : 0.f;
  for (int i = 0; i < p.top; ++i) {
    const int pick = t * p.top + i, place = p.place[pick];
    if (place < 0) continue;
    float o = p.out[(int64_t)place * p.D + c];
    if (p.b2) o += (float)static_cast<const T*>(p.b2)[(int64_t)p.in_idx[pick] * p.D + c];
    y += p.in_wts[pick] * o;
  }
  if (p.bad && p.bad[t]) y = NAN;
  static_cast<T*>(p.Y)[at] = (T)y;
}

// --------------------------------------------------------------------------- launchers

template <typename T>
hipError_t launch_gate(const ExpertArgs& p, hipStream_t s) {
  gate_features_kernel<T><<<dim3((p.d + 3) / 4, (p.T + 3) / 4), 256, 0, s>>>(p);
  gate_pick_kernel<8><<<p.T, 512, 0, s>>>(p);
  return hipGetLastError();
}

template <typename T, int RT, bool GLU, int ACT>
static void launch_expert_products(const ExpertArgs& p, int active, hipStream_t s) {
  constexpr int kOut = GLU ? 8 : 16;
  expert_kernel<T, 4, RT, true, GLU, ACT><<<dim3((p.F + kOut - 1) / kOut, active), 256, 0, s>>>(p);
  expert_kernel<T, 4, RT, false, false, GMM_ACT_NONE><<<dim3((p.D + 15) / 16, active), 256, 0, s>>>(p);
}

template <typename T, int ACT>
static void launch_experts_act(const ExpertArgs& p, hipStream_t s) {
  const int n = p.T * p.top, active = n < p.K ? n : p.K;
  if (p.T <= 16) {
    if (p.glu)
      launch_expert_products<T, 1, true, ACT>(p, active, s);
    else
      launch_expert_products<T, 1, false, ACT>(p, active, s);
  } else {
    if (p.glu)
      launch_expert_products<T, 4, true, ACT>(p, active, s);
    else
      launch_expert_products<T, 4, false, ACT>(p, active, s);
  }
}

template <typename T>
hipError_t launch_experts(int act, const ExpertArgs& p, hipStream_t s) {
  if (act == GMM_ACT_RELU)
    launch_experts_act<T, GMM_ACT_RELU>(p, s);
  else if (act == GMM_ACT_GELU)
    launch_experts_act<T, GMM_ACT_GELU>(p, s);
  else if (act == GMM_ACT_SILU)
    launch_experts_act<T, GMM_ACT_SILU>(p, s);
  else
    launch_experts_act<T, GMM_ACT_NONE>(p, s);
  expert_combine_kernel<T><<<dim3((p.D + 255) / 256, p.T), 256, 0, s>>>(p);
  return hipGetLastError();
}

#define GMM_EXPERTS_TYPE(T)                                          \
  template hipError_t launch_gate<T>(const ExpertArgs&, hipStream_t); \
  template hipError_t launch_experts<T>(int, const ExpertArgs&, hipStream_t);

}  // namespace gmm
