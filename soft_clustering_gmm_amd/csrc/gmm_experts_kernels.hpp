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

typedef double f64x4 __attribute__((ext_vector_type(4)));

// c_k = logw_k - 1/2 (d log 2 pi + sum_j log var_kj), 16 components a block of
// 256 threads, 16 lanes each. The sum is the logarithm of the product of the
// mantissas (at least 2^-128) and the sum of the exponents: one logarithm a
// component.
__device__ __forceinline__ void gate_constants(const ExpertArgs& p, int block) {
  const int l16 = threadIdx.x & 15, k = block * 16 + (threadIdx.x >> 4);
  if (k >= p.K) return;
  double mant = 1.;
  int e = 0;
  for (int j = l16; j < p.d; j += 16) {
    int ej;
    mant *= frexp((double)p.var[(int64_t)k * p.d + j], &ej);
    e += ej;
  }
#pragma unroll
  for (int o = 8; o; o >>= 1) {
    mant *= __shfl_xor(mant, o);
    e += __shfl_xor(e, o);
  }
  const double log2pi = 1.8378770664093454836, ln2 = 0.69314718055994530942;
  if (l16 == 0) p.consts[k] = (double)p.logw[k] - 0.5 * (p.d * log2pi + (log(mant) + e * ln2));
}

// f[t][j] = P_j . x_t on the double-precision matrix instruction, in
// kGateParts parts of the contraction that the next kernel adds up: a row or
// two alone would leave most of the chip idle. A block owns 16 features, 16
// rows and a part, its 4 waves split that again. Every lane loads 16 bytes of
// its row, and element i of all lanes meets in instruction i. The blocks after
// those compute the components' constants.
template <typename T>
__global__ void __launch_bounds__(256) gate_features_kernel(const ExpertArgs p) {
  constexpr int P = Frag<T>::kPer, kStep = 4 * P, U = 4, NW = 4;
  __shared__ double red[NW][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int tiles_j = (p.d + 15) / 16, tiles_t = (p.T + 15) / 16;
  if (blockIdx.x >= tiles_j * tiles_t * kGateParts) {
    gate_constants(p, blockIdx.x - tiles_j * tiles_t * kGateParts);
    return;
  }
  const int z = blockIdx.x / (tiles_j * tiles_t), in = blockIdx.x - z * tiles_j * tiles_t;
  const int j0 = in % tiles_j * 16, t0 = in / tiles_j * 16;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.count[kRowsDone] = 0;
  const T* w = static_cast<const T*>(p.proj) + (int64_t)min(j0 + r, p.d - 1) * p.D + g * P;
  const T* x = static_cast<const T*>(p.X) + (int64_t)min(t0 + r, p.T - 1) * p.D + g * P;
  const int steps = (p.D + kStep - 1) / kStep, per = (steps + NW * kGateParts - 1) / (NW * kGateParts);
  const int s0 = (z * NW + wave) * per, s1 = min(steps, s0 + per);
  f64x4 acc = {0., 0., 0., 0.};
  for (int s = s0; s < s1; s += U) {
    union V {
      u32x4 v;
      T e[P];
    } a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int left = s + u < s1 ? p.D - (s + u) * kStep - g * P : 0;
      a[u].v = load_frag<T>(w + (s + u) * kStep, left);
      b[u].v = load_frag<T>(x + (s + u) * kStep, left);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < P; ++i)
        acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)(float)a[u].e[i], (double)(float)b[u].e[i], acc, 0, 0, 0);
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) red[wave][r][4 * q + g] = acc[q];  // row r, feature 4 q + g
  __syncthreads();
  const int j = threadIdx.x & 15, t = threadIdx.x >> 4;
  if (j0 + j < p.d && t0 + t < p.T) {
    double f = 0.;
#pragma unroll
    for (int v = 0; v < NW; ++v) f += red[v][t][j];
    p.feats[((int64_t)z * p.T + t0 + t) * p.d + j0 + j] = f;
  }
}

// ---------------------------------------------------------------------------
// Experts' products. A block takes one expert with picks and NT * 16 rows of
// its weights, reads them once per 16 RT rows of X (or of h) picked for that
// expert, and multiplies. The waves split the contraction.
// UP: h = act(W1 x + b1), or with GLU act(gate) * up, a tile of 16 weight
// rows being 8 gate rows and their 8 up rows. Otherwise: out = W2 h.
// ---------------------------------------------------------------------------
template <typename T, int NW, int RT, int NT, bool UP, bool GLU, int ACT>
__device__ __forceinline__ void expert_rows_part(const ExpertArgs& p, const T* const* brow, int K, int e, int place0,
                                                 int rows, float (*red)[16][16 * NT + 1]) {
  constexpr int kOut = GLU ? 8 : 16, U = RT * NT > 4 ? 2 : RT + NT > 2 ? 4 : 8;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const T* arow[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int place = place0 + min(16 * t + r, rows - 1);
    arow[t] = UP ? static_cast<const T*>(p.X) + (int64_t)p.row_of[place] * K
                 : static_cast<const T*>(p.h) + (int64_t)place * K;
  }
  f32x4 acc[RT][NT];
  stream_rows<T, NW, RT, NT, U>(brow, arow, K, wave, g, acc);
  const int N = UP ? p.F : p.D, n0 = blockIdx.x * kOut * NT;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    if (16 * t >= rows) break;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) red[wave][r][16 * j + 4 * g + q] = acc[t][j][q];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * kOut * NT; i += 64 * NW) {
      const int n = i % (kOut * NT), m = i / (kOut * NT), at = n / kOut * 16 + n % kOut;  // n's place in the tiles
      if (16 * t + m >= rows || n0 + n >= N) continue;
      float z = 0.f, u = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        z += red[w][m][at];
        if (GLU) u += red[w][m][at + 8];
      }
      const int64_t place = place0 + 16 * t + m;
      if (UP) {
        const T* b1 = static_cast<const T*>(p.b1);
        const int64_t b = (int64_t)e * (GLU ? 2 * p.F : p.F) + n0 + n;
        if (b1) z += (float)b1[b];
        if (GLU && b1) u += (float)b1[b + p.F];
        z = act_value<ACT>(z);
        if (GLU) z *= u;
        // The gathering product adds a row's experts up as it goes, so their
        // weights come in here, as parts of the row's largest.
        if (p.T * p.top <= kGatherPicks) z *= p.weight[place] / p.scale[p.row_of[place]];
        // rounded to the operands' type: what the second product's matrix instruction takes
        static_cast<T*>(p.h)[place * p.F + n0 + n] = (T)z;
      } else {
        p.out[place * p.D + n0 + n] = z;
      }
    }
    __syncthreads();
  }
}

template <typename T, int NW, int RT, int NT, bool UP, bool GLU, int ACT>
__global__ void __launch_bounds__(64 * NW) expert_kernel(const ExpertArgs p) {
  __shared__ float red[NW][16][16 * NT + 1];
  const int a = blockIdx.y;
  const int count = p.count[kExperts], e = p.expert[a], first = p.first[a], rows = p.first[a + 1] - first;
  if (a >= count) return;  // all four loaded at once
  const int r = threadIdx.x & 15;
  const int K = UP ? p.D : p.F, N = UP ? (GLU ? 2 * p.F : p.F) : p.D;
  const T* brow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int tile = blockIdx.x * NT + j;
    const int n = GLU ? (r < 8 ? 0 : p.F) + min(tile * 8 + (r & 7), p.F - 1) : min(tile * 16 + r, N - 1);
    brow[j] = static_cast<const T*>(UP ? p.W1 : p.W2) + ((int64_t)e * N + n) * K;
  }
  if (RT == 1 || rows <= 16) {
    for (int i = 0; i < rows; i += 16)
      expert_rows_part<T, NW, 1, NT, UP, GLU, ACT>(p, brow, K, e, first + i, min(16, rows - i), red);
  } else {
    for (int i = 0; i < rows; i += 16 * RT)
      expert_rows_part<T, NW, RT, NT, UP, GLU, ACT>(p, brow, K, e, first + i, min(16 * RT, rows - i), red);
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
    y += p.weight[place] * o;
  }
  if (p.bad && p.bad[t]) y = NAN;
  static_cast<T*>(p.Y)[at] = (T)y;
}

// The second product and the sum over a row's experts for a few picks: the
// columns of the matrix instruction are the rows of the call, and a block runs
// `cols` columns of Y (at most 16; fewer where that fills the chip) through all
// experts with picks, one long contraction over (expert, k) that its waves
// split evenly. Every expert's part is summed by itself and added only in the
// columns of the rows that picked it: zeros in the other columns would not keep
// out what is not a number in its weights. The weights are in h already, as
// parts of the row's largest, which stands before the whole sum.
template <typename T, int NW>
__global__ void __launch_bounds__(64 * NW) expert_gather_kernel(const ExpertArgs p, int cols) {
  constexpr int P = Frag<T>::kPer, kStep = 4 * P, U = 8, kMost = kGatherPicks;
  __shared__ float red[NW][16][17];
  __shared__ int16_t at[kMost][16];  // [expert][row]: place of the row's pick, -1: none
  __shared__ int expert[kMost];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4, i = threadIdx.x;
  const int n0 = blockIdx.x * cols, count = p.count[kExperts], places = p.count[kPlaces];
  int e = 0, ord = 0, row_of = 0;
  if (i < p.T * p.top) {  // all loaded at once, whatever the counts
    e = p.expert[i];
    ord = p.ord[i];
    row_of = p.row_of[i];
  }
  if (i < kMost * 16) (&at[0][0])[i] = -1;
  __syncthreads();
  if (i < count) expert[i] = e;
  if (i < places) at[ord][row_of] = (int16_t)i;
  __syncthreads();
  const int spe = (p.F + kStep - 1) / kStep, total = count * spe, per = (total + NW - 1) / NW;
  const int t0 = wave * per, t1 = min(total, t0 + per);
  const int64_t brow = min(n0 + r % cols, p.D - 1);
  const T *W2 = static_cast<const T*>(p.W2), *h = static_cast<const T*>(p.h);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f}, sum = {0.f, 0.f, 0.f, 0.f};
  int a = t0 / spe, s = t0 - a * spe;  // the expert and the step in it
  for (int t = t0; t < t1; t += U) {
    u32x4 fb[U], fa[U];
    int place[U];
    bool last[U];  // step of the expert, or of the wave: the same for all lanes
#pragma unroll
    for (int u = 0; u < U; ++u) {
      fb[u] = fa[u] = u32x4{0, 0, 0, 0};
      place[u] = -1;
      last[u] = false;
      if (t + u < t1) {
        const int k = s * kStep + g * P;
        place[u] = at[a][r];
        fb[u] = load_frag<T>(W2 + ((int64_t)expert[a] * p.D + brow) * p.F + k, p.F - k);
        if (place[u] >= 0) fa[u] = load_frag<T>(h + (int64_t)place[u] * p.F + k, p.F - k);
        last[u] = s + 1 == spe || t + u + 1 == t1;
        if (++s == spe) {
          s = 0;
          ++a;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      acc = Frag<T>::mma(fb[u], fa[u], acc);
      if (last[u]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sum[q] += place[u] >= 0 ? acc[q] : 0.f;
          acc[q] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) red[wave][r][4 * g + q] = sum[q];
  __syncthreads();
  if (i < 256) {
    const int n = i & 15, c = n0 + n, row = i >> 4;
    if (row >= p.T || n >= cols || c >= p.D) return;
    float z = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) z += red[w][row][n];
    float y = p.scale[row] * z;
    if (p.b2)
      for (int q = row * p.top; q < (row + 1) * p.top; ++q)
        if (p.place[q] >= 0)
          y += p.weight[p.place[q]] * (float)static_cast<const T*>(p.b2)[(int64_t)p.in_idx[q] * p.D + c];
    const int64_t to = (int64_t)row * p.D + c;
    if (p.residual) y += (float)static_cast<const T*>(p.residual)[to];
    if (p.bad && p.bad[row]) y = NAN;
    static_cast<T*>(p.Y)[to] = (T)y;
  }
}

// --------------------------------------------------------------------------- launchers

hipError_t launch_gate_picks(const ExpertArgs& p, hipStream_t s);

template <typename T>
hipError_t launch_gate(const ExpertArgs& p, hipStream_t s) {
  const int blocks = (p.d + 15) / 16 * ((p.T + 15) / 16) * kGateParts + (p.K + 15) / 16;
  gate_features_kernel<T><<<blocks, 256, 0, s>>>(p);
  return launch_gate_picks(p, s);
}

// One product of all experts with picks. `rows` is the call's, at most as many
// go to one expert. Few blocks: a tile each, and more waves. Many rows and
// blocks: 4 tiles a block beside 4 tiles of rows, which reads a quarter of the
// rows' bytes (128 rows, 23 experts of 4096 x 2048: 184 and 91 us against 194
// and 99 with single tiles; 27 rows, 5 experts of 1001 x 333: 17 and 8 us
// against 11 and 6).
template <typename T, bool UP, bool GLU, int ACT>
static void launch_product_by_expert(const ExpertArgs& p, int active, hipStream_t s) {
  constexpr int kOut = GLU ? 8 : 16;
  const int tiles = ((UP ? p.F : p.D) + kOut - 1) / kOut;
  if (p.T > 16 && (int64_t)tiles * active >= 2048)
    expert_kernel<T, 4, 4, 4, UP, GLU, ACT><<<dim3((tiles + 3) / 4, active), 256, 0, s>>>(p);
  else if (p.T > 16)
    expert_kernel<T, 8, 4, 1, UP, GLU, ACT><<<dim3(tiles, active), 512, 0, s>>>(p);
  else if ((int64_t)tiles * active < 1024)
    expert_kernel<T, 8, 1, 1, UP, GLU, ACT><<<dim3(tiles, active), 512, 0, s>>>(p);
  else
    expert_kernel<T, 4, 1, 1, UP, GLU, ACT><<<dim3(tiles, active), 256, 0, s>>>(p);
}

template <typename T, int ACT>
static void launch_experts_act(const ExpertArgs& p, hipStream_t s) {
  const int n = p.T * p.top, active = n < p.K ? n : p.K;
  if (p.glu)
    launch_product_by_expert<T, true, true, ACT>(p, active, s);
  else
    launch_product_by_expert<T, true, false, ACT>(p, active, s);
  if (n <= kGatherPicks) {
    // 16 columns a block, or 8 or 4 where that leaves CUs without one
    const int cols = p.D >= 16 * 256 ? 16 : p.D >= 8 * 256 ? 8 : 4;
    expert_gather_kernel<T, 16><<<(p.D + cols - 1) / cols, 1024, 0, s>>>(p, cols);
    return;
  }
  launch_product_by_expert<T, false, false, GMM_ACT_NONE>(p, active, s);
  expert_combine_kernel<T><<<dim3((p.D + 255) / 256, p.T), 256, 0, s>>>(p);
}

template <typename T>
hipError_t launch_experts(int act, const ExpertArgs& p, hipStream_t s) {
  return with_act<T, false>(act, false, [&](auto a) {
    launch_experts_act<T, decltype(a)::value>(p, s);
    return hipGetLastError();
  });
}

#define GMM_EXPERTS_TYPE(T)                                          \
  template hipError_t launch_gate<T>(const ExpertArgs&, hipStream_t); \
  template hipError_t launch_experts<T>(int, const ExpertArgs&, hipStream_t);

}  // namespace gmm
