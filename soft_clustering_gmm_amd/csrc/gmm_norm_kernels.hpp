// Kernels of the layer norm, instantiated for the type of X and that of Y
// (gmm_norm_f32.hip, gmm_norm_f16.hip, gmm_norm_bf16.hip).
#pragma once

#include <type_traits>

#include "gmm_norm.hpp"
#include "gmm_product.hpp"

namespace gmm {

// The W weights from column c on; `otherwise` where there are none.
template <typename TY, int W>
__device__ __forceinline__ void load_weights(const void* p, int c, int left, int w_f32, float otherwise, float* out) {
  if (p && left > 0) {
    load_row<TY, W>(p, c, left, w_f32, out);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) out[i] = otherwise;
  }
}

constexpr int norm_threads(int group) { return group > 256 ? group : 256; }

// ---------------------------------------------------------------------------
// Forward. A row stays in the registers of its G threads: its mean, then the
// sums of the deviations d and of d^2, whose mean the first one's rounding has
// left: var = (sum d^2 - (sum d)^2 / D) / D. So a row with a mean far from 0
// loses no more than the rounding of its x. HBM bounds it: X is read once and
// Y written once.
// ---------------------------------------------------------------------------
template <typename TX, typename TY, int G, int C>
__global__ void __launch_bounds__(norm_threads(G)) norm_kernel(const NormArgs p) {
  constexpr int V = 16 / (int)sizeof(TX), kRows = norm_threads(G) / G;
  constexpr bool kKeep = C * V <= kNormKeep;  // the weights stay in registers
  __shared__ float red[2][G > 64 ? G / 64 : 1][2];
  int turn = 0;
  const int t = threadIdx.x % G, D = p.D;
  const float inv = 1.f / (float)D;
  float gamma[kKeep ? C : 1][V], beta[kKeep ? C : 1][V];
  if (kKeep)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * G + t) * V;
      load_weights<TY, V>(p.gamma, col, D - col, p.w_f32, 1.f, gamma[c]);
      load_weights<TY, V>(p.beta, col, D - col, p.w_f32, 0.f, beta[c]);
    }
  for (int64_t row = blockIdx.x * (int64_t)kRows + threadIdx.x / G; row < p.N; row += (int64_t)gridDim.x * kRows) {
    const TX* x = static_cast<const TX*>(p.X) + row * D;
    float d[C][V], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * G + t) * V;
      load_as<TX, V>(x + col, D - col, d[c]);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[0] += d[c][i];
    }
    row_sum<G, 1>(sum, red, turn);
    float mean = sum[0] * inv;
    sum[0] = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        d[c][i] = (c * G + t) * V + i < D ? d[c][i] - mean : 0.f;
        sum[0] += d[c][i];
        sum[1] = fmaf(d[c][i], d[c][i], sum[1]);
      }
    row_sum<G, 2>(sum, red, turn);
    const float shift = sum[0] * inv;
    const float rstd = 1.f / sqrtf(fmaxf(fmaf(-shift, shift, sum[1] * inv), 0.f) + p.eps);
    if (p.stats && t == 0) {
      p.stats[2 * row] = mean + shift;
      p.stats[2 * row + 1] = rstd;
    }
    TY* y = static_cast<TY*>(p.Y) + row * D;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * G + t) * V;
      if (!kKeep) {
        load_weights<TY, V>(p.gamma, col, D - col, p.w_f32, 1.f, gamma[0]);
        load_weights<TY, V>(p.beta, col, D - col, p.w_f32, 0.f, beta[0]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        d[c][i] = fmaf((d[c][i] - shift) * rstd, gamma[kKeep ? c : 0][i], beta[kKeep ? c : 0][i]);
      store_as<TY, V>(y + col, D - col, d[c]);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward. With h = (x - mean) rstd and k = dY gamma,
//   dX = rstd (k - mean(k) - h mean(k h)),  dgamma = sum dY h,  dbeta = sum dY.
// One read of X and dY: a thread keeps its columns' sums over the rows that its
// block takes; they go to `partial` and are added in a fixed order.
// ---------------------------------------------------------------------------
template <typename TX, typename TY, int G, int C>
__global__ void __launch_bounds__(norm_threads(G)) norm_backward_kernel(const NormArgs p) {
  constexpr int V = 16 / (int)sizeof(TX), kThreads = norm_threads(G), kRows = kThreads / G;
  constexpr bool kKeep = C * V <= kNormKeep;
  __shared__ float red[2][G > 64 ? G / 64 : 1][2];
  __shared__ float sums[kKeep && kRows > 1 ? kRows : 1][kKeep && kRows > 1 ? G * C * V : 1];
  int turn = 0;
  const int t = threadIdx.x % G, group = threadIdx.x / G, D = p.D;
  const float inv = 1.f / (float)D;
  float gamma[kKeep ? C : 1][V], dg[kKeep ? C : 1][V], db[kKeep ? C : 1][V];
  if (kKeep)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * G + t) * V;
      load_weights<TY, V>(p.gamma, col, D - col, p.w_f32, 1.f, gamma[c]);
#pragma unroll
      for (int i = 0; i < V; ++i) dg[c][i] = db[c][i] = 0.f;
    }
  for (int64_t row = blockIdx.x * (int64_t)kRows + group; row < p.N; row += (int64_t)gridDim.x * kRows) {
    const TX* x = static_cast<const TX*>(p.X) + row * D;
    const TY* dy = static_cast<const TY*>(p.dY) + row * D;
    const float mean = p.stats[2 * row], rstd = p.stats[2 * row + 1];
    float h[C][V], k[C][V], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * G + t) * V;
      load_as<TX, V>(x + col, D - col, h[c]);
      load_as<TY, V>(dy + col, D - col, k[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * G + t) * V;
      if (!kKeep) load_weights<TY, V>(p.gamma, col, D - col, p.w_f32, 1.f, gamma[0]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        h[c][i] = (h[c][i] - mean) * rstd;
        if (kKeep && col + i < D) {  // beyond the row dY is 0, h need not be finite
          dg[c][i] = fmaf(k[c][i], h[c][i], dg[c][i]);
          db[c][i] += k[c][i];
        }
        if (col + i >= D) h[c][i] = 0.f;
        k[c][i] *= gamma[kKeep ? c : 0][i];
        sum[0] += k[c][i];
        sum[1] = fmaf(k[c][i], h[c][i], sum[1]);
      }
    }
    if (!p.dX) continue;  // the same for all threads
    row_sum<G, 2>(sum, red, turn);
    const float a = sum[0] * inv, b = sum[1] * inv;
    TX* dx = static_cast<TX*>(p.dX) + row * D;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = (c * G + t) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) k[c][i] = rstd * (k[c][i] - fmaf(h[c][i], b, a));
      store_as<TX, V>(dx + col, D - col, k[c]);
    }
  }
  if constexpr (kKeep) {
    if (!p.partial) return;
    float* out = p.partial + (int64_t)blockIdx.x * 2 * D;
    if constexpr (kRows == 1) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int col = (c * G + t) * V;
        store_as<float, V>(out + col, D - col, dg[c]);
        store_as<float, V>(out + D + col, D - col, db[c]);
      }
    } else {
#pragma unroll
      for (int both = 0; both < 2; ++both) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int i = 0; i < V; ++i) sums[group][(c * G + t) * V + i] = both ? db[c][i] : dg[c][i];
        __syncthreads();
        for (int col = threadIdx.x; col < D; col += kThreads) {
          float s = 0.f;
#pragma unroll
          for (int g = 0; g < kRows; ++g) s += sums[g][col];
          out[both * D + col] = s;
        }
      }
    }
  }
}

// The weights' sums of wide rows: a block takes 64 pieces of columns and a
// chunk of rows, 4 of them at a time.
template <typename TX, typename TY>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormArgs p, int across, int64_t chunk) {
  constexpr int V = 16 / (int)sizeof(TX);
  __shared__ float red[2][4][64 * V];
  const int part = blockIdx.x / across, t = threadIdx.x % 64, group = threadIdx.x / 64, D = p.D;
  const int col = ((blockIdx.x % across) * 64 + t) * V;
  const int64_t r1 = min(p.N, (part + 1) * chunk);
  float dg[V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) dg[i] = db[i] = 0.f;
  if (col < D)
#pragma unroll 4
    for (int64_t r = part * chunk + group; r < r1; r += 4) {
      float x[V], k[V];
      load_as<TX, V>(static_cast<const TX*>(p.X) + r * D + col, D - col, x);
      load_as<TY, V>(static_cast<const TY*>(p.dY) + r * D + col, D - col, k);
      const float mean = p.stats[2 * r], rstd = p.stats[2 * r + 1];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dg[i] = fmaf(k[i], (x[i] - mean) * rstd, dg[i]);
        db[i] += k[i];
      }
    }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    red[0][group][t * V + i] = dg[i];
    red[1][group][t * V + i] = db[i];
  }
  __syncthreads();
  float* out = p.partial + (int64_t)part * 2 * D;
  for (int i = threadIdx.x; i < 2 * 64 * V; i += 256) {
    const int both = i / (64 * V), j = i % (64 * V), c = (blockIdx.x % across) * 64 * V + j;
    if (c < D) out[(int64_t)both * D + c] = (red[both][0][j] + red[both][1][j]) + (red[both][2][j] + red[both][3][j]);
  }
}

// dgamma and dbeta from the parts, 64 columns a block.
constexpr int kNormSlices = 16;
template <typename TY>
__global__ void __launch_bounds__(64 * kNormSlices) norm_finish_kernel(const NormArgs p) {
  __shared__ float red[kNormSlices][64];
  const int t = threadIdx.x % 64, slice = threadIdx.x / 64;
  const int64_t col = blockIdx.x * 64ll + t, width = 2ll * p.D;
  float sum = 0.f;
  if (col < width)
#pragma unroll 8
    for (int i = slice; i < p.parts; i += kNormSlices) sum += p.partial[i * width + col];
  red[slice][t] = sum;
  __syncthreads();
  if (slice == 0 && col < width) {
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kNormSlices; ++i) sum += red[i][t];
    void* out = col < p.D ? p.dgamma : p.dbeta;
    if (out) store_row<TY, 1>(out, col < p.D ? col : col - p.D, 1, p.w_f32, &sum);
  }
}

// f with the row shape's group and pieces as constants.
template <int V, typename F>
void with_norm_shape(NormShape s, F&& f) {
  using std::integral_constant;
  auto pieces = [&](auto g, auto most) {
    constexpr int kMost = decltype(most)::value;
    if (s.pieces == 1) return f(g, integral_constant<int, 1>{});
    if constexpr (kMost >= 2)
      if (s.pieces == 2) return f(g, integral_constant<int, 2>{});
    if constexpr (kMost >= 4)
      if (s.pieces == 4) return f(g, integral_constant<int, 4>{});
    if constexpr (kMost >= 8)
      if (s.pieces == 8) return f(g, integral_constant<int, 8>{});
    if constexpr (kMost >= 16) return f(g, integral_constant<int, 16>{});
  };
  constexpr integral_constant<int, kNormKeep / V> few{};
  if (s.group == 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (s.group == 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (s.group == 64) return pieces(integral_constant<int, 64>{}, few);
  if (s.group == 256) return pieces(integral_constant<int, 256>{}, few);
  pieces(integral_constant<int, 1024>{}, integral_constant<int, 64 / V>{});
}

template <typename TX, typename TY>
hipError_t launch_norm(const NormArgs& p, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(TX);
  const NormShape shape = norm_shape(p.D, sizeof(TX));
  with_norm_shape<V>(shape, [&](auto g, auto c) {
    constexpr int G = decltype(g)::value, kThreads = norm_threads(G), kRows = kThreads / G;
    const int64_t blocks = (p.N + kRows - 1) / kRows, most = G == 1024 ? 512 : 2048;
    norm_kernel<TX, TY, G, decltype(c)::value><<<(unsigned)(blocks < most ? blocks : most), kThreads, 0, s>>>(p);
  });
  return hipGetLastError();
}

template <typename TX, typename TY>
hipError_t launch_norm_backward(const NormArgs& p, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(TX);
  const NormShape shape = norm_shape(p.D, sizeof(TX));
  const bool keeps = norm_keeps(shape, sizeof(TX));
  if (p.partial && !keeps) {  // before dX, which may be dY
    const int across = (p.D + 64 * V - 1) / (64 * V);
    norm_columns_kernel<TX, TY><<<across * p.parts, 256, 0, s>>>(p, across, (p.N + p.parts - 1) / p.parts);
  }
  if (p.dX || (p.partial && keeps))
    with_norm_shape<V>(shape, [&](auto g, auto c) {
      constexpr int G = decltype(g)::value;
      norm_backward_kernel<TX, TY, G, decltype(c)::value>
          <<<norm_parts(p.N, keeps ? p.D : 1 << 14, sizeof(TX)), norm_threads(G), 0, s>>>(p);
    });
  if (p.partial) norm_finish_kernel<TY><<<(2 * p.D + 63) / 64, 64 * kNormSlices, 0, s>>>(p);
  return hipGetLastError();
}

#define GMM_NORM_TYPES(TX, TY)                                              \
  template hipError_t launch_norm<TX, TY>(const NormArgs&, hipStream_t);    \
  template hipError_t launch_norm_backward<TX, TY>(const NormArgs&, hipStream_t);

}  // namespace gmm
