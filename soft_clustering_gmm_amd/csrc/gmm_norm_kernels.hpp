// Kernels of the layer norm, instantiated for the type of X and that of Y
// (gmm_norm_f32.hip, gmm_norm_f16.hip, gmm_norm_bf16.hip).
#pragma once

#include <type_traits>

#include "gmm_norm.hpp"
#include "gmm_product.hpp"

namespace gmm {

// How the pieces of a row's threads lie: whole ones; the last one moved back to
// end with the row, so that it begins with elements that the piece before has,
// too; or the row is shorter than a piece. A part of a piece would be loaded
// element by element behind a branch, and waited for there.
enum { kWhole = 0, kMoved = 1, kTiny = 2 };

template <int W, int LIE>
struct Span {
  int at;    // first column
  int skip;  // elements that are not this thread's, from the first on
  int left;  // kTiny: elements of the row from `at` on
  __device__ __forceinline__ Span(int col, int D) {
    at = LIE == kTiny ? col : min(col, D - W);
    skip = LIE == kTiny ? 0 : col - at;
    left = D - at;
  }
  __device__ __forceinline__ bool mine(int i) const {
    return LIE == kTiny ? i < left : LIE == kWhole ? skip == 0 : i >= skip;
  }
  // The elements as they lie in memory; what loads several and then uses the
  // first waits for the first alone. kMoved: all are inside the row, mine or not;
  // else what is not mine is 0.
  template <typename E>
  __device__ __forceinline__ void load(const E* row, E* e) const {
    if constexpr (LIE == kTiny) {
#pragma unroll
      for (int i = 0; i < W; ++i) e[i] = i < left ? row[at + i] : (E)0.f;
    } else if (LIE == kMoved || skip == 0) {
      __builtin_memcpy(e, row + at, sizeof(E) * W);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) e[i] = (E)0.f;
    }
  }
  // Elements that two threads have get the same value from both. ALONE: each
  // stores its own alone, where the other may read the row once more before it
  // does (the output may lie over the input).
  template <bool ALONE, typename E>
  __device__ __forceinline__ void store(E* row, const float* v) const {
    if (LIE == kTiny)
      store_as<E, W>(row + at, left, v);
    else if (ALONE && LIE == kMoved && skip > 0) {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (mine(i)) row[at + i] = (E)v[i];
    } else if (skip < W)
      store_as<E, W>(row + at, W, v);
  }
  // Weights of the row's columns, `otherwise` where there are none.
  template <typename TY>
  __device__ __forceinline__ void weights(const void* p, int w_f32, float otherwise, float* out) const {
    if (p) {
      load_row<TY, W>(p, at, LIE == kTiny ? left : W, w_f32, out);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) out[i] = otherwise;
    }
  }
};

constexpr int norm_threads(int group) { return group > 256 ? group : 256; }

// ---------------------------------------------------------------------------
// Forward. A row stays in the registers of its G threads, as it lies in memory:
// its mean, then the sums of the deviations d and of d^2, whose mean the first
// one's rounding has left: var = (sum d^2 - (sum d)^2 / D) / D. So a row with a
// mean far from 0 loses no more than the rounding of its x. HBM bounds it: X is
// read once and Y written once (32768 x 4096 in bfloat16:
// 104 us, 5.2 TB/s). Rows of more
// than 16384 elements are read three times, the others from the caches: held,
// they would spill.
// ---------------------------------------------------------------------------
template <typename TX, typename TY, int G, int C, int LIE>
__global__ void __launch_bounds__(norm_threads(G)) norm_kernel(const NormArgs p) {
  constexpr int V = 16 / (int)sizeof(TX), kRows = norm_threads(G) / G;
  constexpr bool kKeep = C * V <= kNormKeep;  // row and weights stay in registers
  constexpr bool kAhead = kKeep && G <= 512;  // the next row is on its way while one is finished
  constexpr int kHeld = kKeep ? C : 1, kUnroll = kKeep ? C : 1;
  __shared__ float red[2][G > 64 ? G / 64 : 1][2];
  int turn = 0;
  const int t = threadIdx.x % G, D = p.D;
  const float inv = 1.f / (float)D;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = blockIdx.x * (int64_t)kRows + threadIdx.x / G;
  auto span = [&](int c) { return Span<V, LIE>((c * G + t) * V, D); };
  struct Piece {
    TX e[V];
  } x[kHeld], next[kAhead ? C : 1];
  auto piece = [&](int64_t r, int c, Piece& to) { span(c).load(static_cast<const TX*>(p.X) + r * D, to.e); };
  auto fetch = [&](int64_t r, Piece* to) {
    if (kKeep && r < p.N)
#pragma unroll
      for (int c = 0; c < kHeld; ++c) piece(r, c, to[c]);
  };
  fetch(row, x);
  float gamma[kHeld][V], beta[kHeld][V];
  auto weights = [&](int c, float* ga, float* be) {
    span(c).template weights<TY>(p.gamma, p.w_f32, 1.f, ga);
    span(c).template weights<TY>(p.beta, p.w_f32, 0.f, be);
  };
  if (kKeep)
#pragma unroll
    for (int c = 0; c < kHeld; ++c) weights(c, gamma[c], beta[c]);
  for (; row < p.N; row += step) {
    if constexpr (kAhead) fetch(row + step, next);
    float sum[2] = {0.f, 0.f};
#pragma unroll kUnroll
    for (int c = 0; c < C; ++c) {
      const int w = kKeep ? c : 0;
      const auto own = span(c);
      if (!kKeep) piece(row, c, x[0]);
#pragma unroll
      for (int i = 0; i < V; ++i) sum[0] += LIE != kMoved || own.mine(i) ? (float)x[w].e[i] : 0.f;
    }
    row_sum<G, 1>(sum, red, turn);
    const float mean = sum[0] * inv;
    sum[0] = 0.f;
#pragma unroll kUnroll
    for (int c = 0; c < C; ++c) {
      const int w = kKeep ? c : 0;
      const auto own = span(c);
      if (!kKeep) piece(row, c, x[0]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = own.mine(i) ? (float)x[w].e[i] - mean : 0.f;
        sum[0] += d;
        sum[1] = fmaf(d, d, sum[1]);
      }
    }
    row_sum<G, 2>(sum, red, turn);
    const float shift = sum[0] * inv;
    const float rstd = 1.f / sqrtf(fmaxf(fmaf(-shift, shift, sum[1] * inv), 0.f) + p.eps);
    if (p.stats && t == 0) {
      p.stats[2 * row] = mean + shift;
      p.stats[2 * row + 1] = rstd;
    }
#pragma unroll kUnroll
    for (int c = 0; c < C; ++c) {
      const int w = kKeep ? c : 0;
      if (!kKeep) {
        piece(row, c, x[0]);
        weights(c, gamma[0], beta[0]);
      }
      float out[V];
#pragma unroll
      for (int i = 0; i < V; ++i) out[i] = fmaf(((float)x[w].e[i] - mean - shift) * rstd, gamma[w][i], beta[w][i]);
      span(c).template store<!kKeep>(static_cast<TY*>(p.Y) + row * D, out);
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int c = 0; c < C; ++c) x[c] = next[c];
    } else {
      fetch(row + step, x);
    }
  }
}

// ---------------------------------------------------------------------------
// Backward. With h = (x - mean) rstd and k = dY gamma,
//   dX = rstd (k - mean(k) - h mean(k h)),  dgamma = sum dY h,  dbeta = sum dY.
// One read of X and dY (two of rows of more than 16384 elements, the second from
// the caches): a thread keeps its columns' sums over the rows that its
// block takes; they go to `partial` and are added in a fixed order. HBM bounds
// it (16384 x 2048, float X and bfloat16 dY: 60 us, 5.6 TB/s). 1024 threads have
// 128 registers each, and rows of 8193 to 16384 elements want more: gamma is read
// again, and up to 54 of the registers are kept in memory where X is float and dY
// is not or the pieces are moved (4096 x 16384: float 182 us, bfloat16 114, float
// to bfloat16 158; x 16382: 237, 170 and 265). Wider rows are read by the columns'
// kernel and then twice here (2048 x 32768: 339, 221 and 294 us).
// ---------------------------------------------------------------------------
template <typename TX, typename TY, int G, int C, int LIE>
__global__ void __launch_bounds__(norm_threads(G)) norm_backward_kernel(const NormArgs p) {
  constexpr int V = 16 / (int)sizeof(TX), kThreads = norm_threads(G), kRows = kThreads / G;
  constexpr bool kKeep = C * V <= kNormKeep;
  constexpr bool kAhead = kKeep && G <= 512;  // the next row is on its way while one is finished
  constexpr int kHeld = kKeep ? C : 1, kUnroll = kKeep ? C : 1;
  constexpr bool kGamma = kKeep && G <= 512;  // gamma, too (1024 threads have no room for it)
  __shared__ float red[2][G > 64 ? G / 64 : 1][2];
  __shared__ float sums[kKeep && kRows > 1 ? kRows : 1][kKeep && kRows > 1 ? G * C * V : 1];
  int turn = 0;
  const int t = threadIdx.x % G, group = threadIdx.x / G, D = p.D;
  const float inv = 1.f / (float)D;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = blockIdx.x * (int64_t)kRows + group;
  auto span = [&](int c) { return Span<V, LIE>((c * G + t) * V, D); };
  struct Piece {
    TX x[V];
    TY y[V];
  };
  struct Row {
    Piece e[kHeld];
    float mean, rstd;
  };
  auto piece = [&](int64_t r, int c, Piece& to) {
    span(c).load(static_cast<const TX*>(p.X) + r * D, to.x);
    span(c).load(static_cast<const TY*>(p.dY) + r * D, to.y);
  };
  auto fetch = [&](int64_t r, Row& to) {
    if (r >= p.N) return;
    if (kKeep)
#pragma unroll
      for (int c = 0; c < kHeld; ++c) piece(r, c, to.e[c]);
    to.mean = p.stats[2 * r];
    to.rstd = p.stats[2 * r + 1];
  };
  Row now, next;
  fetch(row, now);
  float gamma[kGamma ? C : 1][V], dg[kHeld][V], db[kHeld][V];
  if (kKeep)
#pragma unroll
    for (int c = 0; c < kHeld; ++c) {
      if (kGamma) span(c).template weights<TY>(p.gamma, p.w_f32, 1.f, gamma[kGamma ? c : 0]);
#pragma unroll
      for (int i = 0; i < V; ++i) dg[c][i] = db[c][i] = 0.f;
    }
  for (; row < p.N; row += step) {
    if constexpr (kAhead) fetch(row + step, next);
    float sum[2] = {0.f, 0.f};
#pragma unroll kUnroll
    for (int c = 0; c < C; ++c) {
      const int w = kKeep ? c : 0;
      const auto own = span(c);
      if (!kKeep) piece(row, c, now.e[0]);
      if (!kGamma) own.template weights<TY>(p.gamma, p.w_f32, 1.f, gamma[0]);
      // Beyond the row x is 0, and (0 - mean) rstd may be beyond float, and no number times dY's 0. 1024 threads have no
      // register left for it, and pass over such pieces (4096 x 16384, float to bfloat16: 158 us, 223 with a rstd of 0
      // there); in the others a branch costs more (16384 x 2048, float to bfloat16: 83, with it 69).
      const bool none = LIE == kWhole && own.skip;
      if (G == 1024 && none) continue;
      const float rstd = none ? 0.f : now.rstd;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // what is another's counts as 0; beyond the row dY is
        const float dy = LIE != kMoved || own.mine(i) ? (float)now.e[w].y[i] : 0.f;
        const float h = LIE == kTiny && !own.mine(i) ? 0.f : ((float)now.e[w].x[i] - now.mean) * rstd;
        if (kKeep) {
          dg[w][i] = fmaf(dy, h, dg[w][i]);
          db[w][i] += dy;
        }
        const float k = dy * gamma[kGamma ? c : 0][i];
        sum[0] += k;
        sum[1] = fmaf(k, h, sum[1]);
      }
    }
    if (p.dX) {  // the same for all threads
      row_sum<G, 2>(sum, red, turn);
      const float a = sum[0] * inv, b = sum[1] * inv;
#pragma unroll kUnroll
      for (int c = 0; c < C; ++c) {
        const int w = kKeep ? c : 0;
        const auto own = span(c);
        if (!kKeep) piece(row, c, now.e[0]);
        if (!kGamma) own.template weights<TY>(p.gamma, p.w_f32, 1.f, gamma[0]);
        float out[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float h = ((float)now.e[w].x[i] - now.mean) * now.rstd;
          out[i] = now.rstd * ((float)now.e[w].y[i] * gamma[kGamma ? c : 0][i] - fmaf(h, b, a));
        }
        own.template store<!kKeep>(static_cast<TX*>(p.dX) + row * D, out);
      }
    }
    if constexpr (kAhead)
      now = next;
    else
      fetch(row + step, now);
  }
  if constexpr (kKeep) {
    if (!p.partial) return;
    float* out = p.partial + (int64_t)blockIdx.x * 2 * D;
    if constexpr (kRows == 1) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const auto own = span(c);
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (own.mine(i)) {
            out[own.at + i] = dg[c][i];
            out[D + own.at + i] = db[c][i];
          }
      }
    } else {
#pragma unroll
      for (int both = 0; both < 2; ++both) {
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const auto own = span(c);
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (own.mine(i)) sums[group][own.at + i] = both ? db[c][i] : dg[c][i];
        }
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
void with_norm_shape(NormShape s, int D, F&& f3) {
  using std::integral_constant;
  auto f = [&](auto g, auto c) {
    if (D % V == 0) return f3(g, c, integral_constant<int, kWhole>{});
    if constexpr (decltype(g)::value == 4)
      if (D < V) return f3(g, c, integral_constant<int, kTiny>{});
    f3(g, c, integral_constant<int, kMoved>{});
  };
  auto pieces = [&](auto g, auto most) {
    constexpr int kMost = decltype(most)::value;
    if (s.pieces == 1) return f(g, integral_constant<int, 1>{});
    if constexpr (kMost >= 2)
      if (s.pieces == 2) return f(g, integral_constant<int, 2>{});
    if constexpr (kMost >= 4) f(g, integral_constant<int, 4>{});
  };
  constexpr integral_constant<int, kNormKeep / V> few{};
  if (s.group == 4) return f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  if (s.group == 8) return f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  if (s.group == 16) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  if (s.group == 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (s.group == 64) return pieces(integral_constant<int, 64>{}, few);
  if (s.group == 256) return pieces(integral_constant<int, 256>{}, few);
  if (s.group == 512) return f(integral_constant<int, 512>{}, few);
  if (s.pieces == few) return f(integral_constant<int, 1024>{}, few);
  if (s.pieces == 2 * few) return f(integral_constant<int, 1024>{}, integral_constant<int, 2 * few>{});
  f(integral_constant<int, 1024>{}, integral_constant<int, 4 * few>{});
}

template <typename TX, typename TY>
hipError_t launch_norm(const NormArgs& p, hipStream_t s) {
  constexpr int V = 16 / (int)sizeof(TX);
  const NormShape shape = norm_shape(p.D, sizeof(TX));
  with_norm_shape<V>(shape, p.D, [&](auto g, auto c, auto lie) {
    constexpr int G = decltype(g)::value, kThreads = norm_threads(G), kRows = kThreads / G;
    const int64_t blocks = (p.N + kRows - 1) / kRows, most = G == 1024 ? 512 : G == 512 ? 1024 : 2048;
    norm_kernel<TX, TY, G, decltype(c)::value, decltype(lie)::value><<<(unsigned)(blocks < most ? blocks : most), kThreads, 0, s>>>(p);
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
    with_norm_shape<V>(shape, p.D, [&](auto g, auto c, auto lie) {
      constexpr int G = decltype(g)::value;
      norm_backward_kernel<TX, TY, G, decltype(c)::value, decltype(lie)::value>
          <<<norm_parts(p.N, keeps ? p.D : 1 << 14, sizeof(TX)), norm_threads(G), 0, s>>>(p);
    });
  if (p.partial) norm_finish_kernel<TY><<<(2 * p.D + 63) / 64, 64 * kNormSlices, 0, s>>>(p);
  return hipGetLastError();
}

#define GMM_NORM_TYPES(TX, TY)                                              \
  template hipError_t launch_norm<TX, TY>(const NormArgs&, hipStream_t);    \
  template hipError_t launch_norm_backward<TX, TY>(const NormArgs&, hipStream_t);

}  // namespace gmm
