// Kernels of the cross entropy of a linear head beside its products,
// instantiated once per element type (gmm_entropy_f32.hip, gmm_entropy_f16.hip,
// gmm_entropy_bf16.hip).
#pragma once

#include <cfloat>
#include <type_traits>

#include "gmm_entropy.hpp"
#include "gmm_product.hpp"

namespace gmm {

// sum exp(z) as s exp(m), m the largest z: what two parts have together. m is
// -infinity where all z are, or where they are not numbers and s is none.
struct LogSum {
  float m, s;
};
__device__ __forceinline__ LogSum join(LogSum a, LogSum b) {
  constexpr float kInf = __builtin_inff();
  const float m = fmaxf(a.m, b.m);
  return {m, (a.m == -kInf ? a.s : a.s * exp_of(a.m - m)) + (b.m == -kInf ? b.s : b.s * exp_of(b.m - m))};
}

// The largest |dloss w| of a row's picks.
__device__ __forceinline__ float row_weight(const RowPicks& picks, const float* dloss, int64_t row, int V) {
  float most = 0.f;
  for (int j = 0; j < picks.top; ++j) most = fmaxf(most, fabsf(pick_of(picks, row, j, V).w));
  return most * fabsf(dloss ? dloss[row] : 1.f);
}
__device__ __forceinline__ bool has_gradient(const RowPicks& picks, const float* dloss, int64_t row, int V) {
  bool on = false;
  if (!dloss || dloss[row] != 0.f)
    for (int j = 0; j < picks.top; ++j) on |= pick_of(picks, row, j, V).w != 0.f;
  return on;
}

// ---------------------------------------------------------------------------
// Work before the products. A row has no gradient where its picks weigh nothing
// or its loss is not asked for; what is not finite in such a row of X would
// reach dW as 0 times it, so dW's product takes a copy with zeros there.
// One launch: of 1001 rows the copies, the clean rows and the range took 4 to 6
// us each in launches of their own. Of up to kOwnPrepPicks picks of rows that need
// no padded copies the loss kernel does the same beside its work.
// ---------------------------------------------------------------------------
template <typename T, int THREADS>
__device__ __forceinline__ void copy_row(const T* from, T* to, int n, int64_t ld, int t) {
  constexpr int V = Frag<T>::kPer;
  for (int64_t c = t * V; c < ld; c += THREADS * V) *reinterpret_cast<u32x4*>(to + c) = load_frag<T>(from + c, (int)(n - c));
}

template <typename T, int L>
__global__ void __launch_bounds__(256) entropy_prep_kernel(const EntropyPrep p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = threadIdx.x % L;
  int block = blockIdx.x, blocks = gridDim.x;
  if (p.all_rows) {  // the largest finite |dloss w|, in parts
    if (block < kEntropyRange) {
      __shared__ float red[4];
      float most = 0.f;
      for (int64_t row = block * 256ll + threadIdx.x; row < p.all_rows; row += kEntropyRange * 256ll) {
        const float a = row_weight(p.picks, p.dloss, row, p.V);
        if (a <= FLT_MAX) most = fmaxf(most, a);
      }
#pragma unroll
      for (int o = 32; o; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
      if (lane == 0) red[wave] = most;
      __syncthreads();
      if (threadIdx.x == 0) p.range[block] = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
      return;
    }
    block -= kEntropyRange;
    blocks -= kEntropyRange;
  }
  const int64_t jobs = p.rows + (p.w ? p.V : 0);
  constexpr int64_t kRows = 256 / L;
  for (int64_t i = block * kRows + threadIdx.x / L; i < jobs; i += blocks * kRows) {
    if (i >= p.rows) {
      const int64_t r = i - p.rows;
      copy_row<T, L>(static_cast<const T*>(p.W) + r * p.d_in, static_cast<T*>(p.w) + r * p.ld, p.d_in, p.ld, t);
      continue;
    }
    const T* x = static_cast<const T*>(p.X) + i * p.d_in;
    if (p.x) copy_row<T, L>(x, static_cast<T*>(p.x) + i * p.ld, p.d_in, p.ld, t);
    if (p.clean) {
      const bool on = has_gradient(p.picks, p.dloss, p.first + i, p.V);
      copy_row<T, L>(x, static_cast<T*>(p.clean) + i * p.ld, on ? p.d_in : 0, p.ld, t);
    }
  }
}

// The scale of G: the largest |dloss w| becomes 2^11 (no entry passes 16 times
// that, 8 picks and the probability's share of as many), and the products take it
// back. So half's range is kept, and where all picks weigh the same, as under a
// mean over labelled rows, the entries dloss (p - 1) of picks of p near 0 lie next
// to 2^11, not next to a number whose rounding all rows share: in bfloat16 the
// gradients of 8192 rows were off by 0.0029 without (1 / 7373 is 0.0024 from its
// neighbour), and are by 0.0017, as by one rounding at the end. Entries of picks
// of any p are rounded on their own besides: 0.0023 at a mean p of one half. In
// every thread of a wave.
__device__ __forceinline__ float gradient_scale(const EntropyArgs& p) {
  float most = 0.f;
  if (p.own_range) {
    for (int64_t row = threadIdx.x & 63; row < p.rows; row += 64) {
      const float a = row_weight(p.picks, p.dloss, row, p.V);
      if (a <= FLT_MAX) most = fmaxf(most, a);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kEntropyRange / 64; ++i) most = fmaxf(most, p.range[i * 64 + (threadIdx.x & 63)]);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
  most = most > 0.f ? fmaxf(most, 1e-30f) : 2048.f;  // the scale and its inverse are normal
  if (blockIdx.x == 0 && threadIdx.x == 0) p.range[kEntropyRange] = most * (1.f / 2048.f);
  return 2048.f / most;
}

// ---------------------------------------------------------------------------
// A row's loss from its log-sum, in parts from the product's tiles (`stats`) or
// from its logits, by THREADS threads:
//   loss = sum_j w_j (log s + (m - z_j)),  lse = m + log s
// z_j is the logit that m and s were taken of, and m - z_j is formed first: both
// terms are at least 0, and a loss near 0 is as exact as the logits' differences,
// down to the half rounding of s next to 1. (With z_j as a sum of its own, in
// another order than the product's, a third of the losses of rows that are sure
// of their pick came out below 0, by 1e-5 to 1e-4.) Latency bounds it, so few
// rows take more threads each.
// ---------------------------------------------------------------------------
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS > 256 ? THREADS : 256) entropy_loss_kernel(const EntropyArgs p) {
  constexpr float kInf = __builtin_inff();
  constexpr int kThreads = THREADS > 256 ? THREADS : 256, kRows = kThreads / THREADS, kWaves = (THREADS + 63) / 64;
  __shared__ LogSum red[kWaves];
  const int t = threadIdx.x % THREADS, lane = threadIdx.x & 63;
  const float scale = p.coef && p.range ? gradient_scale(p) : 1.f;
  const int64_t row = blockIdx.x * (int64_t)kRows + threadIdx.x / THREADS;
  if (row >= p.rows) return;  // whole rows, and only where no barrier follows
  if (p.clean)
    copy_row<T, THREADS>(static_cast<const T*>(p.X) + row * p.d_in, static_cast<T*>(p.clean) + row * p.ldx,
                         has_gradient(p.picks, p.dloss, row, p.V) ? p.d_in : 0, p.ldx, t);
  const float* z = p.Z ? p.Z + row * p.ldz : nullptr;
  LogSum sum{-kInf, 0.f};
  if (p.stats) {
    const float* st = p.stats + row * p.groups * 2;
#pragma unroll 4
    for (int i = t; i < p.groups; i += THREADS) sum = join(sum, LogSum{st[2 * i], st[2 * i + 1]});
  } else {
#pragma unroll 4
    for (int col = t * 4; col < p.V; col += THREADS * 4) {
      float v[4], m = -kInf, s = 0.f;
      load_as<float, 4>(z + col, 4, v);  // a row's memory is whole pieces
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (col + i >= p.V) v[i] = -kInf;
        m = fmaxf(m, v[i]);
      }
      const float base = m == -kInf ? 0.f : m;
#pragma unroll
      for (int i = 0; i < 4; ++i) s += exp_of(v[i] - base);
      sum = join(sum, LogSum{m, s});
    }
  }
  constexpr int kLanes = THREADS < 64 ? THREADS : 64;  // of a row in a wave
#pragma unroll
  for (int o = kLanes / 2; o; o >>= 1) sum = join(sum, LogSum{__shfl_xor(sum.m, o), __shfl_xor(sum.s, o)});
  if constexpr (THREADS > 64) {
    if (lane == 0) red[threadIdx.x / 64] = sum;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    sum = red[0];
    for (int w = 1; w < kWaves; ++w) sum = join(sum, red[w]);
  }
  // one wave goes on, or the row's part of one
  const float log_sum = logf(sum.s);
  float loss = 0.f, share = 0.f;
  RowCoef c{};
  c.v0 = c.v1 = -1;
  for (int j = 0; j < p.picks.top; ++j) {
    const Pick k = pick_of(p.picks, row, j, p.V);
    if (k.w == 0.f) continue;  // the same for the row
    const float of = p.picked ? p.picked[row * p.picks.top + j] : z[k.v];
    share += k.w;
    if (c.v0 < 0 || c.v0 == k.v)
      c.v0 = k.v, c.c0 += k.w;
    else if (c.v1 < 0 || c.v1 == k.v)
      c.v1 = k.v, c.c1 += k.w;
    else
      c.all = 1;
    loss = fmaf(k.w, log_sum + (sum.m - of), loss);
  }
  if (t == 0) {
    p.loss[row] = loss;
    if (p.lse) p.lse[row] = sum.m == -kInf ? sum.s == 0.f ? -kInf : sum.s : sum.m + log_sum;
    if (p.coef) {
      c.d = c.v0 >= 0 ? (p.dloss ? p.dloss[row] : 1.f) * scale : 0.f;
      c.base = sum.m == -kInf ? 0.f : sum.m;
      c.up = c.d * share / sum.s;
      c.c0 *= c.d;
      c.c1 *= c.d;
      p.coef[row] = c;
    }
  }
}

// ---------------------------------------------------------------------------
// The logits' gradient and its column sums (of the rounded values, in float,
// without the scale). A wave takes a row's columns of its block, 16 bytes of G a
// lane, so what belongs to the row is scalar; a block takes a chunk of rows.
// HBM bounds it. GROUPED: 2-byte operands' logits lie in G's place as exp(z - the
// largest z of their row and group of columns), in half: a probability is off by
// 2^-11 of itself, no more than G's rounding puts it off by, and below 2^-29 of the
// largest of its group by 2^-40 of that (8192 x 65536: 394 us, 5.4 TB/s; from
// floats 600, which the product took 240 us more to write).
// ---------------------------------------------------------------------------
template <typename T, bool GROUPED>
__global__ void __launch_bounds__(256) entropy_gradient_kernel(const EntropyArgs p, int across) {
  constexpr int V = Frag<T>::kPer, kAhead = 4;  // rows of logits in flight
  __shared__ float red[4][64 * V];
  const int part = blockIdx.x / across, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int first = (blockIdx.x % across) * 64 * V, col = first + lane * V;
  const int64_t r0 = part * p.chunk + wave, r1 = min(p.rows, (part + 1) * p.chunk);
  const bool mine = col < p.ldz;
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.f;
  for (int64_t r = r0; r < r1; r += 4 * kAhead) {
    using E = std::conditional_t<GROUPED, _Float16, float>;
    struct {
      E e[V];
    } raw[kAhead];
    float most[kAhead], z[V];
    RowCoef c[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (r + 4 * u < r1) {
        const int64_t row = r + 4 * u;
        c[u] = p.coef[row];
        if (mine) {
          const E* from = GROUPED ? static_cast<const E*>(p.G) : reinterpret_cast<const E*>(p.Z);
          __builtin_memcpy(raw[u].e, from + row * p.ldz + col, sizeof(raw[u].e));
          if (GROUPED) most[u] = p.stats[2 * (row * p.groups + min(col, p.V - 1) / p.columns)];
        }
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t row = r + 4 * u;
      if (row >= r1) break;
      float g[V];
#pragma unroll
      for (int i = 0; i < V; ++i) z[i] = (float)raw[u].e[i];
      if (GROUPED)  // most is -infinity where all of the group are
        c[u].up = most[u] == -__builtin_inff() ? 0.f : c[u].up * exp_of(most[u] - c[u].base) * (1.f / kKeptOne);
      logit_gradient<V, GROUPED>(c[u], p.picks, row, col, p.V, z, g);
      if (mine) {
        store_as<T, V>(static_cast<T*>(p.G) + row * p.ldz + col, V, g);
        if (p.parts)
#pragma unroll
          for (int i = 0; i < V; ++i) sum[i] += (float)(T)g[i];
      }
    }
  }
  if (!p.parts) return;
#pragma unroll
  for (int i = 0; i < V; ++i) red[wave][lane * V + i] = sum[i];
  __syncthreads();
  const float unscale = p.range ? p.range[kEntropyRange] : 1.f;
  for (int i = threadIdx.x; i < 64 * V; i += 256)
    if (first + i < p.V)
      p.parts[part * (int64_t)p.V + first + i] = unscale * ((red[0][i] + red[1][i]) + (red[2][i] + red[3][i]));
}

template <typename T>
hipError_t launch_entropy_prep(const EntropyPrep& p, hipStream_t s) {
  auto go = [&](auto lanes) {
    constexpr int L = decltype(lanes)::value, kRows = 256 / L;
    const int64_t jobs = p.rows + (p.w ? p.V : 0), blocks = (jobs + kRows - 1) / kRows;
    const unsigned grid = (unsigned)(blocks < 8192 ? blocks : 8192) + (p.all_rows ? kEntropyRange : 0);
    if (grid) entropy_prep_kernel<T, L><<<grid, 256, 0, s>>>(p);
    return hipGetLastError();
  };
  // short rows share a wave (16384 x 128 in float: 6.1 us, one a wave 9.2)
  if (p.ld * sizeof(T) <= 512) return go(std::integral_constant<int, 16>{});
  return go(std::integral_constant<int, 64>{});
}

template <typename T>
hipError_t launch_entropy_loss(const EntropyArgs& p, hipStream_t s) {
  const int parts = p.stats ? p.groups : p.V / 4;
  // a wave a row where the rows fill the device (8 rows of 1024 parts: 54.1 us for the call, by 256 threads 53.4)
  const int threads = p.rows >= 1024 ? (parts <= 2048 ? 64 : 1024) : parts <= 128 ? 64 : parts <= 4096 ? 256 : 1024;
  // and four rows a wave where they are many and have little each (16384 rows of 16 parts: 21.1 us for the call, one a
  // wave 24.6)
  if (p.rows >= 4096 && parts <= 32)
    entropy_loss_kernel<T, 16><<<(unsigned)((p.rows + 15) / 16), 256, 0, s>>>(p);
  else if (threads == 64)
    entropy_loss_kernel<T, 64><<<(unsigned)((p.rows + 3) / 4), 256, 0, s>>>(p);
  else if (threads == 256)
    entropy_loss_kernel<T, 256><<<(unsigned)p.rows, 256, 0, s>>>(p);
  else
    entropy_loss_kernel<T, 1024><<<(unsigned)p.rows, 1024, 0, s>>>(p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_entropy_gradient(const EntropyArgs& p, hipStream_t s) {
  const int across = (int)((p.ldz + 64 * Frag<T>::kPer - 1) / (64 * Frag<T>::kPer));
  const int64_t chunks = (p.rows + p.chunk - 1) / p.chunk;
  const unsigned grid = (unsigned)(across * chunks);
  if constexpr (sizeof(T) == 2) {
    if (!p.Z) {
      entropy_gradient_kernel<T, true><<<grid, 256, 0, s>>>(p, across);
      return hipGetLastError();
    }
  }
  entropy_gradient_kernel<T, false><<<grid, 256, 0, s>>>(p, across);
  return hipGetLastError();
}

#define GMM_ENTROPY_TYPE(T)                                                    \
  template hipError_t launch_entropy_prep<T>(const EntropyPrep&, hipStream_t); \
  template hipError_t launch_entropy_loss<T>(const EntropyArgs&, hipStream_t); \
  template hipError_t launch_entropy_gradient<T>(const EntropyArgs&, hipStream_t);

}  // namespace gmm
