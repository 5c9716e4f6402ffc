// Host helpers that the entry points of the layers share: argument checks,
// sizes, and the choice of a product's tiles.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "../../include/gmm.h"
#include "gmm_linear.hpp"

namespace gmm {

constexpr int kMaxWidth = 65536;       // d_in, d_out, width, hidden
constexpr int64_t kMaxRows = 1 << 30;  // rows of a call

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int hip_status(hipError_t e) { return e == hipSuccess ? GMM_OK : GMM_EHIP; }
inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
inline int elem_size(int t) { return t == GMM_F32 ? 4 : 2; }
inline bool dtype_ok(int t) { return t == GMM_F32 || t == GMM_F16 || t == GMM_BF16; }
inline bool act_ok(int a) { return a >= GMM_ACT_NONE && a <= GMM_ACT_SILU; }
// Elements of a row rounded up to whole 16-byte pieces.
inline int64_t row_len(int64_t n, int e) { return ceil_div(n, 16 / e) * (16 / e); }

template <typename F>
int with_type(int t, F&& f) {
  if (t == GMM_F16) return f((_Float16*)nullptr);
  if (t == GMM_BF16) return f((__bf16*)nullptr);
  return f((float*)nullptr);
}

// Tile variant and split of the contraction for an M x N x K product: the
// least of a time model, whose us per step were fitted to measurements on an
// MI355X (2-byte elements: 256-row tiles 1263 TFLOP/s at 8192 x 16384 x 4096
// against 1075 with 128-row tiles; 128-row tiles 26.6 us at 2048^3 against 29.9
// with 64-row and 52.9 with 256-row ones; single precision: 128-row tiles 80 us
// at 4096 x 1024 x 1024 against 86 and 104).
struct Cut {
  int variant, splits;
  int64_t split_k;
};

inline Cut choose_cut(int64_t M, int64_t N, int64_t K, int e, int64_t most_parts = 256) {
  struct Rate {
    int per_cu;         // blocks that a CU holds
    double one, full;   // us of a step with one block on a CU, and with all
  };
  static const Rate kRates[2][kTileVariants] = {{{1, 1.7, 1.7}, {2, 0.7, 1.02}, {4, 0.5, 0.82}},
                                                {{1, 7.5, 7.5}, {2, 2.4, 3.8}, {4, 0.8, 2.6}}};
  constexpr int kCus = 256;
  constexpr double kFixedUs = 3., kReduceUs = 3., kBytesPerUs = 3e6;
  const int64_t step = kStepBytes / e, steps = std::max<int64_t>(ceil_div(K, step), 1);
  Cut best{};
  double best_us = 1e30;
  for (int v = 0; v < kTileVariants; ++v) {
    const Rate& r = kRates[e == 4][v];
    const int64_t tiles = ceil_div(M, kTileRows[v]) * ceil_div(N, kTileRows[v]);
    for (int64_t want = 1; want <= std::min<int64_t>(steps, most_parts); want *= 2) {
      const int64_t per = ceil_div(steps, want), parts = ceil_div(steps, per);
      const double moved = parts > 1 ? 8. * parts * M * N : 0.;  // partial sums, written and read
      if (moved > 2e9) break;
      const int64_t blocks = tiles * parts, rounds = blocks / (kCus * r.per_cu), rest = blocks % (kCus * r.per_cu);
      double us = rounds * (per * r.full + kFixedUs);
      if (rest) {
        const int64_t on_cu = ceil_div(rest, kCus);
        const double share = r.per_cu > 1 ? double(on_cu - 1) / (r.per_cu - 1) : 0.;
        us += per * (r.one + share * (r.full - r.one)) + kFixedUs;
      }
      if (parts > 1) us += kReduceUs + moved / kBytesPerUs;
      if (us < best_us) {
        best_us = us;
        best = Cut{v, (int)parts, per * step};
      }
    }
  }
  return best;
}

inline size_t partial_bytes(const Cut& c, int64_t M, int64_t N) {
  return c.splits > 1 ? (size_t)c.splits * M * N * sizeof(float) : 0;
}

inline void set_cut(ProductArgs& p, const Cut& c) {
  p.tiles_m = (int)ceil_div(p.M, kTileRows[c.variant]);
  p.tiles_n = (int)ceil_div(p.N, kTileRows[c.variant]);
  p.splits = c.splits;
  p.split_k = c.split_k;
}

template <typename T>
hipError_t run_product(const Cut& c, bool as, bool bs, int act, ProductArgs& p, hipStream_t s, bool stream = true) {
  set_cut(p, c);
  p.c_stream = stream && p.M * p.N * (p.c_f32 ? 4 : (int64_t)sizeof(T)) >= kStreamBytes;
  hipError_t e = launch_product<T>(c.variant, as, bs, act, p, s);
  p.sum_blocks = 0;  // once
  if (e == hipSuccess && c.splits > 1) e = launch_reduce<T>(act, p, s);
  return e;
}

inline int check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return GMM_OK;
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0 || have < need) return GMM_EWORKSPACE;
  return GMM_OK;
}

}  // namespace gmm
