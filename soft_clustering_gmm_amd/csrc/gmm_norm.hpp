// Internal declarations of the layer norm (gmm_layer_norm, gmm_layer_norm_backward).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gmm {

struct NormArgs {
  const void* X;
  const void *gamma, *beta;  // null: 1 and 0
  int w_f32;                 // gamma, beta and their gradients are float (else Y's type)
  void* Y;
  float* stats;              // [N][2] mean and 1 / sqrt(var + eps); forward: nullable
  int64_t N;
  int D;
  float eps;
  // backward
  const void* dY;
  void* dX;                  // nullable
  void *dgamma, *dbeta;      // each nullable
  float* partial;            // [parts][2][D], where a gradient of the weights is wanted
  int parts;                 // blocks (or chunks of rows) that write partial sums
};

// A row is shared by `group` threads with `pieces` pieces of 16 bytes of X each.
struct NormShape {
  int group, pieces;
};
// Up to so many elements a thread, a backward block keeps the weights' sums of
// its rows in registers; beyond, a second kernel reads X and dY by columns.
constexpr int kNormKeep = 16;

inline NormShape norm_shape(int64_t D, int e) {
  const int v = 16 / e;
  const int64_t pieces = (D + v - 1) / v;
  for (int g : {4, 8, 16, 32})
    if (pieces <= g) return {g, 1};
  for (int c = 1; c * v <= kNormKeep; c *= 2)
    if (pieces <= 64 * c) return {64, c};
  for (int c = 1; c * v <= kNormKeep; c *= 2)
    if (pieces <= 256 * c) return {256, c};
  int c = kNormKeep / v;
  if (pieces <= 512 * c) return {512, c};
  while (pieces > 1024 * c) c *= 2;
  return {1024, c};
}
inline bool norm_keeps(NormShape s, int e) { return s.pieces * 16 / e <= kNormKeep; }

// Blocks of the backward kernel, or chunks of rows of the kernel by columns. Each
// leaves sums, so no more of them than keep HBM busy: fewer where a thread has
// two pieces or more in flight (bfloat16, 16384 x 4096: 86 us with 512 blocks, 107
// with 1024; 8192 x 8192, 512 threads a row: 97 with 256, 107 with 512), not where
// it has one (32768 x 2048: 106 with 512, 88 with 1024).
inline int norm_parts(int64_t N, int64_t D, int e) {
  const NormShape s = norm_shape(D, e);
  if (!norm_keeps(s, e)) return (int)(N < 128 ? N : 128);
  const int64_t at_once = s.group < 256 ? 256 / s.group : 1, blocks = (N + at_once - 1) / at_once;
  const int64_t most = s.group >= 512 ? 256 : s.pieces > 1 ? 512 : 1024;
  return (int)(blocks < most ? blocks : most);
}

template <typename TX, typename TY>
hipError_t launch_norm(const NormArgs& p, hipStream_t s);
template <typename TX, typename TY>
hipError_t launch_norm_backward(const NormArgs& p, hipStream_t s);

}  // namespace gmm
