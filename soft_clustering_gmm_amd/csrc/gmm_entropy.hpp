// Internal declarations of the cross entropy of a linear head
// (gmm_cross_entropy, gmm_cross_entropy_gradients).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gmm_linear.hpp"

namespace gmm {

constexpr int64_t kMaxClasses = 1 << 20;
constexpr int kEntropyRange = 256;     // parts of the largest gradient of a row

// Rows of a call, or of a piece of it.
struct EntropyArgs {
  const void* X;         // [rows][d_in]
  const void* W;         // [V][d_in]
  const void* bias;      // [V] or null
  RowPicks picks;
  const float* dloss;    // [rows] or null: 1
  int64_t rows;
  int d_in, V;
  float *loss, *lse;     // [rows], lse nullable
  const float* stats;    // [rows][groups][2] of the logits' product, or null: from the logits
  int groups, columns;   // of a group
  const float* picked;   // [rows][picks.top] the picks' logits of that product, or null: from the logits
  const float* Z;        // [rows][ldz] logits, or null: not written
  void* G;               // [rows][ldz] their gradient in the operands' type; in its place
                         // before, where Z is null, the logits' exponentials over their group's largest in half
  int64_t ldz;           // a multiple of 8
  RowCoef* coef;         // [rows], or null: no gradient
  float* range;          // [kEntropyRange] and G's scale's inverse behind; null: no scale
  float* parts;          // [chunks][V] column sums of G, or null
  int64_t chunk;         // rows of a chunk
  // what EntropyPrep does otherwise, for the few rows of a call: X without the
  // rows that have no gradient, [rows][ldx], or null; the range of all rows
  void* clean;
  int64_t ldx;
  int own_range;
};
// Every wave reads all picks then (512 features to 300 classes, with a launch
// before and so: 16 rows 28.0 us and 25.7, 512 36.2 and 33.4, 1024 39.1 and 38.6,
// 2048 41.6 and 45.9; 512 rows of 8 picks 46.8 and 51.6).
constexpr int64_t kOwnPrepPicks = 512;

// Work before the products, in one launch: copies of rows of whole pieces of
// 16 bytes of X and of W (no rows: none), a copy of X with zeros for the rows
// that have no gradient, and the parts of `range` over `all_rows` rows.
struct EntropyPrep {
  const void* X;
  void *x, *clean;       // [rows][ld] each, or null
  int64_t rows;
  const void* W;
  void* w;               // [V][ld], or null
  int64_t ld;
  int64_t all_rows;      // 0: no range
  // the picks and losses of all rows, and the first row of X among them
  RowPicks picks;
  const float* dloss;
  int64_t first;
  float* range;
  int d_in, V;
};

template <typename T>
hipError_t launch_entropy_prep(const EntropyPrep& p, hipStream_t s);
// Loss, lse and coef of every row.
template <typename T>
hipError_t launch_entropy_loss(const EntropyArgs& p, hipStream_t s);
// G and its column sums from Z, or the exponentials, and coef.
template <typename T>
hipError_t launch_entropy_gradient(const EntropyArgs& p, hipStream_t s);

// `count` rows of V column sums to `most` or fewer: those of each group of
// fold_rows(count, most) added up. To one row, it may be one of them.
constexpr int kFoldedSums = 256;
inline int64_t fold_rows(int64_t count, int64_t most) { return (count + most - 1) / most; }
hipError_t launch_entropy_fold(const float* parts, int64_t count, int64_t most, int V, float* out, hipStream_t s);

}  // namespace gmm
