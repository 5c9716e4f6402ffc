// Internal declarations of the linear layer (gmm_linear, gmm_linear_backward).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gmm {

// One product C[m][n] = sum_k A(m, k) B(n, k) on 16-byte aligned operands.
// An operand is "k-contiguous" (element (r, k) at p[r * ld + k]) or
// "k-strided" (element (r, k) at p[k * ld + r]); ld * element size is a
// multiple of 16. Elements of a k-contiguous operand between K and the next
// multiple of 16 bytes are zero.
struct ProductArgs {
  const void* A;
  const void* B;
  int64_t lda, ldb;
  int64_t M, K;
  int N;
  int tiles_m, tiles_n;  // output tiles of this launch
  int splits;            // parts of the contraction (> 1: partial sums in `partial`)
  int64_t split_k;       // k per part, a multiple of the k step
  // epilogue (splits == 1): C = act(z + bias) + residual; pre receives z + bias
  const void* bias;      // element type of the operands
  const void* residual;  // type of C
  void* C;
  void* pre;             // type of C
  int c_f32;             // C, residual and pre are float (else the operands' type)
  int c_stream;          // C is written past the caches (kStreamBytes)
  float* partial;        // [splits][M][N]
  // column sums that ride along in blocks of their own (sum_blocks of them, 0:
  // none): sums_out[c] = sum over sums_rows rows of sums[.][c]
  const float* sums;
  void* sums_out;        // type of the operands
  int64_t sums_rows;
  int sums_cols, sum_blocks;
  const float* unscale;  // C = *unscale times the product, where not null (gradients of half operands)
};
constexpr int kSumCols = 16;  // columns of such a block

// Outputs from this size on are written past the caches, a quarter of whose last
// level they would fill (100 MB, the product of 262144 x 1024 rows to 96 float
// columns: 135 us against 139; 268 MB, 8192 x 4096 to 16384: 909 against 913; a
// training step of 2 MB outputs, which the next call finds there: 42 against 40).
constexpr int64_t kStreamBytes = 64ll << 20;

// Tile variants of the product kernel.
enum { kTile256 = 0, kTile128 = 1, kTile64 = 2, kTileVariants = 3 };
constexpr int kTileRows[kTileVariants] = {256, 128, 64};
constexpr int kStepBytes = 128;  // bytes of k per step and operand row

// Few rows: C[m][n] of at most kFewRows rows, operands of any alignment,
// B (the weights) streamed once (bfloat16, 8192 x 16384 weights: 16 rows 49 us
// by this stream; 17 to 64 rows, with the rows of A 4 tiles deep, 82 to 146, by
// the tiled product 46 to 56).
constexpr int kFewRows = 16;

struct FewArgs {
  const void* A;  // [M][K]
  const void* B;  // [N][K]
  int M, N, K;
  const void* bias;
  const void* residual;
  void* C;
  void* pre;
  int c_f32;
};

template <typename T>
hipError_t launch_product(int variant, bool a_strided, bool b_strided, int act, const ProductArgs& p, hipStream_t s);
template <typename T>
hipError_t launch_few(int act, const FewArgs& p, hipStream_t s);
// Rows of `cols` elements copied to rows of `ld` elements, zeros behind (no
// rows: nothing).
struct PadJob {
  const void* src;
  void* dst;
  int64_t rows, ld;
  int cols;
};
template <typename T>
hipError_t launch_pad(const PadJob& a, const PadJob& b, hipStream_t s);
template <typename T>
hipError_t launch_zero(T* p, int64_t n, hipStream_t s);
// Sum of the parts, then the epilogue of ProductArgs.
template <typename T>
hipError_t launch_reduce(int act, const ProductArgs& p, hipStream_t s);
// dZ = dY act'(pre) in the operands' type, rows of ldz elements (zeros
// behind), and per-chunk column sums of the unrounded dZ in db_part; dZ or
// db_part may be null. The two copies run in the same launch. Where `range` is
// not null (launch_dz_range has filled it), dZ is scaled by a power of two and
// *unscale receives its inverse.
template <typename T>
hipError_t launch_dz(int act, const void* dY, const void* pre, int y_f32, int64_t rows, int cols, T* dZ, int64_t ldz,
                     float* db_part, int64_t chunk_rows, const PadJob& px, const PadJob& pw, const float* range,
                     float* unscale, hipStream_t s);
// range[0..kRangeBlocks): their largest is the largest finite |dY act'(pre)|.
constexpr int kRangeBlocks = 256;
template <typename T>
hipError_t launch_dz_range(int act, const float* dY, const float* pre, int64_t n, float* range, hipStream_t s);
// The column sums of `p` alone.
template <typename T>
hipError_t launch_column_sums(const ProductArgs& p, hipStream_t s);

}  // namespace gmm
