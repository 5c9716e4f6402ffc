// C-ABI of a training step around the mixture: the layer norm, the cross entropy
// of a linear head and the AdamW step. Argument checks, workspace planning and dispatch; every check runs on
// the host before anything is enqueued.
#include "../../include/gmm.h"

#include <float.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "gmm_adamw.hpp"
#include "gmm_entropy.hpp"
#include "gmm_layers.hpp"
#include "gmm_norm.hpp"

namespace gmm {

static int check_norm(int64_t N, int32_t D, int32_t x_dtype, int32_t y_dtype, int32_t w_dtype) {
  if (!dtype_ok(x_dtype) || !dtype_ok(y_dtype) || (y_dtype != x_dtype && x_dtype != GMM_F32)) return GMM_EINVAL;
  if (w_dtype != y_dtype && w_dtype != GMM_F32) return GMM_EINVAL;
  if (N < 0 || D < 1) return GMM_EINVAL;
  if (D > kMaxWidth || N > kMaxRows) return GMM_EUNSUPPORTED;
  return GMM_OK;
}

// f with the types of X and Y.
template <typename F>
static int with_norm_types(int x_dtype, int y_dtype, F&& f) {
  return with_type(y_dtype, [&](auto* ty) {
    using TY = std::remove_pointer_t<decltype(ty)>;
    if constexpr (!std::is_same<TY, float>::value)
      if (x_dtype != GMM_F32) return hip_status(f((TY*)nullptr, (TY*)nullptr));
    return hip_status(f((float*)nullptr, (TY*)nullptr));
  });
}

static size_t norm_bytes(int64_t N, int D, int e) {
  return align_up((size_t)norm_parts(N, D, e) * 2 * D * sizeof(float), 256);
}

static bool factor_ok(double beta) { return beta >= 0. && beta < 1.; }
// A size that is a finite float, too.
static bool size_ok(double x) { return x >= 0. && x <= (double)FLT_MAX; }

// The rows of a piece: what the call keeps of a row (`bytes`) within `most`, in
// whole tiles.
static int64_t piece_rows(int64_t N, int64_t bytes, int64_t most) {
  const int64_t rows = std::max<int64_t>(most / bytes / 256 * 256, 256);
  return std::min(N, std::min<int64_t>(rows, 1 << 20));
}
constexpr int64_t kStatPiece = 256ll << 20;   // bytes of a piece's statistics
// Bytes of a piece's logits, were they float: dW is read and written once for
// each (8192 x 2048 to 65536 classes: 5815 us in one piece, 6543 in four, 7617 in
// eight).
constexpr int64_t kLogitPiece = 2048ll << 20;

// Workspace of the loss: [padded rows of X of a piece] [padded W] [statistics]
// [the picks' logits].
struct EntropyPlan {
  bool few, pad;
  int64_t lx, piece;
  int groups;
  Cut cut;
  size_t o_x, o_w, o_stats, o_picked, bytes;
};

static EntropyPlan entropy_plan(int64_t N, int d_in, int V, int e) {
  EntropyPlan l{};
  l.few = N <= kFewRows;
  l.lx = row_len(d_in, e);
  l.pad = l.lx != d_in && !l.few;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  if (l.few) {
    l.piece = N;
    l.groups = (int)ceil_div(V, 16 * few_tiles((int)N, V));
  } else {
    l.piece = piece_rows(N, ceil_div(V, 32) * 8, kStatPiece);
    l.cut = choose_cut(l.piece, V, d_in, e, 1);
    l.groups = stat_groups(l.cut.variant, e, V);
  }
  l.o_x = take(l.pad ? (size_t)l.piece * l.lx * e : 0);
  l.o_w = take(l.pad ? (size_t)V * l.lx * e : 0);
  l.o_stats = take((size_t)l.piece * l.groups * 2 * sizeof(float));
  l.o_picked = take((size_t)l.piece * kMaxPicksRow * sizeof(float));
  l.bytes = off;
  return l;
}

// Up to so many features, and where the logits are more than the caches keep at
// hand, they are computed twice, once for the loss and once for their gradient,
// and not written to memory (8192 rows to 32768 classes in bfloat16, against
// once: 64 features 726 us and 753, 96 755 and 747, 256 912 and 881; to 8192 in
// float: 64 features 433 and 440, 128 669 and 608; 4096 rows to 4096 classes in
// bfloat16, 64 MiB of float: 64 features 74 and 75; 8192 to 1024 in float, 32 MiB:
// 84 and 79).
constexpr int kTwice = 64;
constexpr int64_t kTwiceBytes = 32ll << 20;

// Workspace of the gradients, for a piece of rows: [padded X] [X without the
// rows that have no gradient] [padded W] [logits] [their gradient] [statistics]
// [the picks' logits] [coefficients] [dW so far] [partial sums of the products]
// [column sums of the tiles] [column sums, those of the pieces before first]
// [range and scale].
struct EntropyBackPlan {
  bool few, pad;
  bool twice;  // the logits are computed twice and not written
  int64_t lx, ldz, piece, chunk;
  size_t o_x, o_clean, o_w, o_z, o_g, o_stats, o_picked, o_coef, o_acc, o_part, o_fold, o_db, o_range, bytes;

  // Rows of column sums that a piece finds of those before.
  int64_t carries(int64_t N) const { return piece < N ? 1 : 0; }
  // Tiles of the logits' product: whole sums where it is not written.
  Cut logits(int64_t rows, int V, int d_in, int e) const { return choose_cut(rows, V, d_in, e, twice ? 1 : 256); }
  // Whether they are kept as exponentials over their group's largest, in half, in the place of their gradient.
  bool kept(int64_t rows, int V, int d_in, int e) const {
    return !few && !twice && e == 2 && logits(rows, V, d_in, e).splits == 1;
  }
  // Sums of a column that a piece's gradient leaves, and what is kept of them: those of many tiles are added up first.
  int64_t tile_sums(int64_t rows, int V, int d_in, int e) const {
    return twice ? 2 * ceil_div(rows, kTileRows[logits(rows, V, d_in, e).variant]) : ceil_div(rows, chunk);
  }
  bool folds(int64_t rows, int V, int d_in, int e) const { return twice && tile_sums(rows, V, d_in, e) > kFoldedSums; }
  int64_t sums(int64_t rows, int V, int d_in, int e) const {
    const int64_t n = tile_sums(rows, V, d_in, e);
    return folds(rows, V, d_in, e) ? ceil_div(n, fold_rows(n, kFoldedSums)) : n;
  }
};

static EntropyBackPlan entropy_back_plan(int64_t N, int d_in, int V, int e) {
  EntropyBackPlan l{};
  l.few = N <= kFewRows;
  l.lx = row_len(d_in, e);
  l.pad = l.lx != d_in;
  l.ldz = ceil_div(V, 8) * 8;
  l.piece = piece_rows(N, l.ldz * (int64_t)sizeof(float), kLogitPiece);
  l.twice = !l.few && d_in <= kTwice && l.piece * l.ldz * (int64_t)sizeof(float) > kTwiceBytes;
  // Rows of a block that has columns of G: 16 at least (of 1001 rows and 7777 classes in half 64 make a block a CU, and
  // the call 103.6 us, 16 98), more while 2048 blocks are left, then as many as leave 1024 sums of a column.
  const int64_t across = ceil_div(l.ldz, 64 * (16 / e));
  l.chunk = std::max<int64_t>(16, std::min<int64_t>(64, l.piece * across / 2048 / 16 * 16));
  l.chunk = std::max(l.chunk, ceil_div(ceil_div(l.piece, 1024), 16) * 16);
  l.chunk = std::min(l.piece, l.chunk);
  size_t off = 0, part = 0, stats = 0, fold = 0, sums = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  size_t z = 0, g = 0;
  for (int64_t rows : {l.piece, N % l.piece})
    if (rows) {
      const bool kept = l.kept(rows, V, d_in, e);
      if (!l.twice && !kept) z = std::max(z, (size_t)rows * l.ldz * sizeof(float));
      g = std::max(g, (size_t)rows * l.ldz * e);
      if (!l.few) {
        const Cut c = l.logits(rows, V, d_in, e);
        part = std::max(part, partial_bytes(c, rows, V));
        stats = std::max(stats, (size_t)rows * stat_groups(c.variant, e, V) * 2 * sizeof(float));
      }
      part = std::max(part, partial_bytes(choose_cut(rows, d_in, V, e), rows, d_in));
      part = std::max(part, partial_bytes(choose_cut(V, d_in, rows, e), V, d_in));
      if (l.folds(rows, V, d_in, e)) fold = std::max(fold, (size_t)l.tile_sums(rows, V, d_in, e) * V * sizeof(float));
      sums = std::max(sums, (size_t)(l.sums(rows, V, d_in, e) + l.carries(N)) * V * sizeof(float));
    }
  l.o_x = take(l.pad && !l.few ? (size_t)l.piece * l.lx * e : 0);
  l.o_clean = take((size_t)l.piece * l.lx * e);
  l.o_w = take(l.pad ? (size_t)V * l.lx * e : 0);
  l.o_z = take(z);
  l.o_g = take(g);
  l.o_stats = take(stats);
  l.o_picked = take(l.few ? 0 : (size_t)l.piece * kMaxPicksRow * sizeof(float));
  l.o_coef = take((size_t)l.piece * sizeof(RowCoef));
  l.o_acc = take(l.piece < N && e == 2 ? (size_t)V * d_in * sizeof(float) : 0);
  l.o_part = take(part);
  l.o_fold = take(fold);
  l.o_db = take(sums);
  l.o_range = take((kEntropyRange + 1) * sizeof(float));
  l.bytes = off;
  return l;
}

static int check_entropy(int64_t N, int32_t d_in, int32_t V, int32_t top, int32_t x_dtype) {
  if (!dtype_ok(x_dtype) || N < 0 || d_in < 1 || V < 1 || top < 1) return GMM_EINVAL;
  if (d_in > kMaxWidth || V > kMaxClasses || top > kMaxPicksRow || N > kMaxRows) return GMM_EUNSUPPORTED;
  return GMM_OK;
}

// The first row of a piece in an array of `width` elements a row.
template <typename E>
static E* row_at(E* p, int64_t row, int64_t width) {
  return p ? p + row * width : nullptr;
}

template <typename T>
static hipError_t entropy_forward(EntropyArgs a, int64_t N, char* ws, hipStream_t s) {
  const EntropyPlan l = entropy_plan(N, a.d_in, a.V, sizeof(T));
  const EntropyArgs all = a;
  hipError_t e = hipSuccess;
  ProductArgs p{};
  p.bias = a.bias;
  p.lda = p.ldb = l.lx;
  p.N = a.V;
  p.K = a.d_in;
  for (int64_t r = 0; r < N; r += l.piece) {
    a.rows = std::min(N - r, l.piece);
    a.X = row_at(static_cast<const T*>(all.X), r, a.d_in);
    a.picks.idx = row_at(all.picks.idx, r, a.picks.top);
    a.picks.wts = row_at(all.picks.wts, r, a.picks.top);
    a.loss = row_at(all.loss, r, 1);
    a.lse = row_at(all.lse, r, 1);
    a.stats = p.stats = reinterpret_cast<float*>(ws + l.o_stats);
    a.picked = p.picked = reinterpret_cast<float*>(ws + l.o_picked);
    p.picks = a.picks;
    if (l.few) {
      const FewArgs f{a.X, a.W, (int)N, a.V, a.d_in, a.bias, nullptr, nullptr, nullptr, 1, 0, p.stats, p.picked, p.picks};
      a.groups = l.groups;
      if ((e = launch_few<T>(kRowStats, f, s)) != hipSuccess) return e;
      return launch_entropy_loss<T>(a, s);
    }
    p.A = a.X;
    p.B = a.W;
    if (l.pad) {
      const PadJob px{a.X, ws + l.o_x, a.rows, l.lx, a.d_in}, pw{a.W, ws + l.o_w, r == 0 ? a.V : 0, l.lx, a.d_in};
      if ((e = launch_pad<T>(px, pw, s)) != hipSuccess) return e;
      p.A = ws + l.o_x;
      p.B = ws + l.o_w;
    }
    p.M = a.rows;
    if ((e = run_product<T>(l.cut, false, false, kRowStats, p, s)) != hipSuccess) return e;
    a.groups = l.groups;
    if ((e = launch_entropy_loss<T>(a, s)) != hipSuccess) return e;
  }
  return e;
}

template <typename T>
static hipError_t entropy_gradients(EntropyArgs a, int64_t N, T* dX, T* dW, T* db, char* ws, hipStream_t s) {
  const EntropyBackPlan l = entropy_back_plan(N, a.d_in, a.V, sizeof(T));
  const EntropyArgs all = a;
  const bool scaled = sizeof(T) == 2;
  hipError_t e = hipSuccess;
  a.range = scaled ? reinterpret_cast<float*>(ws + l.o_range) : nullptr;
  a.ldz = l.ldz;
  a.Z = reinterpret_cast<float*>(ws + l.o_z);
  a.G = ws + l.o_g;
  a.coef = reinterpret_cast<RowCoef*>(ws + l.o_coef);
  a.chunk = l.chunk;
  float* sums = reinterpret_cast<float*>(ws + l.o_db);
  a.parts = db ? sums + l.carries(N) * a.V : nullptr;
  const bool pad_w = l.pad && (dX || !l.few), pad_x = l.pad && !l.few;
  const void* W = pad_w ? ws + l.o_w : a.W;
  for (int64_t r = 0; r < N; r += l.piece) {
    const int64_t rows = a.rows = std::min(N - r, l.piece);
    const bool last = r + rows == N;
    a.X = row_at(static_cast<const T*>(all.X), r, a.d_in);
    a.picks.idx = row_at(all.picks.idx, r, a.picks.top);
    a.picks.wts = row_at(all.picks.wts, r, a.picks.top);
    a.dloss = row_at(all.dloss, r, 1);
    a.loss = row_at(all.loss, r, 1);
    a.lse = row_at(all.lse, r, 1);
    // few picks, and rows in their place: the loss kernel does the rest
    const bool alone = N * a.picks.top <= kOwnPrepPicks && !pad_x && !pad_w;
    a.own_range = alone;
    a.clean = alone && dW ? ws + l.o_clean : nullptr;
    a.ldx = l.lx;
    EntropyPrep b{};
    b.X = a.X, b.ld = l.lx, b.d_in = a.d_in, b.V = a.V;
    b.x = pad_x ? ws + l.o_x : nullptr;
    b.clean = dW ? ws + l.o_clean : nullptr;
    b.rows = b.x || b.clean ? rows : 0;
    b.W = a.W, b.w = pad_w && r == 0 ? ws + l.o_w : nullptr;
    b.all_rows = scaled && r == 0 ? N : 0;
    b.picks = all.picks, b.dloss = all.dloss, b.first = r, b.range = a.range;
    if (!alone && (e = launch_entropy_prep<T>(b, s)) != hipSuccess) return e;
    ProductArgs p{};
    p.partial = reinterpret_cast<float*>(ws + l.o_part);
    // the logits, through the caches, which the next kernel finds them in (16384 x 128 to 1024 classes in float: 170 us
    // for the call, past them 172; 2048 x 128 to 32768, 256 MiB: 612 and 605; 2-byte operands within 1 us)
    a.stats = a.picked = nullptr;
    if (l.few) {
      const FewArgs f{a.X, a.W, (int)N, a.V, a.d_in, a.bias, nullptr, const_cast<float*>(a.Z), nullptr, 1, l.ldz};
      e = launch_few<T>(GMM_ACT_NONE, f, s);
    } else {
      p.A = pad_x ? ws + l.o_x : a.X;
      p.B = W, p.lda = p.ldb = l.lx;
      p.M = rows, p.N = a.V, p.K = a.d_in;
      p.bias = a.bias;
      const Cut c = l.logits(rows, a.V, a.d_in, sizeof(T));
      if (c.splits == 1) {  // whole sums: the tiles' statistics with them
        a.stats = p.stats = reinterpret_cast<float*>(ws + l.o_stats);
        a.groups = stat_groups(c.variant, sizeof(T), a.V);
        a.columns = stat_columns(c.variant, sizeof(T));
      }
      const bool kept = l.kept(rows, a.V, a.d_in, sizeof(T));
      a.Z = l.twice || kept ? nullptr : reinterpret_cast<float*>(ws + l.o_z);
      p.picks = a.picks;
      if (!a.Z) a.picked = p.picked = reinterpret_cast<float*>(ws + l.o_picked);
      p.C = kept ? a.G : const_cast<float*>(a.Z);
      p.ldc = l.ldz;
      p.c_f32 = !kept;
      e = run_product<T>(c, false, false, l.twice ? kRowStats : a.stats ? kStatsToo : (int)GMM_ACT_NONE, p, s, false);
      if (e == hipSuccess && l.twice) e = launch_entropy_loss<T>(a, s);
      if (e == hipSuccess && l.twice && (dX || dW || db)) {  // again, for their gradient
        p.coef = a.coef;
        const bool folds = db && l.folds(rows, a.V, a.d_in, sizeof(T));
        p.parts = folds ? reinterpret_cast<float*>(ws + l.o_fold) : a.parts;
        p.parts_unscale = scaled ? a.range + kEntropyRange : nullptr;
        p.C = a.G;
        p.c_f32 = sizeof(T) == 4;
        e = run_product<T>(c, false, false, kLogitGradient, p, s, false);
        if (e == hipSuccess && folds)
          e = launch_entropy_fold(p.parts, l.tile_sums(rows, a.V, a.d_in, sizeof(T)), kFoldedSums, a.V, a.parts, s);
      }
    }
    if (e != hipSuccess) return e;
    if (!l.twice && (e = launch_entropy_loss<T>(a, s)) != hipSuccess) return e;
    if (!dX && !dW && !db) continue;
    if (!l.twice && (e = launch_entropy_gradient<T>(a, s)) != hipSuccess) return e;
    // the column sums of this piece, and of those before in front of them
    const int64_t first = r ? 0 : l.carries(N), count = l.carries(N) + l.sums(rows, a.V, a.d_in, sizeof(T)) - first;
    if (db && !last && (e = launch_entropy_fold(sums + first * a.V, count, 1, a.V, sums, s)) != hipSuccess) return e;
    p = ProductArgs{};
    p.partial = reinterpret_cast<float*>(ws + l.o_part);
    p.N = a.d_in;
    p.ldc = a.d_in;
    p.ldb = l.lx;
    p.unscale = scaled ? a.range + kEntropyRange : nullptr;
    if (db && last) {  // summed beside the next product
      p.sums = sums + first * a.V;
      p.sums_out = db;
      p.sums_rows = count;
      p.sums_cols = a.V;
      p.sum_blocks = (int)ceil_div(a.V, kSumCols);
      if (!dX && !dW) return launch_column_sums<T>(p, s);
    }
    if (dX) {  // dX = G W
      p.A = a.G, p.lda = l.ldz;
      p.B = W;
      p.M = rows, p.K = a.V;
      p.C = row_at(dX, r, a.d_in);
      p.c_f32 = sizeof(T) == 4;
      if ((e = run_product<T>(choose_cut(rows, a.d_in, a.V, sizeof(T)), false, true, GMM_ACT_NONE, p, s)) != hipSuccess)
        return e;
    }
    if (dW) {  // dW = G^T X, over the pieces in float
      float* acc = sizeof(T) == 4 ? reinterpret_cast<float*>(dW) : reinterpret_cast<float*>(ws + l.o_acc);
      p.A = a.G, p.lda = l.ldz;
      p.B = ws + l.o_clean;
      p.M = a.V, p.K = rows;
      p.residual = r ? acc : nullptr;
      p.res_f32 = 1;
      p.C = last ? static_cast<void*>(dW) : acc;
      p.c_f32 = sizeof(T) == 4 || !last;
      if ((e = run_product<T>(choose_cut(a.V, a.d_in, rows, sizeof(T)), true, true, GMM_ACT_NONE, p, s)) != hipSuccess)
        return e;
    }
  }
  return e;
}

}  // namespace gmm

using namespace gmm;

extern "C" {

size_t gmm_layer_norm_workspace_bytes(int64_t N, int32_t D, int32_t x_dtype) {
  if (check_norm(N, D, x_dtype, x_dtype, x_dtype) != GMM_OK) return 0;
  return std::max<size_t>(norm_bytes(N, D, elem_size(x_dtype)), 256);
}

int gmm_layer_norm(const void* X, int32_t x_dtype, int64_t N, int32_t D, const void* gamma, const void* beta,
                   int32_t w_dtype, float eps, void* Y, int32_t y_dtype, float* stats, void* stream) {
  const int st = check_norm(N, D, x_dtype, y_dtype, w_dtype);
  if (st) return st;
  if (!(eps > 0.f) || !isfinite(eps)) return GMM_EINVAL;
  if (N == 0) return GMM_OK;
  if (!X || !Y) return GMM_EINVAL;
  NormArgs p{};
  p.X = X, p.gamma = gamma, p.beta = beta, p.w_f32 = w_dtype == GMM_F32;
  p.Y = Y, p.stats = stats, p.N = N, p.D = D, p.eps = eps;
  return with_norm_types(x_dtype, y_dtype, [&](auto* tx, auto* ty) {
    return launch_norm<std::remove_pointer_t<decltype(tx)>, std::remove_pointer_t<decltype(ty)>>(
        p, static_cast<hipStream_t>(stream));
  });
}

int gmm_layer_norm_backward(const void* dY, int32_t y_dtype, const void* X, int32_t x_dtype, int64_t N, int32_t D,
                            const float* stats, const void* gamma, int32_t w_dtype, void* dX, void* dgamma, void* dbeta,
                            void* workspace, size_t ws_bytes, void* stream) {
  int st = check_norm(N, D, x_dtype, y_dtype, w_dtype);
  if (st) return st;
  if (N > 0 && (!dY || !X || !stats)) return GMM_EINVAL;
  const bool sums = dgamma || dbeta;
  if (N > 0 && sums && (st = check_ws(workspace, ws_bytes, norm_bytes(N, D, elem_size(x_dtype))))) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (N == 0) {  // sums over no rows; zeros are the same bits in every type of a size
    const int e = elem_size(w_dtype);
    hipError_t r = hipSuccess;
    for (void* out : {dgamma, dbeta})
      if (out && r == hipSuccess)
        r = e == 4 ? launch_zero<float>(static_cast<float*>(out), D, s)
                   : launch_zero<_Float16>(static_cast<_Float16*>(out), D, s);
    return hip_status(r);
  }
  if (!dX && !sums) return GMM_OK;
  NormArgs p{};
  p.X = X, p.gamma = gamma, p.w_f32 = w_dtype == GMM_F32;
  p.stats = const_cast<float*>(stats), p.N = N, p.D = D;
  p.dY = dY, p.dX = dX, p.dgamma = dgamma, p.dbeta = dbeta;
  p.partial = sums ? static_cast<float*>(workspace) : nullptr;
  p.parts = norm_parts(N, D, elem_size(x_dtype));
  return with_norm_types(x_dtype, y_dtype, [&](auto* tx, auto* ty) {
    return launch_norm_backward<std::remove_pointer_t<decltype(tx)>, std::remove_pointer_t<decltype(ty)>>(p, s);
  });
}

size_t gmm_cross_entropy_workspace_bytes(int64_t N, int32_t d_in, int32_t V, int32_t x_dtype, int32_t gradients) {
  if (check_entropy(N, d_in, V, 1, x_dtype) != GMM_OK) return 0;
  const int e = elem_size(x_dtype);
  const size_t b = N == 0 ? 0 : gradients ? entropy_back_plan(N, d_in, V, e).bytes : entropy_plan(N, d_in, V, e).bytes;
  return std::max<size_t>(b, 256);
}

int gmm_cross_entropy(const void* X, int32_t x_dtype, int64_t N, int32_t d_in, const void* W, int32_t V,
                      const void* bias, const int32_t* idx, const float* wts, int32_t top, float* loss, float* lse,
                      void* workspace, size_t ws_bytes, void* stream) {
  int st = check_entropy(N, d_in, V, top, x_dtype);
  if (st) return st;
  if (!W || (N > 0 && (!X || !idx || !loss))) return GMM_EINVAL;
  const int e = elem_size(x_dtype);
  if (row_len(d_in, e) == d_in && (!aligned16(X) || !aligned16(W))) return GMM_EINVAL;
  if (N == 0) return GMM_OK;
  if ((st = check_ws(workspace, ws_bytes, entropy_plan(N, d_in, V, e).bytes))) return st;
  EntropyArgs a{};
  a.X = X, a.W = W, a.bias = bias, a.picks = RowPicks{idx, wts, top}, a.d_in = d_in, a.V = V;
  a.loss = loss, a.lse = lse;
  return with_type(x_dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    return hip_status(
        entropy_forward<T>(a, N, static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
  });
}

int gmm_cross_entropy_gradients(const float* dloss, const void* X, int32_t x_dtype, int64_t N, int32_t d_in,
                                const void* W, int32_t V, const void* bias, const int32_t* idx, const float* wts,
                                int32_t top, float* loss, float* lse, void* dX, void* dW, void* db, void* workspace,
                                size_t ws_bytes, void* stream) {
  int st = check_entropy(N, d_in, V, top, x_dtype);
  if (st) return st;
  if (!W || (N > 0 && (!X || !idx || !loss))) return GMM_EINVAL;
  const int e = elem_size(x_dtype);
  if (row_len(d_in, e) == d_in && (!aligned16(X) || !aligned16(W))) return GMM_EINVAL;
  if (N > 0 && (st = check_ws(workspace, ws_bytes, entropy_back_plan(N, d_in, V, e).bytes))) return st;
  EntropyArgs a{};
  a.X = X, a.W = W, a.bias = bias, a.picks = RowPicks{idx, wts, top}, a.dloss = dloss, a.d_in = d_in, a.V = V;
  a.loss = loss, a.lse = lse;
  return with_type(x_dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (N == 0) {  // sums over no rows
      hipError_t r = hipSuccess;
      if (dW) r = launch_zero<T>(static_cast<T*>(dW), (int64_t)V * d_in, s);
      if (r == hipSuccess && db) r = launch_zero<T>(static_cast<T*>(db), V, s);
      return hip_status(r);
    }
    return hip_status(entropy_gradients<T>(a, N, static_cast<T*>(dX), static_cast<T*>(dW), static_cast<T*>(db),
                                           static_cast<char*>(workspace), s));
  });
}

int64_t gmm_adamw_state_elements(int32_t count, const int64_t* sizes) {
  if (count < 0 || (count > 0 && !sizes)) return -1;
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (sizes[i] < 0 || sizes[i] >= (int64_t)1 << 40) return -1;
    total += ceil_div(sizes[i], kStateBlock) * kStateBlock;
  }
  return total;
}

int gmm_adamw_step(int32_t count, const int64_t* sizes, void* const* params, int32_t p_dtype,
                   const void* const* grads, int32_t g_dtype, float* master, void* m, void* v, int32_t state_bits,
                   float* m_scale, float* v_scale, int64_t* step, double lr, double beta1, double beta2, double eps,
                   double weight_decay, const float* lr_factor, const float* grad_factor, void* stream) {
  if (!dtype_ok(p_dtype) || (g_dtype != p_dtype && g_dtype != GMM_F32)) return GMM_EINVAL;
  if (state_bits != 32 && state_bits != 8) return GMM_EINVAL;
  if (!factor_ok(beta1) || !factor_ok(beta2) || !size_ok(lr) || !size_ok(weight_decay)) return GMM_EINVAL;
  // the device's reciprocal takes a denormal number for 0
  if (!size_ok(eps) || (float)eps < FLT_MIN) return GMM_EINVAL;
  const int64_t total = gmm_adamw_state_elements(count, sizes);
  if (total < 0 || !step || reinterpret_cast<uintptr_t>(step) % 8 || (count > 0 && (!params || !grads)))
    return GMM_EINVAL;
  // a float copy of float parameters would be the parameters twice
  if (p_dtype == GMM_F32 && master) return GMM_EINVAL;
  if (total > 0 && (!m || !v || (state_bits == 8 && (!m_scale || !v_scale)))) return GMM_EINVAL;
  if (!aligned16(m) || !aligned16(v) || !aligned16(master)) return GMM_EINVAL;
  for (int32_t i = 0; i < count; ++i)
    if (sizes[i] > 0 && grads[i] && !params[i]) return GMM_EINVAL;
  AdamArgs a{};
  a.master = master;
  a.m = m, a.v = v, a.m_scale = m_scale, a.v_scale = v_scale;
  a.step = step, a.lr_factor = lr_factor, a.grad_factor = grad_factor;
  a.log_beta1 = log(beta1), a.log_beta2 = log(beta2);
  a.beta1 = (float)beta1, a.beta2 = (float)beta2, a.rest1 = (float)(1. - beta1), a.rest2 = (float)(1. - beta2);
  a.lr = (float)lr, a.eps = (float)eps, a.decay = (float)weight_decay;
  a.stream = total * (state_bits == 32 ? 8 : 2) >= kStreamBytes;
  hipStream_t s = static_cast<hipStream_t>(stream);
  int64_t at = 0;
  int32_t i = 0;
  do {  // a launch for each kAdamTensors tensors with work, one for none
    a.count = 0;
    int64_t blocks = 0;
    for (; i < count && a.count < kAdamTensors; ++i) {
      const int64_t mine = ceil_div(sizes[i], kStateBlock);
      if (mine > 0 && grads[i]) {
        a.tensor[a.count++] = AdamArgs::Tensor{params[i], grads[i], sizes[i], at};
        blocks += mine;
      }
      at += mine * kStateBlock;
    }
    // State blocks of a thread block: one a wave up to 2048 thread blocks, then as many as measure best (16 of 32
    // bits, 64 of 8: 268M parameters 1390 and 827 us, with 64 and 16 of them 1472 and 876), more where the grid would
    // pass 2^24.
    const int64_t few = 4 * ceil_div(blocks, 4 * 2048), most = state_bits == 32 ? 16 : 64;
    a.chunk = (int)std::max<int64_t>({4, std::min(few, most), ceil_div(blocks, 1 << 24)});
    a.first[0] = 0;
    for (int k = 0; k < a.count; ++k)
      a.first[k + 1] = a.first[k] + (int)ceil_div(ceil_div(a.tensor[k].n, kStateBlock), a.chunk);
    a.last = i == count;
    const hipError_t e = launch_adamw(p_dtype, g_dtype, state_bits, a, s);
    if (e != hipSuccess) return hip_status(e);
  } while (i < count);
  return GMM_OK;
}

}  // extern "C"
