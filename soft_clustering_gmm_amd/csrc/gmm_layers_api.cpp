// C-ABI of the learned products around the mixture: the linear layer with its
// gradients and the layer of experts. Argument checks, workspace planning and
// dispatch; every check runs on the host before anything is enqueued.
#include "../../include/gmm.h"

#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "gmm_experts.hpp"
#include "gmm_layers.hpp"

namespace gmm {

constexpr int64_t kLaunchRows = 1 << 20;     // rows of one launch (the grid's size)
constexpr int64_t kDzRows = 16;              // rows per column-sum chunk, at least
constexpr int64_t kDzMostRows = 8192;        // and at most: they are added one after the other
constexpr size_t kNoWorkspace = 256;         // what the linear layer's query reports where none is needed
constexpr int64_t kDzBlocks = 2048;          // blocks of the column sums, where the rows allow it

// Workspace of the forward pass: [padded rows of X of one launch] [padded W]
// [partial sums].
struct LinearPlan {
  bool few, pad;
  int64_t kp;  // row length of the operands
  Cut cut;     // of a whole launch
  size_t o_x, o_w, o_part, bytes;
};

static LinearPlan linear_plan(int64_t N, int d_in, int d_out, int e) {
  LinearPlan l{};
  l.few = N <= kFewRows;
  l.kp = row_len(d_in, e);
  l.pad = l.kp != d_in;
  if (l.few || N == 0) return l;
  const int64_t rows = std::min(N, kLaunchRows), tail = N % kLaunchRows;
  l.cut = choose_cut(rows, d_out, d_in, e);
  size_t part = partial_bytes(l.cut, rows, d_out);
  if (N > kLaunchRows && tail) part = std::max(part, partial_bytes(choose_cut(tail, d_out, d_in, e), tail, d_out));
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  l.o_x = take(l.pad ? (size_t)rows * l.kp * e : 0);
  l.o_w = take(l.pad ? (size_t)d_out * l.kp * e : 0);
  l.o_part = take(part);
  l.bytes = off;
  return l;
}

// Workspace of the backward pass: [dZ] [padded X] [padded W] [partial sums of
// dX, then of dW] [column sums] [range of dZ and its scale's inverse].
struct BackwardPlan {
  int64_t lx, lz;  // row lengths of X and W, of dZ
  bool pad, own_dz;
  int64_t chunk, chunks;  // rows per column sum
  size_t o_z, o_x, o_w, o_part, o_db, o_range, bytes;
};

static BackwardPlan backward_plan(int64_t N, int d_in, int d_out, int e, bool plain_dz, bool want_dx, bool want_dw,
                                  bool want_db) {
  BackwardPlan b{};
  b.lx = row_len(d_in, e);
  b.lz = row_len(d_out, e);
  b.pad = b.lx != d_in;
  b.own_dz = !(plain_dz && b.lz == d_out) && (want_dx || want_dw);
  const int64_t across = ceil_div(d_out, 64 * (16 / e));
  b.chunk = std::max(kDzRows, ceil_div(ceil_div(N * across, kDzBlocks), kDzRows) * kDzRows);
  b.chunk = std::min(b.chunk, kDzMostRows);
  b.chunks = ceil_div(N, b.chunk);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  size_t part = 0;
  if (want_dx) {
    const int64_t rows = std::min(N, kLaunchRows), tail = N % kLaunchRows;
    part = partial_bytes(choose_cut(rows, d_in, d_out, e), rows, d_in);
    if (N > kLaunchRows && tail) part = std::max(part, partial_bytes(choose_cut(tail, d_in, d_out, e), tail, d_in));
  }
  if (want_dw) part = std::max(part, partial_bytes(choose_cut(d_out, d_in, N, e), d_out, d_in));
  b.o_z = take(b.own_dz ? (size_t)N * b.lz * e : 0);
  b.o_x = take(b.pad && want_dw ? (size_t)N * b.lx * e : 0);
  b.o_w = take(b.pad && want_dx ? (size_t)d_out * b.lx * e : 0);
  b.o_part = take(part);
  b.o_db = take(want_db ? (size_t)b.chunks * d_out * sizeof(float) : 0);
  b.o_range = take(e == 2 ? (kRangeBlocks + 1) * sizeof(float) : 0);
  b.bytes = off;
  return b;
}

static int check_linear(int64_t N, int32_t d_in, int32_t d_out, int32_t x_dtype, int32_t y_dtype, int32_t act) {
  if (!dtype_ok(x_dtype) || (y_dtype != x_dtype && y_dtype != GMM_F32) || !act_ok(act)) return GMM_EINVAL;
  if (N < 0 || d_in < 1 || d_out < 1) return GMM_EINVAL;
  if (d_in > kMaxWidth || d_out > kMaxWidth || N > kMaxRows) return GMM_EUNSUPPORTED;
  return GMM_OK;
}

template <typename T>
static hipError_t linear_forward(const T* X, int64_t N, int d_in, const T* W, int d_out, const T* bias, int act,
                                 const void* residual, void* Y, int y_f32, void* pre, char* ws, hipStream_t s) {
  const LinearPlan l = linear_plan(N, d_in, d_out, sizeof(T));
  if (l.few) {
    const FewArgs f{X, W, (int)N, d_out, d_in, bias, residual, Y, pre, y_f32, d_out, nullptr};
    return launch_few<T>(act, f, s);
  }
  const int ey = y_f32 ? 4 : (int)sizeof(T);
  ProductArgs p{};
  p.B = W;
  p.lda = p.ldb = l.kp;
  p.N = d_out;
  p.ldc = d_out;
  p.K = d_in;
  p.bias = bias;
  p.c_f32 = y_f32;
  p.partial = reinterpret_cast<float*>(ws + l.o_part);
  hipError_t e = hipSuccess;
  if (l.pad) p.B = ws + l.o_w;
  for (int64_t r = 0; r < N; r += kLaunchRows) {
    const int64_t rows = std::min(N - r, kLaunchRows);
    p.M = rows;
    p.A = X + r * d_in;
    if (l.pad) {
      const PadJob px{X + r * d_in, ws + l.o_x, rows, l.kp, d_in}, pw{W, ws + l.o_w, r == 0 ? d_out : 0, l.kp, d_in};
      if ((e = launch_pad<T>(px, pw, s)) != hipSuccess) return e;
      p.A = ws + l.o_x;
    }
    const size_t at = (size_t)r * d_out * ey;
    p.C = static_cast<char*>(Y) + at;
    p.residual = residual ? static_cast<const char*>(residual) + at : nullptr;
    p.pre = pre ? static_cast<char*>(pre) + at : nullptr;
    e = run_product<T>(r == 0 ? l.cut : choose_cut(rows, d_out, d_in, sizeof(T)), false, false, act, p, s);
    if (e != hipSuccess) return e;
  }
  return e;
}

template <typename T>
static hipError_t linear_gradients(const void* dY, int y_f32, const T* X, int64_t N, int d_in, const T* W, int d_out,
                                   const void* pre, int act, T* dX, T* dW, T* db, char* ws, hipStream_t s) {
  const bool plain = act == GMM_ACT_NONE && (y_f32 != 0) == (sizeof(T) == 4) && aligned16(dY);
  const BackwardPlan b = backward_plan(N, d_in, d_out, sizeof(T), plain, dX != nullptr, dW != nullptr, db != nullptr);
  T* z = reinterpret_cast<T*>(ws + b.o_z);
  float* part = reinterpret_cast<float*>(ws + b.o_db);
  hipError_t e = hipSuccess;
  PadJob px{}, pw{};
  if (b.pad && dW) px = PadJob{X, ws + b.o_x, N, b.lx, d_in};
  if (b.pad && dX) pw = PadJob{W, ws + b.o_w, d_out, b.lx, d_in};
  // Half does not hold every float: dZ is scaled for the products.
  float* range = nullptr;
  if constexpr (std::is_same<T, _Float16>::value)
    if (y_f32 && b.own_dz) {
      range = reinterpret_cast<float*>(ws + b.o_range);
      e = launch_dz_range<T>(act, static_cast<const float*>(dY), static_cast<const float*>(pre), N * d_out, range, s);
      if (e != hipSuccess) return e;
    }
  float* unscale = range ? range + kRangeBlocks : nullptr;
  if (b.own_dz || db)
    e = launch_dz<T>(act, dY, pre, y_f32, N, d_out, b.own_dz ? z : nullptr, b.lz, db ? part : nullptr, b.chunk, px, pw,
                     range, unscale, s);
  else if (px.rows || pw.rows)
    e = launch_pad<T>(px, pw, s);
  if (e != hipSuccess) return e;
  const T* dZ = b.own_dz ? z : static_cast<const T*>(dY);
  ProductArgs p{};
  p.partial = reinterpret_cast<float*>(ws + b.o_part);
  p.c_f32 = sizeof(T) == 4;
  p.N = d_in;
  p.ldc = d_in;
  p.ldb = b.lx;
  p.unscale = unscale;
  if (db) {  // summed beside the first product
    p.sums = part;
    p.sums_out = db;
    p.sums_rows = b.chunks;
    p.sums_cols = d_out;
    p.sum_blocks = (int)ceil_div(d_out, kSumCols);
  }
  if (!dX && !dW) return db ? launch_column_sums<T>(p, s) : hipSuccess;
  if (dX) {  // dX = dZ W
    p.B = b.pad ? ws + b.o_w : static_cast<const void*>(W);
    p.lda = b.lz;
    p.K = d_out;
    for (int64_t r = 0; r < N; r += kLaunchRows) {
      p.M = std::min(N - r, kLaunchRows);
      p.A = dZ + r * b.lz;
      p.C = dX + r * d_in;
      if ((e = run_product<T>(choose_cut(p.M, d_in, d_out, sizeof(T)), false, true, GMM_ACT_NONE, p, s)) != hipSuccess)
        return e;
    }
  }
  if (dW) {  // dW = dZ^T X
    p.B = b.pad ? ws + b.o_x : static_cast<const void*>(X);
    p.A = dZ;
    p.lda = b.lz;
    p.M = d_out;
    p.K = N;
    p.C = dW;
    e = run_product<T>(choose_cut(d_out, d_in, N, sizeof(T)), true, true, GMM_ACT_NONE, p, s);
  }
  return e;
}

// Workspace of the layer of experts.
struct ExpertPlan {
  size_t o_feats, o_consts, o_scores, o_wts, o_bad, o_place, o_row, o_ord, o_weight, o_scale, o_expert, o_first, o_count,
      o_h, o_out, bytes;
};

static ExpertPlan expert_plan(int64_t T, int D, int F, int K, int d, int top, int e) {
  ExpertPlan x{};
  const size_t n = (size_t)T * top;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = align_up(off + bytes, 256);
    return o;
  };
  x.o_feats = take((size_t)kGateParts * T * d * sizeof(double));
  x.o_consts = take(d ? (size_t)K * sizeof(double) : 0);
  x.o_scores = take(d && K > kScoresInLds ? (size_t)T * K * sizeof(double) : 0);
  x.o_wts = take(n * sizeof(float));
  x.o_bad = take(T * sizeof(int32_t));
  x.o_place = take(n * sizeof(int32_t));
  x.o_row = take(n * sizeof(int32_t));
  x.o_ord = take(n * sizeof(int32_t));
  x.o_weight = take(n * sizeof(float));
  x.o_scale = take(T * sizeof(float));
  x.o_expert = take(n * sizeof(int32_t));
  x.o_first = take((n + 1) * sizeof(int32_t));
  x.o_count = take(kCounts * sizeof(int32_t));
  x.o_h = take(n * F * e);
  x.o_out = take(n > kGatherPicks ? n * D * sizeof(float) : 0);
  x.bytes = off;
  return x;
}

static int check_experts(int32_t x_dtype, int64_t T, int32_t D, int32_t K, int32_t F, int32_t top, int32_t act) {
  if (!dtype_ok(x_dtype) || !act_ok(act)) return GMM_EINVAL;
  if (T < 0 || D < 1 || K < 1 || F < 1 || top < 1) return GMM_EINVAL;
  if (T > kMaxLayerRows || top > kMaxTop || D > kMaxWidth || F > kMaxWidth || K > 65536) return GMM_EUNSUPPORTED;
  return GMM_OK;
}

static void place_experts(ExpertArgs& p, const ExpertPlan& x, void* workspace) {
  char* b = static_cast<char*>(workspace);
  p.feats = reinterpret_cast<double*>(b + x.o_feats);
  p.consts = reinterpret_cast<double*>(b + x.o_consts);
  p.scores = reinterpret_cast<double*>(b + x.o_scores);
  p.wts = reinterpret_cast<float*>(b + x.o_wts);
  p.bad = reinterpret_cast<int32_t*>(b + x.o_bad);
  p.place = reinterpret_cast<int32_t*>(b + x.o_place);
  p.row_of = reinterpret_cast<int32_t*>(b + x.o_row);
  p.ord = reinterpret_cast<int32_t*>(b + x.o_ord);
  p.weight = reinterpret_cast<float*>(b + x.o_weight);
  p.scale = reinterpret_cast<float*>(b + x.o_scale);
  p.expert = reinterpret_cast<int32_t*>(b + x.o_expert);
  p.first = reinterpret_cast<int32_t*>(b + x.o_first);
  p.count = reinterpret_cast<int32_t*>(b + x.o_count);
  p.h = b + x.o_h;
  p.out = reinterpret_cast<float*>(b + x.o_out);
}

}  // namespace gmm

using namespace gmm;

extern "C" {

size_t gmm_linear_workspace_bytes(int64_t N, int32_t d_in, int32_t d_out, int32_t x_dtype, int32_t backward) {
  if (check_linear(N, d_in, d_out, x_dtype, x_dtype, GMM_ACT_NONE) != GMM_OK) return 0;
  const int e = elem_size(x_dtype);
  const size_t b = N == 0 ? 0
                   : backward ? backward_plan(N, d_in, d_out, e, false, true, true, true).bytes
                              : linear_plan(N, d_in, d_out, e).bytes;
  return b == 0 ? kNoWorkspace : std::max(b, 2 * kNoWorkspace);  // a need of 256 bytes is not taken for none
}

int gmm_linear(const void* X, int32_t x_dtype, int64_t N, int32_t d_in, const void* W, int32_t d_out,
               const void* bias, int32_t act, const void* residual, void* Y, int32_t y_dtype, void* pre,
               void* workspace, size_t ws_bytes, void* stream) {
  int st = check_linear(N, d_in, d_out, x_dtype, y_dtype, act);
  if (st) return st;
  if (!W || (N > 0 && (!X || !Y))) return GMM_EINVAL;
  const int e = elem_size(x_dtype);
  if (row_len(d_in, e) == d_in && (!aligned16(X) || !aligned16(W))) return GMM_EINVAL;
  if (N == 0) return GMM_OK;
  if ((st = check_ws(workspace, ws_bytes, linear_plan(N, d_in, d_out, e).bytes))) return st;
  return with_type(x_dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    return hip_status(linear_forward<T>(static_cast<const T*>(X), N, d_in, static_cast<const T*>(W), d_out,
                                        static_cast<const T*>(bias), act, residual, Y, y_dtype == GMM_F32, pre,
                                        static_cast<char*>(workspace), static_cast<hipStream_t>(stream)));
  });
}

int gmm_linear_backward(const void* dY, int32_t y_dtype, const void* X, int32_t x_dtype, int64_t N, int32_t d_in,
                        const void* W, int32_t d_out, const void* pre, int32_t act, void* dX, void* dW, void* db,
                        void* workspace, size_t ws_bytes, void* stream) {
  int st = check_linear(N, d_in, d_out, x_dtype, y_dtype, act);
  if (st) return st;
  if (N > 0 && (!dY || (act != GMM_ACT_NONE && !pre) || (dX && !W) || (dW && !X))) return GMM_EINVAL;
  const int e = elem_size(x_dtype);
  if (row_len(d_in, e) == d_in && ((dX && !aligned16(W)) || (dW && !aligned16(X)))) return GMM_EINVAL;
  if (N > 0 && (st = check_ws(workspace, ws_bytes, backward_plan(N, d_in, d_out, e, false, true, true, true).bytes)))
    return st;
  return with_type(x_dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (N == 0) {  // sums over no rows
      hipError_t r = hipSuccess;
      if (dW) r = launch_zero<T>(static_cast<T*>(dW), (int64_t)d_out * d_in, s);
      if (r == hipSuccess && db) r = launch_zero<T>(static_cast<T*>(db), d_out, s);
      return hip_status(r);
    }
    return hip_status(linear_gradients<T>(dY, y_dtype == GMM_F32, static_cast<const T*>(X), N, d_in,
                                          static_cast<const T*>(W), d_out, pre, act, static_cast<T*>(dX),
                                          static_cast<T*>(dW), static_cast<T*>(db), static_cast<char*>(workspace), s));
  });
}

size_t gmm_expert_workspace_bytes(int64_t N, int32_t D, int32_t K, int32_t F, int32_t d, int32_t top,
                                  int32_t x_dtype) {
  if (check_experts(x_dtype, N, D, K, F, top, GMM_ACT_NONE) != GMM_OK || d < 0 || d > 128) return 0;
  return expert_plan(N, D, F, K, d, top, elem_size(x_dtype)).bytes;
}

int gmm_expert_layer(const void* X, int32_t x_dtype, int64_t N, int32_t D, const void* P, int32_t d, const float* mu,
                     const float* var, const float* logw, int32_t K, int32_t top, float border_threshold,
                     int32_t renorm, const void* W1, const void* b1, const void* W2, const void* b2, int32_t F,
                     int32_t act, int32_t glu, const void* residual, void* Y, int32_t* idx, float* resp,
                     void* workspace, size_t ws_bytes, void* stream) {
  int st = check_experts(x_dtype, N, D, K, F, top, act);
  if (st) return st;
  if (d < 1) return GMM_EINVAL;
  if (d > 128) return GMM_EUNSUPPORTED;
  if (!P || !mu || !var || !logw || !W1 || !W2) return GMM_EINVAL;
  if (N == 0) return GMM_OK;
  if (!X || !Y || !idx || !resp) return GMM_EINVAL;
  const ExpertPlan x = expert_plan(N, D, F, K, d, top, elem_size(x_dtype));
  if ((st = check_ws(workspace, ws_bytes, x.bytes))) return st;
  ExpertArgs p{};
  p.X = X, p.residual = residual, p.Y = Y;
  p.T = (int)N, p.D = D, p.F = F, p.K = K, p.top = top, p.glu = glu != 0;
  p.proj = P, p.mu = mu, p.var = var, p.logw = logw, p.d = d, p.renorm = renorm != 0, p.threshold = border_threshold;
  p.idx = idx, p.resp = resp;
  p.W1 = W1, p.b1 = b1, p.W2 = W2, p.b2 = b2;
  place_experts(p, x, workspace);
  p.in_idx = idx, p.in_wts = p.wts;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return with_type(x_dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    hipError_t e = launch_gate<T>(p, s);  // and the lists
    if (e == hipSuccess) e = launch_experts<T>(act, p, s);
    return hip_status(e);
  });
}

int gmm_expert_rows(const void* X, int32_t x_dtype, int64_t N, int32_t D, const int32_t* idx, const float* wts,
                    int32_t top, int32_t K, const void* W1, const void* b1, const void* W2, const void* b2, int32_t F,
                    int32_t act, int32_t glu, const void* residual, void* Y, void* workspace, size_t ws_bytes,
                    void* stream) {
  int st = check_experts(x_dtype, N, D, K, F, top, act);
  if (st) return st;
  if (!W1 || !W2) return GMM_EINVAL;
  if (N == 0) return GMM_OK;
  if (!X || !Y || !idx || !wts) return GMM_EINVAL;
  const ExpertPlan x = expert_plan(N, D, F, K, 0, top, elem_size(x_dtype));
  if ((st = check_ws(workspace, ws_bytes, x.bytes))) return st;
  ExpertArgs p{};
  p.X = X, p.residual = residual, p.Y = Y;
  p.T = (int)N, p.D = D, p.F = F, p.K = K, p.top = top, p.glu = glu != 0;
  p.W1 = W1, p.b1 = b1, p.W2 = W2, p.b2 = b2;
  place_experts(p, x, workspace);
  p.bad = nullptr;
  p.in_idx = idx, p.in_wts = wts;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return with_type(x_dtype, [&](auto* t) {
    using T = std::remove_pointer_t<decltype(t)>;
    hipError_t e = launch_expert_lists(p, s);
    if (e == hipSuccess) e = launch_experts<T>(act, p, s);
    return hip_status(e);
  });
}

}  // extern "C"
