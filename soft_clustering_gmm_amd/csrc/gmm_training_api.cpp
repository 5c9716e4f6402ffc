// C-ABI of a training step around the mixture: the layer norm and the AdamW
// step. Argument checks, workspace planning and dispatch; every check runs on
// the host before anything is enqueued.
#include "../../include/gmm.h"

#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "gmm_adamw.hpp"
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
  if (!factor_ok(beta1) || !factor_ok(beta2) || !((float)eps > 0.f) || !isfinite(eps)) return GMM_EINVAL;
  if (!(lr >= 0.) || !isfinite(lr) || !(weight_decay >= 0.) || !isfinite(weight_decay)) return GMM_EINVAL;
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
