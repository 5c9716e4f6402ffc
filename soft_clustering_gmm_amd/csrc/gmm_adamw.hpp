// Internal declarations of the AdamW step (gmm_adamw_step).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gmm {

constexpr int kStateBlock = 256;  // elements of a state that share a scale
constexpr int kAdamTensors = 96;  // tensors of one launch: its arguments hold them

struct AdamArgs {
  float* master;  // null: the parameters themselves are updated
  void *m, *v;    // float, or 8-bit codes beside the scales
  float *m_scale, *v_scale;
  int64_t* step;  // {steps done, blocks of this launch that are}
  const float *lr_factor, *grad_factor;  // device scalars, null: 1
  double log_beta1, log_beta2;
  float beta1, beta2, rest1, rest2;      // rest = 1 - beta
  float lr, eps, decay;
  int count;
  int chunk;      // state blocks of a block
  int last;       // the launch that counts the step
  int stream;     // past the caches
  struct Tensor {
    void* p;
    const void* g;
    int64_t n, at;  // elements; first element of its part of the state
  } tensor[kAdamTensors];
  int first[kAdamTensors + 1];  // first block of each tensor
};
static_assert(sizeof(AdamArgs) <= 4096, "a kernel's arguments");

hipError_t launch_adamw(int p_dtype, int g_dtype, int bits, const AdamArgs& a, hipStream_t s);

}  // namespace gmm
