// Internal declarations of the layer of experts (gmm_expert_layer, gmm_expert_rows).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gmm {

constexpr int kMaxLayerRows = 128;  // rows of one call
constexpr int kMaxTop = 8;          // picks per row

// A layer's arguments and the pointers into its workspace.
struct ExpertArgs {
  const void* X;        // [T][D]
  const void* residual; // [T][D] or null
  void* Y;              // [T][D]
  int T, D, F, K, top, glu;
  // gate (null proj: the picks are given)
  const void* proj;     // [d][D]
  const float *mu, *var, *logw;
  int d, renorm;
  float threshold;
  int32_t* idx;         // [T][top]
  float* resp;          // [T][top]
  const int32_t* in_idx;
  const float* in_wts;
  // experts
  const void *W1, *b1, *W2, *b2;
  // workspace
  double* feats;        // [T][d]
  double* scores;       // [T][K]
  float* wts;           // [T][top] combination weights
  int32_t* bad;         // [T] rows whose gate is not a number
  int32_t* place;       // [T * top] place of a pick in the order by expert, -1: none
  int32_t* row_of;      // [T * top] row of the pick at a place
  int32_t* expert;      // [T * top] experts with picks, increasing
  int32_t* first;       // [T * top + 1] their first places
  int32_t* count;       // [1] how many experts have picks
  void* h;              // [T * top][F] in the operands' type
  float* out;           // [T * top][D]
};

template <typename T>
hipError_t launch_gate(const ExpertArgs& p, hipStream_t s);
hipError_t launch_expert_lists(const ExpertArgs& p, hipStream_t s);
template <typename T>
hipError_t launch_experts(int act, const ExpertArgs& p, hipStream_t s);

}  // namespace gmm
