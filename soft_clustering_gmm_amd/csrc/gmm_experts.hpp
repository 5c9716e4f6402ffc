// Internal declarations of the layer of experts (gmm_expert_layer, gmm_expert_rows).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gmm {

constexpr int kMaxLayerRows = 128;  // rows of one call
constexpr int kMaxTop = 8;          // picks per row
constexpr int kMaxPicks = kMaxLayerRows * kMaxTop;
// Up to so many picks the second product gathers a row's experts itself, as
// the columns of one matrix instruction (one row of 2 picks, D 4096, F 1408: 6.6
// us against 6.7 and 3.1 for the product by expert and the sum; 16 rows of 2,
// D 2048, F 1024: 23.7 us against 16.0 and 3.9).
constexpr int kGatherPicks = 8;
constexpr int kScoresInLds = 4096;  // components whose scores the gate keeps on chip
constexpr int kGateParts = 8;       // parts of the features' contraction

// Entries of ExpertArgs::count: experts with picks, picks in the lists, rows
// whose gate is done.
enum { kExperts = 0, kPlaces = 1, kRowsDone = 2, kCounts = 3 };

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
  const float* in_wts;  // combination weights
  // experts
  const void *W1, *b1, *W2, *b2;
  // workspace
  double* feats;        // [kGateParts][T][d]
  double* consts;       // [K]
  double* scores;       // [T][K], K > kScoresInLds
  float* wts;           // [T][top] combination weights of the gate
  int32_t* bad;         // [T] rows whose gate is not a number
  int32_t* place;       // [T * top] place of a pick in the order by expert, -1: none
  int32_t* row_of;      // [T * top] row of the pick at a place
  int32_t* ord;         // [T * top] which of the experts with picks the place belongs to
  float* weight;        // [T * top] combination weight of the pick at a place
  float* scale;         // [T] largest weight of a row, repeats added (1 if that is 0)
  int32_t* expert;      // [T * top] experts with picks, increasing
  int32_t* first;       // [T * top + 1] their first places
  int32_t* count;       // [kCounts]
  void* h;              // [T * top][F] in the operands' type
  float* out;           // [T * top][D], more than kGatherPicks picks
};

template <typename T>
hipError_t launch_gate(const ExpertArgs& p, hipStream_t s);
hipError_t launch_expert_lists(const ExpertArgs& p, hipStream_t s);
template <typename T>
hipError_t launch_experts(int act, const ExpertArgs& p, hipStream_t s);

}  // namespace gmm
