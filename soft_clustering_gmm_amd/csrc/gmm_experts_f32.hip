// The layer of experts' kernels for float operands, and the lists of picks,
// which do not depend on the element type.
#include <climits>

#include "gmm_experts_kernels.hpp"

namespace gmm {
GMM_EXPERTS_TYPE(float)

// The picks in the order of their experts (a pick's place: how many picks have
// a lower expert, or the same and a lower number), and each expert's places.
__global__ void __launch_bounds__(1024) expert_lists_kernel(const ExpertArgs p) {
  constexpr int kMost = kMaxLayerRows * kMaxTop;
  __shared__ __align__(16) int key[kMost];
  __shared__ int head[kMost];  // by place: the expert of the pick, INT_MAX behind the last
  __shared__ int waves[16];
  const int n = p.T * p.top, i = threadIdx.x;
  int mine = INT_MAX;
  if (i < n) {
    const int k = p.in_idx[i];
    if (k >= 0 && k < p.K) mine = k;
  }
  key[i] = mine;
  head[i] = INT_MAX;
  __syncthreads();
  int place = 0;
  for (int q = 0; q < n; q += 4) {  // key[] is INT_MAX behind n
    const int4 v = *reinterpret_cast<const int4*>(key + q);
    place += (v.x < mine || (v.x == mine && q < i)) + (v.y < mine || (v.y == mine && q + 1 < i)) +
             (v.z < mine || (v.z == mine && q + 2 < i)) + (v.w < mine || (v.w == mine && q + 3 < i));
  }
  const bool some = mine != INT_MAX;
  if (i < n) p.place[i] = some ? place : -1;
  if (some) {
    head[place] = mine;
    p.row_of[place] = i / p.top;
  }
  __syncthreads();
  // the first place of every expert, numbered by a scan over the places
  const int e = head[i];
  const bool start = e != INT_MAX && (i == 0 || head[i - 1] != e);
  const uint64_t starts = __ballot(start);
  const int lane = i & 63, wave = i >> 6;
  if (lane == 0) waves[wave] = __popcll(starts);
  __syncthreads();
  int before = 0, total = 0;
  for (int w = 0; w < 16; ++w) {
    if (w < wave) before += waves[w];
    total += waves[w];
  }
  if (start) {
    const int a = before + __popcll(starts & ((1ull << lane) - 1));
    p.expert[a] = e;
    p.first[a] = i;
  }
  // the picks end where the INT_MAX begin
  if (e != INT_MAX && (i == kMost - 1 || head[i + 1] == INT_MAX)) p.first[total] = i + 1;
  if (i == 0) *p.count = total;
}

hipError_t launch_expert_lists(const ExpertArgs& p, hipStream_t s) {
  expert_lists_kernel<<<1, 1024, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace gmm
