// The layer of experts' kernels for float operands, and those that do not
// depend on the element type: the gate's picks and the lists of picks.
#include <climits>

#include "gmm_experts_kernels.hpp"

namespace gmm {
GMM_EXPERTS_TYPE(float)

struct Best {
  double s;
  int k;
};
__device__ __forceinline__ bool better(double s, int k, const Best& b) { return s > b.s || (s == b.s && k < b.k); }

struct ListScratch {
  int key[kMaxPicks];   // expert * kMaxPicks + number of a listed pick, INT_MAX: none
  int idx[kMaxPicks];
  float wts[kMaxPicks];
  float sum[kMaxPicks];  // of a listed pick and its repeats
  int head[kMaxPicks + 1];  // by place: the expert of the pick, INT_MAX behind the last
  int waves[16];
};

// The picks in the order of their experts (a pick's place: how many picks have
// a lower expert, or the same and a lower number), and each expert's places.
// A row's further picks of an expert that it has picked already add their
// weight to the first; the row's scale is the largest of these sums, so that no
// weight is more than 1 of it. A thread a pick, with its expert and weight (-1
// behind the last); ONE: at most 64 picks, and only the first wave calls.
template <bool ONE>
__device__ __forceinline__ void expert_lists(const ExpertArgs& p, ListScratch& l, int idx, float wt) {
  static_assert(65536ll * kMaxPicks < INT_MAX, "keys fit");
  const int n = p.T * p.top, i = threadIdx.x, row = i / p.top;
  auto sync = [] {
    if (ONE)
      wave_lds_order();
    else
      __syncthreads();
  };
  l.idx[i] = idx;
  l.wts[i] = wt;
  l.head[i] = INT_MAX;
  if (i == 0) l.head[ONE ? 64 : kMaxPicks] = INT_MAX;
  sync();
  int mine = INT_MAX;
  float w = 0.f, most = 0.f;
  if (idx >= 0 && idx < p.K) {
    mine = idx * kMaxPicks + i;
    for (int q = row * p.top; q < (row + 1) * p.top; ++q)
      if (l.idx[q] == idx) {
        if (q < i) mine = INT_MAX;
        if (q >= i) w += l.wts[q];
      }
  }
  l.key[i] = mine;
  l.sum[i] = w;
  sync();
  const bool some = mine != INT_MAX;
  if (i < n) {
    int place = 0;
    for (int q = 0; q < n; q += 4) {  // key[] is INT_MAX behind n
      const int4 v = *reinterpret_cast<const int4*>(l.key + q);
      place += (v.x < mine) + (v.y < mine) + (v.z < mine) + (v.w < mine);
    }
    p.place[i] = some ? place : -1;
    if (some) {
      l.head[place] = idx;
      p.row_of[place] = row;
      p.weight[place] = w;
    }
  }
  if (i < p.T) {
    for (int q = i * p.top; q < (i + 1) * p.top; ++q)
      if (l.key[q] != INT_MAX) most = fmaxf(most, fabsf(l.sum[q]));
    p.scale[i] = most > 0.f ? most : 1.f;
  }
  sync();
  // the first place of every expert, numbered by a scan over the places
  const int e = l.head[i];
  const bool start = e != INT_MAX && (i == 0 || l.head[i - 1] != e);
  const uint64_t starts = __ballot(start);
  const int lane = i & 63, wave = i >> 6;
  int before = 0, total = __popcll(starts);
  if (!ONE) {
    if (lane == 0) l.waves[wave] = total;
    __syncthreads();
    total = 0;
    for (int v = 0; v < 16; ++v) {
      if (v < wave) before += l.waves[v];
      total += l.waves[v];
    }
  }
  const int a = before + __popcll(starts & (~0ull >> (63 - lane))) - 1;
  if (e != INT_MAX) p.ord[i] = a;
  if (start) {
    p.expert[a] = e;
    p.first[a] = i;
  }
  // the picks end where the INT_MAX begin
  if (e != INT_MAX && l.head[i + 1] == INT_MAX) {
    p.first[total] = i + 1;
    p.count[kPlaces] = i + 1;
  }
  if (i == 0) {
    p.count[kExperts] = total;
    if (total == 0) p.count[kPlaces] = 0;
  }
}

__global__ void __launch_bounds__(1024) expert_lists_kernel(const ExpertArgs p) {
  __shared__ __align__(16) ListScratch l;
  const int i = threadIdx.x, n = p.T * p.top;
  if (n <= 64 && i >= 64) return;
  const int idx = i < n ? p.in_idx[i] : -1;
  const float wt = i < n ? p.in_wts[i] : 0.f;
  if (n <= 64)
    expert_lists<true>(p, l, idx, wt);
  else
    expert_lists<false>(p, l, idx, wt);
}

// 1 / v: the hardware's estimate and two Newton steps (the estimate has 2^-14
// or better, so the result is rounded nearly as a division's). 0 and infinity
// keep the estimate, whose steps would be 0 times infinity.
__device__ __forceinline__ double reciprocal(double v) {
  const double y0 = __builtin_amdgcn_rcp(v);
  double y = fma(fma(-v, y0, 1.), y0, y0);
  y = fma(fma(-v, y, 1.), y, y);
  return y == y ? y : y0;
}

// Scores of one row against all components, its picks, and, in the block that
// is done last, the lists. Sixteen lanes score a component, up to 8 features
// each.
//
// The picks of up to kRanked components are found by rank: all threads share
// the comparisons of every component with every other (K^2 / 1024 each), and
// a component's rank, how many come before it (score down, index up), says
// which pick it is. More components are picked one after the other, each pick
// the best of those after the last.
//
// One block a row is latency from end to end: for one row of 64 components
// (64 features, 2 picks) 13 us with the constants computed here, the maxima
// found by shuffles and the lists behind an acquire of the whole L2, 7 us so.
__global__ void __launch_bounds__(1024) gate_pick_kernel(const ExpertArgs p) {
  constexpr int NW = 16, kPerLane = 8, kRanked = 512;
  __shared__ __align__(16) union {
    double scores[kScoresInLds];
    ListScratch lists;
  } sh;
  __shared__ double feat[128];
  __shared__ Best wave_best[NW];
  __shared__ double wave_sum[NW], pick_s[kMaxTop];
  __shared__ int odd, last_block, pick_k[kMaxTop], rank[kRanked];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, t = blockIdx.x, l16 = lane & 15;
  double* sc = p.K <= kScoresInLds ? sh.scores : p.scores + (int64_t)t * p.K;
  if (tid == 0) odd = 0;
  if (tid < kRanked) rank[tid] = 0;
  if (tid < kMaxTop) pick_s[tid] = -INFINITY;
  double part[kGateParts];
  if (tid < p.d) {
#pragma unroll
    for (int i = 0; i < kGateParts; ++i) part[i] = p.feats[((int64_t)i * p.T + t) * p.d + tid];
  }
  float m[kPerLane], v[kPerLane];
  double c = 0.;
  auto load = [&](int k) {
    const float *mu = p.mu + (int64_t)k * p.d, *var = p.var + (int64_t)k * p.d;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int j = min(l16 + 16 * i, p.d - 1);
      m[i] = mu[j];
      v[i] = var[j];
    }
    c = p.consts[k];
  };
  const int k0 = wave * 4 + (lane >> 4);
  if (k0 < p.K) load(k0);  // on its way while the features are added up
  if (tid < p.d) {
    double sum = 0.;
#pragma unroll
    for (int i = 0; i < kGateParts; ++i) sum += part[i];
    feat[tid] = sum;
  }
  __syncthreads();
  double x[kPerLane];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) x[i] = feat[min(l16 + 16 * i, p.d - 1)];
  for (int k = k0; k < p.K; k += 4 * NW) {
    double q = 0.;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (l16 + 16 * i < p.d) {
        const double u = x[i] - m[i];
        q = fma(u * u, reciprocal(v[i]), q);
      }
    const double ck = c;
    if (k + 4 * NW < p.K) load(k + 4 * NW);
#pragma unroll
    for (int o = 8; o; o >>= 1) q += __shfl_xor(q, o);
    if (l16 == 0) {
      const double s = ck - 0.5 * q;
      sc[k] = s;
      if (!(s < INFINITY)) odd = 1;  // NaN or +inf: the posterior is not a number
    }
  }
  __threadfence_block();
  __syncthreads();

  double top_s, sum = 0.;
  if (p.K <= kRanked) {
    // threads (k, part): k compared with every parts-th component
    int width = 64;
    while (width < p.K) width *= 2;
    const int parts = 64 * NW / width, k = tid & (width - 1), first = tid / width;
    const double s = k < p.K ? sc[k] : 0.;
    if (k < p.K) {
      int before = 0;
#pragma unroll 4
      for (int o = first; o < p.K; o += parts) {
        const double so = sc[o];
        before += so > s || (so == s && o < k);
      }
      atomicAdd(&rank[k], before);
    }
    __syncthreads();
    if (first == 0 && k < p.K) {
      const int r = rank[k];
      if (r < p.top) {
        pick_s[r] = s;
        pick_k[r] = k;
      }
    }
    __syncthreads();
    top_s = pick_s[0];
    if (tid < width) {  // whole waves
      double z = k < p.K ? exp(s - top_s) : 0.;
#pragma unroll
      for (int o = 32; o; o >>= 1) z += __shfl_xor(z, o);
      if (lane == 0) wave_sum[wave] = z;
    }
    __syncthreads();
    for (int w = 0; w < width / 64; ++w) sum += wave_sum[w];
  } else {
    Best last{INFINITY, -1};
    for (int pick = 0; pick < p.top; ++pick) {
      Best b{-INFINITY, INT_MAX};
      for (int k = tid; k < p.K; k += 64 * NW) {
        const double s = sc[k];
        // after the last pick
        if ((s < last.s || (s == last.s && k > last.k)) && better(s, k, b)) b = Best{s, k};
      }
#pragma unroll
      for (int o = 32; o; o >>= 1) {
        const double s = __shfl_xor(b.s, o);
        const int k = __shfl_xor(b.k, o);
        if (better(s, k, b)) b = Best{s, k};
      }
      if (lane == 0) wave_best[wave] = b;
      __syncthreads();
      b = wave_best[0];
      for (int w = 1; w < NW; ++w)
        if (better(wave_best[w].s, wave_best[w].k, b)) b = wave_best[w];
      __syncthreads();
      if (tid == 0 && b.k != INT_MAX) {
        pick_s[pick] = b.s;
        pick_k[pick] = b.k;
      }
      last = b;
    }
    __syncthreads();
    top_s = pick_s[0];
    double z = 0.;
    for (int k = tid; k < p.K; k += 64 * NW) z += exp(sc[k] - top_s);
#pragma unroll
    for (int o = 32; o; o >>= 1) z += __shfl_xor(z, o);
    if (lane == 0) wave_sum[wave] = z;
    __syncthreads();
    for (int w = 0; w < NW; ++w) sum += wave_sum[w];
  }

  int idx = -1;
  float wt = 0.f;
  if (wave == 0) {  // a lane per pick
    const bool bad = odd || !(top_s > -INFINITY);
    // components of weight zero (score -inf) are no picks
    const double s = lane < p.top && !bad ? pick_s[lane] : -INFINITY;
    const double r = s > -INFINITY ? exp(s - top_s) / sum : 0.;
    const bool keep = s > -INFINITY && (lane == 0 || r >= (double)p.threshold);
    double kept = keep ? r : 0.;
#pragma unroll
    for (int o = kMaxTop / 2; o; o >>= 1) kept += __shfl_xor(kept, o);
    if (keep) {
      idx = pick_k[lane];
      wt = (float)(p.renorm ? r / kept : r);
    }
    if (lane < p.top) {
      const int at = t * p.top + lane;
      p.idx[at] = idx;
      p.resp[at] = (float)(keep ? r : 0.);
      p.wts[at] = wt;
    }
    if (lane == 0) p.bad[t] = bad;
    // The block that counts the last row lists the picks of all.
    if (p.T > 1) {
      __threadfence();
      if (lane == 0) last_block = atomicAdd(p.count + kRowsDone, 1) == p.T - 1;
    }
  }
  const int n = p.T * p.top;
  __syncthreads();  // the scores' memory is free
  if ((p.T > 1 && !last_block) || (n <= 64 && wave > 0)) return;
  if (p.T > 1) {  // past the caches, as other blocks wrote them
    idx = tid < n ? __hip_atomic_load(p.in_idx + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : -1;
    wt = tid < n ? __hip_atomic_load(p.in_wts + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.f;
  }
  if (n <= 64)
    expert_lists<true>(p, sh.lists, idx, wt);
  else
    expert_lists<false>(p, sh.lists, idx, wt);
}

hipError_t launch_gate_picks(const ExpertArgs& p, hipStream_t s) {
  gate_pick_kernel<<<p.T, 1024, 0, s>>>(p);
  return hipGetLastError();
}

hipError_t launch_expert_lists(const ExpertArgs& p, hipStream_t s) {
  expert_lists_kernel<<<1, 1024, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace gmm
