// Kernels of the linear layer, instantiated once per element type
// (gmm_linear_f32.hip, gmm_linear_f16.hip, gmm_linear_bf16.hip).
#pragma once

#include <cfloat>
#include <type_traits>

#include "gmm_linear.hpp"
#include "gmm_product.hpp"

namespace gmm {

typedef __attribute__((address_space(3))) void* lds_ptr;

__device__ __forceinline__ lds_ptr to_lds(const void* p) {
  return reinterpret_cast<lds_ptr>(reinterpret_cast<uintptr_t>(p));
}

// ---------------------------------------------------------------------------
// Tiled product. A block computes a BM x BN tile of C with WM x WN waves; a
// step of the contraction brings kStepBytes of k of both operands into one of
// two slots of LDS, by loads that go to LDS directly. A's tile is two halves of
// rows, and every wave owns rows in both.
//
// A step has four phases (half of A, half of k), and the fragments of the next
// phase are read from LDS between the matrix instructions of the present one:
//   phase 0: multiply A0, first k;   read A0 and B, second k
//   barrier: A1 of this step has arrived; A0 and B are read out -> load theirs
//            of step s + 2
//   phase 1: multiply A0, second k;  read A1, first k
//   phase 2: multiply A1, first k;   read A1, second k
//   barrier: A0 and B of the next step have arrived; A1 is read out -> load it
//   phase 3: multiply A1, second k;  read A0 and B, first k, of the next step
// A load so has one and a half steps to arrive. That is what bounds the large
// shapes: with one step (both barriers in one place) the loads alone took 692 us
// at 8192 x 16384 x 4096 in bfloat16, the matrix instructions alone 535 and the
// LDS reads alone 430; with two steps in flight and 4 tile rows side by side
// instead of 8 the loads took 546.
//
// The matrix instruction gets B's rows (n) as its first operand and A's rows
// (m) as its second, so a lane's results are 4 consecutive n of one m.
//
// LDS layouts, in 16-byte chunks, the chunk's place XORed with a key of its
// row so that the fragment reads of a wave spread over the banks:
//   k-contiguous: [row][8 chunks of k], key from the row;
//   k-strided:    [k][BR / kPer chunks of rows], key from k.
// ---------------------------------------------------------------------------

typedef int i32x4 __attribute__((ext_vector_type(4)));

// One kilobyte per wave, 16 bytes a lane, from a buffer straight into LDS at
// `lds` (the same for the whole wave); offsets past the buffer's end give
// zeros. Written out because the compiler makes every transposing LDS read
// wait for such loads in flight, which would undo the double buffering; the
// kernel's own waits are in step_barrier(). Nothing is returned in registers.
// The wait states cover M0, and a buffer word that a vector instruction wrote.
__device__ __forceinline__ void load_to_lds(uint32_t lds, uint32_t offset, i32x4 buffer) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(offset), "s"(buffer)
               : "m0");
}

// All but the last PENDING loads of this wave have arrived in LDS and its LDS
// reads are done; then the block's barrier. `lds` ties the tiles' memory to it.
template <int PENDING>
__device__ __forceinline__ void step_barrier(const void* lds) {
  asm volatile("s_waitcnt vmcnt(%1) lgkmcnt(0)\n\ts_barrier" : : "v"(to_lds(lds)), "n"(PENDING) : "memory");
}

template <typename T, int BR, int NWAVES, bool STRIDED>
struct Operand {
  static constexpr int kPer = Frag<T>::kPer;
  static constexpr int kStep = kStepBytes / (int)sizeof(T);  // k per step
  static constexpr int kBytes = BR * kStepBytes;
  static constexpr int kLoads = kBytes / 1024 / NWAVES;  // wave loads of 1 KB
  static constexpr int kRowChunks = BR * (int)sizeof(T) / 16;  // k-strided: chunks per k

  uintptr_t base;        // element (first row of the tile, first k of the part)
  int64_t step_bytes;    // from one step to the next
  int64_t left;          // bytes from base to the end of the operand's rows (of the part's k)
  int rows_left;         // k-strided: elements from the tile's first row to the end of a k
  uint32_t off[kLoads];  // byte offset of this lane's chunk from base
  static constexpr uint32_t kNowhere = 0x80000000u;  // beyond any buffer: zeros

  // Key of a k-strided tile's k. A k is 64, 128, 256 or 512 bytes; what 32 lanes
  // read at once should be 256 different bytes of the banks' 256.
  // 2-byte elements (transposing reads): 32 bytes of each of k = 0..3 and 8..11.
  // 4-byte elements: 64 bytes of each of k = 0, 4, 8, 12.
  static __device__ __forceinline__ int key(int k) {
    if (sizeof(T) == 4) return kRowChunks >= 16 ? (k & 12) : (k & 4);
    if (kRowChunks >= 16) return ((k & 3) << 1) | (k & 8);
    if (kRowChunks == 8) return (k & 2) | ((k & 8) >> 1);
    return (k & 8) >> 2;
  }

  // First k, within the step, of the chunk that this lane brings in load j.
  static __device__ __forceinline__ int chunk_k(int j, int wave, int lane) {
    const int ch = (wave * kLoads + j) * 64 + lane;
    if (STRIDED) return ch / kRowChunks;
    const int r = ch / 8;
    return ((ch % 8) ^ (r & 7)) * kPer;
  }

  // The same for its first row (k-strided).
  static __device__ __forceinline__ int chunk_row(int j, int wave, int lane) {
    const int ch = (wave * kLoads + j) * 64 + lane;
    return ((ch % kRowChunks) ^ key(ch / kRowChunks)) * kPer;
  }

  __device__ __forceinline__ void init(const void* p, int64_t ld, int64_t r0, int64_t rows, int64_t k0, int64_t k1,
                                       int wave, int lane) {
    const int e = sizeof(T);
    if (STRIDED) {
      base = reinterpret_cast<uintptr_t>(p) + (k0 * ld + r0) * e;
      step_bytes = kStep * ld * e;
      left = ((k1 - k0) * ld - r0) * e;
      rows_left = (int)(ld - r0);
    } else {
      base = reinterpret_cast<uintptr_t>(p) + (r0 * ld + k0) * e;
      step_bytes = kStepBytes;
      left = ((rows - r0) * ld - k0) * e;
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int ch = (wave * kLoads + j) * 64 + lane;  // chunk of the tile in LDS order
      if (STRIDED) {
        off[j] = (uint32_t)(ch / kRowChunks * ld * e + chunk_row(j, wave, lane) * e);
      } else {
        off[j] = (uint32_t)((ch / 8) * ld * e + chunk_k(j, wave, lane) * e);
      }
    }
  }

  // Loads of step `step` of the part, of whose k `k_left` remain, from row
  // `skip` of the tile on (its other half), `ahead` bytes further. What is read
  // is inside the operand: k is held to k_left and the rows of a k-strided one
  // to rows_left; a k-contiguous one's rows past the last are beyond the buffer,
  // whose size is that seen from step 0.
  __device__ __forceinline__ void load(uint32_t lds, int step, int k_left, int wave, int lane, int skip,
                                       int64_t ahead) const {
    const uintptr_t b = base + step * step_bytes + ahead;
    const int64_t n = left - ahead;
    i32x4 buffer;
    buffer[0] = (int)(uint32_t)b;
    buffer[1] = (int)((uint32_t)(b >> 32) & 0xffff);
    buffer[2] = n < 0 ? 0 : n > 0x7fffffff ? 0x7fffffff : (int)n;
    buffer[3] = 0x00027000;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const bool inside = chunk_k(j, wave, lane) < k_left && (!STRIDED || chunk_row(j, wave, lane) < rows_left - skip);
      load_to_lds(lds + (wave * kLoads + j) * 1024, inside ? off[j] : kNowhere, buffer);
    }
  }

  // Fragment of the 16 rows of tile i (of a wave whose rows start at w0), k
  // chunks 4 kk + l / 16 of the step.
  static __device__ __forceinline__ u32x4 frag(const char* lds, int w0, int i, int kk, int lane) {
    const int r = lane & 15, g = lane >> 4;
    if (!STRIDED) {
      const int row = w0 + 16 * i + r;
      const int c = (4 * kk + g) ^ (row & 7);
      return *reinterpret_cast<const u32x4*>(lds + row * kStepBytes + 16 * c);
    }
    if constexpr (sizeof(T) == 4) {
      const int row = w0 + 16 * i + r;
      u32x4 v;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = 16 * kk + 4 * g + q;
        const int c = (row >> 2) ^ key(k);
        v[q] = *reinterpret_cast<const uint32_t*>(lds + (k * kRowChunks + c) * 16 + 4 * (row & 3));
      }
      return v;
    } else {
      // Two transposing reads: over 16 lanes, lane t gives the address of 4
      // consecutive rows of k = t / 4, and receives 4 consecutive k of row t.
      const int row = w0 + 16 * i + 4 * (r & 3);
      u32x4 v;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 32 * kk + 8 * g + 4 * h + (r >> 2);
        const int c = (row >> 3) ^ key(k);
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)to_lds(lds + (k * kRowChunks + c) * 16 + 2 * (row & 7)));
        const uint2 y = __builtin_bit_cast(uint2, x);
        v[2 * h] = y.x;
        v[2 * h + 1] = y.y;
      }
      return v;
    }
  }
};

// The residual of W consecutive n of one row, where there is one.
template <typename T, int W>
__device__ __forceinline__ void load_residual(const ProductArgs& p, int64_t m, int n, float* res) {
  if (p.residual) load_row<T, W>(p.residual, m * p.ldc + n, p.N - n, p.c_f32 | p.res_f32, res);
}

// z + bias -> pre, act(.) + residual -> C for W consecutive n of one row.
template <typename T, int ACT, int W>
__device__ __forceinline__ void finish_row(const ProductArgs& p, int64_t m, int n, float* z, const float* bias,
                                           const float* res) {
  const int64_t at = m * p.ldc + n;
  const int left = p.N - n;
#pragma unroll
  for (int i = 0; i < W; ++i) z[i] += bias[i];
  if constexpr (ACT == kLogitGradient) {
    RowCoef c;
    __builtin_memcpy(&c, res, sizeof(c));
    float g[W];
    logit_gradient<W>(c, p.picks, m, n, p.N, z, g);
    if (p.c_stream)
      store_as<T, W, true>(static_cast<T*>(p.C) + at, W, g);
    else
      store_as<T, W>(static_cast<T*>(p.C) + at, W, g);
#pragma unroll
    for (int i = 0; i < W; ++i) z[i] = (float)(T)g[i];  // for the column sums
    return;
  }
  if (p.pre) store_row<T, W>(p.pre, at, left, p.c_f32, z);
#pragma unroll
  for (int i = 0; i < W; ++i) z[i] = act_value<ACT>(z[i]);
  if (p.residual)
#pragma unroll
    for (int i = 0; i < W; ++i) z[i] += res[i];
  if (p.c_stream)
    store_row<T, W, true>(p.C, at, left, p.c_f32, z);
  else
    store_row<T, W>(p.C, at, left, p.c_f32, z);
}

// A block's tile and part of the contraction. Tiles go in groups of 4 tile
// rows, column by column within a group, so that the blocks an XCD runs
// together share rows of A and of B in its L2.
struct Place {
  int part, n0;
  int64_t m0, k0, k1;
};
__device__ __forceinline__ Place tile_place(const ProductArgs& p, int bm, int bn) {
  const int tiles = p.tiles_m * p.tiles_n;
  Place at;
  at.part = blockIdx.x / tiles;
  const int t = xcd_place(blockIdx.x - at.part * tiles, tiles);
  constexpr int G = 4;
  const int group = t / (G * p.tiles_n), first = group * G;
  const int height = min(G, p.tiles_m - first), in = t - group * G * p.tiles_n;
  at.m0 = (int64_t)(first + in % height) * bm;
  at.n0 = in / height * bn;
  at.k0 = at.part * p.split_k;
  at.k1 = min(p.K, at.k0 + p.split_k);
  return at;
}

// Column sums: kSumCols columns a block, kSumSlices rows at a time by its first
// 256 threads, in the same order whatever kernel they ride in.
constexpr int kSumSlices = 256 / kSumCols;
template <typename T>
__device__ __forceinline__ void column_sums(const ProductArgs& p, int block, float (*red)[kSumCols + 1]) {
  const int x = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
  const int c = block * kSumCols + x;
  if (y < kSumSlices) {
    float sum = 0.f;
    if (c < p.sums_cols) {
#pragma unroll 8
      for (int64_t i = y; i < p.sums_rows; i += kSumSlices) sum += p.sums[i * p.sums_cols + c];
    }
    red[y][x] = sum;
  }
  __syncthreads();
  if (y == 0 && c < p.sums_cols) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kSumSlices; ++i) sum += red[i][x];
    static_cast<T*>(p.sums_out)[c] = (T)sum;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) column_sums_kernel(const ProductArgs p) {
  __shared__ float red[kSumSlices][kSumCols + 1];
  column_sums<T>(p, blockIdx.x, red);
}

// The logits of the rows' picks in a wave's TI x NI tiles: whichever lane has one
// writes it. The same float that the statistics are taken of, so that no pick's
// lies above its row's largest. `mine` are the picks of the tile's rows from m0 on.
// Most waves have none, so all rows are looked at first.
template <int TI, int NI, typename F>
__device__ __forceinline__ void store_picks(const ProductArgs& p, const f32x4 (*acc)[NI], const float (*bias)[4],
                                            F&& first_row, const int* mine, int64_t m0, int n0, int lane) {
  const int top = p.picks.top, n = n0 + 4 * (lane >> 4);  // this lane's columns are n + 16 j + q
  for (int k = 0; k < top; ++k) {
    bool some = false;
#pragma unroll
    for (int r = 0; r < 16 * TI; r += 64) {
      const int i = r / 16 + lane / 16;
      if (i < TI) {
        const int v = mine[((int)(first_row(i) - m0) + (lane & 15)) * top + k];
        some |= v >= n0 && v < min(p.N, n0 + 16 * NI);
      }
    }
    if (!__any(some)) continue;
    int v[TI];
#pragma unroll
    for (int i = 0; i < TI; ++i) v[i] = mine[((int)(first_row(i) - m0) + (lane & 15)) * top + k];
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int d = v[i] - n;
      if (v[i] < p.N && (unsigned)d < 16u * NI && (d & 12) == 0) {
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (d == 16 * j + q) z = acc[i][j][q] + bias[j][q];
        p.picked[(first_row(i) + (lane & 15)) * top + k] = z;
      }
    }
  }
}

// The statistics of a wave's TI x NI tiles, straight from the registers: a lane
// has 4 NI columns of a row, which 4 lanes share. KEEP: acc becomes kKeptOne
// exp(z - the largest of its row).
template <typename T, int TI, int NI, bool KEEP, bool PICKS, typename F>
__device__ __forceinline__ void row_stats(const ProductArgs& p, f32x4 (*acc)[NI], F&& first_row, const int* picks,
                                          int64_t m0, int n0, int group, int groups, int lane) {
  constexpr float kInf = __builtin_inff();
  float bias[NI][4];
#pragma unroll
  for (int j = 0; j < NI; ++j) {
    const int n = n0 + 16 * j + 4 * (lane >> 4);
    if (p.bias)
      load_as<T, 4>(static_cast<const T*>(p.bias) + n, p.N - n, bias[j]);
    else
#pragma unroll
      for (int q = 0; q < 4; ++q) bias[j][q] = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q >= p.N) bias[j][q] = -kInf;  // the products there are 0
  }
  if (PICKS && p.picked) store_picks<TI, NI>(p, acc, bias, first_row, picks, m0, n0, lane);
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    float most = -kInf, z[NI][4], sum = 0.f;
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        z[j][q] = acc[i][j][q] + bias[j][q];
        most = fmaxf(most, z[j][q]);
      }
    most = fmaxf(most, __shfl_xor(most, 16));
    most = fmaxf(most, __shfl_xor(most, 32));
    const float base = most == -kInf ? 0.f : most;
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float e = exp_of(z[j][q] - base);
        sum += e;
        if (KEEP) acc[i][j][q] = kKeptOne * e;
      }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    const int64_t m = first_row(i) + (lane & 15);
    if (lane < 16 && m < p.M) {
      float* out = p.stats + 2 * (m * groups + group);
      out[0] = most;
      out[1] = sum;
    }
  }
}

// Logits that leave as their exponentials over their row's largest, in half.
template <typename T, int ACT>
constexpr bool kKept = ACT == kStatsToo && sizeof(T) == 2;

// Products that may be unscaled: the gradients' of 2-byte operands (B k-strided).
template <typename T, bool BS>
constexpr bool kScaled = BS && sizeof(T) == 2;

template <typename T, int BM, int BN, int WM, int WN, bool AS, bool BS, int ACT>
__global__ void __launch_bounds__(64 * WM * WN, 2)
product_kernel(const ProductArgs p) {
  constexpr int NW = WM * WN, HM = BM / 2, TM = HM / WM, TN = BN / WN, MI = TM / 16, NI = TN / 16;
  using OA = Operand<T, HM, NW, AS>;
  using OB = Operand<T, BN, NW, BS>;
  constexpr int kSlot = 2 * OA::kBytes + OB::kBytes, kPending = 2 * OA::kLoads + OB::kLoads;
  __shared__ __align__(1024) char lds[2 * kSlot];
  constexpr bool kPicks = ACT == kRowStats || kKept<T, ACT>;  // float logits in memory hold them
  __shared__ int picks[kPicks ? BM * kMaxPicksRow : 1];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  if ((int)blockIdx.x >= p.tiles_m * p.tiles_n * p.splits) {
    column_sums<T>(p, blockIdx.x - p.tiles_m * p.tiles_n * p.splits, reinterpret_cast<float(*)[kSumCols + 1]>(lds));
    return;
  }
  const Place at = tile_place(p, BM, BN);
  const int64_t k0 = at.k0, k1 = at.k1;

  OA a;
  OB b;
  a.init(p.A, p.lda, at.m0, p.M, k0, k1, wave, lane);
  b.init(p.B, p.ldb, at.n0, p.N, k0, k1, wave, lane);

  f32x4 acc[2][MI][NI];
#pragma unroll
  for (int i = 0; i < 2 * MI * NI; ++i) (&acc[0][0][0])[i] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int k_all = (int)(k1 - k0);  // at most 2^30
  const int steps = (k_all + OA::kStep - 1) / OA::kStep;
  const int64_t half = (AS ? HM : HM * p.lda) * (int)sizeof(T);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)reinterpret_cast<uintptr_t>(to_lds(lds)));
  // Steps past the end bring zeros and no traffic, so that the number of loads
  // in flight is the same at every barrier.
  auto load_a = [&](int s, int h) {
    a.load(lds0 + (s & 1) * kSlot + h * OA::kBytes, s, k_all - s * OA::kStep, wave, lane, h * HM,
           h * half);
  };
  auto load_b = [&](int s) {
    b.load(lds0 + (s & 1) * kSlot + 2 * OA::kBytes, s, k_all - s * OA::kStep, wave, lane, 0, 0);
  };
  u32x4 fa[2][MI], fb[2][NI];  // by half of k
  auto read_a = [&](int s, int h, int kk) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
      fa[kk][i] = OA::frag(lds + (s & 1) * kSlot + h * OA::kBytes, wm * TM, i, kk, lane);
  };
  auto read_b = [&](int s, int kk) {
#pragma unroll
    for (int j = 0; j < NI; ++j) fb[kk][j] = OB::frag(lds + (s & 1) * kSlot + 2 * OA::kBytes, wn * TN, j, kk, lane);
  };
  // The multiplication of a phase, one of its reads after every few matrix instructions.
  constexpr int kPerA = !AS ? 1 : sizeof(T) == 4 ? 4 : 2, kPerB = !BS ? 1 : sizeof(T) == 4 ? 4 : 2;
  constexpr int kMma = MI * NI * (sizeof(T) == 4 ? 4 : 1);
  auto multiply = [&](int h, int kk, auto with_b) {
    Frag<T>::template mma_tiles<MI, NI>(fb[kk], fa[kk], acc[h]);
    constexpr int reads = MI * kPerA + (decltype(with_b)::value ? NI * kPerB : 0);
    constexpr int between = kMma / reads > 1 ? kMma / reads : 1;
#pragma unroll
    for (int i = 0; i < reads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, between, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // the rows' picks, for the end (asked for there, a tile of 256 rows took 1.1 us more)
  constexpr int kPickLoads = kPicks ? BM * kMaxPicksRow / (64 * NW) : 1;
  int pick[kPickLoads];
  if (kPicks && p.picked)
#pragma unroll
    for (int u = 0; u < kPickLoads; ++u) {
      const int i = u * 64 * NW + threadIdx.x;
      const int64_t in = at.m0 * p.picks.top + i;
      pick[u] = i < BM * p.picks.top && in < p.M * p.picks.top ? p.picks.idx[in] : -1;
    }
  load_a(0, 0), load_b(0), load_a(0, 1);
  load_a(1, 0), load_b(1), load_a(1, 1);
  step_barrier<kPending + OA::kLoads>(lds);
  read_a(0, 0, 0);
  read_b(0, 0);
  __builtin_amdgcn_sched_barrier(0);
  for (int s = 0; s < steps; ++s) {
    read_a(s, 0, 1);
    read_b(s, 1);
    multiply(0, 0, std::true_type{});
    step_barrier<kPending>(lds);
    load_a(s + 2, 0);
    load_b(s + 2);
    __builtin_amdgcn_sched_barrier(0);
    read_a(s, 1, 0);
    multiply(0, 1, std::false_type{});
    read_a(s, 1, 1);
    multiply(1, 0, std::false_type{});
    step_barrier<kPending>(lds);
    load_a(s + 2, 1);
    __builtin_amdgcn_sched_barrier(0);
    read_a(s + 1, 0, 0);  // after the last step: zeros, not used
    read_b(s + 1, 0);
    multiply(1, 1, std::true_type{});
  }
  if (kPicks && p.picked)
#pragma unroll
    for (int u = 0; u < kPickLoads; ++u)
      if (u * 64 * NW + (int)threadIdx.x < BM * p.picks.top) picks[u * 64 * NW + threadIdx.x] = pick[u];
  step_barrier<0>(lds);  // nobody reads the slots, and nothing arrives in them any more
  if constexpr (ACT == kRowStats || ACT == kStatsToo)
    row_stats<T, 2 * MI, NI, kKept<T, ACT>, kPicks>(
        p, acc[0], [&](int i) { return at.m0 + i / MI * HM + wm * TM + 16 * (i % MI); }, picks, at.m0, at.n0 + wn * TN,
        at.n0 / BN * WN + wn, p.tiles_n * WN, lane);
  if constexpr (ACT == kRowStats) return;

  // The results go through LDS, 16 rows of m at a time in memory of the wave's
  // own, so that neighbouring lanes access one row: whole lines for C, residual
  // and pre. Straight from the registers, 16 n of a row per lane, the product
  // to 96 float columns (262144 x 1024 rows) took 152 us, so 141; a bfloat16 one
  // with no residual is 2% slower this way (8192 x 16384: 921 against 940).
  // Padded rows spread the writes over the banks.
  constexpr int W = Frag<T>::kPer;  // n of a lane: 16 bytes of the operands' type
  constexpr int kRow = TN * 4 + 16, kChunks = TN / W, kRows = 64 / kChunks, Q = 16 / kRows;
  static_assert(NW * 16 * kRow <= 2 * kSlot, "fits the slots");
  char* mine = lds + wave * 16 * kRow;
  const int n = at.n0 + wn * TN + lane % kChunks * W;
  const bool whole = p.splits == 1;
  const float unscale = kScaled<T, BS> && whole && p.unscale ? *p.unscale : 1.f;
  float bias[W];
#pragma unroll
  for (int i = 0; i < W; ++i) bias[i] = 0.f;
  if (whole && p.bias && n < p.N && !kKept<T, ACT>) load_as<T, W>(static_cast<const T*>(p.bias) + n, p.N - n, bias);
  // The next 16 rows' residual is on its way while these are finished: C may be
  // the residual, so the compiler keeps a load behind the stores before it.
  constexpr int R = ACT == kLogitGradient ? sizeof(RowCoef) / 4 : W;  // or the row's coefficients in its place
  float res[2][Q][R];
  auto row_of = [&](int i, int q) {
    return at.m0 + i / MI * HM + wm * TM + 16 * (i % MI) + q * kRows + lane / kChunks;
  };
  auto fetch = [&](int i) {
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (whole && row_of(i, q) < p.M && n < p.N) {
        if constexpr (ACT == kLogitGradient)
          load_as<float, R>(reinterpret_cast<const float*>(p.coef + row_of(i, q)), R, res[i & 1][q]);
        else
          load_residual<T, W>(p, row_of(i, q), n, res[i & 1][q]);
      }
  };
  fetch(0);
  float cols[W];
#pragma unroll
  for (int i = 0; i < W; ++i) cols[i] = 0.f;
#pragma unroll
  for (int i = 0; i < 2 * MI; ++i) {
    if (i + 1 < 2 * MI) fetch(i + 1);
#pragma unroll
    for (int j = 0; j < NI; ++j)
      *reinterpret_cast<f32x4*>(mine + (lane & 15) * kRow + 64 * j + (lane >> 4) * 16) = acc[i / MI][i % MI][j];
    wave_lds_order();
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float z[W];
      const char* from = mine + (q * kRows + lane / kChunks) * kRow + lane % kChunks * W * 4;
#pragma unroll
      for (int k = 0; k < W; k += 4) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(from + 4 * k);
#pragma unroll
        for (int c = 0; c < 4; ++c) z[k + c] = v[c];
      }
      if (kScaled<T, BS>)
#pragma unroll
        for (int k = 0; k < W; ++k) z[k] *= unscale;
      const int64_t m = row_of(i, q);
      if (m < p.M && n < p.N) {
        if constexpr (kKept<T, ACT>) {
          store_as<_Float16, W>(static_cast<_Float16*>(p.C) + m * p.ldc + n, p.N - n, z);
        } else if (whole) {
          finish_row<T, ACT, W>(p, m, n, z, bias, res[i & 1][q]);
          if (ACT == kLogitGradient)
#pragma unroll
            for (int k = 0; k < W; ++k) cols[k] += z[k];
        } else
          store_as<float, W>(p.partial + ((int64_t)at.part * p.M + m) * p.N + n, p.N - n, z);
      }
    }
    wave_lds_order();
  }
  if constexpr (ACT == kLogitGradient) {
    if (!p.parts) return;
    const float unscaled = p.parts_unscale ? *p.parts_unscale : 1.f;
#pragma unroll
    for (int o = kChunks; o < 64; o *= 2)
#pragma unroll
      for (int k = 0; k < W; ++k) cols[k] += __shfl_xor(cols[k], o);
#pragma unroll
    for (int k = 0; k < W; ++k) cols[k] *= unscaled;
    static_assert(WM == 2, "two sums for a tile's rows");
    if (lane < kChunks && n < p.N) store_as<float, W>(p.parts + (at.m0 / BM * WM + wm) * (int64_t)p.N + n, p.N - n, cols);
  }
}

// C from the partial sums. A block takes 64 groups of W consecutive n, and its
// 4 waves a quarter of the parts each: few outputs of many parts would
// otherwise be few threads with one long chain of loads each.
template <typename T, int ACT, int W>
__global__ void __launch_bounds__(256) product_reduce_kernel(const ProductArgs p) {
  __shared__ float red[4][64][W + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per_row = (p.N + W - 1) / W;
  const int64_t total = p.M * per_row, part = p.M * p.N;
  const int quarter = (p.splits + 3) / 4, s0 = wave * quarter, s1 = min(p.splits, s0 + quarter);
  const float unscale = kScaled<T, ACT == GMM_ACT_NONE> && p.unscale ? *p.unscale : 1.f;
  for (int64_t i0 = blockIdx.x * 64ll; i0 < total; i0 += gridDim.x * 64ll) {
    const int64_t i = i0 + lane, m = i / per_row;
    const int n = (int)(i - m * per_row) * W;
    float z[W], bias[W];
#pragma unroll
    for (int k = 0; k < W; ++k) z[k] = bias[k] = 0.f;
    if (i < total) {
      const float* q = p.partial + m * p.N + n;
      for (int s = s0; s < s1; ++s) {
        float v[W];
        load_as<float, W>(q + s * part, W, v);
#pragma unroll
        for (int k = 0; k < W; ++k) z[k] += v[k];
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < W; ++k) red[wave][lane][k] = z[k];
    __syncthreads();
    // each wave finishes 16 of the groups
    const int mine = wave * 16 + lane;
    const int64_t at = i0 + mine, row = at / per_row;
    if (lane < 16 && at < total) {
      const int col = (int)(at - row * per_row) * W;
#pragma unroll
      for (int k = 0; k < W; ++k)
        z[k] = unscale * ((red[0][mine][k] + red[1][mine][k]) + (red[2][mine][k] + red[3][mine][k]));
      if (p.bias) load_as<T, W>(static_cast<const T*>(p.bias) + col, W, bias);
      float res[W];
      load_residual<T, W>(p, row, col, res);
      finish_row<T, ACT, W>(p, row, col, z, bias, res);
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows. The weights are read once and everything else is small, so the
// kernel is a stream over B: a block owns NT * 16 rows of B, its waves split
// the contraction. The rows of A come from the caches as the second operand.
// ---------------------------------------------------------------------------
template <typename T, int NW, int NT, int ACT>
__global__ void __launch_bounds__(64 * NW) few_kernel(const FewArgs p) {
  constexpr int NB = 16 * NT;
  __shared__ float red[NW][16][NB + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * NB;
  const T *brow[NT], *arow = static_cast<const T*>(p.A) + (int64_t)min(r, p.M - 1) * p.K;
#pragma unroll
  for (int j = 0; j < NT; ++j) brow[j] = static_cast<const T*>(p.B) + (int64_t)min(n0 + 16 * j + r, p.N - 1) * p.K;
  f32x4 acc[1][NT];
  stream_rows<T, NW, 1, NT, 8 / NT>(brow, &arow, p.K, wave, g, acc);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) red[wave][r][16 * j + 4 * g + q] = acc[0][j][q];
  __syncthreads();
  if constexpr (ACT == kRowStats) {
    constexpr float kInf = __builtin_inff();
    for (int i = threadIdx.x; i < 16 * NB; i += 64 * NW) {
      const int n = i % NB, m = i / NB;
      float z = -kInf;
      if (n0 + n < p.N) {
        z = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) z += red[w][m][n];
        if (p.bias) z += (float)static_cast<const T*>(p.bias)[n0 + n];
        if (m < p.M)
          for (int k = 0; k < p.picks.top; ++k)
            if (p.picks.idx[m * p.picks.top + k] == n0 + n) p.picked[m * p.picks.top + k] = z;
      }
      float most = z;
#pragma unroll
      for (int o = NB / 2; o; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
      float sum = exp_of(z - (most == -kInf ? 0.f : most));
#pragma unroll
      for (int o = NB / 2; o; o >>= 1) sum += __shfl_xor(sum, o);
      if (n == 0 && m < p.M) {
        float* out = p.stats + 2 * ((int64_t)m * gridDim.x + blockIdx.x);
        out[0] = most;
        out[1] = sum;
      }
    }
    return;
  }
  for (int i = threadIdx.x; i < 16 * NB; i += 64 * NW) {
    const int n = i % NB, m = i / NB;
    if (m >= p.M || n0 + n >= p.N) continue;
    float z = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) z += red[w][m][n];
    ProductArgs e;
    e.N = p.N;
    e.ldc = p.ldc;
    e.res_f32 = 0;
    e.residual = p.residual;
    e.C = p.C;
    e.pre = p.pre;
    e.c_f32 = p.c_f32;
    e.c_stream = 0;
    float bias = p.bias ? (float)static_cast<const T*>(p.bias)[n0 + n] : 0.f;
    float res;
    load_residual<T, 1>(e, m, n0 + n, &res);
    finish_row<T, ACT, 1>(e, m, n0 + n, &z, &bias, &res);
  }
}

// Rows of any length and start copied to rows of whole 16-byte pieces, zeros
// behind: pieces i0, i0 + stride, ...
template <typename T>
__device__ __forceinline__ void pad_rows(const PadJob& j, int64_t i0, int64_t stride) {
  constexpr int P = Frag<T>::kPer;
  const int pieces = (int)(j.ld / P);
  const int64_t total = j.rows * pieces;
  for (int64_t i = i0; i < total; i += stride) {
    // a 64-bit division is a hundred instructions, a 32-bit one twenty
    const int64_t r = total < (1ll << 31) ? (int64_t)((uint32_t)i / (uint32_t)pieces) : i / pieces;
    const int c = (int)(i - r * pieces) * P;
    *reinterpret_cast<u32x4*>(static_cast<T*>(j.dst) + r * j.ld + c) =
        load_frag<T>(static_cast<const T*>(j.src) + r * j.cols + c, j.cols - c);
  }
}

// Two copies in one launch, half of the blocks each.
template <typename T>
__global__ void __launch_bounds__(256) pad_kernel(const PadJob a, const PadJob b) {
  const int half = gridDim.x / 2;
  if ((int)blockIdx.x < half)
    pad_rows<T>(a, blockIdx.x * 256ll + threadIdx.x, half * 256ll);
  else
    pad_rows<T>(b, (blockIdx.x - half) * 256ll + threadIdx.x, half * 256ll);
}

template <typename T>
__global__ void __launch_bounds__(256) zero_kernel(T* p, int64_t n) {
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) p[i] = (T)0.f;
}

// The largest finite |dY act'(pre)|, in parts, for the scale of a half dZ. One
// more read of dY and pre, by a block of 16 waves a CU: the backward pass of half
// operands and a float dY takes 388 us with it and 334 without at 4096 x 2048 to
// 8192 (268 MB, 4.9 TB/s), 31 and 26 at 1001 x 516 to 1000.
constexpr int kRangeThreads = 1024;
template <int ACT>
__global__ void __launch_bounds__(kRangeThreads)
dz_range_kernel(const float* __restrict__ dY, const float* __restrict__ pre, int64_t n, float* __restrict__ range) {
  constexpr int U = 4, V = 4;  // 4 loads of 16 bytes in flight
  __shared__ float red[kRangeThreads / 64];
  const int64_t stride = (int64_t)kRangeBlocks * kRangeThreads * V;
  float most = 0.f;
  for (int64_t i = ((int64_t)blockIdx.x * kRangeThreads + threadIdx.x) * V; i < n; i += U * stride) {
    float v[U][V], z[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = i + u * stride;
      const int left = at < n ? (int)min((int64_t)V, n - at) : 0;
      load_as<float, V>(dY + at, left, v[u]);
      if (ACT != GMM_ACT_NONE) load_as<float, V>(pre + at, left, z[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float a = fabsf(ACT == GMM_ACT_NONE ? v[u][k] : v[u][k] * act_slope<ACT>(z[u][k]));
        if (a <= FLT_MAX) most = fmaxf(most, a);
      }
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = most;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kRangeThreads / 64; ++w) most = fmaxf(most, red[w]);
    range[blockIdx.x] = most;
  }
}

// The exponent of the largest power of two that keeps the largest of `range`
// within half's 65504, in every thread of a block of kRangeBlocks: half then
// holds dZ with its 11 bits down to 2^-29 of the largest, wherever dY lies, and
// what half holds as it is loses nothing. 0 for no values.
__device__ __forceinline__ int dz_scale(const float* range) {
  __shared__ float red[kRangeBlocks / 64];
  float most = range[threadIdx.x];
#pragma unroll
  for (int o = 32; o; o >>= 1) most = fmaxf(most, __shfl_xor(most, o));
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRangeBlocks / 64; ++w) most = fmaxf(most, red[w]);
  if (!(most > 0.f)) return 0;
  int e;
  const float m = frexpf(most, &e);
  return min(126, max(-126, (m > 65504.f / 65536.f ? 15 : 16) - e));  // the scale and its inverse are normal
}

// dZ and the column sums of a chunk of rows. A thread owns V consecutive
// columns (16 bytes of the operands' type), 256 / CG rows go at a time; the
// rows' sums meet in LDS at the end. The last `pads`
// blocks copy X and W to padded rows, where the products need that. SCALED: dZ
// is scaled by dz_scale, the column sums are not.
template <typename T, int ACT, int V, int CG, bool SCALED>
__global__ void __launch_bounds__(256)
dz_kernel(const void* __restrict__ dY, const void* __restrict__ pre, int y_f32, int64_t rows, int cols,
          T* __restrict__ dZ, int64_t ldz, float* __restrict__ db_part, int64_t chunk_rows, int across, int pads,
          const PadJob px, const PadJob pw, const float* __restrict__ range, float* __restrict__ unscale) {
  constexpr int RG = 256 / CG;
  static_assert(kRangeBlocks == 256, "a thread each");
  __shared__ float red[RG][CG * V];
  const int pad = (int)blockIdx.x - ((int)gridDim.x - pads);
  if (pad >= 0) {
    pad_rows<T>(px, pad * 256ll + threadIdx.x, pads * 256ll);
    pad_rows<T>(pw, pad * 256ll + threadIdx.x, pads * 256ll);
    return;
  }
  float scale = 1.f;
  if (SCALED) {
    const int e = dz_scale(range);
    scale = ldexpf(1.f, e);
    if (blockIdx.x == 0 && threadIdx.x == 0) *unscale = ldexpf(1.f, -e);
  }
  const int bx = blockIdx.x % across, by = blockIdx.x / across;
  const int cg = threadIdx.x % CG, rg = threadIdx.x / CG;
  const int64_t c = ((int64_t)bx * CG + cg) * V;
  const int64_t r0 = by * chunk_rows, r1 = min(rows, r0 + chunk_rows);
  const int left = (int)min((int64_t)V, cols - c);  // of this thread's columns
  float sum[V];
#pragma unroll
  for (int i = 0; i < V; ++i) sum[i] = 0.f;
  if (c < cols) {  // dZ's padding, less than V, is behind the last of them: loaded as zeros
    constexpr int U = 4;  // rows in flight
    for (int64_t r = r0 + rg; r < r1; r += U * RG) {
      float v[U][V], z[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r + u * RG < r1) {
          load_row<T, V>(dY, (r + u * RG) * cols + c, left, y_f32, v[u]);
          if (ACT != GMM_ACT_NONE) load_row<T, V>(pre, (r + u * RG) * cols + c, left, y_f32, z[u]);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r + u * RG < r1) {
          if (ACT != GMM_ACT_NONE)
#pragma unroll
            for (int i = 0; i < V; ++i) v[u][i] *= act_slope<ACT>(z[u][i]);
#pragma unroll
          for (int i = 0; i < V; ++i) sum[i] += v[u][i];
          if (SCALED)
#pragma unroll
            for (int i = 0; i < V; ++i) v[u][i] *= scale;
          if (dZ) store_as<T, V>(dZ + (r + u * RG) * ldz + c, (int)min((int64_t)V, ldz - c), v[u]);
        }
    }
  }
  if (!db_part) return;
#pragma unroll
  for (int i = 0; i < V; ++i) red[rg][cg * V + i] = sum[i];
  __syncthreads();
  for (int i = threadIdx.x; i < CG * V; i += 256) {
    const int64_t col = (int64_t)bx * CG * V + i;
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < RG; ++g) t += red[g][i];
    if (col < cols) db_part[by * (int64_t)cols + col] = t;
  }
}

// --------------------------------------------------------------------------- launchers

template <typename T, bool AS, bool BS, int ACT>
static void launch_tile(int variant, const ProductArgs& p, hipStream_t s) {
  const dim3 grid(p.tiles_m * p.tiles_n * p.splits + p.sum_blocks);
  if (variant == kTile256)
    product_kernel<T, 256, 256, 2, 4, AS, BS, ACT><<<grid, 512, 0, s>>>(p);
  else if (variant == kTile128 && sizeof(T) == 4)
    // single precision is matrix-bound, and one block on a CU is common: two
    // waves a SIMD (4096 x 1024 x 1024 with its epilogue: 82.4 us against 83.8)
    product_kernel<T, 128, 128, 2, 4, AS, BS, ACT><<<grid, 512, 0, s>>>(p);
  else if (variant == kTile128)
    product_kernel<T, 128, 128, 2, 2, AS, BS, ACT><<<grid, 256, 0, s>>>(p);
  else
    product_kernel<T, 64, 64, 2, 2, AS, BS, ACT><<<grid, 256, 0, s>>>(p);
}

template <typename T>
hipError_t launch_product(int variant, bool a_strided, bool b_strided, int act, const ProductArgs& p, hipStream_t s) {
  if (act == kRowStats) {  // of k-contiguous operands
    launch_tile<T, false, false, kRowStats>(variant, p, s);
    return hipGetLastError();
  }
  if (act == kStatsToo) {
    launch_tile<T, false, false, kStatsToo>(variant, p, s);
    return hipGetLastError();
  }
  if (act == kLogitGradient) {
    launch_tile<T, false, false, kLogitGradient>(variant, p, s);
    return hipGetLastError();
  }
  if (!a_strided && !b_strided)
    return with_act<T, true>(act, p.c_f32, [&](auto a) {
      launch_tile<T, false, false, decltype(a)::value>(variant, p, s);
      return hipGetLastError();
    });
  // the gradients' products have no activation
  if (!a_strided)
    launch_tile<T, false, true, GMM_ACT_NONE>(variant, p, s);
  else
    launch_tile<T, true, true, GMM_ACT_NONE>(variant, p, s);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_few(int act, const FewArgs& p, hipStream_t s) {
  auto go = [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    if (few_tiles(p.M, p.N) == 2)
      few_kernel<T, 8, 2, ACT><<<(p.N + 31) / 32, 512, 0, s>>>(p);
    else
      few_kernel<T, 8, 1, ACT><<<(p.N + 15) / 16, 512, 0, s>>>(p);
    return hipGetLastError();
  };
  if (act == kRowStats) return go(std::integral_constant<int, kRowStats>{});
  return with_act<T, true>(act, p.c_f32, go);
}

static unsigned blocks_for(int64_t items) {
  const int64_t b = (items + 255) / 256;
  return (unsigned)(b < 16384 ? b : 16384);
}

template <typename T>
hipError_t launch_pad(const PadJob& a, const PadJob& b, hipStream_t s) {
  const int64_t pieces = (a.rows * a.ld > b.rows * b.ld ? a.rows * a.ld : b.rows * b.ld) / Frag<T>::kPer;
  pad_kernel<T><<<2 * blocks_for(pieces), 256, 0, s>>>(a, b);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_zero(T* p, int64_t n, hipStream_t s) {
  zero_kernel<T><<<blocks_for(n), 256, 0, s>>>(p, n);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_reduce(int act, const ProductArgs& p, hipStream_t s) {
  return with_act<T, true>(act, p.c_f32, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    if (p.N % 4 == 0)
      product_reduce_kernel<T, ACT, 4><<<blocks_for(p.M * (p.N / 4) * 4), 256, 0, s>>>(p);
    else
      product_reduce_kernel<T, ACT, 1><<<blocks_for(p.M * p.N * 4), 256, 0, s>>>(p);
    return hipGetLastError();
  });
}

template <typename T, int ACT, bool SCALED>
static void launch_dz_columns(const void* dY, const void* pre, int y_f32, int64_t rows, int cols, T* dZ, int64_t ldz,
                              float* db_part, int64_t chunk_rows, const PadJob& px, const PadJob& pw, const float* range,
                              float* unscale, hipStream_t s) {
  constexpr int V = Frag<T>::kPer;
  const int64_t groups = (cols + V - 1) / V, chunks = (rows + chunk_rows - 1) / chunk_rows;
  const int64_t pieces = (px.rows * px.ld + pw.rows * pw.ld) / V;
  const int pads = pieces ? (int)blocks_for(pieces) : 0;
  const int across = groups > 16 ? (int)((groups + 63) / 64) : 1;
  const unsigned grid = (unsigned)(across * chunks + pads);
  if (groups > 16)
    dz_kernel<T, ACT, V, 64, SCALED><<<grid, 256, 0, s>>>(dY, pre, y_f32, rows, cols, dZ, ldz, db_part, chunk_rows,
                                                          across, pads, px, pw, range, unscale);
  else  // narrow rows: more of them at a time
    dz_kernel<T, ACT, V, 16, SCALED><<<grid, 256, 0, s>>>(dY, pre, y_f32, rows, cols, dZ, ldz, db_part, chunk_rows,
                                                          across, pads, px, pw, range, unscale);
}

template <typename T>
hipError_t launch_dz(int act, const void* dY, const void* pre, int y_f32, int64_t rows, int cols, T* dZ, int64_t ldz,
                     float* db_part, int64_t chunk_rows, const PadJob& px, const PadJob& pw, const float* range,
                     float* unscale, hipStream_t s) {
  return with_act<T, false>(act, false, [&](auto a) {
    constexpr int ACT = decltype(a)::value;
    if constexpr (std::is_same<T, _Float16>::value) {
      if (range) {
        launch_dz_columns<T, ACT, true>(dY, pre, y_f32, rows, cols, dZ, ldz, db_part, chunk_rows, px, pw, range, unscale,
                                        s);
        return hipGetLastError();
      }
    }
    launch_dz_columns<T, ACT, false>(dY, pre, y_f32, rows, cols, dZ, ldz, db_part, chunk_rows, px, pw, range, unscale, s);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t launch_dz_range(int act, const float* dY, const float* pre, int64_t n, float* range, hipStream_t s) {
  return with_act<T, false>(act, false, [&](auto a) {
    dz_range_kernel<decltype(a)::value><<<kRangeBlocks, kRangeThreads, 0, s>>>(dY, pre, n, range);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t launch_column_sums(const ProductArgs& p, hipStream_t s) {
  column_sums_kernel<T><<<p.sum_blocks, 256, 0, s>>>(p);
  return hipGetLastError();
}

#define GMM_LINEAR_TYPE(T)                                                                                         \
  template hipError_t launch_product<T>(int, bool, bool, int, const ProductArgs&, hipStream_t);                    \
  template hipError_t launch_few<T>(int, const FewArgs&, hipStream_t);                                             \
  template hipError_t launch_pad<T>(const PadJob&, const PadJob&, hipStream_t);                                    \
  template hipError_t launch_zero<T>(T*, int64_t, hipStream_t);                                                    \
  template hipError_t launch_reduce<T>(int, const ProductArgs&, hipStream_t);                                      \
  template hipError_t launch_dz<T>(int, const void*, const void*, int, int64_t, int, T*, int64_t, float*, int64_t, \
                                   const PadJob&, const PadJob&, const float*, float*, hipStream_t);               \
  template hipError_t launch_column_sums<T>(const ProductArgs&, hipStream_t);

}  // namespace gmm
