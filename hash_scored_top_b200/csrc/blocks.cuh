// Blocks of keys chosen by a cheap score.
//
// A block's summary is the minimum and the maximum of its keys per channel,
// rounded outwards to bf16, so that sum_c max(q_c mn_c, q_c mx_c) bounds q.k
// over the block from above. Since mn <= mx the larger product is q_c mx_c for
// q_c > 0 and q_c mn_c otherwise, so the bounds of a group's heads add up to
// one product of length 2 D:
//   score_b = T- . mn_b + T+ . mx_b,  T- = sum_h min(q_h, 0), T+ = sum_h max(q_h, 0).
// The products are summed in f64 and the score rounded once to f32: which
// block is chosen does not depend on the order of the sum, and equal f32
// scores go to the lower block.
#pragma once

#include "cache_attend.cuh"

namespace hst {

struct SummaryParams {
  const void* K;             // [pairs][Ncap][D]
  const float* scales;       // 8-bit formats
  __nv_bfloat16* bsum;       // [pairs][NB][2][D]
  RowRange rows;
  int Hkv, NB, block;
};

constexpr int SUMMARY_THREADS = 256;

// One warp per block that holds new rows: its summary over the block's rows
// below the end of the new ones. grid = (warps' worth of blocks, pairs).
template <int D, int FMT>
__global__ void __launch_bounds__(SUMMARY_THREADS) block_summarize_kernel(const SummaryParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pair = blockIdx.y, b = pair / p.Hkv;
  const int start = p.rows.start(b);
  const long long stop = (long long)start + p.rows.n_count;
  const int end = (int)(stop < p.rows.end(b) ? stop : p.rows.end(b));
  const int first = max(start, 0);
  const int blk = first / p.block + blockIdx.x * (SUMMARY_THREADS / 32) + warp;
  if (start >= end || blk * (long long)p.block >= end) return;
  if (end <= 0) return;
  const int r0 = blk * p.block, r1 = min(r0 + p.block, end);
  const size_t base = (size_t)pair * p.rows.Ncap;
  if (lane >= D / 4) return;
  float mn[4], mx[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mn[i] = INFINITY;
    mx[i] = -INFINITY;
  }
#pragma unroll 8
  for (int r = r0; r < r1; ++r) {
    float4 v = row_quad<FMT>(p.K, base + r, D, lane);
    if constexpr (FMT == KV_INT8 || FMT == KV_E4M3) {
      const float s = __ldg(p.scales + 2 * (base + r));
      v.x *= s;
      v.y *= s;
      v.z *= s;
      v.w *= s;
    }
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mn[i] = fminf(mn[i], x[i]);
      mx[i] = fmaxf(mx[i], x[i]);
    }
  }
  __nv_bfloat16* out = p.bsum + ((size_t)pair * p.NB + blk) * 2 * D + 4 * lane;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[i] = __float2bfloat16_rd(mn[i]);
    out[D + i] = __float2bfloat16_ru(mx[i]);
  }
}

struct BlockSelectParams {
  const void* Q;             // [B][Hq][D]
  const __nv_bfloat16* bsum; // [pairs][NB][2][D]
  const int* lens;           // optional [B]
  uint32_t* keys;            // [pairs][NB]: the scores as ordered integers
  int* idx;                  // [pairs][k]
  int Hq, Hkv, NB, N, block, k, n_first, n_last;
};

// f32 -> an unsigned integer of the same order (-0 like +0, NaN below all).
__device__ __forceinline__ uint32_t ordered_bits(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

constexpr int BSCORE_THREADS = 256;

// One warp per block. grid = (chunks of blocks, pairs).
template <int D, typename QT>
__global__ void __launch_bounds__(BSCORE_THREADS) block_score_kernel(const BlockSelectParams p) {
  __shared__ double T[2 * D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pair = blockIdx.y, b = pair / p.Hkv, G = p.Hq / p.Hkv;
  const QT* Qg = reinterpret_cast<const QT*>(p.Q) + ((size_t)b * p.Hq + (pair % p.Hkv) * G) * D;
  for (int c = threadIdx.x; c < D; c += BSCORE_THREADS) {
    double lo = 0.0, hi = 0.0;
    for (int g = 0; g < G; ++g) {
      const double q = (double)(float)Qg[g * D + c];
      lo += fmin(q, 0.0);
      hi += fmax(q, 0.0);
    }
    T[c] = lo;
    T[D + c] = hi;
  }
  __syncthreads();
  const int nb = (seq_len(p.lens, b, p.N) + p.block - 1) / p.block;
  const int stride = gridDim.x * (BSCORE_THREADS / 32);
  for (int j = blockIdx.x * (BSCORE_THREADS / 32) + warp; j < nb; j += stride) {
    const __nv_bfloat16* s = p.bsum + ((size_t)pair * p.NB + j) * 2 * D;
    double a = 0.0;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) a = fma(T[32 * i + lane], (double)__bfloat162float(s[32 * i + lane]), a);
    a = warp_sum(a);
    if (lane == 0) {
      const bool forced = j < p.n_first || j >= nb - p.n_last;
      p.keys[(size_t)pair * p.NB + j] = forced ? 0xffffffffu : ordered_bits((float)a);
    }
  }
}

constexpr int BTOPK_THREADS = 1024;

// The k largest keys of a pair, ties to the lower block: the k-th key digit by
// digit (8 bits a pass), then the blocks above it and as many of those equal
// to it as are left, in ascending order. grid = pairs.
__global__ void __launch_bounds__(BTOPK_THREADS) block_topk_kernel(const BlockSelectParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t sh_prefix, sh_left;
  __shared__ uint32_t wsum[2][BTOPK_THREADS / 32];
  const int pair = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int nb = (seq_len(p.lens, pair / p.Hkv, p.N) + p.block - 1) / p.block;
  int* out = p.idx + (size_t)pair * p.k;
  const int k = min(p.k, nb);
  for (int i = k + threadIdx.x; i < p.k; i += BTOPK_THREADS) out[i] = -1;
  if (k == 0) return;
  const uint32_t* keys = p.keys + (size_t)pair * p.NB;
  uint32_t prefix = 0u, left = (uint32_t)k;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0u;
    __syncthreads();
    for (int j = threadIdx.x; j < nb; j += BTOPK_THREADS) {
      const uint32_t u = __ldcg(keys + j);
      if (shift == 24 || (u >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(u >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t n = left, d = 255u;
      for (;; --d) {
        if (hist[d] >= n || d == 0u) break;
        n -= hist[d];
      }
      sh_prefix = prefix | (d << shift);
      sh_left = n;
    }
    __syncthreads();
    prefix = sh_prefix;
    left = sh_left;
  }
  // ordered compaction: running counts of keys above and equal to the k-th
  uint32_t above = 0u, equal = 0u;
  for (int j0 = 0; j0 < nb; j0 += BTOPK_THREADS) {
    const int j = j0 + threadIdx.x;
    const uint32_t u = j < nb ? __ldcg(keys + j) : 0u;
    const uint32_t ba = __ballot_sync(FULL, j < nb && u > prefix), be = __ballot_sync(FULL, j < nb && u == prefix);
    if (lane == 0) {
      wsum[0][warp] = __popc(ba);
      wsum[1][warp] = __popc(be);
    }
    __syncthreads();
    uint32_t a = above, e = equal, ta = 0u, te = 0u;
    for (int w = 0; w < BTOPK_THREADS / 32; ++w) {
      if (w < warp) {
        a += wsum[0][w];
        e += wsum[1][w];
      }
      ta += wsum[0][w];
      te += wsum[1][w];
    }
    a += __popc(ba & lanemask_lt());
    e += __popc(be & lanemask_lt());
    if (j < nb && (u > prefix || (u == prefix && e < left))) out[a + min(e, left)] = j;
    above += ta;
    equal += te;
    __syncthreads();
  }
}

}  // namespace hst
