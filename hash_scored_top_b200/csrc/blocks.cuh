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

// 16 bytes of a row as pairs of f32 minima and maxima: VPL values.
template <int FMT>
struct SummaryLane {
  static constexpr int VPL = 16 / kv_elem_bytes(FMT);
  float mn[VPL], mx[VPL];
  __device__ __forceinline__ void init() {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      mn[i] = INFINITY;
      mx[i] = -INFINITY;
    }
  }
  __device__ __forceinline__ void take(uint4 v, float s) {
    float x[VPL];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (FMT == KV_F32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
    } else if constexpr (FMT == KV_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo_to_f32(w[i]);
        x[2 * i + 1] = bf16hi_to_f32(w[i]);
      }
    } else {
      float y[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        decode8<FMT>(make_uint2(w[2 * i], w[2 * i + 1]), s, y);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[8 * i + k] = y[k];
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      mn[i] = fminf(mn[i], x[i]);
      mx[i] = fmaxf(mx[i], x[i]);
    }
  }
  __device__ __forceinline__ void join(int mask) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      mn[i] = fminf(mn[i], __shfl_xor_sync(FULL, mn[i], mask));
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(FULL, mx[i], mask));
    }
  }
};

// One warp per block that holds new rows: its summary over the block's rows
// below the end of the new ones. Bound by the bytes of K: 16 bytes per lane, as
// many rows at a time as fill the warp, eight such loads in flight.
// grid = (warps' worth of blocks, pairs).
template <int D, int FMT>
__global__ void __launch_bounds__(SUMMARY_THREADS) block_summarize_kernel(const SummaryParams p) {
  constexpr int ROW = D * kv_elem_bytes(FMT), LPR = ROW / 16, RPW = 32 / LPR > 0 ? 32 / LPR : 1, UNROLL = 8;
  static_assert(LPR <= 32, "a row is at most a warp's load");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pair = blockIdx.y, b = pair / p.Hkv;
  const int start = p.rows.start(b);
  const long long stop = (long long)start + p.rows.n_count;
  const int end = (int)(stop < p.rows.end(b) ? stop : p.rows.end(b));
  const long long blk_l = max(start, 0) / p.block + (long long)blockIdx.x * (SUMMARY_THREADS / 32) + warp;
  if (start >= end || end <= 0 || blk_l * p.block >= end) return;
  const int blk = (int)blk_l, r0 = blk * p.block, r1 = min(r0 + p.block, end);
  const size_t base = (size_t)pair * p.rows.Ncap;
  const int sub = lane / LPR, piece = lane % LPR;
  const unsigned char* src = reinterpret_cast<const unsigned char*>(p.K) + base * ROW + 16 * piece;
  SummaryLane<FMT> sl;
  sl.init();
  for (int r = r0 + sub; r < r1; r += RPW * UNROLL) {
    uint4 v[UNROLL];
    float s[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int at = min(r + u * RPW, r1 - 1);             // the last row again: the same minimum
      v[u] = ldg_stream(src + (size_t)at * ROW);
      s[u] = FMT == KV_INT8 || FMT == KV_E4M3 ? __ldg(p.scales + 2 * (base + at)) : 1.f;
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) sl.take(v[u], s[u]);
  }
  __syncwarp();
#pragma unroll
  for (int mask = LPR; mask < 32; mask <<= 1) sl.join(mask);
  if (sub != 0) return;
  constexpr int VPL = SummaryLane<FMT>::VPL;
  __nv_bfloat16* out = p.bsum + ((size_t)pair * p.NB + blk) * 2 * D + VPL * piece;
  uint32_t lo[VPL / 2], hi[VPL / 2];
#pragma unroll
  for (int i = 0; i < VPL / 2; ++i) {
    const __nv_bfloat16 a[4] = {__float2bfloat16_rd(sl.mn[2 * i]), __float2bfloat16_rd(sl.mn[2 * i + 1]),
                                __float2bfloat16_ru(sl.mx[2 * i]), __float2bfloat16_ru(sl.mx[2 * i + 1])};
    lo[i] = (uint32_t)__bfloat16_as_ushort(a[0]) | (uint32_t)__bfloat16_as_ushort(a[1]) << 16;
    hi[i] = (uint32_t)__bfloat16_as_ushort(a[2]) | (uint32_t)__bfloat16_as_ushort(a[3]) << 16;
  }
#pragma unroll
  for (int i = 0; i < VPL / 2; i += 2) {
    *reinterpret_cast<uint2*>(out + 2 * i) = make_uint2(lo[i], lo[i + 1]);
    *reinterpret_cast<uint2*>(out + D + 2 * i) = make_uint2(hi[i], hi[i + 1]);
  }
}

struct BlockSelectParams {
  const void* Q;             // [B][Hq][D]
  const __nv_bfloat16* bsum; // [pairs][NB][2][D]
  const int* lens;           // optional [B]
  uint32_t* keys;            // [pairs][NB] scores as ordered integers, where they do not fit in shared memory (else null)
  int* idx;                  // [pairs][k]
  int Hq, Hkv, NB, N, block, k, n_first, n_last;
};

// f32 -> an unsigned integer of the same order (-0 like +0, NaN below all).
__device__ __forceinline__ uint32_t ordered_bits(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}

constexpr int BSEL_THREADS = 512;
constexpr int BSEL_WARPS = BSEL_THREADS / 32;
constexpr int BSEL_MAX_KEYS = 51200;         // a pair's keys in the first CTA's shared memory

// A cluster of C CTAs per pair. Its warps score the pair's blocks, C * 16 warps
// side by side, into the first CTA's shared memory; that CTA then finds the k-th key
// bit by bit, counting (it may stop once a bound has just k keys above it), and
// writes the blocks above it and as many of those equal to it as are left, in
// ascending order.
// Scoring is bound by the summaries' bytes (4 D per block): 16 bytes per lane, one
// summary (D = 128) or two to a warp's load, 8 loads in flight; a lane keeps its 8
// channels of T in f64 registers. (Making the f64 from bf16 bits with integer
// operations instead of the conversion took 99 instructions per block, not 40: 29 us
// for 102400 blocks of D = 128, whose bytes take 8.)
template <int D, typename QT>
__global__ void __launch_bounds__(BSEL_THREADS) block_select_kernel(const BlockSelectParams p, int C) {
  extern __shared__ uint32_t keys_s[];
  __shared__ uint32_t count_s[34];
  __shared__ uint32_t wsum[2][BSEL_WARPS];
  constexpr int LPB = D / 4, BPW = 32 / LPB, UNROLL = 8;   // lanes per block, blocks per warp load
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  const int pair = blockIdx.x / C, b = pair / p.Hkv, G = p.Hq / p.Hkv;
  const int nb = (seq_len(p.lens, b, p.N) + p.block - 1) / p.block;
  if (threadIdx.x < 34) count_s[threadIdx.x] = 0u;
  if (C > 1) cluster_arrive_relaxed();                     // every CTA has started before anyone writes into the first
  // ---- T of this lane's channels: the summary's bytes 16 * piece .. (minima first)
  const int piece = lane % LPB, sub = lane / LPB;
  double T[8];
  {
    const QT* Qg = reinterpret_cast<const QT*>(p.Q) + ((size_t)b * p.Hq + (pair % p.Hkv) * G) * D + (8 * piece) % D;
#pragma unroll
    for (int i = 0; i < 8; ++i) T[i] = 0.0;
    for (int g = 0; g < G; ++g) {
      float q[8];
      load8(Qg + g * D, q);
#pragma unroll
      for (int i = 0; i < 8; ++i) T[i] += (double)(8 * piece < D ? fminf(q[i], 0.f) : fmaxf(q[i], 0.f));
    }
  }
  const uint32_t keys0 = smem_u32(keys_s);
  const uint32_t dst = C > 1 ? mapa(keys0, 0) : keys0;
  if (C > 1) cluster_wait();
  const __nv_bfloat16* src = p.bsum + (size_t)pair * p.NB * 2 * D + 8 * piece;
  const int stride = C * BSEL_WARPS * BPW;
  for (int j0 = (rank * BSEL_WARPS + warp) * BPW; j0 < nb; j0 += stride * UNROLL) {
    uint4 v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int j = min(j0 + u * stride + sub, nb - 1);
      v[u] = ldg_stream(src + (size_t)j * 2 * D);
    }
    double a[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      double x = 0.0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x = fma(T[2 * i], (double)bf16lo_to_f32(w[i]), x);
        x = fma(T[2 * i + 1], (double)bf16hi_to_f32(w[i]), x);
      }
      a[u] = x;
    }
    // ---- sums over the block's lanes, 8 blocks at once: each step halves the number of sums a lane holds
    double r[4], s2[2], t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool up = lane & 1;
      const double give = up ? a[i] : a[i + 4], keep = up ? a[i + 4] : a[i];
      r[i] = keep + __shfl_xor_sync(FULL, give, 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool up = lane & 2;
      const double give = up ? r[i] : r[i + 2], keep = up ? r[i + 2] : r[i];
      s2[i] = keep + __shfl_xor_sync(FULL, give, 2);
    }
    {
      const bool up = lane & 4;
      const double give = up ? s2[0] : s2[1], keep = up ? s2[1] : s2[0];
      t = keep + __shfl_xor_sync(FULL, give, 4);
    }
#pragma unroll
    for (int o = 8; o < LPB; o <<= 1) t += __shfl_xor_sync(FULL, t, o);
    const int u = (lane & 1) * 4 + (lane & 2) + ((lane & 4) >> 2);         // the sum that this lane ended with
    const int j = j0 + u * stride + sub;
    if (piece < 8 && j < nb) {
      const bool forced = j < p.n_first || j >= nb - p.n_last;
      const uint32_t key = forced ? 0xffffffffu : ordered_bits((float)t);
      if (p.keys) p.keys[(size_t)pair * p.NB + j] = key;
      else if (C > 1) st_cluster_u32(dst + 4u * (uint32_t)j, key);
      else keys_s[j] = key;
    }
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  if (rank != 0) return;

  // ---- the k-th key
  auto key_at = [&](int j) { return p.keys ? __ldcg(p.keys + (size_t)pair * p.NB + j) : keys_s[j]; };
  int* out = p.idx + (size_t)pair * p.k;
  const int k = min(p.k, nb);
  for (int i = k + threadIdx.x; i < p.k; i += BSEL_THREADS) out[i] = -1;
  if (k == 0) return;
  // keys of at least `bound`; a counter of its own for each count, so one barrier each
  auto count = [&](uint32_t bound, int slot) -> uint32_t {
    uint32_t n = 0u;
    for (int j = threadIdx.x; j < nb; j += BSEL_THREADS) n += key_at(j) >= bound ? 1u : 0u;
    n = __reduce_add_sync(FULL, n);
    if (lane == 0 && n > 0u) atomicAdd(&count_s[slot], n);
    __syncthreads();
    return *reinterpret_cast<volatile uint32_t*>(&count_s[slot]);
  };
  uint32_t kth = 0u, left = 0u;                            // keys of at least kth; `left` of those equal to it
  bool exact = false;
  for (int bit = 31; bit >= 0 && !exact; --bit) {
    const uint32_t n = count(kth | 1u << bit, bit);
    if (n >= (uint32_t)k) kth |= 1u << bit;
    exact = n == (uint32_t)k;
  }
  if (!exact) left = (uint32_t)k - (kth == 0xffffffffu ? 0u : count(kth + 1u, 32));
  // ---- ordered compaction: a thread takes `per` blocks in a row
  const int per = (nb + BSEL_THREADS - 1) / BSEL_THREADS, ja = min((int)threadIdx.x * per, nb), je = min(ja + per, nb);
  uint32_t above = 0u, equal = 0u;
  for (int j = ja; j < je; ++j) {
    const uint32_t u = key_at(j);
    above += u > kth || (exact && u == kth) ? 1u : 0u;
    equal += !exact && u == kth ? 1u : 0u;
  }
  uint32_t sa = above, se = equal;                         // inclusive sums over the warp, then over the warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(FULL, sa, o), y = __shfl_up_sync(FULL, se, o);
    if (lane >= o) {
      sa += x;
      se += y;
    }
  }
  if (lane == 31) {
    wsum[0][warp] = sa;
    wsum[1][warp] = se;
  }
  __syncthreads();
  uint32_t pa = sa - above, pe = se - equal;
  for (int w = 0; w < warp; ++w) {
    pa += wsum[0][w];
    pe += wsum[1][w];
  }
  for (int j = ja; j < je; ++j) {
    const uint32_t u = key_at(j);
    const bool is_above = u > kth || (exact && u == kth), is_equal = !exact && u == kth;
    if (is_above || (is_equal && pe < left)) out[pa + min(pe, left)] = j;
    pa += is_above;
    pe += is_equal;
  }
}

}  // namespace hst
