// Blocks of keys chosen by a cheap score.
//
// A block's summary is the minimum and the maximum of its keys per channel,
// rounded outwards to bf16, so that sum_c max(q_c mn_c, q_c mx_c) bounds q.k
// over the block from above. Since mn <= mx the larger product is q_c mx_c for
// q_c > 0 and q_c mn_c otherwise, so the bounds of a group's heads add up to
// one product of length 2 D:
//   score_b = T- . mn_b + T+ . mx_b,  T- = sum_h min(q_h, 0), T+ = sum_h max(q_h, 0).
// That product is the definition, also of summaries that are not finite: an
// infinite minimum or maximum where T- or T+ is 0 gives NaN.
// The score is that of the sums in f64, rounded once to f32: which block is
// chosen does not depend on the order of the sum, and equal f32 scores go to
// the lower block.
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
// many rows at a time as fill the warp, eight such loads in flight: 137 us for
// 102400 bf16 keys of 32 pairs, D = 128 (6.1 TB/s of the 6.46 of a copy).
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

__device__ __forceinline__ float ordered_value(uint32_t u) { return __uint_as_float(u >> 31 ? u & 0x7fffffffu : ~u); }

// The smaller and the larger; a NaN if either is one. (Comparisons and a choice in their place took the selection from 25.6 to
// 28 us: the compiler made branches of them, and the heads' loads followed one another.)
__device__ __forceinline__ float min_nan(float a, float b) {
  float v;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float v;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(a), "f"(b));
  return v;
}

constexpr int BSEL_THREADS = 512;
constexpr int BSEL_WARPS = BSEL_THREADS / 32;
constexpr int BSEL_MAX_KEYS = 51200;         // a pair's keys in the first CTA's shared memory

// A cluster of C CTAs per pair. Its warps score the pair's blocks, C * 16 warps
// side by side, into the first CTA's shared memory; that CTA then finds the k-th
// key and writes the blocks above it and as many of those equal to it as are left, in
// ascending order. (Bit by bit, with a count of the keys for each, the search took
// 10 us of 27; the histograms take 1.)
// Scoring is bound by the summaries' bytes (4 D per block): 16 bytes per lane, one
// summary (D = 128) or two to a warp's load, 8 loads and the next 8 in flight. The choice is that
// of the f64 sums, but conversions to f64 run at 5 values a clock and SM (29 us for
// 102400 blocks of D = 128, whose bytes take 8). So the scores are f32 sums first,
// and beside each goes A = sum |T m|, which bounds its error: T and the products'
// sum (a chain of 4, 2, then 5 levels) round 12 times, 12 * 2^-24 A; with A itself summed in
// bf16 (at most 4 * 2^-8 too small) 2^-20 A is safe. Where the gap between the k-th
// score and the next is wider than the bound, the choice is settled; else the blocks
// in doubt, a handful, are scored again in f64.
// 97 of 3200 blocks, 32 pairs, D = 128: 16 us with warm caches, 8 of them scoring.
template <int D, typename QT>
__global__ void __launch_bounds__(BSEL_THREADS) block_select_kernel(const BlockSelectParams p, int C) {
  extern __shared__ uint32_t keys_s[];
  __shared__ uint32_t hist_s[2048];
  __shared__ uint32_t edge_s[4], found_s[3], last_s[3], worst_s[8 * BSEL_WARPS];
  __shared__ uint32_t wsum[2][BSEL_WARPS];
  constexpr int LPB = D / 4, BPW = 32 / LPB, UNROLL = 8;   // lanes per block, blocks per warp load
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = C > 1 ? (int)cluster_ctarank() : 0;
  const int pair = blockIdx.x / C, b = pair / p.Hkv, G = p.Hq / p.Hkv;
  const int nb = (seq_len(p.lens, b, p.N) + p.block - 1) / p.block;
  if (threadIdx.x < 3) last_s[threadIdx.x] = threadIdx.x == 0 ? 0xffffffffu : 0u;
  if (C > 1) cluster_arrive_relaxed();                     // every CTA has started before anyone writes into the first
  // ---- the first summaries are on their way while T is made. This lane has bytes 16 * piece .. (minima first)
  const int piece = lane % LPB, sub = lane / LPB;
  const __nv_bfloat16* src = p.bsum + (size_t)pair * p.NB * 2 * D + 8 * piece;
  const int stride = C * BSEL_WARPS * BPW, jw = (rank * BSEL_WARPS + warp) * BPW;
  uint4 next[UNROLL];
  auto load = [&](int j0) {
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (j0 + u * stride < nb) next[u] = ldg_stream(src + (size_t)min(j0 + u * stride + sub, nb - 1) * 2 * D);
  };
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) next[u] = make_uint4(0u, 0u, 0u, 0u);
  load(jw);
  double T[8];
  {
    const QT* Qg = reinterpret_cast<const QT*>(p.Q) + ((size_t)b * p.Hq + (pair % p.Hkv) * G) * D + (8 * piece) % D;
#pragma unroll
    for (int i = 0; i < 8; ++i) T[i] = 0.0;
    for (int g = 0; g < G; ++g) {
      float q[8];
      load8(Qg + g * D, q);
#pragma unroll
      for (int i = 0; i < 8; ++i) T[i] += (double)(8 * piece < D ? min_nan(q[i], 0.f) : max_nan(q[i], 0.f));
    }
  }
  uint64_t T2[4];                                          // as f32, and the magnitudes as bf16, rounded up
  __nv_bfloat162 A2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = (float)T[2 * i], y = (float)T[2 * i + 1];
    T2[i] = pack_f32x2(x, y);
    A2[i] = __halves2bfloat162(__float2bfloat16_ru(fabsf(x)), __float2bfloat16_ru(fabsf(y)));
  }
  const uint32_t keys0 = smem_u32(keys_s);
  const uint32_t dst = C > 1 ? mapa(keys0, 0) : keys0;
  if (C > 1) cluster_wait();
  uint32_t worst = 0u;                                     // the largest A's bits: infinity and NaN come above every number
  for (int j0 = jw; j0 < nb; j0 += stride * UNROLL) {
    uint4 v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) v[u] = next[u];
    load(j0 + stride * UNROLL);
    float a[2][UNROLL];                                    // the score, and A
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      uint64_t x2 = 0ull;                                  // (0, 0)
      __nv_bfloat162 y2 = __halves2bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x2 = fma_f32x2(T2[i], pack_f32x2(bf16lo_to_f32(w[i]), bf16hi_to_f32(w[i])), x2);
        const uint32_t m = w[i] & 0x7fff7fffu;
        y2 = __hfma2(A2[i], *reinterpret_cast<const __nv_bfloat162*>(&m), y2);
      }
      float x, y;
      unpack_f32x2(x2, x, y);
      a[0][u] = x + y;
      a[1][u] = __bfloat162float(y2.x) + __bfloat162float(y2.y);
    }
    // ---- sums over the block's lanes, 8 blocks at once: each step halves the number of sums a lane holds
    float t[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      float r[4], s2[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float give = lane & 1 ? a[z][i] : a[z][i + 4], keep = lane & 1 ? a[z][i + 4] : a[z][i];
        r[i] = keep + __shfl_xor_sync(FULL, give, 1);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float give = lane & 2 ? r[i] : r[i + 2], keep = lane & 2 ? r[i + 2] : r[i];
        s2[i] = keep + __shfl_xor_sync(FULL, give, 2);
      }
      const float give = lane & 4 ? s2[0] : s2[1], keep = lane & 4 ? s2[1] : s2[0];
      t[z] = keep + __shfl_xor_sync(FULL, give, 4);
#pragma unroll
      for (int o = 8; o < LPB; o <<= 1) t[z] += __shfl_xor_sync(FULL, t[z], o);
    }
    const int u = (lane & 1) * 4 + (lane & 2) + ((lane & 4) >> 2);         // the block that this lane ended with
    const int j = j0 + u * stride + sub;
    if (piece < 8 && j < nb) {
      const bool forced = j < p.n_first || j >= nb - p.n_last;
      if (!forced) worst = max(worst, __float_as_uint(t[1]) & 0x7fffffffu);
      const uint32_t key = forced ? 0xffffffffu : ordered_bits(t[0]);
      if (p.keys) p.keys[(size_t)pair * p.NB + j] = key;
      else if (C > 1) st_cluster_u32(dst + 4u * (uint32_t)j, key);
      else keys_s[j] = key;
    }
  }
  {
    const uint32_t bits = __reduce_max_sync(FULL, worst);
    const uint32_t at = smem_u32(&worst_s[rank * BSEL_WARPS + warp]);
    if (lane == 0) {
      if (C > 1) st_cluster_u32(mapa(at, 0), bits);
      else worst_s[warp] = bits;
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
  auto set_key = [&](int j, uint32_t u) {
    if (p.keys) p.keys[(size_t)pair * p.NB + j] = u;
    else keys_s[j] = u;
  };
  // a thread has `per` blocks in a row, up to 8 of them in registers
  const int per = (nb + BSEL_THREADS - 1) / BSEL_THREADS, ja = min((int)threadIdx.x * per, nb), je = min(ja + per, nb);
  uint32_t mine[8];
  auto hold = [&] {
    if (per > 8) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) mine[i] = ja + i < je ? key_at(ja + i) : 0u;
  };
  auto each = [&](auto f) {                                // f(block, key)
    if (per <= 8) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (ja + i < je) f(ja + i, mine[i]);
    } else {
      for (int j = ja; j < je; ++j) f(j, key_at(j));
    }
  };
  uint32_t kth, left;                                      // the choice: keys above kth and `left` of those equal to it,
  bool exact;                                              // or (exact) keys of at least kth
  // The k-th key by histograms of 2048 bins over the range that it lies in: scores share their leading digits, so the
  // first range is that of the keys there are (without the forced ones), and a bin of the first one mostly holds a few.
  auto search = [&] {
    hold();
    if (threadIdx.x < 4) edge_s[threadIdx.x] = threadIdx.x == 0 ? 0xffffffffu : 0u;
    __syncthreads();
    uint32_t lo = 0xffffffffu, hi = 0u, nf = 0u;
    each([&](int, uint32_t u) {
      if (u == 0xffffffffu) {
        ++nf;
      } else {
        lo = min(lo, u);
        hi = max(hi, u);
      }
    });
    lo = __reduce_min_sync(FULL, lo);
    hi = __reduce_max_sync(FULL, hi);
    nf = __reduce_add_sync(FULL, nf);
    if (lane == 0) {
      atomicMin(&edge_s[0], lo);
      atomicMax(&edge_s[1], hi);
      atomicAdd(&edge_s[2], nf);
    }
    __syncthreads();
    lo = edge_s[0];
    hi = edge_s[1];
    nf = edge_s[2];
    kth = 0xffffffffu;
    left = 0u;
    exact = true;
    if (nf >= (uint32_t)k) return;                         // (they are k at most)
    left = (uint32_t)k - nf;
    int bits = 32 - __clz((int)(hi - lo));                 // keys lo .. lo + 2^bits - 1
    for (;;) {
      const int sh = max(bits - 11, 0);
      const uint32_t bins = 1u << (bits - sh);             // of the range: the keys behind it were counted by the pass before
      for (int i = threadIdx.x; i < 2048; i += BSEL_THREADS) hist_s[i] = 0u;
      __syncthreads();
      each([&](int, uint32_t u) {
        const uint32_t d = (u - lo) >> sh;
        if (u != 0xffffffffu && u >= lo && d < bins) atomicAdd(&hist_s[d], 1u);
      });
      __syncthreads();
      uint32_t c[4], sum = 0u;                             // bins 2047 - 4 thread downwards
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = hist_s[2047 - 4 * (int)threadIdx.x - i];
        sum += c[i];
      }
      uint32_t before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(FULL, before, o);
        if (lane >= o) before += x;
      }
      if (lane == 31) wsum[0][warp] = before;
      __syncthreads();
      before -= sum;
      for (int w = 0; w < warp; ++w) before += wsum[0][w];
      if (before < left && left <= before + sum) {         // one thread
        uint32_t n = left - before;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (n > 0u && n <= c[i]) {
            found_s[0] = 2047u - 4u * threadIdx.x - i;
            found_s[1] = n;
            found_s[2] = c[i];
            n = 0u;
          } else if (n > 0u) {
            n -= c[i];
          }
        }
      }
      __syncthreads();
      lo += found_s[0] << sh;
      left = found_s[1];
      exact = found_s[2] == left;                          // the whole bin is in
      bits = sh;
      if (exact || sh == 0) break;
    }
    kth = lo;
    if (exact) left = 0u;
  };
  search();
  // ---- is the choice settled? The smallest key in and the largest key out
  uint32_t lo = 0xffffffffu, hi = 0u, wb = 0u;
  each([&](int, uint32_t u) {
    if (u >= kth) lo = min(lo, u);
    else hi = max(hi, u);
  });
  lo = __reduce_min_sync(FULL, lo);
  hi = __reduce_max_sync(FULL, hi);
  for (int i = threadIdx.x; i < C * BSEL_WARPS; i += BSEL_THREADS) wb = max(wb, worst_s[i]);
  wb = __reduce_max_sync(FULL, wb);
  if (lane == 0) {
    atomicMin(&last_s[0], lo);
    atomicMax(&last_s[1], hi);
    atomicMax(&last_s[2], wb);
  }
  __syncthreads();
  lo = last_s[0];
  hi = last_s[1];
  const float err = __fmul_ru(__uint_as_float(last_s[2]), 0x1p-20f) + 0x1p-126f;
  const float in = ordered_value(lo), out_v = ordered_value(hi);
  // (nothing is out; only forced blocks are in; or the gap is wider than both errors, of finite scores)
  const bool settled = exact && (k == nb || lo == 0xffffffffu || (lo != 0u && hi != 0u && __fsub_rd(in, out_v) > 2.f * err));
  if (!settled) {
    // blocks within the errors of the edge are scored again; those above and below it are out of doubt. With scores or
    // errors that are not finite, all are.
    const bool all = !(err < 0x1p100f) || lo == 0u || lo == 0xffffffffu || !(fabsf(in) < 0x1p126f);
    const uint32_t sure_out = all ? 0u : ordered_bits(__fsub_rd(in, 2.f * err)), sure_in = all ? 0xffffffffu : ordered_bits(__fadd_ru(in, 2.f * err));
    for (int j0 = warp * 32; j0 < nb; j0 += BSEL_THREADS) {
      const int j = j0 + lane;
      const uint32_t u = j < nb ? key_at(j) : 0u;
      const bool forced = u == 0xffffffffu;
      const bool doubt = j < nb && !forced && (all || (u >= sure_out && u <= sure_in));
      if (j < nb && !forced && !doubt) set_key(j, u > sure_in ? 0xffffffffu : 0u);
      for (uint32_t todo = __ballot_sync(FULL, doubt); todo != 0u; todo &= todo - 1u) {
        const int jj = j0 + __ffs(todo) - 1;
        const uint4 v = ldg_stream(src + (size_t)jj * 2 * D);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        double x = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x = fma(T[2 * i], (double)bf16lo_to_f32(w[i]), x);
          x = fma(T[2 * i + 1], (double)bf16hi_to_f32(w[i]), x);
        }
#pragma unroll
        for (int o = 1; o < LPB; o <<= 1) x += __shfl_xor_sync(FULL, x, o);
        const uint32_t key = ordered_bits((float)x);
        if (lane == 0) set_key(jj, all ? key : min(max(key, 1u), 0xfffffffeu));
      }
    }
    __syncthreads();
    search();
  }
  // ---- ordered compaction
  uint32_t above = 0u, equal = 0u;
  each([&](int, uint32_t u) {
    above += u > kth || (exact && u == kth) ? 1u : 0u;
    equal += !exact && u == kth ? 1u : 0u;
  });
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
  each([&](int j, uint32_t u) {
    const bool is_above = u > kth || (exact && u == kth), is_equal = !exact && u == kth;
    if (is_above || (is_equal && pe < left)) out[pa + min(pe, left)] = j;
    pa += is_above;
    pe += is_equal;
  });
}

}  // namespace hst
