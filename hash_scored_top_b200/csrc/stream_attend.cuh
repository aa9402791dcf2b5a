// Attention of one token's G <= 8 query heads over a bf16 or 8-bit cache: all
// keys of a sequence, listed rows, or listed blocks (see cache_attend.cuh).
//
// The kernel is bound by the cache's bytes: 4 D (bf16) or 2 D + 8 (8 bits) per
// key and pair, against 4 D G flops. Everything follows from keeping those
// bytes in flight and the work per byte small:
//   * One persistent block per SM. The tiles of all pairs form one list, of
//     which every block takes an equal run, whatever the lengths of the
//     sequences are. A run that crosses a pair's end gives a partial
//     (m, l, o[D]) per head for each side; stream_merge_kernel joins a pair's
//     partials in order.
//   * A tile (32 positions, 16 for bf16 with D = 128) is a warp's own work,
//     copied to the warp's own stages in shared memory (cp.async): no block
//     barriers, and the next tile in flight costs no registers. Every copy
//     instruction of a warp takes 512 bytes in a row where the rows lie so:
//     with 64-byte pieces of eight rows to an instruction, so that each lane
//     copied what it used, reads ended at 5.1 TB/s of 7.2. 16-byte chunks are
//     placed so that the operands' reads do not meet in a bank.
//   * Tensor cores, m16n8k16. S[heads x keys] = Q . K^T has the heads in rows
//     0..7 of M; rows 8..15 carry the low parts of an f32 query. O^T[D x heads]
//     = V^T . P^T has P on the N side, and S's accumulators are that operand as
//     they lie: a lane's two keys of head r. The order of the head dimension
//     inside S's products and of the columns of O is free, so a lane's 16 bytes
//     of K are its operand, and its 16 bytes of four V rows are the four
//     contraction rows of 16 (bf16: 8) columns. (P on the M side, its high and
//     low parts in rows 0..7 and 8..15, takes as many products but twice the
//     accumulators: 64 registers, which spilled.)
//   * 8-bit codes become f16 exactly. Queries are scaled by a power of two to
//     fill f16 (an 11-bit high part holds a bf16 value; an f32 one takes two).
//     A key's scale multiplies its logit, a value's scale its weight; weights
//     are kept below 2^15 by a running power of two, from the largest exponent
//     of a value scale so far, next to the running maximum, and enter as two
//     f16 terms (22 bits). bf16 caches use bf16 products, weights in three
//     terms (24 bits).
// 102400 keys of 32 pairs, D = 128, G = 4: bf16 6.9 TB/s, int8 6.0, e4m3 5.4 (its
// conversions to f16); D = 64 8-bit rows 4.5 to 4.9, where the work per byte is
// the largest. Short lists (32 pairs of 3103 rows: 19 us, whose bytes take 4) pay
// for what a block does once for a pair: the query, the first copies, the join of
// its warps, each behind the last.
#pragma once

#include "cache_attend.cuh"

namespace hst {

// A stage of a warp's ring: HALVES x 16 positions, each of 16 K rows, 16 V rows
// and their scales.
template <int D, int FMT>
struct StreamShape {
  static constexpr bool B16 = FMT == KV_BF16;
  static constexpr int ROW = B16 ? 2 * D : D;             // bytes of a cache row: 64, 128 or 256
  static constexpr int KC = ROW / 64;                     // 16-byte chunks of a K row per lane (4 lanes a row)
  static constexpr int VB = ROW / 8;                      // bytes of a V row per lane (8 lanes a row): 8, 16 or 32
  static constexpr int HALF = 32 * ROW + (B16 ? 0 : 128);
  static constexpr int HALVES = HALF > 8000 ? 1 : 2;
  static constexpr int WARPS = 12;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int TILE = 16 * HALVES;                // positions
  static constexpr int STAGE = HALVES * HALF;
  // 12 warps x 2 stages of 8 KB, or 3 of the 4 KB of 8 bits and D = 64
  static constexpr int STAGES = STAGE > 6000 ? 2 : 3;
  static constexpr int SMEM = WARPS * STAGES * STAGE;
  static_assert(STAGES * STAGE >= (8 * D + 16) * 4, "a warp's partial lies in its own stages");

  // Place of chunk j of row n (of 16) among the K or V rows of a half. K is
  // read chunk c (+ 4 i) of rows r: two neighbouring rows in a phase of eight
  // lanes; V chunk r (+ 8 k) of rows 2 c: four rows, every other one.
  __host__ __device__ static constexpr int k_place(int n, int j) {
    return ROW == 64 ? 64 * n + 16 * j : ROW * n + 16 * (j ^ (4 * (n & 1)));
  }
  __host__ __device__ static constexpr int v_place(int n, int j) {
    return ROW == 64 ? 128 * (n >> 1) + 16 * ((4 * (n & 1) + j) ^ (2 * ((n >> 1) & 3))) : ROW * n + 16 * (j ^ (n & 6));
  }
};

struct StreamParams {
  CacheAttendParams a;
};

// Tiles of a sequence's pairs.
template <int TILE>
__device__ __forceinline__ int stream_tiles(const CacheAttendParams& a, int b) {
  return ((a.mode == KEYS_ALL ? seq_len(a.lens, b, a.N) : a.n) + TILE - 1) / TILE;
}

// The list of all pairs' tiles (fewer than 2^31, checked on the host), cut into
// one run per block: the first `rem` runs have one tile more than the others.
struct StreamRuns {
  int total, q, rem;
  template <int TILE>
  __device__ __forceinline__ static StreamRuns make(const CacheAttendParams& a, int B, int blocks) {
    StreamRuns s;
    if (a.mode != KEYS_ALL || a.lens == nullptr) {
      s.total = B * a.Hkv * stream_tiles<TILE>(a, 0);
    } else {
      s.total = 0;
      for (int b = 0; b < B; ++b) s.total += a.Hkv * stream_tiles<TILE>(a, b);
    }
    s.q = (int)((uint32_t)s.total / (uint32_t)blocks);
    s.rem = s.total - s.q * blocks;
    return s;
  }
  __device__ __forceinline__ int begin(int i) const { return i * q + min(i, rem); }
  // the run that tile x lies in
  __device__ __forceinline__ int of(int x) const {
    const int cut = rem * (q + 1);
    if (x < cut) return (int)((uint32_t)x / (uint32_t)(q + 1));
    return rem + (int)((uint32_t)(x - cut) / (uint32_t)q);       // q > 0: there are tiles behind the cut
  }
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// (mma_bf16_16816 of attend.cuh, free to be moved)
__device__ __forceinline__ void mma_b16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Copies `bytes` (0 to 16, or 8) and fills up with zeros; with 0 nothing is read.
__device__ __forceinline__ void async_copy16(uint32_t dst, const void* src, int bytes = 16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void async_copy8(uint32_t dst, const void* src, int bytes = 8) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// Two f16 from the low (HI = false) or high pair of a word of codes. int8: the
// code plus 128 in the mantissa of 1024.., less 1152; exact.
template <int FMT, bool HI>
__device__ __forceinline__ uint32_t codes_to_f16x2(uint32_t w) {
  if constexpr (FMT == KV_INT8) {
    const uint32_t m = __byte_perm(w ^ 0x80808080u, 0x64646464u, HI ? 0x4342 : 0x4140);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&m), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(HI ? w >> 16 : w & 0xffffu), __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
  }
}

// 2^e as f32, |e| <= 126 (anything outside: the nearest of those).
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 126) + 127) << 23); }

// 2^x, 2 units in the last place; 0 below 2^-126.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, int FMT, bool QF32, bool LISTED>
__global__ void __launch_bounds__(StreamShape<D, FMT>::THREADS, 1) stream_attend_kernel(const StreamParams sp, int B) {
  using SH = StreamShape<D, FMT>;
  constexpr bool B16 = SH::B16;
  constexpr int KS = D / 16, NT = D / 16;                  // steps of Q.K, column tiles of O
  constexpr int SA_WARPS = SH::WARPS, SA_THREADS = SH::THREADS;
  constexpr int KC = SH::KC, STAGES = SH::STAGES, HALVES = SH::HALVES, ROW = SH::ROW, TILE = SH::TILE;
  extern __shared__ __align__(1024) unsigned char dyn[];
  __shared__ float sm_w[SA_WARPS][8];                      // a warp's factor in the block's partial
  __shared__ float sm_m[8], sm_l[8];
  const CacheAttendParams& a = sp.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
  const int G = a.G;
  const uint32_t ring = smem_u32(dyn) + (uint32_t)(warp * STAGES * SH::STAGE);
  asm volatile("griddepcontrol.wait;" ::: "memory");       // idx may be the previous kernel's
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // this block's run of the list of tiles
  const StreamRuns runs = StreamRuns::make<TILE>(a, B, gridDim.x);
  int t0 = runs.begin(blockIdx.x);
  const int t1 = runs.begin(blockIdx.x + 1);
  int b = 0, first = 0;                                    // first tile of sequence b's pairs
  while (t0 < t1) {
    int per;
    for (;; ++b) {
      per = stream_tiles<TILE>(a, b);
      if (t0 - first < a.Hkv * per) break;
      first += a.Hkv * per;
    }
    const int h = (int)((uint32_t)(t0 - first) / (uint32_t)per), pair = b * a.Hkv + h;
    const int ta = t0 - first - h * per;
    const int te = min(per, ta + (t1 - t0));
    const int len = seq_len(a.lens, b, a.N);
    const size_t base = (size_t)pair * a.Ncap;
    const unsigned char* Kp = reinterpret_cast<const unsigned char*>(a.K) + base * ROW;
    const unsigned char* Vp = reinterpret_cast<const unsigned char*>(a.V) + base * ROW;
    const float* Sp = a.scales + 2 * base;
    // a copy instruction i of a warp takes bytes 512 i + 16 lane of a half's rows
    constexpr int CP = ROW / 32;
    const int lane_n = 16 * lane / ROW, lane_j = lane % (ROW / 16);

    // ---- the copies of a tile. Listed: lane i holds position i's row. Else a half's 16 positions are 16 rows from
    // `row` on, the first `cnt` of which are seen.
    struct Half {
      int row, cnt;
    };
    auto half_at = [&](int t, int hf) -> Half {
      Half x = {0, 0};
      const int j = TILE * t + 16 * hf;
      if (t >= te || j >= a.n) return x;
      x.row = j;
      if (a.mode == KEYS_BLOCKS) {
        const int bl = __ldcg(a.idx + (size_t)pair * a.k + j / a.block);
        if (bl < 0 || bl > (len - 1) / a.block) return x;
        x.row = bl * a.block + j % a.block;
      }
      x.cnt = min(max(len - x.row, 0), 16);
      if (x.cnt == 0) x.row = 0;
      return x;
    };
    auto listed_at = [&](int t) -> int {
      const int j = TILE * t + lane;
      return t < te && lane < TILE && j < a.n ? key_row(a, pair, b, 0, len, j) : -1;
    };
    uint32_t seen[3] = {0u, 0u, 0u};                       // a bit per position of the tiles in flight, newest first
    auto shift_in = [&](uint32_t bits) {
      seen[2] = seen[1];
      seen[1] = seen[0];
      seen[0] = bits;
    };
    Half nx[HALVES];
    int nl = -1;
    int next = ta + warp;                                  // next tile to copy
    auto look = [&](int t) {                               // a tile's rows, ahead of its copies
      if constexpr (LISTED) {
        nl = listed_at(t);
      } else {
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) nx[hf] = half_at(t, hf);
      }
    };
    auto issue = [&](int stage) {
      uint32_t bits = 0u;
#pragma unroll
      for (int hf = 0; hf < HALVES; ++hf) {
        const uint32_t dst = ring + (uint32_t)(stage * SH::STAGE + hf * SH::HALF), sdst = dst + 32u * ROW;
        if constexpr (LISTED) {
#pragma unroll
          for (int i = 0; i < CP; ++i) {
            const int n = (512 * i) / ROW + lane_n;
            const int row = __shfl_sync(FULL, nl, 16 * hf + n);
            const size_t at = (size_t)max(row, 0) * ROW + 16 * lane_j;
            const int on = row >= 0 ? 16 : 0;
            async_copy16(dst + SH::k_place(n, lane_j), Kp + at, on);
            async_copy16(dst + 16u * ROW + SH::v_place(n, lane_j), Vp + at, on);
          }
          if constexpr (!B16) {
            const int row = __shfl_sync(FULL, nl, 16 * hf + (lane & 15));
            if (lane < 16) async_copy8(sdst + 8u * lane, Sp + 2 * (size_t)max(row, 0), row >= 0 ? 8 : 0);
          }
        } else {
          const Half x = nx[hf];
          bits |= ((1u << x.cnt) - 1u) << (16 * hf);
          const size_t at = (size_t)x.row * ROW + 16 * lane;
          if (x.cnt == 16) {                               // the common case: constant offsets
#pragma unroll
            for (int i = 0; i < CP; ++i) {
              const int n = (512 * i) / ROW + lane_n;
              async_copy16(dst + SH::k_place(n, lane_j), Kp + at + 512 * i);
              async_copy16(dst + 16u * ROW + SH::v_place(n, lane_j), Vp + at + 512 * i);
            }
            if constexpr (!B16)
              if (lane < 8) async_copy16(sdst + 16u * lane, Sp + 2 * (size_t)(x.row + 2 * lane));
          } else {                                         // rows past the end are not read: zeros
#pragma unroll
            for (int i = 0; i < CP; ++i) {
              const int n = (512 * i) / ROW + lane_n;
              const bool on = n < x.cnt;
              const size_t from = on ? at + 512 * i : 0;
              async_copy16(dst + SH::k_place(n, lane_j), Kp + from, on ? 16 : 0);
              async_copy16(dst + 16u * ROW + SH::v_place(n, lane_j), Vp + from, on ? 16 : 0);
            }
            if constexpr (!B16)
              if (lane < 8)
                async_copy16(sdst + 16u * lane, Sp + 2 * (size_t)(x.row + min(2 * lane, 14)),
                             min(max(8 * (x.cnt - 2 * lane), 0), 16));
          }
        }
      }
      if constexpr (LISTED) bits = __ballot_sync(FULL, nl >= 0);
      shift_in(bits);
      next += SA_WARPS;
      look(next);
    };
    const int mine = te - ta > warp ? (te - ta - warp + SA_WARPS - 1) / SA_WARPS : 0;
    look(next);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
      if (s < mine) issue(s);
      else shift_in(0u);
      async_commit();
    }

    // ---- the query rows as operands: word s of a lane covers dimensions dim(s) .. dim(s) + 3
    uint32_t qh[KS][2], ql[QF32 ? KS : 1][2];
    float qscale = a.scale_log2;
    {
      const size_t q0 = ((size_t)b * a.Hq + h * G + r) * D;
      float4 q[KS];
      float mx = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int dim = B16 ? 32 * (s >> 1) + 8 * c + 4 * (s & 1) : 64 * (s >> 2) + 16 * c + 4 * (s & 3);
        q[s] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < G) {
          if constexpr (QF32) q[s] = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.Q) + q0 + dim);
          else q[s] = row_quad<KV_BF16>(reinterpret_cast<const __nv_bfloat16*>(a.Q) + q0, 0, D, dim / 4);
        }
        mx = fmaxf(mx, fmaxf(fmaxf(fabsf(q[s].x), fabsf(q[s].y)), fmaxf(fabsf(q[s].z), fabsf(q[s].w))));
      }
      if constexpr (B16) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          qh[s][0] = pack_bf16x2(q[s].x, q[s].y);
          qh[s][1] = pack_bf16x2(q[s].z, q[s].w);
        }
      } else {
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
        const int e = max((int)(__float_as_uint(mx) >> 23) - 127, -112);     // 2^(13 - e) stays a number
        const float f = pow2i(13 - e);
        // two factors: their product may leave f32 where each does not
        qscale = a.scale_log2 * pow2i((e - 13) / 2) * pow2i((e - 13) - (e - 13) / 2);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const float x = q[s].x * f, y = q[s].y * f, z = q[s].z * f, w = q[s].w * f;
          qh[s][0] = pack_f16x2(x, y);
          qh[s][1] = pack_f16x2(z, w);
          if constexpr (QF32) {
            const float2 lo = __half22float2(*reinterpret_cast<__half2*>(&qh[s][0]));
            const float2 hi = __half22float2(*reinterpret_cast<__half2*>(&qh[s][1]));
            ql[s][0] = pack_f16x2(x - lo.x, y - lo.y);
            ql[s][1] = pack_f16x2(z - hi.x, w - hi.y);
          }
        }
      }
    }

    // ---- this warp's tiles ta + warp, ta + warp + SA_WARPS, ...
    float acc[NT][4], m = -INFINITY, l = 0.f;
    int E = -127;
    float vf = pow2i(13 - E);                              // weights' factor
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    int stage = 0;
    for (int i = 0; i < mine; ++i) {
      {
        const int ahead = stage == 0 ? STAGES - 1 : stage - 1;
        if (i + STAGES - 1 < mine) issue(ahead);
        else shift_in(0u);
        async_commit();
      }
      async_wait<STAGES - 1>();
      __syncwarp();                                        // other lanes' copies too
      const uint32_t src = ring + (uint32_t)(stage * SH::STAGE);
      const uint32_t ksrc = src + SH::k_place(r, c), ssrc = src + 32u * ROW + 16u * c;
      const uint32_t vsrc0 = src + 16u * ROW + (SH::VB == 8 ? SH::v_place(2 * c, r >> 1) + 8u * (r & 1) : SH::v_place(2 * c, r));
      stage = stage == STAGES - 1 ? 0 : stage + 1;
      const uint32_t live = seen[STAGES - 1];

      // ---- S = Q . K^T: n counts groups of 8 keys
      float S[2 * HALVES][4];
#pragma unroll
      for (int n = 0; n < 2 * HALVES; ++n) S[n][0] = S[n][1] = S[n][2] = S[n][3] = 0.f;
#pragma unroll
      for (int i2 = 0; i2 < KC; ++i2) {
#pragma unroll
        for (int n = 0; n < 2 * HALVES; ++n) {
          // chunk 4 i2 + c of row r + 8 (n & 1): k_place's exclusive or reaches the 64s only
          const uint4 v = lds128((ROW == 64 ? ksrc : (ksrc ^ (64u * (i2 & 1)))  + 128u * (i2 >> 1)) + (uint32_t)((n >> 1) * SH::HALF + 8 * ROW * (n & 1)));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if constexpr (B16) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
              mma_b16_16816(S[n], qh[2 * i2 + u][0], 0u, qh[2 * i2 + u][1], 0u, w[2 * u], w[2 * u + 1]);
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int s = 4 * i2 + u;
              mma_f16_16816(S[n], qh[s][0], QF32 ? ql[QF32 ? s : 0][0] : 0u, qh[s][1], QF32 ? ql[QF32 ? s : 0][1] : 0u,
                            codes_to_f16x2<FMT, false>(w[u]), codes_to_f16x2<FMT, true>(w[u]));
            }
          }
        }
      }

      // ---- weights of head r for the keys 2c, 2c + 1 of each group
      constexpr int NW = 4 * HALVES;
      float s[NW], ks[B16 ? 1 : NW], vs[B16 ? 1 : NW];
      int e = E;
#pragma unroll
      for (int n = 0; n < 2 * HALVES; ++n) {
        s[2 * n] = QF32 ? S[n][0] + S[n][2] : S[n][0];
        s[2 * n + 1] = QF32 ? S[n][1] + S[n][3] : S[n][1];
      }
      if constexpr (!B16) {
        float vm = 0.f;
#pragma unroll
        for (int n = 0; n < 2 * HALVES; ++n) {             // (scale of K, scale of V) of two rows
          const uint4 x = lds128(ssrc + (uint32_t)((n >> 1) * SH::HALF) + 64u * (n & 1));
          ks[2 * n] = __uint_as_float(x.x) * qscale;       // (S times either alone may leave f32 where the logit does not)
          ks[2 * n + 1] = __uint_as_float(x.z) * qscale;
          vs[2 * n] = __uint_as_float(x.y);
          vs[2 * n + 1] = __uint_as_float(x.w);
          vm = fmaxf(vm, fmaxf(fabsf(vs[2 * n]), fabsf(vs[2 * n + 1])));
        }
        vm = fmaxf(vm, __shfl_xor_sync(FULL, vm, 1));
        vm = fmaxf(vm, __shfl_xor_sync(FULL, vm, 2));
        if (vm < INFINITY) e = max(E, (int)(__float_as_uint(vm) >> 23) - 127);      // not a NaN either
      }
      float mt = -INFINITY;
      if (live == (TILE == 32 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
        for (int k = 0; k < NW; ++k) s[k] *= B16 ? qscale : ks[B16 ? 0 : k];
      } else {
        const uint32_t my = live >> (2 * c);
#pragma unroll
        for (int k = 0; k < NW; ++k) s[k] = (my >> ((k & 1) + 8 * (k >> 1))) & 1u ? s[k] * (B16 ? qscale : ks[B16 ? 0 : k]) : -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < NW; ++k) mt = fmaxf(mt, s[k]);
      mt = fmaxf(mt, __shfl_xor_sync(FULL, mt, 1));
      mt = fmaxf(mt, __shfl_xor_sync(FULL, mt, 2));
      if (__any_sync(FULL, mt > m || e > E)) {             // rare once the maximum has settled
        const float mn = fmaxf(m, mt);
        float f = mn == -INFINITY ? 1.f : ex2(m - mn);
        m = mn;
        l *= f;
        if constexpr (!B16) {
          const float nf = pow2i(13 - e);
          f *= nf / vf;                                    // a power of two
          vf = nf;
          E = e;
        }
        // the accumulators are those of heads 2c and 2c + 1, whose factors lie in lanes 8c and 8c + 4
        const float f0 = __shfl_sync(FULL, f, 8 * c), f1 = __shfl_sync(FULL, f, 8 * c + 4);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          acc[j][0] *= f0;
          acc[j][1] *= f1;
          acc[j][2] *= f0;
          acc[j][3] *= f1;
        }
      }
      const float ms = m == -INFINITY ? 0.f : m;           // no finite logit yet: all weights are 0
      float w[NW];
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        w[k] = ex2(s[k] - ms);
        l += w[k];
        if constexpr (!B16) w[k] *= vs[k] * vf;
      }

      // ---- O += P . V, half by half, column tile by column tile
#pragma unroll
      for (int hf = 0; hf < HALVES; ++hf) {
        const uint32_t vsrc = vsrc0 + (uint32_t)(hf * SH::HALF);      // rows 2c, 2c + 1, 2c + 8, 2c + 9 from here
        uint32_t p0[2], p1[2], p2[2];                      // the weights' terms, two keys to a word
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float x = w[4 * hf + 2 * k], y = w[4 * hf + 2 * k + 1];
          if constexpr (B16) {
            p0[k] = pack_bf16x2(x, y);
            const float x1 = x - bf16lo_to_f32(p0[k]), y1 = y - bf16hi_to_f32(p0[k]);
            p1[k] = pack_bf16x2(x1, y1);
            p2[k] = pack_bf16x2(x1 - bf16lo_to_f32(p1[k]), y1 - bf16hi_to_f32(p1[k]));
          } else {
            p0[k] = pack_f16x2(x, y);
            const float2 hi = __half22float2(*reinterpret_cast<__half2*>(&p0[k]));
            p1[k] = pack_f16x2(x - hi.x, y - hi.y);
          }
        }
        if constexpr (B16) {
#pragma unroll
          for (int k = 0; k < SH::VB / 16; ++k) {
            uint32_t v[4][4];
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2) {
              const uint4 x = lds128(vsrc + (uint32_t)(ROW * ((i2 & 1) + 8 * (i2 >> 1)) + 128 * k));
              v[i2][0] = x.x;
              v[i2][1] = x.y;
              v[i2][2] = x.z;
              v[i2][3] = x.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {                  // columns 2 j, 2 j + 1 of the lane's eight
              const uint32_t a0 = __byte_perm(v[0][j], v[1][j], 0x5410), a1 = __byte_perm(v[0][j], v[1][j], 0x7632);
              const uint32_t a2 = __byte_perm(v[2][j], v[3][j], 0x5410), a3 = __byte_perm(v[2][j], v[3][j], 0x7632);
              mma_b16_16816(acc[4 * k + j], a0, a1, a2, a3, p0[0], p0[1]);
              mma_b16_16816(acc[4 * k + j], a0, a1, a2, a3, p1[0], p1[1]);
              mma_b16_16816(acc[4 * k + j], a0, a1, a2, a3, p2[0], p2[1]);
            }
          }
        } else {
          uint32_t v[4][SH::VB / 4];
          if constexpr (SH::VB == 16) {
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2) {
              const uint4 x = lds128(vsrc + (uint32_t)(ROW * ((i2 & 1) + 8 * (i2 >> 1))));
              v[i2][0] = x.x;
              v[i2][1] = x.y;
              v[i2][2] = x.z;
              v[i2][3] = x.w;
            }
          } else {
#pragma unroll
            for (int i2 = 0; i2 < 4; ++i2) {               // the odd rows of a pair lie 64 bytes off, by exclusive or
              const uint2 x = lds64((i2 & 1 ? vsrc ^ 64u : vsrc) + 512u * (i2 >> 1));
              v[i2][0] = x.x;
              v[i2][1] = x.y;
            }
          }
#pragma unroll
          for (int q = 0; q < SH::VB / 4; ++q) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {                  // columns 4 q + 2 u, 4 q + 2 u + 1 of the lane's
              const int sel = u ? 0x7362 : 0x5140;
              const uint32_t x = __byte_perm(v[0][q], v[1][q], sel), y = __byte_perm(v[2][q], v[3][q], sel);
              const uint32_t a0 = codes_to_f16x2<FMT, false>(x), a1 = codes_to_f16x2<FMT, true>(x);
              const uint32_t a2 = codes_to_f16x2<FMT, false>(y), a3 = codes_to_f16x2<FMT, true>(y);
              mma_f16_16816(acc[2 * q + u], a0, a1, a2, a3, p0[0], p0[1]);
              mma_f16_16816(acc[2 * q + u], a0, a1, a2, a3, p1[0], p1[1]);
            }
          }
        }
      }
      __syncwarp();                                        // every lane has read the stage: it may be overwritten
    }
    async_wait<0>();

    // ---- the block's partial: every warp's (m, l, o) into its own stages, joined in warp order
    l += __shfl_xor_sync(FULL, l, 1);
    l += __shfl_xor_sync(FULL, l, 2);
    float* mine_s = reinterpret_cast<float*>(dyn + (size_t)warp * STAGES * SH::STAGE);
    __syncwarp();                                          // other lanes' slots of the ring are done with
    if (r < G && c == 0) {
      mine_s[r] = m;
      mine_s[8 + r] = l;
    }
    {
      const float of = B16 ? 1.f : 1.f / vf;               // a power of two
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {                      // head 2c + (k & 1), second column of the two for k >= 2
          const int col = (B16 ? 64 * (j >> 2) + 8 * r + 2 * (j & 3) : SH::VB * r + 2 * j) + (k >> 1);
          if (2 * c + (k & 1) < G) mine_s[16 + (2 * c + (k & 1)) * D + col] = acc[j][k] * of;
        }
      }
    }
    __syncthreads();
    if (threadIdx.x < 8 && threadIdx.x < G) {
      const int g = threadIdx.x;
      float mm = -INFINITY, ls = 0.f;
#pragma unroll
      for (int w = 0; w < SA_WARPS; ++w)
        mm = fmaxf(mm, reinterpret_cast<float*>(dyn + (size_t)w * STAGES * SH::STAGE)[g]);
#pragma unroll
      for (int w = 0; w < SA_WARPS; ++w) {
        const float* p = reinterpret_cast<float*>(dyn + (size_t)w * STAGES * SH::STAGE);
        const float f = mm == -INFINITY ? 1.f : ex2(p[g] - mm);
        sm_w[w][g] = f;
        ls = fmaf(f, p[8 + g], ls);
      }
      sm_m[g] = mm;
      sm_l[g] = ls;
    }
    __syncthreads();
    float* out = a.part + ((size_t)blockIdx.x + pair) * G * (D + 2);
    for (int x = threadIdx.x; x < G * D; x += SA_THREADS) {
      const int g = x / D, col = x % D;
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < SA_WARPS; ++w)
        o = fmaf(sm_w[w][g], reinterpret_cast<float*>(dyn + (size_t)w * STAGES * SH::STAGE)[16 + x], o);
      out[g * (D + 2) + 2 + col] = o;
    }
    if (threadIdx.x < G) {
      out[threadIdx.x * (D + 2)] = sm_m[threadIdx.x];
      out[threadIdx.x * (D + 2) + 1] = sm_l[threadIdx.x];
    }
    t0 += te - ta;
    __syncthreads();                                       // the stages are free for the next pair
  }
}

// Joins a pair's partials (those of blocks i0 .. i1, in order). grid = (G, pairs); 4 groups of D threads take a quarter
// of the partials each.
template <int D, int TILE>
__global__ void __launch_bounds__(4 * D) stream_merge_kernel(const StreamParams sp, float* O, int B, int blocks) {
  __shared__ float sm[4], sl[4], so[4][D];
  const CacheAttendParams& a = sp.a;
  const int g = blockIdx.x, pair = blockIdx.y, b = pair / a.Hkv, h = pair % a.Hkv;
  const int col = threadIdx.x % D, grp = threadIdx.x / D;
  const int per = stream_tiles<TILE>(a, b);
  const StreamRuns runs = StreamRuns::make<TILE>(a, B, blocks);
  int first = pair * per;                                  // the pair's first tile
  if (a.mode == KEYS_ALL && a.lens != nullptr) {
    first = h * per;
    for (int i = 0; i < b; ++i) first += a.Hkv * stream_tiles<TILE>(a, i);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float* out = O + ((size_t)b * a.Hq + h * a.G + g) * D;
  if (per == 0) {                                          // no keys
    if (grp == 0) out[col] = 0.f;
    return;
  }
  const int i0 = runs.of(first), i1 = runs.of(first + per - 1);
  const float* part = a.part + (size_t)g * (D + 2);
  const size_t step = (size_t)a.G * (D + 2);
  float m = -INFINITY, l = 0.f, o = 0.f;
#pragma unroll 4
  for (int i = i0 + grp; i <= i1; i += 4) {
    const float* p = part + (size_t)(i + pair) * step;
    const float pm = __ldcg(p), pl = __ldcg(p + 1), po = __ldcg(p + 2 + col);
    const float mn = fmaxf(m, pm);
    const float f0 = mn == -INFINITY ? 1.f : exp2f(m - mn), f1 = mn == -INFINITY ? 1.f : exp2f(pm - mn);
    m = mn;
    l = fmaf(f1, pl, l * f0);
    o = fmaf(f1, po, o * f0);
  }
  if (col == 0) {
    sm[grp] = m;
    sl[grp] = l;
  }
  so[grp][col] = o;
  __syncthreads();
  if (grp > 0) return;
  const float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  l = o = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float f = mm == -INFINITY ? 1.f : exp2f(sm[k] - mm);
    l = fmaf(f, sl[k], l);
    o = fmaf(f, so[k][col], o);
  }
  out[col] = l == 0.f ? 0.f : o / l;
}

}  // namespace hst
