// Attention of T drafted tokens over a bf16 or 8-bit cache on tcgen05
// (tree_decode; see cache_attend.cuh for what a token sees).
//
// A KV head's R = T * G query rows are the M side of two products per tile of
// KT keys: S[128 x KT] = Q . K^T and O[128 x D] += P . V. A cache byte is used by
// all rows at once, so up to about a hundred rows the cache's bytes bound the
// kernel (4 D per key and pair), beyond that the two products (4 D R flops).
//
// Roles of a block (one per SM, 320 threads):
//   warp 8    copies K and V tiles by TMA (128-byte swizzle) into a ring of
//             slots, K and V alternating;
//   warp 9    issues the MMAs: S of a job into tensor memory, and, when its
//             weights are there, O += P . V with P as the tensor-memory operand
//             and V as it lies (N-major);
//   warps 0-7 are softmax threads, one row (lane of tensor memory) each. Up to
//             128 rows are one team of 256: two threads share a row, half of a
//             tile's columns each, and exchange the half maxima. More rows (WIDE)
//             are two teams of 128 threads and rows, which share the tiles.
// S has two buffers per team: the product of the next tile runs while the
// weights of this one are taken (with one buffer a tile took S, softmax and P . V
// one after the other: 5100 clocks per 128 keys where the cache's bytes take
// 2500). The weights are written over the S that they come from. O is rescaled
// only when a row's maximum has grown by more than 2^8 since the last time: weights
// up to 2^8 lose nothing. (8-bit caches: 2^1, so that their f16 weights, below 2^15,
// go down to 2^-38 of the largest.)
// The weights enter the second product as NT bf16 terms: one for bf16 outputs
// (each is off by at most 2^-8, as the output's own rounding is), three (24
// bits) for f32. An MMA takes 128 rows, however many there are: with R <= 64 (32)
// the rows are laid out twice (four times), every copy takes the same weights, and the
// copies hold different terms, so that three terms take two products (one) instead of
// three. The accumulator of an MMA is cut off, not rounded: over a run of 140 tiles O
// came out 1.2e-5 off, so f32 outputs add it up in plain arithmetic every 8 tiles (1e-6).
// Tensor memory holds O, that sum and two buffers of S and the third term (for 128
// rows and D = 128 with tiles of 64 keys: 128 + 128 + 2 * 96 columns). Two teams fit with tiles
// of 64 keys and one term, so f32 outputs of more than 128 rows are taken 128 at a time.
//
// 8-bit caches: warp 8 copies the codes as they lie into a second ring, and four
// more warps turn them into f16 tiles (exactly), in the layout that TMA gives a
// bf16 tile, and put the rows' scales beside them. Queries are f16 too, scaled by
// a power of two per row. A key's scale multiplies its column of S, a value's its
// weights, which are kept below 2^15 by the largest exponent of a value scale so
// far, as in stream_attend.cuh; one f16 term (11 bits) for bf16 outputs, two (22) for f32.
// With R <= 64 the two copies of the rows share a tile's keys there (16 tokens of 4 heads over
// 102384 int8 keys, 32 pairs, f32 outputs, in a loop: 348 us; with a term of the weights to each
// copy 552. 305 alone).
// f32 queries are two f16 tiles, high and low parts, whose products with K add up in S
// (over tiles of 64 keys, to make room).
//
// The list of all (pair, group of rows, tile) is cut into one even run per
// block, as in stream_attend.cuh; a run that crosses a unit's end gives a partial for
// each side, which tree_merge_kernel joins in order.
//
// Four sequences of up to 102400 keys, 8 KV heads of 4 queries, D = 128: 16 tokens with f32
// outputs 283 us (4.8 TB/s; the tensor pipe 51% busy), 64 tokens with bf16 outputs 381 (the
// exponentials and the products 50% each); in a loop the GPU's power limit makes that
// 310 to 330 and 420 to 450. 7 tokens over int8, 32761 keys of 8 pairs: 47 us (the conversion,
// about 3000 clocks a tile), with f32 queries and outputs 63. The 8-bit kernels of one copy (R > 64,
// or f32 queries) spill 8 to 232 bytes, most with f32 outputs: 448 threads leave 128 registers to each.
//
// Drafted keys lie behind the cached ones, in the last tiles. Their S is masked
// per row. A V row that is not finite must reach only the rows that see it,
// which a product cannot do (0 * NaN): such rows (and the rows behind the
// sequence) are cleared in shared memory, and what a drafted one gives to the
// rows that see it is added at the end, in plain arithmetic. (e4m3: its NaN codes
// alone are cleared, and make that column NaN for the rows that see them.)
#pragma once

#include <type_traits>

#include "cache_attend.cuh"
#include "stream_attend.cuh"
#include "tcgen05.cuh"

namespace hst {

constexpr int TR_MAX_SLOTS = 12;
constexpr uint32_t TR_SMEM_MAX = 229376;     // dynamic; of a block's 232448, 3 KB are the kernel's static arrays
constexpr int TR_MAX_DRAFT_WORDS = 8;

template <int D, int KT, bool WIDE, bool Q8, bool QF32 = false>
struct TreeShape {
  static constexpr int THREADS = Q8 ? 448 : 320;
  static constexpr int QBYTES = 128 * D * 2;               // one Q tile
  static constexpr int SLOT = KT * D * 2;                  // one K or V tile
  static constexpr int QTILES = WIDE || QF32 ? 2 : 1;     // f32 queries: high and low parts
  static constexpr int FIT = ((int)TR_SMEM_MAX - QTILES * QBYTES) / SLOT;
  static constexpr int SLOTS = Q8 ? 4 : FIT < TR_MAX_SLOTS ? FIT : TR_MAX_SLOTS;
  // 8 bits: RAWS tiles of codes with their scales, and the scales of four tiles as the softmax reads them
  static constexpr int RAW = KT * D + KT * 8;
  static constexpr int RAW_FIT = ((int)TR_SMEM_MAX - QTILES * QBYTES - SLOTS * SLOT - 4 * KT * 8) / RAW;
  static constexpr int RAWS = !Q8 ? 0 : RAW_FIT < 6 ? RAW_FIT : 6;
  static constexpr int SMEM = QTILES * QBYTES + SLOTS * SLOT + RAWS * RAW + (Q8 ? 4 * KT * 8 : 0);
  static_assert(Q8 ? RAWS >= 3 : SLOTS >= 6, "the tiles of both buffers and one in flight");
  static_assert(SMEM <= (int)TR_SMEM_MAX, "dynamic shared memory");
};

struct TreeParams {
  CacheAttendParams a;
  int groups;                // groups of 128 (WIDE: 256) rows of a pair
  int rows;                  // rows of a partial: min(R, 128)
  int parts;                 // partials of a run: teams, or copies of the rows
};

// Tiles of a sequence's units: its cached and its drafted keys.
template <int KT>
__device__ __forceinline__ int tree_tiles(const CacheAttendParams& a, int b) {
  return (seq_len(a.lens, b, a.N) + a.T + KT - 1) / KT;
}

template <int KT>
__device__ __forceinline__ StreamRuns tree_runs(const TreeParams& p, int B, int blocks) {
  StreamRuns s;
  s.total = 0;
  for (int b = 0; b < B; ++b) s.total += p.a.Hkv * p.groups * tree_tiles<KT>(p.a, b);
  s.q = (int)((uint32_t)s.total / (uint32_t)blocks);
  s.rem = s.total - s.q * blocks;
  return s;
}

// Bits of the positions j0 .. j0 + 31 that the token sees.
struct TreeRow {
  const uint32_t* mask;      // the token's words, or null: a chain
  int t, len, T;
  __device__ __forceinline__ uint32_t drafts(int w) const {      // drafted keys 32 w ..
    const int left = T - 32 * w;
    if (left <= 0 || w < 0) return 0u;
    const uint32_t in = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
    if (mask) return __ldg(mask + w) & in;
    const int n = t + 1 - 32 * w;
    return n >= 32 ? in : n <= 0 ? 0u : ((1u << n) - 1u) & in;
  }
  __device__ __forceinline__ uint32_t sees(int j0) const {
    const int a = len - j0;                                      // cached positions from here
    if (a >= 32) return 0xffffffffu;
    if (a > 0) return ((1u << a) - 1u) | (drafts(0) << a);
    const int w = (-a) >> 5, s = (-a) & 31;
    return s == 0 ? drafts(w) : (drafts(w) >> s) | (drafts(w + 1) << (32 - s));
  }
};

// The operand descriptors of this kernel are those of umma_desc_sw128 (K-major)
// and, for V as it lies, N-major with the 128-byte swizzle: atoms of 64 columns
// x 8 rows (rows 128 bytes apart), `lbo` bytes between atoms along the columns
// and 1024 along the rows. Their upper words are the same for all tiles; an MMA
// then costs its thread one addition per operand. (Building the descriptors for
// every MMA took the issuing thread 105 clocks each, which bound the kernel.)
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);         // stride 1024, version 1, 128-byte swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); }

// D[tmem] (+)= A[smem] . B[smem]^T, bf16, both K-major.
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"(kDescHi)
      : "memory");
}
// D[tmem] (+)= A[tmem] . B[smem], bf16: A is M x 16, two values to a column; B N-major.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"((uint32_t)accumulate), "r"(kDescHi)
      : "memory");
}
// f32 accumulators, bf16 (f16) operands, M = 128; B is N-major if b_mn.
__device__ __forceinline__ constexpr uint32_t tree_idesc(int n, bool b_mn, bool f16 = false) {
  return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0u;
}

// Two f32 from shared memory.
__device__ __forceinline__ uint64_t lds_f32x2(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr));
  return v;
}

// Clears the NaN codes among 16 e4m3 codes; whether there were any.
__device__ __forceinline__ bool drop_nan_codes(uint4& v) {
  const uint32_t x = __vcmpeq4(v.x & 0x7f7f7f7fu, 0x7f7f7f7fu), y = __vcmpeq4(v.y & 0x7f7f7f7fu, 0x7f7f7f7fu);
  const uint32_t z = __vcmpeq4(v.z & 0x7f7f7f7fu, 0x7f7f7f7fu), w = __vcmpeq4(v.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
  v = make_uint4(v.x & ~x, v.y & ~y, v.z & ~z, v.w & ~w);
  return (x | y | z | w) != 0u;
}

// The value that a bf16 of x's upper half has: x cut off to 8 bits.
__device__ __forceinline__ float cut_bf16(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

// NT terms of the weights in COPIES copies of the rows. Over 8-bit caches the (two) copies share the keys instead: each takes
// half of a tile's, with a maximum, a sum and an O of its own, and its weights for the others are 0.
template <int D, int KT, int NT, bool WIDE, int COPIES, int FMT, bool QF32 = false>
__global__ void __launch_bounds__(TreeShape<D, KT, WIDE, FMT != KV_BF16, QF32>::THREADS, 1)
    tree_attend_kernel(const TreeParams p, int B, const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV) {
  constexpr bool Q8 = FMT != KV_BF16;
  using SH = TreeShape<D, KT, WIDE, Q8, QF32>;
  static_assert(!QF32 || (Q8 && !WIDE), "f32 queries: 8-bit caches");
  constexpr int NS = SH::SLOTS, NR = SH::RAWS, ATOMS = D / 64, TEAMS = WIDE ? 2 : 1, TEAM = WIDE ? 128 : 256;
  // tensor memory: O of team w at w * D; buffer sb of its S (and P over it) behind them. Chunk q of 32 keys holds S at
  // 32 q, then P of the first two products at 32 q and 32 q + 16, of the third at KT + 16 q.
  constexpr bool SPLIT = Q8 && COPIES == 2;
  constexpr int NP = SPLIT ? NT : (NT + COPIES - 1) / COPIES;      // products per tile
  constexpr uint32_t SCOLS = NP == 3 ? KT + KT / 2 : KT;
  static_assert(!WIDE || COPIES == 1, "a team has all its rows");
  // f32 outputs: O is added to a second one, which the MMAs do not touch, after every FLUSH tiles
  constexpr bool LONG = NT > 1;
  constexpr uint32_t LCOL = TEAMS * (D + 2 * SCOLS);
  constexpr int FLUSH = 8;
  static_assert(LCOL + (LONG ? D : 0) <= 512, "tensor memory");
  auto s_col = [](int w, int sb) { return (uint32_t)(TEAMS * D) + (uint32_t)(2 * w + sb) * SCOLS; };
  extern __shared__ __align__(1024) unsigned char dyn[];
  __shared__ __align__(8) uint64_t bars[2 * TR_MAX_SLOTS + 16 + (Q8 ? 16 : 0)];
  __shared__ float vmax_s[4][4];                           // 8 bits: the largest value scale of a tile, by quarters of its rows
  __shared__ uint32_t nan_s;                               // e4m3: set once a drafted row of V has a NaN code
  // drafted keys whose V was cleared, by the parity of the segment: they are cleared for a segment while others may
  // still read the last one's
  __shared__ uint32_t bad_s[2][TR_MAX_DRAFT_WORDS];
  __shared__ float half_s[2][2][128];                      // maxima (at the end sums) of half a row, by the parity of the tile
  __shared__ uint32_t tbase_s;
  static_assert(sizeof(bars) + sizeof(vmax_s) + sizeof(nan_s) + sizeof(bad_s) + sizeof(half_s) + sizeof(tbase_s) <= 232448 - TR_SMEM_MAX,
                "static shared memory");
  const CacheAttendParams& a = p.a;
  const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
  const uint32_t s0 = smem_u32(dyn), q0 = s0, slots = s0 + SH::QTILES * SH::QBYTES;
  const uint32_t b0 = smem_u32(bars), full = b0, empty = b0 + 8 * TR_MAX_SLOTS, sfull = b0 + 16 * TR_MAX_SLOTS;
  const uint32_t pready = sfull + 32, pvdone = sfull + 64, qready = sfull + 96, halves = sfull + 104, drain = sfull + 112;
  const uint32_t rfull = sfull + 128, rempty = rfull + 48, scales_in = rempty + 48;      // (8 bits: rings of codes, scales)
  const uint32_t raws = slots + (uint32_t)(NS * SH::SLOT), scs = raws + (uint32_t)(NR * SH::RAW);
  if (warp == 0) {
    tmem_alloc(smem_u32(&tbase_s), 512u);
    tmem_relinquish();
  }
  if (tid == 0) {
    nan_s = 0u;
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + 8 * i, Q8 ? 128 : 1);
      mbar_init(empty + 8 * i, TEAMS);                     // one commit per team
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(rfull + 8 * i, 1);
      mbar_init(rempty + 8 * i, 128);
    }
    for (int i = 0; i < (Q8 ? 4 : 0); ++i) mbar_init(scales_in + 8 * i, 128);
    for (int i = 0; i < 4; ++i) {                          // team w, buffer sb: 2 w + sb
      mbar_init(sfull + 8 * i, 1);
      mbar_init(pready + 8 * i, TEAM);
      mbar_init(pvdone + 8 * i, 1);
    }
    mbar_init(qready, 256);
    mbar_init(halves, 256);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tb = tbase_s;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // the block's run, walked by every role on its own
  const StreamRuns runs = tree_runs<KT>(p, B, gridDim.x);
  const int t1 = runs.begin(blockIdx.x + 1);
  struct Segment {
    int t0, b, first;                                      // walking state
    int unit, pair, grp, len, ta, te;
  };
  auto next_segment = [&](Segment& s) -> bool {
    if (s.t0 >= t1) return false;
    int per;
    for (;; ++s.b) {
      per = tree_tiles<KT>(a, s.b);
      const int all = a.Hkv * p.groups * per;
      if (s.t0 - s.first < all) break;
      s.first += all;
    }
    const int u = (s.t0 - s.first) / per;
    s.unit = s.b * a.Hkv * p.groups + u;
    s.pair = s.unit / p.groups;
    s.grp = s.unit % p.groups;
    s.len = seq_len(a.lens, s.b, a.N);
    s.ta = s.t0 - s.first - u * per;
    s.te = min(per, s.ta + (t1 - s.t0));
    s.t0 += s.te - s.ta;
    return true;
  };
  Segment seg = {};
  seg.t0 = runs.begin(blockIdx.x);
  const int R = a.T * a.G;
  // J counts the block's tiles: their K and V lie in slots 2 J and 2 J + 1 (modulo the ring), their S in buffer J & 1
  auto slot_of = [&](int n) { return slots + (uint32_t)(n % NS) * (uint32_t)SH::SLOT; };
  auto bar_of = [](uint32_t bars4, int w, int J) { return bars4 + 8u * (uint32_t)(2 * w + (J & 1)); };
  auto par_of = [](int J) { return (uint32_t)((J >> 1) & 1); };

  if (warp == 8) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      constexpr int RING = Q8 ? NR : NS;
      const uint32_t in = Q8 ? rfull : full, out = Q8 ? rempty : empty;
      int n = 0;
      bool ok = true;
      while (ok && next_segment(seg)) {
        for (int i = seg.ta; i < seg.te && ok; ++i) {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const int s = n % RING;
            if (n >= RING && !mbar_wait_bounded(out + 8 * s, (uint32_t)((n / RING - 1) & 1))) {
              ok = false;
              break;
            }
            if constexpr (Q8) {
              // the rows that there are, of codes, and (with K) their scales, an even number for 16 bytes
              const int rows = min(KT, seg.len + a.T - i * KT), even = (rows + 1) & ~1;
              const size_t at = (size_t)seg.pair * a.Ncap + (size_t)i * KT;
              const uint32_t dst = raws + (uint32_t)(s * SH::RAW);
              mbar_arrive_expect_tx(in + 8 * s, (uint32_t)(rows * D + (kv ? 0 : even * 8)));
              bulk_copy_g2s(dst, reinterpret_cast<const unsigned char*>(kv ? a.V : a.K) + at * D, (uint32_t)(rows * D), in + 8 * s);
              if (!kv) bulk_copy_g2s(dst + KT * D, a.scales + 2 * at, (uint32_t)(even * 8), in + 8 * s);
            } else {
              mbar_arrive_expect_tx(in + 8 * s, (uint32_t)SH::SLOT);
#pragma unroll
              for (int at = 0; at < ATOMS; ++at)
                tma_load_2d(slot_of(n) + (uint32_t)(at * KT * 128), kv ? &mapV : &mapK, 64 * at, seg.pair * a.Ncap + i * KT,
                            in + 8 * s);
            }
          }
        }
      }
      // nothing stays in flight, whatever the others did
      for (int j = max(0, n - RING); j < n; ++j) mbar_wait_bounded(in + 8 * (j % RING), (uint32_t)((j / RING) & 1));
    }
  } else if (warp == 9) {
    // ---------------------------------------------------------------- MMAs
    // elect.sync, not a lane's number: the compiler then knows that one thread is left and keeps the operands in
    // uniform registers (an MMA costs its thread 85 clocks instead of 125, with nothing else between them)
    if (elect_one()) {
      bool ok = true;
      int J0 = 0, seg_n = 0;
      constexpr uint32_t idS = tree_idesc(KT, false, Q8), idO = tree_idesc(D, true, Q8);
      auto waits = [&](uint32_t bar, uint32_t parity) {
        ok = ok && mbar_wait_bounded(bar, parity);
        return ok;
      };
      auto issue_s = [&](int w, int J) {
        const int n = 2 * J;
        if (!waits(full + 8 * (n % NS), (uint32_t)((n / NS) & 1))) return;
        tc_fence_after_sync();
        const uint32_t ks = desc_lo(slot_of(n), 16u), qs = desc_lo(q0 + (uint32_t)(w * SH::QBYTES), 16u), sd = tb + s_col(w, J & 1);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          tc_mma_ss(sd, qs + (uint32_t)(((s >> 2) * 128 * 128 + (s & 3) * 32) >> 4),
                    ks + (uint32_t)(((s >> 2) * KT * 128 + (s & 3) * 32) >> 4), idS, s > 0);
        if constexpr (QF32) {                              // + the low parts' product
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            tc_mma_ss(sd, qs + (uint32_t)((SH::QBYTES + (s >> 2) * 128 * 128 + (s & 3) * 32) >> 4),
                      ks + (uint32_t)(((s >> 2) * KT * 128 + (s & 3) * 32) >> 4), idS, true);
        }
        tc_commit(bar_of(sfull, w, J));
        tc_commit(empty + 8 * (n % NS));
      };
      while (ok && next_segment(seg)) {
        const int nt = seg.te - seg.ta;
        if (!waits(qready, (uint32_t)(seg_n & 1))) break;
        for (int i = 0; i < 2 && i < nt; ++i)
          for (int w = 0; w < TEAMS && ok; ++w) issue_s(w, J0 + i);
        for (int i = 0; i < nt && ok; ++i) {
          const int J = J0 + i, n = 2 * J + 1;
          if (!waits(full + 8 * (n % NS), (uint32_t)((n / NS) & 1))) break;
          const uint32_t vs = desc_lo(slot_of(n), KT * 128u);
#pragma unroll
          for (int w = 0; w < TEAMS; ++w) {
            if (!waits(bar_of(pready, w, J), par_of(J))) break;
            tc_fence_after_sync();
            const uint32_t ps = tb + s_col(w, J & 1);
#pragma unroll
            for (int s = 0; s < KT / 16; ++s) {
#pragma unroll
              for (int k = 0; k < NP; ++k) {
                const uint32_t at = k < 2 ? 32u * (s >> 1) + 16u * k + 8u * (s & 1) : KT + 8u * s;
                tc_mma_ts(tb + w * D, ps + at, vs + (uint32_t)(s * 2048 >> 4), idO, s > 0 || k > 0 || (LONG ? i % FLUSH != 0 : i > 0));
              }
            }
            tc_commit(bar_of(pvdone, w, J));
            tc_commit(empty + 8 * (n % NS));
            if (i + 2 < nt) issue_s(w, J + 2);             // over the P that the product before it reads
          }
        }
        J0 += nt;
        ++seg_n;
      }
      tc_commit(drain);                                    // every MMA issued is done before tensor memory is freed
      mbar_wait_bounded(drain, 0u);
    }
  } else if (Q8 && warp >= 10) {
    // ---------------------------------------------------------------- 8 bits: codes to f16 tiles
    if constexpr (Q8) {
      const int ct = tid - 320;                            // of 128 threads
      constexpr int CR = D / 16;                           // 16-byte pieces of a row
      int n = 0, J = 0;
      bool ok = true;
      while (ok && next_segment(seg)) {
        for (int i = seg.ta; i < seg.te && ok; ++i, ++J) {
          const int rows = min(KT, seg.len + a.T - i * KT);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const int r = n % NR, s = n % NS;
            if (!mbar_wait_bounded(rfull + 8 * r, (uint32_t)((n / NR) & 1)) ||
                (n >= NS && !mbar_wait_bounded(empty + 8 * s, (uint32_t)((n / NS - 1) & 1)))) {
              ok = false;
              break;
            }
            const uint32_t src = raws + (uint32_t)(r * SH::RAW), dst = slot_of(n);
            if (kv == 0) {                                 // the tile's scales, 0 behind the last row
              float2 x = make_float2(0.f, 0.f);
              if (ct < rows) {
                const uint2 u = lds64(src + KT * D + 8u * ct);
                x = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
              }
              if (ct < KT) {
                const uint32_t to = scs + (uint32_t)((J & 3) * KT * 8) + 4u * ct;
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(x.x) : "memory");
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + 4u * KT), "f"(x.y) : "memory");
              }
              float vm = fabsf(x.y);
              vm = vm < INFINITY ? vm : 0.f;               // a NaN says nothing of the others' size
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) vm = fmaxf(vm, __shfl_xor_sync(FULL, vm, o));
              if (lane == 0) vmax_s[J & 3][warp - 10] = vm;
              mbar_arrive(scales_in + 8 * (J & 3));
            }
            constexpr int PER = KT * CR / 128, AT_ONCE = PER < 8 ? PER : 8;      // pieces of a thread; all read, then all written
            static_assert(PER % AT_ONCE == 0, "pieces");
#pragma unroll 1
            for (int x0 = 0; x0 < PER; x0 += AT_ONCE) {
              uint4 v[AT_ONCE];
#pragma unroll
              for (int x = 0; x < AT_ONCE; ++x) v[x] = lds128(src + 16u * (ct + 128 * (x0 + x)));
              if constexpr (FMT == KV_E4M3) {              // NaN codes of drafted values stay out of the product
                if (kv == 1 && (i + 1) * KT > seg.len) {
#pragma unroll
                  for (int x = 0; x < AT_ONCE; ++x) {
                    const int row = (ct + 128 * (x0 + x)) / CR;
                    if (i * KT + row >= seg.len && row < rows && drop_nan_codes(v[x])) atomicOr(&nan_s, 1u);
                  }
                }
              }
#pragma unroll
              for (int x = 0; x < AT_ONCE; ++x) {
                const int piece = ct + 128 * (x0 + x), row = piece / CR, c = piece % CR;
                // pieces c and c + 4 of a row go to the same banks of two atoms: they write their halves in turn
                const bool on = row < rows, turn = c >> 2;
                const uint32_t w[4] = {!on ? 0u : turn ? v[x].z : v[x].x, !on ? 0u : turn ? v[x].w : v[x].y,
                                       !on ? 0u : turn ? v[x].x : v[x].z, !on ? 0u : turn ? v[x].y : v[x].w};
                const uint32_t at = dst + (uint32_t)((c >> 2) * KT * 128 + row * 128), k = 2 * (c & 3) + turn;
#pragma unroll
                for (int y = 0; y < 2; ++y)
                  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + (((k ^ y) ^ row) & 7) * 16),
                               "r"(codes_to_f16x2<FMT, false>(w[2 * y])), "r"(codes_to_f16x2<FMT, true>(w[2 * y])),
                               "r"(codes_to_f16x2<FMT, false>(w[2 * y + 1])), "r"(codes_to_f16x2<FMT, true>(w[2 * y + 1]))
                               : "memory");
              }
            }
            fence_proxy_async_shared();
            mbar_arrive(full + 8 * s);
            mbar_arrive(rempty + 8 * r);
          }
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    static_assert(COPIES == 1 || SPLIT || NT == 3, "copies");
    constexpr int COLS = WIDE ? KT : KT / (SPLIT ? 4 : 2), NQ = COLS / 32;      // columns of a tile per thread
    static_assert(COLS == 32 || COLS == 64, "a thread's columns");
    constexpr int OC = WIDE ? D : D / 2;                   // columns of O that it looks after
    constexpr int RC = 128 / COPIES;                       // rows of a copy
    const int hw = warp >> 2, lrow = tid & 127;            // WIDE: team, else half of the columns; row of its tile
    const int copy = COPIES == 1 ? 0 : (warp & 3) * 32 / RC, row = COPIES == 1 ? lrow : lrow % RC;
    const int w = WIDE ? hw : 0, chunk0 = WIDE ? 0 : SPLIT ? 2 * copy + hw : NQ * hw;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t to = tb + lanes + w * D + (WIDE ? 0u : (uint32_t)(hw * OC));
    bool ok = true;
    int J0 = 0, seg_n = 0, exchanges = 0;
    // the other half's value of this row (WIDE: none)
    auto exchange = [&](float x, float& other) -> bool {
      half_s[exchanges & 1][hw][lrow] = x;
      mbar_arrive(halves);
      if (!mbar_wait_bounded(halves, (uint32_t)(exchanges & 1))) return false;
      other = half_s[exchanges & 1][hw ^ 1][lrow];
      ++exchanges;
      return true;
    };
    while (ok && next_segment(seg)) {
      const int nt = seg.te - seg.ta;
      const int h = seg.pair % a.Hkv;
      const int my_row = (WIDE ? 256 * seg.grp + 128 * w : 128 * seg.grp) + row;      // of the pair's R
      const bool live = my_row < R && (SPLIT || copy < NT);
      // a warp whose rows are all past R (or a copy without a term): their Q and so their S are zero, which as P is zero too. It takes no weights.
      const bool idle = my_row - lane >= R || (!SPLIT && copy >= NT);
      const int t = live ? my_row / a.G : 0, g = live ? my_row % a.G : 0;
      uint32_t* bad = bad_s[seg_n & 1];
      const TreeRow vis = {a.mask ? a.mask + ((size_t)seg.b * a.T + t) * a.mask_words : nullptr, t, seg.len, a.T};
      const size_t qrow = ((size_t)seg.b * a.T + t) * a.Hq + h * a.G + g;
      // ---- Q: WIDE each team its own tile, else the two halves every other chunk. 8 bits: f16, filled by a power of
      // two, which the row's scale takes back
      float row_scale_log2 = a.scale_log2;
      {
        const uint32_t dst = q0 + (uint32_t)(w * SH::QBYTES) + (uint32_t)lrow * 128u;
        auto put = [&](uint32_t tile, int c, uint4 v) {
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(tile + (uint32_t)((c >> 3) * 128 * 128 + ((c ^ lrow) & 7) * 16)),
                       "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
        };
        if constexpr (QF32) {
          const float* src = reinterpret_cast<const float*>(a.Q) + qrow * D;
          uint32_t mx = 0u;                                // the largest magnitude's bits
#pragma unroll 4
          for (int c = 0; c < D / 4; ++c) {
            const uint4 v = live ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0u, 0u, 0u, 0u);
            mx = max(max(mx, max(v.x & 0x7fffffffu, v.y & 0x7fffffffu)), max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
          }
          const int e = max((int)(mx >> 23) - 127, -112);
          const float f = pow2i(13 - e);
          row_scale_log2 = a.scale_log2 * pow2i((e - 13) / 2) * pow2i((e - 13) - (e - 13) / 2);
#pragma unroll 2
          for (int c = hw; c < D / 8; c += 2) {
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (live) load8(src + 8 * c, x);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              hi[k] = pack_f16x2(x[2 * k] * f, x[2 * k + 1] * f);
              const float2 h2 = __half22float2(*reinterpret_cast<const __half2*>(&hi[k]));
              lo[k] = pack_f16x2(x[2 * k] * f - h2.x, x[2 * k + 1] * f - h2.y);
            }
            put(dst, c, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            put(dst + SH::QBYTES, c, make_uint4(lo[0], lo[1], lo[2], lo[3]));
          }
        } else {
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.Q) + qrow * D);
          float f = 1.f;
          if constexpr (Q8) {
            uint32_t mx = 0u;                              // largest exponent field of a bf16
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const uint4 v = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
              const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) mx = max(mx, max((u[k] >> 7) & 0xffu, (u[k] >> 23) & 0xffu));
            }
            const int e = max((int)mx - 127, -112);
            f = pow2i(13 - e);
            row_scale_log2 = a.scale_log2 * pow2i((e - 13) / 2) * pow2i((e - 13) - (e - 13) / 2);
          }
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            if (!WIDE && (c & 1) != hw) continue;
            uint4 v = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
            if constexpr (Q8)
              v = make_uint4(pack_f16x2(bf16lo_to_f32(v.x) * f, bf16hi_to_f32(v.x) * f), pack_f16x2(bf16lo_to_f32(v.y) * f, bf16hi_to_f32(v.y) * f),
                             pack_f16x2(bf16lo_to_f32(v.z) * f, bf16hi_to_f32(v.z) * f), pack_f16x2(bf16lo_to_f32(v.w) * f, bf16hi_to_f32(v.w) * f));
            put(dst, c, v);
          }
        }
        if (tid < TR_MAX_DRAFT_WORDS) bad[tid] = 0u;
        fence_proxy_async_shared();
        mbar_arrive(qready);
      }
      // the rows of V that a product must not meet (done by the first team, whose product with a tile comes first)
      auto clear_rows = [&](int J, int j0) -> bool {
        const int n = 2 * J + 1;
        if (!mbar_wait_bounded(full + 8 * (n % NS), (uint32_t)((n / NS) & 1))) return false;
        const int pos = j0 + lrow;
        if (lrow < KT && pos >= seg.len) {
          const uint32_t vr = slot_of(n) + (uint32_t)lrow * 128u;
          bool clear = pos >= seg.len + a.T;
          if (!clear) {
            bool odd = false;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const uint4 x = lds128(vr + (uint32_t)((c >> 3) * KT * 128 + ((c ^ lrow) & 7) * 16));
              const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) odd |= (u[k] & 0x7f80u) == 0x7f80u || (u[k] & 0x7f800000u) == 0x7f800000u;
            }
            if (odd) {
              atomicOr(&bad[(pos - seg.len) >> 5], 1u << ((pos - seg.len) & 31));
              clear = true;
            }
          }
          if (clear) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
              asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(vr + (uint32_t)((c >> 3) * KT * 128 + c % 8 * 16)), "r"(0u)
                           : "memory");
          }
        }
        fence_proxy_async_shared();
        return true;
      };
      // how far (log2) a row's maximum may outgrow the m that its weights are relative to
      constexpr float LAZY = Q8 ? 1.f : 8.f;
      float m = -INFINITY, l = 0.f;
      int E = -127;                                        // 8 bits: weights are times vf = 2^(13 - E) and the value's scale
      float vf = pow2i(13 - E);
      for (int i = 0; i < nt && idle; ++i) {
        const int J = J0 + i, j0 = (seg.ta + i) * KT;
        float other;
        if (!mbar_wait_bounded(bar_of(sfull, w, J), par_of(J)) || (!WIDE && !exchange(-INFINITY, other)) ||
            (!WIDE && Q8 && j0 + KT > seg.len && !exchange(0.f, other)) ||
            (!Q8 && hw == 0 && j0 + KT > seg.len && !clear_rows(J, j0))) {
          ok = false;
          break;
        }
        mbar_arrive(bar_of(pready, w, J));
      }
      for (int i = 0; i < nt && !idle; ++i) {
        const int J = J0 + i, j0 = (seg.ta + i) * KT, jc = j0 + 32 * chunk0;
        const bool tail = j0 + KT > seg.len;
        if (!mbar_wait_bounded(bar_of(sfull, w, J), par_of(J))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t ts = tb + lanes + s_col(w, J & 1);
        uint32_t v[NQ][32];
        if constexpr (NQ == 2) tmem_ld64(ts + 32u * chunk0, v[0], v[NQ - 1]);
        else tmem_ld32(ts + 32u * chunk0, v[0]);
        int e = E;
        const uint32_t kss = scs + (uint32_t)((J & 3) * KT * 8) + 128u * chunk0;      // scales of this thread's keys, of their values
        if constexpr (Q8) {
          if (!mbar_wait_bounded(scales_in + 8 * (J & 3), (uint32_t)((J >> 2) & 1))) {
            ok = false;
            break;
          }
          float vm = 0.f;
          if (tail) {                                      // of the values that the row sees: an unseen one may be any size
#pragma unroll 1
            for (int q = 0; q < NQ; ++q) {
              uint32_t see = vis.sees(jc + 32 * q);
#pragma unroll 4
              for (int k = 0; k < 32; ++k, see >>= 1) {
                const float x = fabsf(lds_f32(kss + 4u * KT + 128u * q + 4u * k));
                if ((see & 1u) && x < INFINITY) vm = fmaxf(vm, x);
              }
            }
            if constexpr (!WIDE) {
              float other;
              if (!exchange(vm, other)) {
                ok = false;
                break;
              }
              vm = fmaxf(vm, other);
            }
          } else {
            vm = fmaxf(fmaxf(vmax_s[J & 3][0], vmax_s[J & 3][1]), fmaxf(vmax_s[J & 3][2], vmax_s[J & 3][3]));
          }
          e = max(E, (int)(__float_as_uint(vm) >> 23) - 127);
          // from here on v holds the logits: S times the row's or the key's scale alone may leave f32 where they do not
          const uint64_t rs2 = pack_f32x2(row_scale_log2, row_scale_log2);
#pragma unroll
          for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float x, y;
              unpack_f32x2(mul_f32x2(pack_f32x2(__uint_as_float(v[q][k]), __uint_as_float(v[q][k + 1])), mul_f32x2(lds_f32x2(kss + 128u * q + 4u * k), rs2)), x, y);
              v[q][k] = __float_as_uint(x);
              v[q][k + 1] = __float_as_uint(y);
            }
        }
        // ---- the row's maximum
        float mt = -INFINITY;
        const float logit_scale = Q8 ? 1.f : row_scale_log2;
        if (!tail && (Q8 || a.scale_log2 >= 0.f)) {
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            float x = __uint_as_float(v[q][0]), y = __uint_as_float(v[q][1]);      // two chains
#pragma unroll
            for (int k = 2; k < 32; k += 4) {
              x = max3(x, __uint_as_float(v[q][k]), __uint_as_float(v[q][k + 1]));
              if (k + 2 < 32) y = max3(y, __uint_as_float(v[q][k + 2]), __uint_as_float(v[q][k + 3]));
            }
            mt = max3(mt, x, y);
          }
          mt *= logit_scale;
        } else {                                           // masked, or an order that the scale turns round
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            const uint32_t see = vis.sees(jc + 32 * q);
#pragma unroll
            for (int k = 0; k < 32; ++k) mt = fmaxf(mt, (see >> k) & 1u ? __uint_as_float(v[q][k]) * logit_scale : -INFINITY);
          }
        }
        if constexpr (!WIDE) {
          float other;
          if (!exchange(mt, other)) {
            ok = false;
            break;
          }
          mt = fmaxf(mt, other);
        }
        bool fresh = i == 0;                               // the next product begins an O
        if constexpr (LONG) {
          if (i > 0 && i % FLUSH == 0) {
            if (!mbar_wait_bounded(bar_of(pvdone, w, J - 1), par_of(J - 1))) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            fresh = true;
#pragma unroll 1
            for (int q = 0; q < OC / 32; ++q) {
              uint32_t o[32], x[16], y[16];
              tmem_ld32(to + 32u * q, o);
              if (i > FLUSH) {
                uint32_t z[32];
                tmem_ld32(to + LCOL + 32u * q, z);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) + __uint_as_float(z[k]));
              }
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                x[k] = o[k];
                y[k] = o[16 + k];
              }
              tmem_st16(to + LCOL + 32u * q, x);
              tmem_st16(to + LCOL + 32u * q + 16u, y);
            }
            tmem_wait_st();
          }
        }
        // (both halves of a row come to the same answer: they have the same m and mt)
        if (__any_sync(FULL, mt > m + LAZY || (m == -INFINITY && mt > m) || e > E)) {
          const float mn = fmaxf(m, mt);
          float f = mn == -INFINITY ? 1.f : ex2(m - mn);
          m = mn;
          l *= f;
          if constexpr (Q8) {
            const float nf = pow2i(13 - e);
            f *= nf / vf;                                  // a power of two
            vf = nf;
            E = e;
          }
          // O (once the product before has left it at rest) and the long sum
          auto rescale = [&](uint32_t at) {
#pragma unroll 1
            for (int q = 0; q < OC / 32; ++q) {
              uint32_t o[32], x[16], y[16];
              tmem_ld32(at + 32u * q, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                x[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                y[k] = __float_as_uint(__uint_as_float(o[16 + k]) * f);
              }
              tmem_st16(at + 32u * q, x);
              tmem_st16(at + 32u * q + 16u, y);
            }
          };
          if (LONG && i >= FLUSH) rescale(to + LCOL);
          if (!fresh) {
            if (!mbar_wait_bounded(bar_of(pvdone, w, J - 1), par_of(J - 1))) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            rescale(to);
          }
        }
        const float ms = m == -INFINITY ? 0.f : m;
        // ---- weights, over the S that they come from
        auto weights = [&](auto mask_tag) {
          constexpr bool masked = decltype(mask_tag)::value;
          const uint64_t sc2 = pack_f32x2(logit_scale, logit_scale), ms2 = pack_f32x2(-ms, -ms);
          [[maybe_unused]] const uint64_t vf2 = pack_f32x2(vf, vf);
          uint64_t sum = 0ull;                             // (0, 0)
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            uint32_t t0[16];
            [[maybe_unused]] uint32_t t1v[16], t2[16];
            [[maybe_unused]] const uint32_t see = masked ? vis.sees(jc + 32 * q) : 0u;
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float x, y;
              const uint64_t s2 = pack_f32x2(__uint_as_float(v[q][k]), __uint_as_float(v[q][k + 1]));
              unpack_f32x2(Q8 ? add_f32x2(s2, ms2) : fma_f32x2(s2, sc2, ms2), x, y);
              x = ex2(x);
              y = ex2(y);
              if constexpr (masked) {
                if (!((see >> k) & 1u)) x = 0.f;
                if (!((see >> (k + 1)) & 1u)) y = 0.f;
              }
              sum = add_f32x2(sum, pack_f32x2(x, y));
              if constexpr (Q8) {
                unpack_f32x2(mul_f32x2(pack_f32x2(x, y), mul_f32x2(lds_f32x2(kss + 4u * KT + 128u * q + 4u * k), vf2)), x, y);
                if constexpr (masked) {                    // (0 times a NaN scale)
                  if (!((see >> k) & 1u)) x = 0.f;
                  if (!((see >> (k + 1)) & 1u)) y = 0.f;
                }
                t0[k / 2] = pack_f16x2(x, y);
                if constexpr (NT == 2) {
                  const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&t0[k / 2]));
                  t1v[k / 2] = pack_f16x2(x - hi.x, y - hi.y);
                }
              } else if constexpr (NT == 1) {
                t0[k / 2] = pack_bf16x2(x, y);
              } else {                                     // 8 bits cut off, 8 more, the rest rounded: 24 bits
                const float x1 = x - cut_bf16(x), y1 = y - cut_bf16(y);
                t0[k / 2] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
                t1v[k / 2] = __byte_perm(__float_as_uint(x1), __float_as_uint(y1), 0x7632);
                t2[k / 2] = pack_bf16x2(x1 - cut_bf16(x1), y1 - cut_bf16(y1));
              }
            }
            const uint32_t at = ts + 32u * (chunk0 + q);
            if constexpr (NT < 3) {
              tmem_st16(at, t0);
              if constexpr (NT == 2) tmem_st16(at + 16u, t1v);
              if constexpr (SPLIT) {
                uint32_t none[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) none[k] = 0u;
                const uint32_t others = ts + 32u * (chunk0 ^ 2);         // the same share of the other copy's keys
                tmem_st16(others, none);
                if constexpr (NT == 2) tmem_st16(others + 16u, none);
              }
            } else if constexpr (COPIES == 1) {
              tmem_st16(at, t0);
              tmem_st16(at + 16u, t1v);
              tmem_st16(ts + KT + 16u * (chunk0 + q), t2);
            } else if constexpr (COPIES == 2) {            // high | middle, then low | nothing
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                t0[k] = copy == 0 ? t0[k] : t1v[k];
                t2[k] = copy == 0 ? t2[k] : 0u;
              }
              tmem_st16(at, t0);
              tmem_st16(at + 16u, t2);
            } else {                                       // high | middle | low
#pragma unroll
              for (int k = 0; k < 16; ++k) t0[k] = copy == 0 ? t0[k] : copy == 1 ? t1v[k] : t2[k];
              tmem_st16(at, t0);
            }
          }
          float x, y;
          unpack_f32x2(sum, x, y);
          l += x + y;
        };
        if (tail) weights(std::true_type{});
        else weights(std::false_type{});
        if (!Q8 && tail && hw == 0 && !clear_rows(J, j0)) {
          ok = false;
          break;
        }
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(bar_of(pready, w, J));
      }
      if (!ok) break;
      if constexpr (!WIDE) {
        float other;
        if (!exchange(l, other)) {
          ok = false;
          break;
        }
        l = hw == 0 ? l + other : other + l;
      }
      J0 += nt;
      if (!mbar_wait_bounded(bar_of(pvdone, w, J0 - 1), par_of(J0 - 1))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      // ---- the team's partial of the row
      // (copies that hold terms of the same weights add up, and the sum of weights is the first one's)
      float* out = a.part + (((size_t)(blockIdx.x + seg.unit) * p.parts + (WIDE ? w : copy)) * p.rows + row) * (D + 2);
      if (!SPLIT && copy > 0) l = 0.f;
      uint32_t any_bad = 0u;
#pragma unroll
      for (int k = 0; k < TR_MAX_DRAFT_WORDS; ++k) any_bad |= bad[k];
#pragma unroll 1
      for (int q = 0; q < OC / 32 && !idle; ++q) {
        const int col = (WIDE ? 0 : hw * OC) + 32 * q;
        uint32_t o[32];
        tmem_ld32(to + 32u * q, o);
        if constexpr (LONG) {
          if (nt > FLUSH) {
            uint32_t z[32];
            tmem_ld32(to + LCOL + 32u * q, z);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) + __uint_as_float(z[k]));
          }
        }
        if constexpr (Q8) {
          const float of = 1.f / vf;                       // a power of two
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * of);
        }
        if (!Q8 && any_bad != 0u && live && copy == 0) {                       // rare: drafted keys left out of the products
          for (int i = 0; i < a.T; ++i) {
            if (!((bad[i >> 5] >> (i & 31)) & 1u) || !((vis.drafts(i >> 5) >> (i & 31)) & 1u)) continue;
            const size_t kr = ((size_t)seg.pair * a.Ncap + seg.len + i) * D;
            const __nv_bfloat16 *qp = reinterpret_cast<const __nv_bfloat16*>(a.Q) + qrow * D,
                                *kp = reinterpret_cast<const __nv_bfloat16*>(a.K) + kr,
                                *vp = reinterpret_cast<const __nv_bfloat16*>(a.V) + kr + col;
            float s = 0.f;
            for (int c = 0; c < D; ++c) s = fmaf(__bfloat162float(qp[c]), __bfloat162float(kp[c]), s);
            const float x = ex2(s * a.scale_log2 - (m == -INFINITY ? 0.f : m));
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(fmaf(x, __bfloat162float(vp[k]), __uint_as_float(o[k])));
          }
        }
        if (row < p.rows) {
#pragma unroll
          for (int k = 0; k < 32; k += 2) *reinterpret_cast<uint2*>(out + 2 + col + k) = make_uint2(o[k], o[k + 1]);
        }
      }
      if constexpr (FMT == KV_E4M3) {                      // rare: a weight times a NaN, for the rows that see its key
        if (nan_s != 0u && live) {
          int unit = seg.unit, r = my_row;                 // all else anew: kept in registers up to here it cost the tiles 2 to 3%
          asm volatile("" : "+r"(unit), "+r"(r));
          const int pair = unit / p.groups, b = pair / a.Hkv, len = seq_len(a.lens, b, a.N), col = WIDE ? 0 : hw * OC;
          const TreeRow sees = {a.mask ? a.mask + ((size_t)b * a.T + r / a.G) * a.mask_words : nullptr, r / a.G, len, a.T};
          const unsigned char* vp = reinterpret_cast<const unsigned char*>(a.V) + ((size_t)pair * a.Ncap + len) * D + col;
#pragma unroll 1
          for (int i = 0; i < a.T; ++i, vp += D) {
            if (!((sees.drafts(i >> 5) >> (i & 31)) & 1u)) continue;
#pragma unroll 1
            for (int c = 0; c < OC; ++c)
              if ((vp[c] & 0x7f) == 0x7f) out[2 + col + c] = __uint_as_float(0x7fc00000u);
          }
        }
        __syncwarp();
      }
      if (row < p.rows && !idle && (WIDE || hw == 0)) *reinterpret_cast<float2*>(out) = make_float2(m, l);
      tc_fence_before_sync();                              // O has been read before the next segment's products
      ++seg_n;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after_sync();
    tmem_dealloc(tb, 512u);
  }
}

// Joins the rows' partials in order: 8 / WPR rows to a block, WPR warps to a row, each taking every WPR-th partial (a few
// pairs on many blocks leave many partials to a row). grid = (ceil(R WPR / 8), pairs).
template <int D, int KT, bool WIDE, int WPR, typename OT>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeParams p, OT* O, int B, int blocks) {
  __shared__ float sm[8], sl[8];
  __shared__ float2 so[8][D / 2];
  const CacheAttendParams& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % WPR;
  const int my_row = blockIdx.x * (8 / WPR) + warp / WPR;
  const int pair = blockIdx.y, b = pair / a.Hkv, h = pair % a.Hkv;
  const int per = tree_tiles<KT>(a, b);
  const StreamRuns runs = tree_runs<KT>(p, B, blocks);
  const int grp = my_row / (WIDE ? 256 : 128), row = my_row % 128;
  // a run has one partial of a row, or one for each copy
  const int k0 = WIDE ? (my_row >> 7) & 1 : 0, kn = WIDE ? 1 : min(p.parts, 3);
  const int unit = pair * p.groups + grp;
  int first = (h * p.groups + grp) * per;                  // the unit's first tile
  for (int i = 0; i < b; ++i) first += a.Hkv * p.groups * tree_tiles<KT>(a, i);
  const int i0 = runs.of(first), i1 = runs.of(first + per - 1);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int C = D / 64;                                // pairs of columns per lane
  const bool live = my_row < a.T * a.G;
  float m = -INFINITY, l = 0.f;
  float2 o[C];
#pragma unroll
  for (int c = 0; c < C; ++c) o[c] = make_float2(0.f, 0.f);
  auto add = [&](float pm, float pl, const float2 (&po)[C]) {
    const float mn = fmaxf(m, pm);
    const float f0 = mn == -INFINITY ? 1.f : ex2(m - mn), f1 = mn == -INFINITY ? 1.f : ex2(pm - mn);
    m = mn;
    l = fmaf(f1, pl, l * f0);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      o[c].x = fmaf(f1, po[c].x, o[c].x * f0);
      o[c].y = fmaf(f1, po[c].y, o[c].y * f0);
    }
  };
  if (live) {
#pragma unroll 2
    for (int i = i0 + part; i <= i1; i += WPR) {
      for (int k = k0; k < k0 + kn; ++k) {
        const float2* q = reinterpret_cast<const float2*>(a.part + (((size_t)(i + unit) * p.parts + k) * p.rows + row) * (D + 2));
        const float2 ml = __ldcg(q);
        float2 x[C];
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = __ldcg(q + 1 + 32 * c + lane);
        add(ml.x, ml.y, x);
      }
    }
  }
  if constexpr (WPR > 1) {
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) so[warp][32 * c + lane] = o[c];
    __syncthreads();
    if (part > 0) return;
    for (int x = 1; x < WPR; ++x) {
      float2 y[C];
#pragma unroll
      for (int c = 0; c < C; ++c) y[c] = so[warp + x][32 * c + lane];
      add(sm[warp + x], sl[warp + x], y);
    }
  }
  if (!live) return;
  OT* out = O + (((size_t)b * a.T + my_row / a.G) * a.Hq + h * a.G + my_row % a.G) * D;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const float x = l == 0.f ? 0.f : o[c].x / l, y = l == 0.f ? 0.f : o[c].y / l;
    if constexpr (sizeof(OT) == 2) *reinterpret_cast<uint32_t*>(out + 64 * c + 2 * lane) = pack_bf16x2(x, y);
    else *reinterpret_cast<float2*>(out + 64 * c + 2 * lane) = make_float2(x, y);
  }
}

}  // namespace hst
