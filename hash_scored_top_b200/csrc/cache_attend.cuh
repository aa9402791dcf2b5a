// Attention over a cache in any of its formats, for R = T * G query rows per
// KV head: T query tokens of a sequence times the G query heads of the group
// (row t * G + g). The keys of a pair are a run of positions:
//   all     position j is row j of the cache, seen if j < the sequence's length;
//   listed  position j is row idx[j], seen if that is a row of the cache;
//   blocks  position j is row j % block of block idx[j / block], seen if the
//           entry is not negative and the row lies below the length;
//   tree    positions below the length are seen by every token, and position
//           length + i, drafted key i < T, by the tokens whose mask has bit i.
//
// Softmax in the log2 domain with a running maximum m and sum l per row, all
// in f32; a key that a row does not see is never read for it, so what lies in
// its place (infinities, NaN) cannot reach the row. A split of the positions
// gives (m, l, o[D]) per row; the merge adds the splits in their order and
// divides, which makes the result independent of the order the splits ran in.
// A row that sees nothing gets 0.
#pragma once

#include "attend.cuh"
#include "quant.cuh"

namespace hst {

enum KeyMode { KEYS_ALL = 0, KEYS_LISTED = 1, KEYS_BLOCKS = 2, KEYS_TREE = 3 };

struct CacheAttendParams {
  const void* Q;             // [B][T][Hq][D], f32 or bf16
  const void* K;             // [pairs][Ncap][D]
  const void* V;
  const float* scales;       // [pairs][Ncap][2] (8-bit formats)
  const int* lens;           // optional [B]
  const int* idx;            // listed: [pairs][k] rows; blocks: [pairs][k] blocks
  const uint32_t* mask;      // tree: optional [B][T][mask_words]; null: token t sees drafts 0 .. t
  float* part;               // [pairs][R][splits][D + 2]: (m, l, o[D])
  int Hq, Hkv, T, G, Ncap, N, k, block, mask_words;
  int n;                     // positions (an upper bound of a pair's)
  int mode;                  // KeyMode
  int splits;
  float scale_log2;          // scale * log2(e)
};

__device__ __forceinline__ int seq_len(const int* lens, int b, int N) {
  return lens ? min(max(__ldg(lens + b), 0), N) : N;
}

// What position j of a pair is (but for KEYS_ALL): its cache row, or -1 when it is not seen. The list may be the previous
// kernel's, which still runs when this one starts, so it is not read as constant data (__ldg).
__device__ __forceinline__ int key_row(const CacheAttendParams& p, int pair, int b, int t, int len, int j) {
  if (p.mode == KEYS_LISTED) {
    const int r = __ldcg(p.idx + (size_t)pair * p.k + j);
    return r >= 0 && r < p.Ncap ? r : -1;
  }
  if (p.mode == KEYS_BLOCKS) {
    const int bl = __ldcg(p.idx + (size_t)pair * p.k + j / p.block);
    if (bl < 0 || bl > (len - 1) / p.block) return -1;
    const int r = bl * p.block + j % p.block;
    return r < len ? r : -1;
  }
  if (j < len) return j;
  const int i = j - len;
  if (i >= p.T) return -1;
  const bool sees = p.mask ? (__ldg(p.mask + ((size_t)b * p.T + t) * p.mask_words + (i >> 5)) >> (i & 31)) & 1u : i <= t;
  return sees ? j : -1;
}

// Values 4q .. 4q + 3 of a row of f32 or bf16.
template <int FMT>
__device__ __forceinline__ float4 row_quad(const void* base, size_t row, int D, int q) {
  const size_t e = row * D + 4 * q;
  if constexpr (FMT == KV_F32) return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + e);
  const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(base) + e);
  return make_float4(bf16lo_to_f32(w.x), bf16hi_to_f32(w.x), bf16lo_to_f32(w.y), bf16hi_to_f32(w.y));
}

constexpr int CACHE_THREADS = 256;

// The simple kernel, for f32 caches: a warp per key. Bound by its instructions:
// 97 chosen blocks of 32 keys, 32 pairs, G = 4, D = 128 take 92 us, where
// stream_attend_kernel takes 16 for a bf16 cache.
// grid = (splits, R, pairs); warp w takes the split's positions w, w + 8, ...
// and its lanes the head dimension.
template <int D>
__global__ void __launch_bounds__(CACHE_THREADS) cache_attend_rows_kernel(const CacheAttendParams p) {
  constexpr int NW = CACHE_THREADS / 32, QL = D / 4;      // QL lanes hold a row (4 values each)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int split = blockIdx.x, R = p.T * p.G;
  const int row = blockIdx.y, pair = blockIdx.z, b = pair / p.Hkv, t = row / p.G;
  const int head = (pair % p.Hkv) * p.G + row % p.G;
  const int len = seq_len(p.lens, b, p.N);
  float q[4] = {0.f, 0.f, 0.f, 0.f};
  const bool on = lane < QL;
  if (on) {
    const size_t row0 = ((size_t)b * p.T + t) * p.Hq + head;
    const float4 v = row_quad<KV_F32>(p.Q, row0, D, lane);
    q[0] = v.x * p.scale_log2;
    q[1] = v.y * p.scale_log2;
    q[2] = v.z * p.scale_log2;
    q[3] = v.w * p.scale_log2;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");      // idx may be the previous kernel's
  const int j0 = (int)((long long)split * p.n / p.splits), j1 = (int)((long long)(split + 1) * p.n / p.splits);
  const size_t base = (size_t)pair * p.Ncap;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = j0 + warp; j < j1; j += NW) {
    const int r = key_row(p, pair, b, t, len, j);
    if (r < 0) continue;
    float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
    if (on) {
      kv = row_quad<KV_F32>(p.K, base + r, D, lane);
      vv = row_quad<KV_F32>(p.V, base + r, D, lane);
    }
    float s = warp_sum(fmaf(q[0], kv.x, fmaf(q[1], kv.y, fmaf(q[2], kv.z, q[3] * kv.w))));
    const float mn = fmaxf(m, s);
    const float al = mn == -INFINITY ? 1.f : exp2f(m - mn);
    const float pr = s == -INFINITY ? 0.f : exp2f(s - mn);    // a NaN logit stays one
    m = mn;
    l = fmaf(l, al, pr);
    o[0] = fmaf(o[0], al, pr * vv.x);
    o[1] = fmaf(o[1], al, pr * vv.y);
    o[2] = fmaf(o[2], al, pr * vv.z);
    o[3] = fmaf(o[3], al, pr * vv.w);
  }
  __shared__ float sm[NW], sl[NW], so[NW][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  if (on) *reinterpret_cast<float4*>(&so[warp][4 * lane]) = make_float4(o[0], o[1], o[2], o[3]);
  __syncthreads();
  float mm = -INFINITY;
#pragma unroll
  for (int w = 0; w < NW; ++w) mm = fmaxf(mm, sm[w]);
  float* out = p.part + (((size_t)pair * R + row) * p.splits + split) * (D + 2);
  for (int e = threadIdx.x; e < D + 1; e += CACHE_THREADS) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = mm == -INFINITY ? 0.f : exp2f(sm[w] - mm);
      a = fmaf(f, e < D ? so[w][e] : sl[w], a);
    }
    out[e < D ? 2 + e : 1] = a;
  }
  if (threadIdx.x == 0) out[0] = mm;
}

// Adds a row's splits in order: O = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.
// grid = (R, pairs), one warp per 32 columns.
struct CacheMergeParams {
  const float* part;
  void* O;                   // [B][T][Hq][D], f32 or bf16
  int Hq, Hkv, T, G, splits;
};

template <int D, typename OT>
__global__ void __launch_bounds__(D) cache_merge_kernel(const CacheMergeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int row = blockIdx.x, pair = blockIdx.y, R = p.T * p.G, c = threadIdx.x;
  const float* part = p.part + ((size_t)pair * R + row) * p.splits * (D + 2);
  float mm = -INFINITY;
  for (int s = 0; s < p.splits; ++s) mm = fmaxf(mm, __ldcg(part + (size_t)s * (D + 2)));
  float l = 0.f, o = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float* q = part + (size_t)s * (D + 2);
    const float m = __ldcg(q);
    if (m == -INFINITY && !(__ldcg(q + 1) != 0.f)) continue;      // nothing seen (a NaN sum still counts)
    const float f = m == -INFINITY ? 1.f : exp2f(m - mm);
    l = fmaf(f, __ldcg(q + 1), l);
    o = fmaf(f, __ldcg(q + 2 + c), o);
  }
  const int head = (pair % p.Hkv) * p.G + row % p.G;
  const size_t at = (((size_t)(pair / p.Hkv) * p.T + row / p.G) * p.Hq + head) * D + c;
  const float v = l == 0.f ? 0.f : o / l;
  reinterpret_cast<OT*>(p.O)[at] = (OT)v;
}

}  // namespace hst
