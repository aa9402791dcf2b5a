// C ABI of the operators over quantised, block-selected and drafted caches:
// argument validation, launch planning and launches, under the rules of
// api.cu (everything is checked on the host before anything is launched,
// nothing is allocated, all work is asynchronous on the caller's stream).
#include <algorithm>
#include <atomic>
#include <climits>

#include "host.cuh"
#include "blocks.cuh"
#include "cache_attend.cuh"
#include "quant.cuh"
#include "stream_attend.cuh"
#include "tree_attend.cuh"

using namespace hst;

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// A kernel launch, as the programmatic dependent of the kernel before it on
// the stream if `pdl` (it waits before it reads what that kernel writes).
template <typename... Params>
int launch(void (*kern)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, bool pdl, const char* what,
           const std::type_identity_t<Params>&... p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p...);
  if (e != cudaSuccess) return fail(SK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

// ---------------------------------------------------------------- checks
bool is_8bit(int kv) { return kv == SK_INT8 || kv == SK_E4M3; }

int check_8bit(sk_dtype kv) {
  if (!is_8bit(kv)) return fail(SK_ERR_INVALID_ARG, "cache dtype %d: SK_INT8 or SK_E4M3 expected", (int)kv);
  return SK_OK;
}

// Any format of cache, its scales, and a query type that goes with it.
int check_formats(sk_dtype q, sk_dtype kv, const float* scales) {
  SK_TRY(check_dtype(q));
  if (is_8bit(kv)) {
    SK_NONNULL(scales);
    SK_ALIGNED(scales, 16);
    return SK_OK;
  }
  SK_TRY(check_dtype(kv));
  if (q != kv) return fail(SK_ERR_INVALID_ARG, "Q has dtype %d, the cache %d: they must be the same", (int)q, (int)kv);
  return SK_OK;
}

int check_grid(int B, int Hq, int Hkv, int d) {
  SK_TRY(check_heads(B, Hq, Hkv, d));
  if ((long long)B * Hkv > 65535) return fail(SK_ERR_UNSUPPORTED, "B * Hkv = %lld > 65535", (long long)B * Hkv);
  if (Hq / Hkv > 8) return fail(SK_ERR_UNSUPPORTED, "group size G=%d > 8", Hq / Hkv);
  return SK_OK;
}

// Rows of a pair at most: a tile's, or a block's, more can be counted in 32 bits.
constexpr int kMaxRows = INT_MAX - 512;
// Keys that one call attends to, or writes, per pair at most.
constexpr int kMaxPositions = 1 << 30;

int check_ncap(int Ncap) {
  if (Ncap > kMaxRows) return fail(SK_ERR_UNSUPPORTED, "Ncap=%d: at most %d rows per pair", Ncap, kMaxRows);
  if (Ncap < 32 || Ncap % 32) return fail(SK_ERR_INVALID_ARG, "Ncap=%d must be a positive multiple of 32", Ncap);
  return SK_OK;
}

int check_rows(const int* starts, int Ncap, int n_begin, int n_count) {
  SK_TRY(check_ncap(Ncap));
  if (n_count < 0 || n_count > kMaxPositions)
    return fail(SK_ERR_INVALID_ARG, "n_count=%d must be in [0, %d]", n_count, kMaxPositions);
  if (starts == nullptr && (n_begin < 0 || (long long)n_begin + n_count > Ncap))
    return fail(SK_ERR_INVALID_ARG, "key range [%d, %d+%d) outside [0, Ncap=%d)", n_begin, n_begin, n_count, Ncap);
  return SK_OK;
}

int check_block(int block) {
  if (block != 16 && block != 32 && block != 64 && block != 128)
    return fail(SK_ERR_UNSUPPORTED, "block=%d: 16, 32, 64 or 128 keys", block);
  return SK_OK;
}

int check_ws(const void* ws, size_t got, size_t need) {
  if (need > 0 && (ws == nullptr || got < need))
    return fail(SK_ERR_WORKSPACE, "workspace: need %zu bytes, got %zu", need, ws == nullptr ? (size_t)0 : got);
  SK_ALIGNED(ws, 16);
  return SK_OK;
}

// ---------------------------------------------------------------- attention
// Splits of a pair's positions: about four blocks per SM over all rows.
int rows_splits(int pairs, int R, int n) {
  const long long rows = (long long)pairs * R;
  const long long want = (4LL * kNumSMs + rows - 1) / rows;
  return (int)std::max(1LL, std::min(want, (long long)(n + 63) / 64));
}

// Blocks of the stream kernel: one per SM, fewer when there are fewer than 12
// tiles (one for each warp) to a block. A block takes its pairs one after another,
// so pairs of one or two tiles leave most of its warps idle: 64 pairs of 32 keys
// run on 6 blocks and take 56 us, 512 pairs of 100 keys on 148 and 26.
int stream_blocks(int pairs, int n) {
  const long long tiles = (long long)pairs * ((n + 31) / 32);
  return (int)std::max(1LL, std::min((long long)kNumSMs, (tiles + 11) / 12));
}

// Query rows that a block of the tree kernel takes at once: 128, or, for more
// rows and bf16 outputs, 256 (two teams that share each K and V tile).
bool tree_wide(int R, sk_dtype o) { return R > 128 && o == SK_BF16; }
int tree_groups(int R, bool wide) { return wide ? (R + 255) / 256 : (R + 127) / 128; }

// Copies of the rows that share 128 rows of an MMA, at most. bf16 caches and f32
// outputs: they hold the three terms of the weights (two products for 64 rows, one
// for 32). 8-bit caches: two, which share a tile's keys, so that the softmax threads
// of all lanes are busy.
int tree_copies(int R) { return R > 64 ? 1 : R > 32 ? 2 : 4; }

// Partials: (blocks + units) runs of one or two teams', or copies', rows.
size_t tree_bytes(int pairs, int R, int d) {
  size_t most = 0;
  for (const sk_dtype o : {SK_F32, SK_BF16}) {
    const bool wide = tree_wide(R, o);
    most = std::max(most, (kNumSMs + (size_t)pairs * tree_groups(R, wide)) * (wide ? 2 : tree_copies(R)));
  }
  return align256(most * std::min(R, 128) * (d + 2) * sizeof(float));
}

// Workspace of the attention of R rows per pair: the larger of what its
// kernels need (the query does not know the cache's format).
size_t attend_bytes(int pairs, int R, int n, int d) {
  const size_t rows = (size_t)pairs * R * rows_splits(pairs, R, n) * (d + 2) * sizeof(float);
  const size_t stream = R <= 8 ? (size_t)(stream_blocks(pairs, n) + pairs) * R * (d + 2) * sizeof(float) : 0;
  return align256(std::max(rows, stream));
}

// Allows a kernel its dynamic shared memory on the current device (once per
// kernel and device; setting it twice does no harm).
template <auto Kern>
int allow_smem(size_t smem) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch("cudaGetDevice");
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return SK_OK;
  if (cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return check_launch("cudaFuncSetAttribute");
  done.fetch_or(bit, std::memory_order_relaxed);
  return SK_OK;
}

template <int D, int FMT, bool QF32>
int launch_stream(const CacheAttendParams& p, int B, float* O, bool pdl, cudaStream_t s) {
  using SH = StreamShape<D, FMT>;
  StreamParams sp;
  sp.a = p;
  const int blocks = stream_blocks(B * p.Hkv, p.n);
  // listed rows are those of a quantised cache: bf16 caches have socket_sparse_attend
  constexpr bool CAN_LIST = FMT != KV_BF16;
  if (CAN_LIST && p.mode == KEYS_LISTED) {
    SK_TRY((allow_smem<stream_attend_kernel<D, FMT, QF32, CAN_LIST>>(SH::SMEM)));
    SK_TRY(launch(stream_attend_kernel<D, FMT, QF32, CAN_LIST>, dim3(blocks), SH::THREADS, SH::SMEM, s, pdl,
                  "stream_attend_kernel", sp, B));
  } else {
    SK_TRY((allow_smem<stream_attend_kernel<D, FMT, QF32, false>>(SH::SMEM)));
    SK_TRY(launch(stream_attend_kernel<D, FMT, QF32, false>, dim3(blocks), SH::THREADS, SH::SMEM, s, pdl,
                  "stream_attend_kernel", sp, B));
  }
  return launch(stream_merge_kernel<D, SH::TILE>, dim3(p.G, B * p.Hkv), 4 * D, 0, s, true, "stream_merge_kernel", sp, O, B,
                blocks);
}

template <int D>
int stream_attend(const CacheAttendParams& p, sk_dtype q, sk_dtype kv, int B, float* O, bool pdl, cudaStream_t s) {
  const bool f = q == SK_F32;
  return kv == SK_BF16   ? launch_stream<D, KV_BF16, false>(p, B, O, pdl, s)
         : kv == SK_INT8 ? (f ? launch_stream<D, KV_INT8, true>(p, B, O, pdl, s) : launch_stream<D, KV_INT8, false>(p, B, O, pdl, s))
                         : (f ? launch_stream<D, KV_E4M3, true>(p, B, O, pdl, s) : launch_stream<D, KV_E4M3, false>(p, B, O, pdl, s));
}

// Drafted tokens over a bf16 or 8-bit cache, on tcgen05.
template <int D, int KT, int NT, bool WIDE, int COPIES, int FMT, bool QF32 = false, typename OT>
int launch_tree(const CacheAttendParams& a, int B, OT* O, cudaStream_t s) {
  using SH = TreeShape<D, KT, WIDE, FMT != KV_BF16, QF32>;
  TreeParams p;
  p.a = a;
  p.groups = tree_groups(a.T * a.G, WIDE);
  p.rows = std::min(a.T * a.G, 128);
  p.parts = WIDE ? 2 : COPIES;
  const int pairs = B * a.Hkv, R = a.T * a.G;
  const long long units = (long long)pairs * p.groups, tiles = units * ((a.n + KT - 1) / KT);
  const int blocks = (int)std::min((long long)kNumSMs, tiles);
  CUtensorMap mk = {}, mv = {};
  if (FMT == KV_BF16) {
    SK_TRY(encode_rows_map(&mk, a.K, (long)pairs * a.Ncap, D, KT));
    SK_TRY(encode_rows_map(&mv, a.V, (long)pairs * a.Ncap, D, KT));
  }
  SK_TRY((allow_smem<tree_attend_kernel<D, KT, NT, WIDE, COPIES, FMT, QF32>>(SH::SMEM)));
  SK_TRY(launch(tree_attend_kernel<D, KT, NT, WIDE, COPIES, FMT, QF32>, dim3(blocks), SH::THREADS, SH::SMEM, s, false,
                "tree_attend_kernel", p, B, mk, mv));
  // about blocks / units partials to a row: one warp takes a few, eight take many
  if (blocks > 6 * units)
    return launch(tree_merge_kernel<D, KT, WIDE, 8, OT>, dim3(R, pairs), 256, 0, s, true, "tree_merge_kernel", p, O, B, blocks);
  return launch(tree_merge_kernel<D, KT, WIDE, 1, OT>, dim3((R + 7) / 8, pairs), 256, 0, s, true, "tree_merge_kernel", p, O, B,
                blocks);
}

template <int D, int FMT>
int tree_attend(const CacheAttendParams& a, sk_dtype q, int B, void* O, sk_dtype o, cudaStream_t s) {
  const int R = a.T * a.G;
  if constexpr (FMT != KV_BF16) {
    constexpr int KT = 64;                                 // (two Q tiles of D = 128 leave no room for tiles of 128 keys)
    if (q == SK_F32)
      return o == SK_F32 ? launch_tree<D, KT, 2, false, 1, FMT, true>(a, B, reinterpret_cast<float*>(O), s)
                         : launch_tree<D, KT, 2, false, 1, FMT, true>(a, B, reinterpret_cast<__nv_bfloat16*>(O), s);
  }
  if (o == SK_F32) {
    float* out = reinterpret_cast<float*>(O);
    if constexpr (FMT == KV_BF16) {
      const int copies = tree_copies(R);
      return copies == 4   ? launch_tree<D, 128, 3, false, 4, FMT>(a, B, out, s)
             : copies == 2 ? launch_tree<D, 128, 3, false, 2, FMT>(a, B, out, s)
                           : launch_tree<D, D == 128 ? 64 : 128, 3, false, 1, FMT>(a, B, out, s);
    } else {
      return R <= 64 ? launch_tree<D, 128, 2, false, 2, FMT>(a, B, out, s) : launch_tree<D, 128, 2, false, 1, FMT>(a, B, out, s);
    }
  }
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(O);
  if constexpr (FMT != KV_BF16)
    if (R <= 64) return launch_tree<D, 128, 1, false, 2, FMT>(a, B, out, s);
  return tree_wide(R, o) ? launch_tree<D, 64, 1, true, 1, FMT>(a, B, out, s) : launch_tree<D, 128, 1, false, 1, FMT>(a, B, out, s);
}

template <int D>
int tree_attend(const CacheAttendParams& a, sk_dtype q, sk_dtype kv, int B, void* O, sk_dtype o, cudaStream_t s) {
  return kv == SK_BF16   ? tree_attend<D, KV_BF16>(a, q, B, O, o, s)
         : kv == SK_INT8 ? tree_attend<D, KV_INT8>(a, q, B, O, o, s)
                         : tree_attend<D, KV_E4M3>(a, q, B, O, o, s);
}

// Attention over the positions that `p` describes (all of it but part, splits
// and the query's place), then the merge of its splits into O.
int attend(CacheAttendParams p, sk_dtype q, sk_dtype kv, int B, int d, float scale, void* O, sk_dtype o, void* ws,
           bool pdl, cudaStream_t s) {
  const int pairs = B * p.Hkv, R = p.T * p.G;
  if ((long long)pairs * ((p.n + 15LL) / 16) > INT_MAX)
    return fail(SK_ERR_UNSUPPORTED, "more than 2^31 - 1 tiles of 16 keys");
  p.scale_log2 = scale * kLog2e;
  p.part = reinterpret_cast<float*>(ws);
  if (kv != SK_F32 && p.mode != KEYS_TREE)
    return d == 128 ? stream_attend<128>(p, q, kv, B, reinterpret_cast<float*>(O), pdl, s)
                    : stream_attend<64>(p, q, kv, B, reinterpret_cast<float*>(O), pdl, s);
  if (kv != SK_F32)
    return d == 128 ? tree_attend<128>(p, q, kv, B, O, o, s) : tree_attend<64>(p, q, kv, B, O, o, s);
  p.splits = rows_splits(pairs, R, p.n);
  SK_TRY(launch(d == 128 ? cache_attend_rows_kernel<128> : cache_attend_rows_kernel<64>, dim3(p.splits, R, pairs), CACHE_THREADS, 0,
                s, pdl, "cache_attend_rows_kernel", p));
  CacheMergeParams m;
  m.part = p.part;
  m.O = O;
  m.Hq = p.Hq;
  m.Hkv = p.Hkv;
  m.T = p.T;
  m.G = p.G;
  m.splits = p.splits;
  auto merge = d == 128 ? (o == SK_BF16 ? cache_merge_kernel<128, __nv_bfloat16> : cache_merge_kernel<128, float>)
                        : (o == SK_BF16 ? cache_merge_kernel<64, __nv_bfloat16> : cache_merge_kernel<64, float>);
  return launch(merge, dim3(R, pairs), d, 0, s, true, "cache_merge_kernel", m);
}

CacheAttendParams cache_params(const void* Q, const void* K, const void* V, const float* scales, const int* lens, int Hq,
                               int Hkv, int Ncap, int N) {
  CacheAttendParams p = {};
  p.Q = Q;
  p.K = K;
  p.V = V;
  p.scales = scales;
  p.lens = lens;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.T = 1;
  p.G = Hq / Hkv;
  p.Ncap = Ncap;
  p.N = N;
  return p;
}

// ---------------------------------------------------------------- blocks
int num_blocks(int Ncap, int block) { return (Ncap + block - 1) / block; }

size_t select_bytes(int pairs, int Ncap, int block) { return align256((size_t)pairs * num_blocks(Ncap, block) * 4); }

int check_select(const void* Q, sk_dtype q, const void* bsum, int B, int Hq, int Hkv, int Ncap, int N, int d, int block,
                 int k, int n_first, int n_last) {
  SK_NONNULL(Q);
  SK_NONNULL(bsum);
  SK_ALIGNED(Q, 16);
  SK_ALIGNED(bsum, 16);
  SK_TRY(check_dtype(q));
  SK_TRY(check_grid(B, Hq, Hkv, d));
  SK_TRY(check_ncap(Ncap));
  SK_TRY(check_cache(Ncap, N));
  SK_TRY(check_block(block));
  if (k < 1 || (long long)k * block > kMaxPositions) return fail(SK_ERR_INVALID_ARG, "k=%d blocks of %d keys", k, block);
  if (n_first < 0 || n_last < 0 || (long long)n_first + n_last > k)
    return fail(SK_ERR_INVALID_ARG, "n_first=%d and n_last=%d must be >= 0 and at most k=%d together", n_first, n_last, k);
  return SK_OK;
}

template <int D, typename QT>
int launch_select(const BlockSelectParams& p, int pairs, int C, size_t smem, cudaStream_t s) {
  SK_TRY((allow_smem<block_select_kernel<D, QT>>(BSEL_MAX_KEYS * 4)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pairs * C);
  cfg.blockDim = dim3(BSEL_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, block_select_kernel<D, QT>, p, C);
  if (e != cudaSuccess) return fail(SK_ERR_CUDA, "block_select_kernel: %s", cudaGetErrorString(e));
  return check_launch("block_select_kernel");
}

int select_impl(const void* Q, sk_dtype q, const void* bsum, const int* lens, int B, int Hq, int Hkv, int Ncap, int N,
                int d, int block, int k, int n_first, int n_last, int* idx, void* ws, cudaStream_t s) {
  BlockSelectParams p;
  p.Q = Q;
  p.bsum = reinterpret_cast<const __nv_bfloat16*>(bsum);
  p.lens = lens;
  p.keys = reinterpret_cast<uint32_t*>(ws);
  p.idx = idx;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.NB = num_blocks(Ncap, block);
  p.N = N;
  p.block = block;
  p.k = k;
  p.n_first = n_first;
  p.n_last = n_last;
  const int pairs = B * Hkv, most = num_blocks(N, block);
  const bool on_chip = most <= BSEL_MAX_KEYS;
  if (on_chip) p.keys = nullptr;
  // the largest cluster (up to 8) with which every pair still runs at once, no larger than there is work for
  int C = 1;
  while (C < 8 && 2 * C * pairs <= kNumSMs && most > 64 * C) C *= 2;
  const size_t smem = on_chip ? (size_t)most * 4 : 0;
  return d == 128 ? (q == SK_BF16 ? launch_select<128, __nv_bfloat16>(p, pairs, C, smem, s) : launch_select<128, float>(p, pairs, C, smem, s))
                  : (q == SK_BF16 ? launch_select<64, __nv_bfloat16>(p, pairs, C, smem, s) : launch_select<64, float>(p, pairs, C, smem, s));
}

int check_cache_args(const void* Q, sk_dtype q, const void* K, const void* V, sk_dtype kv, const float* scales, int B,
                     int Hq, int Hkv, int Ncap, int d, const void* O) {
  SK_NONNULL(Q);
  SK_NONNULL(K);
  SK_NONNULL(V);
  SK_NONNULL(O);
  SK_ALIGNED(Q, 16);
  SK_ALIGNED(K, 16);
  SK_ALIGNED(V, 16);
  SK_ALIGNED(O, 16);
  SK_TRY(check_formats(q, kv, scales));
  SK_TRY(check_grid(B, Hq, Hkv, d));
  return check_ncap(Ncap);
}

int block_attend_impl(const void* Q, sk_dtype q, const void* K, const void* V, sk_dtype kv, const float* scales,
                      const int* lens, const int* idx, int B, int Hq, int Hkv, int Ncap, int N, int d, int block, int k,
                      float scale, float* O, void* ws, bool pdl, cudaStream_t s) {
  CacheAttendParams p = cache_params(Q, K, V, scales, lens, Hq, Hkv, Ncap, N);
  p.mode = KEYS_BLOCKS;
  p.idx = idx;
  p.k = k;
  p.block = block;
  p.n = k * block;
  return attend(p, q, kv, B, d, scale, O, SK_F32, ws, pdl, s);
}

constexpr int kMaxDrafts = 256;

}  // namespace

// ---------------------------------------------------------------- for api.cu
size_t hst::cache_workspace_bytes(int op, int B, int Hq, int Hkv, int Ncap, int N, int d, int block, int k) {
  const size_t bad = (size_t)-1;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq / Hkv > 8 || (long long)B * Hkv > 65535 || (d != 64 && d != 128) ||
      Ncap > kMaxRows || N > kMaxRows)
    return bad;
  const int pairs = B * Hkv, G = Hq / Hkv;
  switch (op) {
    case SK_OP_QUANT_DECODE:
      return N < 1 ? bad : attend_bytes(pairs, G, N, d);
    case SK_OP_QUANT_SPARSE_ATTEND:
      return k < 1 || k > kMaxPositions ? bad : attend_bytes(pairs, G, k, d);
    case SK_OP_BLOCK_SELECT:
    case SK_OP_BLOCK_ATTEND:
    case SK_OP_BLOCK_DECODE: {
      if (k < 1 || Ncap < 32 || (block != 16 && block != 32 && block != 64 && block != 128) ||
          (long long)k * block > kMaxPositions)
        return bad;
      if (op == SK_OP_BLOCK_SELECT) return select_bytes(pairs, Ncap, block);
      const size_t at = attend_bytes(pairs, G, k * block, d);
      if (op == SK_OP_BLOCK_ATTEND) return at;
      return select_bytes(pairs, Ncap, block) + align256((size_t)pairs * k * 4) + at;
    }
    case SK_OP_TREE_DECODE:
      if (k < 1 || k > kMaxDrafts || N < 0 || N > kMaxRows - k) return bad;
      return std::max(attend_bytes(pairs, k * G, N + k, d), tree_bytes(pairs, k * G, d));
    default:
      return bad;
  }
}

cudaError_t hst::cache_take_error(unsigned int* word) {
  cudaError_t e = cudaMemcpyFromSymbol(word, g_error_word, sizeof(*word));
  if (e == cudaSuccess && *word) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_error_word, &zero, sizeof(zero));
  }
  return e;
}

int hst::quant_list_check(const void* Q, sk_dtype q, const void* Kq, const void* Vq, sk_dtype kv, const float* scales,
                          int B, int Hq, int Hkv, int Ncap, int d, int k, const float* O) {
  SK_NONNULL(Kq);
  SK_NONNULL(Vq);
  SK_TRY(check_8bit(kv));
  SK_TRY(check_cache_args(Q, q, Kq, Vq, kv, scales, B, Hq, Hkv, Ncap, d, O));
  if (k < 1 || k > kMaxPositions) return fail(SK_ERR_INVALID_ARG, "k=%d must be in [1, 2^30]", k);
  return SK_OK;
}

int hst::quant_list_launch(const void* Q, sk_dtype q, const void* Kq, const void* Vq, sk_dtype kv, const float* scales,
                           const int* idx, int B, int Hq, int Hkv, int Ncap, int d, int k, float scale, float* O,
                           void* ws, cudaStream_t s, bool pdl) {
  CacheAttendParams p = cache_params(Q, Kq, Vq, scales, nullptr, Hq, Hkv, Ncap, Ncap);
  p.mode = KEYS_LISTED;
  p.idx = idx;
  p.k = k;
  p.n = k;
  return attend(p, q, kv, B, d, scale, O, SK_F32, ws, pdl, s);
}

extern "C" {

int quant_append(const void* K_new, const void* V_new, sk_dtype src, long long stride_b, long long stride_h,
                 long long stride_n, const int* starts, const int* lens, int B, int Hkv, int Ncap, int n_begin,
                 int n_count, int d, void* Kq, void* Vq, sk_dtype kv, float* scales, void* stream) {
  if (n_count != 0) {            // (an empty tensor has no address)
    SK_NONNULL(K_new);
    SK_NONNULL(V_new);
  }
  SK_NONNULL(Kq);
  SK_NONNULL(Vq);
  SK_NONNULL(scales);
  SK_ALIGNED(K_new, 16);
  SK_ALIGNED(V_new, 16);
  SK_ALIGNED(Kq, 16);
  SK_ALIGNED(Vq, 16);
  SK_ALIGNED(scales, 16);
  SK_TRY(check_dtype(src));
  SK_TRY(check_8bit(kv));
  SK_TRY(check_grid(B, Hkv, Hkv, d));
  SK_TRY(check_rows(starts, Ncap, n_begin, n_count));
  const long long per16 = src == SK_BF16 ? 8 : 4;
  if (stride_b % per16 || stride_h % per16 || stride_n % per16)
    return fail(SK_ERR_INVALID_ARG, "strides (%lld, %lld, %lld) must be multiples of 16 bytes (%lld elements)", stride_b,
                stride_h, stride_n, per16);
  if (n_count == 0) return SK_OK;
  QuantParams p = {};
  p.src[0] = K_new;
  p.src[1] = V_new;
  p.sb = stride_b;
  p.sh = stride_h;
  p.sn = stride_n;
  p.codes[0] = Kq;
  p.codes[1] = Vq;
  p.scales = scales;
  p.rows = {starts, lens, n_begin, n_count, Ncap};
  p.Hkv = Hkv;
  p.pairs = B * Hkv;
  const int per_block = d == 128 ? append_rows<128>() : append_rows<64>();
  auto kern = d == 128 ? (src == SK_BF16 ? (kv == SK_INT8 ? quant_append_kernel<128, __nv_bfloat16, KV_INT8>
                                                         : quant_append_kernel<128, __nv_bfloat16, KV_E4M3>)
                                         : (kv == SK_INT8 ? quant_append_kernel<128, float, KV_INT8>
                                                         : quant_append_kernel<128, float, KV_E4M3>))
                       : (src == SK_BF16 ? (kv == SK_INT8 ? quant_append_kernel<64, __nv_bfloat16, KV_INT8>
                                                         : quant_append_kernel<64, __nv_bfloat16, KV_E4M3>)
                                         : (kv == SK_INT8 ? quant_append_kernel<64, float, KV_INT8>
                                                         : quant_append_kernel<64, float, KV_E4M3>));
  return launch(kern, dim3((n_count + per_block - 1) / per_block, B * Hkv), QUANT_THREADS, 0, as_stream(stream), false,
                "quant_append_kernel", p);
}

int quant_read(const void* Kq, const void* Vq, sk_dtype kv, const float* scales, const int* starts, const int* lens,
               int B, int Hkv, int Ncap, int n_begin, int n_count, int d, void* K, void* V, sk_dtype dst, void* stream) {
  SK_NONNULL(Kq);
  SK_NONNULL(Vq);
  SK_NONNULL(scales);
  if (n_count != 0) {            // (an empty tensor has no address)
    SK_NONNULL(K);
    SK_NONNULL(V);
  }
  SK_ALIGNED(Kq, 16);
  SK_ALIGNED(Vq, 16);
  SK_ALIGNED(scales, 16);
  SK_ALIGNED(K, 16);
  SK_ALIGNED(V, 16);
  SK_TRY(check_8bit(kv));
  SK_TRY(check_dtype(dst));
  SK_TRY(check_grid(B, Hkv, Hkv, d));
  SK_TRY(check_rows(starts, Ncap, n_begin, n_count));
  if (n_count == 0) return SK_OK;
  QuantParams p = {};
  p.codes[0] = const_cast<void*>(Kq);
  p.codes[1] = const_cast<void*>(Vq);
  p.scales = const_cast<float*>(scales);
  p.dst[0] = K;
  p.dst[1] = V;
  p.rows = {starts, lens, n_begin, n_count, Ncap};
  p.Hkv = Hkv;
  p.pairs = B * Hkv;
  const int per_block = d == 128 ? read_rows<128>() : read_rows<64>();
  auto kern = d == 128 ? (dst == SK_BF16 ? (kv == SK_INT8 ? quant_read_kernel<128, __nv_bfloat16, KV_INT8>
                                                         : quant_read_kernel<128, __nv_bfloat16, KV_E4M3>)
                                         : (kv == SK_INT8 ? quant_read_kernel<128, float, KV_INT8>
                                                         : quant_read_kernel<128, float, KV_E4M3>))
                       : (dst == SK_BF16 ? (kv == SK_INT8 ? quant_read_kernel<64, __nv_bfloat16, KV_INT8>
                                                         : quant_read_kernel<64, __nv_bfloat16, KV_E4M3>)
                                         : (kv == SK_INT8 ? quant_read_kernel<64, float, KV_INT8>
                                                         : quant_read_kernel<64, float, KV_E4M3>));
  return launch(kern, dim3((n_count + per_block - 1) / per_block, B * Hkv), QUANT_THREADS, 0, as_stream(stream), false,
                "quant_read_kernel", p);
}

int quant_decode(const void* Q, sk_dtype q, const void* Kq, const void* Vq, sk_dtype kv, const float* scales,
                 const int* lens, int B, int Hq, int Hkv, int Ncap, int N, int d, float scale, float* O, void* ws,
                 size_t ws_bytes, void* stream) {
  SK_TRY(check_8bit(kv));
  SK_TRY(check_cache_args(Q, q, Kq, Vq, kv, scales, B, Hq, Hkv, Ncap, d, O));
  SK_TRY(check_cache(Ncap, N));
  SK_TRY(check_ws(ws, ws_bytes, cache_workspace_bytes(SK_OP_QUANT_DECODE, B, Hq, Hkv, Ncap, N, d, 0, 0)));
  CacheAttendParams p = cache_params(Q, Kq, Vq, scales, lens, Hq, Hkv, Ncap, N);
  p.mode = KEYS_ALL;
  p.n = N;
  return attend(p, q, kv, B, d, scale, O, SK_F32, ws, false, as_stream(stream));
}

int quant_sparse_attend(const void* Q, sk_dtype q, const void* Kq, const void* Vq, sk_dtype kv, const float* scales,
                        const int* idx, int B, int Hq, int Hkv, int Ncap, int d, int k, float scale, float* O, void* ws,
                        size_t ws_bytes, void* stream) {
  SK_NONNULL(idx);
  SK_TRY(quant_list_check(Q, q, Kq, Vq, kv, scales, B, Hq, Hkv, Ncap, d, k, O));
  SK_TRY(check_ws(ws, ws_bytes, cache_workspace_bytes(SK_OP_QUANT_SPARSE_ATTEND, B, Hq, Hkv, Ncap, 0, d, 0, k)));
  return quant_list_launch(Q, q, Kq, Vq, kv, scales, idx, B, Hq, Hkv, Ncap, d, k, scale, O, ws, as_stream(stream), false);
}

int block_summarize(const void* K, sk_dtype kv, const float* scales, const int* starts, const int* lens, int B, int Hkv,
                    int Ncap, int n_begin, int n_count, int d, int block, void* bsum, void* stream) {
  SK_NONNULL(K);
  SK_NONNULL(bsum);
  SK_ALIGNED(K, 16);
  SK_ALIGNED(bsum, 16);
  SK_TRY(check_formats(kv == SK_F32 ? SK_F32 : SK_BF16, kv, scales));
  SK_TRY(check_grid(B, Hkv, Hkv, d));
  SK_TRY(check_block(block));
  SK_TRY(check_rows(starts, Ncap, n_begin, n_count));
  if (n_count == 0) return SK_OK;
  SummaryParams p;
  p.K = K;
  p.scales = scales;
  p.bsum = reinterpret_cast<__nv_bfloat16*>(bsum);
  p.rows = {starts, lens, n_begin, n_count, Ncap};
  p.Hkv = Hkv;
  p.NB = num_blocks(Ncap, block);
  p.block = block;
  // n_count rows lie in at most this many blocks, wherever they start
  const int most = std::min((int)(((long long)n_count + block - 2) / block + 1), p.NB);
  const int warps = SUMMARY_THREADS / 32;
  auto kern = d == 128 ? (kv == SK_F32    ? block_summarize_kernel<128, KV_F32>
                          : kv == SK_BF16 ? block_summarize_kernel<128, KV_BF16>
                          : kv == SK_INT8 ? block_summarize_kernel<128, KV_INT8>
                                          : block_summarize_kernel<128, KV_E4M3>)
                       : (kv == SK_F32    ? block_summarize_kernel<64, KV_F32>
                          : kv == SK_BF16 ? block_summarize_kernel<64, KV_BF16>
                          : kv == SK_INT8 ? block_summarize_kernel<64, KV_INT8>
                                          : block_summarize_kernel<64, KV_E4M3>);
  return launch(kern, dim3((most + warps - 1) / warps, B * Hkv), SUMMARY_THREADS, 0, as_stream(stream), false,
                "block_summarize_kernel", p);
}

int block_select(const void* Q, sk_dtype q, const void* bsum, const int* lens, int B, int Hq, int Hkv, int Ncap, int N,
                 int d, int block, int k, int n_first, int n_last, int* idx, void* ws, size_t ws_bytes, void* stream) {
  SK_TRY(check_select(Q, q, bsum, B, Hq, Hkv, Ncap, N, d, block, k, n_first, n_last));
  SK_NONNULL(idx);
  SK_TRY(check_ws(ws, ws_bytes, cache_workspace_bytes(SK_OP_BLOCK_SELECT, B, Hq, Hkv, Ncap, N, d, block, k)));
  return select_impl(Q, q, bsum, lens, B, Hq, Hkv, Ncap, N, d, block, k, n_first, n_last, idx, ws, as_stream(stream));
}

int block_attend(const void* Q, sk_dtype q, const void* K, const void* V, sk_dtype kv, const float* scales,
                 const int* lens, const int* idx, int B, int Hq, int Hkv, int Ncap, int N, int d, int block, int k,
                 float scale, float* O, void* ws, size_t ws_bytes, void* stream) {
  SK_NONNULL(idx);
  SK_TRY(check_cache_args(Q, q, K, V, kv, scales, B, Hq, Hkv, Ncap, d, O));
  SK_TRY(check_cache(Ncap, N));
  SK_TRY(check_block(block));
  if (k < 1 || (long long)k * block > kMaxPositions) return fail(SK_ERR_INVALID_ARG, "k=%d blocks of %d keys", k, block);
  SK_TRY(check_ws(ws, ws_bytes, cache_workspace_bytes(SK_OP_BLOCK_ATTEND, B, Hq, Hkv, Ncap, N, d, block, k)));
  return block_attend_impl(Q, q, K, V, kv, scales, lens, idx, B, Hq, Hkv, Ncap, N, d, block, k, scale, O, ws, false,
                           as_stream(stream));
}

int block_decode(const void* Q, sk_dtype q, const void* K, const void* V, sk_dtype kv, const float* scales,
                 const void* bsum, const int* lens, int B, int Hq, int Hkv, int Ncap, int N, int d, int block, int k,
                 int n_first, int n_last, float scale, float* O, int* idx_out, void* ws, size_t ws_bytes, void* stream) {
  SK_TRY(check_cache_args(Q, q, K, V, kv, scales, B, Hq, Hkv, Ncap, d, O));
  SK_TRY(check_select(Q, q, bsum, B, Hq, Hkv, Ncap, N, d, block, k, n_first, n_last));
  SK_TRY(check_ws(ws, ws_bytes, cache_workspace_bytes(SK_OP_BLOCK_DECODE, B, Hq, Hkv, Ncap, N, d, block, k)));
  const cudaStream_t s = as_stream(stream);
  char* w = reinterpret_cast<char*>(ws);
  const size_t sel = select_bytes(B * Hkv, Ncap, block);
  int* idx = idx_out ? idx_out : reinterpret_cast<int*>(w + sel);
  SK_TRY(select_impl(Q, q, bsum, lens, B, Hq, Hkv, Ncap, N, d, block, k, n_first, n_last, idx, w, s));
  return block_attend_impl(Q, q, K, V, kv, scales, lens, idx, B, Hq, Hkv, Ncap, N, d, block, k, scale, O,
                           w + sel + align256((size_t)B * Hkv * k * 4), true, s);
}

int tree_decode(const void* Q, sk_dtype q, const void* K, const void* V, sk_dtype kv, const float* scales,
                const int* lens, const int* mask, int B, int T, int Hq, int Hkv, int Ncap, int N, int d, float scale,
                void* O, sk_dtype o, void* ws, size_t ws_bytes, void* stream) {
  SK_TRY(check_cache_args(Q, q, K, V, kv, scales, B, Hq, Hkv, Ncap, d, O));
  SK_TRY(check_dtype(o));
  if (T < 1 || T > kMaxDrafts) return fail(SK_ERR_UNSUPPORTED, "T=%d: 1 <= T <= %d drafted tokens", T, kMaxDrafts);
  if (N < 0 || (long long)N + T > Ncap)
    return fail(SK_ERR_INVALID_ARG, "N=%d cached and T=%d drafted keys do not fit Ncap=%d", N, T, Ncap);
  if ((long long)B * Hkv * Ncap > INT_MAX - 128)
    return fail(SK_ERR_UNSUPPORTED, "a cache of more than 2^31 - 129 rows (B * Hkv * Ncap)");
  SK_TRY(check_ws(ws, ws_bytes, cache_workspace_bytes(SK_OP_TREE_DECODE, B, Hq, Hkv, Ncap, N, d, 0, T)));
  CacheAttendParams p = cache_params(Q, K, V, scales, lens, Hq, Hkv, Ncap, N);
  p.mode = KEYS_TREE;
  p.T = T;
  p.mask = reinterpret_cast<const uint32_t*>(mask);
  p.mask_words = (T + 31) / 32;
  p.n = N + T;
  return attend(p, q, kv, B, d, scale, O, o, ws, false, as_stream(stream));
}

}  // extern "C"
