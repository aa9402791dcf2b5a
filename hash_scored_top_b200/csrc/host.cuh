// What the library's translation units share on the host: the error message,
// argument checks, launches, and the calls one makes of the other.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/hash_scored_top.h"

#define HST_HIDDEN __attribute__((visibility("hidden")))

namespace hst {

// Records the thread's error message (sk_last_error) and returns `code`.
HST_HIDDEN int fail(int code, const char* fmt, ...);

inline int check_launch(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SK_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return SK_OK;
}

inline cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

constexpr int kMaxL = 64;
constexpr int kNumSMs = 148;

// Shapes common to the decode-side calls.
inline int check_heads(int B, int Hq, int Hkv, int d) {
  if (B < 1 || Hq < 1 || Hkv < 1) return fail(SK_ERR_INVALID_ARG, "B, Hq, Hkv must be >= 1");
  if (Hq % Hkv) return fail(SK_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d)", Hq, Hkv);
  if (d != 64 && d != 128) return fail(SK_ERR_UNSUPPORTED, "head dim d=%d: only 64 and 128 are supported", d);
  return SK_OK;
}

inline int check_cache(int Ncap, int N) {
  if (Ncap < 32 || Ncap % 32) return fail(SK_ERR_INVALID_ARG, "Ncap=%d must be a positive multiple of 32", Ncap);
  if (N < 1 || N > Ncap) return fail(SK_ERR_INVALID_ARG, "N=%d must be in [1, Ncap=%d]", N, Ncap);
  return SK_OK;
}

inline int check_tables(int L, int P, float tau) {
  if (P < 1 || P > 8) return fail(SK_ERR_UNSUPPORTED, "P=%d: 1 <= P <= 8 (bucket IDs are bytes)", P);
  if (L < 1 || L > kMaxL) return fail(SK_ERR_UNSUPPORTED, "L=%d: 1 <= L <= %d", L, kMaxL);
  if (!(tau > 0.f)) return fail(SK_ERR_INVALID_ARG, "tau must be > 0");
  return SK_OK;
}

inline int check_dtype(sk_dtype t) {
  if (t != SK_F32 && t != SK_BF16) return fail(SK_ERR_INVALID_ARG, "unknown dtype %d", (int)t);
  return SK_OK;
}

#define SK_TRY(expr)            \
  do {                          \
    const int _rc = (expr);     \
    if (_rc != SK_OK) return _rc; \
  } while (0)

#define SK_NONNULL(ptr)                                                          \
  do {                                                                           \
    if ((ptr) == nullptr) return fail(SK_ERR_INVALID_ARG, "%s is NULL", #ptr);   \
  } while (0)

// Alignment the kernels' vector loads and bulk copies rely on.
#define SK_ALIGNED(ptr, bytes)                                                                   \
  do {                                                                                           \
    if (reinterpret_cast<uintptr_t>(ptr) % (bytes))                                              \
      return fail(SK_ERR_INVALID_ARG, "%s must be %d-byte aligned", #ptr, (int)(bytes));         \
  } while (0)

// 2-D tensor map of a [rows][d] bf16 matrix: TMA tiles of 64 columns x box_rows
// rows with the 128-byte swizzle. (api.cu)
HST_HIDDEN int encode_rows_map(CUtensorMap* map, const void* base, long rows, int d, int box_rows);

// ---- cache_api.cu, for api.cu
// Workspace of the operators over quantised, block-selected and drafted caches.
HST_HIDDEN size_t cache_workspace_bytes(int op, int B, int Hq, int Hkv, int Ncap, int N, int d, int block, int k);
// The argument checks and the launch of quant_sparse_attend; pdl: as the
// programmatic dependent of the kernel that writes idx.
HST_HIDDEN int quant_list_check(const void* Q, sk_dtype q, const void* Kq, const void* Vq, sk_dtype kv, const float* scales,
                                int B, int Hq, int Hkv, int Ncap, int d, int k, const float* O);
HST_HIDDEN int quant_list_launch(const void* Q, sk_dtype q, const void* Kq, const void* Vq, sk_dtype kv,
                                 const float* scales, const int* idx, int B, int Hq, int Hkv, int Ncap, int d, int k,
                                 float scale, float* O, void* ws, cudaStream_t s, bool pdl);
// Reads and clears that unit's device error word.
HST_HIDDEN cudaError_t cache_take_error(unsigned int* word);

}  // namespace hst
