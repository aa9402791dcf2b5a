// Rows quantised to 8 bits as they are written to the cache, and read back.
//
// Per row x of D values (one key or one value of one KV head), a = max |x_c|:
//   int8  s = max(a / 127, 2^-126) rounded once to f32, code = the integer
//         nearest x / s (ties to even, of the exact quotient), |code| <= 127;
//   e4m3  s = 2^e with the smallest e >= -126 that gives a <= 448 * 2^e,
//         code = x / s rounded once to e4m3. A power of two costs an e4m3 code
//         no precision (its steps are relative) and makes x / s and code * s
//         exact.
// A row of zeros has s = 0; a row with an infinity or a NaN has s = NaN and
// zero codes, so that all of it reads back as NaN.
//
// Both kernels move each byte once, so HBM should bound them. It does bound
// quant_read: 33 us for 32768 rows of 8 heads, D = 128, int8 to bf16 (6.2 TB/s).
// quant_append to e4m3 takes 36 us the other way (5.6 TB/s), to int8 46 (4.4): no
// pipe of it is full (issue slots 61%, ALU 54%), but a block loads first and rounds
// then, and only other blocks fill the gaps. Rows without outliers have more codes
// on a half (values of half the row's largest), which the division settles: 82 us
// for Gaussian rows. When it writes, a row is D / 16 lanes of two
// pieces of 8 values, a half row apart (16-byte loads of bf16 rows, 128 bytes in
// a row): the scale's arithmetic and the exchanges are shared by 16 values. The
// lanes of a warp take a K row and its V row side by side, so that the row's two
// scales leave as one 8-byte store.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace hst {

// Formats of a cache: the values of sk_dtype.
constexpr int KV_F32 = 0, KV_BF16 = 1, KV_INT8 = 2, KV_E4M3 = 3;
__host__ __device__ constexpr int kv_elem_bytes(int fmt) { return fmt == KV_F32 ? 4 : fmt == KV_BF16 ? 2 : 1; }

// The rows that a call writes or reads: for sequence b rows start .. start +
// count - 1 of the cache, as far as they lie below the sequence's end.
struct RowRange {
  const int* starts;   // optional [B]: first row, instead of n_begin
  const int* lens;     // optional [B]: rows at or behind lens[b] are left out
  int n_begin, n_count, Ncap;
  __device__ __forceinline__ int start(int b) const { return starts ? __ldg(starts + b) : n_begin; }
  __device__ __forceinline__ int end(int b) const { return lens ? min(__ldg(lens + b), Ncap) : Ncap; }
};

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_to_f32(w[i]);
    x[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}
// 8 values of a row as loaded, and the bits of their largest magnitude.
struct Raw8F32 {
  float x[8];
  __device__ __forceinline__ void load(const float* p) { load8(p, x); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
  }
  // with the other piece, of the LPR lanes that share the row
  template <int LPR>
  __device__ __forceinline__ uint32_t amax(const Raw8F32& y) const {
    uint32_t a = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, max(__float_as_uint(x[i]) & 0x7fffffffu, __float_as_uint(y.x[i]) & 0x7fffffffu));
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(FULL, a, o));
    return a;
  }
  __device__ __forceinline__ void get(float (&y)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
  }
};
struct Raw8B16 {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = ldg_stream(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  static __device__ __forceinline__ uint32_t two(uint4 w) {
    return __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
  }
  template <int LPR>
  __device__ __forceinline__ uint32_t amax(const Raw8B16& y) const {     // two 16-bit maxima at a time
    uint32_t a = __vmaxu2(two(v), two(y.v));
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) a = __vmaxu2(a, __shfl_xor_sync(FULL, a, o));
    return max(a << 16, a & 0xffff0000u);
  }
  __device__ __forceinline__ void get(float (&y)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = bf16lo_to_f32(w[i]);
      y[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
  }
};
template <typename T> struct Raw8Of { using type = Raw8F32; };
template <> struct Raw8Of<__nv_bfloat16> { using type = Raw8B16; };

__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// The row's scale from the bits of its largest magnitude (bits of |x| order
// like the magnitudes, NaN above infinity above every number).
template <int FMT>
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  if (amax_bits == 0u) return 0.f;
  const float a = __uint_as_float(amax_bits);
  if constexpr (FMT == KV_INT8) return fmaxf(a / 127.f, 0x1p-126f);
  // a = m 2^E with 1 <= m < 2: 448 = 1.75 * 2^8, so e = E - 8 or E - 7
  const int E = (int)(amax_bits >> 23) - 127;             // subnormals: E = -127, clamped below
  const int e = max(E - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0), -126);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Nearest integer to x / s, ties to even. The f32 quotient may round onto a
// half; the sign of x - (n +- 1/2) s, exact in one fma, settles it.
__device__ __forceinline__ int nearest_quotient(float x, float s) {
  float n = rintf(x / s);
  if (fmaf(-(n + 0.5f), s, x) > 0.f) n += 1.f;
  else if (fmaf(-(n - 0.5f), s, x) < 0.f) n -= 1.f;
  return max(-127, min(127, (int)n));
}

// The codes of 8 values. x / s is x times the approximate reciprocal, off by at
// most 127 * 2^-22 (its unit in the last place and the sum's rounding); added to 1.5 * 2^23 it rounds to
// the integer in the low bits. Where it lies within 2^-15 of a half, the
// quotient decides. (A division for each value took the kernel 106 us where the bytes
// of 32768 rows of 8 heads take 31; this takes 46.)
__device__ __forceinline__ uint2 encode_int8(const float (&x)[8], float s) {
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  float t[8], far = 0.f;
  const uint64_t inv2 = pack_f32x2(inv, inv), magic = pack_f32x2(12582912.f, 12582912.f), minus = pack_f32x2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint64_t x2 = pack_f32x2(x[i], x[i + 1]), t2 = fma_f32x2(x2, inv2, magic);
    unpack_f32x2(t2, t[i], t[i + 1]);
    float a, b;
    unpack_f32x2(fma_f32x2(x2, inv2, fma_f32x2(t2, minus, magic)), a, b);      // what was rounded off
    far = max3(far, fabsf(a), fabsf(b));
  }
  if (far > 0.5f - 0x1p-15f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = 12582912.f + (float)nearest_quotient(x[i], s);
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = __byte_perm(__byte_perm(__float_as_uint(t[4 * i]), __float_as_uint(t[4 * i + 1]), 0x0040),
                       __byte_perm(__float_as_uint(t[4 * i + 2]), __float_as_uint(t[4 * i + 3]), 0x0040), 0x5410);
  return make_uint2(w[0], w[1]);
}

template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float s) {
  uint32_t w[2] = {0u, 0u};
  if (s > 0.f) {                                          // not zero, not NaN
    if constexpr (FMT == KV_INT8) {
      return encode_int8(x, s);
    } else {
      const float inv = __uint_as_float(0x7f000000u - __float_as_uint(s));   // 2^-e, exact for -126 <= e <= 126
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t v =
            __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        w[i >> 1] |= (uint32_t)v << (16 * (i & 1));
      }
    }
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(__half2(h));
}

template <int FMT>
__device__ __forceinline__ void decode8(uint2 w, float s, float (&x)[8]) {
  const uint32_t v[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = (v[i >> 1] >> (16 * (i & 1))) & 0xffffu;
    if constexpr (FMT == KV_INT8) {
      x[2 * i] = (float)(int)(signed char)(two & 255u) * s;
      x[2 * i + 1] = (float)(int)(signed char)(two >> 8) * s;
    } else {
      const float2 f = e4m3x2_to_f32(two);
      x[2 * i] = f.x * s;
      x[2 * i + 1] = f.y * s;
    }
  }
}

struct QuantParams {
  const void* src[2];        // K and V rows, element strides below (append)
  long long sb, sh, sn;
  void* codes[2];            // [pairs][Ncap][D]
  float* scales;             // [pairs][Ncap][2]: of the K row, of the V row
  void* dst[2];              // [pairs][n_count][D] (read)
  RowRange rows;
  int Hkv, pairs;
};

constexpr int QUANT_THREADS = 256;
constexpr int QUANT_UNROLL = 4;      // row pairs in flight per group of lanes

// Row pairs that a block of quant_append_kernel (quant_read_kernel) takes.
template <int D>
__host__ __device__ constexpr int append_rows() { return QUANT_THREADS / (2 * (D / 16)) * QUANT_UNROLL; }
template <int D>
__host__ __device__ constexpr int read_rows() { return QUANT_THREADS / (2 * (D / 8)) * QUANT_UNROLL; }

// grid = (chunks of rows, pairs).
template <int D, typename ST, int FMT>
__global__ void __launch_bounds__(QUANT_THREADS) quant_append_kernel(const QuantParams p) {
  constexpr int LPR = D / 16;                        // lanes per row
  constexpr int RPB = append_rows<D>() / QUANT_UNROLL;     // row pairs per pass of the block
  const int sub = threadIdx.x % LPR, which = (threadIdx.x / LPR) & 1, slot = threadIdx.x / (2 * LPR);
  const int pair = blockIdx.y, b = pair / p.Hkv, h = pair % p.Hkv;
  const int start = p.rows.start(b), end = p.rows.end(b);
  const ST* src = reinterpret_cast<const ST*>(p.src[which]) + b * p.sb + h * p.sh + 8 * sub;
  const size_t row0 = (size_t)pair * p.rows.Ncap;
  const int i0 = blockIdx.x * append_rows<D>() + slot;
  typename Raw8Of<ST>::type x[QUANT_UNROLL][2];
  bool live[QUANT_UNROLL];
  // (for the whole block) all its rows are there and have a place
  const int last = (blockIdx.x + 1) * append_rows<D>() - 1;
  const bool inside = last < p.rows.n_count && start >= 0 && (long long)start + last < end;
#pragma unroll
  for (int u = 0; u < QUANT_UNROLL; ++u) {
    const int i = i0 + u * RPB;
    live[u] = true;
    if (!inside) {
      const long long r = (long long)start + i;
      live[u] = i < p.rows.n_count && r >= 0 && r < end;
      // a row that the lengths do not leave out but the cache has no place for
      if (i < p.rows.n_count && !live[u] && (r < 0 || r >= p.rows.Ncap) && (!p.rows.lens || r < __ldg(p.rows.lens + b)))
        atomicOr(&g_error_word, ERR_ROWS);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (live[u]) x[u][k].load(src + i * p.sn + k * (D / 2));
      else x[u][k].zero();
    }
  }
#pragma unroll
  for (int u = 0; u < QUANT_UNROLL; ++u) {
    const float s = row_scale<FMT>(x[u][0].template amax<LPR>(x[u][1]));
    const float sv = __shfl_xor_sync(FULL, s, LPR);  // the V row's scale, in the K row's lanes
    if (!live[u]) continue;
    const size_t row = row0 + (size_t)(start + i0 + u * RPB);
    unsigned char* out = reinterpret_cast<unsigned char*>(p.codes[which]) + row * D + 8 * sub;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float y[8];
      x[u][k].get(y);
      *reinterpret_cast<uint2*>(out + k * (D / 2)) = encode8<FMT>(y, s);
    }
    if (which == 0 && sub == 0) *reinterpret_cast<float2*>(p.scales + 2 * row) = make_float2(s, sv);
  }
}

template <int D, typename ST, int FMT>
__global__ void __launch_bounds__(QUANT_THREADS) quant_read_kernel(const QuantParams p) {
  constexpr int LPR = D / 8;
  constexpr int RPB = read_rows<D>() / QUANT_UNROLL;
  const int sub = threadIdx.x % LPR, which = (threadIdx.x / LPR) & 1, slot = threadIdx.x / (2 * LPR);
  const int pair = blockIdx.y, b = pair / p.Hkv;
  const int start = p.rows.start(b), end = p.rows.end(b);
  const unsigned char* codes = reinterpret_cast<const unsigned char*>(p.codes[which]) + 8 * sub;
  ST* dst = reinterpret_cast<ST*>(p.dst[which]) + (size_t)pair * p.rows.n_count * D + 8 * sub;
  const size_t row0 = (size_t)pair * p.rows.Ncap;
  const int i0 = blockIdx.x * (RPB * QUANT_UNROLL) + slot;
  uint2 w[QUANT_UNROLL];
  float s[QUANT_UNROLL];
  bool live[QUANT_UNROLL];
#pragma unroll
  for (int u = 0; u < QUANT_UNROLL; ++u) {
    const int i = i0 + u * RPB;
    const long long r = (long long)start + i;
    live[u] = i < p.rows.n_count && r >= 0 && r < end;
    w[u] = make_uint2(0u, 0u);
    s[u] = 0.f;
    if (live[u]) {
      const size_t row = row0 + (size_t)r;
      w[u] = *reinterpret_cast<const uint2*>(codes + row * D);
      s[u] = __ldg(p.scales + 2 * row + which);
    }
  }
#pragma unroll
  for (int u = 0; u < QUANT_UNROLL; ++u) {
    if (!live[u]) continue;
    float x[8];
    decode8<FMT>(w[u], s[u], x);
    store8(dst + (size_t)(i0 + u * RPB) * D, x);
  }
}

}  // namespace hst
