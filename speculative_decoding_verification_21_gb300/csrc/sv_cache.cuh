// sv_cache.cuh -- the paged cache as the kernels see it: a sequence's tokens, where a
// token of it sits in the pool, e4m3 codes and scales, 4-bit codes, steps and zeros.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "specverify.h"

namespace sv {

// The device arrays of one call and the sizes that bound every index into them.
struct CacheView {
  char* k;
  char* v;
  uint8_t* ks;  // e4m3: scale bytes; 4 bits: words of a step (low half) and a zero
  uint8_t* vs;
  int64_t page_bytes, head_bytes, token_bytes;  // strides in bytes
  int num_pages, kv_heads, page_size, head_dim;
  int page_shift;  // log2 of the page size, or -1
};

struct BatchView {
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* kv_len;
  int total, B, max_pages;
};

// How a cache holds an element: 16 bits, an e4m3 code, or a 4-bit code.
enum Format { kHalf, kE4m3, kU4 };
inline Format format_of(int dtype) { return dtype == SV_E4M3 ? kE4m3 : dtype == SV_U4 ? kU4 : kHalf; }

inline CacheView cache_view(const sv_kv_cache& c) {
  const int halves = c.dtype == SV_U4 ? 1 : c.dtype == SV_E4M3 ? 2 : 4;  // half bytes an element
  CacheView v{};
  v.k = (char*)c.k;
  v.v = (char*)c.v;
  v.ks = c.k_scale;
  v.vs = c.v_scale;
  v.page_bytes = c.page_stride * halves / 2;
  v.head_bytes = c.head_stride * halves / 2;
  v.token_bytes = c.token_stride * halves / 2;
  v.num_pages = (int)c.num_pages;
  v.kv_heads = c.kv_heads;
  v.page_size = c.page_size;
  v.head_dim = c.head_dim;
  v.page_shift = (c.page_size & (c.page_size - 1)) ? -1 : __builtin_ctz((unsigned)c.page_size);
  return v;
}

// Rows tok0 .. tok0+n-1 of the packed arrays; the first of them sits at position
// pos0 = len - n (negative where the chunk is longer than the sequence).  A bad
// q_start empties the sequence, a bad kv_len is clamped into what the table's
// pages hold, so that nothing derived from them leaves an array.
struct Seq {
  int tok0, n, len, pos0;
  bool bad;
};

__device__ __forceinline__ Seq make_seq(int s0, int s1, int len, int total, int64_t held) {
  Seq q;
  const bool order = s0 >= 0 && s1 >= s0 && s1 <= total;
  q.tok0 = s0;
  q.n = order ? s1 - s0 : 0;
  q.len = len < 0 ? 0 : ((int64_t)len > held ? (int)held : len);
  q.bad = !order || q.len != len;
  q.pos0 = q.len - q.n;
  return q;
}

__device__ __forceinline__ Seq load_seq(const BatchView& bv, int b, int page_size) {
  return make_seq(__ldg(bv.q_start + b), __ldg(bv.q_start + b + 1), __ldg(bv.kv_len + b), bv.total,
                  (int64_t)bv.max_pages * page_size);
}

// The sequence that owns packed row t < total (one warp, all its lanes; B where none
// does).  The entries of a well-formed start rise, so it is the number of entries of
// start[1..B] that are <= t.  Where that sequence does not hold the row, some entry is
// bad: the first sequence whose own two entries hold it is looked for, so that a bad
// entry costs the two sequences beside it their rows and nobody else.
__device__ __forceinline__ int owner_of(const int32_t* start, int B, int t, int total) {
  const int lane = threadIdx.x & 31;
  auto holds = [&](int b) {
    const int s0 = __ldg(start + b), s1 = __ldg(start + b + 1);
    return s0 >= 0 && s0 <= t && t < s1 && s1 <= total;
  };
  int n = 0;
  for (int j = 0; j < B; j += 32) {
    const bool le = j + lane < B && __ldg(start + 1 + j + lane) <= t;
    n += __popc(__ballot_sync(0xffffffffu, le));
  }
  if (n == B || holds(n)) return n;  // (all of start[1..B] are <= t: nobody's)
  for (int j = 0; j < B; j += 32) {
    const unsigned in = __ballot_sync(0xffffffffu, j + lane < B && holds(j + lane));
    if (in) return j + __ffs(in) - 1;
  }
  return B;
}

__device__ __forceinline__ void page_of(const CacheView& c, int pos, int& page, int& slot) {
  if (c.page_shift >= 0) {
    page = pos >> c.page_shift;
    slot = pos & (c.page_size - 1);
  } else {
    page = pos / c.page_size;
    slot = pos - page * c.page_size;
  }
}

// 2^(s - 127) of a scale byte 1 <= s <= 254 (0 reads as 0, 255 as infinity).
__device__ __forceinline__ float scale_of(uint32_t s) { return __uint_as_float(s << 23); }

// Two e4m3 codes (low byte first) as fp32 (exact; the NaN code as NaN).
__device__ __forceinline__ float2 e4m3x2(uint16_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(__half2(h));
}

// 16-bit floats as fp32 and back (to nearest), by type.
template <int DT>
struct F16;
template <>
struct F16<SV_BF16> {
  static __device__ __forceinline__ float2 up(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};
template <>
struct F16<SV_F16> {
  static __device__ __forceinline__ float2 up(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
};

// Step and zero of a 4-bit row's word.
__device__ __forceinline__ float step_of(uint32_t sz) { return __uint_as_float(sz << 16); }
__device__ __forceinline__ float zero_of(uint32_t sz) { return __uint_as_float(sz & 0xFFFF0000u); }

// The code in nibble e of a word, as a float: 2^23 + c is the float whose bits end in c.
__device__ __forceinline__ float code_of(uint32_t w, int e) {
  return __uint_as_float(0x4B000000u | ((w >> (4 * e)) & 15u)) - 8388608.0f;
}

// ---------------------------------------------------------------------------
// Rows into codes.  A row's lanes form an aligned group of 1 << group_shift; each has 16
// of its elements.
// ---------------------------------------------------------------------------
constexpr int kMinScaleExp = -120;

// e4m3: with the row's largest finite |x| = f 2^e, 1 <= f < 2, the largest code
// 448 = 1.75 2^8 holds it over 2^k for k = e - 8 if f <= 1.75 and k = e - 7 else; x 2^-k
// is exact in fp32 (k >= -120 keeps 2^-k finite), so each code is rounded once.  m: the
// lane's largest |x|, NaNs passed over.
__device__ __forceinline__ uint4 encode_e4m3(float (&f)[16], float m, int group_shift, int& k) {
  const float inf = __int_as_float(0x7f800000);
  if (__any_sync(0xffffffffu, m == inf)) {
    // the largest finite one instead; infinities become the NaN code (the conversion
    // would make them the largest)
    m = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      if (fabsf(f[j]) == inf) f[j] = __int_as_float(0x7fffffff);
      m = fmaxf(m, fabsf(f[j]));
    }
  }
  for (int o = 1; o < (1 << group_shift); o <<= 1)
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const uint32_t bits = __float_as_uint(m);
  k = (int)(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
  k = k < kMinScaleExp ? kMinScaleExp : k;
  const float inv = __uint_as_float((uint32_t)(127 - k) << 23);
  uint32_t o4[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * j] * inv, f[4 * j + 1] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * j + 2] * inv, f[4 * j + 3] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    o4[j] = lo | (hi << 16);
  }
  return make_uint4(o4[0], o4[1], o4[2], o4[3]);
}

// (a NaN on either side stays one, unlike with fmaxf)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 4 bits: z = bf16(lo), s = max(bf16((hi/2 - z/2) fl(2/15)), 2^-120), c the integer nearest
// to the fp32 quotient (x/2 - z/2) / (s/2), within 0..15.  lo, hi: the lane's smallest and
// largest (NaN if it has one; +inf and -inf of a lane without elements).  The halves keep
// differences in range.  The quotient is d r with r = 1 / (s/2) and one correction by the
// remainder, which is exact: that rounds it correctly (a quotient of a 24-bit and an
// 8-bit number is no closer than 2^-33 to a midpoint unless it is one, and it is none), so
// ties, which bf16 rows have many of, are ties here too.
__device__ __forceinline__ uint2 encode_u4(const float (&f)[16], float lo, float hi, int group_shift,
                                           uint32_t& sz) {
  for (int o = 1; o < (1 << group_shift); o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const float inf = __int_as_float(0x7f800000);
  const uint32_t zb = __bfloat16_as_ushort(__float2bfloat16_rn(lo));
  const float half = __uint_as_float(zb << 16) * 0.5f;
  const float span = __fmul_rn(__fmaf_rn(hi, 0.5f, -half), 0.13333334f);
  const uint32_t sb = __bfloat16_as_ushort(__float2bfloat16_rn(fmaxf(span, 0x1p-120f)));
  const bool sound = fabsf(hi) < inf && fabsf(half) < inf && (sb & 0x7f80u) != 0x7f80u;
  sz = sound ? sb | (zb << 16) : 0x7fff7fffu;
  const float s2 = sound ? __uint_as_float(sb << 16) * 0.5f : 1.0f;
  const float r = __frcp_rn(s2);
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
#pragma unroll
    for (int e = 7; e >= 0; --e) {
      const float d = __fmaf_rn(f[8 * j + e], 0.5f, -half);
      const float q0 = __fmul_rn(d, r);
      const float q = __fmaf_rn(__fmaf_rn(-q0, s2, d), r, q0);
      // 1.5 2^23 + c is the float whose bits end in c
      const uint32_t b = __float_as_uint(__fadd_rn(fminf(fmaxf(q, 0.0f), 15.0f), 12582912.0f));
      w[j] = e == 7 ? b : (w[j] << 4) + b;
    }
    // (the sum of the 0x4B400000 16^e of the eight)
    w[j] -= 0x40000000u + 0xB4000000u + 0x4B400000u;
  }
  return sound ? make_uint2(w[0], w[1]) : make_uint2(0, 0);
}

// 16 elements of 16-bit floats as fp32; the lane's largest |x|, NaNs passed over.
template <int DT>
__device__ __forceinline__ void widen16(const uint4& x0, const uint4& x1, float (&f)[16]) {
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 p = F16<DT>::up(w[j]);
    f[2 * j] = p.x;
    f[2 * j + 1] = p.y;
  }
}
__device__ __forceinline__ float amax16(const float (&f)[16]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(f[2 * j]), fabsf(f[2 * j + 1])));
  return m;
}
__device__ __forceinline__ void range16(const float (&f)[16], bool on, float& lo, float& hi) {
  lo = __int_as_float(0x7f800000);
  hi = -lo;
  if (!on) return;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    lo = min_nan(lo, f[j]);
    hi = max_nan(hi, f[j]);
  }
}

}  // namespace sv
