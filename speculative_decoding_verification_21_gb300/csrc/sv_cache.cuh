// sv_cache.cuh -- the paged cache as the kernels see it: a sequence's tokens,
// where a token of it sits in the pool, and the e4m3 codes and scales.
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
  uint8_t* ks;
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

inline CacheView cache_view(const sv_kv_cache& c) {
  const int es = c.dtype == SV_E4M3 ? 1 : 2;
  CacheView v{};
  v.k = (char*)c.k;
  v.v = (char*)c.v;
  v.ks = c.k_scale;
  v.vs = c.v_scale;
  v.page_bytes = c.page_stride * es;
  v.head_bytes = c.head_stride * es;
  v.token_bytes = c.token_stride * es;
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

}  // namespace sv
