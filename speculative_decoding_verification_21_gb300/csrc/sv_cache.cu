// sv_cache.cu -- spec_kv_append and spec_kv_read: new keys and values into the
// pages of the cache, and tokens out of them.
//
// Both are copies by an index, bound by HBM: a token's rows (kv_heads vectors of
// k and of v) are contiguous on the packed side, and head_dim-long runs on the
// pool's.  One warp takes one token or four, so that the search for its sequence and
// its page is done once for all of its rows; a lane moves 16 elements of a row (two
// 16-byte vectors of 16-bit floats, one of codes), and a row's lanes form an
// aligned group of 1, 2, 4, 8 or 16 so that its largest value is a few shuffles.
//
// e4m3: with amax = f 2^e, 1 <= f < 2, the largest code 448 = 1.75 2^8 holds
// amax / 2^k for k = e - 8 if f <= 1.75 and k = e - 7 else; x 2^-k is exact in
// fp32 (k >= -120 keeps 2^-k finite), so each code is rounded once.
//
// Measured on GB300: 84 thousand tokens of 8 heads of 128 into e4m3 94 us, 5.5 TB/s
// (0.81 of a copy's rate; what is missing is the arithmetic between loads and stores);
// 174 thousand out of e4m3 171 us, 6.3 TB/s (0.93); 320 tokens 4 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "specverify.h"
#include "sv_cache.cuh"
#include "sv_device.cuh"
#include "sv_launch.h"
#include "sv_tma.cuh"

namespace sv {
namespace {

constexpr int kMoveWarps = 8;
constexpr int kMinScaleExp = -120;

struct MoveArgs {
  CacheView c;
  const int32_t* table;
  const int32_t* start;   // [B+1]
  const int32_t* at;      // append: kv_len [B]; read: first [B]
  const char* in_k;       // append: new keys; read: unused
  const char* in_v;
  char* out_k;            // read: packed outputs
  char* out_v;
  uint8_t* flags;
  int64_t in_token, in_head;  // strides of the new rows in bytes
  int total, B, max_pages;
  int move_blocks;        // blocks that move tokens; the rest write flags
};

// Rows tok0 .. tok0+n-1 of sequence b, the position of the first (as the lengths say,
// wherever that is: a row whose position lies outside the pages has no place), and
// whether the entries are sound.
struct MoveSeq {
  int tok0, n;
  int64_t pos0;
  bool bad;
};
template <bool APPEND>
__device__ __forceinline__ MoveSeq move_seq(const MoveArgs& a, int b) {
  const int s0 = __ldg(a.start + b), s1 = __ldg(a.start + b + 1), at = __ldg(a.at + b);
  const int64_t held = (int64_t)a.max_pages * a.c.page_size;
  const Seq q = make_seq(s0, s1, APPEND ? at : 0, a.total, held);
  MoveSeq m{q.tok0, q.n, APPEND ? (int64_t)at - q.n : at, q.bad};
  m.bad |= m.n && (m.pos0 < 0 || m.pos0 + m.n > held);
  return m;
}

__device__ __forceinline__ bool in_pages(int64_t pos, int64_t held) { return pos >= 0 && pos < held; }

// Flags of sequence b from its lengths and the table entries of its rows (one warp).
template <bool APPEND>
__device__ void write_flags(const MoveArgs& a, int b) {
  const int lane = threadIdx.x & 31;
  const MoveSeq q = move_seq<APPEND>(a, b);
  const int64_t held = (int64_t)a.max_pages * a.c.page_size;
  int64_t lo = q.pos0, hi = lo + q.n;
  lo = lo < 0 ? 0 : lo;
  hi = hi > held ? held : hi;
  bool page_bad = false;
  if (hi > lo) {
    const int p0 = (int)(lo / a.c.page_size), p1 = (int)((hi - 1) / a.c.page_size);
    for (int p = p0 + lane; p <= p1; p += 32) {
      const int page = __ldg(a.table + (int64_t)b * a.max_pages + p);
      page_bad |= page < 0 || page >= a.c.num_pages;
    }
  }
  const bool any = __any_sync(0xffffffffu, page_bad);
  if (lane == 0)
    a.flags[b] = (uint8_t)((q.bad ? SV_FLAG_BAD_LENGTH : 0) | (any ? SV_FLAG_BAD_PAGE : 0));
}

// 16 values as codes: the row's largest finite |x| over its group of lanes, the
// exponent, the codes.
template <int DT>
__device__ __forceinline__ uint4 encode16(const uint4& x0, const uint4& x1, int group_shift, int& k) {
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  const float inf = __int_as_float(0x7f800000);
  float f[16], m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 p = F16<DT>::up(w[j]);
    f[2 * j] = p.x;
    f[2 * j + 1] = p.y;
    m = fmaxf(m, fmaxf(fabsf(p.x), fabsf(p.y)));  // (a NaN is passed over)
  }
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

// 16 codes times 2^(byte - 127) as 16-bit values.
template <int DT>
__device__ __forceinline__ void decode16(const uint4& x, uint32_t byte, uint4& x0, uint4& x1) {
  const float s = scale_of(byte);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t o8[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 lo = e4m3x2((uint16_t)w[j]), hi = e4m3x2((uint16_t)(w[j] >> 16));
    o8[2 * j] = F16<DT>::down(lo.x * s, lo.y * s);
    o8[2 * j + 1] = F16<DT>::down(hi.x * s, hi.y * s);
  }
  x0 = make_uint4(o8[0], o8[1], o8[2], o8[3]);
  x1 = make_uint4(o8[4], o8[5], o8[6], o8[7]);
}

// Where packed row t goes or comes from: page -2: nowhere (no sequence has the row),
// -1: a bad place.
struct Place {
  int page, slot;
};
template <bool APPEND>
__device__ __forceinline__ Place place_of(const MoveArgs& a, int b, int t, int64_t held) {
  Place p{-2, 0};
  if (b >= a.B) return p;  // rows behind the last sequence
  const MoveSeq q = move_seq<APPEND>(a, b);
  const int i = t - q.tok0;
  if (i < 0 || i >= q.n) return p;  // start does not rise
  const int64_t pos = q.pos0 + i;
  p.page = -1;
  if (!in_pages(pos, held)) return p;
  int index;
  page_of(a.c, (int)pos, index, p.slot);
  const int page = __ldg(a.table + (int64_t)b * a.max_pages + index);
  if (page >= 0 && page < a.c.num_pages) p.page = page;
  return p;
}

// A warp moves `per` consecutive tokens.  Their places are found together, one token a
// lane: with one token a warp the chain q_start, kv_len, table stood before every 8 KB.
// A row's lanes: head_dim / 16 rounded up to a power of two (1 << group_shift).
// Encoding keeps two steps' loads in flight (its shuffles hold back later ones) in 32
// warps an SM; copies and decoding do better with single steps in 64 warps.  Measured:
// 84 thousand tokens of 8 heads of 128 into e4m3: 94 us (5.5 TB/s), with four steps 98,
// with one 116; 175 thousand out of e4m3: 171 us (6.3 TB/s), with 48 warps 176, with four
// steps 204.
constexpr int batch_of(bool e4m3, bool append) { return e4m3 && append ? 2 : 1; }

template <int DT, bool E4M3, bool APPEND>
__global__ void __launch_bounds__(kMoveWarps * 32, batch_of(E4M3, APPEND) > 1 ? 4 : APPEND ? 6 : 8) k_move(const __grid_constant__ MoveArgs a,
                                                          int group_shift, int per) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int)blockIdx.x >= a.move_blocks) {
    const int b = ((int)blockIdx.x - a.move_blocks) * kMoveWarps + warp;
    if (b < a.B) write_flags<APPEND>(a, b);
    return;
  }
  const CacheView& c = a.c;
  const int64_t held = (int64_t)a.max_pages * c.page_size;
  const int64_t first = ((int64_t)blockIdx.x * kMoveWarps + warp) * per;
  if (first >= a.total) return;
  const int t0 = (int)first, n = min(per, a.total - t0);
  // the sequence of the first token, and mostly of all
  const int b0 = owner_of(a.start, a.B, t0, a.total);
  const bool same = n == 1 || (b0 < a.B && t0 + n <= __ldg(a.start + b0 + 1));
  Place mine{-2, 0};
  if (same) {
    if (lane < n) mine = place_of<APPEND>(a, b0, t0 + lane, held);
  } else {
    for (int j = 0; j < n; ++j) {
      const int b = owner_of(a.start, a.B, t0 + j, a.total);
      if (lane == j) mine = place_of<APPEND>(a, b, t0 + j, held);
    }
  }
  const int sub = lane & ((1 << group_shift) - 1);  // 16-element piece of the row
  const int row = lane >> group_shift;              // row of a step
  const bool on = sub * 16 < c.head_dim;
  const int rows = 2 * c.kv_heads;                  // k heads, then v heads
  const int at_once = 32 >> group_shift;
  const int steps = (rows + at_once - 1) / at_once;
  // the loads of a batch of steps, then the rest of them
  constexpr int kBatch = batch_of(E4M3, APPEND);
  const int all = n * steps;
  int j = 0, step = 0;
  for (int e0 = 0; e0 < all; e0 += kBatch) {
    uint4 x0[kBatch], x1[kBatch];
    char* out[kBatch];        // append: the row in the pool; read: the packed row
    int64_t at[kBatch];       // append: index of the row's scale
    bool is_v[kBatch], live[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int page = __shfl_sync(0xffffffffu, mine.page, j & 31);
      const int slot = __shfl_sync(0xffffffffu, mine.slot, j & 31);
      const int64_t t = t0 + j;
      const int r = step * at_once + row;
      live[i] = e0 + i < all && r < rows && on && (APPEND ? page >= 0 : page > -2);
      if (++step == steps) {
        step = 0;
        ++j;
      }
      is_v[i] = r >= c.kv_heads;
      const int h = is_v[i] ? r - c.kv_heads : r;
      char* pool = (is_v[i] ? c.v : c.k) + (int64_t)page * c.page_bytes +
                   (int64_t)h * c.head_bytes + (int64_t)slot * c.token_bytes;
      at[i] = ((int64_t)page * c.kv_heads + h) * c.page_size + slot;
      x0[i] = x1[i] = make_uint4(0, 0, 0, 0);
      if (APPEND) {
        const char* src = (is_v[i] ? a.in_v : a.in_k) + t * a.in_token + (int64_t)h * a.in_head;
        out[i] = pool;
        if (live[i]) {
          x0[i] = ld_stream16(src + 32 * sub);
          x1[i] = ld_stream16(src + 32 * sub + 16);
        }
      } else {
        out[i] = (is_v[i] ? a.out_v : a.out_k) + ((t * c.kv_heads + h) * c.head_dim) * 2;
        if (live[i] && page >= 0) {
          if (E4M3) {
            x0[i] = ld_stream16(pool + 16 * sub);
            x1[i].x = __ldg((is_v[i] ? c.vs : c.ks) + at[i]);
          } else {
            x0[i] = ld_stream16(pool + 32 * sub);
            x1[i] = ld_stream16(pool + 32 * sub + 16);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      uint4* const dst = reinterpret_cast<uint4*>(out[i]);
      if (APPEND && E4M3) {
        int k;
        const uint4 o = encode16<DT>(x0[i], x1[i], group_shift, k);
        if (live[i]) {
          dst[sub] = o;
          if (sub == 0) (is_v[i] ? c.vs : c.ks)[at[i]] = (uint8_t)(k + 127);
        }
        continue;
      }
      if (E4M3) decode16<DT>(x0[i], x1[i].x, x0[i], x1[i]);
      if (live[i]) {
        dst[2 * sub] = x0[i];
        dst[2 * sub + 1] = x1[i];
      }
    }
  }
}

template <bool APPEND>
cudaError_t launch_move(MoveArgs a, int dtype, bool e4m3, cudaStream_t stream) {
  int shift = 0;
  while ((16 << shift) < a.c.head_dim) ++shift;
  // four tokens a warp where that still gives every SM 16 warps
  const int per = a.total >= 152 * 16 * 4 ? 4 : 1;
  a.move_blocks = (int)(((int64_t)a.total + kMoveWarps * per - 1) / (kMoveWarps * per));
  const int flag_blocks = a.flags ? (a.B + kMoveWarps - 1) / kMoveWarps : 0;
  if (a.move_blocks + flag_blocks == 0) return cudaSuccess;
  auto* k = e4m3 ? (dtype == SV_BF16 ? k_move<SV_BF16, true, APPEND> : k_move<SV_F16, true, APPEND>)
                 : k_move<SV_BF16, false, APPEND>;  // a plain copy of 16-bit values
  return launch_pdl(k, dim3(a.move_blocks + flag_blocks), dim3(kMoveWarps * 32), 0, stream, a, shift, per);
}

}  // namespace

cudaError_t launch_kv_append(const sv_kv_cache& c, const sv_kv_batch& b, const void* new_k,
                             const void* new_v, int dtype, int64_t token_stride,
                             int64_t head_stride, uint8_t* out_flags, cudaStream_t stream) {
  MoveArgs a{};
  a.c = cache_view(c);
  a.table = b.block_table;
  a.start = b.q_start;
  a.at = b.kv_len;
  a.in_k = (const char*)new_k;
  a.in_v = (const char*)new_v;
  a.in_token = token_stride * 2;
  a.in_head = head_stride * 2;
  a.flags = out_flags;
  a.total = (int)b.total;
  a.B = b.B;
  a.max_pages = b.max_pages;
  return launch_move<true>(a, dtype, c.dtype == SV_E4M3, stream);
}

cudaError_t launch_kv_read(const sv_kv_cache& c, const int32_t* block_table, const int32_t* first,
                           const int32_t* out_start, int B, int max_pages, int64_t total,
                           void* out_k, void* out_v, int dtype, uint8_t* out_flags,
                           cudaStream_t stream) {
  MoveArgs a{};
  a.c = cache_view(c);
  a.table = block_table;
  a.start = out_start;
  a.at = first;
  a.out_k = (char*)out_k;
  a.out_v = (char*)out_v;
  a.flags = out_flags;
  a.total = (int)total;
  a.B = B;
  a.max_pages = max_pages;
  return launch_move<false>(a, dtype, c.dtype == SV_E4M3, stream);
}

}  // namespace sv
