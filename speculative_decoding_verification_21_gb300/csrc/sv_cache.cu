// sv_cache.cu -- spec_kv_append and spec_kv_read: new keys and values into the
// pages of the cache, and tokens out of them.
//
// Both are copies by an index, bound by HBM: a token's rows (kv_heads vectors of
// k and of v) are contiguous on the packed side, and head_dim-long runs on the
// pool's.  One warp takes one token, so that the search for its sequence and its
// page is done once for all of its rows; a lane moves 16 elements of a row (two
// 16-byte vectors of 16-bit floats, one of codes), and a row's lanes form an
// aligned group of 1, 2, 4, 8 or 16 so that its largest value is a few shuffles.
//
// e4m3: with amax = f 2^e, 1 <= f < 2, the largest code 448 = 1.75 2^8 holds
// amax / 2^k for k = e - 8 if f <= 1.75 and k = e - 7 else; x 2^-k is exact in
// fp32 (k >= -120 keeps 2^-k finite), so each code is rounded once.
#include <cuda_runtime.h>

#include <cstdint>

#include "specverify.h"
#include "sv_cache.cuh"
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

// Position of the first row of sequence b, and whether its entries are sound.
template <bool APPEND>
__device__ __forceinline__ Seq move_seq(const MoveArgs& a, int b) {
  const int s0 = __ldg(a.start + b), s1 = __ldg(a.start + b + 1), at = __ldg(a.at + b);
  const int64_t held = (int64_t)a.max_pages * a.c.page_size;
  if (APPEND) return make_seq(s0, s1, at, a.total, held);
  Seq q = make_seq(s0, s1, 0, a.total, held);
  q.pos0 = at;
  q.bad = q.bad || (q.n && (at < 0 || (int64_t)at + q.n > held));
  return q;
}

__device__ __forceinline__ bool in_pages(int64_t pos, int64_t held) { return pos >= 0 && pos < held; }

// Flags of sequence b from its lengths and the table entries of its rows (one warp).
template <bool APPEND>
__device__ void write_flags(const MoveArgs& a, int b) {
  const int lane = threadIdx.x & 31;
  const Seq q = move_seq<APPEND>(a, b);
  const int64_t held = (int64_t)a.max_pages * a.c.page_size;
  int64_t lo = q.pos0, hi = lo + q.n;
  bool bad = q.bad || (q.n && lo < 0);
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
    a.flags[b] = (uint8_t)((bad ? SV_FLAG_BAD_LENGTH : 0) | (any ? SV_FLAG_BAD_PAGE : 0));
}

// Lanes of a row's group: head_dim / 16 rounded up to a power of two.
template <int DT, bool E4M3, bool APPEND>
__global__ void __launch_bounds__(kMoveWarps * 32) k_move(MoveArgs a, int group_shift) {
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
  const int sub = lane & ((1 << group_shift) - 1);  // 16-element piece of the row
  const int rows = 2 * c.kv_heads;                  // k heads, then v heads
  const int per = 32 >> group_shift;                // rows per step of the warp
  const bool on = sub * 16 < c.head_dim;
  for (int64_t t = (int64_t)blockIdx.x * kMoveWarps + warp; t < a.total;
       t += (int64_t)a.move_blocks * kMoveWarps) {
    const int b = owner_of(a.start, a.B, (int)t);
    if (b >= a.B) continue;  // rows behind the last sequence
    const Seq q = move_seq<APPEND>(a, b);
    const int i = (int)t - q.tok0;
    if (i < 0 || i >= q.n) continue;  // start does not rise
    const int64_t pos = (int64_t)q.pos0 + i;
    int page = -1, slot = 0;
    if (in_pages(pos, held)) {
      page_of(c, (int)pos, page, slot);
      page = __ldg(a.table + (int64_t)b * a.max_pages + page);
    }
    const bool sound = page >= 0 && page < c.num_pages;
    if (APPEND && !sound) continue;
#pragma unroll 4
    for (int r0 = 0; r0 < rows; r0 += per) {
      const int r = r0 + (lane >> group_shift);
      const bool live = r < rows && on;
      const bool is_v = r >= c.kv_heads;
      const int h = is_v ? r - c.kv_heads : r;
      char* pool = (is_v ? c.v : c.k) + (int64_t)page * c.page_bytes + (int64_t)h * c.head_bytes +
                   (int64_t)slot * c.token_bytes;
      uint8_t* scale = (is_v ? c.vs : c.ks) + ((int64_t)page * c.kv_heads + h) * c.page_size + slot;
      if (APPEND) {
        const char* src = (is_v ? a.in_v : a.in_k) + t * a.in_token + (int64_t)h * a.in_head;
        uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
        if (live) {
          x0 = __ldg(reinterpret_cast<const uint4*>(src) + 2 * sub);
          x1 = __ldg(reinterpret_cast<const uint4*>(src) + 2 * sub + 1);
        }
        if (!E4M3) {
          if (live) {
            reinterpret_cast<uint4*>(pool)[2 * sub] = x0;
            reinterpret_cast<uint4*>(pool)[2 * sub + 1] = x1;
          }
        } else {
          const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
          float f[16], m = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 p = F16<DT>::up(w[j]);
            f[2 * j] = p.x;
            f[2 * j + 1] = p.y;
            const float u = fabsf(p.x), v = fabsf(p.y);
            if (u < __int_as_float(0x7f800000)) m = fmaxf(m, u);
            if (v < __int_as_float(0x7f800000)) m = fmaxf(m, v);
          }
          for (int o = 1; o < (1 << group_shift); o <<= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const uint32_t bits = __float_as_uint(m);
          int k = (int)(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
          k = k < kMinScaleExp ? kMinScaleExp : k;
          const float inv = __uint_as_float((uint32_t)(127 - k) << 23);
          if (live) {
            uint32_t o4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t word = 0;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float u = f[4 * j + 2 * e] * inv, v = f[4 * j + 2 * e + 1] * inv;
                // infinities become the NaN code (the conversion would saturate)
                u = fabsf(u) < __int_as_float(0x7f800000) ? u : __int_as_float(0x7fffffff);
                v = fabsf(v) < __int_as_float(0x7f800000) ? v : __int_as_float(0x7fffffff);
                const uint32_t two =
                    __nv_cvt_float2_to_fp8x2(make_float2(u, v), __NV_SATFINITE, __NV_E4M3);
                word |= two << (16 * e);
              }
              o4[j] = word;
            }
            reinterpret_cast<uint4*>(pool)[sub] = make_uint4(o4[0], o4[1], o4[2], o4[3]);
            if (sub == 0) *scale = (uint8_t)(k + 127);
          }
        }
      } else {
        char* dst = (is_v ? a.out_v : a.out_k) + ((t * c.kv_heads + h) * c.head_dim) * 2;
        uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
        if (live && sound) {
          if (!E4M3) {
            x0 = __ldg(reinterpret_cast<const uint4*>(pool) + 2 * sub);
            x1 = __ldg(reinterpret_cast<const uint4*>(pool) + 2 * sub + 1);
          } else {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(pool) + sub);
            const float s = scale_of(__ldg(scale));
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
        }
        if (live) {
          reinterpret_cast<uint4*>(dst)[2 * sub] = x0;
          reinterpret_cast<uint4*>(dst)[2 * sub + 1] = x1;
        }
      }
    }
  }
}

template <bool APPEND>
cudaError_t launch_move(MoveArgs a, int dtype, bool e4m3, cudaStream_t stream) {
  int shift = 0;
  while ((16 << shift) < a.c.head_dim) ++shift;
  const int64_t want = ((int64_t)a.total + kMoveWarps - 1) / kMoveWarps;
  a.move_blocks = (int)(want < (1 << 20) ? want : (1 << 20));
  const int flag_blocks = a.flags ? (a.B + kMoveWarps - 1) / kMoveWarps : 0;
  if (a.move_blocks + flag_blocks == 0) return cudaSuccess;
  auto* k = e4m3 ? (dtype == SV_BF16 ? k_move<SV_BF16, true, APPEND> : k_move<SV_F16, true, APPEND>)
                 : k_move<SV_BF16, false, APPEND>;  // a plain copy of 16-bit values
  return launch_pdl(k, dim3(a.move_blocks + flag_blocks), dim3(kMoveWarps * 32), 0, stream, a, shift);
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
