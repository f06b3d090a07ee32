// sv_rope.cu -- spec_kv_append_rope: a chunk's queries and keys rotated by their positions,
// the keys and values into the pages of the cache.
//
//   x' = x c - y s,  y' = y c + x s   for the pairs of a head's first rot elements,
//   (c, s) from row t of a table for a token at position t; fp32, each operation rounded,
//   so that equal inputs give equal codes whatever computes them.
//
// Bound by HBM: rows in, rows and codes out.  A warp takes one token (or a part of its
// rows, where there are few tokens; or two tokens, where there are many).  A lane has 16
// elements of a row as two pieces of 8, chosen so that both halves of a pair are its own:
// [8p, 8p + 8) and [rot/2 + 8p, ...) of pairs (i, i + rot/2), neighbours else.  Its eight
// cosines and sines are then the same for every row of the token: 64 bytes read once.
//
// Measured: 94 thousand tokens of 32 + 8 + 8 heads of 128 into 4 bits, and their reading back,
// 2.4 GB, 457 us, 5.3 TB/s (0.80 of a copy's rate); what is missing is the arithmetic between
// loads and stores, more than half of the issue slots.  Steps on the way: a step's rows loaded
// while those before are turned 514 -> 488 us; 32 warps an SM instead of 24 (64 registers) 470,
// 40 warps 544 (what is spilled then); two tokens a warp instead of four 457, one 461.  7387
// tokens of 28 heads of 96 into 4 bits 23 us; 320 tokens into e4m3 6 us in a graph, 24 as a call
// from Python.
#include <cuda_runtime.h>

#include <cstdint>

#include "specverify.h"
#include "sv_cache.cuh"
#include "sv_device.cuh"
#include "sv_launch.h"
#include "sv_tma.cuh"

namespace sv {
namespace {

constexpr int kRopeWarps = 8;

struct RopeArgs {
  CacheView c;
  BatchView b;
  const char* in_k;
  const char* in_v;
  const char* q;
  char* out_q;
  const float* table;         // [positions][rot]
  uint8_t* flags;
  int64_t in_token, in_head;  // strides of the new rows in bytes
  int64_t q_token, q_head;
  int positions, rot, heads;
  int group_shift;            // lanes of a row: 1 << group_shift
  int per;                    // tokens of a warp
  int parts, part_steps;      // warps of a token (1 unless per is 1), and steps of each
  int move_blocks;            // blocks that move rows; the rest write flags
};

// Rows tok0 .. tok0+n-1 of sequence b, the first of them at position pos0.
struct Chunk {
  int tok0, n;
  int64_t pos0;
  bool bad;
};
__device__ __forceinline__ Chunk load_chunk(const RopeArgs& a, int b) {
  const int s0 = __ldg(a.b.q_start + b), s1 = __ldg(a.b.q_start + b + 1);
  const int len = __ldg(a.b.kv_len + b);
  const int64_t held = (int64_t)a.b.max_pages * a.c.page_size;
  const Seq q = make_seq(s0, s1, len, a.b.total, held);
  Chunk k{q.tok0, q.n, (int64_t)len - q.n, q.bad};
  k.bad |= k.n && (k.pos0 < 0 || k.pos0 + k.n > (held < a.positions ? held : (int64_t)a.positions));
  return k;
}

// Flags of sequence b from its lengths and the table entries of its rows (one warp).
__device__ void rope_flags(const RopeArgs& a, int b) {
  const int lane = threadIdx.x & 31;
  const Chunk q = load_chunk(a, b);
  const int64_t held = (int64_t)a.b.max_pages * a.c.page_size;
  const int64_t top = held < a.positions ? held : (int64_t)a.positions;
  const int64_t lo = q.pos0 < 0 ? 0 : q.pos0, end = q.pos0 + q.n, hi = end > top ? top : end;
  bool page_bad = false;
  if (hi > lo) {
    const int p0 = (int)(lo / a.c.page_size), p1 = (int)((hi - 1) / a.c.page_size);
    for (int p = p0 + lane; p <= p1; p += 32) {
      const int page = __ldg(a.b.table + (int64_t)b * a.b.max_pages + p);
      page_bad |= page < 0 || page >= a.c.num_pages;
    }
  }
  const bool any = __any_sync(0xffffffffu, page_bad);
  if (lane == 0)
    a.flags[b] = (uint8_t)((q.bad ? SV_FLAG_BAD_LENGTH : 0) | (any ? SV_FLAG_BAD_PAGE : 0));
}

// Where packed row t belongs.  page: -1 nowhere in the cache, -2 no sequence has the row;
// angle: its row of the table, -1 outside it (the cache's page is then -1 too).
struct Place {
  int page, slot, angle;
};
__device__ __forceinline__ Place place_of(const RopeArgs& a, int b, int t) {
  Place p{-2, 0, -1};
  if (b >= a.b.B) return p;  // rows behind the last sequence
  const Chunk q = load_chunk(a, b);
  const int i = t - q.tok0;
  if (i < 0 || i >= q.n) return p;  // start does not rise
  const int64_t pos = q.pos0 + i;
  p.page = -1;
  if (pos < 0 || pos >= a.positions) return p;
  p.angle = (int)pos;
  if (pos >= (int64_t)a.b.max_pages * a.c.page_size) return p;
  int index;
  page_of(a.c, (int)pos, index, p.slot);
  const int page = __ldg(a.b.table + (int64_t)b * a.b.max_pages + index);
  if (page >= 0 && page < a.c.num_pages) p.page = page;
  return p;
}

// (not the read-only path: the output of a query may be its own place)
__device__ __forceinline__ uint4 ld_row16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// The lane's pairs turned by its cosines and sines.
template <bool NEXT>
__device__ __forceinline__ void turn(float (&f)[16], const float (&cs)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    constexpr int kStep = NEXT ? 2 : 1, kOther = NEXT ? 1 : 8;
    float& x = f[kStep * i];
    float& y = f[kStep * i + kOther];
    const float u = __fsub_rn(__fmul_rn(x, cs[i]), __fmul_rn(y, cs[8 + i]));
    y = __fadd_rn(__fmul_rn(y, cs[i]), __fmul_rn(x, cs[8 + i]));
    x = u;
  }
}

template <int DT>
__device__ __forceinline__ void narrow16(const float (&f)[16], uint4& x0, uint4& x1) {
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = F16<DT>::down(f[2 * j], f[2 * j + 1]);
  x0 = make_uint4(w[0], w[1], w[2], w[3]);
  x1 = make_uint4(w[4], w[5], w[6], w[7]);
}

// NEXT: pairs (2i, 2i + 1).
template <int DT, int FMT, bool NEXT>
__global__ void __launch_bounds__(kRopeWarps * 32, 4)
    k_append_rope(const __grid_constant__ RopeArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int)blockIdx.x >= a.move_blocks) {
    const int b = ((int)blockIdx.x - a.move_blocks) * kRopeWarps + warp;
    if (b < a.b.B) rope_flags(a, b);
    return;
  }
  const CacheView& c = a.c;
  const int64_t unit = (int64_t)blockIdx.x * kRopeWarps + warp;
  const int64_t first = unit / a.parts * a.per;
  const int part = (int)(unit % a.parts);
  if (first >= a.b.total) return;
  const int t0 = (int)first, n = min(a.per, a.b.total - t0);
  // the sequence of the first token, and mostly of all
  const int b0 = owner_of(a.b.q_start, a.b.B, t0, a.b.total);
  const bool same = n == 1 || (b0 < a.b.B && t0 + n <= __ldg(a.b.q_start + b0 + 1));
  Place mine{-2, 0, -1};
  if (same) {
    if (lane < n) mine = place_of(a, b0, t0 + lane);
  } else {
    for (int j = 0; j < n; ++j) {
      const int b = owner_of(a.b.q_start, a.b.B, t0 + j, a.b.total);
      if (lane == j) mine = place_of(a, b, t0 + j);
    }
  }
  const int sub = lane & ((1 << a.group_shift) - 1);  // the lane's 16 elements of a row
  const int row = lane >> a.group_shift;              // row of a step
  const bool on = sub * 16 < c.head_dim, turned = sub * 16 < a.rot;
  const int e0 = turned && !NEXT ? 8 * sub : 16 * sub;
  const int e1 = turned && !NEXT ? a.rot / 2 + 8 * sub : 16 * sub + 8;
  const int at_once = 32 >> a.group_shift;
  const int q_steps = (a.heads + at_once - 1) / at_once;
  const int kv_steps = (2 * c.kv_heads + at_once - 1) / at_once;
  const int from = part * a.part_steps, upto = min(q_steps + kv_steps, from + a.part_steps);
  for (int j = 0; j < n; ++j) {
    const int page = __shfl_sync(0xffffffffu, mine.page, j);
    const int slot = __shfl_sync(0xffffffffu, mine.slot, j);
    const int angle = __shfl_sync(0xffffffffu, mine.angle, j);
    if (page == -2) continue;
    const int64_t t = t0 + j;
    float cs[16] = {};
    if (turned && angle >= 0) {
      const float* r = a.table + (int64_t)angle * a.rot + 8 * sub;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // eight cosines, eight sines
        const float4 x = __ldg(reinterpret_cast<const float4*>(r + (i >> 1) * (a.rot / 2)) + (i & 1));
        cs[4 * i] = x.x;
        cs[4 * i + 1] = x.y;
        cs[4 * i + 2] = x.z;
        cs[4 * i + 3] = x.w;
      }
    }
    // A step's rows are loaded while those of the step before are turned and stored.
    const int last = page < 0 ? min(upto, q_steps) : upto;
    uint4 n0 = make_uint4(0, 0, 0, 0), n1 = n0;
    auto fetch = [&](int step) {
      if (step < q_steps) {
        const int h = step * at_once + row;
        if (h < a.heads && on && angle >= 0) {
          const char* src = a.q + t * a.q_token + (int64_t)h * a.q_head;
          n0 = ld_row16(src + 2 * e0);
          n1 = ld_row16(src + 2 * e1);
        }
      } else {
        const int r = (step - q_steps) * at_once + row;
        n0 = n1 = make_uint4(0, 0, 0, 0);
        if (r < 2 * c.kv_heads && on) {
          const int h = r >= c.kv_heads ? r - c.kv_heads : r;
          const char* src = (r >= c.kv_heads ? a.in_v : a.in_k) + t * a.in_token + (int64_t)h * a.in_head;
          n0 = ld_stream16(src + 2 * e0);
          n1 = ld_stream16(src + 2 * e1);
        }
      }
    };
    if (from < last) fetch(from);
    for (int step = from; step < last; ++step) {
      uint4 x0 = n0, x1 = n1;
      if (step + 1 < last) fetch(step + 1);
      if (step < q_steps) {  // queries
        const int h = step * at_once + row;
        if (h >= a.heads || !on) continue;
        if (turned && angle >= 0) {
          float f[16];
          widen16<DT>(x0, x1, f);
          turn<NEXT>(f, cs);
          narrow16<DT>(f, x0, x1);
        }
        char* dst = a.out_q + (t * a.heads + h) * c.head_dim * 2;
        *reinterpret_cast<uint4*>(dst + 2 * e0) = x0;
        *reinterpret_cast<uint4*>(dst + 2 * e1) = x1;
        continue;
      }
      // keys, then values
      const int r = (step - q_steps) * at_once + row;
      const bool live = r < 2 * c.kv_heads && on, is_v = r >= c.kv_heads;
      const int h = is_v ? r - c.kv_heads : r;
      char* dst = (is_v ? c.v : c.k) + (int64_t)page * c.page_bytes + (int64_t)h * c.head_bytes +
                  (int64_t)slot * c.token_bytes;
      const int64_t at = ((int64_t)page * c.kv_heads + h) * c.page_size + slot;
      const bool turns = turned && !is_v;
      if (FMT == kHalf) {
        if (turns) {
          float f[16];
          widen16<DT>(x0, x1, f);
          turn<NEXT>(f, cs);
          narrow16<DT>(f, x0, x1);
        }
        if (live) {
          *reinterpret_cast<uint4*>(dst + 2 * e0) = x0;
          *reinterpret_cast<uint4*>(dst + 2 * e1) = x1;
        }
        continue;
      }
      float f[16];
      widen16<DT>(x0, x1, f);
      if (turns) turn<NEXT>(f, cs);
      if (FMT == kE4m3) {
        int k;
        const uint4 o = encode_e4m3(f, amax16(f), a.group_shift, k);
        if (live) {
          *reinterpret_cast<uint2*>(dst + e0) = make_uint2(o.x, o.y);
          *reinterpret_cast<uint2*>(dst + e1) = make_uint2(o.z, o.w);
          if (sub == 0) (is_v ? c.vs : c.ks)[at] = (uint8_t)(k + 127);
        }
      } else {
        float lo, hi;
        uint32_t sz;
        range16(f, on, lo, hi);
        const uint2 o = encode_u4(f, lo, hi, a.group_shift, sz);
        if (live) {
          *reinterpret_cast<uint32_t*>(dst + e0 / 2) = o.x;
          *reinterpret_cast<uint32_t*>(dst + e1 / 2) = o.y;
          if (sub == 0) reinterpret_cast<uint32_t*>(is_v ? c.vs : c.ks)[at] = sz;
        }
      }
    }
  }
}

template <int FMT>
auto rope_kernel(int dtype, bool next) {
  return dtype == SV_BF16 ? (next ? k_append_rope<SV_BF16, FMT, true> : k_append_rope<SV_BF16, FMT, false>)
                          : (next ? k_append_rope<SV_F16, FMT, true> : k_append_rope<SV_F16, FMT, false>);
}

}  // namespace

cudaError_t launch_kv_append_rope(const sv_kv_cache& c, const sv_kv_batch& b, const sv_rope& rope,
                                  const void* new_k, const void* new_v, int dtype,
                                  int64_t token_stride, int64_t head_stride, const void* q,
                                  int heads, int64_t q_token_stride, int64_t q_head_stride,
                                  void* out_q, uint8_t* out_flags, cudaStream_t stream) {
  RopeArgs a{};
  a.c = cache_view(c);
  a.b = BatchView{b.block_table, b.q_start, b.kv_len, (int)b.total, b.B, b.max_pages};
  a.in_k = (const char*)new_k;
  a.in_v = (const char*)new_v;
  a.q = (const char*)q;
  a.out_q = (char*)out_q;
  a.table = rope.cos_sin;
  a.flags = out_flags;
  a.in_token = token_stride * 2;
  a.in_head = head_stride * 2;
  a.q_token = q_token_stride * 2;
  a.q_head = q_head_stride * 2;
  a.positions = (int)rope.positions;
  a.rot = rope.rot_dim;
  a.heads = heads;
  while ((16 << a.group_shift) < c.head_dim) ++a.group_shift;
  const int at_once = 32 >> a.group_shift;
  const int steps = (heads + at_once - 1) / at_once + (2 * c.kv_heads + at_once - 1) / at_once;
  // two tokens a warp where that still gives every SM 16 warps; fewer tokens than that
  // are cut into parts for as many warps
  constexpr int64_t kWarps = 152 * 16;
  a.per = b.total >= kWarps * 2 ? 2 : 1;
  a.parts = 1;
  a.part_steps = steps;
  if (b.total > 0 && b.total < kWarps) {
    const int64_t want = kWarps / b.total;
    a.part_steps = want >= steps ? 1 : (int)((steps + want - 1) / want);
    a.parts = (steps + a.part_steps - 1) / a.part_steps;
  }
  const int64_t units = ((b.total + a.per - 1) / a.per) * a.parts;
  a.move_blocks = (int)((units + kRopeWarps - 1) / kRopeWarps);
  const int flag_blocks = a.flags ? (b.B + kRopeWarps - 1) / kRopeWarps : 0;
  if (a.move_blocks + flag_blocks == 0) return cudaSuccess;
  const Format fmt = format_of(c.dtype);
  const bool next = rope.interleaved != 0;
  auto* k = fmt == kE4m3 ? rope_kernel<kE4m3>(dtype, next)
            : fmt == kU4 ? rope_kernel<kU4>(dtype, next) : rope_kernel<kHalf>(dtype, next);
  return launch_pdl(k, dim3(a.move_blocks + flag_blocks), dim3(kRopeWarps * 32), 0, stream, a);
}

}  // namespace sv
