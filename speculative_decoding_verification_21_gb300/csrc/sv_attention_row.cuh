// sv_attention_row.cuh -- one query row of spec_chunk_attention in plain arithmetic: the
// row kernel's loop, and what the tile kernel's join mends rows with.
#pragma once

#include <cstdint>

#include "sv_attention.h"
#include "sv_cache.cuh"
#include "sv_device.cuh"

namespace sv {

// One warp takes every `step`-th block of 32 keys of [lo, hi), from block `first_block`
// on: a lane has one key of the block for the scores and eight columns for the products
// with v.  sq: the query times scale_log2 (shared memory).  m: the warp's running
// maximum; l: the lane's share of the sum; o: the lane's columns.  Nothing outside
// [lo, hi) is read.  UNROLL: of the loops over columns and keys (1 where registers count).
template <int DT, bool E4M3, int UNROLL>
__device__ __forceinline__ void attend_blocks(const AttendArgs& a, int b, int h, int lo, int hi,
                                              const float* sq, int first_block, int step, float& m,
                                              float& l, float (&o)[8]) {
  const CacheView& c = a.c;
  const int lane = threadIdx.x & 31, D = c.head_dim;
  const int32_t* table = a.b.table + (int64_t)b * a.b.max_pages;
  for (int j0 = lo / 32 * 32 + 32 * first_block; j0 < hi; j0 += 32 * step) {
    const int j = j0 + lane;
    const bool seen = j >= lo && j < hi;
    int page = -1, slot = 0;
    if (seen) {
      page_of(c, j, page, slot);
      page = __ldg(table + page);
      if (page < 0 || page >= c.num_pages) page = -1;
    }
    const int64_t at = (int64_t)page * c.page_bytes + (int64_t)h * c.head_bytes +
                       (int64_t)slot * c.token_bytes;
    const int64_t sat = ((int64_t)page * c.kv_heads + h) * c.page_size + slot;
    float s = seen ? 0.0f : -kInf, vs = 1.0f;
    if (page >= 0) {
      if (E4M3) {
        vs = scale_of(__ldg(c.vs + sat));
        const float ks = scale_of(__ldg(c.ks + sat));
#pragma unroll UNROLL
        for (int d = 0; d < D; d += 16) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(c.k + at + d));
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 f = e4m3x2((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
            const float2 r = F16<DT>::up(F16<DT>::down(f.x * ks, f.y * ks));
            s = fmaf(r.x, sq[d + 2 * e], s);
            s = fmaf(r.y, sq[d + 2 * e + 1], s);
          }
        }
      } else {
#pragma unroll UNROLL
        for (int d = 0; d < D; d += 8) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(c.k + at + 2 * d));
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 r = F16<DT>::up(w[e]);
            s = fmaf(r.x, sq[d + 2 * e], s);
            s = fmaf(r.y, sq[d + 2 * e + 1], s);
          }
        }
      }
    }
    const float bm = fmaxf(m, warp_max(s));
    if (bm > m) {
      const float f = m == -kInf ? 0.0f : ex2(m - bm);
      l *= f;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= f;
      m = bm;
    }
    // a NaN score (fmaxf passes it over) keeps its NaN here
    const float p = seen ? (m == -kInf ? (s == s ? 0.0f : s) : ex2(s - m)) : 0.0f;
    l += p;
    const int first = max(0, lo - j0), last = min(32, hi - j0);
#pragma unroll UNROLL
    for (int e = first; e < last; ++e) {
      const int64_t vat = __shfl_sync(0xffffffffu, at, e);
      const int vpage = __shfl_sync(0xffffffffu, page, e);
      const float pe = __shfl_sync(0xffffffffu, p, e), ve = __shfl_sync(0xffffffffu, vs, e);
      if (vpage < 0 || lane * 8 >= D) continue;
      if (E4M3) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(c.v + vat) + lane);
        const uint32_t w[2] = {x.x, x.y};
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float2 f = e4m3x2((uint16_t)(w[d >> 1] >> (16 * (d & 1))));
          const float2 r = F16<DT>::up(F16<DT>::down(f.x * ve, f.y * ve));
          o[2 * d] = fmaf(pe, r.x, o[2 * d]);
          o[2 * d + 1] = fmaf(pe, r.y, o[2 * d + 1]);
        }
      } else {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(c.v + vat) + lane);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const float2 r = F16<DT>::up(w[d]);
          o[2 * d] = fmaf(pe, r.x, o[2 * d]);
          o[2 * d + 1] = fmaf(pe, r.y, o[2 * d + 1]);
        }
      }
    }
  }
}

}  // namespace sv
