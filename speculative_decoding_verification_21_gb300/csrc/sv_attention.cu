// sv_attention.cu -- spec_chunk_attention for caches that the tile kernel does not
// take (tiles_take): causal attention of each sequence's chunk of new tokens over
// its pages, one query row per CTA.
//
//   s_j = scale q.k_j over the keys seen, m = max_j s_j, p_j = exp(s_j - m),
//   out = (sum_j p_j v_j) / (sum_j p_j),  lse = m + log sum_j p_j
//
// in one pass over the keys with a running m: when it rises by d, the sums so far
// are multiplied by exp(-d).
#include <cuda_runtime.h>

#include <cstdint>

#include "specverify.h"
#include "sv_attention.h"
#include "sv_cache.cuh"
#include "sv_device.cuh"
#include "sv_launch.h"
#include "sv_tma.cuh"

namespace sv {
namespace {

constexpr int kRowWarps = 4;
constexpr int kMaxHeadDim = 256;

// One CTA per query row (token and head): its warps take blocks of 32 keys in
// turn, a lane one key of the block for the scores and eight columns for the
// products with v, and their sums meet in shared memory.
template <int DT, bool E4M3>
__global__ void __launch_bounds__(kRowWarps * 32) k_attend_rows(AttendArgs a) {
  __shared__ float sq[kMaxHeadDim];
  __shared__ float so[kRowWarps][kMaxHeadDim];
  __shared__ float sm[kRowWarps], sl[kRowWarps];
  pdl_launch_dependents();
  pdl_wait();
  const CacheView& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = c.head_dim;
  const int t = (int)(blockIdx.x / a.heads), hq = (int)(blockIdx.x - (unsigned)t * a.heads);
  const int b = owner_of(a.b.q_start, a.b.B, t);
  if (b >= a.b.B) return;
  const Seq q = load_seq(a.b, b, c.page_size);
  const int i = t - q.tok0;
  if (i < 0 || i >= q.n) return;
  const int pos = q.pos0 + i;
  const int hi = pos + 1 < 0 ? 0 : pos + 1;
  const int lo = a.window && hi > a.window ? hi - a.window : 0;
  const int h = hq / (a.heads / c.kv_heads);
  const char* qrow = a.q + (int64_t)t * a.q_token + (int64_t)hq * a.q_head;
  for (int d = threadIdx.x; d < D / 2; d += kRowWarps * 32) {
    const float2 f = F16<DT>::up(__ldg(reinterpret_cast<const uint32_t*>(qrow) + d));
    sq[2 * d] = f.x * a.scale_log2;
    sq[2 * d + 1] = f.y * a.scale_log2;
  }
  __syncthreads();
  const int32_t* table = a.b.table + (int64_t)b * a.b.max_pages;
  float m = -kInf, l = 0.0f, o[8] = {};
  for (int j0 = lo / 32 * 32 + warp * 32; j0 < hi; j0 += kRowWarps * 32) {
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
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  if (lane * 8 < D)
#pragma unroll
    for (int e = 0; e < 8; ++e) so[warp][lane * 8 + e] = o[e];
  __syncthreads();
  float M = -kInf, L = 0.0f;
  for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, sm[w]);
  float f[kRowWarps];
  for (int w = 0; w < kRowWarps; ++w) {
    f[w] = sm[w] == -kInf ? (sl[w] == 0.0f ? 0.0f : 1.0f) : ex2(sm[w] - M);
    L += f[w] * sl[w];
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  char* orow = a.out + ((int64_t)t * a.heads + hq) * D * 2;
  for (int d = threadIdx.x; d < D / 2; d += kRowWarps * 32) {
    float x = 0.0f, y = 0.0f;
    for (int w = 0; w < kRowWarps; ++w) {
      x = fmaf(f[w], so[w][2 * d], x);
      y = fmaf(f[w], so[w][2 * d + 1], y);
    }
    reinterpret_cast<uint32_t*>(orow)[d] = F16<DT>::down(x * inv, y * inv);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(int64_t)t * a.heads + hq] = L == 0.0f ? -kInf : (M == -kInf ? 0.0f : M) * kLn2 + logf(L);
}

__global__ void __launch_bounds__(256) k_attend_flags(AttendArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = (int)(blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5));
  if (b >= a.b.B) return;
  const uint8_t f = sequence_flags(a, b);
  if ((threadIdx.x & 31) == 0) a.flags[b] = f;
}

}  // namespace

size_t attention_workspace_bytes(const CacheView& c, bool e4m3) {
  return tiles_take(c, e4m3) ? attention_tiles_workspace(c.head_dim) : 0;
}

cudaError_t launch_attention(const AttendArgs& a, int dtype, bool e4m3, cudaStream_t stream) {
  if (tiles_take(a.c, e4m3) && a.scale_log2 >= 0.0f) {
    bool taken = false;
    const cudaError_t e = launch_attention_tiles(a, dtype, e4m3, stream, &taken);
    if (e != cudaSuccess || taken) return e;
  }
  if (a.flags) {
    const cudaError_t e = launch_pdl(k_attend_flags, dim3((a.b.B + 7) / 8), dim3(256), 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  if (a.b.total == 0) return cudaSuccess;
  auto* k = dtype == SV_BF16 ? (e4m3 ? k_attend_rows<SV_BF16, true> : k_attend_rows<SV_BF16, false>)
                             : (e4m3 ? k_attend_rows<SV_F16, true> : k_attend_rows<SV_F16, false>);
  return launch_pdl(k, dim3((unsigned)((int64_t)a.b.total * a.heads)), dim3(kRowWarps * 32), 0,
                    stream, a);
}

}  // namespace sv
