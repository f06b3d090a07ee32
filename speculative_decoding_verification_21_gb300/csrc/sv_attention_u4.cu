// sv_attention_u4.cu -- spec_chunk_attention over a cache of 4-bit codes.
//
//   k_j = z_j + s_j c_j:  score_j = z_j sum(q) + s_j (q.c_j),
//   out = (sum_j (p_j s_j) c_j + sum_j p_j z_j) / sum_j p_j
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

// What the tile kernels do not take: head sizes above 128, pages that are no power of two or below
// 16 tokens, more than 80 query heads to a key head, steps and zeros off 16 bytes.  Plain fp32,
// right and not fast (rounds of 64 sequences on up to 8192 keys, 128 wide, took it 5.2 ms); bound
// by its instructions, a product, a mask and a conversion for every query row and code.
//
// One CTA per query row (token and head): its warps take blocks of 32 keys in turn, a lane
// one key of the block for the scores and eight columns for the products with v, and their
// sums meet in shared memory.
template <int DT>
__global__ void __launch_bounds__(kRowWarps * 32) k_attend_rows_u4(AttendArgs a) {
  __shared__ float sq[kMaxHeadDim];
  __shared__ float so[kRowWarps][kMaxHeadDim];
  __shared__ float sm[kRowWarps], sl[kRowWarps], part[kRowWarps];
  pdl_launch_dependents();
  pdl_wait();
  const CacheView& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = c.head_dim;
  const int t = (int)(blockIdx.x / a.heads), hq = (int)(blockIdx.x - (unsigned)t * a.heads);
  const int b = owner_of(a.b.q_start, a.b.B, t, a.b.total);
  if (b >= a.b.B) return;
  const Seq q = load_seq(a.b, b, c.page_size);
  const int i = t - q.tok0;
  if (i < 0 || i >= q.n) return;
  const int hi = max(0, q.pos0 + i + 1);
  const int lo = a.window && hi > a.window ? hi - a.window : 0;
  const int h = hq / (a.heads / c.kv_heads);
  const char* qrow = a.q + (int64_t)t * a.q_token + (int64_t)hq * a.q_head;
  float sum = 0.0f;
  for (int d = threadIdx.x; d < D / 2; d += kRowWarps * 32) {
    const float2 f = F16<DT>::up(__ldg(reinterpret_cast<const uint32_t*>(qrow) + d));
    sq[2 * d] = f.x;
    sq[2 * d + 1] = f.y;
    sum += f.x + f.y;
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  sum = part[0] + part[1] + part[2] + part[3];
  float m = -kInf, l = 0.0f, o[8] = {};
  const int32_t* table = a.b.table + (int64_t)b * a.b.max_pages;
  for (int j0 = lo / 32 * 32 + 32 * warp; j0 < hi; j0 += 32 * kRowWarps) {
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
    float s = seen ? 0.0f : -kInf;
    uint32_t vsz = 0;
    if (page >= 0) {
      const uint32_t ksz = __ldg(reinterpret_cast<const uint32_t*>(c.ks) + sat);
      vsz = __ldg(reinterpret_cast<const uint32_t*>(c.vs) + sat);
      float dot = 0.0f;
      for (int d = 0; d < D; d += 32) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(c.k + at + d / 2));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 32; ++e) dot = fmaf(code_of(w[e >> 3], e & 7), sq[d + e], dot);
      }
      s = fmaf(zero_of(ksz), sum, step_of(ksz) * dot) * a.scale_log2;
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
      const float pe = __shfl_sync(0xffffffffu, p, e);
      const uint32_t sz = __shfl_sync(0xffffffffu, vsz, e);
      if (vpage < 0 || lane * 8 >= D) continue;
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(c.v + vat) + lane);
#pragma unroll
      for (int d = 0; d < 8; ++d)
        o[d] = fmaf(pe, fmaf(step_of(sz), code_of(w, d), zero_of(sz)), o[d]);
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

}  // namespace

cudaError_t launch_attention_rows_u4(const AttendArgs& a, int dtype, cudaStream_t stream) {
  auto* k = dtype == SV_BF16 ? k_attend_rows_u4<SV_BF16> : k_attend_rows_u4<SV_F16>;
  return launch_pdl(k, dim3((unsigned)((int64_t)a.b.total * a.heads)), dim3(kRowWarps * 32), 0, stream, a);
}

}  // namespace sv
