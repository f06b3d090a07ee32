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
#include "sv_attention_row.cuh"
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
  const int b = owner_of(a.b.q_start, a.b.B, t, a.b.total);
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
  float m = -kInf, l = 0.0f, o[8] = {};
  attend_blocks<DT, E4M3, 4>(a, b, h, lo, hi, sq, warp, kRowWarps, m, l, o);
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
