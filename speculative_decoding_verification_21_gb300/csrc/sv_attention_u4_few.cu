// sv_attention_u4_few.cu -- spec_chunk_attention over a cache of 4-bit codes, for items of few
// query rows: single tokens and short rounds.
//
//   k_j = z_j + s_j c_j:  t_jn = scale log2e (z_j sum(q_n) + s_j (q_n.c_j)) - m_n,
//   p = 2^t,  l_n += p,  Z_n += p (z_j + 8 s_j),  O_n += (p s_j) (c_j - 8);  out_n = (O_n + Z_n) / l_n
//
// Eight warps multiply.  Each has 16 of a tile's 128 keys and works by itself, on two tiles at
// once: products of 16 keys by 8 rows (S^T = K Q^T) and of 16 dimensions by 8 rows (O^T += V^T
// P^T), weights and O in registers, maxima and sums of its own.  They meet at an item's end, where
// their results are added up in shared memory, always in the same order.  A ninth warp fetches
// pages, a tenth the next item's queries, so that neither costs the eight an instruction.
//
// Why not the tensor memory that many rows use (sv_attention_u4_tiles.cu): there a tile costs
// some 2300 clocks of hand-overs between roles, whatever its rows.  Here one of 24 rows takes 1370,
// one of 8 rows 1050 (sequences of 16000 keys on average; both and what follows with raw codes of v,
// centring them adds 2%), where HBM would allow 756: up to 24 rows
// of 128 dimensions are faster here, 32 are not (O no longer fits the registers).  Narrower heads
// leave room for more; the bounds are kFew's.  (Where keys are few it takes many rows too, as more
// items: the rule stands where the calls are told apart.)
//
// What bounds it: latency.  Two warps share a scheduler, O's registers allow no more; of a
// stage's 3000 clocks (two tiles, 24 rows) the products take 1570, the exponentials 400, waits 360.
//
// Tried: a ring of asynchronous copies for each warp (no page warp: 567 instructions for 16 keys
// and 24 rows, now 350; 228 us); sixteen warps, half the rows each, at 104 registers (they spill:
// 260 us).
//
// Work: items of one row tile, cut into equal shares of key tiles (sv_attention_line.cuh).
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "specverify.h"
#include "sv_attention.h"
#include "sv_attention_line.cuh"
#include "sv_attention_u4.cuh"
#include "sv_cache.cuh"
#include "sv_device.cuh"
#include "sv_launch.h"
#include "sv_tma.cuh"

namespace sv {
namespace {

// The eight warps that multiply; one that copies, one that converts queries, and two that make up
// their group, for the registers: a thread has kLaunchRegs at launch, and then by role (the sum
// must not pass what the launch gave, or the takers would wait forever).
constexpr int kFewWarps = 8, kFewThreads = 32 * (kFewWarps + 4);
constexpr int kLaunchRegs = 168, kCopyRegs = 64, kWorkRegs = 216;
static_assert(32 * kFewWarps * kWorkRegs + 128 * kCopyRegs <= kFewThreads * kLaunchRegs, "registers");
constexpr int kFewN = 48;                  // rows of an item, at most
constexpr int kBlock = 16;                 // keys of a tile that are a warp's
constexpr size_t kFewSmem = 227 * 1024;

template <bool FP16>
struct FewArgs : U4ArgsOf<FP16> {
  // (3, 5, 6, 8, 11: rounds of 64 sequences 139, 131, 130, 132, 136 us)
  static constexpr int kItemUnits = 6;
};

struct FewCtl {
  uint64_t full[kMaxStages], empty[kMaxStages], segfull[4], segempty[4], qfull[2], qempty[2];
  int abort;
  int two;                               // (find_share's; not used)
  int b, h, qt, off;
  long long left, share;
  long long warp_units[kFewThreads / 32];
  Seg seg[4];                            // the items (n = 0: no more)
  Walk walk;
  float4 ends[kFewWarps][kFewN];         // a warp's m, l, Z, E of its rows
  float qsum[2][kFewN], qfac[2][kFewN];  // a query row's sum; its factor back to kQShift
  int odd[2];                            // some row has a factor of its own
};

// The warps that multiply, all of them.
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory");
}
__device__ __forceinline__ bool consumers_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "n"(32 * kFewWarps)
      : "memory");
  return r != 0;
}
// c[0], c[1]: row lane / 4, columns 2 (lane % 4) and + 1; c[2], c[3]: the row eight on.
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                      uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}
__device__ __forceinline__ void mma16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                           uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y), "f"(0.0f));
}
// An 8 x 8 matrix of 16-bit entries, two of a row to a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void ld_transposed2(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(addr)
               : "memory");
}
// W consecutive words (of eight codes).
template <int W>
__device__ __forceinline__ void ld_words(uint32_t addr, uint32_t (&w)[W]) {
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr)
                 : "memory");
  else if constexpr (W == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
  else
#pragma unroll
    for (int i = 0; i < W; ++i)
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[i]) : "r"(addr + 4 * i) : "memory");
}

// W: words of a lane (head_dim = 32 W).  NT: eight-row tiles of an item.  EXACT: queries and outputs
// are fp16, and items of few keys have exact weights (kExactKeys).
template <int W, int NT, bool EXACT>
__global__ void __launch_bounds__(kFewThreads, 1)
    k_attend_u4_few(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const __grid_constant__ FewArgs<EXACT> t) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int D = 32 * W, N = 8 * NT;
  constexpr bool bf16 = !EXACT;
  const AttendArgs& a = t.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
  const int wid = (int)blockIdx.x;
  uint8_t* const ring = smem;
  float4* const obuf = reinterpret_cast<float4*>(ring + (size_t)t.ring.n * t.stage_bytes);
  uint4* const qbuf = reinterpret_cast<uint4*>(obuf + 4 * W * NT * 64);  // [2][NT][W][lane]
  FewCtl& ctl = *reinterpret_cast<FewCtl*>(qbuf + 2 * NT * W * 32);
  const Guard guard{&ctl.abort, t.wait_clocks};
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    ctl.two = 0;
    ctl.abort = (smem_u32(smem) & 1023u) ? 1 : 0;  // the swizzles need this alignment
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(ctl.full + i, 33);
      mbar_init(ctl.empty + i, kFewWarps);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(ctl.segfull + i, 1);
      mbar_init(ctl.segempty + i, kFewWarps + 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(ctl.qfull + i, 1);
      mbar_init(ctl.qempty + i, kFewWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  if (threadIdx.x == 0) t.rec[wid].more = 0;  // (the call before may have been reading it till here)
  find_share(t, ctl);
  bool ok = *guard.flag == 0;

  if (warp >= kFewWarps) {
    give_regs<kCopyRegs>();
    if (warp == kFewWarps) copy_tiles(mk, mv, t, ctl, ring, guard, ok);
    if (warp == kFewWarps + 1) {
      // Queries, an item ahead: a lane 8 W elements of a row, in the order of the codes' pairs.
      for (uint32_t items = 0; ok; ++items) {
        const Seg& s = ctl.seg[items & 3u];
        const uint32_t b = items & 1u;
        if (!wait_held(ctl.segfull + (items & 3u), (items >> 2) & 1u, guard, kWaitItem) || s.n == 0 ||
            !wait_held(ctl.qempty + b, ((items >> 1) & 1u) ^ 1u, guard, kWaitQ))
          break;
        bool odd = false;
#pragma unroll 1
        for (int nt = 0; nt < NT; ++nt) {
          const int n = 8 * nt + g;
          uint32_t x[4 * W];
#pragma unroll
          for (int e = 0; e < 4 * W; ++e) x[e] = 0;
          if (n < s.ntok * t.group) {
            const int tok = (int)(n * t.group_inv >> 16), hd = n - tok * t.group;
            const uint4* from = reinterpret_cast<const uint4*>(a.q + (int64_t)(s.row0 + tok) * a.q_token +
                                                               (int64_t)(s.h * t.group + hd) * a.q_head) + q4 * W;
#pragma unroll
            for (int w = 0; w < W; ++w) {
              const uint4 v = __ldg(from + w);
              x[4 * w] = v.x, x[4 * w + 1] = v.y, x[4 * w + 2] = v.z, x[4 * w + 3] = v.w;
            }
          }
          auto up = [&](uint32_t v) { return bf16 ? F16<SV_BF16>::up(v) : F16<SV_F16>::up(v); };
          float top = 0.0f, sum = 0.0f;
#pragma unroll
          for (int e = 0; e < 4 * W; ++e) {
            const float2 p = up(x[e]);
            top = fmaxf(top, fmaxf(fabsf(p.x), fabsf(p.y)));
            sum += p.x + p.y;
          }
#pragma unroll
          for (int d = 1; d < 4; d <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            sum += __shfl_xor_sync(0xffffffffu, sum, d);
          }
          int shift = kQShift;
          if (!(top >= 0.0625f && top < 512.0f) && top > 0.0f && top < kInf) {
            // the largest value into [2^14, 2^15)
            shift = min(126, 14 + 127 - (int)(__float_as_uint(top) >> 23));
            odd = true;
          }
          const float f0 = pow2f(shift), f1 = f0 * 0.0625f;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float2 v0 = up(x[4 * w]), v1 = up(x[4 * w + 1]), v2 = up(x[4 * w + 2]), v3 = up(x[4 * w + 3]);
            qbuf[(((int)b * NT + nt) * W + w) * 32 + lane] =
                make_uint4(F16<SV_F16>::down(v0.x * f0, v2.x * f0), F16<SV_F16>::down(v0.y * f1, v2.y * f1),
                           F16<SV_F16>::down(v1.x * f0, v3.x * f0), F16<SV_F16>::down(v1.y * f1, v3.y * f1));
          }
          if (q4 == 0) {
            ctl.qsum[b][n] = sum;
            ctl.qfac[b][n] = pow2f(kQShift - shift);
          }
        }
        odd = __any_sync(0xffffffffu, odd);
        if (lane == 0) ctl.odd[b] = odd;
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ctl.segempty + (items & 3u));
          // (a test may withhold a CTA's first queries: the waits for them then run out)
          if (t.stall != wid || items) mbar_arrive(ctl.qfull + b);
        }
      }
    }
  } else {
    take_regs<kWorkRegs>();
    constexpr float kUndo = (float)(1 << (24 - kQShift));  // the codes' and the queries' powers
    uint32_t slot = 0, phase = 0;
    for (uint32_t items = 0;; ++items) {
      const Seg& s = ctl.seg[items & 3u];
      bool go = ok && wait_held(ctl.segfull + (items & 3u), (items >> 2) & 1u, guard, kWaitItem) && s.n > 0;
      go = go && wait_held(ctl.qfull + (items & 1u), (items >> 1) & 1u, guard, kWaitQ);
      if (rare(!go)) {  // (the end, or a wait ran out: whoever may be in an item learns of it)
        consumers_any(true);
        break;
      }
      const uint4* const qb = qbuf + (items & 1u) * (NT * W * 32) + lane;
      const float* const qsum = ctl.qsum[items & 1u] + 2 * q4;
      const bool odd = ctl.odd[items & 1u] != 0;
      const int tiles = s.n;
      uint64_t M2[NT], l2[NT], z2[NT];  // -m, sums: of rows 8 nt + 2 q4, + 1
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) M2[nt] = l2[nt] = z2[nt] = 0;
      uint32_t unset = (1u << 2 * NT) - 1;  // bits 2 nt + r: rows that have seen nothing yet
      float lag = -FLT_MAX;                 // what may pass: kLag, nothing while there are such rows
      bool opened = false;                  // O holds something
      float o[2 * W][NT][4];
#pragma unroll
      for (int m = 0; m < 2 * W; ++m)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[m][nt][e] = 0.0f;
      float E = 0.0f, e_up = 0.0f;  // largest step so far, up to a power of two; kUp over it
      // This warp's keys of tile i are first_key + i kTile and on.  Those of tiles [seen0, seen1)
      // are seen, those of tiles [whole0, whole1) by all tokens.
      const int first_key = s.t0 * kTile + kBlock * warp;
      const int seen0 = (max(0, s.lo - first_key - kBlock + 1) + kTile - 1) / kTile;
      const int seen1 = s.hi > first_key ? min(tiles, (s.hi - first_key - 1) / kTile + 1) : 0;
      const int whole1 = (s.pos + 1) / kTile - s.t0;
      const int whole0 = a.window ? max(0, s.pos + s.ntok - 1 - a.window) / kTile + 1 - s.t0 : 0;

      // Two loops, for the registers: a window of 1000 keys, in fp16 and 96 wide, takes 388 us without
      // the exact one, 408 with it, 445 with a branch in one loop for both, and 410 with two bodies of
      // all that an item takes.
      auto all_tiles = [&](auto exact) {
        constexpr int U = exact ? 1 : 2;  // tiles at once (what is exact takes registers)
#pragma unroll 1
        for (int i = 0; i < tiles; i += 2) {
          ok = wait_held(ctl.full + slot, phase, guard, kWaitSlot);
          if (rare(!ok)) break;
#pragma unroll 1
          for (int v = 0; v < 2; v += U) {
            // Block u is tile i + v + u's (of one that is not there, or not seen, all is hidden).
            const int i0 = i + v;
            if (i0 >= seen1 || i0 + U <= seen0) continue;
            constexpr int kCode = kTile * D / 2;
            const uint32_t stage = smem_u32(ring) + slot * t.stage_bytes,
                           block = stage + 2 * kCode * v + kBlock * 16 * W * warp;
            uint32_t words[U][4];  // of K, K + 8, V, V + 8
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                asm volatile("ld.shared.u32 %0, [%1];"
                             : "=r"(words[u][e])
                             : "r"(stage + 4 * kCode + 1024 * (v + u) + 4 * kBlock * warp + 4 * kTile * (e >> 1) +
                                   4 * (g + 8 * (e & 1)))
                             : "memory");
            // ---- S: keys g and g + 8 ----
            float x[U][NT][4];
            {
              uint32_t k0[U][W], k1[U][W];
              // (a lane's words of a row lie in one 16-byte chunk, or W is 1 or 3 and nothing is swizzled)
              const uint32_t in = W == 4   ? 16 * code_chunk(D, g, q4)
                                  : W == 2 ? 16 * code_chunk(D, g, q4 >> 1) + 8 * (q4 & 1)
                                           : 4 * W * q4;
              const uint32_t in8 = W == 4   ? 16 * code_chunk(D, g + 8, q4)
                                   : W == 2 ? 16 * code_chunk(D, g + 8, q4 >> 1) + 8 * (q4 & 1)
                                            : 4 * W * q4;
#pragma unroll
              for (int u = 0; u < U; ++u) {
                ld_words<W>(block + 2 * kCode * u + g * 16 * W + in, k0[u]);
                ld_words<W>(block + 2 * kCode * u + (g + 8) * 16 * W + in8, k1[u]);
              }
#pragma unroll
              for (int w = 0; w < W; ++w) {
                uint32_t a0[U][4], a1[U][4];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                  spread(k0[u][w], a0[u]);
                  spread(k1[u][w], a1[u]);
                }
                uint4 q[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) q[nt] = qb[(nt * W + w) * 32];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int u = 0; u < U; ++u)
                    if (w == 0)
                      mma16_zero(x[u][nt], a0[u][0], a1[u][0], a0[u][1], a1[u][1], make_uint2(q[nt].x, q[nt].y));
                    else
                      mma16(x[u][nt], a0[u][0], a1[u][0], a0[u][1], a1[u][1], make_uint2(q[nt].x, q[nt].y));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int u = 0; u < U; ++u)
                    mma16(x[u][nt], a0[u][2], a1[u][2], a0[u][3], a1[u][3], make_uint2(q[nt].z, q[nt].w));
              }
            }
            if (rare(odd)) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const float2 f = *reinterpret_cast<const float2*>(ctl.qfac[items & 1u] + 8 * nt + 2 * q4);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                  x[u][nt][0] *= f.x;
                  x[u][nt][1] *= f.y;
                  x[u][nt][2] *= f.x;
                  x[u][nt][3] *= f.y;
                }
              }
            }
            // ---- exponents: key 2 u + e is g + 8 e of block u ----
            float step[2 * U], zero[2 * U];
            float top = -kInf;
            bool sound = true;  // no step is larger than E, and no value row is not finite
#pragma unroll
            for (int u = 0; u < U; ++u) {
              uint64_t A2[2], B2[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float A = step_of(words[u][e]) * t.c * kUndo, B = zero_of(words[u][e]) * t.c;
                A2[e] = pack2(A, A);
                B2[e] = pack2(B, B);
                step[2 * u + e] = step_of(words[u][2 + e]);
                zero[2 * u + e] = centre_of(words[u][2 + e]);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const float2 sum = *reinterpret_cast<const float2*>(qsum + 8 * nt);
                const uint64_t Q = pack2(sum.x, sum.y);
                float* const c = x[u][nt];
                unpack2(ffma2(pack2(c[0], c[1]), A2[0], ffma2(Q, B2[0], M2[nt])), c[0], c[1]);
                unpack2(ffma2(pack2(c[2], c[3]), A2[1], ffma2(Q, B2[1], M2[nt])), c[2], c[3]);
              }
            }
            if (rare(i0 + U > whole1 || i0 < whole0 || i0 + U > tiles)) {
              // the rows that see a key: [first, first + span)
#pragma unroll
              for (int k = 0; k < 2 * U; ++k) {
                // token j sees a key if key - pos <= j < key - pos + window
                const int key = first_key + (i0 + (k >> 1)) * kTile + g + 8 * (k & 1), d = key - s.pos;
                const int t0 = max(0, min(d, t.tpt));
                const int t1 = a.window && d <= t.tpt - a.window ? max(0, d + a.window) : t.tpt;
                const int first = t0 * t.group;
                int span = max(0, (t1 == t.tpt ? N : t1 * t.group) - first);
                if (key < s.lo || key >= s.hi || i0 + (k >> 1) >= tiles) span = 0;
                if (!span) step[k] = zero[k] = 0.0f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int r = 0; r < 2; ++r)
                    if ((unsigned)(8 * nt + 2 * q4 + r - first) >= (unsigned)span)
                      x[k >> 1][nt][2 * (k & 1) + r] = -kInf;
              }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                top = max3(max3(top, x[u][nt][0], x[u][nt][1]), x[u][nt][2], x[u][nt][3]);
#pragma unroll
            for (int k = 0; k < 2 * U; ++k) sound &= fabsf(fmaf(zero[k], 0.0f, step[k])) <= E;
            if (rare(__any_sync(0xffffffffu, top > lag || !sound))) {
              // a maximum rises, or the largest step; or a value row is not finite: it weighs nothing
              // (0 times it would not be 0 where it is not seen), the rows that see it get their NaN
              // here
              float ws = 0.0f;
              bool bad = false;
#pragma unroll
              for (int k = 0; k < 2 * U; ++k) {
                const bool finite = fabsf(fmaf(zero[k], 0.0f, step[k])) < kInf;
                bad |= !finite;
                ws = fmaxf(ws, finite ? fabsf(step[k]) : 0.0f);
              }
              if (rare(__any_sync(0xffffffffu, bad))) {
                const float nan = __int_as_float(0x7fffffff);
#pragma unroll
                for (int k = 0; k < 2 * U; ++k)
                  if (!(fabsf(fmaf(zero[k], 0.0f, step[k])) < kInf)) {
                    step[k] = zero[k] = 0.0f;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                      const float* c = x[k >> 1][nt] + 2 * (k & 1);
                      z2[nt] = fadd2(z2[nt], pack2(c[0] == -kInf ? 0.0f : nan, c[1] == -kInf ? 0.0f : nan));
                    }
                  }
              }
              ws = warp_max(ws);
              const float e_now = fmaxf(E, step_bound(ws));
              const float fe = E < e_now ? E * (1.0f / e_now) : 1.0f;
              if (E < e_now) {
                E = e_now;
                e_up = kUp / e_now;
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float m[2], f[2];  // (-m)
                unpack2(M2[nt], m[0], m[1]);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  float most = fmaxf(x[0][nt][r], x[0][nt][2 + r]);
                  if constexpr (U == 2) most = max3(most, x[U - 1][nt][r], x[U - 1][nt][2 + r]);
#pragma unroll
                  for (int d = 4; d < 32; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                  const bool first = (unset >> (2 * nt + r)) & 1u;
                  f[r] = 1.0f;
                  if (first ? most > -kInf : most > kLag) {
                    unset &= ~(1u << (2 * nt + r));
                    f[r] = first ? 0.0f : ex2(-most);
                    m[r] -= most;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                      x[u][nt][r] -= most;
                      x[u][nt][2 + r] -= most;
                    }
                  }
                }
                M2[nt] = pack2(m[0], m[1]);
                // (a row that is seen first has no sums yet but such a NaN)
                const uint64_t f2 = pack2(f[0], f[1]);
                l2[nt] = fmul2(l2[nt], f2);
                z2[nt] = fmul2(z2[nt], f2);
                if (opened) {
#pragma unroll
                  for (int mt = 0; mt < 2 * W; ++mt) {
                    o[mt][nt][0] *= f[0] * fe;
                    o[mt][nt][1] *= f[1] * fe;
                    o[mt][nt][2] *= f[0] * fe;
                    o[mt][nt][3] *= f[1] * fe;
                  }
                }
              }
              if (__all_sync(0xffffffffu, unset == 0)) lag = kLag;
            }
            // ---- weights, as the second operand of V^T P^T ----
            uint2 p[U][NT], rest[U][exact ? NT : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const uint64_t u0 = pack2(step[2 * u] * e_up, step[2 * u] * e_up),
                             u1 = pack2(step[2 * u + 1] * e_up, step[2 * u + 1] * e_up);
              const uint64_t v0 = pack2(zero[2 * u], zero[2 * u]), v1 = pack2(zero[2 * u + 1], zero[2 * u + 1]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const float* c = x[u][nt];
                const uint64_t p0 = pack2(ex2(c[0]), ex2(c[1])), p1 = pack2(ex2(c[2]), ex2(c[3]));
                l2[nt] = fadd2(l2[nt], fadd2(p0, p1));
                z2[nt] = ffma2(p0, v0, ffma2(p1, v1, z2[nt]));
                float w[4];
                unpack2(fmul2(p0, u0), w[0], w[1]);
                unpack2(fmul2(p1, u1), w[2], w[3]);
                const uint32_t h0 = F16<SV_F16>::down(w[0], w[1]), h1 = F16<SV_F16>::down(w[2], w[3]);
                p[u][nt] = make_uint2(transposed(h0), transposed(h1));
                if constexpr (exact) {
                  const float2 r0 = F16<SV_F16>::up(h0), r1 = F16<SV_F16>::up(h1);
                  rest[u][nt] = make_uint2(transposed(F16<SV_F16>::down(w[0] - r0.x, w[1] - r0.y)),
                                           transposed(F16<SV_F16>::down(w[2] - r1.x, w[3] - r1.y)));
                }
              }
            }
            opened = true;
            // ---- O: 32 dimensions to a chunk, dimension 4 c + i of them to class i of column c ----
            const int vr = 8 * ((lane >> 3) & 1) + (lane & 7);
            const uint32_t vrow = block + kCode + vr * 16 * W;
#pragma unroll 1
            for (int turn = 0; turn < (exact ? 2 : 1); ++turn) {
#pragma unroll
              for (int q = 0; q < W; q += 2) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                  uint32_t r[4];
                  if (q + 1 < W)
                    ld_transposed4(vrow + 2 * kCode * u + 16 * code_chunk(D, vr, q + (lane >> 4)), r);
                  else
                    ld_transposed2(vrow + 2 * kCode * u + 16 * code_chunk(D, vr, q), r);
#pragma unroll
                  for (int e = 0; e < 2 && q + e < W; ++e) {
                    uint32_t y0[4], y1[4];
                    spread_centred(r[2 * e], y0);
                    spread_centred(r[2 * e + 1], y1);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                      for (int nt = 0; nt < NT; ++nt)
                        mma16(o[2 * (q + e) + h][nt], y0[2 * h], y0[2 * h + 1], y1[2 * h], y1[2 * h + 1], p[u][nt]);
                  }
                }
              }
              if constexpr (exact) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) p[u][nt] = rest[u][nt];
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(ctl.empty + slot);
          if (++slot == t.ring.n) {
            slot = 0;
            phase ^= 1u;
          }
        }
      };
      if constexpr (EXACT) {
        if (rare(t.exact(s.pos))) all_tiles(std::true_type{});
        else all_tiles(std::false_type{});
      } else {
        all_tiles(std::false_type{});
      }
      // ---- the item's end: the warps' results into one ----
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float l[2], z[2], m[2];
        unpack2(l2[nt], l[0], l[1]);
        unpack2(z2[nt], z[0], z[1]);
        unpack2(M2[nt], m[0], m[1]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
            z[r] += __shfl_xor_sync(0xffffffffu, z[r], d);
          }
          if (g == 0) {
            // (a row that has seen nothing, or nothing but -inf, has l = 0)
            const bool none = (unset >> (2 * nt + r)) & 1u;
            ctl.ends[warp][8 * nt + 2 * q4 + r] = make_float4(none ? -kInf : -m[r], l[r], z[r], E);
          }
        }
      }
      if (consumers_any(!ok)) break;
      const int rows = s.ntok * t.group;
      const int64_t prow = (int64_t)(2 * wid + (s.slot > 0 ? 1 : 0)) * kMaxN;
      // Every warp for itself: of row `lane` (and `lane` + 32), the factor of its O and what is added.
      constexpr int kSets = (N + 31) / 32;
      float co[kSets], add[kSets];
#pragma unroll
      for (int k = 0; k < kSets; ++k) {
        const int n = 32 * k + lane;
        co[k] = add[k] = 0.0f;
        if (n < N) {
          float m = -kInf, L = 0.0f, Z = 0.0f;
#pragma unroll
          for (int w = 0; w < kFewWarps; ++w) m = fmaxf(m, ctl.ends[w][n].x);
#pragma unroll
          for (int w = 0; w < kFewWarps; ++w) {
            const float4 e = ctl.ends[w][n];
            const float f = ex2(e.x - m);
            if (e.y != 0.0f) {  // (a warp that saw nothing has l = 0)
              L += f * e.y;
              Z += f * e.z;
              if (w == warp) co[k] = f * e.w * (pow2f(kDown) / kUp);
            }
          }
          const float inv = s.slot >= 0 ? 1.0f : L == 0.0f ? 0.0f : 1.0f / L;
          co[k] *= inv;
          if (L != 0.0f) add[k] = Z * inv;
          if (warp == 0 && n < rows) {
            if (s.slot >= 0) {
              t.ml[prow + n] = make_float2(m, L);
            } else if (a.lse) {
              const int tok = (int)(n * t.group_inv >> 16), hd = n - tok * t.group;
              a.lse[(int64_t)(s.row0 + tok) * a.heads + s.h * t.group + hd] = lse_of(m, L);
            }
          }
        }
      }
      // Half of the warps hand their O to the other half, which adds its own; then a warp adds up
      // 32 dimensions of eight rows and stores them.
      const bool giver = warp >= kFewWarps / 2;
      float4* const mine = obuf + (warp & 3) * (2 * W * NT * 32) + lane;
#pragma unroll 1
      for (int turn = 0; turn < 2; ++turn) {
        if (giver == (turn == 0)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 f = make_float2(__shfl_sync(0xffffffffu, co[nt / 4], (8 * nt + 2 * q4) & 31),
                                         __shfl_sync(0xffffffffu, co[nt / 4], (8 * nt + 2 * q4 + 1) & 31));
#pragma unroll
            for (int mt = 0; mt < 2 * W; ++mt) {
              const float* x = o[mt][nt];
              float4 y = make_float4(0, 0, 0, 0);
              if (turn) y = mine[(mt * NT + nt) * 32];
              // (an O of no weight is not finite only where nothing may be read from it)
              if (f.x != 0.0f) {
                y.x += x[0] * f.x;
                y.z += x[2] * f.x;
              }
              if (f.y != 0.0f) {
                y.y += x[1] * f.y;
                y.w += x[3] * f.y;
              }
              mine[(mt * NT + nt) * 32] = y;
            }
          }
        }
        consumers_sync();
      }
      for (int u = warp; u < NT * W; u += kFewWarps) {
        const int nt = u / W, q = u - nt * W;
        const float4* from = obuf + lane;
        float4 x = make_float4(0, 0, 0, 0), y = x;
#pragma unroll
        for (int p = 0; p < kFewWarps / 2; ++p) {
          const float4 v = from[p * (2 * W * NT * 32) + (2 * q * NT + nt) * 32];
          const float4 w = from[p * (2 * W * NT * 32) + ((2 * q + 1) * NT + nt) * 32];
          x.x += v.x, x.y += v.y, x.z += v.z, x.w += v.w;
          y.x += w.x, y.y += w.y, y.z += w.z, y.w += w.w;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int n = 8 * nt + 2 * q4 + r, d = 32 * q + 4 * g;
          float z = __shfl_sync(0xffffffffu, add[0], n & 31);
          if constexpr (kSets > 1) {
            const float high = __shfl_sync(0xffffffffu, add[kSets - 1], n & 31);
            if (n >= 32) z = high;
          }
          if (n < rows) {
            const float v[4] = {(r ? x.y : x.x) + z, (r ? x.w : x.z) + z, (r ? y.y : y.x) + z,
                                (r ? y.w : y.z) + z};
            if (s.slot < 0) {
              const int tok = (int)(n * t.group_inv >> 16), hd = n - tok * t.group;
              const int64_t orow = (int64_t)(s.row0 + tok) * a.heads + s.h * t.group + hd;
              *reinterpret_cast<uint2*>(a.out + (orow * D + d) * 2) =
                  bf16 ? make_uint2(F16<SV_BF16>::down(v[0], v[1]), F16<SV_BF16>::down(v[2], v[3]))
                       : make_uint2(F16<SV_F16>::down(v[0], v[1]), F16<SV_F16>::down(v[2], v[3]));
            } else {
              *reinterpret_cast<float4*>(t.part + (prow + n) * D + d) = make_float4(v[0], v[1], v[2], v[3]);
            }
          }
        }
      }
      if (threadIdx.x == 0 && s.slot == 1) t.rec[wid] = Rec{s.more, s.row0, s.ntok, s.h};
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ctl.qempty + (items & 1u));
        mbar_arrive(ctl.segempty + (items & 3u));
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) t.err[wid] = ctl.abort ? kLate | ctl.abort << 8 : 0;
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
template <bool FP16>
using FewKernel = void (*)(const CUtensorMap, const CUtensorMap, const FewArgs<FP16>);
struct Few {
  FewKernel<false> bf16;
  FewKernel<true> fp16;
  int dim, rows, fixed;  // head_dim; rows of an item; bytes of shared memory beside the ring
};
template <int W, int NT>
constexpr Few few() {
  return Few{k_attend_u4_few<W, NT, false>, k_attend_u4_few<W, NT, true>, 32 * W, 8 * NT,
             4 * W * NT * 64 * 16 + 2 * NT * W * 32 * 16 + (int)sizeof(FewCtl)};
}
// By width, the items' rows that there are: as many as the warps' registers hold.  Rounds of 64
// sequences, us here and with the tensor memory: 128 wide 5 rows 106 and 157, 15 rows 110 and
// 157, 20 rows 134 and 157, 30 rows 264 and 155; 96 wide, 20 rows 116 and 146, 30 rows 138 and 147;
// 64 wide, 20 rows 111 and 140, 45 rows 173 and 178; 32 wide, 20 rows 103 and 135.
const Few kFew[] = {few<4, 1>(), few<4, 2>(), few<4, 3>(), few<3, 1>(), few<3, 2>(), few<3, 3>(), few<3, 4>(),
                    few<2, 1>(), few<2, 2>(), few<2, 4>(), few<2, 6>(), few<1, 1>(), few<1, 2>(), few<1, 4>()};

std::mutex g_few_mu;
int g_few_sms[64] = {};

cudaError_t few_ready(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_few_mu);
  if (!g_few_sms[dev]) {
    for (const Few& f : kFew)
      for (const void* k : {(const void*)f.bf16, (const void*)f.fp16}) {
        cudaFuncAttributes attr{};
        e = cudaFuncGetAttributes(&attr, k);
        if (e != cudaSuccess) return e;
        if (attr.numRegs < kLaunchRegs) return cudaErrorInvalidKernelImage;  // the roles' shares count on them
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewSmem);
        if (e != cudaSuccess) return e;
      }
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    g_few_sms[dev] = n;
  }
  *sms = g_few_sms[dev];
  return cudaSuccess;
}

// The smallest that takes `rows` rows, or else the largest there is.
const Few* few_for(int dim, int rows) {
  const Few* best = nullptr;
  for (const Few& f : kFew)
    if (f.dim == dim && !(best && best->rows >= rows)) best = &f;
  return best;
}

}  // namespace

int u4_few_rows(int head_dim, int rows) { return few_for(head_dim, rows)->rows; }

cudaError_t launch_attention_u4_few(const U4Args& call, const CUtensorMap& mk, const CUtensorMap& mv,
                                    int rows, int dtype, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = few_ready(&sms);
  if (e != cudaSuccess) return e;
  U4Args t = call;
  const Few& f = *few_for(t.a.c.head_dim, rows);
  t.tpt = f.rows / t.group;
  t.ring = make_ring(((int)kFewSmem - f.fixed) / t.stage_bytes, kMaxStages);
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  e = dtype == SV_BF16 ? launch_pdl(f.bf16, dim3(ctas), dim3(kFewThreads), kFewSmem, stream, mk, mv, FewArgs<false>{t})
                       : launch_pdl(f.fp16, dim3(ctas), dim3(kFewThreads), kFewSmem, stream, mk, mv,
                                    FewArgs<true>{U4ExactArgs{t}});
  return e == cudaSuccess ? launch_u4_join(t, dtype, ctas, stream) : e;
}

}  // namespace sv
