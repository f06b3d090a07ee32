// sv_attention_u4_tiles.cu -- spec_chunk_attention over a cache of 4-bit codes on the tensor
// cores: tiles of 128 keys against up to 80 query rows, transposed.
//
//   k_j = z_j + s_j c_j:  t_jn = scale log2e (z_j sum(q_n) + s_j (q_n.c_j)) - m_n,
//   p = 2^t,  l_n += p,  Z_n += p z_j,  O_n += (p s_j) c_j;  out_n = (O_n + Z_n) / l_n
//
// A code c in 0..15 is a 16-bit float by itself: the subnormal c 2^-24, or c 2^-20 four bits
// further up.  So a word of eight codes becomes four pairs of tensor-core operands by four
// masks and a shift, nothing is dequantised, and the powers of two go into the queries
// and the outputs.  The products are exact; steps and zeros act in fp32 on the scores (a row
// of k) and on the weights (a row of v).
//
// The codes are operand A and go through tensor memory, a key (of K) or a dimension (of V)
// to a lane:  S^T [128 keys x N rows] = K Q^T,  O^T [dims x N rows] += V^T P^T.  Shared memory
// then carries the codes once (4 bits), Q, and P; and the products cost by the query rows
// that there are, not by 128.  N is 16 to 80, the rows of an item: tokens of a chunk times
// the query heads that share a key head.
//
// Work: items of one row tile, cut into equal shares of key tiles (sv_attention_line.cuh).
//
// Roles of the 16 or 20 warps: 0 fetches pages (tensor copies; steps and zeros by bulk
// copies), 1 issues the products, 2 and 3 convert queries, then four or eight spread K's and
// V's codes, and eight are two softmax groups of half the columns each.  A softmax thread has one key and N/2
// rows.  The running maxima are columns: they are looked at again only when some score
// passes one by kLag (a vote of the group's threads), so a tile needs no reduction across
// lanes, and the sums stay per thread to the item's end.
//
// Every wait is bounded; one that gives up ends the CTA's roles and flags the call.  The
// softmax warps, which meet at barriers of their own, then go through their tiles without
// waiting for anything.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "specverify.h"
#include "sv_attention.h"
#include "sv_attention_line.cuh"
#include "sv_cache.cuh"
#include "sv_device.cuh"
#include "sv_launch.h"
#include "sv_tma.cuh"
#include "sv_umma.cuh"

namespace sv {
namespace {

constexpr int kMaxN = 80;              // 3 N columns beside 256 of operands in tensor memory
constexpr int kMaxStages = 12;
constexpr int kSpan = 16384;           // 128 rows of a 128-byte swizzle span
constexpr size_t kSmemBytes = 227 * 1024;
// By N: groups of four warps that spread codes, threads, and the registers of a thread at
// launch and then by role (the roles' sum must not pass what the launch gave, or the takers
// would wait forever).
template <int N>
struct Shape {
  static constexpr int kSpread = N <= 32 ? 2 : 1;
  static constexpr int kWarps = 4 + 4 * kSpread + 8, kThreads = 32 * kWarps;
  static constexpr int kRegs = kSpread == 2 ? 96 : 128;
  static constexpr int kHelpRegs = 64, kSoftRegs = kSpread == 2 ? 144 : 192;
  static_assert((kThreads - 256) * kHelpRegs + 256 * kSoftRegs <= kThreads * kRegs, "registers");
};
// A maximum may lag by this many powers of two, and a weight p s is at most 2^kLag kUp = 2^15
// in fp16, s relative to the largest step seen: weights keep all their bits down to 2^-23
// of that, and some to 2^-33.
constexpr float kLag = 6.0f;
constexpr float kUp = 512.0f;
// Queries times 2^kQShift (and 2^-4 of that where the code sits four bits higher): rows with
// a largest value within [2^-4, 2^9) fit fp16 so, to the last bit of all that matters (what
// is below 2^-19 is rounded to 2^-27).  Other rows get a factor of their own.
constexpr int kQShift = 6;

struct U4Args {
  static constexpr int kItemUnits = 3, kRowTiles = 1, kSlotRows = kMaxN;
  AttendArgs a;
  int group, tpt;      // query heads per key head; tokens per row tile
  int box;             // tokens per copy: min(page_size, 128)
  int spans;           // of 64 dimensions, of a query row: 1 or 2
  Ring ring;
  int stage_bytes;
  int stall;           // test only: the CTA whose first scores are withheld (-1: none)
  long long wait_clocks;
  float c;             // scale log2 e
  float* part;         // [2 * kMaxCtas][kMaxN][head_dim]
  float2* ml;          // [2 * kMaxCtas][kMaxN]
  Rec* rec;            // [kMaxCtas]
  int* err;            // [kMaxCtas]
};

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t qfull[2], qempty[2], kfull[2], kfree[2], vfull[2], sfull[2], pfull[2], pfree[2];
  uint64_t ofull, oempty, fin;
  uint32_t tmem;
  int abort;
  int two;             // (find_share's; not used)
  int b, h, qt, off;   // start of the CTA's share (off in units)
  long long left, share;
  long long warp_units[Shape<16>::kWarps];
  float qsum[2][kMaxN], qfac[2][kMaxN];  // of each query row: sum, factor back to kQShift
  int odd[2][2];                         // a row (of a converting warp) has a factor of its own
  // by softmax group:
  float4 qm[2][kMaxN / 4];               // of two rows: sums, -m
  float m[2][kMaxN / 2];
  float fac[2][kMaxN / 2];               // of a rise: old over new weights
  float wmax[2][4][kMaxN / 2], wstep[2][4];
  float2 lz[2][4][kMaxN / 2];            // sums of a warp's keys
  float2 fin_lz[2][kMaxN / 2];           // factor of O, what is added
};

// ---------------------------------------------------------------------------
// Primitives.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_ld8_async(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
// 16 lanes: registers 2j and 2j+1 of thread t go to lanes t/4 and t/4 + 8, column 4j + t%4.
__device__ __forceinline__ void tmem_st_rows8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(taddr)
      : "memory");
}
// Four 8 x 8 matrices of 16-bit entries, transposed: thread t gets entries t/4 of rows
// 2(t%4) and 2(t%4)+1 of each; lane l gives the address of row l%8 of matrix l/8.
__device__ __forceinline__ void ld_transposed4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// The 128 threads of a softmax group.
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// The 16-byte chunk of a code row that holds its i-th, as the copies lay it out (a 64- or
// 32-byte swizzle where rows of 16 bytes' steps would meet in the banks).
__device__ __forceinline__ int code_chunk(int D, int row, int i) {
  return D == 128 ? i ^ ((row >> 1) & 3) : D == 64 ? i ^ ((row >> 2) & 1) : i;
}
// Eight codes as four pairs (i, i + 4), i = 0..3.
__device__ __forceinline__ void spread(uint32_t w, uint32_t* r) {
  const uint32_t v = w >> 8;
  r[0] = w & 0x000F000Fu;
  r[1] = w & 0x00F000F0u;
  r[2] = v & 0x000F000Fu;
  r[3] = v & 0x00F000F0u;
}

enum WaitId { kWaitSlot = 1, kWaitQ, kWaitK, kWaitV, kWaitP, kWaitQFree, kWaitS, kWaitO, kWaitCodes,
              kWaitFree };

// Sums (or largest, NaNs passed over) over a warp's lanes of C values (a multiple of 8)
// each: lane l ends with those of C / 8 columns from first_column(l) on, in v[0..].
template <int C, bool MAX>
__device__ __forceinline__ void over_lanes(float (&v)[C]) {
  const int lane = threadIdx.x & 31;
  auto join = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int o = 16, n = C / 2; o >= 4; o >>= 1, n >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? v[n + i] : v[i], send = up ? v[i] : v[n + i];
      v[i] = join(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
#pragma unroll
  for (int o = 2; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < C / 8; ++i) v[i] = join(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
}
template <int C>
__device__ __forceinline__ int first_column(int lane) {
  return (lane & 16 ? C / 2 : 0) + (lane & 8 ? C / 4 : 0) + (lane & 4 ? C / 8 : 0);
}

// Of row n of two (Q: sums, M: -m): n = 2i, 2i+1.
__device__ __forceinline__ void set_m(float4* qm, int n, float neg_m) {
  reinterpret_cast<float*>(qm + (n >> 1))[2 + (n & 1)] = neg_m;
}

template <int DT, int N>
__global__ void __launch_bounds__(Shape<N>::kThreads, 1)
    k_attend_u4(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                const __grid_constant__ U4Args t) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int C = N / 2;                            // rows of a softmax group
  constexpr int kSpread = Shape<N>::kSpread, kSoft = 4 + 4 * kSpread;  // first softmax warp
  constexpr int kPBytes = N > 64 ? 2 * kSpan : kSpan;
  constexpr uint32_t kColV = 128, kColS = 256, kColO = 256 + 2 * N;  // tensor memory
  const AttendArgs& a = t.a;
  const int D = a.c.head_dim;
  const int q_bytes = t.spans * N * 128, code_bytes = kTile * D / 2;
  uint8_t* const pbuf = smem;
  uint8_t* const qbuf = pbuf + 2 * kPBytes;
  uint8_t* const ring = qbuf + 2 * q_bytes;
  Ctl& ctl = *reinterpret_cast<Ctl*>(ring + (size_t)t.ring.n * t.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wid = (int)blockIdx.x;
  const Guard guard{&ctl.abort, t.wait_clocks};

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    ctl.two = 0;
    ctl.abort = (smem_u32(smem) & 1023u) ? 1 : 0;  // the swizzles need this alignment
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(ctl.full + i, 1);
      mbar_init(ctl.empty + i, 4 * kSpread + 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(ctl.qfull + i, 2);
      mbar_init(ctl.qempty + i, 1 + 8);
      mbar_init(ctl.kfull + i, 4);
      mbar_init(ctl.kfree + i, 1);
      mbar_init(ctl.vfull + i, 4);
      mbar_init(ctl.sfull + i, 1);
      mbar_init(ctl.pfull + i, 8);
      mbar_init(ctl.pfree + i, 1);
    }
    mbar_init(&ctl.ofull, 1);
    mbar_init(&ctl.oempty, 8);
    mbar_init(&ctl.fin, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = ctl.tmem;
  pdl_wait();
  find_share(t, ctl);
  Walk walk(ctl);
  Seg s;
  bool ok = *guard.flag == 0;
  if (warp < kSoft) give_regs<Shape<N>::kHelpRegs>();

  if (warp == 0) {
    // ---------------- fetch key and value pages ----------------
    // Lanes 0-7 and 16-23 hold a tile's copies of K and of V; page numbers are read a tile
    // ahead.
    const uint64_t pol = l2_policy_evict_first();
    const int which = lane >> 4, part = lane & 15;
    const int copies = kTile / t.box;
    uint32_t k = 0;
    while (ok && walk.next(t, ctl, s)) {
      const int32_t* table = a.b.table + (int64_t)s.b * a.b.max_pages;
      auto look = [&](int i, int& from, int& upto) {
        const int key0 = (s.t0 + i) * kTile;
        from = max(0, s.lo - key0) / t.box;
        upto = min(copies, (max(0, s.hi - key0) + t.box - 1) / t.box);
        return part >= from && part < upto ? __ldg(table + ((key0 + part * t.box) >> a.c.page_shift)) : -1;
      };
      int from, upto;
      int page = look(0, from, upto);
      for (int i = 0; ok && i < s.n; ++i) {
        const Slot at(k, t.ring);
        ok = wait_warp(ctl.empty + at.i, at.ph ^ 1u, guard, kWaitSlot);
        if (!ok) break;
        uint8_t* const stage = ring + (size_t)at.i * t.stage_bytes;
        const int live = max(0, upto - from);
        const bool mine = part >= from && part < upto;
        const bool sound = page >= 0 && page < a.c.num_pages;  // (then `mine` too)
        const int in_page = ((s.t0 + i) * kTile + part * t.box) & (a.c.page_size - 1);
        uint8_t* const words = stage + 2 * code_bytes + (which * kTile + part * t.box) * 4;
        // a page outside the pool arrives as zeros; so do its steps and zeros
        if (mine && !sound)
          for (int e = 0; e < 4 * t.box; e += 16)
            *reinterpret_cast<uint4*>(words + e) = make_uint4(0, 0, 0, 0);
        const uint32_t bytes = (uint32_t)(2 * live * t.box * (D / 2)) +
                               __popc(__ballot_sync(0xffffffffu, sound)) * 4 * t.box;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(ctl.full + at.i, bytes);
        __syncwarp();
        if (mine) {
          tma_load_4d_hint(stage + which * code_bytes + part * t.box * (D / 2), which ? &mv : &mk, 0,
                           in_page, s.h, page, ctl.full + at.i, pol);
          if (sound)
            bulk_load(words,
                      (which ? a.c.vs : a.c.ks) +
                          (((int64_t)page * a.c.kv_heads + s.h) * a.c.page_size + in_page) * 4,
                      (uint32_t)(4 * t.box), ctl.full + at.i);
        }
        __syncwarp();
        ++k;
        if (i + 1 < s.n) page = look(i + 1, from, upto);
      }
    }
    // every copy has landed before the CTA may exit
    for (uint32_t i = k > t.ring.n ? k - t.ring.n : 0; i < k; ++i) {
      const Slot at(i, t.ring);
      if (lane == 0) wait_end(ctl.full + at.i, at.ph, guard);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- issue the products ----------------
    const uint32_t leader = elect_leader();
    const uint32_t idesc_s = umma_idesc_16(false, kTile, N, false);
    const uint32_t idesc_o = umma_idesc_16(false, kTile, N, true);
    const uint32_t tb = (uint32_t)uniform((int)tbase);
    const int ksteps = D / 16;
    const uint64_t qdesc = umma_smem_desc(smem_u32(qbuf), 16, 1024);
    const uint64_t pdesc = umma_smem_desc(smem_u32(pbuf), kSpan, 1024);
    uint32_t g = 0, qn = 0;  // tiles and items before
    while (ok && walk.next(t, ctl, s)) {
      const int n = uniform(s.n);
      const uint32_t qb = qn & 1u;
      auto scores = [&](uint32_t j, bool last) {
        const uint32_t b = j & 1u;
        if (!wait_warp(ctl.kfull + b, (j >> 1) & 1u, guard, kWaitK)) return false;
        tc_fence_after();
        const uint32_t acc = tb + kColS + b * N, ka = tb + b * 64;
        const uint64_t qd = qdesc + qb * ((uint32_t)q_bytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t o = (uint64_t)((kk >> 2) * (N * 128 >> 4) + (kk & 3) * 2);
          if (kk < ksteps) umma_ts_if(leader, acc, ka + kk * 8, qd + o, idesc_s, kk != 0);
        }
        umma_commit_if(leader, ctl.kfree + b);
        // (a test may withhold a CTA's first scores: the softmax's wait then runs out)
        umma_commit_if(t.stall == wid && j == 0 ? 0u : leader, ctl.sfull + b);
        if (last) umma_commit_if(leader, ctl.qempty + qb);
        return true;
      };
      ok = wait_warp(ctl.qfull + qb, (qn >> 1) & 1u, guard, kWaitQ) && scores(g, n == 1);
      for (int i = 0; ok && i < n; ++i) {
        const uint32_t j = g + (uint32_t)i, b = j & 1u;
        if (i + 1 < n) ok = scores(j + 1, i + 2 == n);
        ok = ok && wait_warp(ctl.vfull + b, (j >> 1) & 1u, guard, kWaitV) &&
             (i > 0 || wait_warp(&ctl.oempty, (qn & 1u) ^ 1u, guard, kWaitO)) &&
             wait_warp(ctl.pfull + b, (j >> 1) & 1u, guard, kWaitP);
        if (!ok) break;
        tc_fence_after();
        const uint32_t va = tb + kColV + b * 64;
        const uint64_t pd = pdesc + b * (kPBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ts_if(leader, tb + kColO, va + kk * 8, pd + (uint64_t)(kk * 128), idesc_o, kk || i);
        umma_commit_if(leader, ctl.pfree + b);
        if (i == n - 1) umma_commit_if(leader, &ctl.ofull);
      }
      g += (uint32_t)n;
      ++qn;
    }
    // all products complete before tensor memory is released
    umma_commit_if(leader, &ctl.fin);
    wait_end(&ctl.fin, 0, guard);
  } else if (warp < 4) {
    // ---------------- convert queries ----------------
    // Half a warp to a row, eight elements a lane, in the order of the codes' pairs:
    // 0 4 1 5 2 6 3 7.
    const int sub = lane & 15, side = 2 * (warp - 2) + (lane >> 4);
    uint32_t qn = 0;
    if (warp == 2 && lane == 0) t.rec[wid].more = 0;
    for (; ok && walk.next(t, ctl, s); ++qn) {
      if (warp == 2 && lane == 0 && s.slot == 1) t.rec[wid] = Rec{s.more, s.row0, s.ntok, s.h};
      const uint32_t qb = qn & 1u;
      ok = wait_warp(ctl.qempty + qb, ((qn >> 1) & 1u) ^ 1u, guard, kWaitQFree);
      if (!ok) break;
      bool odd = false;
      const int rows = s.ntok * t.group;
#pragma unroll 2
      for (int n = side; n < N; n += 4) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (n < rows && sub * 8 < D) {
          const int tok = n / t.group, hd = n - tok * t.group;
          x = __ldg(reinterpret_cast<const uint4*>(a.q + (int64_t)(s.row0 + tok) * a.q_token +
                                                   (int64_t)(s.h * t.group + hd) * a.q_head) + sub);
        }
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        float f[8], top = 0.0f, sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 p = F16<DT>::up(w[e]);
          f[2 * e] = p.x;
          f[2 * e + 1] = p.y;
          top = fmaxf(top, fmaxf(fabsf(p.x), fabsf(p.y)));
          sum += p.x + p.y;
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        int shift = kQShift;
        if (!(top >= 0.0625f && top < 512.0f) && top > 0.0f && top < kInf) {
          // the largest value into [2^14, 2^15)
          shift = min(126, 14 + 127 - (int)(__float_as_uint(top) >> 23));
          odd = true;
        }
        const float f0 = pow2f(shift), f1 = f0 * 0.0625f;
        if (sub * 8 < D) {
          uint8_t* const to = qbuf + qb * q_bytes + (sub >> 3) * (N * 128) + n * 128 + (((sub & 7) ^ (n & 7)) << 4);
          *reinterpret_cast<uint4*>(to) =
              make_uint4(F16<SV_F16>::down(f[0] * f0, f[4] * f0), F16<SV_F16>::down(f[1] * f1, f[5] * f1),
                         F16<SV_F16>::down(f[2] * f0, f[6] * f0), F16<SV_F16>::down(f[3] * f1, f[7] * f1));
        }
        if (sub == 0) {
          ctl.qsum[qb][n] = sum;
          ctl.qfac[qb][n] = pow2f(kQShift - shift);
        }
      }
      const bool any = __any_sync(0xffffffffu, odd);
      if (lane == 0) ctl.odd[qb][warp - 2] = any;
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(ctl.qfull + qb);
    }
  } else if (warp < kSoft) {
    // ---------------- spread codes ----------------
    // One group of four warps for K and one for V, or one for both.
    const int quad = warp & 3, row = 32 * quad + lane;
    const bool does_k = kSpread == 1 || warp < 8, does_v = kSpread == 1 || warp >= 8;
    const uint32_t lanes = tbase + ((uint32_t)(32 * quad) << 16);
    uint32_t j = 0;
    while (ok && walk.next(t, ctl, s)) {
      for (int i = 0; i < s.n; ++i, ++j) {
        const Slot at(j, t.ring);
        const uint32_t b = j & 1u, ph = (j >> 1) & 1u;
        const uint8_t* const codes = ring + (size_t)at.i * t.stage_bytes;
        ok = wait_warp(ctl.full + at.i, at.ph, guard, kWaitCodes);
        if (!ok) break;
        if (does_k) {
          ok = wait_warp(ctl.kfree + b, ph ^ 1u, guard, kWaitFree);
          if (!ok) break;
          tc_fence_after();
          // a key to a lane: pairs (i, i + 4) of each eight dimensions
#pragma unroll 2
          for (int ch = 0; ch < D / 32; ++ch) {
            const uint4 x = *reinterpret_cast<const uint4*>(codes + row * (D / 2) + 16 * code_chunk(D, row, ch));
            uint32_t r[16];
            spread(x.x, r);
            spread(x.y, r + 4);
            spread(x.z, r + 8);
            spread(x.w, r + 12);
            tmem_st16(lanes + b * 64 + 16 * ch, r);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ctl.kfull + b);
        }
        if (does_v) {
          ok = wait_warp(ctl.pfree + b, ph ^ 1u, guard, kWaitFree);
          if (!ok) break;
          tc_fence_after();
          // a dimension to a lane, pairs of tokens: lane 8i + c of the warp's 32 takes
          // dimension 4c + i of its 32
          if (32 * quad < D) {
            const uint32_t base = smem_u32(codes + code_bytes);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t lo[16], hi[16];
#pragma unroll
              for (int m4 = 0; m4 < 2; ++m4) {
                const int token = 64 * half + 32 * m4 + lane;
                uint32_t x[4];
                ld_transposed4(base + token * (D / 2) + 16 * code_chunk(D, token, quad), x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t r[4];
                  spread(x[e], r);
                  lo[8 * m4 + 2 * e] = r[0];
                  lo[8 * m4 + 2 * e + 1] = r[1];
                  hi[8 * m4 + 2 * e] = r[2];
                  hi[8 * m4 + 2 * e + 1] = r[3];
                }
              }
              tmem_st_rows8(lanes + kColV + b * 64 + 32 * half, lo);
              tmem_st_rows8(lanes + (16u << 16) + kColV + b * 64 + 32 * half, hi);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ctl.vfull + b);
        }
        if (lane == 0) mbar_arrive(ctl.empty + at.i);
      }
    }
  } else {
    // ---------------- softmax and output ----------------
    take_regs<Shape<N>::kSoftRegs>();
    const int wg = (warp - kSoft) >> 2, quad = warp & 3, row = 32 * quad + lane, id = 1 + wg;
    const int tid = row;                          // of the group's 128
    const uint32_t lanes = tbase + ((uint32_t)(32 * quad) << 16);
    const uint32_t o_tm = lanes + kColO + wg * C;
    const int n0 = wg * C;                        // the group's first row
    float4* const qm = ctl.qm[wg];
    const float c18 = t.c * pow2f(24 - kQShift);  // undoes the codes' and the queries' powers
    uint32_t g = 0, qn = 0;
    for (; walk.next(t, ctl, s); ++qn) {
      const uint32_t qb = qn & 1u;
      if (ok) ok = wait_warp(ctl.qfull + qb, (qn >> 1) & 1u, guard, kWaitQ);
      if (tid < C) {
        reinterpret_cast<float*>(qm + (tid >> 1))[tid & 1] = ctl.qsum[qb][n0 + tid];
        set_m(qm, tid, kInf);
        ctl.m[wg][tid] = -kInf;
      }
      const bool odd = ctl.odd[qb][0] | ctl.odd[qb][1];
      group_sync(id);
      uint64_t l2[C / 2], z2[C / 2];
#pragma unroll
      for (int i = 0; i < C / 2; ++i) l2[i] = z2[i] = 0;
      float E = 0.0f, inv_e = 0.0f;  // largest step so far, up to a power of two; its inverse
      for (int i = 0; i < s.n; ++i, ++g) {
        const Slot at(g, t.ring);
        const uint32_t b = g & 1u, ph = (g >> 1) & 1u;
        const uint32_t s_tm = lanes + kColS + b * N + wg * C;
        // S is there, so the tile's steps and zeros are too, and O's product of two tiles ago
        // is done (it was issued before this S): P's place is free
        if (ok) ok = wait_warp(ctl.sfull + b, ph, guard, kWaitS);
        tc_fence_after();
        // the key's step and zero, and the rows that see it: [first, first + span) of the group's
        const uint32_t* const words =
            reinterpret_cast<const uint32_t*>(ring + (size_t)at.i * t.stage_bytes + 2 * code_bytes);
        uint32_t ksz = words[row], vsz = words[kTile + row];
        const int key = (s.t0 + i) * kTile + row;
        int first = 0, span = C;
        const bool edge = (s.t0 + i + 1) * kTile > s.pos + 1 ||
                          (a.window && (s.t0 + i) * kTile <= s.pos + s.ntok - 1 - a.window);
        if (edge) {
          // token i sees it if key - pos <= i < key - pos + window
          const int d = key - s.pos;
          const int t0 = max(0, min(d, t.tpt));
          const int t1 = a.window && d <= t.tpt - a.window ? max(0, d + a.window) : t.tpt;
          const int r0 = max(0, t0 * t.group - n0);
          const int r1 = t1 == t.tpt ? C : min(C, t1 * t.group - n0);
          first = r0;
          span = max(0, r1 - r0);
          if (key < s.lo || key >= s.hi) span = 0;
          if (!span) ksz = vsz = 0;
        }
        const bool masked = edge && __any_sync(0xffffffffu, span < C);
        const float A = step_of(ksz) * c18, B = zero_of(ksz) * t.c;
        const float step = step_of(vsz), zero = zero_of(vsz);
        uint32_t r[C];
        auto load = [&]() {
#pragma unroll
          for (int u = 0; u < C; u += 8) tmem_ld8_async(s_tm + u, r + u);
          tmem_wait_ld();
          if (odd) {
#pragma unroll
            for (int n = 0; n < C; ++n)
              r[n] = __float_as_uint(__uint_as_float(r[n]) * ctl.qfac[qb][n0 + n]);
          }
        };
        // t of all rows
        auto exponents = [&]() {
          const uint64_t A2 = pack2(A, A), B2 = pack2(B, B);
#pragma unroll
          for (int n = 0; n < C; n += 2) {
            const float4 k = qm[n >> 1];
            float x, y;
            unpack2(ffma2(pack2(__uint_as_float(r[n]), __uint_as_float(r[n + 1])), A2,
                          ffma2(pack2(k.x, k.y), B2, pack2(k.z, k.w))), x, y);
            r[n] = __float_as_uint(x);
            r[n + 1] = __float_as_uint(y);
          }
          if (masked) {
#pragma unroll
            for (int n = 0; n < C; ++n)
              if ((unsigned)(n - first) >= (unsigned)span) r[n] = 0xff800000u;
          }
        };
        load();
        exponents();
        float top = -kInf;
#pragma unroll
        for (int n = 0; n < C; ++n) top = fmaxf(top, __uint_as_float(r[n]));
        if (group_any(id, top > kLag || step > E)) {
          // some maximum rises, or the largest step
          load();
          const uint64_t A2 = pack2(A, A), B2 = pack2(B, B);
          float v[C];
#pragma unroll
          for (int n = 0; n < C; n += 2) {
            const float4 k = qm[n >> 1];
            unpack2(ffma2(pack2(__uint_as_float(r[n]), __uint_as_float(r[n + 1])), A2,
                          fmul2(pack2(k.x, k.y), B2)), v[n], v[n + 1]);
            if ((unsigned)(n - first) >= (unsigned)span) v[n] = -kInf;
            if ((unsigned)(n + 1 - first) >= (unsigned)span) v[n + 1] = -kInf;
          }
          over_lanes<C, true>(v);
          if ((lane & 3) == 0)
#pragma unroll
            for (int n = 0; n < C / 8; ++n) ctl.wmax[wg][quad][first_column<C>(lane) + n] = v[n];
          const float ws = warp_max(step < kInf ? step : 0.0f);
          if (lane == 0) ctl.wstep[wg][quad] = ws;
          group_sync(id);
          if (tid < C) {
            const float was = ctl.m[wg][tid];
            float now = was;
#pragma unroll
            for (int w = 0; w < 4; ++w) now = fmaxf(now, ctl.wmax[wg][w][tid]);
            ctl.m[wg][tid] = now;
            ctl.fac[wg][tid] = now > was ? ex2(was - now) : 1.0f;
            set_m(qm, tid, -now);
          }
          float most = 0.0f;
#pragma unroll
          for (int w = 0; w < 4; ++w) most = fmaxf(most, ctl.wstep[wg][w]);
          const uint32_t up = (__float_as_uint(most) + 0x7fffffu) & 0x7f800000u;  // to a power of two
          const float e_now = fmaxf(E, __uint_as_float(up));
          const float fe = E < e_now ? E * (1.0f / e_now) : 1.0f;
          group_sync(id);
          if (i) {
#pragma unroll
            for (int n = 0; n < C; n += 2) {
              const float2 f = *reinterpret_cast<const float2*>(ctl.fac[wg] + n);
              l2[n / 2] = fmul2(l2[n / 2], pack2(f.x, f.y));
              z2[n / 2] = fmul2(z2[n / 2], pack2(f.x, f.y));
            }
            // O: the product of the tile before is done
            if (ok) ok = wait_warp(ctl.pfree + (b ^ 1u), ((g - 1) >> 1) & 1u, guard, kWaitFree);
            tc_fence_after();
#pragma unroll 1
            for (int u = 0; u < C; u += 8) {
              uint32_t o[8];
              float f[8];
              bool still = true;
#pragma unroll
              for (int n = 0; n < 8; ++n) {
                f[n] = ctl.fac[wg][u + n] * fe;
                still = still && f[n] == 1.0f;
              }
              if (still) continue;  // (the same for all threads)
              tmem_ld8_async(o_tm + u, o);
              tmem_wait_ld();
#pragma unroll
              for (int n = 0; n < 8; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * f[n]);
              tmem_st8(o_tm + u, o);
            }
            tmem_wait_st();
          }
          if (E < e_now) {
            E = e_now;
            inv_e = 1.0f / e_now;
          }
          load();
          exponents();
        }
        // weights.  A value row that is not finite weighs nothing here (0 times it would not
        // be 0 where it is not seen); the rows that do see it get their NaN below
        const bool bad = !(step < kInf && fabsf(zero) < kInf);
        const float up = bad ? 0.0f : step * inv_e * kUp, zero_in = bad ? 0.0f : zero;
        const uint64_t up2 = pack2(up, up), zero2 = pack2(zero_in, zero_in);
        uint8_t* const prow = pbuf + b * kPBytes + row * 128;
#pragma unroll
        for (int u = 0; u < C; u += 8) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int n = u + e;
            const uint64_t p = pack2(ex2(__uint_as_float(r[n])), ex2(__uint_as_float(r[n + 1])));
            l2[n / 2] = fadd2(l2[n / 2], p);
            z2[n / 2] = ffma2(p, zero2, z2[n / 2]);
            float x, y;
            unpack2(fmul2(p, up2), x, y);
            w[e / 2] = F16<SV_F16>::down(x, y);
          }
          const int ch = (n0 + u) >> 3;
          *reinterpret_cast<uint4*>(prow + (ch >> 3) * kSpan + (((ch & 7) ^ (row & 7)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (__any_sync(0xffffffffu, bad)) {
          const float nan = bad ? __int_as_float(0x7fffffff) : 0.0f;
#pragma unroll
          for (int n = 0; n < C; n += 2)
            z2[n / 2] = fadd2(z2[n / 2], pack2((unsigned)(n - first) < (unsigned)span ? nan : 0.0f,
                                               (unsigned)(n + 1 - first) < (unsigned)span ? nan : 0.0f));
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ctl.pfull + b);
          mbar_arrive(ctl.empty + at.i);
        }
      }
      // ---- the item's end: sums over the keys, then O ----
      {
        float v[C];
#pragma unroll
        for (int n = 0; n < C; n += 2) unpack2(l2[n / 2], v[n], v[n + 1]);
        over_lanes<C, false>(v);
        const int col = first_column<C>(lane);
        if ((lane & 3) == 0)
#pragma unroll
          for (int n = 0; n < C / 8; ++n) ctl.lz[wg][quad][col + n].x = v[n];
#pragma unroll
        for (int n = 0; n < C; n += 2) unpack2(z2[n / 2], v[n], v[n + 1]);
        over_lanes<C, false>(v);
        if ((lane & 3) == 0)
#pragma unroll
          for (int n = 0; n < C / 8; ++n) ctl.lz[wg][quad][col + n].y = v[n];
      }
      group_sync(id);
      const int rows = s.ntok * t.group;  // live ones of the item
      const int64_t prow = (int64_t)(2 * wid + (s.slot > 0 ? 1 : 0)) * kMaxN + n0;
      if (tid < C) {
        float L = 0.0f, Z = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 x = ctl.lz[wg][w][tid];
          L += x.x;
          Z += x.y;
        }
        const float m = ctl.m[wg][tid];
        if (s.slot >= 0) {
          ctl.fin_lz[wg][tid] = make_float2(1.0f, Z);
          if (n0 + tid < rows) t.ml[prow + tid] = make_float2(m, L);
        } else {
          const float inv = L == 0.0f ? 0.0f : 1.0f / L;
          ctl.fin_lz[wg][tid] = make_float2(inv, L == 0.0f ? 0.0f : Z * inv);
          if (a.lse && n0 + tid < rows) {
            const int tok = (n0 + tid) / t.group, hd = n0 + tid - tok * t.group;
            a.lse[(int64_t)(s.row0 + tok) * a.heads + s.h * t.group + hd] = lse_of(m, L);
          }
        }
      }
      group_sync(id);
      if (ok) ok = wait_warp(&ctl.ofull, qn & 1u, guard, kWaitO);
      tc_fence_after();
      // lane 8i + c of the warp's 32 has dimension 4c + i, with codes 2^-24 or 2^-20 high
      const int dim = 32 * quad + 4 * (lane & 7) + (lane >> 3);
      const float back = (lane & 8 ? pow2f(20) : pow2f(24)) / kUp;
      int tok = n0 / t.group, hd = n0 - tok * t.group;
#pragma unroll 1
      for (int u = 0; u < C; u += 8) {
        uint32_t o[8];
        __syncwarp();
        tmem_ld8_async(o_tm + u, o);
        tmem_wait_ld();
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          if (n0 + u + n < rows && dim < D) {
            const float2 f = ctl.fin_lz[wg][u + n];
            // (rows that saw nothing: O was never weighed, f is 0)
            const float x = E == 0.0f ? 0.0f : __uint_as_float(o[n]) * back * E;
            const float y = fmaf(x, f.x, f.y);
            if (s.slot < 0) {
              const int64_t orow = (int64_t)(s.row0 + tok) * a.heads + s.h * t.group + hd;
              reinterpret_cast<uint16_t*>(a.out)[orow * D + dim] = (uint16_t)F16<DT>::down(y, 0.0f);
            } else {
              t.part[(prow + u + n) * D + dim] = y;
            }
          }
          if (++hd == t.group) {
            hd = 0;
            ++tok;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl.oempty);
        mbar_arrive(ctl.qempty + qb);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 512);
  if (threadIdx.x == 0) t.err[wid] = ctl.abort ? kLate | ctl.abort << 8 : 0;
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
std::mutex g_mu;
EncodeTiled g_encode = nullptr;
int g_sms[64] = {};

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const U4Args);
int threads_of(int n) { return n <= 32 ? Shape<16>::kThreads : Shape<80>::kThreads; }
int regs_of(int n) { return n <= 32 ? Shape<16>::kRegs : Shape<80>::kRegs; }
template <int DT>
Kernel kernel_of(int n) {
  switch (n) {
    case 16: return k_attend_u4<DT, 16>;
    case 32: return k_attend_u4<DT, 32>;
    case 48: return k_attend_u4<DT, 48>;
    case 64: return k_attend_u4<DT, 64>;
    default: return k_attend_u4<DT, 80>;
  }
}

cudaError_t device_ready(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_encode) {
    e = tensor_encoder(&g_encode);
    if (e != cudaSuccess) return e;
  }
  if (!g_sms[dev]) {
    for (int n = 16; n <= kMaxN; n += 16)
      for (Kernel k : {kernel_of<SV_BF16>(n), kernel_of<SV_F16>(n)}) {
        cudaFuncAttributes attr{};
        e = cudaFuncGetAttributes(&attr, (const void*)k);
        if (e != cudaSuccess) return e;
        if (attr.numRegs < regs_of(n)) return cudaErrorInvalidKernelImage;  // the roles' shares count on them
        e = cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
        if (e != cudaSuccess) return e;
      }
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    g_sms[dev] = n;
  }
  *sms = g_sms[dev];
  return cudaSuccess;
}

// A pool [pages][kv_heads][page_size][dim / 2] of bytes, `box` tokens at a time.
bool encode_codes(CUtensorMap* map, const CacheView& c, const void* base, int box) {
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim / 2, (cuuint64_t)c.page_size,
                              (cuuint64_t)c.kv_heads, (cuuint64_t)c.num_pages};
  // a dimension of one entry is never stepped along: any legal stride will do
  const cuuint64_t strides[3] = {(cuuint64_t)c.token_bytes,
                                 (cuuint64_t)(c.kv_heads > 1 ? c.head_bytes : c.token_bytes),
                                 (cuuint64_t)(c.num_pages > 1 ? c.page_bytes : c.token_bytes)};
  const cuuint32_t bx[4] = {(cuuint32_t)c.head_dim / 2, (cuuint32_t)box, 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle swizzle = c.head_dim == 128  ? CU_TENSOR_MAP_SWIZZLE_64B
                                     : c.head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_32B
                                                        : CU_TENSOR_MAP_SWIZZLE_NONE;
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, bx, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kRecBytes = 4096, kMlBytes = sizeof(float2) * 2 * kMaxCtas * kMaxN;
static_assert(kMaxCtas * (sizeof(Rec) + sizeof(int)) <= kRecBytes, "records");
static_assert(kMlBytes % 256 == 0, "alignment");

}  // namespace

bool u4_tiles_take(const CacheView& c, int group) {
  return c.head_dim <= 128 && c.num_pages > 0 && c.page_shift >= 4 && group <= kMaxN &&
         ((uintptr_t)c.ks | (uintptr_t)c.vs) % 16 == 0;
}

size_t attention_u4_workspace(int head_dim) {
  return kRecBytes + kMlBytes + sizeof(float) * 2 * kMaxCtas * kMaxN * (size_t)head_dim;
}

cudaError_t launch_attention_u4_tiles(const AttendArgs& a, int dtype, cudaStream_t stream, bool* taken) {
  int sms = 0;
  cudaError_t e = device_ready(&sms);
  if (e != cudaSuccess) return e;
  const CacheView& c = a.c;
  U4Args t{};
  t.a = a;
  t.group = a.heads / c.kv_heads;
  // Rows of an item: an average chunk's tokens, in as few items as hold them.
  const int most = kMaxN / t.group;  // tokens
  const int64_t chunk = a.b.B ? ((int64_t)a.b.total + a.b.B - 1) / a.b.B : 1;
  const int64_t items = chunk > most ? (chunk + most - 1) / most : 1;
  t.tpt = (int)(chunk < 1 ? 1 : (chunk + items - 1) / items);
  const int N = (t.tpt * t.group + 15) / 16 * 16;
  t.tpt = N / t.group;
  t.box = c.page_size < kTile ? c.page_size : kTile;
  t.spans = c.head_dim > 64 ? 2 : 1;
  t.stage_bytes = kTile * c.head_dim + 1024;
  const int fixed = 2 * (N > 64 ? 2 : 1) * kSpan + 2 * t.spans * N * 128 + (int)sizeof(Ctl);
  t.ring = make_ring(((int)kSmemBytes - fixed) / t.stage_bytes, kMaxStages);
  t.stall = attention_test().stall_cta;
  t.wait_clocks = attention_test().wait_clocks;
  t.c = a.scale_log2;
  t.rec = reinterpret_cast<Rec*>(a.ws);
  t.err = reinterpret_cast<int*>(a.ws + kMaxCtas * sizeof(Rec));
  t.ml = reinterpret_cast<float2*>(a.ws + kRecBytes);
  t.part = reinterpret_cast<float*>(a.ws + kRecBytes + kMlBytes);
  alignas(64) CUtensorMap mk{}, mv{};
  *taken = encode_codes(&mk, c, c.k, t.box) && encode_codes(&mv, c, c.v, t.box);
  if (!*taken) return cudaSuccess;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  e = launch_pdl(dtype == SV_BF16 ? kernel_of<SV_BF16>(N) : kernel_of<SV_F16>(N), dim3(ctas),
                 dim3(threads_of(N)), kSmemBytes, stream, mk, mv, t);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.b.total * a.heads;
  const int join_blocks = (int)(rows < 6 * ctas ? rows : 6 * ctas);
  const int flag_blocks = a.flags ? (a.b.B + kJoinThreads / 32 - 1) / (kJoinThreads / 32) : 0;
  if (join_blocks + flag_blocks == 0) return cudaSuccess;
  auto* j = dtype == SV_BF16 ? k_attend_join<U4Args, SV_BF16, false> : k_attend_join<U4Args, SV_F16, false>;
  return launch_pdl(j, dim3(join_blocks + flag_blocks), dim3(kJoinThreads), 0, stream, t, ctas, join_blocks);
}

}  // namespace sv
