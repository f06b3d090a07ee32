// sv_attention_u4_tiles.cu -- spec_chunk_attention over a cache of 4-bit codes on the tensor
// cores: tiles of 128 keys against up to 80 query rows, transposed.
//
//   k_j = z_j + s_j c_j:  t_jn = scale log2e (z_j sum(q_n) + s_j (q_n.c_j)) - m_n,
//   p = 2^t,  l_n += p,  Z_n += p (z_j + 8 s_j),  O_n += (p s_j) (c_j - 8);  out_n = (O_n + Z_n) / l_n
//
// Codes as operands: sv_attention_u4.cuh.
//
// The codes are operand A and go through tensor memory, a key (of K) or a dimension (of V)
// to a lane:  S^T [128 keys x N rows] = K Q^T,  O^T [dims x N rows] += V^T P^T.  Shared memory
// then carries the codes once (4 bits), Q, and P; and the products cost by the query rows
// that there are, not by 128.  N is 32 to 80, the rows of an item: tokens of a chunk times
// the query heads that share a key head (fewer rows: sv_attention_u4_few.cu).
//
// Work: items of one row tile, cut into equal shares of key tiles (sv_attention_line.cuh).
//
// Roles of the 20 warps: 0 finds the items and fetches their pages, 1 and 3 issue the
// products S and O, 2 converts queries, 4-7 and 8-11 spread K's and V's codes, 12-19 are two
// softmax groups.  A softmax thread has one key and N/2 rows.  The running maxima are columns:
// they are looked at again only when some score passes one by kLag (a vote of the group's
// threads), so a tile needs no reduction across lanes, and the sums stay per thread to the
// item's end.  Maxima and zeros enter S through one more product (16 deep, in bf16 parts).
//
// Measured: 32 sequences on up to 40000 keys, 9 tokens of 8 heads to a key head, 400 us (2.0 TB/s,
// 0.54 PFLOP/s); prompts of 4096 tokens 1060 us (0.56 PFLOP/s), in fp16 1140.  What bounds it:
// instructions, some 6300 a tile of 128 keys and 80 rows at 2 a clock and SM; loops are short and
// paths few because the roles' code shares the instruction caches (forty instructions more in the
// softmax's loop cost 10%).  A tile takes some 3200 clocks, its products 680.  Fewer rows an item
// are slower: prompts in items of 80, 64, 48 rows 1068, 1140, 1419 us (of raw codes).
//
// Every wait is bounded; one that gives up ends the CTA's roles and flags the call.
#include <cuda.h>
#include <cuda_runtime.h>

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
#include "sv_umma.cuh"

namespace sv {
namespace {

constexpr int kSpan = 16384;           // 128 rows of a 128-byte swizzle span
constexpr size_t kSmemBytes = 227 * 1024;
// Registers of a thread at launch, and then by role (the roles' sum must not pass what the
// launch gave, or the takers would wait forever).
constexpr int kThreads = 640, kSoft = 12;  // first softmax warp
template <int N>
struct Regs {
  static constexpr int kLaunch = 96, kHelp = N <= 64 ? 64 : 48, kSoft = N <= 64 ? 144 : 168;
  static_assert((kThreads - 256) * kHelp + 256 * kSoft <= kThreads * kLaunch, "registers");
};
// What small steps of keys are measured against, by an item's queries (small_of).
struct Small {
  float codes, step;  // steps below the one do not matter; the other is used in their place
};
struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t qfull[2], qempty[2], kfull[2], kfree[2], sfull[2], sfree[2], pvfull[2], pvfree[2];
  uint64_t ofull, oempty, fin[2], segfull[4], segempty[4];
  uint32_t tmem;
  int abort;
  int two;             // (find_share's; not used)
  int b, h, qt, off;   // start of the CTA's share (off in units)
  long long left, share;
  long long warp_units[kThreads / 32];
  float qfac[2][kMaxN];                  // of each query row: factor back to kQShift
  int odd[2];                            // some row has a factor of its own
  Small small[2];
  Seg seg[4];                            // the items, as warp 0 finds them (n = 0: no more)
  Walk walk;                             // where it is (no registers between items)
  float2 kv[4][kTile];                   // by tile: a key's factor of the product; V's step and zero
  // by softmax group (of kMaxN / 2 rows, or of all where the groups take tiles in turn):
  float m[2][kMaxN / 2];                 // maxima (-inf: nothing seen yet)
  float2 mv[2][2][kMaxN / 2];            // by S buffer: the m in its product; that of before less m
  float fac[2][kMaxN / 2];               // of a rise: old over new weights
  float wmax[2][4][kMaxN / 2], wstep[2][4];
  int rose[2];                           // some maximum rose; some row has seen nothing yet
  int unset[2];
  float2 lz[2][4][kMaxN / 2];            // sums of a warp's keys
  float4 ends[2][kMaxN / 2];              // a group's m, l, Z, E
  float4 out[kMaxN];                     // of a row: factors of the two O, what is added
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
__device__ __forceinline__ void tmem_st_rows4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
// The 128 threads of a softmax group (or the 256 of both).
__device__ __forceinline__ void group_sync(int id) {
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}
template <int THREADS = 128>
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u), "r"(id), "n"(THREADS)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void st_shared16(uint32_t addr, const uint32_t* w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}

// A key's row of codes into tensor memory (this thread's lane).
__device__ __forceinline__ void spread_row(const uint8_t* from, int D, int row, bool drop, uint32_t to) {
  const int swizzled = code_chunk(D, row, 0);
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint4 x = *reinterpret_cast<const uint4*>(from + 16 * (c ^ swizzled));
    if (drop) x = make_uint4(0, 0, 0, 0);
    uint32_t r[16];
    spread(x.x, r);
    spread(x.y, r + 4);
    spread(x.z, r + 8);
    spread(x.w, r + 12);
    tmem_st16(to + 16 * c, r);
  }
}


// Sums (or largest, NaNs passed over) over a warp's lanes of C values (a multiple of 8)
// each: lane l ends with those of C / 8 columns from first_column(l) on, in v[0..].
template <int C, bool MAX, class T>
__device__ __forceinline__ void over_lanes(T (&v)[C]) {
  static_assert(sizeof(T) == 4, "floats, or their bits");
  const int lane = threadIdx.x & 31;
  auto join = [](T a, T b) -> T {
    float x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    x = MAX ? fmaxf(x, y) : x + y;
    memcpy(&a, &x, 4);
    return a;
  };
#pragma unroll
  for (int o = 16, n = C / 2; o >= 4; o >>= 1, n >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const T keep = up ? v[n + i] : v[i], send = up ? v[i] : v[n + i];
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

// ---------------------------------------------------------------------------
// The affine part of a score as one more product, of 16 in bf16: with a key's step s and zero
// z, and a row's sum Q of queries and maximum m,
//   t = s c (q.code + (z / s) Q - m / (s c)),
// both 1 / s and z / s times a number of the row.  Each of the four numbers is a sum of three
// bf16 (24 bits), and the six largest products of their parts are taken, in this order:
//   1 / s: 1 1 2 1 2 3 0 0, m: 1 2 1 3 2 1 0 0; z / s and Q alike in the other eight.
// ---------------------------------------------------------------------------
struct Parts {
  uint32_t p1, p2, p3;  // bf16 bits
};
__device__ __forceinline__ Parts parts_of(float x) {
  Parts p;
  p.p1 = __bfloat16_as_ushort(__float2bfloat16_rn(x));
  const float r = x - __uint_as_float(p.p1 << 16);
  p.p2 = __bfloat16_as_ushort(__float2bfloat16_rn(r));
  p.p3 = __bfloat16_as_ushort(__float2bfloat16_rn(r - __uint_as_float(p.p2 << 16)));
  return p;
}
__device__ __forceinline__ uint4 key_side(const Parts& p) {
  return make_uint4(p.p1 | p.p1 << 16, p.p2 | p.p1 << 16, p.p2 | p.p3 << 16, 0);
}
__device__ __forceinline__ uint4 row_side(const Parts& p) {
  return make_uint4(p.p1 | p.p2 << 16, p.p1 | p.p3 << 16, p.p2 | p.p1 << 16, 0);
}
// The step that a key's products are in.  Codes that cannot matter are dropped: beside their zero
// (a constant row has the smallest step there is, or none), or because all of them together move
// no exponent by 2^-29 (zeros that were appended, bad pages).  Such a row has a step from its zero
// instead, or one that keeps m / (s c) in range.
//
// c: scale log2 e; top: the exponent of the largest of the query rows' factors (-1000: all rows
// are zeros).  Their elements are below 2^(9 + top), so codes move an exponent by less than
// 15 2^(16 + top) s c.  A maximum enters the product as m 2^-18 / (s c) over its row's factor, and
// comes out times that: c s = 2^(-top / 2) keeps both from the ends of the range.
__device__ __forceinline__ Small small_of(float c, int top) {
  const int e = (int)((__float_as_uint(c) >> 23) & 255u) - 127;
  return Small{pow2f(max(-120, min(100, -50 - e - top))), pow2f(max(-120, min(100, -e - top / 2)))};
}
__device__ __forceinline__ float working_step(float s, float z, const Small& small, bool& drop) {
  drop = fabsf(s) < fmaxf(fabsf(z) * 0x1p-40f, small.codes);
  return drop ? fmaxf(fabsf(z) * 0x1p-30f, small.step) : s;
}
// Where row n has its eight entries for m (half 0) or Q (half 1): rows of 32 bytes, swizzled.
__device__ __forceinline__ uint4* row_entries(uint8_t* tile, int n, int half) {
  return reinterpret_cast<uint4*>(tile + n * 32 + ((half ^ ((n >> 2) & 1)) << 4));
}
__device__ __forceinline__ uint64_t umma_desc_32(uint32_t smem_addr) {  // 32-byte swizzle
  return (uint64_t)((smem_addr >> 4) & 0x3FFFu) | (uint64_t)1 << 16 | (uint64_t)(256 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)6 << 61;
}

// Places of P, a key tile's weights each.
constexpr int p_places(bool fp16, int n) { return fp16 && n <= 32 ? 4 : 2; }

template <int DT, int N>
__global__ void __launch_bounds__(kThreads, 1)
    k_attend_u4(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                const __grid_constant__ U4ArgsOf<DT == SV_F16> t) {
  extern __shared__ __align__(1024) uint8_t smem[];
  // Few rows: the two softmax groups take tiles in turn, all rows each, with sums, maxima and O
  // of their own that the item's end adds up; a tile's fixed costs then fall on half the
  // warps.  More rows would not fit a thread's registers: the groups take half the rows each.
  constexpr bool kTurns = N <= 32;
  constexpr int C = kTurns ? N : N / 2;               // rows of a softmax group
  constexpr int kPBytes = N > 64 ? 2 * kSpan : kSpan;
  // What the rounding takes off an exact item's weights has the place of the tile before, whose
  // product is then waited for (in turns, where that is the other group's, one of its own).
  constexpr bool kExact = DT == SV_F16;
  constexpr int kRest = kTurns ? 2 : 1;  // from P's place b: b + 2, or b ^ 1
  constexpr uint32_t kColK = 72, kColV = 144, kColS = 272, kColO = 272 + 2 * N;  // tensor memory
  const AttendArgs& a = t.a;
  const int D = a.c.head_dim;
  const int q_bytes = t.spans * N * 128, code_bytes = kTile * D / 2;
  uint8_t* const pbuf = smem;
  uint8_t* const qbuf = pbuf + p_places(DT == SV_F16, N) * kPBytes;
  uint8_t* const affine = qbuf + 2 * q_bytes;  // [query tile][S buffer][N] rows of 32 bytes
  uint8_t* const ring = affine + 4 * N * 32;
  Ctl& ctl = *reinterpret_cast<Ctl*>(ring + (size_t)t.ring.n * t.stage_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wid = (int)blockIdx.x;
  const Guard guard{&ctl.abort, t.wait_clocks};

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    ctl.two = 0;
    ctl.abort = (smem_u32(smem) & 1023u) ? 1 : 0;  // the swizzles need this alignment
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(ctl.full + i, 33);
      mbar_init(ctl.empty + i, 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(ctl.qfull + i, 1);
      mbar_init(ctl.qempty + i, 1 + 8);
      mbar_init(ctl.kfull + i, 4);
      mbar_init(ctl.kfree + i, 1);
      mbar_init(ctl.sfull + i, 1);
      mbar_init(ctl.sfree + i, kTurns ? 4 : 8);
      mbar_init(ctl.pvfull + i, 4 + (kTurns ? 4 : 8));
      mbar_init(ctl.pvfree + i, 1);
      mbar_init(ctl.fin + i, 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(ctl.segfull + i, 1);
      mbar_init(ctl.segempty + i, 19);
    }
    mbar_init(&ctl.ofull, 1);
    mbar_init(&ctl.oempty, 8);
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
  bool ok = *guard.flag == 0;
  // The CTA's items, one after another: warp 0 writes them down, everybody else takes them.
  uint32_t items = 0;
  auto take = [&](Seg& s) {
    const uint32_t i = items & 3u;
    if (!wait_held(ctl.segfull + i, (items >> 2) & 1u, guard, kWaitItem)) return false;
    s = ctl.seg[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(ctl.segempty + i);
    ++items;
    return s.n > 0;
  };
  Seg s;
  if (warp < kSoft) give_regs<Regs<N>::kHelp>();

  if (warp == 0) {
    // ---------------- items, and their key and value pages ----------------
    copy_tiles(mk, mv, t, ctl, ring, guard, ok);
  } else if (warp == 1) {
    // ---------------- issue the products S ----------------
    const uint32_t leader = elect_leader();
    const uint32_t idesc_s = umma_idesc_16(false, kTile, N, false);
    const uint32_t idesc_a = umma_idesc_16(true, kTile, N, false);
    const uint32_t tb = (uint32_t)uniform((int)tbase);
    const int ksteps = D / 16;
    const uint64_t qdesc = umma_smem_desc(smem_u32(qbuf), 16, 1024);
    const uint64_t adesc = umma_desc_32(smem_u32(affine));
    uint32_t j = 0, qn = 0;  // tiles and items before
    for (; ok && take(s); ++qn) {
      const int n = uniform(s.n);
      const uint32_t qb = qn & 1u;
      const uint64_t qd = qdesc + qb * ((uint32_t)q_bytes >> 4);
      ok = wait_held(ctl.qfull + qb, (qn >> 1) & 1u, guard, kWaitQ);
      for (int i = 0; ok && i < n; ++i, ++j) {
        const uint32_t b = j & 1u, ph = (j >> 1) & 1u;
        ok = wait_held(ctl.sfree + b, ph ^ 1u, guard, kWaitS) && wait_held(ctl.kfull + b, ph, guard, kWaitK);
        if (rare(!ok)) break;
        tc_fence_after();
        const uint32_t acc = tb + kColS + b * N, ka = tb + b * kColK;
        umma_ts_if(leader, acc, ka + 64, adesc + (2 * qb + b) * (uint32_t)(N * 32 >> 4), idesc_a, false);
#pragma unroll 1
        for (int kk = 0; kk < ksteps; ++kk)
          umma_ts_if(leader, acc, ka + kk * 8, qd + (uint64_t)((kk >> 2) * (N * 128 >> 4) + (kk & 3) * 2), idesc_s, true);
        // (a test may withhold a CTA's first scores: the softmax's wait then runs out)
        umma_commit_if(t.stall == wid && j == 0 ? 0u : leader, ctl.sfull + b);
        umma_commit_if(leader, ctl.kfree + b);
        if (i == n - 1) umma_commit_if(leader, ctl.qempty + qb);
      }
    }
    // all products complete before tensor memory is released
    umma_commit_if(leader, ctl.fin);
    wait_end(ctl.fin, 0, guard);
  } else if (warp == 3) {
    // ---------------- issue the products O ----------------
    const uint32_t leader = elect_leader();
    const uint32_t idesc_o = umma_idesc_16(false, kTile, N, true);
    const uint32_t tb = (uint32_t)uniform((int)tbase);
    const uint64_t pdesc = umma_smem_desc(smem_u32(pbuf), kSpan, 1024);
    uint32_t j = 0, qn = 0;
    for (; ok && take(s); ++qn) {
      const int n = uniform(s.n);
      const bool exact = kExact && t.exact(uniform(s.pos));
      ok = wait_held(&ctl.oempty, (qn & 1u) ^ 1u, guard, kWaitO);
      for (int i = 0; ok && i < n; ++i, ++j) {
        const uint32_t b = j & 1u;
        ok = wait_held(ctl.pvfull + b, (j >> 1) & 1u, guard, kWaitP);
        if (rare(!ok)) break;
        tc_fence_after();
        const uint32_t va = tb + kColV + b * 64, acc = tb + kColO + (kTurns ? b * N : 0);
        const uint64_t pd = pdesc + b * (kPBytes >> 4);
        const bool more = i > (kTurns ? 1 : 0);
#pragma unroll 1
        for (int kk = 0; kk < 8; ++kk)
          umma_ts_if(leader, acc, va + kk * 8, pd + (uint64_t)(kk * 128), idesc_o, kk || more);
        if (kExact && exact) {
          const uint64_t rd = pdesc + (kTurns ? b + kRest : b ^ kRest) * (kPBytes >> 4);
#pragma unroll 1
          for (int kk = 0; kk < 8; ++kk)
            umma_ts_if(leader, acc, va + kk * 8, rd + (uint64_t)(kk * 128), idesc_o, true);
        }
        umma_commit_if(leader, ctl.pvfree + b);
      }
      if (ok) umma_commit_if(leader, &ctl.ofull);
    }
    umma_commit_if(leader, ctl.fin + 1);
    wait_end(ctl.fin + 1, 0, guard);
  } else if (warp == 2) {
    // ---------------- convert queries ----------------
    // Half a warp to a row, eight elements a lane, in the order of the codes' pairs:
    // 0 4 1 5 2 6 3 7.
    const int sub = lane & 15, side = lane >> 4;
    uint32_t qn = 0;
    if (lane == 0) t.rec[wid].more = 0;
    for (; ok && take(s); ++qn) {
      if (lane == 0 && s.slot == 1) t.rec[wid] = Rec{s.more, s.row0, s.ntok, s.h};
      const uint32_t qb = qn & 1u;
      ok = wait_held(ctl.qempty + qb, ((qn >> 1) & 1u) ^ 1u, guard, kWaitQFree);
      if (!ok) break;
      bool odd = false;
      int largest = -1000;
      const int rows = s.ntok * t.group;
      constexpr int kAtOnce = 4;  // rows whose loads stand together
#pragma unroll 1
      for (int base = side; base < N; base += 2 * kAtOnce) {
        uint4 x[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int n = base + 2 * j;
          x[j] = make_uint4(0, 0, 0, 0);
          if (n < rows && sub * 8 < D) {
            const int tok = (int)(n * t.group_inv >> 16), hd = n - tok * t.group;
            x[j] = __ldg(reinterpret_cast<const uint4*>(a.q + (int64_t)(s.row0 + tok) * a.q_token +
                                                        (int64_t)(s.h * t.group + hd) * a.q_head) + sub);
          }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int n = base + 2 * j;
          const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
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
          if (top > 0.0f && top < kInf) largest = max(largest, kQShift - shift);
          const float f0 = pow2f(shift), f1 = f0 * 0.0625f;
          if (sub * 8 < D && n < N) {
            uint8_t* const to =
                qbuf + qb * q_bytes + (sub >> 3) * (N * 128) + n * 128 + (((sub & 7) ^ (n & 7)) << 4);
            *reinterpret_cast<uint4*>(to) =
                make_uint4(F16<SV_F16>::down(f[0] * f0, f[4] * f0), F16<SV_F16>::down(f[1] * f1, f[5] * f1),
                           F16<SV_F16>::down(f[2] * f0, f[6] * f0), F16<SV_F16>::down(f[3] * f1, f[7] * f1));
          }
          if (sub == 0 && n < N) {
            const uint4 none = make_uint4(0, 0, 0, 0);
            const uint4 q = row_side(parts_of(sum * pow2f(shift - kQShift) * pow2f(kQShift - 24)));
            ctl.qfac[qb][n] = pow2f(kQShift - shift);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              uint8_t* const tile = affine + (2 * qb + b) * (N * 32);
              *row_entries(tile, n, 0) = none;
              *row_entries(tile, n, 1) = q;
            }
          }
        }
      }
      const bool any = __any_sync(0xffffffffu, odd);
      largest = uniform(largest);
      if (lane == 0) {
        ctl.odd[qb] = any;
        ctl.small[qb] = small_of(t.c, largest);
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(ctl.qfull + qb);
    }
  } else if (warp < kSoft) {
    // ---------------- spread codes ----------------
    // Warps 4-7 those of K, 8-11 those of V.
    const int quad = warp & 3, row = 32 * quad + lane;
    const bool is_k = warp < 8;
    constexpr float kUndo = (float)(1 << (24 - kQShift));  // the codes' and the queries' powers
    const uint32_t lanes = tbase + ((uint32_t)(32 * quad) << 16);
    uint32_t j = 0, k = 0, qn = 0;  // tiles, stages and items before
    for (; ok && take(s); ++qn) {
      if (is_k) ok = wait_held(ctl.qfull + (qn & 1u), (qn >> 1) & 1u, guard, kWaitQ);
      for (int i = 0; ok && i < s.n; ++i, ++j) {
        const Slot at(k, t.ring);
        const uint32_t b = j & 1u, ph = (j >> 1) & 1u;
        const uint8_t* const stage = ring + (size_t)at.i * t.stage_bytes;
        const uint8_t* const codes = stage + (2 * (i & 1) + (is_k ? 0 : 1)) * code_bytes;
        if (!(i & 1)) ok = wait_held(ctl.full + at.i, at.ph, guard, kWaitCodes);
        if (rare(!ok)) break;
        if (is_k) {
          // a key to a lane: pairs (i, i + 4) of each eight dimensions, and its 1 / s and z / s
          const uint32_t* const words =
              reinterpret_cast<const uint32_t*>(stage + 4 * code_bytes + (i & 1) * 1024);
          const uint32_t sz = words[row];
          bool drop;
          const float step = working_step(step_of(sz), zero_of(sz), ctl.small[qn & 1u], drop);
          const float inv = __frcp_rn(step);
          const uint4 m4 = key_side(parts_of(inv)), q4 = key_side(parts_of(zero_of(sz) * inv));
          ok = wait_held(ctl.kfree + b, ph ^ 1u, guard, kWaitFree);
          if (rare(!ok)) break;
          tc_fence_after();
          ctl.kv[j & 3u][row] = make_float2(step * t.c * kUndo, __uint_as_float(words[kTile + row]));
          const uint32_t e[8] = {m4.x, m4.y, m4.z, m4.w, q4.x, q4.y, q4.z, q4.w};
          tmem_st8(lanes + b * kColK + 64, e);
          const uint8_t* const from = codes + row * (D / 2);
          const uint32_t to = lanes + b * kColK;
          spread_row(from, D, row, drop, to);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ctl.kfull + b);
        } else {
          // a dimension to a lane, pairs of tokens: lane 8i + c of the warp's 32 takes
          // dimension 4c + i of its 32
          ok = wait_held(ctl.pvfree + b, ph ^ 1u, guard, kWaitFree);
          if (rare(!ok)) break;
          tc_fence_after();
          if (32 * quad < D) {
            const uint32_t base = smem_u32(codes) + lane * (D / 2) + 16 * code_chunk(D, lane, quad);
            const uint32_t to = lanes + kColV + b * 64;
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
              uint32_t x[4], lo[8], hi[8];
              ld_transposed4(base + m * 16 * D, x);  // (of tokens 32 m + lane)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t r[4];
                spread_centred(x[e], r);
                lo[2 * e] = r[0];
                lo[2 * e + 1] = r[1];
                hi[2 * e] = r[2];
                hi[2 * e + 1] = r[3];
              }
              tmem_st_rows4(to + 16 * m, lo);
              tmem_st_rows4(to + (16u << 16) + 16 * m, hi);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ctl.pvfull + b);
        }
        if ((i & 1) || i == s.n - 1) {
          if (lane == 0) mbar_arrive(ctl.empty + at.i);
          ++k;
        }
      }
    }
  } else {
    // ---------------- softmax and output ----------------
    take_regs<Regs<N>::kSoft>();
    const int wg = (warp - kSoft) >> 2, quad = warp & 3, row = 32 * quad + lane, id = 1 + wg;
    const int tid = row;                          // of the group's 128
    const uint32_t lanes = tbase + ((uint32_t)(32 * quad) << 16);
    const int n0 = kTurns ? 0 : wg * C;           // the group's first row
    const uint32_t o_tm = lanes + kColO + (kTurns ? wg * N : n0);
    // maxima go into the products (unless the scale is next to nothing, or so large that m / c is:
    // then all tiles take the slow way)
    const bool applies = fabsf(t.c) >= 0x1p-100f && fabsf(t.c) <= 0x1p100f;
    const float inv_c = applies ? 1.0f / t.c : 0.0f;
    // (one of the warps whose wait gave up goes on as far as the next vote, where its group
    // leaves the item, and both groups leave together: they meet at barriers without a limit)
    uint32_t g = 0, qn = 0;
    for (;; ++qn) {
      const Seg& seg = ctl.seg[items & 3u];  // (given back at the item's end)
      ok = ok && wait_held(ctl.segfull + (items & 3u), (items >> 2) & 1u, guard, kWaitItem);
      if (group_any<256>(3, !ok || seg.n == 0)) break;
      const int tiles = seg.n, tile0 = seg.t0, pos = seg.pos;
      const int rows = seg.ntok * t.group;  // live ones of the item
      // tiles [whole0, whole1) hold keys that all tokens see
      const int whole1 = (pos + 1) / kTile - tile0;
      const int whole0 = a.window ? max(0, pos + seg.ntok - 1 - a.window) / kTile + 1 - tile0 : 0;
      const uint32_t qb = qn & 1u;
      ok = wait_held(ctl.qfull + qb, (qn >> 1) & 1u, guard, kWaitQ);
      if (tid < C) {
        ctl.m[wg][tid] = -kInf;
        ctl.mv[wg][0][tid] = ctl.mv[wg][1][tid] = make_float2(0.0f, 0.0f);
      }
      bool unset = true;                    // some row has seen nothing yet
      bool stale[2] = {true, true};         // a buffer's products lack the present maxima
      const bool odd = ctl.odd[qb];
      group_sync(id);
      uint64_t l2[C / 2], z2[C / 2];
#pragma unroll
      for (int i = 0; i < C / 2; ++i) l2[i] = z2[i] = 0;
      float E = 0.0f, e_up = 0.0f;  // largest step so far, up to a power of two; kUp over it
      bool late = false;
      // (in turns a group's tiles are those of one S buffer, whose products always have the
      // present maxima in them: they change before the buffer's next one is issued)
      // Two loops: a prompt chunk in fp16, which has no exact item, takes 1085 us without the exact
      // loop, 1126 with it, and 1233 with a branch in one loop for both.
      auto all_tiles = [&](auto exact) {
        for (int i = kTurns ? (wg ^ (int)(g & 1u)) : 0; i < tiles; i += kTurns ? 2 : 1) {
          const uint32_t j = g + (uint32_t)i, b = kTurns ? (uint32_t)wg : j & 1u, ph = (j >> 1) & 1u;
          const uint32_t s_tm = lanes + kColS + b * N + n0;
          ok = wait_held(ctl.sfull + b, ph, guard, kWaitS);  // (then the tile's factors are there too)
          tc_fence_after();
          const float2 kv = ctl.kv[j & 3u][row];
          float step = step_of(__float_as_uint(kv.y)), zero = centre_of(__float_as_uint(kv.y));
          // the rows that see the key: [first, first + span) of the group's
          int first = 0, span = C;
          const bool edge = i >= whole1 || i < whole0;
          if (rare(edge)) {
            // token i sees it if key - pos <= i < key - pos + window
            const int key = (tile0 + i) * kTile + row, d = key - pos;
            const int t0 = max(0, min(d, t.tpt));
            const int t1 = a.window && d <= t.tpt - a.window ? max(0, d + a.window) : t.tpt;
            first = max(0, t0 * t.group - n0);
            span = max(0, (t1 == t.tpt ? C : min(C, t1 * t.group - n0)) - first);
            if (key < seg.lo || key >= seg.hi) span = 0;
            if (!span) step = zero = 0.0f;
          }
          const bool masked = edge && __any_sync(0xffffffffu, span < C);
          const uint64_t A2 = pack2(kv.x, kv.x);
          uint32_t r[C];
          auto load = [&]() {
            if constexpr (C % 32 == 0) {
              tmem_ld32_async(s_tm, r);
            } else if constexpr (C % 16 == 0) {
              tmem_ld16_async(s_tm, r);
            } else {
#pragma unroll
              for (int u = 0; u < C; u += 8) tmem_ld8_async(s_tm + u, r + u);
            }
            tmem_wait_ld();
            if (rare(odd)) {
#pragma unroll
              for (int n = 0; n < C; ++n)
                r[n] = __float_as_uint(__uint_as_float(r[n]) * ctl.qfac[qb][n0 + n]);
            }
          };
          auto hide = [&]() {
            if (rare(masked)) {
#pragma unroll
              for (int n = 0; n < C; ++n)
                if ((unsigned)(n - first) >= (unsigned)span) r[n] = 0xff800000u;
            }
          };
          load();
          bool slow = unset || (!kTurns && (b ? stale[1] : stale[0]));  // (the same for the group)
          if (!slow) {
#pragma unroll
            for (int n = 0; n < C; n += 2) {
              float x, y;
              unpack2(fmul2(pack2(__uint_as_float(r[n]), __uint_as_float(r[n + 1])), A2), x, y);
              r[n] = __float_as_uint(x);
              r[n + 1] = __float_as_uint(y);
            }
            hide();
            float top = __uint_as_float(r[0]), top2 = __uint_as_float(r[1]);
#pragma unroll
            for (int n = 2; n < C; n += 4) {
              top = max3(top, __uint_as_float(r[n]), __uint_as_float(r[n + 1]));
              if (n + 2 < C) top2 = max3(top2, __uint_as_float(r[n + 2]), __uint_as_float(r[n + 3]));
            }
            // (a step or zero that is not finite takes the slow way too)
            slow = group_any(id, fmaxf(top, top2) > kLag || !(fabsf(fmaf(zero, 0.0f, step)) <= E) || !ok);
            if (rare(slow)) load();
          }
          if (rare(slow)) {
            // a maximum rises, or the largest step, or the product was issued with older maxima
            if (group_any(id, !ok)) {
              late = true;
              break;
            }
            // scores, maxima taken off from column `off` of mv
            auto scores = [&](int off) {
#pragma unroll
              for (int n = 0; n < C; n += 2) {
                const float* k = reinterpret_cast<const float*>(ctl.mv[wg][b] + n) + off;
                float x, y;
                unpack2(ffma2(pack2(__uint_as_float(r[n]), __uint_as_float(r[n + 1])), A2, pack2(k[0], k[2])), x, y);
                r[n] = __float_as_uint(x);
                r[n + 1] = __float_as_uint(y);
              }
              hide();
            };
            scores(0);
            over_lanes<C, true>(r);
            if ((lane & 3) == 0)
#pragma unroll
              for (int n = 0; n < C / 8; ++n)
                ctl.wmax[wg][quad][first_column<C>(lane) + n] = __uint_as_float(r[n]);
            const bool bad = !(fabsf(fmaf(zero, 0.0f, step)) < kInf);
            const float ws = warp_max(bad ? 0.0f : fabsf(step));
            if (lane == 0) ctl.wstep[wg][quad] = ws;
            if (tid == 0) ctl.rose[wg] = ctl.unset[wg] = 0;
            group_sync(id);
            if (tid < C) {
              float most = -kInf;
#pragma unroll
              for (int w = 0; w < 4; ++w) most = fmaxf(most, ctl.wmax[wg][w][tid]);
              const float was = ctl.m[wg][tid], now = most > was + kLag ? most : was;
              ctl.m[wg][tid] = now;
              ctl.fac[wg][tid] = now > was ? ex2(was - now) : 1.0f;
              if (now > was) ctl.rose[wg] = 1;
              const bool none = now == -kInf;
              if (none && n0 + tid < rows) ctl.unset[wg] = 1;
              // the buffer's next product (two tiles on) has the present maximum in it
              const float m = none ? 0.0f : now, in = applies && fabsf(m) < kInf ? m : 0.0f;
              // (and this one: with the maximum that it was issued with, less the present one)
              ctl.mv[wg][b][tid] = make_float2(in, ctl.mv[wg][b][tid].x - m);
              *row_entries(affine + (2 * qb + b) * (N * 32), n0 + tid, 0) =
                  row_side(parts_of(-in * inv_c * (pow2f(kQShift - 24) / ctl.qfac[qb][n0 + tid])));
            }
            float most = 0.0f;
#pragma unroll
            for (int w = 0; w < 4; ++w) most = fmaxf(most, ctl.wstep[wg][w]);
            const float e_now = fmaxf(E, step_bound(most));
            const float fe = E < e_now ? E * (1.0f / e_now) : 1.0f;
            group_sync(id);
            const bool rose = ctl.rose[wg] != 0;
            unset = ctl.unset[wg] != 0 || (kTurns && !applies);
            stale[0] = b ? stale[0] || rose || !applies : !applies;
            stale[1] = b ? !applies : stale[1] || rose || !applies;
            const bool opened = kTurns ? i > 1 : i > 0;  // O holds something of the item
            if (opened && (rose || fe != 1.0f)) {
#pragma unroll
              for (int n = 0; n < C; n += 2) {
                const float2 f = *reinterpret_cast<const float2*>(ctl.fac[wg] + n);
                l2[n / 2] = fmul2(l2[n / 2], pack2(f.x, f.y));
                z2[n / 2] = fmul2(z2[n / 2], pack2(f.x, f.y));
              }
              // O: its last product is done (in turns that of two tiles ago)
              ok = kTurns ? wait_held(ctl.pvfree + b, ph ^ 1u, guard, kWaitFree)
                          : wait_held(ctl.pvfree + (b ^ 1u), ((j - 1) >> 1) & 1u, guard, kWaitFree);
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
              e_up = kUp / e_now;
            }
            if (__any_sync(0xffffffffu, bad)) {
              // a value row that is not finite weighs nothing (0 times it would not be 0 where
              // it is not seen); the rows that do see it get their NaN here
              const float nan = bad ? __int_as_float(0x7fffffff) : 0.0f;
#pragma unroll
              for (int n = 0; n < C; n += 2)
                z2[n / 2] = fadd2(z2[n / 2], pack2((unsigned)(n - first) < (unsigned)span ? nan : 0.0f,
                                                   (unsigned)(n + 1 - first) < (unsigned)span ? nan : 0.0f));
              if (bad) step = zero = 0.0f;
            }
            load();
            scores(1);
            group_sync(id);  // (mv and the maxima's votes are written again by the next slow tile)
          }
          // S has been read, and the next product in its place has the present maxima to take
          fence_proxy_async();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ctl.sfree + b);
          // weights, into P's place of two tiles ago
          ok = wait_held(ctl.pvfree + b, ph ^ 1u, guard, kWaitFree);
          if (exact && !kTurns)
            ok = wait_held(ctl.pvfree + (b ^ 1u), ((j - 1) >> 1) & 1u, guard, kWaitFree) && ok;
          const float up = step * e_up;
          const uint64_t up2 = pack2(up, up), zero2 = pack2(zero, zero);
          const uint32_t prow = smem_u32(pbuf + b * kPBytes + row * 128) | ((row & 7) << 4);
          // where what the rounding takes off goes, from there
          const uint32_t rest = ((kTurns ? b + kRest : b ^ kRest) - b) * kPBytes;
#pragma unroll
          for (int u = 0; u < C; u += 8) {
            uint32_t w[4], v[4];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const int n = u + e;
              const uint64_t p = pack2(ex2(__uint_as_float(r[n])), ex2(__uint_as_float(r[n + 1])));
              l2[n / 2] = fadd2(l2[n / 2], p);
              z2[n / 2] = ffma2(p, zero2, z2[n / 2]);
              float x, y;
              unpack2(fmul2(p, up2), x, y);
              w[e / 2] = F16<SV_F16>::down(x, y);
              if constexpr (exact) {
                const float2 had = F16<SV_F16>::up(w[e / 2]);
                v[e / 2] = F16<SV_F16>::down(x - had.x, y - had.y);
              }
            }
            const int ch = (n0 + u) >> 3;
            const uint32_t to = (prow ^ ((ch & 7) << 4)) + (ch >> 3) * kSpan;
            st_shared16(to, w);
            if constexpr (exact) st_shared16(to + rest, v);
          }
          fence_proxy_async();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ctl.pvfull + b);
        }
      };
      if constexpr (kExact) {
        if (rare(t.exact(pos))) all_tiles(std::true_type{});
        else all_tiles(std::false_type{});
      } else {
        all_tiles(std::false_type{});
      }
      g += (uint32_t)tiles;
      // ---- the item's end: sums over the keys, then O ----
      auto sum_up = [&](uint64_t (&x2)[C / 2], int which) {
        float v[C];
#pragma unroll
        for (int n = 0; n < C; n += 2) unpack2(x2[n / 2], v[n], v[n + 1]);
        over_lanes<C, false>(v);
        if ((lane & 3) == 0)
#pragma unroll
          for (int n = 0; n < C / 8; ++n)
            reinterpret_cast<float*>(ctl.lz[wg][quad] + first_column<C>(lane) + n)[which] = v[n];
      };
      sum_up(l2, 0);
      sum_up(z2, 1);
      group_sync(id);
      if (tid < C) {
        float L = 0.0f, Z = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 x = ctl.lz[wg][w][tid];
          L += x.x;
          Z += x.y;
        }
        ctl.ends[wg][tid] = make_float4(ctl.m[wg][tid], L, Z, E);
      }
      if (group_any<256>(3, late)) break;
      // half the rows' outputs each
      constexpr int kOut = N / 2;
      const int r0 = wg * kOut;
      const int64_t prow = (int64_t)(2 * wid + (seg.slot > 0 ? 1 : 0)) * kMaxN;
      if (tid < kOut) {
        const int n = r0 + tid;
        const float4 x = ctl.ends[kTurns ? 0 : wg][kTurns ? n : tid];
        float m = x.x, L = x.y, Z = x.z, f0 = x.w, f1 = 0.0f;
        if (kTurns) {
          const float4 y = ctl.ends[1][n];
          m = fmaxf(x.x, y.x);
          // (a group that saw nothing: l is 0, and its O was never written)
          const float a0 = x.y == 0.0f ? 0.0f : ex2(x.x - m), a1 = y.y == 0.0f ? 0.0f : ex2(y.x - m);
          L = (x.y == 0.0f ? 0.0f : a0 * x.y) + (y.y == 0.0f ? 0.0f : a1 * y.y);
          Z = (x.y == 0.0f ? 0.0f : a0 * x.z) + (y.y == 0.0f ? 0.0f : a1 * y.z);
          f0 = a0 * x.w;
          f1 = a1 * y.w;
        }
        const float inv = seg.slot >= 0 ? 1.0f : L == 0.0f ? 0.0f : 1.0f / L;
        ctl.out[n] = make_float4(f0 * inv * (pow2f(kDown) / kUp), f1 * inv * (pow2f(kDown) / kUp), L == 0.0f ? 0.0f : Z * inv, 0.0f);
        if (n < rows) {
          if (seg.slot >= 0) {
            t.ml[prow + n] = make_float2(m, L);
          } else if (a.lse) {
            const int tok = (int)(n * t.group_inv >> 16), hd = n - tok * t.group;
            a.lse[(int64_t)(seg.row0 + tok) * a.heads + seg.h * t.group + hd] = lse_of(m, L);
          }
        }
      }
      group_sync(id);
      ok = wait_held(&ctl.ofull, qn & 1u, guard, kWaitO);
      tc_fence_after();
      // lane 8i + c of the warp's 32 has dimension 4c + i
      const int dim = 32 * quad + 4 * (lane & 7) + (lane >> 3);
      // Outputs go by way of shared memory (P's place: the item's last product is done, and both
      // groups meet before the next one's first), so that the stores are 16 bytes of a row: two
      // bytes at a time an item's 80 rows took 6000 clocks.
      const int pitch = 2 * D + 16;
      uint8_t* const staged = pbuf + wg * (kOut * (2 * 128 + 16));
      const bool whole = seg.slot < 0;
      float* const part = t.part + (prow + r0) * D + dim;
#pragma unroll 1
      for (int u = 0; u < kOut; u += 8) {
        uint32_t o[8], q[8];
        __syncwarp();
        tmem_ld8_async(lanes + kColO + r0 + u, o);
        if (kTurns) tmem_ld8_async(lanes + kColO + N + r0 + u, q);
        tmem_wait_ld();
        if (32 * quad >= D) continue;
        float y[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float4 f = ctl.out[r0 + u + n];
          // (an O without weights is not read: it may hold anything)
          y[n] = f.z;
          if (f.x != 0.0f) y[n] = fmaf(__uint_as_float(o[n]), f.x, y[n]);
          if (kTurns && f.y != 0.0f) y[n] = fmaf(__uint_as_float(q[n]), f.y, y[n]);
        }
        if (whole) {
#pragma unroll
          for (int n = 0; n < 8; ++n)
            *reinterpret_cast<uint16_t*>(staged + (u + n) * pitch + 2 * dim) =
                (uint16_t)F16<DT>::down(y[n], 0.0f);
        } else {
#pragma unroll
          for (int n = 0; n < 8; ++n)
            if (r0 + u + n < rows) part[(u + n) * D] = y[n];
        }
      }
      if (whole) {
        group_sync(id);
        for (int n = r0 + (tid >> 4); n < min(r0 + kOut, rows); n += 8) {
          const int ch = tid & 15, tok = (int)(n * t.group_inv >> 16), hd = n - tok * t.group;
          if (8 * ch < D)
            reinterpret_cast<uint4*>(a.out + ((int64_t)(seg.row0 + tok) * a.heads + seg.h * t.group + hd) * D * 2)[ch] =
                *reinterpret_cast<const uint4*>(staged + (n - r0) * pitch + 16 * ch);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&ctl.oempty);
        mbar_arrive(ctl.qempty + qb);
        mbar_arrive(ctl.segempty + (items & 3u));
      }
      ++items;
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

// f of the kernel for items of up to n rows.
template <int DT, class Fn>
cudaError_t with_kernel(int n, Fn f) {
  switch (n) {
    case 32: return f(k_attend_u4<DT, 32>);
    case 48: return f(k_attend_u4<DT, 48>);
    case 64: return f(k_attend_u4<DT, 64>);
    default: return f(k_attend_u4<DT, 80>);
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
    auto ready = [](auto* k) {
      cudaFuncAttributes attr{};
      const cudaError_t e = cudaFuncGetAttributes(&attr, (const void*)k);
      if (e != cudaSuccess) return e;
      if (attr.numRegs < Regs<32>::kLaunch) return cudaErrorInvalidKernelImage;  // the roles' shares count on them
      return cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    };
    for (int n = 32; n <= kMaxN; n += 16) {
      e = with_kernel<SV_BF16>(n, ready);
      if (e == cudaSuccess) e = with_kernel<SV_F16>(n, ready);
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
  // Rows of one head that lie apart (token-major pages): what L2 fetches beside them is other
  // heads', and gone again before those are read (rows of 64 bytes, 512 apart: 10.5 bytes a
  // clock and SM with 256-byte fetches, 22.7 with 64).
  const CUtensorMapL2promotion promotion = c.token_bytes == c.head_dim / 2
                                               ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                               : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, bx, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
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
  t.group_inv = (uint32_t)((65536 + t.group - 1) / t.group);
  t.c = a.scale_log2;
  t.rec = reinterpret_cast<Rec*>(a.ws);
  t.err = reinterpret_cast<int*>(a.ws + kMaxCtas * sizeof(Rec));
  t.ml = reinterpret_cast<float2*>(a.ws + kRecBytes);
  t.part = reinterpret_cast<float*>(a.ws + kRecBytes + kMlBytes);
  t.box = c.page_size < kTile ? c.page_size : kTile;
  t.stage_bytes = 2 * (kTile * c.head_dim + 1024);
  t.stall = attention_test().stall_cta;
  t.wait_clocks = attention_test().wait_clocks;
  alignas(64) CUtensorMap mk{}, mv{};
  *taken = encode_codes(&mk, c, c.k, t.box) && encode_codes(&mv, c, c.v, t.box);
  if (!*taken) return cudaSuccess;
  const int rows = t.tpt * t.group;
  // Keys of an item, at most.  (The lengths are on the device: without a window the table's width
  // counts, not what of it is used.)
  const int64_t held = (int64_t)a.b.max_pages * c.page_size;
  const int64_t keys = a.window && a.window < held - t.tpt ? a.window + t.tpt : held;
  // Up to the rows of its items the kernel of few rows takes a call.  More rows are several items
  // there, whose starts and ends cost it less than they cost this kernel: with narrow heads, items
  // nearly full and few keys it is ahead for many rows too.  us there and here, prompts of up to
  // 2001 tokens in a window, groups of 5 heads:
  //   window     1000        2000        2600        3300        4500
  //   32 wide  295  430    458  527    538  564    608  586    698  625
  //   64 wide  371  430    491  533    541  574    590  592    661  631
  //   96 wide  402  431    527  524    616  565    694  595    791  633
  // and tables of 2000, 3300, 4500 keys as wide as the prompts are long: 32 wide 484 603, 1007 1062,
  // 2002 1898; 96 wide 587 640, 1152 1144, 2279 1935; 64 wide ahead throughout.  By an item's rows,
  // window of 1000: 96 wide, of 32 rows 27 (235 and 244) and 24 (340 and 318), 17 (659 and 448); 64
  // wide, of 48 rows 42 (162 and 180), 40 (851 and 807), 34 (435 and 419), 32 (844 and 715); 32 wide, of
  // 32 rows 24 (242 and 305), 17 (469 and 427).  128 wide: 543 and 413.
  const int fit = u4_few_rows(c.head_dim, rows), live = fit / t.group * t.group;
  const bool few_keys = c.head_dim == 32   ? keys <= 25 * kTile && live >= 24
                        : c.head_dim == 64 ? keys <= 32 * kTile && live >= 41
                                           : c.head_dim == 96 && keys <= 16 * kTile && live >= 26;
  if (rows <= fit || few_keys)
    return launch_attention_u4_few(t, mk, mv, rows, dtype, stream);
  const int N = (t.tpt * t.group + 15) / 16 * 16;
  t.tpt = N / t.group;
  t.spans = c.head_dim > 64 ? 2 : 1;
  const int fixed = p_places(dtype == SV_F16, N) * (N > 64 ? 2 : 1) * kSpan + 2 * t.spans * N * 128 +
                    4 * N * 32 + (int)sizeof(Ctl);
  t.ring = make_ring(((int)kSmemBytes - fixed) / t.stage_bytes, kMaxStages);
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  auto launch = [&](auto* k, auto args) {
    return launch_pdl(k, dim3(ctas), dim3(kThreads), kSmemBytes, stream, mk, mv, args);
  };
  e = dtype == SV_BF16 ? with_kernel<SV_BF16>(N, [&](auto* k) { return launch(k, t); })
                       : with_kernel<SV_F16>(N, [&](auto* k) { return launch(k, U4ExactArgs{t}); });
  return e == cudaSuccess ? launch_u4_join(t, dtype, ctas, stream) : e;
}

cudaError_t launch_u4_join(const U4Args& t, int dtype, int ctas, cudaStream_t stream) {
  const AttendArgs& a = t.a;
  const int64_t rows = (int64_t)a.b.total * a.heads;
  const int join_blocks = (int)(rows < 6 * ctas ? rows : 6 * ctas);
  const int flag_blocks = a.flags ? (a.b.B + kJoinThreads / 32 - 1) / (kJoinThreads / 32) : 0;
  if (join_blocks + flag_blocks == 0) return cudaSuccess;
  auto* j = dtype == SV_BF16 ? k_attend_join<U4Args, SV_BF16, false> : k_attend_join<U4Args, SV_F16, false>;
  return launch_pdl(j, dim3(join_blocks + flag_blocks), dim3(kJoinThreads), 0, stream, t, ctas, join_blocks);
}

}  // namespace sv
