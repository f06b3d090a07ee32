// sv_attention_u4.cuh -- what the kernels of spec_chunk_attention over 4-bit codes share.
//
// A code c in 0..15 is a 16-bit float by itself: the subnormal c 2^-24, or c 2^-20 four bits
// further up.  So a word of eight codes of k becomes four pairs of tensor-core operands by four
// masks and a shift, nothing is dequantised, and the powers of two go into the queries.  Codes
// of v are centred as well, (c - 8) 2^-10, by a multiply-add a pair: what a sum loses (the tensor
// cores cut its last bits) and what the weights' rounding costs go by the size of what is summed,
// and raw codes would sum up to some 7.5 times the weights, for the zeros to take off again
// (sequences of up to 40000 keys in bf16: an error of 1.78e-3 with raw codes and 1.69e-3, the
// output's own rounding, with centred ones; a window of 1000 keys in fp16: 2.4e-4 and 2.1e-4).
// The products are exact; steps and zeros act in fp32 on the scores (a row of k) and on the
// weights (a row of v, whose value at code 8, z + 8 s, stands for its zero).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "sv_attention.h"
#include "sv_attention_line.cuh"
#include "sv_cache.cuh"
#include "sv_device.cuh"
#include "sv_tma.cuh"

namespace sv {

constexpr int kMaxN = 80;              // query rows of an item, at most
constexpr int kMaxStages = 6;          // of two key tiles
// A weight p s is rounded to fp16, as an fp16 output is.  Among many keys that averages out, among a
// few it would show (22, 100, 500 keys: errors of 2.29e-4, 2.19e-4, 2.16e-4 of the values, the
// output's rounding alone 2.07e-4, 2.06e-4, 2.09e-4), so rows of fp16 outputs that see at most so
// many keys get what the rounding takes off through a second product.  It goes by the item: its
// first row sees the fewest.
constexpr int kExactKeys = 512;

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
  // An item's start and end count as so many tiles (its queries, the first maxima, sums and
  // outputs, and a join if it is cut).  3, 8, 12, 18: a window of 1000 keys 534, 442, 418, 408
  // us, long rounds 400, 391, 394, 397.
  static constexpr int kItemUnits = 12;
  static constexpr int kRowTiles = 1, kSlotRows = kMaxN;
  static __device__ __forceinline__ bool exact(int) { return false; }
  static __device__ __forceinline__ int slow_units(int, int) { return 0; }
  AttendArgs a;
  int group, tpt;      // query heads per key head; tokens per row tile
  uint32_t group_inv;  // ceil(2^16 / group): row n of an item is of token n group_inv >> 16
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
// The same of a call with fp16 outputs.  (A type of its own: the question costs prompts in bf16, where
// the answer is no, 18 of 1065 us.)
struct U4ExactArgs : U4Args {
  // Whether an item's weights are good to 2^-22 (the first of its tokens at position pos), and what
  // that costs its tiles.  (Of 0, 1/4, 1/2 and all of them: a window of 1000 keys over prompts, a
  // tenth of whose rows see few keys, 445, 420, 410, 413 us.)
  __device__ __forceinline__ bool exact(int pos) const {
    return pos < kExactKeys || (a.window && a.window <= kExactKeys);
  }
  __device__ __forceinline__ int slow_units(int pos, int count) const { return exact(pos) ? (count + 1) / 2 : 0; }
};
template <bool FP16>
using U4ArgsOf = std::conditional_t<FP16, U4ExactArgs, U4Args>;

// ---------------------------------------------------------------------------
// Primitives.
// ---------------------------------------------------------------------------
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
__device__ __forceinline__ float max3(float a, float b, float c) {  // NaNs are passed over
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 16 bytes into shared memory (zeros if not `real`), asynchronously.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
               "l"(__cvta_generic_to_global(src)), "r"(real ? 16 : 0)
               : "memory");
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
// The same as (c - 8) 2^-kDown.  (1024 + c and 64 + c, an OR each, less 1032 and 72, cost a round
// of 64 sequences 4 us more.)
constexpr int kDown = 10;
__device__ __forceinline__ uint32_t fma_halves(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ void spread_centred(uint32_t w, uint32_t* r) {
  const uint32_t v = w >> 8;
  r[0] = fma_halves(w & 0x000F000Fu, 0x74007400u, 0xA000A000u);
  r[1] = fma_halves(w & 0x00F000F0u, 0x64006400u, 0xA000A000u);
  r[2] = fma_halves(v & 0x000F000Fu, 0x74007400u, 0xA000A000u);
  r[3] = fma_halves(v & 0x00F000F0u, 0x64006400u, 0xA000A000u);
}
// What code 8 of a row stands for (0 if it has neither step nor zero).
__device__ __forceinline__ float centre_of(uint32_t sz) { return fmaf(8.0f, step_of(sz), zero_of(sz)); }

// The E of a largest step: the next power of two, 2^-100 at least (kUp over it is finite, and what
// weighs by so small a step is nothing); 0 where there is none.
__device__ __forceinline__ float step_bound(float most) {
  const float up = __uint_as_float((__float_as_uint(most) + 0x7fffffu) & 0x7f800000u);
  return up > 0.0f ? fmaxf(up, 0x1p-100f) : 0.0f;
}

// (code for what is rare goes out of the way: the warps' eight pieces of code share instruction
// caches that do not hold them all)
__device__ __forceinline__ bool rare(bool x) { return __builtin_expect(x, false); }

enum WaitId { kWaitItem = 12, kWaitSlot = 1, kWaitQ, kWaitK, kWaitV, kWaitP, kWaitQFree, kWaitS, kWaitO, kWaitCodes,
              kWaitFree };

// This thread's arrival at a barrier once all its copies so far have landed.
__device__ __forceinline__ void arrive_when_copied(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// One warp's work: the CTA's items, written down one after another (an item ahead of its tiles:
// queries take a while), and their key and value pages, two tiles to a stage of the ring.
template <class Args, class Ctl>
__device__ __forceinline__ void copy_tiles(const CUtensorMap& mk, const CUtensorMap& mv, const Args& t, Ctl& ctl,
                                           uint8_t* ring, const Guard& guard, bool ok) {
  const AttendArgs& a = t.a;
  const int lane = threadIdx.x & 31, D = a.c.head_dim, code_bytes = kTile * D / 2;
  uint32_t items = 0;
  // A copy takes the issuing warp about 53 clocks, so a stage has two tiles, and all its
  // copies are lanes of one instruction: lane 16 t + 8 v + p has part p of K (v = 0) or V of
  // tile t.  Steps and zeros come 16 bytes a lane (of a page outside the pool codes, steps
  // and zeros arrive as zeros).  The page numbers of 32 copies are read together, a batch of
  // tiles ahead.
  const uint64_t pol = l2_policy_evict_first();
  const int tile = lane >> 4, is_v = (lane >> 3) & 1, part = lane & 7;
  const int copies = kTile / t.box, batch = 32 / copies;
  const int word_part = 4 * lane / t.box;  // the copy beside this lane's steps and zeros
  const uint32_t half_bytes = (uint32_t)(t.box * (D / 2));
  uint32_t k = 0;
  if (lane == 0) ctl.walk = Walk(ctl);
  __syncwarp();
  auto write_down = [&]() {  // (an item ahead of the tiles: its queries take a while)
    Walk w = ctl.walk;
    Seg x;
    if (!w.next(t, ctl, x)) x.n = 0;
    const uint32_t i = items & 3u;
    ok = wait_held(ctl.segempty + i, ((items >> 2) & 1u) ^ 1u, guard, kWaitItem);
    if (lane == 0) {
      ctl.walk = w;
      ctl.seg[i] = x;
      mbar_arrive(ctl.segfull + i);
    }
    __syncwarp();
    ++items;
  };
  write_down();
  while (ok && ctl.seg[(items - 1) & 3u].n > 0) {
    write_down();
    const Seg& s = ctl.seg[(items - 2) & 3u];  // (stays while this warp has not come round to it)
    const int n = s.n, t0 = s.t0, lo = s.lo, hi = s.hi, h = s.h;
    const int32_t* table = a.b.table + (int64_t)s.b * a.b.max_pages;
    const int64_t head = (int64_t)h * a.c.page_size;
    auto seen = [&](int key) { return key + t.box > lo && key < hi; };
    auto look = [&](int i0) {  // pages of the tiles from i0 on
      const int i = i0 + lane / copies, key = (t0 + i) * kTile + lane % copies * t.box;
      return i < n && seen(key) ? __ldg(table + (key >> a.c.page_shift)) : -1;
    };
    int next = look(0), pages = 0, at_tile = batch;
    for (int i = 0; ok && i < n; i += 2, ++k) {
      if (at_tile == batch) {
        at_tile = 0;
        pages = next;
        if (i + batch < n) next = look(i + batch);
      }
      const Slot at(k, t.ring);
      const int first = at_tile * copies, key0 = (t0 + i) * kTile;
      at_tile += 2;
      const int key = key0 + tile * kTile + part * t.box;
      const int page = __shfl_sync(0xffffffffu, pages, (first + tile * copies + part) & 31);
      const bool mine = part < copies && i + tile < n && seen(key);
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * half_bytes;
      uint8_t* const stage = ring + (size_t)at.i * t.stage_bytes;
      ok = wait_held(ctl.empty + at.i, at.ph ^ 1u, guard, kWaitSlot);
      if (rare(!ok)) break;
      if (lane == 0) mbar_arrive_expect_tx(ctl.full + at.i, bytes);
      __syncwarp();
      if (mine)
        tma_load_4d_hint(stage + (2 * tile + is_v) * code_bytes + part * half_bytes, is_v ? &mv : &mk, 0,
                         key & (a.c.page_size - 1), h, page, ctl.full + at.i, pol);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int word_page = __shfl_sync(0xffffffffu, pages, (first + e * copies + word_part) & 31);
        const int word_key = key0 + e * kTile + 4 * lane;
        if (i + e < n && seen(word_key - (4 * lane & (t.box - 1)))) {
          const bool sound = word_page >= 0 && word_page < a.c.num_pages;
          const int64_t from =
              sound ? ((int64_t)word_page * a.c.kv_heads * a.c.page_size + head + (word_key & (a.c.page_size - 1))) * 4
                    : 0;
          uint8_t* const words = stage + 4 * code_bytes + e * 1024 + 16 * lane;
          copy16(words, a.c.ks + from, sound);
          copy16(words + 4 * kTile, a.c.vs + from, sound);
        }
      }
      arrive_when_copied(ctl.full + at.i);
    }
  }
  // every copy has landed before the CTA may exit
  __syncwarp();
  for (uint32_t i = k > t.ring.n ? k - t.ring.n : 0; i < k; ++i) {
    const Slot at(i, t.ring);
    if (lane == 0) wait_end(ctl.full + at.i, at.ph, guard);
  }
  __syncwarp();
}

// Adds up the shares of items that were cut (and raises the flags of a call that gave up).
cudaError_t launch_u4_join(const U4Args& t, int dtype, int ctas, cudaStream_t stream);
// The kernel of few rows (sv_attention_u4_few.cu).  The rows of the items that it would make of
// `rows` (fewer, where it does not take as many); the call, with all of U4Args set but what belongs
// to the kernel.
int u4_few_rows(int head_dim, int rows);
cudaError_t launch_attention_u4_few(const U4Args& call, const CUtensorMap& mk, const CUtensorMap& mv,
                                    int rows, int dtype, cudaStream_t stream);

}  // namespace sv
