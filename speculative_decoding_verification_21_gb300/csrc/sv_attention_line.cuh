// sv_attention_line.cuh -- what the tile kernels of spec_chunk_attention share: the line of
// work and its shares, bounded waits, rings of tiles, the join of cut items.
//
// Balance: all key tiles of all items form one line, an item's start worth some
// tiles more (start_units), cut into equal shares, one per CTA (one CTA per SM).  An
// item cut by a share's end leaves partial (m, l, O) in the workspace, at most two per
// CTA, which k_attend_join adds up; an item inside a share is written at once.  Lengths
// live on the device, so every CTA finds its own place in the line at its start.
//
// Args, a kernel's arguments, has: a (AttendArgs), group, tpt (tokens of a row tile), ml,
// part, rec, err (workspace), kRowTiles (row tiles of an item), kSlotRows (rows of a partial
// slot), kItemUnits and slow_units(pos, count): what an item costs beside its `count` tiles, any
// item and one whose first token is at position pos, in tiles.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "specverify.h"
#include "sv_attention.h"
#include "sv_cache.cuh"
#include "sv_device.cuh"
#include "sv_tma.cuh"
#include "sv_umma.cuh"

namespace sv {

constexpr int kTile = 128;          // keys per tile
constexpr int kMaxCtas = 160;       // shares (GB300: 152 SMs)
constexpr int kJoinThreads = 256;

// A CTA's err word: a wait gave up; a row that it wrote holds something that is not finite.
constexpr int kLate = 1, kMend = 2;

// Slots of a ring, and ceil(2^32 / slots): slot and turn of tile k without a division.
struct Ring {
  uint32_t n, inv;
};

// What a CTA leaves for the join: the item that it began and did not end.
struct Rec {
  int more;            // further CTAs with a part of it (0: nothing to join)
  int row0, ntok, h;   // first packed row, tokens, key head
};

// ---------------------------------------------------------------------------
// The line of work.
// ---------------------------------------------------------------------------
struct Span {
  int lo, hi;        // keys [lo, hi) that some row of the item sees
  int first, count;  // key tiles; count >= 1 (a masked one if nothing is seen)
};

__device__ __forceinline__ Span item_span(const Seq& q, int per_item, int qt, int window) {
  const int i0 = qt * per_item, i1 = min(q.n, i0 + per_item);
  Span s;
  const int seen = q.pos0 + i0 + 1;  // keys up to the first row's own; negative in front of token 0
  s.hi = max(0, q.pos0 + i1);
  s.lo = window && seen > window ? seen - window : 0;
  if (s.hi <= s.lo) {
    s.lo = s.hi = s.first = 0;
    s.count = 1;
  } else {
    s.first = s.lo / kTile;
    s.count = (s.hi + kTile - 1) / kTile - s.first;
  }
  return s;
}

__device__ __forceinline__ long long warp_sum64(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ long long warp_scan64(long long v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// Units of an item's start, and of all of it.
template <class Args>
__device__ __forceinline__ int start_units(const Args& t, const Seq& q, int per_item, int qt, int count) {
  return Args::kItemUnits + t.slow_units(q.pos0 + qt * per_item, count);
}
template <class Args>
__device__ __forceinline__ int item_units(const Args& t, const Seq& q, int per_item, int qt) {
  const int count = item_span(q, per_item, qt, t.a.window).count;
  return start_units(t, q, per_item, qt, count) + count;
}

// Units of one head of the lane's sequence (n = 0: none).  A sequence of many
// items is summed by the whole warp.
template <class Args>
__device__ __forceinline__ long long head_units(const Args& args, const Seq& q, int per_item) {
  const int lane = threadIdx.x & 31;
  const int nqt = (q.n + per_item - 1) / per_item;
  long long u = 0;
  if (nqt <= 4)
    for (int t = 0; t < nqt; ++t) u += item_units(args, q, per_item, t);
  unsigned big = __ballot_sync(0xffffffffu, nqt > 4);
  while (big) {
    const int src = __ffs(big) - 1;
    big &= big - 1;
    Seq s{};
    s.n = __shfl_sync(0xffffffffu, q.n, src);
    s.pos0 = __shfl_sync(0xffffffffu, q.pos0, src);
    long long v = 0;
    const int m = (s.n + per_item - 1) / per_item;
    for (int t = lane; t < m; t += 32) v += item_units(args, s, per_item, t);
    v = warp_sum64(v);
    if (lane == src) u = v;
  }
  return u;
}

// a / b and a % b of non-negative numbers, in 32 bits where they fit (a 64-bit division
// is a long subroutine).
__device__ __forceinline__ long long divide(long long a, long long b, long long& rest) {
  if (((a | b) >> 32) == 0) {
    const uint32_t q = (uint32_t)a / (uint32_t)b;
    rest = (uint32_t)a - q * (uint32_t)b;
    return q;
  }
  const long long q = a / b;
  rest = a - q * b;
  return q;
}

// The start of this CTA's share (all threads; ends with a barrier).  Each warp looks
// at its stretch of the sequences, 32 at a time.
template <class Args, class Ctl>
__device__ void find_share(const Args& t, Ctl& ctl) {
  const BatchView& bv = t.a.b;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (int)(blockDim.x >> 5);
  const int per_item = t.tpt * Args::kRowTiles, H = t.a.c.kv_heads, ps = t.a.c.page_size;
  const int chunk = (bv.B + nw - 1) / nw;
  const int b0 = min(bv.B, warp * chunk), b1 = min(bv.B, b0 + chunk);
  Seq q{};
  long long per_head = 0, sum = 0;
  auto look = [&](int base) {
    q = Seq{};
    if (base + lane < b1) q = load_seq(bv, base + lane, ps);
    per_head = head_units(t, q, per_item);
  };
  for (int base = b0; base < b1; base += 32) {
    look(base);
    sum += warp_sum64(per_head * H);
    if (q.n > t.tpt) ctl.two = 1;
  }
  if (lane == 0) ctl.warp_units[warp] = sum;
  if (threadIdx.x == 0) {
    ctl.left = 0;
    ctl.b = bv.B;
    ctl.h = ctl.qt = ctl.off = 0;
  }
  __syncthreads();
  // the units of the warps before this one, and of all
  const long long mine = lane < nw ? ctl.warp_units[lane] : 0;
  const long long total = warp_sum64(mine);
  long long before = __shfl_sync(0xffffffffu, warp_scan64(mine) - mine, warp);
  long long rest;
  const long long share = max(1ll, divide(total + gridDim.x - 1, (long long)gridDim.x, rest));
  const long long start = share * blockIdx.x;
  if (start >= before && start < before + sum) {  // this warp's sequences hold the start
    for (int base = b0; base < b1; base += 32) {
      if (b1 - b0 > 32) look(base);  // (else they are still here)
      const long long scan = warp_scan64(per_head * H);
      const unsigned hit = __ballot_sync(0xffffffffu, start < before + scan);
      if (!hit) {
        before += __shfl_sync(0xffffffffu, scan, 31);
        continue;
      }
      const int src = __ffs(hit) - 1;
      Seq s{};
      s.n = __shfl_sync(0xffffffffu, q.n, src);
      s.pos0 = __shfl_sync(0xffffffffu, q.pos0, src);
      const long long ph = __shfl_sync(0xffffffffu, per_head, src);
      long long r = start - before - __shfl_sync(0xffffffffu, scan - per_head * H, src);
      const int h = (int)divide(r, ph, r);
      const int m = (s.n + per_item - 1) / per_item;
      for (int q0 = 0; q0 < m; q0 += 32) {
        const long long c = q0 + lane < m ? item_units(t, s, per_item, q0 + lane) : 0;
        const long long sc = warp_scan64(c);
        const unsigned in = __ballot_sync(0xffffffffu, r < sc);
        if (!in) {
          r -= __shfl_sync(0xffffffffu, sc, 31);
          continue;
        }
        const int l = __ffs(in) - 1;
        const long long off = r - __shfl_sync(0xffffffffu, sc - c, l);
        if (lane == 0) {
          ctl.b = base + src;
          ctl.h = h;
          ctl.qt = q0 + l;
          ctl.off = (int)off;
          ctl.left = min(share, total - start);
        }
        break;
      }
      break;
    }
  }
  if (threadIdx.x == 0) ctl.share = share;
  __syncthreads();
}

// One CTA's part of one item.
struct Seg {
  int b, h;
  int row0, ntok;    // first packed row, tokens
  int pos;           // position of the first token
  int lo, hi;
  int t0, n;         // key tiles t0 .. t0+n-1
  bool two;          // two row tiles
  int slot;          // -1: the whole item; else the partial slot of the CTA (0, 1)
  int more;          // slot 1: further CTAs with a part of it
};

struct Walk {
  int b, h, qt, off, nqt;
  long long left;
  Seq q;
  bool loaded;

  template <class Ctl>
  __device__ __forceinline__ Walk(const Ctl& c)
      : b(c.b), h(c.h), qt(c.qt), off(c.off), nqt(0), left(c.left), loaded(false) {}

  template <class Args, class Ctl>
  __device__ __forceinline__ bool next(const Args& t, const Ctl& ctl, Seg& s) {
    if (left <= 0) return false;
    const int per_item = t.tpt * Args::kRowTiles;
    while (!loaded) {
      if (b >= t.a.b.B) return false;
      q = load_seq(t.a.b, b, t.a.c.page_size);
      nqt = (q.n + per_item - 1) / per_item;
      if (nqt) loaded = true;
      else ++b;
    }
    const Span sp = item_span(q, per_item, qt, t.a.window);
    // units off .. off + take of the item: its start, then a unit a tile
    const int start = start_units(t, q, per_item, qt, sp.count), avail = sp.count + start - off;
    const int take = (int)min((long long)avail, left);
    const int t0 = max(0, off - start), t1 = off + take - start;
    left -= take;
    if (t1 <= t0) return false;  // the share ends in front of the item's first tile
    s.b = b;
    s.h = h;
    s.row0 = q.tok0 + qt * per_item;
    s.ntok = min(per_item, q.n - qt * per_item);
    s.pos = q.pos0 + qt * per_item;
    s.lo = sp.lo;
    s.hi = sp.hi;
    s.t0 = sp.first + t0;
    s.n = t1 - t0;
    s.two = s.ntok > t.tpt;
    s.slot = s.n == sp.count ? -1 : (t0 ? 0 : 1);
    s.more = s.slot == 1 ? (int)((avail - take + ctl.share - 1) / ctl.share) : 0;
    off = 0;
    if (++qt == nqt) {
      qt = 0;
      if (++h == t.a.c.kv_heads) {
        h = 0;
        ++b;
        loaded = false;
      }
    }
    return true;
  }
};

// Slot and phase of the k-th tile of a ring (k < 2^32 / 12).
struct Slot {
  uint32_t i, ph;
  __device__ __forceinline__ Slot(uint32_t k, const Ring& r) {
    const uint32_t turn = __umulhi(k, r.inv);
    i = k - turn * r.n;
    ph = turn & 1u;
  }
};

// A value that is the same in all lanes, in a form that the compiler knows to be.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

// ---------------------------------------------------------------------------
// Waits.
// ---------------------------------------------------------------------------
// A whole warp.  All lanes test and go on together: one that went ahead could let
// the barrier move a phase further before another tests it.
struct Guard {
  volatile int* flag;  // the CTA's abort flag
  long long clocks;    // limit of a wait
};
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Guard& guard, int id) {
  for (int i = 0; i < 64; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  for (;;) {
    for (int i = 0; i < 16; ++i)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const bool late = clock64() - t0 >= guard.clocks;
    if (__any_sync(0xffffffffu, late)) *guard.flag = id;
    if (__any_sync(0xffffffffu, late || *guard.flag != 0)) return false;
  }
}
// The same in a shorter form, for a kernel of many roles (a try holds the warp for some 8000
// clocks before it gives up, so the loop goes round rarely).
__device__ __forceinline__ bool wait_held(uint64_t* bar, uint32_t parity, const Guard& guard, int id) {
  if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar, parity)), true)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    const bool late = clock64() - t0 >= guard.clocks;
    if (__any_sync(0xffffffffu, late)) *guard.flag = id;
    if (__any_sync(0xffffffffu, late || *guard.flag != 0)) return false;
  }
}
// What must have ended before the CTA may go, whether or not the call is aborted.
__device__ __forceinline__ void wait_end(uint64_t* bar, uint32_t parity, const Guard& guard) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity) && clock64() - t0 < guard.clocks) {
  }
}

__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.0f ? -kInf : ((m == -kInf ? 0.0f : m) + log2f(l)) * kLn2;
}

template <int REGS>
__device__ __forceinline__ void take_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void give_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// ---------------------------------------------------------------------------
// The join: items cut by a share's end, and the flags.
// ---------------------------------------------------------------------------
// One row from its parts (at most one per CTA).  The (m, l) of all parts are read at
// once, a part per lane; the warp then adds up every `stride`-th part's O from `first`
// on, 32 lanes by four columns.  Returns this lane's columns; M, L: of all parts.
template <class Args>
__device__ __forceinline__ float4 join_parts(const Args& t, int c, int parts, int row, int first,
                                             int stride, float& M, float& L) {
  constexpr int kSets = (kMaxCtas + 31) / 32;
  const int lane = threadIdx.x & 31, D = t.a.c.head_dim;
  auto place = [&](int p) { return (int64_t)(p ? 2 * (c + p) : 2 * c + 1) * Args::kSlotRows + row; };
  float2 ml[kSets];
  M = -kInf;
#pragma unroll
  for (int k = 0; k < kSets; ++k) {
    ml[k] = make_float2(-kInf, 0.0f);
    if (32 * k + lane < parts) ml[k] = __ldcg(t.ml + place(32 * k + lane));
    M = fmaxf(M, ml[k].x);
  }
  M = warp_max(M);
  if (M == -kInf) M = 0.0f;
  L = 0.0f;
  float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
  for (int k = 0; k < kSets; ++k) {
    if (32 * k >= parts) break;
    // (a part that sees nothing has l = 0, and its O was never written)
    const float f = ml[k].y == 0.0f ? 0.0f : ex2(ml[k].x - M);
    float l = ml[k].y == 0.0f ? 0.0f : f * ml[k].y;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    L += l;
    const unsigned seen = __ballot_sync(0xffffffffu, ml[k].y != 0.0f);
    const int last = min(32, parts - 32 * k);
#pragma unroll 8
    for (int q = first; q < last; q += stride) {
      const float g = __shfl_sync(0xffffffffu, f, q);
      if (((seen >> q) & 1u) && lane * 4 < D) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(t.part + place(32 * k + q) * D) + lane);
        o.x += g * x.x;
        o.y += g * x.y;
        o.z += g * x.z;
        o.w += g * x.w;
      }
    }
  }
  return o;
}

// MEND: look for outputs that are not finite (Args::mend).
template <class Args, int DT, bool MEND>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(const __grid_constant__ Args t,
                                                              int ctas, int join_blocks) {
  constexpr int kWarps = kJoinThreads / 32;
  __shared__ Rec rec[kMaxCtas];
  __shared__ int rows_to[kMaxCtas];  // rows of records 0..c
  __shared__ int warp_rows[kWarps];
  __shared__ int most;
  __shared__ float4 so[kWarps][32];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const AttendArgs& a = t.a;
  if ((int)blockIdx.x >= join_blocks) {
    const int b = ((int)blockIdx.x - join_blocks) * kWarps + warp;
    if (b >= a.b.B) return;
    bool late = false;
    for (int c = lane; c < ctas; c += 32) late |= (__ldcg(t.err + c) & kLate) != 0;
    late = __any_sync(0xffffffffu, late);
    const uint8_t f = sequence_flags(a, b);
    if (lane == 0) a.flags[b] = f | (late ? SV_FLAG_TIMEOUT : 0);
    return;
  }
  // records, and the rows before each (kMaxCtas <= kJoinThreads)
  static_assert(kMaxCtas <= kJoinThreads, "one record per thread");
  if (threadIdx.x == 0) most = 0;
  __syncthreads();
  int n = 0, err = 0;
  if ((int)threadIdx.x < ctas) {
    const Rec r = t.rec[threadIdx.x];
    err = __ldcg(t.err + threadIdx.x);
    rec[threadIdx.x] = r;
    n = r.more ? r.ntok * t.group : 0;
    if (r.more) atomicMax(&most, r.more);
  }
  int scan = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) warp_rows[warp] = scan;
  __syncthreads();
  for (int w = 0; w < warp; ++w) scan += warp_rows[w];
  if (threadIdx.x < kMaxCtas) rows_to[threadIdx.x] = scan;
  __syncthreads();
  const int total = rows_to[kMaxCtas - 1];
  // few rows of many parts: a whole block to a row; else a warp to a row
  const bool wide = most >= 8 && total <= 2 * join_blocks;
  const int step = wide ? join_blocks : join_blocks * kWarps;
  const int begin = wide ? (int)blockIdx.x : (int)blockIdx.x * kWarps + warp;
  auto locate = [&](int j, int& c, int& tok, int& hd) {
    c = 0;
    for (int half = 128; half; half >>= 1)
      if (c + half <= ctas && rows_to[c + half - 1] <= j) c += half;
    const int k = j - (c ? rows_to[c - 1] : 0);
    tok = k / t.group;
    hd = k - tok * t.group;
  };
  bool odd = false;
  for (int j = begin; j < total; j += step) {
    int c, tok, hd;
    locate(j, c, tok, hd);
    const Rec r = rec[c];
    const int row = tok / t.tpt * kTile + tok % t.tpt * t.group + hd;
    const int parts = r.more + 1;
    float M, L;
    float4 o = join_parts(t, c, parts, row, wide ? warp : 0, wide ? kWarps : 1, M, L);
    if (wide) {
      __syncthreads();
      so[warp][lane] = o;
      __syncthreads();
      if (warp) continue;
      for (int w = 1; w < kWarps; ++w) {
        const float4 x = so[w][lane];
        o.x += x.x;
        o.y += x.y;
        o.z += x.z;
        o.w += x.w;
      }
    }
    const int64_t orow = (int64_t)(r.row0 + tok) * a.heads + r.h * t.group + hd;
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int D = a.c.head_dim;
    if (lane * 4 < D) {
      if (MEND) odd |= L == L && !(fabsf(o.x * inv + o.y * inv + o.z * inv + o.w * inv) < kInf);
      const uint2 w = make_uint2(F16<DT>::down(o.x * inv, o.y * inv),
                                 F16<DT>::down(o.z * inv, o.w * inv));
      reinterpret_cast<uint2*>(a.out + orow * D * 2)[lane] = w;
    }
    if (lane == 0 && a.lse) a.lse[orow] = lse_of(M, L);
  }
  if constexpr (MEND) {
    if (!__syncthreads_or(odd || (err & kMend))) return;
    // rare: the rows joined here, and those that the tile kernel wrote itself
    float* sq = reinterpret_cast<float*>(so[warp]);
    if (!wide || !warp)
      for (int j = begin; j < total; j += step) {
        int c, tok, hd;
        locate(j, c, tok, hd);
        Args::template mend<DT>(a, rec[c].row0 + tok, rec[c].h * t.group + hd, sq);
      }
    if (!__syncthreads_or(err & kMend)) return;
    const int64_t rows = (int64_t)a.b.total * a.heads;
    for (int64_t j = (int64_t)blockIdx.x * kWarps + warp; j < rows; j += (int64_t)join_blocks * kWarps) {
      const int tok = (int)(j / a.heads), hq = (int)(j - (int64_t)tok * a.heads);
      bool cut = false;
      for (int c = lane; c < ctas; c += 32)
        cut |= rec[c].more && rec[c].h == hq / t.group && tok >= rec[c].row0 &&
               tok - rec[c].row0 < rec[c].ntok;
      if (!__any_sync(0xffffffffu, cut)) Args::template mend<DT>(a, tok, hq, sq);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline cudaError_t tensor_encoder(EncodeTiled* out) {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q{};
  const cudaError_t e =
      cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
  if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
  *out = reinterpret_cast<EncodeTiled>(fn);
  return cudaSuccess;
}

inline Ring make_ring(int n, int most) {
  const uint32_t k = (uint32_t)(n < most ? n : most);
  return Ring{k, (uint32_t)((0x100000000ull + k - 1) / k)};
}

}  // namespace sv
