// sv_attention_tiles.cu -- spec_chunk_attention on the tensor cores: tiles of 128
// query rows against tiles of 128 keys.
//
//   S = Q K^T (tcgen05, fp32 in tensor memory), P = 2^(c S - m) with the running
//   row maximum m, O += P V (P from tensor memory), l += row sums of P;
//   out = O / l, lse = (m + log2 l) ln 2.
//
// Rows: the `group` query heads of a key head share its keys, so the rows of a
// tile are (token, head of the group) pairs, floor(128 / group) tokens of them; a
// key tile is read once for all of them.  An item is up to two such tiles of one
// (sequence, key head); its keys are cut into tiles of 128 counted from token 0.
//
// Balance: all key tiles of all items form one line, an item's start worth kItemUnits
// tiles more, cut into equal shares, one per CTA (one CTA per SM).  An item cut by a share's end leaves partial (m, l, O)
// in the workspace, at most two per CTA, which k_attend_join adds up; an item
// inside a share is written at once.  Lengths live on the device, so every CTA
// finds its own place in the line at its start.
//
// Two softmax warpgroups keep the tensor cores busy: while one works on its S,
// the other's products run.  An item of two row tiles gives one to each; an item
// of one row tile (a round's few tokens) gives them the key tiles alternately, and
// their (m, l, O) are added up at its end.
//
// Roles: warps 0 and 3 fetch key and value pages (tensor copies, 128-byte swizzle),
// warp 1 issues the products, warp 2 fetches queries, warps 4-11 are the softmax,
// and for e4m3 caches warps 12-19 widen the codes to 16 bits between the copies
// and the products.  Every wait is bounded; one that gives up ends the CTA's roles
// and flags the call.
//
// What bounds it, measured on GB300 (152 SMs, one CTA each):
//   a round (5 tokens, 64 sequences up to 8192, 32/8 heads of 128, bf16): HBM; 197 to
//     203 us for 1.27 GB, 6.3 TB/s, 0.93 of a copy's rate;
//   a prompt chunk (4096 and 1605 tokens, 32/8 heads of 128, bf16): the chain softmax,
//     P V, Q K^T of a stage (about 3200 clocks for 2048 of products) and the power
//     limit; 440 to 500 us, 1.2 to 1.35 PFLOP/s, 0.62 to 0.70 of a large library
//     product's rate;
//   a round on e4m3 (9 tokens, 32 sequences up to 40000, 64/8 heads of 128): the widening
//     of codes, by its length rather than by a full unit; 449 to 455 us, 3.4 TB/s of codes,
//     0.50 of a copy's.  Per tile of 128 keys and values an SM issues about 1800
//     instructions a scheduler (half of them widen codes), and has 1370 clocks at HBM's
//     rate; 60% of the issue slots are used and no pipe more than 41%, while the tiles'
//     three widened slots are waited for on both sides.
//   small calls: the chain lengths, page numbers, copies, products, join; 16 us for one
//     token on 777, of them 3 to find the shares, 3 to the first scores, 5 for the join.
// The 128 x 128 tile keeps S, P and O of two stages in tensor memory's 512 columns; the
// operands leave room for five tiles of 32 KB in flight, what HBM's latency asks for.
//
// Waits of one CTA, by barrier: full/empty (key and value tiles in 16 bits),
// rawfull/rawempty (e4m3 codes), qfull/qempty (query tiles), sfull (S ready),
// pfull (P written, so S is free), ofull (last product of a stage done), xbar
// (the two warpgroups at the end of a one-tile item).  Two warps (or two groups of
// converters) that take a ring's tiles in turn leave out turns of a slot, and a
// waiter who leaves out turns can take one phase of a barrier for another; so the
// barriers that such waiters wait on are those of a ring of twice the slots, whose
// every place belongs to one of the two.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "specverify.h"
#include "sv_attention.h"
#include "sv_attention_row.cuh"
#include "sv_cache.cuh"
#include "sv_device.cuh"
#include "sv_launch.h"
#include "sv_tma.cuh"
#include "sv_umma.cuh"

namespace sv {
namespace {

constexpr int kTile = 128;          // query rows and keys per tile
constexpr int kSpan = 16384;        // 128 rows of one 128-byte swizzle span
constexpr int kMaxCtas = 160;       // shares (GB300: 152 SMs)
constexpr int kMaxRows = 2 * kTile;
constexpr int kMaxStages = 12, kMaxRaw = 8;
constexpr long long kWaitClocks = 1ll << 32;  // about two seconds
// The wait limit and the CTA whose first scores are never handed over in the next calls
// (a failure test sets them through sv_test_attention_stall; not thread-safe).
long long g_wait_clocks = kWaitClocks;
int g_stall_cta = -1;
constexpr size_t kSmemBytes = 227 * 1024;
constexpr int kQBytes = 2 * kSpan;                // one query tile
// Shared memory: two query tiles, then 160 KB.  A 16-bit cache's ring of key and value
// tiles (5 of 32 KB, or 10 of 16 KB) takes those; an e4m3 cache's codes take the first
// 64 KB and the widened tiles (3 or 6) the rest.  In a call without an item of two row
// tiles the second query tile is not used, and the first of the rings starts there (a
// round of 64 sequences of bf16, 6 tiles in flight instead of 5: 203 us instead of 212).
constexpr int kCodes = 64 * 1024, kRing16 = 160 * 1024, kRing8 = 96 * 1024;
constexpr int kScaleBytes = kMaxRaw * kTile;
// What an item costs beside its key tiles (its queries, the end of its pipeline, its
// outputs), in key tiles.  (Shares of key tiles alone: a round of 64 sequences 203 us,
// with 1, 2, 3, 4 a start 201, 198, 197, 197; the prompt chunk 449 and 443, 439, 439, 440.)
constexpr int kItemUnits = 3;
constexpr int kJoinThreads = 256;
// The running maximum may lag by this many powers of two before O is rescaled: P
// stays within 2^8, exact enough in 16-bit floats and far from their range.
constexpr float kLag = 8.0f;
// Threads, and the registers a thread is launched with and then takes by role (the
// roles' sum must not pass what the launch gave, or the takers would wait forever).
constexpr int kThreads16 = 384, kWideWarps = 4, kThreads8 = 384 + 64 * kWideWarps;
// (At these counts the kernels spill 28 to 50 words a thread, outside the loops over key
// tiles: eight times the keys leave the number of their loads and stores the same.)
constexpr int kRegs16 = 168, kRegs8 = 96;
constexpr int kHelpRegs16 = 88, kSoftRegs16 = 208;
constexpr int kHelpRegs8 = 64, kSoftRegs8 = 128, kWideRegs8 = 80;
static_assert(128 * kHelpRegs16 + 256 * kSoftRegs16 <= kThreads16 * kRegs16, "registers");
static_assert(128 * kHelpRegs8 + 256 * kSoftRegs8 + 64 * kWideWarps * kWideRegs8 <= kThreads8 * kRegs8, "registers");

// Slots of a ring, and ceil(2^32 / slots): slot and turn of tile k without a division.
struct Ring {
  uint32_t n, inv;
};

struct TileArgs {
  AttendArgs a;
  int group, tpt;      // query heads per key head; tokens per row tile
  int nhalf;           // swizzle spans per row: 1 (head_dim <= 64) or 2
  Ring tiles[2], codes[2];  // of 16-bit tiles and of codes, without and with items of two
  Ring tiles2[2], codes2[2];  // twice their slots (see the barriers)
  int box;             // tokens per copy: min(page_size, 128)
  int fetchers;        // warps that fetch key and value tiles
  int stall;           // test only: the CTA whose first scores are withheld (-1: none)
  long long wait_clocks;
  int wide;            // outputs sit on 32-byte boundaries
  float c;             // scale log2 e, positive
  float* part;         // [2 * kMaxCtas][kMaxRows][head_dim]
  float2* ml;          // [2 * kMaxCtas][kMaxRows]
  struct Rec* rec;     // [kMaxCtas]
  int* err;            // [kMaxCtas]: kLate, kMend; above 8 bits a wait that gave up
};

constexpr int kLate = 1, kMend = 2;

// What a CTA leaves for the join: the item that it began and did not end.
struct Rec {
  int more;            // further CTAs with a part of it (0: nothing to join)
  int row0, ntok, h;   // first packed row, tokens, key head
};

// Control words of a CTA.
struct Ctl {
  uint64_t full[kMaxStages], empty[2 * kMaxStages], rawfull[2 * kMaxRaw], rawempty[2 * kMaxRaw];
  uint64_t qfull[2], qempty[2], sfull[2], pfull[2], ofull[2], xbar, fin;
  uint32_t tmem;
  int abort;
  int mend;            // a row written by this CTA holds something that is not finite
  int two;             // some item of the call has two row tiles
  int b, h, qt, off;   // start of the CTA's share (off in units)
  long long left, share;
  union {
    long long warp_units[kThreads8 / 32];
    float2 xch[kTile];  // (m, l) from one warpgroup to the other
  };
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

// Units of one head of the lane's sequence (n = 0: none).  A sequence of many
// items is summed by the whole warp.
__device__ __forceinline__ long long head_units(const Seq& q, int per_item, int window) {
  const int lane = threadIdx.x & 31;
  const int nqt = (q.n + per_item - 1) / per_item;
  long long u = 0;
  if (nqt <= 4)
    for (int t = 0; t < nqt; ++t) u += kItemUnits + item_span(q, per_item, t, window).count;
  unsigned big = __ballot_sync(0xffffffffu, nqt > 4);
  while (big) {
    const int src = __ffs(big) - 1;
    big &= big - 1;
    Seq s{};
    s.n = __shfl_sync(0xffffffffu, q.n, src);
    s.pos0 = __shfl_sync(0xffffffffu, q.pos0, src);
    long long v = 0;
    const int m = (s.n + per_item - 1) / per_item;
    for (int t = lane; t < m; t += 32) v += kItemUnits + item_span(s, per_item, t, window).count;
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
__device__ void find_share(const TileArgs& t, Ctl& ctl) {
  const BatchView& bv = t.a.b;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = (int)(blockDim.x >> 5);
  const int per_item = 2 * t.tpt, H = t.a.c.kv_heads, ps = t.a.c.page_size;
  const int chunk = (bv.B + nw - 1) / nw;
  const int b0 = min(bv.B, warp * chunk), b1 = min(bv.B, b0 + chunk);
  Seq q{};
  long long per_head = 0, sum = 0;
  auto look = [&](int base) {
    q = Seq{};
    if (base + lane < b1) q = load_seq(bv, base + lane, ps);
    per_head = head_units(q, per_item, t.a.window);
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
        const long long c =
            q0 + lane < m ? kItemUnits + item_span(s, per_item, q0 + lane, t.a.window).count : 0;
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

  __device__ __forceinline__ Walk(const Ctl& c)
      : b(c.b), h(c.h), qt(c.qt), off(c.off), nqt(0), left(c.left), loaded(false) {}

  __device__ __forceinline__ bool next(const TileArgs& t, const Ctl& ctl, Seg& s) {
    if (left <= 0) return false;
    const int per_item = 2 * t.tpt;
    while (!loaded) {
      if (b >= t.a.b.B) return false;
      q = load_seq(t.a.b, b, t.a.c.page_size);
      nqt = (q.n + per_item - 1) / per_item;
      if (nqt) loaded = true;
      else ++b;
    }
    const Span sp = item_span(q, per_item, qt, t.a.window);
    // units off .. off + take of the item: its start, then a unit a tile
    const int avail = sp.count + kItemUnits - off;
    const int take = (int)min((long long)avail, left);
    const int t0 = max(0, off - kItemUnits), t1 = off + take - kItemUnits;
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

// Ring order of an item part's tiles: K0 K1 V0 K2 V1 ... V(n-1), as the products
// need them when the next S is computed one product ahead.
__device__ __forceinline__ int k_index(int i) { return i ? 2 * i - 1 : 0; }
__device__ __forceinline__ int v_index(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }
__device__ __forceinline__ void tile_of(int idx, int n, bool& is_v, int& tile) {
  is_v = idx == 2 * n - 1 || (idx > 0 && (idx & 1) == 0);
  tile = is_v ? (idx == 2 * n - 1 ? n - 1 : idx / 2 - 1) : (idx + 1) / 2;
}

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

// Keys of a tile that some row sees, in steps of 16 (a product's depth).
__device__ __forceinline__ void key_steps(int lo, int hi, int tile, int& s0, int& s1) {
  const int key0 = tile * kTile;
  s0 = max(0, lo - key0) / 16;
  s1 = max(s0, (min(kTile, hi - key0) + 15) / 16);
}

// ---------------------------------------------------------------------------
// Waits.
// ---------------------------------------------------------------------------
// Which wait gave up, in the CTA's err word, for whoever looks at the workspace after a timeout.
enum WaitId { kWaitSlot = 1, kWaitQ, kWaitK, kWaitV, kWaitP, kWaitQFree, kWaitS, kWaitO, kWaitX, kWaitRaw,
              kWaitWide };

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
// What must have ended before the CTA may go, whether or not the call is aborted.
__device__ __forceinline__ void wait_end(uint64_t* bar, uint32_t parity, const Guard& guard) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity) && clock64() - t0 < guard.clocks) {
  }
}

// ---------------------------------------------------------------------------
// Softmax of one S tile row (this thread's), 128 scores in tensor memory.
// ---------------------------------------------------------------------------
// Scores of columns that the row does not see become -inf; it sees [first, first + span).
template <int N>
__device__ __forceinline__ void hide(uint32_t* r, int first, int span) {
#pragma unroll
  for (int j = 0; j < N; ++j)
    if ((unsigned)(j - first) >= (unsigned)span) r[j] = 0xff800000u;
}
template <int N>
__device__ __forceinline__ float max_of(const uint32_t* r) {
  float m[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
  for (int j = 0; j < N; ++j) m[j & 3] = fmaxf(m[j & 3], __uint_as_float(r[j]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// P = 2^(c s - m) of N scores in pairs of 16-bit floats into tensor memory; adds to
// the four pairs of sums.  P is rounded to the values' type because the product takes
// both operands in one 16-bit type, and a second product for what the rounding leaves
// would double the time of P V; the sums are of the unrounded weights.  Measured against
// 64 bits: an error of 2.1e-3 to 2.3e-3 in bf16, where rounding the output alone leaves
// 1.7e-3, and 2.9e-4 in fp16, of 2.1e-4.
template <int PT, int N>
__device__ __forceinline__ void exp_of(const uint32_t* r, float c, float m, uint32_t p_tm,
                                       uint64_t* acc) {
  const uint64_t cc = pack2(c, c), mm = pack2(-m, -m);
#pragma unroll
  for (int k = 0; k < N; k += 32) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float x, y;
      unpack2(ffma2(pack2(__uint_as_float(r[k + 2 * j]), __uint_as_float(r[k + 2 * j + 1])), cc, mm),
              x, y);
      x = ex2(x);
      y = ex2(y);
      acc[j & 3] = fadd2(acc[j & 3], pack2(x, y));
      w[j] = F16<PT>::down(x, y);
    }
    tmem_st16(p_tm + k / 2, w);
  }
}
__device__ __forceinline__ float sum_of(const uint64_t* acc) {
  float a, b;
  unpack2(fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3])), a, b);
  return a + b;
}

// Two e4m3 values times 2^(sc - 127) in 16 bits.  bf16: the codes fit bf16 and a power
// of two changes no digit, so the packed product is exact; fp16 rounds once from fp32.
template <int DT>
__device__ __forceinline__ uint32_t scaled(float2 v, uint32_t sc) {
  if (DT == SV_F16) {
    const float f = scale_of(sc);
    return F16<DT>::down(v.x * f, v.y * f);
  }
  const uint32_t f2 = (sc << 7) | (sc << 23), c = F16<SV_BF16>::down(v.x, v.y);
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(c), "r"(f2));
  return r;
}

// O *= f (rows that need none have f = 1).
__device__ __forceinline__ void rescale(uint32_t o_tm, int units, float f) {
  for (int u = 0; u < units; ++u) {
    uint32_t r[16];
    __syncwarp();
    tmem_ld16_async(o_tm + 16 * u, r);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * f);
    tmem_st16(o_tm + 16 * u, r);
  }
  tmem_wait_st();
}

// A lane's 16 outputs of one row: one 32-byte store (a whole sector) where that is aligned.
template <int DT>
__device__ __forceinline__ void store16(char* at, const float* x, bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = F16<DT>::down(x[2 * j], x[2 * j + 1]);
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
    return;
  }
  reinterpret_cast<uint4*>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void store16f(float* at, const float* x) {  // 32-byte aligned
#pragma unroll
  for (int j = 0; j < 16; j += 8)
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at + j), "f"(x[j]),
                 "f"(x[j + 1]), "f"(x[j + 2]), "f"(x[j + 3]), "f"(x[j + 4]), "f"(x[j + 5]),
                 "f"(x[j + 6]), "f"(x[j + 7])
                 : "memory");
}

// (not finite if one of them is not)
__device__ __forceinline__ float sum16(const float* x) {
  uint64_t s[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    s[j] = fadd2(pack2(x[4 * j], x[4 * j + 1]), pack2(x[4 * j + 2], x[4 * j + 3]));
  return sum_of(s);
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

template <int DT, bool E4M3>
__global__ void __launch_bounds__(E4M3 ? kThreads8 : kThreads16, 1)
k_attend_tiles(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ TileArgs t) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int kPT = DT;
  constexpr float kShift = kPT == SV_F16 ? 6.0f : 0.0f;  // fp16 P within 2^14: small ones keep bits
  uint8_t* const qbuf = smem;
  uint8_t* const scale_area = smem + 2 * kQBytes + kRing16;  // e4m3: [kMaxRaw][128]
  Ctl& ctl = *reinterpret_cast<Ctl*>(scale_area + kScaleBytes);
  static_assert(2 * kQBytes + kRing16 + kScaleBytes + sizeof(Ctl) <= kSmemBytes, "shared memory");
  static_assert(kCodes + kRing8 == kRing16, "shared memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttendArgs& a = t.a;
  const int D = a.c.head_dim;
  const int stage_bytes = t.nhalf * kSpan, raw_bytes = kTile * D;
  const Guard guard{&ctl.abort, t.wait_clocks};

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    ctl.two = 0;
    ctl.mend = 0;
    ctl.abort = (smem_u32(smem) & 1023u) ? 1 : 0;  // the swizzle needs this alignment
    for (int i = 0; i < kMaxStages; ++i) mbar_init(ctl.full + i, E4M3 ? kWideWarps : 1);
    for (int i = 0; i < 2 * kMaxStages; ++i) mbar_init(ctl.empty + i, 1);
    for (int i = 0; i < 2 * kMaxRaw; ++i) {
      mbar_init(ctl.rawfull + i, 1);
      mbar_init(ctl.rawempty + i, kWideWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(ctl.qfull + i, 1);
      mbar_init(ctl.qempty + i, 1);
      mbar_init(ctl.sfull + i, 1);
      mbar_init(ctl.pfull + i, 4);
      mbar_init(ctl.ofull + i, 1);
    }
    mbar_init(&ctl.xbar, 8);
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
  const int wid = (int)blockIdx.x;
  const int pair = ctl.two;                       // query tiles held: 1 + pair
  const Ring rt = t.tiles[pair], rc = t.codes[pair], rt2 = t.tiles2[pair], rc2 = t.codes2[pair];
  uint8_t* const first = smem + (1 + pair) * kQBytes;
  uint8_t* const raw = first;                     // e4m3: codes
  uint8_t* const ring = E4M3 ? smem + 2 * kQBytes + kCodes : first;
  Walk walk(ctl);
  Seg s;
  bool ok = *guard.flag == 0;
  if (warp < 4) give_regs<E4M3 ? kHelpRegs8 : kHelpRegs16>();

  if (warp == 0 || (warp == 3 && t.fetchers == 2)) {
    // ---------------- fetch key and value pages ----------------
    // Two warps take the tiles in turn where one alone (page numbers, a wait, up to 16
    // copies a tile) is slower than HBM.  The lanes hold a tile's copies; its page
    // numbers are read a tile ahead.
    const uint64_t pol = l2_policy_evict_first();
    const uint32_t turn = warp == 3 ? 1u : 0u;
    const Ring rs = E4M3 ? rc : rt, rs2 = E4M3 ? rc2 : rt2;
    uint64_t* const freeb = E4M3 ? ctl.rawempty : ctl.empty;
    uint32_t issued = 0, done = 0;  // tiles before the part; behind this warp's last
    const int copies = kTile / t.box;                                  // along a tile
    const int part = E4M3 ? lane : (t.nhalf == 2 ? lane >> 1 : lane);  // this lane's copy ...
    const int half = E4M3 ? 0 : (t.nhalf == 2 ? lane & 1 : 0);         // ... and span
    for (; ok && walk.next(t, ctl, s); issued += 2u * (uint32_t)s.n) {
      const int32_t* table = a.b.table + (int64_t)s.b * a.b.max_pages;
      // the copies of a tile that hold keys somebody sees, and this lane's page
      auto look = [&](int idx, int& key0, int& from, int& upto, bool& is_v) {
        int tile;
        tile_of(idx, s.n, is_v, tile);
        key0 = (s.t0 + tile) * kTile;
        from = max(0, s.lo - key0) / t.box;
        upto = min(copies, (max(0, s.hi - key0) + t.box - 1) / t.box);
        const int mine = key0 + part * t.box;
        return part >= from && part < upto ? __ldg(table + (mine >> a.c.page_shift)) : -1;
      };
      int key0, from, upto;
      bool is_v;
      int idx = (int)turn;  // (a part has 2 n tiles: issued is even)
      int page = look(idx, key0, from, upto, is_v);
      for (; ok && idx < 2 * s.n; idx += t.fetchers) {
        const uint32_t k = issued + (uint32_t)idx, slot = Slot(k, rs).i;
        const Slot at2(k, rs2);
        uint64_t* const fullb = E4M3 ? ctl.rawfull + at2.i : ctl.full + slot;
        ok = wait_warp(freeb + at2.i, at2.i < rs.n ? at2.ph ^ 1u : at2.ph, guard, kWaitSlot);
        if (!ok) break;
        const int live = max(0, upto - from);
        const bool mine = part >= from && part < upto;
        const int in_page = (key0 + part * t.box) & (a.c.page_size - 1);
        uint32_t bytes = (uint32_t)(live * t.box * (E4M3 ? D : t.nhalf * 128));
        if (E4M3) {
          // a page outside the pool arrives as zeros; so do its scales
          uint8_t* const dst = raw + (size_t)slot * raw_bytes + part * t.box * D;
          uint8_t* const scales = scale_area + slot * kTile + part * t.box;
          const bool sound = page >= 0 && page < a.c.num_pages;
          bytes += __popc(__ballot_sync(0xffffffffu, sound)) * t.box;
          if (mine && !sound)
            for (int e = 0; e < t.box; e += 16)
              *reinterpret_cast<uint4*>(scales + e) = make_uint4(0, 0, 0, 0);
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(fullb, bytes);
          __syncwarp();
          if (mine) {
            tma_load_4d_hint(dst, is_v ? &mv : &mk, 0, in_page, s.h, page, fullb, pol);
            if (sound)
              bulk_load(scales,
                        (is_v ? a.c.vs : a.c.ks) +
                            ((int64_t)page * a.c.kv_heads + s.h) * a.c.page_size + in_page,
                        (uint32_t)t.box, fullb);
          }
        } else {
          uint8_t* const dst =
              ring + (size_t)slot * stage_bytes + half * kSpan + part * t.box * 128;
          if (lane == 0) mbar_arrive_expect_tx(fullb, bytes);
          __syncwarp();
          if (mine)
            tma_load_4d_hint(dst, is_v ? &mv : &mk, 64 * half, in_page, s.h, page, fullb, pol);
        }
        __syncwarp();
        done = k + 1;
        if (idx + t.fetchers < 2 * s.n) page = look(idx + t.fetchers, key0, from, upto, is_v);
      }
    }
    // every copy has landed before the CTA may exit
    const uint32_t end = ok ? issued : done;
    for (uint32_t k = end > rs.n ? end - rs.n : 0; k < end; ++k) {
      const Slot at(k, E4M3 ? rc2 : rt);
      if (lane == 0 && (t.fetchers == 1 || (k & 1u) == turn)) wait_end((E4M3 ? ctl.rawfull : ctl.full) + at.i, at.ph, guard);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- issue the products ----------------
    const uint32_t leader = elect_leader();
    const uint32_t idesc_s = umma_idesc_16(DT == SV_BF16, kTile, kTile, false);
    const uint32_t idesc_o = umma_idesc_16(kPT == SV_BF16, kTile, D, true);
    const int ksteps = D / 16;
    const uint64_t qdesc = umma_smem_desc(smem_u32(qbuf), 16, 1024);
    const uint64_t kdesc = umma_smem_desc(smem_u32(ring), 16, 1024);
    const uint64_t vdesc = umma_smem_desc(smem_u32(ring), kSpan, 1024);
    const uint32_t stage16 = (uint32_t)stage_bytes >> 4, tb = (uint32_t)uniform((int)tbase);
    const int pr = uniform(pair);
    uint32_t base = 0, qn = 0;          // tiles and query tiles used so far
    uint32_t pph = 0;                   // phases of the two stages' P
    while (ok && walk.next(t, ctl, s)) {
      const int n = uniform(s.n), two = uniform(s.two ? 1 : 0);
      const int lo = uniform(s.lo), hi = uniform(s.hi), t0 = uniform(s.t0);
      const int jobs = n << two;
      // S of job j (stage j & 1), once its tiles are there
      auto key_slot = [&](int j) {
        return Slot(base + (uint32_t)k_index(j >> two), rt);
      };
      // whoever waits for tile k's slot waits for tile k + n, the slot's next
      auto freed = [&](uint32_t k) { return ctl.empty + Slot(k + rt.n, rt2).i; };
      auto scores = [&](int j, uint32_t slot, uint32_t tell) {
        const int i = j >> two, st = j & 1;
        const uint32_t qb = (qn + (uint32_t)(two & st)) & (uint32_t)pr;
        const uint64_t ad = qdesc + qb * (kQBytes >> 4), bd = kdesc + slot * stage16;
        const uint32_t acc = tb + st * kTile;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t o = (uint64_t)((kk >> 2) * (kSpan >> 4) + (kk & 3) * 2);
          if (kk < ksteps) umma_ss_if(leader, acc, ad + o, bd + o, idesc_s, kk != 0);
        }
        umma_commit_if(tell, ctl.sfull + st);
        if (!two || st) umma_commit_if(leader, freed(base + (uint32_t)k_index(i)));
        if (i == n - 1) umma_commit_if(leader, ctl.qempty + qb);
      };
      for (int j = 0; j < 2 && j < jobs; ++j) {
        const Slot k = key_slot(j);
        const uint32_t qk = qn + (uint32_t)(two & j);
        ok = wait_warp(ctl.qfull + (qk & (uint32_t)pr), (qk >> pr) & 1u, guard, kWaitQ) &&
             wait_warp(ctl.full + k.i, k.ph, guard, kWaitK);
        if (!ok) break;
        tc_fence_after();
        // (a test may withhold a CTA's first scores: the softmax's wait then runs out)
        scores(j, k.i, t.stall == wid && base == 0 && j == 0 ? 0u : leader);
      }
      for (int j = 0; ok && j < jobs; ++j) {
        const int i = j >> two, st = j & 1;
        const bool more = j + 2 < jobs;
        const Slot v(base + (uint32_t)v_index(i, n), rt);
        const Slot k = key_slot(more ? j + 2 : j);
        int s0, s1;
        key_steps(lo, hi, t0 + i, s0, s1);
        const uint64_t bd = vdesc + v.i * stage16;
        const uint32_t acc = tb + 256 + st * kTile, p = tb + st * kTile;
        const bool fresh = two ? i == 0 : j < 2;
        // P is awaited last: nothing then stands between it and the products.  (The key
        // tile of job j + 2 does not depend on job j: its slot was freed by an earlier
        // one.  Of an e4m3 cache's three slots that one is freed late: there the key
        // tile is awaited behind the product with V.)
        ok = wait_warp(ctl.full + v.i, v.ph, guard, kWaitV) &&
             (E4M3 || !more || wait_warp(ctl.full + k.i, k.ph, guard, kWaitK)) &&
             wait_warp(ctl.pfull + st, (pph >> st) & 1u, guard, kWaitP);
        if (!ok) break;
        pph ^= 1u << st;
        tc_fence_after();
        if (s0 == 0 && s1 == 8) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts_if(leader, acc, p + kk * 8, bd + (uint64_t)(kk * 128), idesc_o, kk || !fresh);
        } else {
          for (int kk = s0; kk < s1; ++kk)
            umma_ts_if(leader, acc, p + kk * 8, bd + (uint64_t)(kk * 128), idesc_o, kk != s0 || !fresh);
        }
        if (!two || st) umma_commit_if(leader, freed(base + (uint32_t)v_index(i, n)));
        if (E4M3 && more) {
          ok = wait_warp(ctl.full + k.i, k.ph, guard, kWaitK);
          if (!ok) break;
          tc_fence_after();
        }
        if (more) scores(j + 2, k.i, leader);
        else umma_commit_if(leader, ctl.ofull + st);
      }
      base += 2u * (uint32_t)n;
      qn += 1u + (uint32_t)two;
    }
    // all products complete before tensor memory is released
    umma_commit_if(leader, &ctl.fin);
    wait_end(&ctl.fin, 0, guard);
  } else if (warp == 2) {
    // ---------------- fetch query tiles ----------------
    // A copy takes tpt tokens by group heads, rows in the order of the tile.  Tokens
    // behind the sequence's last are other sequences' or zeros: nobody reads their rows.
    const uint64_t pol = l2_policy_evict_first();
    uint32_t qn = 0;
    if (lane == 0) t.rec[wid].more = 0;
    while (ok && walk.next(t, ctl, s)) {
      if (lane == 0 && s.slot == 1) t.rec[wid] = Rec{s.more, s.row0, s.ntok, s.h};
      for (int st = 0; ok && st < (s.two ? 2 : 1); ++st, ++qn) {
        const uint32_t qb = qn & (uint32_t)pair;
        ok = wait_warp(ctl.qempty + qb, ((qn >> pair) & 1u) ^ 1u, guard, kWaitQFree);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(ctl.qfull + qb, (uint32_t)(t.nhalf * t.tpt * t.group * 128));
          for (int h = 0; h < t.nhalf; ++h)
            tma_load_3d_hint(qbuf + qb * kQBytes + h * kSpan, &mq, 64 * h, s.h * t.group,
                             s.row0 + st * t.tpt, ctl.qfull + qb, pol);
        }
        __syncwarp();
      }
    }
    // every copy has landed before the CTA may exit
    const uint32_t held = 1u + (uint32_t)pair;
    for (uint32_t i = qn > held ? qn - held : 0; i < qn; ++i)
      if (lane == 0) wait_end(ctl.qfull + (i & (uint32_t)pair), (i >> pair) & 1u, guard);
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // ---------------- softmax and output ----------------
    take_regs<E4M3 ? kSoftRegs8 : kSoftRegs16>();
    const int st = (warp - 4) >> 2, quad = warp & 3, row = 32 * quad + lane;
    const uint32_t lanes = tbase + ((uint32_t)(32 * quad) << 16);
    const uint32_t s_tm = lanes + st * kTile, o_tm = lanes + 256 + st * kTile;
    const int units = D / 16;
    const int my_tok = row / t.group, my_head = row - my_tok * t.group;
    uint32_t sph = 0, oph = 0, xph = 0;
    uint32_t base = 0;  // tiles of the parts before
    for (; ok && walk.next(t, ctl, s); base += 2u * (uint32_t)s.n) {
      const int shift = s.two ? 0 : 1;
      const int jobs = s.two ? s.n : (s.n + 1 - st) >> 1;
      const int tok_off = s.two ? st * t.tpt : 0;
      const int ntok = min(t.tpt, s.ntok - tok_off);
      const bool live = my_tok < ntok;
      const bool warp_live = 32 * quad < ntok * t.group;
      const int pos = s.pos + tok_off + my_tok;
      const int see1 = live ? pos + 1 : 0;  // keys [see0, see1)
      const int see0 = a.window && see1 > a.window ? see1 - a.window : 0;
      float m = -kInf, l = 0.0f;
      for (int k = 0; ok && k < jobs; ++k) {
        if (!wait_warp(ctl.sfull + st, sph, guard, kWaitS)) {
          ok = false;
          break;
        }
        sph ^= 1u;
        tc_fence_after();
        const int i = shift ? 2 * k + st : k;  // key tile
        if (warp_live) {
          const int key0 = (s.t0 + i) * kTile;
          const int first = max(0, see0 - key0), span = max(0, min(kTile, see1 - key0) - first);
          const bool masked = __any_sync(0xffffffffu, live && span < kTile);
          // beside the converters a thread has no room for all of its scores: it reads
          // them twice, 64 at a time (P lies over scores that were read by then)
          constexpr int kHeld = E4M3 ? 64 : kTile;
          uint32_t r[kHeld];
          float tm = -kInf;
#pragma unroll 1
          for (int c0 = 0; c0 < kTile; c0 += kHeld) {
#pragma unroll
            for (int c = 0; c < kHeld; c += 32) tmem_ld32_async(s_tm + c0 + c, r + c);
            tmem_wait_ld();
            if (masked) hide<kHeld>(r, first - c0, span);
            tm = fmaxf(tm, max_of<kHeld>(r));
          }
          tm = tm * t.c - kShift;
          const bool rise = tm > m + kLag || (m == -kInf && tm > m);
          if (__any_sync(0xffffffffu, rise)) {
            const float nm = rise ? tm : m;
            if (k) {
              const float f = rise ? ex2(m - nm) : 1.0f;
              l *= f;
              rescale(o_tm, units, f);
            }
            m = nm;
          }
          const float mu = m == -kInf ? 0.0f : m;
          uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll 1
          for (int c0 = 0; c0 < kTile; c0 += kHeld) {
            if (E4M3) {
#pragma unroll
              for (int c = 0; c < kHeld; c += 32) tmem_ld32_async(s_tm + c0 + c, r + c);
              tmem_wait_ld();
              if (masked) hide<kHeld>(r, first - c0, span);
            }
            exp_of<kPT, kHeld>(r, t.c, mu, s_tm + c0 / 2, acc);
          }
          l += sum_of(acc);
          tmem_wait_st();
        }
        if (!E4M3 && !(s.two && st) && (i == 0 || i == s.n - 1)) {
          // value rows of the first and last step that nobody sees may hold anything:
          // zeros (their P is 0, but 0 times infinity is not)
          const int key0 = (s.t0 + i) * kTile;
          const int v0 = max(0, s.lo - key0), v1 = min(kTile, s.hi - key0);
          if (((v0 | v1) & 15) && v1 > v0) {
            const Slot vk(base + (uint32_t)v_index(i, s.n), rt);
            if (!wait_warp(ctl.full + vk.i, vk.ph, guard, kWaitV)) {
              ok = false;
              break;
            }
            uint8_t* const vt = ring + (size_t)vk.i * stage_bytes;
            const int pre = v0 & 15, post = -v1 & 15, chunks = t.nhalf * 8;
            for (int e = row; e < (pre + post) * chunks; e += kTile) {
              const int r = e / chunks, ch = e - r * chunks;
              const int vr = r < pre ? v0 - pre + r : v1 + r - pre;
              *reinterpret_cast<uint4*>(vt + (ch >> 3) * kSpan + vr * 128 + (ch & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
          }
        }
        __syncwarp();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ctl.pfull + st);
      }
      if (!ok) break;
      if (jobs) {
        if (!wait_warp(ctl.ofull + st, oph, guard, kWaitO)) {
          ok = false;
          break;
        }
        oph ^= 1u;
        tc_fence_after();
      }
      const int64_t prow = ((int64_t)(2 * wid + (s.slot > 0 ? 1 : 0)) * kMaxRows + (s.two ? st * kTile : 0) + row);
      const int64_t orow = (int64_t)(s.row0 + tok_off + my_tok) * a.heads + s.h * t.group + my_head;
      if (s.two || s.n == 1) {  // (of a single key tile, all is warpgroup 0's)
        if (warp_live && (s.two || st == 0)) {
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          for (int u = 0; u < units; ++u) {
            uint32_t r[16];
            float x[16];
            __syncwarp();  // the lanes parted at the stores
            tmem_ld16_async(o_tm + 16 * u, r);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              x[j] = __uint_as_float(r[j]);
              if (s.slot < 0) x[j] = l == 0.0f ? 0.0f : x[j] * inv;
            }
            if (live) {
              if (s.slot < 0) {
                if (l == l && !(fabsf(sum16(x)) < kInf)) ctl.mend = kMend;
                store16<DT>(a.out + (orow * D + 16 * u) * 2, x, t.wide);
              } else {
                store16f(t.part + prow * D + 16 * u, x);
              }
            }
          }
          if (live) {
            if (s.slot < 0) {
              if (a.lse) a.lse[orow] = lse_of(m, l);
            } else {
              t.ml[prow] = make_float2(m, l);
            }
          }
        }
      } else {
        // stage 1's (m, l) to warpgroup 0, then stage 0's to warpgroup 1
        float2 p0 = make_float2(m, l), p1 = p0;
        for (int turn = 0; ok && turn < 2; ++turn) {
          if (st != turn) ctl.xch[row] = make_float2(m, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl.xbar);
          ok = wait_warp(&ctl.xbar, xph, guard, kWaitX);
          xph ^= 1u;
          if (st == turn) (st ? p0 : p1) = ctl.xch[row];
          __syncwarp();
        }
        if (!ok) break;
        tc_fence_after();
        if (warp_live) {
          const float M = fmaxf(p0.x, p1.x);
          const float f0 = p0.y == 0.0f ? 0.0f : ex2(p0.x - (M == -kInf ? 0.0f : M));
          const float f1 = p1.y == 0.0f ? 0.0f : ex2(p1.x - (M == -kInf ? 0.0f : M));
          const float L = (p0.y == 0.0f ? 0.0f : f0 * p0.y) + (p1.y == 0.0f ? 0.0f : f1 * p1.y);
          const float inv = s.slot >= 0 ? 1.0f : (L == 0.0f ? 0.0f : 1.0f / L);
          const int u0 = st ? (units + 1) / 2 : 0, u1 = st ? units : (units + 1) / 2;
          for (int u = u0; u < u1; ++u) {
            uint32_t r0[16], r1[16];
            float x[16];
            __syncwarp();  // the lanes parted at the stores
            tmem_ld16_async(lanes + 256 + 16 * u, r0);
            tmem_ld16_async(lanes + 256 + kTile + 16 * u, r1);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              // a stage without keys left its O as it was: not read
              const float y0 = p0.y == 0.0f ? 0.0f : f0 * __uint_as_float(r0[j]);
              const float y1 = p1.y == 0.0f ? 0.0f : f1 * __uint_as_float(r1[j]);
              x[j] = (y0 + y1) * inv;
            }
            if (live) {
              if (s.slot < 0) {
                if (L == L && !(fabsf(sum16(x)) < kInf)) ctl.mend = kMend;
                store16<DT>(a.out + (orow * D + 16 * u) * 2, x, t.wide);
              } else {
                store16f(t.part + prow * D + 16 * u, x);
              }
            }
          }
          if (live && st == 0) {
            if (s.slot < 0) {
              if (a.lse) a.lse[orow] = lse_of(M, L);
            } else {
              t.ml[prow] = make_float2(M, L);
            }
          }
        }
        // the other warpgroup has read this stage's O and (m, l)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.xbar);
        if (!wait_warp(&ctl.xbar, xph, guard, kWaitX)) {
          ok = false;
          break;
        }
        xph ^= 1u;
        tc_fence_after();
      }
    }
  } else if (E4M3 && warp >= 12) {
    // ---------------- widen e4m3 codes ----------------
    // Two groups of four warps take the tiles in turn, so that one tile's loads and
    // stores stand beside the other's arithmetic.  (Groups of eight leave 72 registers
    // a thread instead of 96 and hide no more: round 448 us instead of 445, window 141
    // instead of 137; converters with 64 registers and softmax with 144: 465 us.)
    // A lane widens 16 codes of a row (two 16-byte chunks of a swizzle span).  Four
    // lanes take one span of a row and the next four that span of the row below, so
    // that the eight lanes of a store's phase write different banks; four loads at a
    // time, 16 rows a warp and step.
    give_regs<kWideRegs8>();
    constexpr int kRows = kTile / kWideWarps;  // of a warp
    const int cw = (warp - 12) % kWideWarps;
    const uint32_t group = (uint32_t)(warp - 12) / kWideWarps;
    const int span = (lane >> 3) & 1, ch = (lane & 3) + 4 * span;
    const int g = ((lane >> 2) & 1) + 2 * (lane >> 4);
    uint32_t k = 0;
    while (ok && walk.next(t, ctl, s)) {
      for (int idx = 0; ok && idx < 2 * s.n; ++idx, ++k) {
        if ((k & 1u) != group) continue;
        bool is_v;
        int tile;
        tile_of(idx, s.n, is_v, tile);
        const int key0 = (s.t0 + tile) * kTile;
        const uint32_t rs = Slot(k, rc).i, slot = Slot(k, rt).i;
        const Slot from(k, rc2), to(k, rt2);
        if (!wait_warp(ctl.rawfull + from.i, from.ph, guard, kWaitRaw) ||
            !wait_warp(ctl.empty + to.i, to.i < rt.n ? to.ph ^ 1u : to.ph, guard, kWaitWide)) {
          ok = false;
          break;
        }
        // only the part's first and last tiles hold rows that nobody sees: those
        // become zeros whatever they hold
        const int row0 = key0 + kRows * cw;
        const bool edge = row0 < s.lo || row0 + kRows > s.hi;
        if (ch * 16 < D) {
#pragma unroll 1
          for (int q = kRows * cw + g; q < kRows * (cw + 1); q += 16) {
            const uint8_t* src = raw + (size_t)rs * raw_bytes + q * D + ch * 16;
            uint8_t* dst = ring + (size_t)slot * stage_bytes + span * kSpan + q * 128;
            const uint8_t* scales = scale_area + rs * kTile + q;
            uint4 x[4];
            uint32_t sc[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              x[p] = *reinterpret_cast<const uint4*>(src + 4 * p * D);
              sc[p] = scales[4 * p];
            }
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
              uint32_t o[8];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 u = e4m3x2((uint16_t)w[j]), v = e4m3x2((uint16_t)(w[j] >> 16));
                o[2 * j] = scaled<DT>(u, sc[p]);
                o[2 * j + 1] = scaled<DT>(v, sc[p]);
              }
              if (edge && (key0 + q + 4 * p < s.lo || key0 + q + 4 * p >= s.hi)) {
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = 0;
              }
              const int sw = (4 * p + g) & 7, c1 = 2 * (lane & 3);  // (q is g and a multiple of 16)
              *reinterpret_cast<uint4*>(dst + 4 * p * 128 + ((c1 ^ sw) << 4)) =
                  make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4*>(dst + 4 * p * 128 + (((c1 + 1) ^ sw) << 4)) =
                  make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(ctl.full + slot);
          mbar_arrive(ctl.rawempty + Slot(k + rc.n, rc2).i);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 512);
  if (threadIdx.x == 0) t.err[wid] = (ctl.abort ? kLate | ctl.abort << 8 : 0) | ctl.mend;
}

// ---------------------------------------------------------------------------
// The join: items cut by a share's end, and the flags.
// ---------------------------------------------------------------------------
// One row from its parts (at most one per CTA).  The (m, l) of all parts are read at
// once, a part per lane; the warp then adds up every `stride`-th part's O from `first`
// on, 32 lanes by four columns.  Returns this lane's columns; M, L: of all parts.
__device__ __forceinline__ float4 join_parts(const TileArgs& t, int c, int parts, int row, int first,
                                             int stride, float& M, float& L) {
  constexpr int kSets = (kMaxCtas + 31) / 32;
  const int lane = threadIdx.x & 31, D = t.a.c.head_dim;
  auto place = [&](int p) { return (int64_t)(p ? 2 * (c + p) : 2 * c + 1) * kMaxRows + row; };
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

// The products of a tile weigh every value of it, and 0 times an infinity is NaN: a value
// that is not finite reaches rows that do not see it.  So what is not finite in a row's
// outputs is found again, one warp to the row, from the keys that it sees alone.  (Not
// where the sum of the weights is NaN, from the query or a key that the row does see: its
// outputs are NaN by the definition.  Rows like that alone set off no mending.)  sq:
// shared memory for the warp's query.
template <int DT, bool E4M3>
__device__ __forceinline__ void mend_row(const AttendArgs& a, int t, int hq, float* sq) {
  const int lane = threadIdx.x & 31, D = a.c.head_dim;
  __syncwarp();  // the row's stores
  if (a.lse) {
    const float lse = __ldcg(a.lse + (int64_t)t * a.heads + hq);
    if (lse != lse) return;
  }
  uint4 w = make_uint4(0, 0, 0, 0);
  uint4* at = reinterpret_cast<uint4*>(a.out + ((int64_t)t * a.heads + hq) * D * 2) + lane;
  if (lane * 8 < D) w = __ldcg(at);
  uint32_t v[4] = {w.x, w.y, w.z, w.w};
  bool odd = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = F16<DT>::up(v[e]);
    odd |= !(fabsf(f.x) < kInf && fabsf(f.y) < kInf);
  }
  if (!__any_sync(0xffffffffu, odd)) return;
  const int b = owner_of(a.b.q_start, a.b.B, t, a.b.total);
  if (b >= a.b.B) return;
  const Seq q = load_seq(a.b, b, a.c.page_size);
  const int i = t - q.tok0;
  if (i < 0 || i >= q.n) return;
  const int hi = max(0, q.pos0 + i + 1);
  const int lo = a.window && hi > a.window ? hi - a.window : 0;
  const char* qrow = a.q + (int64_t)t * a.q_token + (int64_t)hq * a.q_head;
  for (int d = lane; d < D / 2; d += 32) {
    const float2 f = F16<DT>::up(__ldg(reinterpret_cast<const uint32_t*>(qrow) + d));
    sq[2 * d] = f.x * a.scale_log2;
    sq[2 * d + 1] = f.y * a.scale_log2;
  }
  __syncwarp();
  float m = -kInf, l = 0.0f, o[8] = {};
  attend_blocks<DT, E4M3, 1>(a, b, hq / (a.heads / a.c.kv_heads), lo, hi, sq, 0, 1, m, l, o);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
  __syncwarp();
  if (lane * 8 >= D) return;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = F16<DT>::up(v[e]);
    const uint32_t y = F16<DT>::down(o[2 * e] * inv, o[2 * e + 1] * inv);
    if (!(fabsf(f.x) < kInf)) v[e] = (v[e] & 0xffff0000u) | (y & 0xffffu);
    if (!(fabsf(f.y) < kInf)) v[e] = (v[e] & 0xffffu) | (y & 0xffff0000u);
  }
  *at = make_uint4(v[0], v[1], v[2], v[3]);
}

template <int DT, bool E4M3>
__global__ void __launch_bounds__(kJoinThreads) k_attend_join(const __grid_constant__ TileArgs t,
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
      odd |= L == L && !(fabsf(o.x * inv + o.y * inv + o.z * inv + o.w * inv) < kInf);
      const uint2 w = make_uint2(F16<DT>::down(o.x * inv, o.y * inv),
                                 F16<DT>::down(o.z * inv, o.w * inv));
      reinterpret_cast<uint2*>(a.out + orow * D * 2)[lane] = w;
    }
    if (lane == 0 && a.lse) a.lse[orow] = lse_of(M, L);
  }
  if (!__syncthreads_or(odd || (err & kMend))) return;
  // rare: the rows joined here, and those that the tile kernel wrote itself
  float* sq = reinterpret_cast<float*>(so[warp]);
  if (!wide || !warp)
    for (int j = begin; j < total; j += step) {
      int c, tok, hd;
      locate(j, c, tok, hd);
      mend_row<DT, E4M3>(a, rec[c].row0 + tok, rec[c].h * t.group + hd, sq);
    }
  if (!__syncthreads_or(err & kMend)) return;
  const int64_t rows = (int64_t)a.b.total * a.heads;
  for (int64_t j = (int64_t)blockIdx.x * kWarps + warp; j < rows; j += (int64_t)join_blocks * kWarps) {
    const int tok = (int)(j / a.heads), hq = (int)(j - (int64_t)tok * a.heads);
    bool cut = false;
    for (int c = lane; c < ctas; c += 32)
      cut |= rec[c].more && rec[c].h == hq / t.group && tok >= rec[c].row0 &&
             tok - rec[c].row0 < rec[c].ntok;
    if (!__any_sync(0xffffffffu, cut)) mend_row<DT, E4M3>(a, tok, hq, sq);
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

std::mutex g_mu;
EncodeTiled g_encode = nullptr;
int g_sms[64] = {};

cudaError_t device_ready(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_mu);
  if (!g_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
    g_encode = reinterpret_cast<EncodeTiled>(fn);
  }
  if (!g_sms[dev]) {
    const struct {
      const void* kernel;
      int regs;
    } all[] = {{(const void*)k_attend_tiles<SV_BF16, false>, kRegs16},
               {(const void*)k_attend_tiles<SV_F16, false>, kRegs16},
               {(const void*)k_attend_tiles<SV_BF16, true>, kRegs8},
               {(const void*)k_attend_tiles<SV_F16, true>, kRegs8}};
    for (const auto& k : all) {
      cudaFuncAttributes attr{};
      e = cudaFuncGetAttributes(&attr, k.kernel);
      if (e != cudaSuccess) return e;
      if (attr.numRegs < k.regs) return cudaErrorInvalidKernelImage;  // the roles' shares count on them
      e = cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)kSmemBytes);
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

// A pool [pages][kv_heads][page_size][dim] by its strides (in bytes), one box of
// `span` entries and `box` tokens at a time.
bool encode_pool(CUtensorMap* map, const CacheView& c, const void* base, CUtensorMapDataType type,
                 CUtensorMapSwizzle swizzle, int span, int box) {
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size,
                              (cuuint64_t)c.kv_heads, (cuuint64_t)c.num_pages};
  // a dimension of one entry is never stepped along: any legal stride will do
  const cuuint64_t strides[3] = {(cuuint64_t)c.token_bytes,
                                 (cuuint64_t)(c.kv_heads > 1 ? c.head_bytes : c.token_bytes),
                                 (cuuint64_t)(c.num_pages > 1 ? c.page_bytes : c.token_bytes)};
  const cuuint32_t bx[4] = {(cuuint32_t)span, (cuuint32_t)box, 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return g_encode(map, type, 4, const_cast<void*>(base), dims, strides, bx, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries [total][heads][dim] by their strides, tpt tokens by group heads at a time.
bool encode_queries(CUtensorMap* map, const AttendArgs& a, int dim, int group, int tpt) {
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)a.heads, (cuuint64_t)a.b.total};
  // a dimension of one entry is never stepped along: any legal stride will do
  const cuuint64_t row = (cuuint64_t)dim * 2;
  const cuuint64_t strides[2] = {a.heads > 1 ? (cuuint64_t)a.q_head : row,
                                 a.b.total > 1 ? (cuuint64_t)a.q_token : row};
  const cuuint32_t bx[3] = {64, (cuuint32_t)group, (cuuint32_t)tpt};
  const cuuint32_t one[3] = {1, 1, 1};
  return a.b.total > 0 &&
         g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<char*>(a.q), dims, strides,
                  bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Ring make_ring(int n, int most) {
  const uint32_t k = (uint32_t)(n < most ? n : most);
  return Ring{k, (uint32_t)((0x100000000ull + k - 1) / k)};
}

constexpr size_t kRecBytes = 4096, kMlBytes = sizeof(float2) * 2 * kMaxCtas * kMaxRows;
static_assert(kMaxCtas * (sizeof(Rec) + sizeof(int)) <= kRecBytes, "records");

}  // namespace

void set_attention_stall(int cta, long long clocks) {
  g_stall_cta = cta;
  g_wait_clocks = clocks > 0 ? clocks : kWaitClocks;
}

size_t attention_tiles_workspace(int head_dim) {
  return kRecBytes + kMlBytes + sizeof(float) * 2 * kMaxCtas * kMaxRows * (size_t)head_dim;
}

cudaError_t launch_attention_tiles(const AttendArgs& a, int dtype, bool e4m3, cudaStream_t stream,
                                   bool* taken) {
  int sms = 0;
  cudaError_t e = device_ready(&sms);
  if (e != cudaSuccess) return e;
  const CacheView& c = a.c;
  TileArgs t{};
  t.a = a;
  t.group = a.heads / c.kv_heads;
  t.tpt = kTile / t.group;
  t.nhalf = c.head_dim > 64 ? 2 : 1;
  const int stage = t.nhalf * kSpan, codes = kTile * c.head_dim;
  for (int two = 0; two < 2; ++two) {
    const int spare = two ? 0 : kQBytes;
    t.tiles[two] = make_ring(e4m3 ? kRing8 / stage : (kRing16 + spare) / stage, kMaxStages);
    t.codes[two] = make_ring((kCodes + spare) / codes, kMaxRaw);
    t.tiles2[two] = make_ring(2 * t.tiles[two].n, 2 * kMaxStages);
    t.codes2[two] = make_ring(2 * t.codes[two].n, 2 * kMaxRaw);
  }
  t.box = c.page_size < kTile ? c.page_size : kTile;
  t.wide = ((uintptr_t)a.out & 31) == 0;
  t.stall = g_stall_cta;
  t.wait_clocks = g_wait_clocks;
  // a second warp fetches from four copies a tile on (32 sequences of e4m3 in pages of
  // 64: 552 -> 466 us; one sequence of 64-wide heads in pages of 128: 36 us with one
  // warp, 40 with two)
  t.fetchers = kTile / t.box * (e4m3 ? 2 : t.nhalf) >= 4 ? 2 : 1;
  // a scale of zero: every finite product times 2^-149 is below 2^-20, and the -inf of a
  // key that is not seen stays one
  t.c = a.scale_log2 == 0.0f ? 0x1p-149f : a.scale_log2;
  t.rec = reinterpret_cast<Rec*>(a.ws);
  t.err = reinterpret_cast<int*>(a.ws + kMaxCtas * sizeof(Rec));
  t.ml = reinterpret_cast<float2*>(a.ws + kRecBytes);
  t.part = reinterpret_cast<float*>(a.ws + kRecBytes + kMlBytes);
  alignas(64) CUtensorMap mq{}, mk{}, mv{};
  *taken = encode_queries(&mq, a, c.head_dim, t.group, t.tpt);
  if (e4m3) {
    *taken = *taken &&
             encode_pool(&mk, c, c.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE,
                         c.head_dim, t.box) &&
             encode_pool(&mv, c, c.v, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE,
                         c.head_dim, t.box);
  } else {
    *taken = *taken &&
             encode_pool(&mk, c, c.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         CU_TENSOR_MAP_SWIZZLE_128B, 64, t.box) &&
             encode_pool(&mv, c, c.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         CU_TENSOR_MAP_SWIZZLE_128B, 64, t.box);
  }
  if (!*taken) return cudaSuccess;
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  auto* k = dtype == SV_BF16 ? (e4m3 ? k_attend_tiles<SV_BF16, true> : k_attend_tiles<SV_BF16, false>)
                             : (e4m3 ? k_attend_tiles<SV_F16, true> : k_attend_tiles<SV_F16, false>);
  e = launch_pdl(k, dim3(ctas), dim3(e4m3 ? kThreads8 : kThreads16), kSmemBytes, stream, mq, mk, mv, t);
  if (e != cudaSuccess) return e;
  // Blocks of the join: two rounds of the three that fit an SM, or for e4m3, whose mending
  // leaves room for two, one round (round of 64: 197 us, with two an SM 200; e4m3 round 449,
  // with four 452), but no more blocks than rows.
  const int64_t rows = (int64_t)a.b.total * a.heads;
  const int most = (e4m3 ? 2 : 6) * ctas;
  const int join_blocks = (int)(rows < most ? rows : most);
  const int flag_blocks = a.flags ? (a.b.B + kJoinThreads / 32 - 1) / (kJoinThreads / 32) : 0;
  auto* j = dtype == SV_BF16 ? (e4m3 ? k_attend_join<SV_BF16, true> : k_attend_join<SV_BF16, false>)
                             : (e4m3 ? k_attend_join<SV_F16, true> : k_attend_join<SV_F16, false>);
  return launch_pdl(j, dim3(join_blocks + flag_blocks), dim3(kJoinThreads), 0, stream, t, ctas,
                    join_blocks);
}

}  // namespace sv
