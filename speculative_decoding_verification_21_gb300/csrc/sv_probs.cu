// sv_probs.cu -- spec_verify_probs: the round from given probabilities and given
// uniforms.
//
//   n = first i with not (u_i <= p_i(x_i) / q_i(x_i)), else gamma
//   w = max(0, p_n - q_n) (p_n where that is empty, p_gamma for n = gamma)
//   t = smallest v with W_v > u W_{V-1},  W_v = w_0 + ... + w_v
//
// Bound by HBM: the rows p_n and q_n are read once, 2 V values per batch row.  A
// row is cut over a cluster of CTAs and their warps; each warp sums its run of
// the row, the totals are exchanged through shared memory (distributed between
// the CTAs), and the one warp whose run holds the target reads that run again
// (from L2) and stops inside it.  W is an integer in units of 2^-61, so the split
// changes nothing, and the target floor(u W) is exact: u = m 2^-e with a 24-bit m,
// so u W is a 128-bit product shifted right.
//
// Units without 64-bit conversions or shifts (those bound the kernel at three times
// the time of its reads): adding a constant M rounds w to a multiple of M's last
// place, and the sum's bits less M's are that multiple.  Three constants peel w into
// multiples of 2^-21, 2^-44 and 2^-61; what each leaves is exact in fp32.  Two
// entries share an instruction, and the three 32-bit sums of a batch of entries are
// put together in 64 bits once a batch.
//
// Measured on GB300: 256 rows of 152064 fp32 (269 MB) 65 us, 4.1 TB/s (0.61 of a copy's
// rate: the search behind a row's reads leaves the memory idle, and only other rows' CTAs
// fill the gap); one row of 32000 6 us.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "specverify.h"
#include "sv_device.cuh"
#include "sv_launch.h"
#include "sv_plan.h"
#include "sv_tma.cuh"

namespace sv {
namespace {

namespace cg = cooperative_groups;

constexpr int kProbWarps = 8;
constexpr int kProbThreads = kProbWarps * 32;
constexpr int kProbMaxCluster = 8;

struct ProbArgs {
  const void* p;
  const void* q;
  const int32_t* x;
  const float* u;
  int B, gamma;
  int64_t V;
  int32_t* out_tokens;
  int32_t* out_counts;
  uint8_t* out_flags;
};

// A probability as given: 0 where it is none (and `odd` is set).
__device__ __forceinline__ float sane(float p, bool& odd) {
  const bool ok = p >= 0.0f && p <= 2.0f;
  odd |= !ok;
  return ok ? p : 0.0f;
}

// Constants whose last places are 2^-21, 2^-44 and 2^-61.
constexpr float kM1 = 4.0f, kM2 = 1.5f * 0x1p-21f, kM3 = 1.5f * 0x1p-38f;

// Sums of the three parts' bits over a batch; the constants' own bits are taken off
// at its end.
struct Parts {
  uint32_t a = 0, b = 0, c = 0;
};

// Two weights 0 <= w <= 2 into the parts.
__device__ __forceinline__ void add_parts(Parts& s, float w0, float w1) {
  const uint64_t w = pack2(w0, w1), minus = pack2(-1.0f, -1.0f);
  const uint64_t t1 = fadd2(w, pack2(kM1, kM1));
  const uint64_t l1 = ffma2(fadd2(t1, pack2(-kM1, -kM1)), minus, w);
  const uint64_t t2 = fadd2(l1, pack2(kM2, kM2));
  const uint64_t l2 = ffma2(fadd2(t2, pack2(-kM2, -kM2)), minus, l1);
  const uint64_t t3 = fadd2(l2, pack2(kM3, kM3));
  float x, y;
  unpack2(t1, x, y);
  s.a += __float_as_uint(x) + __float_as_uint(y);
  unpack2(t2, x, y);
  s.b += __float_as_uint(x) + __float_as_uint(y);
  unpack2(t3, x, y);
  s.c += __float_as_uint(x) + __float_as_uint(y);
}
// The batch's sum in units of 2^-61 (n entries, n <= 64: no part passes 31 bits).
__device__ __forceinline__ unsigned long long units(const Parts& s, int n) {
  const int a = (int)(s.a - (uint32_t)n * __float_as_uint(kM1));
  const int b = (int)(s.b - (uint32_t)n * __float_as_uint(kM2));
  const int c = (int)(s.c - (uint32_t)n * __float_as_uint(kM3));
  return (unsigned long long)(((long long)a << 40) + ((long long)b << 17) + c);
}
// One weight.
__device__ __forceinline__ unsigned long long units(float w) {
  Parts s;
  add_parts(s, w, 0.0f);
  return units(s, 2);
}

// floor(u w) for 0 <= u < 1.
__device__ __forceinline__ unsigned long long times(float u, unsigned long long w) {
  const uint32_t bits = __float_as_uint(u);
  const int e = (int)(bits >> 23);  // u = m 2^(e - 150) (e = 0: m 2^-149, no hidden bit)
  const unsigned long long m = e ? ((bits & 0x7fffffu) | 0x800000u) : (bits & 0x7fffffu);
  const int sh = 150 - (e ? e : 1);  // >= 24
  const unsigned long long hi = __umul64hi(w, m), lo = w * m;
  if (sh >= 128) return 0;
  if (sh >= 64) return hi >> (sh - 64);
  return (hi << (64 - sh)) | (lo >> sh);
}

struct Weights {
  const void* p;
  const void* q;  // null: w = p
};

// Weights of elements i .. i+N-1 of the row (N consecutive ones, aligned if VEC).
template <int DT, bool VEC>
struct Piece {
  static constexpr int N = VEC ? VecInfo<DT>::kElems : 1;
};

// Raw vectors (or single entries) of p and q, and the weights that they hold.
template <int DT, bool VEC>
struct Entry;
template <int DT>
struct Entry<DT, true> {
  uint4 p, q;
  __device__ __forceinline__ void load(const Weights& r, int64_t i) {
    constexpr int es = DT == SV_F32 ? 4 : 2;
    p = ld_stream16((const char*)r.p + i * es);
    q = r.q ? ld_stream16((const char*)r.q + i * es) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float* fp, float* fq) const {
    unpack<DT>(p, fp);
    unpack<DT>(q, fq);
  }
};
template <int DT>
struct Entry<DT, false> {
  float p, q;
  __device__ __forceinline__ void load(const Weights& r, int64_t i) {
    p = load_logit<DT>(r.p, i);
    q = r.q ? load_logit<DT>(r.q, i) : 0.0f;
  }
  __device__ __forceinline__ void get(float* fp, float* fq) const {
    fp[0] = p;
    fq[0] = q;
  }
};

// max(0, p - q) of one entry's values.  A value is a probability for certain when
// neither of its two highest bits is set (0 <= p < 2); only where some is set is each
// looked at by itself.
template <int N>
__device__ __forceinline__ void weights_of(float* fp, float* fq, float* w, bool& odd) {
  uint32_t all = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) all |= __float_as_uint(fp[j]) | __float_as_uint(fq[j]);
  if (all & 0xC0000000u) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      fp[j] = sane(fp[j], odd);
      fq[j] = sane(fq[j], odd);
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) w[j] = fmaxf(0.0f, fp[j] - fq[j]);
}

template <int DT, bool VEC>
__device__ __forceinline__ void load_weights(const Weights& r, int64_t i, float* w, bool& odd) {
  constexpr int N = Piece<DT, VEC>::N;
  Entry<DT, VEC> e;
  float fp[N], fq[N];
  e.load(r, i);
  e.get(fp, fq);
  weights_of<N>(fp, fq, w, odd);
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct ProbShared {
  unsigned long long warp_total[kProbWarps];
  unsigned long long total;
  int any;   // some weight of this CTA is positive
  int odd;   // some value was no probability
  int n, flags;
};

// The accept tests of batch row b (one warp): n, and the flags they raise (lane 0's).
struct Accept {
  int n, flags;
};
template <int DT>
__device__ Accept accept_tests(const ProbArgs& a, int b) {
  const int lane = threadIdx.x & 31, g = a.gamma;
  bool ok = false, bad_token = false, odd = false;
  if (lane < g) {
    const int x = __ldg(a.x + (int64_t)b * g + lane);
    const float u = __ldg(a.u + (int64_t)b * (g + 1) + lane);
    float p = 0.0f, q = 0.0f;
    bad_token = x < 0 || (int64_t)x >= a.V;
    if (!bad_token) {
      p = sane(load_logit<DT>(a.p, ((int64_t)b * (g + 1) + lane) * a.V + x), odd);
      q = sane(load_logit<DT>(a.q, ((int64_t)b * g + lane) * a.V + x), odd);
    }
    ok = u <= p / q;
    odd |= !(u >= 0.0f && u < 1.0f) || (!bad_token && q == 0.0f);
  }
  const unsigned fail = __ballot_sync(0xffffffffu, lane < g && !ok);
  const int n = fail ? __ffs(fail) - 1 : g;
  // only what was tested says something about the round
  const unsigned seen = n >= 31 ? 0xffffffffu : (2u << n) - 1u;
  const unsigned bt = __ballot_sync(0xffffffffu, bad_token) & seen;
  const unsigned od = __ballot_sync(0xffffffffu, odd) & seen;
  return Accept{n, (bt ? SV_FLAG_BAD_TOKEN : 0) | (od ? SV_FLAG_NONFINITE : 0)};
}

// The accept tests of all rows ahead of the rows' reads, one warp to a row: out_counts
// holds n and, above 8 bits, the flags, until the row's own CTAs have ended.
constexpr int kAcceptWarps = 4;
template <int DT>
__global__ void __launch_bounds__(kAcceptWarps * 32) k_accept(ProbArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = (int)blockIdx.x * kAcceptWarps + (int)(threadIdx.x >> 5);
  if (b >= a.B) return;
  const Accept t = accept_tests<DT>(a, b);
  if ((threadIdx.x & 31) == 0) a.out_counts[b] = t.n | t.flags << 8;
}

// This warp's run of the row: its share of the CTA's slice.
struct Run {
  int64_t lo, hi;
};
template <int DT, bool VEC>
__device__ __forceinline__ Run run_of(int64_t V, int parts, int part) {
  constexpr int N = Piece<DT, VEC>::N;
  const int64_t pieces = V / N;  // VEC: V is a multiple of N
  return Run{pieces * part / parts * N, pieces * (part + 1) / parts * N};
}

template <int DT, bool VEC>
__device__ __forceinline__ unsigned long long sum_run(const Weights& r, Run run, bool& any,
                                                      bool& odd) {
  constexpr int N = Piece<DT, VEC>::N, U = VEC ? 4 : 8;  // entries of a batch in flight
  const int lane = threadIdx.x & 31;
  unsigned long long s = 0;
  uint32_t some = 0;  // bits of any weight
  for (int64_t i = run.lo + (int64_t)lane * N; i < run.hi; i += U * 32 * N) {
    Entry<DT, VEC> e[U];
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (k == 0 || i + k * 32 * N < run.hi) e[k].load(r, i + k * 32 * N);
      else e[k] = Entry<DT, VEC>{};
    Parts parts;
    float last = 0.0f;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      float fp[N], fq[N], w[N];
      e[k].get(fp, fq);
      weights_of<N>(fp, fq, w, odd);
#pragma unroll
      for (int j = 0; j < N; ++j) some |= __float_as_uint(w[j]);
      if (N == 1) {  // two single entries make a pair
        if (k & 1) add_parts(parts, last, w[0]);
        last = w[0];
      } else {
#pragma unroll
        for (int j = 0; j + 1 < N; j += 2) add_parts(parts, w[j], w[j + 1]);
      }
    }
    s += units(parts, U * N);
  }
  any |= some != 0;
  return s;
}

// The first element of the run at which the running sum, `before` in front of
// the run, passes `target`; -1 if none does.  Four pieces are read at a time, so that
// the search waits for memory once in 512 entries.
template <int DT, bool VEC>
__device__ int64_t find_in_run(const Weights& r, Run run, unsigned long long before,
                               unsigned long long target) {
  constexpr int N = Piece<DT, VEC>::N, U = 4;
  const int lane = threadIdx.x & 31;
  bool odd = false;
  for (int64_t base = run.lo; base < run.hi; base += U * 32 * N) {
    Entry<DT, VEC> e[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t i = base + (k * 32 + lane) * N;
      if (i < run.hi) e[k].load(r, i);
      else e[k] = Entry<DT, VEC>{};
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      float fp[N], fq[N], w[N];
      e[k].get(fp, fq);
      weights_of<N>(fp, fq, w, odd);
      unsigned long long mine = 0;
#pragma unroll
      for (int j = 0; j < N; ++j) mine += units(w[j]);
      unsigned long long scan = mine;  // inclusive over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + scan > target);
      if (hit) {
        const int l = __ffs(hit) - 1;
        int at = 0;
        if (lane == l) {
          unsigned long long c = before + scan - mine;
          bool found = false;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            c += units(w[j]);
            if (!found && c > target) {
              at = j;
              found = true;
            }
          }
        }
        at = __shfl_sync(0xffffffffu, at, l);
        return base + (int64_t)(k * 32 + l) * N + at;
      }
      before += __shfl_sync(0xffffffffu, scan, 31);
    }
  }
  return -1;
}

template <int DT, bool VEC, bool AHEAD>
__global__ void __launch_bounds__(kProbThreads, 4) k_verify_probs(ProbArgs a) {
  __shared__ ProbShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int b = (int)(blockIdx.x / C), g = a.gamma;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  if (threadIdx.x == 0) {
    sh.any = 0;
    sh.odd = 0;
  }
  if (AHEAD) {
    if (threadIdx.x == 0) {
      const int packed = a.out_counts[b];
      sh.n = packed & 255;
      sh.flags = packed >> 8;
    }
  } else if (warp == 0) {
    const Accept t = accept_tests<DT>(a, b);
    if (lane == 0) {
      sh.n = t.n;
      sh.flags = t.flags;
    }
  }
  __syncthreads();
  const int n = sh.n;
  constexpr int es = DT == SV_F32 ? 4 : 2;
  Weights r;
  r.p = (const char*)a.p + ((int64_t)b * (g + 1) + n) * a.V * es;
  r.q = n < g ? (const char*)a.q + ((int64_t)b * g + n) * a.V * es : nullptr;
  const Run run = run_of<DT, VEC>(a.V, C * kProbWarps, rank * kProbWarps + warp);
  int flags = sh.flags;
  unsigned long long total = 0, before = 0;
  bool cluster_any = false, cluster_odd = false;
  // once, and again on p_n where the residual is empty
  for (int pass = 0; pass < 2; ++pass) {
    bool any = false, odd = false;
    const unsigned long long mine = warp_sum(sum_run<DT, VEC>(r, run, any, odd));
    any = __any_sync(0xffffffffu, any);
    odd = __any_sync(0xffffffffu, odd);
    if (lane == 0) {
      sh.warp_total[warp] = mine;
      if (any) sh.any = 1;
      if (odd) sh.odd = 1;
    }
    __syncthreads();
    if (warp == 0) {
      const unsigned long long s = warp_sum(lane < kProbWarps ? sh.warp_total[lane] : 0ull);
      if (lane == 0) sh.total = s;
    }
    cluster.sync();
    total = before = 0;
    cluster_any = false;
    for (int c = 0; c < C; ++c) {
      const ProbShared* o = cluster.map_shared_rank(&sh, c);
      const unsigned long long s = o->total;
      if (c < rank) before += s;
      total += s;
      cluster_any |= o->any != 0;
      cluster_odd |= o->odd != 0;
    }
    cluster.barrier_arrive();  // its totals are read: the wait stands where they change or end
    if (cluster_any || !r.q) break;
    cluster.barrier_wait();
    flags |= SV_FLAG_RESIDUAL_FALLBACK;
    r.q = nullptr;
  }
  float u = __ldg(a.u + (int64_t)b * (g + 1) + g);
  if (!(u >= 0.0f && u < 1.0f)) {
    flags |= SV_FLAG_NONFINITE;
    u = u >= 1.0f ? 0x1.fffffep-1f : 0.0f;
  }
  if (cluster_odd) flags |= SV_FLAG_NONFINITE;
  if (!cluster_any) flags |= SV_FLAG_ZERO_MASS;
  const unsigned long long target = times(u, total);
  int32_t* out = a.out_tokens + (int64_t)b * (g + 1);
  for (int w = 0; w < warp; ++w) before += sh.warp_total[w];
  if (total > 0 && before <= target && target < before + sh.warp_total[warp]) {
    const int64_t t = find_in_run<DT, VEC>(r, run, before, target);
    if (lane == 0) out[n] = (int32_t)(t < 0 ? 0 : t);
  }
  if (rank == 0) {
    if (threadIdx.x <= g && (int)threadIdx.x != n)
      out[threadIdx.x] = (int)threadIdx.x < n ? __ldg(a.x + (int64_t)b * g + threadIdx.x) : -1;
    if (threadIdx.x == 0) {
      if (total == 0) out[n] = 0;  // no mass (or none as large as a unit)
      a.out_counts[b] = n;
      if (a.out_flags) a.out_flags[b] = (uint8_t)flags;
    }
  }
  cluster.barrier_wait();
}

template <int DT>
cudaError_t launch_dt(const ProbArgs& a, int cluster, cudaStream_t stream) {
  constexpr int es = DT == SV_F32 ? 4 : 2;
  // 16-byte loads where every row starts on a 16-byte boundary
  const bool vec = (a.V * es) % 16 == 0;
  // More CTAs than stand at once (four to an SM): each would begin with the accept tests'
  // three dependent loads while its share of the memory idles, so they go ahead in a
  // kernel of their own (256 rows of 152064: 68 us without it, 65 with; one row takes 6 us
  // either way, but the call a launch more: 18.7 us of the host instead of 17.7).
  const bool ahead = (int64_t)a.B * cluster > 4 * 152;
  if (ahead) {
    const cudaError_t e = launch_pdl(k_accept<DT>, dim3((a.B + kAcceptWarps - 1) / kAcceptWarps),
                                     dim3(kAcceptWarps * 32), 0, stream, a);
    if (e != cudaSuccess) return e;
  }
  auto* k = vec ? (ahead ? k_verify_probs<DT, true, true> : k_verify_probs<DT, true, false>)
                : (ahead ? k_verify_probs<DT, false, true> : k_verify_probs<DT, false, false>);
  return launch_pdl_cluster(k, dim3((unsigned)(a.B * cluster)), dim3(kProbThreads), 0,
                            (unsigned)cluster, stream, a);
}

}  // namespace

cudaError_t launch_verify_probs(const void* p, const void* q, const int32_t* x, const float* u,
                                int B, int gamma, int64_t V, int dtype, int32_t* out_tokens,
                                int32_t* out_counts, uint8_t* out_flags, cudaStream_t stream) {
  const ProbArgs a{p, q, x, u, B, gamma, V, out_tokens, out_counts, out_flags};
  // CTAs per batch row: as many as give each of 152 SMs a dozen (a batch of 256 rows of
  // 152064: 72 us with 2048 CTAs of 256 threads, 100 us with 512; an SM then has rows of
  // one and of two vectors to read, and others' reads while one searches), while a CTA
  // keeps at least 2048 entries.
  int c = 1;
  while (c < kProbMaxCluster && (int64_t)B * c < 2048 && V / (2 * c) >= 2048) c *= 2;
  return dtype == SV_F32 ? launch_dt<SV_F32>(a, c, stream) : launch_dt<SV_BF16>(a, c, stream);
}

}  // namespace sv
