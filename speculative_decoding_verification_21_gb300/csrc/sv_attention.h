// sv_attention.h -- the arguments of spec_chunk_attention's kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "sv_cache.cuh"

namespace sv {

struct AttendArgs {
  CacheView c;
  BatchView b;
  const char* q;
  int64_t q_token, q_head;  // strides of the queries in bytes
  int heads;
  float scale_log2;         // scale * log2 e: scores are kept in log2 units
  int window;
  char* out;
  float* lse;
  uint8_t* flags;
  char* ws;
};

// Whether the tile kernel takes a cache: head_dim up to 128, and pages of a power of two
// of tokens (they divide a tile of 128 or are whole tiles), at least 8 (one swizzle
// group), or 16 where their scale bytes are copied 16 at a time.  The row kernel takes the rest,
// and negative scales (a row's maximum is then not its largest product).
inline bool tiles_take(const CacheView& c, bool e4m3) {
  if (c.head_dim > 128 || c.num_pages == 0) return false;
  if (!e4m3) return c.page_shift >= 3;
  return c.page_shift >= 4 && ((uintptr_t)c.ks | (uintptr_t)c.vs) % 16 == 0;
}

// Flags of sequence b (one warp): its lengths, and the pages of the keys it sees.
__device__ __forceinline__ uint8_t sequence_flags(const AttendArgs& a, int b) {
  const Seq q = load_seq(a.b, b, a.c.page_size);
  bool bad = false;
  if (q.n) {
    const int first = q.pos0 + 1;
    const int lo = a.window && first > a.window ? first - a.window : 0;
    for (int p = lo / a.c.page_size + (threadIdx.x & 31); (int64_t)p * a.c.page_size < q.len; p += 32) {
      const int page = __ldg(a.b.table + (int64_t)b * a.b.max_pages + p);
      bad |= page < 0 || page >= a.c.num_pages;
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  return (uint8_t)((q.bad ? SV_FLAG_BAD_LENGTH : 0) | (bad ? SV_FLAG_BAD_PAGE : 0));
}

// cache_dtype: the sv_dtype of the cache; group: query heads to a key head.
size_t attention_workspace_bytes(const CacheView& c, int cache_dtype, int group);
size_t attention_tiles_workspace(int head_dim);
cudaError_t launch_attention(const AttendArgs& a, int dtype, int cache_dtype, cudaStream_t stream);
cudaError_t launch_attention_rows_u4(const AttendArgs& a, int dtype, cudaStream_t stream);

// Whether the tile kernel of 4-bit caches takes one: head_dim up to 128, pages of a power of
// two of tokens, at least 16, at most 80 query heads to a key head, steps and zeros on
// 16-byte boundaries.
bool u4_tiles_take(const CacheView& c, int group);
size_t attention_u4_workspace(int head_dim);
// *taken = false: the cache cannot be described by a tensor map; nothing was queued.
cudaError_t launch_attention_u4_tiles(const AttendArgs& a, int dtype, cudaStream_t stream, bool* taken);

// Test only (sv_test_attention_stall).
void set_attention_stall(int cta, long long clocks);
struct AttentionTest {
  int stall_cta;         // -1: none
  long long wait_clocks; // limit of a wait
};
AttentionTest attention_test();

// *taken = false: the cache cannot be described by a tensor map; nothing was queued.
cudaError_t launch_attention_tiles(const AttendArgs& a, int dtype, bool e4m3, cudaStream_t stream,
                                   bool* taken);

}  // namespace sv
