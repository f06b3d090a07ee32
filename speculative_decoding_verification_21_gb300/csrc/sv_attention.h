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

size_t attention_workspace_bytes(int head_dim);
cudaError_t launch_attention(const AttendArgs& a, int dtype, bool e4m3, cudaStream_t stream);

}  // namespace sv
