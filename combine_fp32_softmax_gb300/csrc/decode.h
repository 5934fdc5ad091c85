// The layer for a few tokens and its linear form (host launchers; the entry
// points in api.cu check the arguments).
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"

namespace moe {

// One weight array: bf16 (scales null) or 4-bit codes with bf16 scales of
// groups of `group` columns (q4.cuh).
struct DecodeWeight {
  const void* w;
  const uint16_t* scales;
};

struct DecodeArgs {
  moe_cfg c;
  int group;  // 0: bf16 weights
  const float* logits;
  const uint16_t* x;
  DecodeWeight W1, W3, W2;
  void* y;
  int y_type;
  int32_t* topk_idx;
  float* topk_w;
  void* ws;
  int grid_limit;  // most CTAs, 0: no limit
};

struct LinearArgs {
  int T, n, K, group;
  const uint16_t* x;
  DecodeWeight W;
  void* y;
  int y_type;
  void* ws;
  int grid_limit;
};

size_t decode_workspace_bytes(const moe_cfg& c);
size_t linear_workspace_bytes();
// Clears the error word and the counters of either workspace.
int decode_ws_init(void* ws, cudaStream_t s);
int launch_decode(const DecodeArgs& a, cudaStream_t s);
int launch_linear(const LinearArgs& a, cudaStream_t s);

}  // namespace moe
