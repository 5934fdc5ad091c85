// Softmax cross entropy over a vocabulary (host launchers).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace moe {

struct XentArgs {
  int T, V, d;
  const uint16_t* x;
  const uint16_t* W;
  const void* target;
  int target_type;
  float* loss;  // written by the forward, read by the backward
  float* lse;
  // backward
  const float* dloss;
  const float* dlse;
  void* dx;
  void* dW;
  int dx_type, dW_type;
  void* ws;
  int grid_limit;
};

size_t xent_workspace_bytes(int T, int V, int d, int backward);
// Both return MOE_OK or a negative MOE_ERR_*.
int launch_xent_fwd(const XentArgs& a, cudaStream_t s);
int launch_xent_bwd(const XentArgs& a, cudaStream_t s);

}  // namespace moe
