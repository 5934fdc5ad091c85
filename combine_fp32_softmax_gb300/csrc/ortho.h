// Orthogonalised matrices (host launcher).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "common.cuh"

namespace moe {

struct OrthoArgs {
  int mats, rows, cols;
  const void* G;
  int g_type;
  uint16_t* O;
  int steps;
  void* ws;
  int grid_limit;
};

size_t ortho_workspace_bytes(int mats, int rows, int cols);
int launch_ortho(const OrthoArgs& a, cudaStream_t s);
// Matrices whose smaller side is at most 128, while a cluster each runs at one
// time: all steps in one launch (ortho_small.cu).
bool ortho_small(int mats, int rows, int cols);
int launch_ortho_small(const OrthoArgs& a, cudaStream_t s);

}  // namespace moe
