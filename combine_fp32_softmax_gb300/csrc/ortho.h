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

}  // namespace moe
