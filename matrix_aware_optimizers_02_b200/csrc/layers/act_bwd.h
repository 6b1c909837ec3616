// The elementwise pass of the linear layer's backward (act_bwd.cu).
#pragma once

#include "layer_host.h"

namespace mao {

// Rows per chunk; the pass writes ceil(rows / chunk) partial rows of column sums.
int act_bwd_chunk(int rows, int cols);

struct ActBwd {
  const void* dy;
  long long ld_dy;
  const void* z;  // nullptr: read zk
  long long ld_z;
  CkptView zk;
  int act;
  int rows, cols;  // of dy; rows >= 1
  void* dz;        // nullptr: not written (no activation: dz is dy)
  long long ld_dz;
  float* part;     // partial column sums of dz, or nullptr
  CkptView xk;     // read back to xr (rows x x_cols, dense), unless that is nullptr
  void* xr;
  int x_cols;
};

mao_status act_bwd_launch(const ActBwd& b, int dtype, cudaStream_t stream);

}  // namespace mao
