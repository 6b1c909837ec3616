// The elementwise pass of the linear layer's backward (act_bwd.cu).
#pragma once

#include "layer_host.h"

namespace mao {

// Rows per chunk; the pass writes ceil(rows / chunk) partial rows of column sums.
int act_bwd_chunk(int rows, int cols);

// rows, cols >= 1; dz == nullptr: column sums only; part == nullptr: no column sums.
mao_status act_bwd_launch(const void* dy, long long ld_dy, const void* z, long long ld_z, const CkptView& k, bool kept,
                          int act, int dtype, int rows, int cols, void* dz, long long ld_dz, float* part,
                          cudaStream_t stream);

}  // namespace mao
