// Host side shared by the trained-layer entry points: argument checks and the
// operators that one entry point calls of another.
#pragma once

#include <atomic>
#include <climits>

#include "host_common.h"
#include "layer_math.cuh"

namespace mao {

inline int elem_size(int dtype) { return dtype == MAO_F32 ? 4 : 2; }
inline int ckpt_blocks(int cols) { return (cols + 31) / 32; }
inline bool is16(int dtype) { return dtype == MAO_BF16 || dtype == MAO_F16; }

// rows x cols of activations with the module's row rule (see "trained layers" in mao.h)
inline mao_status check_acts(const void* p, int rows, int cols, long long ld) {
  if (rows > 0 && p == nullptr) return MAO_ERR_INVALID_ARG;
  if (ld < cols || (ld & 7) || ld > (1ll << 36)) return MAO_ERR_SHAPE;
  return aligned16(p) ? MAO_OK : MAO_ERR_ALIGN;
}
// at most 2^30 each way: row and column numbers rounded up to a tile, or a grid past the end,
// stay in 32 bits
inline mao_status check_dims(int rows, int cols) {
  constexpr int most = 1 << 30;
  return (rows < 0 || rows > most || cols < 1 || cols > most || (cols & 7)) ? MAO_ERR_SHAPE : MAO_OK;
}
inline mao_status check_ckpt(const mao_ckpt8& c, int rows, int cols) {
  if (rows > 0 && (c.q == nullptr || c.e == nullptr)) return MAO_ERR_INVALID_ARG;
  if (c.ld_q < cols || (c.ld_q & 31) || c.ld_q > (1ll << 36) || c.ld_e < ckpt_blocks(cols) || c.ld_e > (1ll << 36))
    return MAO_ERR_SHAPE;
  return aligned16(c.q) ? MAO_OK : MAO_ERR_ALIGN;
}
inline CkptView view(const mao_ckpt8& c) { return CkptView{c.q, c.e, c.ld_q, c.ld_e}; }

inline mao_status launched() { return cudaGetLastError() == cudaSuccess ? MAO_OK : MAO_ERR_CUDA; }

// A kernel's dynamic shared memory limit, raised once per device.
template <class K>
mao_status allow_smem(K kern, int bytes, std::atomic<bool> (&done)[64]) {
  int d = 0;
  MAO_CUDA_TRY(cudaGetDevice(&d));  // device_info has bounded it
  if (!done[d].load(std::memory_order_acquire)) {
    MAO_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    done[d].store(true, std::memory_order_release);
  }
  return MAO_OK;
}

// Launch as a programmatic dependent of the kernel before it in the stream, which must be one
// of this call's: launch latency and set-up overlap that kernel's end.  The kernel calls
// wait_for_previous() before it touches global memory, and takes what the kernel before wrote
// by plain pointers: __restrict__ would say that nothing writes there while it runs, and allow
// read-only loads that the wait does not order.
template <class... P, class... A>
mao_status launch_dependent(void (*kern)(P...), dim3 grid, int block, int smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(block);
  c.dynamicSmemBytes = smem;
  c.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, args...) == cudaSuccess ? MAO_OK : MAO_ERR_CUDA;
}

// y = act(value of c); arguments checked by the caller, rows >= 1
mao_status restore_launch(const CkptView& c, int rows, int cols, int act, void* y, int dtype, long long ld_y,
                          cudaStream_t stream);

// out[col] = sum over parts of part[p * cols + col], in a fixed order; follows the kernel that
// wrote the parts
mao_status col_sum_launch(const float* part, int parts, int cols, float* out, cudaStream_t stream);

}  // namespace mao
