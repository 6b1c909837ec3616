// 8-bit activation checkpoints: written from and read back to fp32, bf16 or fp16
// (format: mao_ckpt8 in mao.h).
//
// Both passes are HBM-bound: a 16-bit element costs 2 + 1 + 1/32 bytes either way.  A lane
// owns 8 columns (16 bytes of a 16-bit type), 4 lanes a block of 32, whose largest magnitude
// takes two shuffles; a thread keeps kUnroll vectors in flight.
#include "ckpt8.cuh"
#include "layer_host.h"

namespace mao {
namespace {

constexpr int kThreads = kCkptThreads;
constexpr int kUnroll = kCkptUnroll;

template <class T>
__global__ void __launch_bounds__(kThreads) ckpt8_kernel(const T* __restrict__ x, long long ld_x, CkptView k, Steps st,
                                                         int cols) {
  Walk at(st, blockIdx.x);
  const long long tile = kThreads * kUnroll;
  // uniform over the block: lanes behind the last vector take part in the shuffles
  for (long long i = blockIdx.x * tile; i < st.total; i += gridDim.x * tile) {
    Vec8<T> v[kUnroll];
    long long row[kUnroll];
    int col[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      row[u] = at.row;
      col[u] = at.v * 8;
      if (at.row < st.rows && col[u] < cols) v[u].load(x + at.row * ld_x + col[u]);
      else v[u].zero();
      at.move(st.dr, st.dv, st.vpr);
    }
    at.move(st.tr, st.tv, st.vpr);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t amax = v[u].block_max();  // 4 | vpr: a block's lanes are all in or all out
      f2 f[4];
      v[u].get(f);
      if (row[u] < st.rows)
        ckpt_store8(k.q + row[u] * k.ld_q + col[u], (col[u] & 31) ? nullptr : k.e + row[u] * k.ld_e + (col[u] >> 5), f, amax);
    }
  }
}

template <class T, int ACT>
__global__ void __launch_bounds__(kThreads) restore_kernel(CkptView k, T* __restrict__ y, long long ld_y, Steps st) {
  restore_block<T, ACT>(k, y, ld_y, st, blockIdx.x);
}

template <class T>
mao_status pack(const void* x, long long ld_x, const CkptView& k, int rows, int cols, cudaStream_t stream) {
  const int vpr = ckpt_blocks(cols) * 4;
  DeviceInfo* dev = nullptr;
  MAO_TRY(device_info(&dev));
  Steps st;
  const unsigned grid = steps_of(rows, vpr, dev->sm_count, &st);
  LaunchScope ls(stream, MAO_K_CKPT8, 0.0, (double)rows * cols * (sizeof(T) + 1.0 + 1.0 / 32));
  ckpt8_kernel<T><<<grid, kThreads, 0, stream>>>(static_cast<const T*>(x), ld_x, k, st, cols);
  return launched();
}

template <class T>
mao_status restore(const CkptView& k, int rows, int cols, int act, void* y, long long ld_y, cudaStream_t stream) {
  const int vpr = cols / 8;
  DeviceInfo* dev = nullptr;
  MAO_TRY(device_info(&dev));
  Steps st;
  const unsigned grid = steps_of(rows, vpr, dev->sm_count, &st);
  T* o = static_cast<T*>(y);
  LaunchScope ls(stream, MAO_K_CKPT8_RESTORE, 0.0, (double)rows * cols * (sizeof(T) + 1.0 + 1.0 / 32));
  switch (act) {
    case MAO_ACT_NONE: restore_kernel<T, MAO_ACT_NONE><<<grid, kThreads, 0, stream>>>(k, o, ld_y, st); break;
    case MAO_ACT_RELU: restore_kernel<T, MAO_ACT_RELU><<<grid, kThreads, 0, stream>>>(k, o, ld_y, st); break;
    case MAO_ACT_RELU2: restore_kernel<T, MAO_ACT_RELU2><<<grid, kThreads, 0, stream>>>(k, o, ld_y, st); break;
    case MAO_ACT_GELU: restore_kernel<T, MAO_ACT_GELU><<<grid, kThreads, 0, stream>>>(k, o, ld_y, st); break;
    case MAO_ACT_GELU_TANH:
      restore_kernel<T, MAO_ACT_GELU_TANH><<<grid, kThreads, 0, stream>>>(k, o, ld_y, st);
      break;
    case MAO_ACT_SILU: restore_kernel<T, MAO_ACT_SILU><<<grid, kThreads, 0, stream>>>(k, o, ld_y, st); break;
    default: return MAO_ERR_INVALID_ARG;
  }
  return launched();
}

}  // namespace

mao_status restore_launch(const CkptView& c, int rows, int cols, int act, void* y, int dtype, long long ld_y,
                          cudaStream_t stream) {
  switch (dtype) {
    case MAO_F32: return restore<float>(c, rows, cols, act, y, ld_y, stream);
    case MAO_BF16: return restore<__nv_bfloat16>(c, rows, cols, act, y, ld_y, stream);
    default: return restore<__half>(c, rows, cols, act, y, ld_y, stream);
  }
}

}  // namespace mao

using namespace mao;

extern "C" mao_status mao_checkpoint8(const void* x, int32_t dtype, int32_t rows, int32_t cols, int64_t ld_x,
                                      const mao_ckpt8* c, mao_stream_t stream_) {
  if (c == nullptr) return MAO_ERR_INVALID_ARG;
  if (dtype != MAO_F32 && !is16(dtype)) return MAO_ERR_DTYPE;
  MAO_TRY(check_dims(rows, cols));
  MAO_TRY(check_acts(x, rows, cols, ld_x));
  MAO_TRY(check_ckpt(*c, rows, cols));
  DeviceInfo* dev = nullptr;
  MAO_TRY(device_info(&dev));
  if (rows == 0) return MAO_OK;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  switch (dtype) {
    case MAO_F32: return pack<float>(x, ld_x, view(*c), rows, cols, stream);
    case MAO_BF16: return pack<__nv_bfloat16>(x, ld_x, view(*c), rows, cols, stream);
    default: return pack<__half>(x, ld_x, view(*c), rows, cols, stream);
  }
}

extern "C" mao_status mao_checkpoint8_restore(const mao_ckpt8* c, int32_t rows, int32_t cols, int32_t act, void* y,
                                              int32_t dtype, int64_t ld_y, mao_stream_t stream_) {
  if (c == nullptr) return MAO_ERR_INVALID_ARG;
  if (dtype != MAO_F32 && !is16(dtype)) return MAO_ERR_DTYPE;
  if (act < MAO_ACT_NONE || act > MAO_ACT_SILU) return MAO_ERR_INVALID_ARG;
  MAO_TRY(check_dims(rows, cols));
  MAO_TRY(check_acts(y, rows, cols, ld_y));
  MAO_TRY(check_ckpt(*c, rows, cols));
  DeviceInfo* dev = nullptr;
  MAO_TRY(device_info(&dev));
  if (rows == 0) return MAO_OK;
  return restore_launch(view(*c), rows, cols, act, y, dtype, ld_y, reinterpret_cast<cudaStream_t>(stream_));
}
