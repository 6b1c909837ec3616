// 8-bit activation checkpoints: written from and read back to fp32, bf16 or fp16
// (format: mao_ckpt8 in mao.h).
//
// Both passes are HBM-bound: a 16-bit element costs 2 + 1 + 1/32 bytes either way.  A lane
// owns 8 columns (16 bytes of a 16-bit type), 4 lanes a block of 32, whose largest magnitude
// takes two shuffles; a thread keeps kUnroll vectors in flight.
#include "layer_host.h"

namespace mao {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;

// Vector index -> (row, column).  `vpr` vectors per row, rows padded to whole blocks.
struct Split {
  long long row;
  int col;
  __device__ __forceinline__ Split(long long i, int vpr) {
    if (i < (1ll << 32)) {
      const uint32_t r = (uint32_t)i / (uint32_t)vpr;
      row = r;
      col = ((uint32_t)i - r * (uint32_t)vpr) * 8;
    } else {
      row = i / vpr;
      col = (int)(i - row * vpr) * 8;
    }
  }
};

template <class T>
__global__ void __launch_bounds__(kThreads) ckpt8_kernel(const T* __restrict__ x, long long ld_x, CkptView k,
                                                         long long total, int vpr, int cols) {
  const long long base = (long long)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  Vec8<T> v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = base + u * kThreads;
    v[u].zero();
    if (i < total) {
      const Split s(i, vpr);
      if (s.col < cols) v[u].load(x + s.row * ld_x + s.col);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = base + u * kThreads;
    const Split s(i < total ? i : 0, vpr);
    float f[8];
    v[u].get(f);
    ckpt_store8(k, s.row, s.col, f, i < total);  // 4 | vpr: a block's lanes are all in or all out
  }
}

template <class T, int ACT>
__global__ void __launch_bounds__(kThreads) restore_kernel(CkptView k, T* __restrict__ y, long long ld_y,
                                                           long long total, int vpr) {
  const long long base = (long long)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
  CkptVec8 v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = base + u * kThreads;
    if (i < total) {
      const Split s(i, vpr);
      v[u].load(k, s.row, s.col);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const long long i = base + u * kThreads;
    if (i >= total) continue;
    const Split s(i, vpr);
    float f[8];
    v[u].get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = act_value<ACT, sizeof(T) == 4>(f[j]);
    Vec8<T> o;
    o.set(f);
    o.store(y + s.row * ld_y + s.col);
  }
}

bool grid_of(long long total, unsigned* grid) {
  const long long g = (total + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  *grid = (unsigned)g;
  return g <= INT_MAX;
}

template <class T>
mao_status pack(const void* x, long long ld_x, const CkptView& k, int rows, int cols, cudaStream_t stream) {
  const int vpr = ckpt_blocks(cols) * 4;
  const long long total = (long long)rows * vpr;
  unsigned grid;
  if (!grid_of(total, &grid)) return MAO_ERR_SHAPE;
  LaunchScope ls(stream, MAO_K_CKPT8, 0.0, (double)rows * cols * (sizeof(T) + 1.0 + 1.0 / 32));
  ckpt8_kernel<T><<<grid, kThreads, 0, stream>>>(static_cast<const T*>(x), ld_x, k, total, vpr, cols);
  return launched();
}

template <class T>
mao_status restore(const CkptView& k, int rows, int cols, int act, void* y, long long ld_y, cudaStream_t stream) {
  const int vpr = cols / 8;
  const long long total = (long long)rows * vpr;
  unsigned grid;
  if (!grid_of(total, &grid)) return MAO_ERR_SHAPE;
  T* o = static_cast<T*>(y);
  LaunchScope ls(stream, MAO_K_CKPT8_RESTORE, 0.0, (double)rows * cols * (sizeof(T) + 1.0 + 1.0 / 32));
  switch (act) {
    case MAO_ACT_NONE: restore_kernel<T, MAO_ACT_NONE><<<grid, kThreads, 0, stream>>>(k, o, ld_y, total, vpr); break;
    case MAO_ACT_RELU: restore_kernel<T, MAO_ACT_RELU><<<grid, kThreads, 0, stream>>>(k, o, ld_y, total, vpr); break;
    case MAO_ACT_RELU2: restore_kernel<T, MAO_ACT_RELU2><<<grid, kThreads, 0, stream>>>(k, o, ld_y, total, vpr); break;
    case MAO_ACT_GELU: restore_kernel<T, MAO_ACT_GELU><<<grid, kThreads, 0, stream>>>(k, o, ld_y, total, vpr); break;
    case MAO_ACT_GELU_TANH:
      restore_kernel<T, MAO_ACT_GELU_TANH><<<grid, kThreads, 0, stream>>>(k, o, ld_y, total, vpr);
      break;
    case MAO_ACT_SILU: restore_kernel<T, MAO_ACT_SILU><<<grid, kThreads, 0, stream>>>(k, o, ld_y, total, vpr); break;
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
