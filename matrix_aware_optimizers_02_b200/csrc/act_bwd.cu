// dz = dy act'(z), rounded to the activations' type for the two products that read it, with
// the column sums of the unrounded dz for the bias gradient in the same pass.
//
// HBM-bound: dy 2 + z 2 (or 1 + 1/32 from a checkpoint) + dz 2 bytes per element.  A lane
// owns 8 columns, a block 256 columns of a chunk of rows; each chunk leaves one partial row
// of column sums, joined in order by a second kernel (no atomics: the same bits every run).
#include "act_bwd.h"

namespace mao {
namespace {

struct ActArgs {
  const void* dy;
  const void* z;
  CkptView k;
  void* dz;     // nullptr: column sums only
  float* part;  // [chunks][cols], or nullptr
  long long ld_dy, ld_z, ld_dz;
  int rows, cols, chunk;
};

constexpr int kRowsInFlight = 4;

template <class T, int ACT, bool KEPT>
__global__ void __launch_bounds__(256) act_bwd_kernel(const ActArgs a) {
  __shared__ float2 sh[8][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * 8;
  const long long r_end = min((long long)a.rows, ((long long)blockIdx.y + 1) * a.chunk);
  f2 sum[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) sum[j] = dup2(0.0f);
  if (c < a.cols) {
    for (long long r0 = (long long)blockIdx.y * a.chunk + warp; r0 < r_end; r0 += 8 * kRowsInFlight) {
      Vec8<T> g[kRowsInFlight];
      Vec8<T> z[kRowsInFlight];
      CkptVec8 zk[kRowsInFlight];
#pragma unroll
      for (int i = 0; i < kRowsInFlight; ++i) {
        const long long r = r0 + 8 * i;
        if (r < r_end) {
          g[i].load(static_cast<const T*>(a.dy) + r * a.ld_dy + c);
          if constexpr (ACT != MAO_ACT_NONE) {
            if constexpr (KEPT) zk[i].load(a.k, r, c);
            else z[i].load(static_cast<const T*>(a.z) + r * a.ld_z + c);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kRowsInFlight; ++i) {
        const long long r = r0 + 8 * i;
        if (r < r_end) {
          f2 d[4];
          g[i].get(d);
          if constexpr (ACT != MAO_ACT_NONE) {
            f2 f[4];
            if constexpr (KEPT) zk[i].get(f);
            else z[i].get(f);
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = mul2(d[j], act_slope<ACT>(f[j]));
            Vec8<T> o;
            o.set(d);
            if (a.dz != nullptr) o.store(static_cast<T*>(a.dz) + r * a.ld_dz + c);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[j] = add2(sum[j], d[j]);
        }
      }
    }
  }
  if (a.part == nullptr) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) sh[warp][lane * 4 + j] = sum[j];
  __syncthreads();
  const float* p = reinterpret_cast<const float*>(sh);
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) s += p[w * 256 + threadIdx.x];
  const int col = blockIdx.x * 256 + threadIdx.x;
  if (col < a.cols) a.part[(long long)blockIdx.y * a.cols + col] = s;
}

template <class T, bool KEPT>
mao_status run(const ActArgs& a, int act, dim3 grid, cudaStream_t s) {
  switch (act) {
    case MAO_ACT_NONE: act_bwd_kernel<T, MAO_ACT_NONE, false><<<grid, 256, 0, s>>>(a); break;
    case MAO_ACT_RELU: act_bwd_kernel<T, MAO_ACT_RELU, KEPT><<<grid, 256, 0, s>>>(a); break;
    case MAO_ACT_RELU2: act_bwd_kernel<T, MAO_ACT_RELU2, KEPT><<<grid, 256, 0, s>>>(a); break;
    case MAO_ACT_GELU: act_bwd_kernel<T, MAO_ACT_GELU, KEPT><<<grid, 256, 0, s>>>(a); break;
    case MAO_ACT_GELU_TANH: act_bwd_kernel<T, MAO_ACT_GELU_TANH, KEPT><<<grid, 256, 0, s>>>(a); break;
    case MAO_ACT_SILU: act_bwd_kernel<T, MAO_ACT_SILU, KEPT><<<grid, 256, 0, s>>>(a); break;
    default: return MAO_ERR_INVALID_ARG;
  }
  return launched();
}

}  // namespace

// About eight waves of the three blocks that an SM of a B200 holds, so that the last wave's
// idle share is small, at least 32 rows each; chunks <= 3552 fits grid.y.
int act_bwd_chunk(int rows, int cols) {
  const int strips = (cols + 255) / 256;
  const int want = std::max(1, 3552 / strips);
  const int chunks = std::max(1, std::min(want, (rows + 31) / 32));
  return (rows + chunks - 1) / chunks;
}

mao_status act_bwd_launch(const void* dy, long long ld_dy, const void* z, long long ld_z, const CkptView& k, bool kept,
                          int act, int dtype, int rows, int cols, void* dz, long long ld_dz, float* part,
                          cudaStream_t stream) {
  ActArgs a;
  a.dy = dy, a.z = z, a.k = k, a.dz = dz, a.part = part;
  a.ld_dy = ld_dy, a.ld_z = ld_z, a.ld_dz = ld_dz;
  a.rows = rows, a.cols = cols;
  a.chunk = act_bwd_chunk(rows, cols);
  const dim3 grid((cols + 255) / 256, (rows + a.chunk - 1) / a.chunk);
  const double z_bytes = act == MAO_ACT_NONE ? 0.0 : (kept ? 1.0 + 1.0 / 32 : 2.0);
  LaunchScope ls(stream, MAO_K_ACT_BWD, 0.0, (double)rows * cols * (2.0 + z_bytes + (dz ? 2.0 : 0.0)));
  if (dtype == MAO_BF16)
    return kept ? run<__nv_bfloat16, true>(a, act, grid, stream) : run<__nv_bfloat16, false>(a, act, grid, stream);
  return kept ? run<__half, true>(a, act, grid, stream) : run<__half, false>(a, act, grid, stream);
}

}  // namespace mao
