// Layer norm and its gradient (mao_layer_norm, mao_layer_norm_backward).
//
// Both are HBM-bound, one pass over the activations: a row lives in the registers of the
// G threads that own it (8 * VPT consecutive-by-8 columns each) from its load to its store.
// Blocks walk rows with a stride, so a thread's columns stay the same: the weight and the
// bias are read once per block, the next row's loads are issued before the present row's
// reductions, and in the backward pass the column sums of dw and db accumulate in
// registers, each block leaving one partial row for a second, small kernel.
//
// Mean and variance: two passes over the registers (sum of x, then of (x - mean)^2), so
// a large mean costs no digits.
#include "layer_host.h"

namespace mao {
namespace {

// Sums of N values over the G threads of a row; every thread of the block calls this.
// `sh` holds N floats per warp; two buffers alternate between calls, so one barrier per
// call is enough: a buffer is written again only after the barrier of the call between.
template <int G, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if constexpr (G > 32) {
    constexpr int W = G / 32;  // warps of a row
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) sh[warp * N + i] = v[i];
    }
    __syncthreads();
    const float* r = sh + (warp / W) * W * N;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += r[w * N + i];
  }
}

template <int G>
constexpr int kBlock = G < 128 ? 128 : G;

// ------------------------------------------------------------------ forward
struct FwdArgs {
  const void* x;
  const void* w;
  const void* b;
  void* y;
  float* mean;
  float* rstd;
  CkptView k;
  long long ld_x, ld_y;
  int rows, cols;
  int w_f32;
  float eps, inv_cols;
};

template <class T, int G, int VPT>
__global__ void __launch_bounds__(kBlock<G>) norm_kernel(const FwdArgs a) {
  constexpr int B = kBlock<G>, R = B / G;  // rows per block at a time
  __shared__ float sh[2][32];
  const int t = threadIdx.x % G;
  const int cols = a.cols;
  const T* x = static_cast<const T*>(a.x);
  float w[VPT][8], b[VPT][8];
  Vec8<T> next[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * G + t) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = b[i][j] = 0.0f;
    if (c < cols) {
      load_param8<T>(a.w, a.w_f32, c, w[i]);
      if (a.b != nullptr) load_param8<T>(a.b, a.w_f32, c, b[i]);
    }
  }
  const long long step = (long long)gridDim.x * R;
  long long row = (long long)blockIdx.x * R + threadIdx.x / G;
  auto fetch = [&](long long r) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * G + t) * 8;
      if (r < a.rows && c < cols) next[i].load(x + r * a.ld_x + c);
      else next[i].zero();
    }
  };
  fetch(row);
  // the trip count is the block's: rows behind the last take part in the reductions
  for (long long r0 = (long long)blockIdx.x * R; r0 < a.rows; r0 += step, row += step) {
    float v[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) next[i].get(v[i]);
    fetch(row + step);
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] += v[i][j];
    row_sum<G, 1>(s, sh[0]);
    const float mean = s[0] * a.inv_cols;
    s[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const bool in = (i * G + t) * 8 < cols;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] -= mean;
        if (in) s[0] = fmaf(v[i][j], v[i][j], s[0]);
      }
    }
    row_sum<G, 1>(s, sh[1]);
    const float rstd = 1.0f / sqrtf(s[0] * a.inv_cols + a.eps);
    const bool live = row < a.rows;
    if (live && t == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * G + t) * 8;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = fmaf(v[i][j] * rstd, w[i][j], b[i][j]);
      Vec8<T> p;
      p.set(o);
      if (live && c < cols) p.store(static_cast<T*>(a.y) + row * a.ld_y + c);
      if (a.k.q != nullptr) {
        // the checkpoint is of y as stored; lanes behind the last column hold zeros
        p.get(o);
        if (c >= cols) {
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = 0.0f;
        }
        ckpt_store8(a.k, row, c, o, live && (c & ~31) < cols);
      }
    }
  }
}

// ------------------------------------------------------------------ backward
struct BwdArgs {
  const void* dy;
  const void* x;
  const void* w;
  const void* dres;
  void* dx;
  const float* mean;
  const float* rstd;
  float* part;  // [2][gridDim.x][cols]: partial sums of dw, then of db (each only if asked for)
  CkptView k;
  long long ld_dy, ld_x, ld_dres, ld_dx;
  int rows, cols;
  int w_f32;
  float inv_cols;
};

template <class T, bool KEPT>
struct XVec {
  Vec8<T> v;
  __device__ __forceinline__ void load(const BwdArgs& a, long long r, int c) {
    v.load(static_cast<const T*>(a.x) + r * a.ld_x + c);
  }
  __device__ __forceinline__ void zero() { v.zero(); }
  __device__ __forceinline__ void get(float (&f)[8]) const { v.get(f); }
};
template <class T>
struct XVec<T, true> {
  CkptVec8 v;
  __device__ __forceinline__ void load(const BwdArgs& a, long long r, int c) { v.load(a.k, r, c); }
  __device__ __forceinline__ void zero() { v.zero(); }
  __device__ __forceinline__ void get(float (&f)[8]) const { v.get(f); }
};

template <class T, bool KEPT, int G, int VPT>
__global__ void __launch_bounds__(kBlock<G>) norm_bwd_kernel(const BwdArgs a) {
  constexpr int B = kBlock<G>, R = B / G;
  __shared__ float sh[2][64];
  const int t = threadIdx.x % G;
  const int cols = a.cols;
  const T* dy = static_cast<const T*>(a.dy);
  float w[VPT][8], dw[VPT][8], db[VPT][8];
  Vec8<T> next_g[VPT];
  XVec<T, KEPT> next_x[VPT];
  float next_mean = 0.0f, next_rstd = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * G + t) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = dw[i][j] = db[i][j] = 0.0f;
    if (c < cols) load_param8<T>(a.w, a.w_f32, c, w[i]);
  }
  const long long step = (long long)gridDim.x * R;
  long long row = (long long)blockIdx.x * R + threadIdx.x / G;
  auto fetch = [&](long long r) {
    const bool in_rows = r < a.rows;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * G + t) * 8;
      if (in_rows && c < cols) {
        next_g[i].load(dy + r * a.ld_dy + c);
        next_x[i].load(a, r, c);
      } else {
        next_g[i].zero();
        next_x[i].zero();
      }
    }
    next_mean = in_rows ? a.mean[r] : 0.0f;
    next_rstd = in_rows ? a.rstd[r] : 0.0f;
  };
  fetch(row);
  int buf = 0;
  for (long long r0 = (long long)blockIdx.x * R; r0 < a.rows; r0 += step, row += step, buf ^= 1) {
    const float mean = next_mean, rstd = next_rstd;
    const bool live = row < a.rows;
    float u[VPT][8], h[VPT][8];
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const bool in = live && (i * G + t) * 8 < cols;
      next_g[i].get(u[i]);
      next_x[i].get(h[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] = in ? (h[i][j] - mean) * rstd : 0.0f;
        dw[i][j] = fmaf(u[i][j], h[i][j], dw[i][j]);
        db[i][j] += u[i][j];
        u[i][j] *= w[i][j];
        s[0] += u[i][j];
        s[1] = fmaf(u[i][j], h[i][j], s[1]);
      }
    }
    Vec8<T> res[VPT];
    if (a.dres != nullptr) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * G + t) * 8;
        if (live && c < cols) res[i].load(static_cast<const T*>(a.dres) + row * a.ld_dres + c);
        else res[i].zero();
      }
    }
    fetch(row + step);
    row_sum<G, 2>(s, sh[buf]);
    const float mu = s[0] * a.inv_cols, mh = s[1] * a.inv_cols;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * G + t) * 8;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = rstd * (u[i][j] - mu - h[i][j] * mh);
      if (a.dres != nullptr) {
        float r[8];
        res[i].get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += r[j];
      }
      Vec8<T> p;
      p.set(o);
      if (live && c < cols) p.store(static_cast<T*>(a.dx) + row * a.ld_dx + c);
    }
  }
  if (a.part == nullptr) return;
  // the block's column sums: its R row groups joined in a fixed order
  float* pw = a.part + (long long)blockIdx.x * cols;
  float* pb = pw + (long long)gridDim.x * cols;
  if constexpr (R == 1) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * G + t) * 8;
      if (c < cols) {
        Vec8<float> p;
        p.set(dw[i]);
        p.store(pw + c);
        p.set(db[i]);
        p.store(pb + c);
      }
    }
  } else {
    __shared__ float acc[R][G * 8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[threadIdx.x / G][t * 8 + j] = which ? db[i][j] : dw[i][j];
        __syncthreads();
        for (int e = threadIdx.x; e < G * 8; e += B) {
          float sum = 0.0f;
#pragma unroll
          for (int r = 0; r < R; ++r) sum += acc[r][e];
          const int c = i * G * 8 + e;
          if (c < cols) (which ? pb : pw)[c] = sum;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ column reduction
// One warp-wide column strip per block: 32 columns x 8 lanes of parts, joined in a fixed
// order, so the sums do not depend on how blocks are scheduled.
__global__ void __launch_bounds__(256) col_reduce_kernel(const float* __restrict__ part, int parts, int cols,
                                                         float* __restrict__ out) {
  __shared__ float sh[8][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31);
  const int g = threadIdx.x >> 5;
  float s = 0.0f;
  if (c < cols)
    for (int p = g; p < parts; p += 8) s += part[(long long)p * cols + c];
  sh[g][threadIdx.x & 31] = s;
  __syncthreads();
  if (g == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sh[i][threadIdx.x];
    out[c] = s;
  }
}

// ------------------------------------------------------------------ dispatch
// (G threads, VPT vectors of 8) per row: the fewest vectors per thread that keep a row in
// at most 1024 threads, two where the row allows, so that two loads are in flight.
#define MAO_NORM_SIZES(CALL)              \
  if (cols <= 256) CALL(32, 1)            \
  else if (cols <= 512) CALL(32, 2)       \
  else if (cols <= 1024) CALL(64, 2)      \
  else if (cols <= 2048) CALL(128, 2)     \
  else if (cols <= 4096) CALL(256, 2)     \
  else if (cols <= 8192) CALL(512, 2)     \
  else if (cols <= 16384) CALL(1024, 2)   \
  else CALL(1024, 4)

// Blocks of a walk over `rows`: as many as are resident at once, never more than there is
// work for.  The backward pass writes 8 * cols bytes of partial sums per block.
int threads_of(int cols) {
  int b = 0;
#define MAO_CASE(G, V) b = kBlock<G>;
  MAO_NORM_SIZES(MAO_CASE)
#undef MAO_CASE
  return b;
}
int rows_per_block(int cols) {
  int r = 0;
#define MAO_CASE(G, V) r = kBlock<G> / G;
  MAO_NORM_SIZES(MAO_CASE)
#undef MAO_CASE
  return r;
}
int walk_blocks(int rows, int cols, int sm_count, int threads_per_sm) {
  const int per_sm = std::max(1, threads_per_sm / threads_of(cols));
  const int rpb = rows_per_block(cols);
  return std::min((rows + rpb - 1) / rpb, per_sm * sm_count);
}
constexpr int kFwdThreads = 1024, kBwdThreads = 512;  // resident threads per SM that registers allow
constexpr int kSizingSms = 160;                       // at least the SMs of any sm_100 part, for workspace sizes

template <class T>
mao_status fwd(const FwdArgs& a, int sms, cudaStream_t stream) {
  const int cols = a.cols;
  const int grid = walk_blocks(a.rows, cols, sms, kFwdThreads);
  LaunchScope ls(stream, MAO_K_LAYER_NORM, 0.0,
                 (double)a.rows * cols * (2.0 * sizeof(T) + (a.k.q ? 1.0 + 1.0 / 32 : 0.0)));
#define MAO_CASE(G, V) norm_kernel<T, G, V><<<grid, kBlock<G>, 0, stream>>>(a);
  MAO_NORM_SIZES(MAO_CASE)
#undef MAO_CASE
  return launched();
}

template <class T, bool KEPT>
mao_status bwd(const BwdArgs& a, int grid, cudaStream_t stream) {
  const int cols = a.cols;
  LaunchScope ls(stream, MAO_K_LAYER_NORM_BWD, 0.0,
                 (double)a.rows * cols * (2.0 * sizeof(T) + (KEPT ? 1.0 + 1.0 / 32 : sizeof(T)) + (a.dres ? sizeof(T) : 0)));
#define MAO_CASE(G, V) norm_bwd_kernel<T, KEPT, G, V><<<grid, kBlock<G>, 0, stream>>>(a);
  MAO_NORM_SIZES(MAO_CASE)
#undef MAO_CASE
  return launched();
}

mao_status check_w(int w_dtype, int dtype) {
  return (w_dtype == MAO_F32 || w_dtype == dtype) ? MAO_OK : MAO_ERR_DTYPE;
}

mao_status check_bwd(const mao_layer_norm_backward_args* a) {
  if (a == nullptr) return MAO_ERR_INVALID_ARG;
  if (a->dtype != MAO_F32 && !is16(a->dtype)) return MAO_ERR_DTYPE;
  MAO_TRY(check_w(a->w_dtype, a->dtype));
  MAO_TRY(check_dims(a->rows, a->cols));
  if (a->cols > MAO_LAYER_NORM_MAX_COLS) return MAO_ERR_UNSUPPORTED;
  return MAO_OK;
}

size_t bwd_bytes(const mao_layer_norm_backward_args* a, int sms) {
  if (a->dw == nullptr && a->db == nullptr) return 0;
  return sizeof(float) * 2 * (size_t)walk_blocks(a->rows, a->cols, sms, kBwdThreads) * (size_t)a->cols;
}

}  // namespace

mao_status col_reduce_launch(const float* part, int parts, int cols, float* out, cudaStream_t stream) {
  LaunchScope ls(stream, MAO_K_COL_REDUCE, 0.0, 4.0 * (double)parts * cols);
  col_reduce_kernel<<<(cols + 31) / 32, 256, 0, stream>>>(part, parts, cols, out);
  return launched();
}

}  // namespace mao

using namespace mao;

extern "C" mao_status mao_layer_norm(const mao_layer_norm_args* a, mao_stream_t stream_) {
  if (a == nullptr) return MAO_ERR_INVALID_ARG;
  if (a->dtype != MAO_F32 && !is16(a->dtype)) return MAO_ERR_DTYPE;
  MAO_TRY(check_w(a->w_dtype, a->dtype));
  MAO_TRY(check_dims(a->rows, a->cols));
  if (a->cols > MAO_LAYER_NORM_MAX_COLS) return MAO_ERR_UNSUPPORTED;
  if (a->w == nullptr || !(a->eps >= 0.0f)) return MAO_ERR_INVALID_ARG;
  MAO_TRY(check_acts(a->x, a->rows, a->cols, a->ld_x));
  MAO_TRY(check_acts(a->y, a->rows, a->cols, a->ld_y));
  if (a->rows > 0 && (a->mean == nullptr || a->rstd == nullptr)) return MAO_ERR_INVALID_ARG;
  if (!aligned16(a->w) || !aligned16(a->b)) return MAO_ERR_ALIGN;
  if (a->yc.q != nullptr) MAO_TRY(check_ckpt(a->yc, a->rows, a->cols));
  DeviceInfo* dev = nullptr;
  MAO_TRY(device_info(&dev));
  if (a->rows == 0) return MAO_OK;
  FwdArgs f;
  f.x = a->x, f.w = a->w, f.b = a->b, f.y = a->y, f.mean = a->mean, f.rstd = a->rstd;
  f.k = view(a->yc);
  f.ld_x = a->ld_x, f.ld_y = a->ld_y;
  f.rows = a->rows, f.cols = a->cols;
  f.w_f32 = a->w_dtype == MAO_F32;
  f.eps = a->eps;
  f.inv_cols = 1.0f / (float)a->cols;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  switch (a->dtype) {
    case MAO_F32: return fwd<float>(f, dev->sm_count, stream);
    case MAO_BF16: return fwd<__nv_bfloat16>(f, dev->sm_count, stream);
    default: return fwd<__half>(f, dev->sm_count, stream);
  }
}

extern "C" mao_status mao_layer_norm_backward_workspace_size(const mao_layer_norm_backward_args* a, size_t* bytes) {
  if (bytes == nullptr) return MAO_ERR_INVALID_ARG;
  MAO_TRY(check_bwd(a));
  *bytes = align_up(bwd_bytes(a, kSizingSms), 256);
  return MAO_OK;
}

extern "C" mao_status mao_layer_norm_backward(const mao_layer_norm_backward_args* a, void* workspace, size_t ws_bytes,
                                              mao_stream_t stream_) {
  MAO_TRY(check_bwd(a));
  if (a->w == nullptr) return MAO_ERR_INVALID_ARG;
  const bool kept = a->x == nullptr && a->xc.q != nullptr;
  MAO_TRY(check_acts(a->dy, a->rows, a->cols, a->ld_dy));
  if (kept) {
    MAO_TRY(check_ckpt(a->xc, a->rows, a->cols));
  } else {
    MAO_TRY(check_acts(a->x, a->rows, a->cols, a->ld_x));
  }
  if (a->dres != nullptr) MAO_TRY(check_acts(a->dres, a->rows, a->cols, a->ld_dres));
  MAO_TRY(check_acts(a->dx, a->rows, a->cols, a->ld_dx));
  if (a->rows > 0 && (a->mean == nullptr || a->rstd == nullptr)) return MAO_ERR_INVALID_ARG;
  if (!aligned16(a->w) || !aligned16(a->dw) || !aligned16(a->db)) return MAO_ERR_ALIGN;
  const size_t need = align_up(bwd_bytes(a, kSizingSms), 256);
  if (need > 0) {
    if (workspace == nullptr || ws_bytes < need) return MAO_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return MAO_ERR_ALIGN;
  }
  DeviceInfo* dev = nullptr;
  MAO_TRY(device_info(&dev));
  if (dev->sm_count > kSizingSms) return MAO_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (a->rows == 0) {
    if (a->dw) MAO_CUDA_TRY(cudaMemsetAsync(a->dw, 0, sizeof(float) * a->cols, stream));
    if (a->db) MAO_CUDA_TRY(cudaMemsetAsync(a->db, 0, sizeof(float) * a->cols, stream));
    return MAO_OK;
  }
  BwdArgs g;
  g.dy = a->dy, g.x = a->x, g.w = a->w, g.dres = a->dres, g.dx = a->dx;
  g.mean = a->mean, g.rstd = a->rstd;
  g.part = need > 0 ? static_cast<float*>(workspace) : nullptr;
  g.k = view(a->xc);
  g.ld_dy = a->ld_dy, g.ld_x = a->ld_x, g.ld_dres = a->ld_dres, g.ld_dx = a->ld_dx;
  g.rows = a->rows, g.cols = a->cols;
  g.w_f32 = a->w_dtype == MAO_F32;
  g.inv_cols = 1.0f / (float)a->cols;
  const int grid = walk_blocks(a->rows, a->cols, dev->sm_count, kBwdThreads);
  mao_status st;
  switch (a->dtype) {
    case MAO_F32: st = kept ? bwd<float, true>(g, grid, stream) : bwd<float, false>(g, grid, stream); break;
    case MAO_BF16:
      st = kept ? bwd<__nv_bfloat16, true>(g, grid, stream) : bwd<__nv_bfloat16, false>(g, grid, stream);
      break;
    default: st = kept ? bwd<__half, true>(g, grid, stream) : bwd<__half, false>(g, grid, stream); break;
  }
  if (st != MAO_OK) return st;
  if (a->dw) MAO_TRY(col_reduce_launch(g.part, grid, a->cols, a->dw, stream));
  if (a->db) MAO_TRY(col_reduce_launch(g.part + (size_t)grid * a->cols, grid, a->cols, a->db, stream));
  return MAO_OK;
}
