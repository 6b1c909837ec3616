// Layer norm and its gradient (mao_layer_norm, mao_layer_norm_backward).
//
// Both are HBM-bound, one pass over the activations: a row lives in the registers of the
// G threads that own it (8 * VPT consecutive-by-8 columns each) from its load to its store.
// Blocks walk rows with a stride, so a thread's columns stay the same: the weight and the
// bias are read once per block, and in the backward pass the column sums of dw and db
// accumulate in registers, each block leaving one partial row for a second, small kernel.
// A thread reads its share of the next rows ahead, by cp.async into a ring of its own in
// shared memory: up to 200 KB in flight per SM, where the same loads held in registers, one
// row ahead, left the passes waiting (backward 8191 x 1536 with residual: 49 us).
//
// Mean and variance: two passes over the registers (sum of x, then of (x - m)^2).  m, a rounded
// sum times a rounded reciprocal, is off by a few steps of itself, which a row far from zero
// shows rstd-fold (a constant 10944 in 14336 columns: y off by 0.3).  Rows whose |m| is more than
// kFar deviations therefore sum x - m as well: delta = mean(x - m) corrects the mean, the variance
// (less delta^2) and y, and what is left of the error is a few steps of delta.  Nearer rows skip
// that: m's error, a few 2^-24 of at most kFar deviations, is that of their other roundings
// (16384 x 4096 bf16 with checkpoint: 67.6 us, far rows 76.7, without any of this 65.5).
#include "layer_host.h"

namespace mao {
namespace {

// Sums of N values over the G threads of a row; every thread of the block calls this.
// `sh` holds N floats per warp; two buffers alternate between calls, so one barrier per
// call is enough: a buffer is written again only after the barrier of the call between.
template <int G, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* sh) {
  const bool low = (threadIdx.x & 16) == 0;
  float s = v[0];
  if constexpr (N == 2) {
    // lanes 0-15 go on with the first sum, lanes 16-31 with the second
    const float mine = low ? v[0] : v[1], other = low ? v[1] : v[0];
    s = mine + __shfl_xor_sync(0xffffffffu, other, 16);
  } else {
    s += __shfl_xor_sync(0xffffffffu, s, 16);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if constexpr (G > 32) {
    constexpr int W = G / 32;  // warps of a row
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & (N == 2 ? 15 : 31)) == 0) sh[warp * N + (low ? 0 : 1)] = s;
    __syncthreads();
    const float* r = sh + (warp / W) * W * N;
    f2 p = dup2(0.0f);  // N = 1: even and odd warps; N = 2: the two sums
    if constexpr (W * N >= 4) {
#pragma unroll
      for (int w = 0; w < W * N / 4; ++w) {
        const float4 q = reinterpret_cast<const float4*>(r)[w];
        p = add2(p, add2(make_float2(q.x, q.y), make_float2(q.z, q.w)));
      }
    } else {
      p = *reinterpret_cast<const float2*>(r);
    }
    if constexpr (N == 1) v[0] = p.x + p.y;
    else v[0] = p.x, v[1] = p.y;
  } else if constexpr (N == 1) {
    v[0] = s;
  } else {
    v[0] = __shfl_sync(0xffffffffu, s, 0), v[1] = __shfl_sync(0xffffffffu, s, 16);
  }
}

template <int G>
constexpr int kBlock = G < 128 ? 128 : G;

// Stages of a thread's ring: as deep as kRingBytes of shared memory per SM allow at the
// resident thread count, up to kMostStages; 0, plain loads into registers, where not one
// fits (fp32 rows above 16384 columns).
constexpr int kRingBytes = 200 * 1024;
constexpr int kMostStages = 4;
constexpr int ring_stages(int bytes_per_thread, int resident) {
  const int n = kRingBytes / (bytes_per_thread * resident);
  return n > kMostStages ? kMostStages : n;
}

// Row indices are unsigned: a row ahead of the last one does not overflow.
template <class T>
__device__ __forceinline__ Vec8<T> load_vec(const T* p, bool ok) {
  Vec8<T> x;
  if (ok) x.load(p);
  else x.zero();
  return x;
}

// ------------------------------------------------------------------ forward
constexpr float kFar = 4.0f;

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

constexpr int kFwdThreads = 768;  // resident threads per SM that registers allow (blocks of 1024: one)
template <class T, int G, int VPT>
struct FwdCfg {
  static constexpr int B = kBlock<G>;
  static constexpr int kPerSm = B >= kFwdThreads ? 1 : kFwdThreads / B;
  static constexpr int kStages = ring_stages(VPT * Slot8<T>::kBytes, kPerSm * B);
  static constexpr int kSmem = kStages * VPT * Slot8<T>::kBytes * B;
};

template <class T, bool KEEP, int G, int VPT>
__global__ void __launch_bounds__(kBlock<G>, FwdCfg<T, G, VPT>::kPerSm) norm_kernel(const FwdArgs a) {
  using Cfg = FwdCfg<T, G, VPT>;
  constexpr int B = Cfg::B, R = B / G;  // rows per block at a time
  constexpr int D = Cfg::kStages;
  constexpr uint32_t kVec = Slot8<T>::kBytes * B;  // one vector of every thread
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float sh[3][32];
  const uint32_t slot0 = smem_u32(ring) + threadIdx.x * 16;
  const int t = threadIdx.x % G;
  const int cols = a.cols;
  const uint32_t step = gridDim.x * R, rows = (uint32_t)a.rows;
  const uint32_t row0 = blockIdx.x * R + threadIdx.x / G;
  bool in[VPT];  // vectors inside the row
#pragma unroll
  for (int i = 0; i < VPT; ++i) in[i] = (i * G + t) * 8 < cols;
  // where the row ahead and the present row's results lie, moved on by a step per row
  const T* ahead = static_cast<const T*>(a.x) + (long long)row0 * a.ld_x + t * 8;
  const long long ahead_step = (long long)step * a.ld_x, y_step = (long long)step * a.ld_y;
  T* y = static_cast<T*>(a.y) + (long long)row0 * a.ld_y + t * 8;
  int8_t* kq = a.k.q + (long long)row0 * a.k.ld_q + t * 8;
  uint8_t* ke = a.k.e + (long long)row0 * a.k.ld_e + t / 4;
  const long long kq_step = (long long)step * a.k.ld_q, ke_step = (long long)step * a.k.ld_e;
  uint32_t row_ahead = row0;
  auto fetch = [&](int stage) {
    if (row_ahead < rows) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (in[i]) Slot8<T>::fetch(slot0 + (stage * VPT + i) * kVec, B * 16, ahead + i * G * 8);
    }
    cp_async_commit();
    row_ahead += step;
    ahead += ahead_step;
  };
  if constexpr (D > 0) {
    // slots behind the last column hold zeros for good
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (!in[i]) Slot8<T>::zero(slot0 + (d * VPT + i) * kVec, B * 16);
#pragma unroll
    for (int d = 0; d < D - 1; ++d) fetch(d);
  }
  // the weight and the bias stay in registers, but for rows of 4 vectors a thread, where they would
  // be spilled: those read them anew for each row (4096 x 20480 bf16: 121 us, held and spilled 182)
  constexpr bool kHold = VPT < 4;
  f2 w[kHold ? VPT : 1][4], b[kHold ? VPT : 1][4];
  auto params = [&](int i, f2 (&wi)[4], f2 (&bi)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) wi[j] = bi[j] = dup2(0.0f);
    if (in[i]) {
      load_param8<T>(a.w, a.w_f32, (i * G + t) * 8, wi);
      if (a.b != nullptr) load_param8<T>(a.b, a.w_f32, (i * G + t) * 8, bi);
    }
  };
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) params(i, w[i], b[i]);
  }
  uint32_t row = row0;
  int stage = 0;
  // the trip count is the block's: rows behind the last take part in the reductions, with
  // whatever their slots hold, and write nothing
  for (uint32_t r0 = blockIdx.x * R; r0 < rows; r0 += step, row += step, y += y_step, kq += kq_step, ke += ke_step) {
    const bool live = row < rows;
    f2 v[VPT][4];
    if constexpr (D > 0) {
      // the slot read in the iteration before is free: its values are in registers and used
      fetch(stage == 0 ? D - 1 : stage - 1);
      cp_async_wait<D - 1>();
#pragma unroll
      for (int i = 0; i < VPT; ++i) Slot8<T>::get(slot0 + (stage * VPT + i) * kVec, B * 16).get(v[i]);
      stage = stage >= D - 1 ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) load_vec(ahead + i * G * 8, live && in[i]).get(v[i]);
      ahead += ahead_step;
    }
    f2 p = dup2(0.0f);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) p = add2(p, v[i][j]);
    float s[1] = {p.x + p.y};
    row_sum<G, 1>(s, sh[0]);
    const float m = s[0] * a.inv_cols;
    p = dup2(0.0f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][j] = add2(v[i][j], dup2(-m));
      if (in[i]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) p = fma2(v[i][j], v[i][j], p);
      }
    }
    s[0] = p.x + p.y;
    row_sum<G, 1>(s, sh[1]);
    float var = s[0] * a.inv_cols, mean = m;
    // all threads of a row hold the same sums; a block of two rows has barriers that both take part in
    const bool far = m * m > kFar * kFar * (var + a.eps);
    if ((R > 1 && G > 32) ? __syncthreads_or(far) : far) {
      f2 d = dup2(0.0f);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (in[i]) {
#pragma unroll
          for (int j = 0; j < 4; ++j) d = add2(d, v[i][j]);
        }
      s[0] = d.x + d.y;
      row_sum<G, 1>(s, sh[2]);
      if (far) {
        const float delta = s[0] * a.inv_cols;
        mean += delta;
        var = fmaxf(fmaf(-delta, delta, var), 0.0f);  // not NaN here: far rows compare
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i][j] = add2(v[i][j], dup2(-delta));
      }
    }
    const float rstd = rsqrtf(var + a.eps);  // off by at most 2 steps
    if (live && t == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      f2 o[4];
      if constexpr (!kHold) params(i, w[0], b[0]);
      constexpr int kStep = kHold ? 1 : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fma2(mul2(v[i][j], dup2(rstd)), w[i * kStep][j], b[i * kStep][j]);
      Vec8<T> q;
      q.set(o);
      if (live && in[i]) q.store(y + i * G * 8);
      if constexpr (KEEP) {
        // the checkpoint is of y as stored; lanes behind the last column hold zeros
        if (!in[i]) q.zero();
        const uint32_t amax = q.block_max();
        q.get(o);
        if (live && ((i * G + t) * 8 & ~31) < cols)
          ckpt_store8(kq + i * G * 8, (t & 3) ? nullptr : ke + i * (G / 4), o, amax);
      }
    }
  }
  cp_async_wait<0>();
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
  float* part;  // [2][gridDim.x][cols]: partial sums of dw, then of db
  CkptView k;
  long long ld_dy, ld_x, ld_dres, ld_dx;
  int rows, cols;
  int w_f32;
  float inv_cols;
};

constexpr int kBwdThreads = 512;  // resident threads per SM that registers allow (blocks of 1024: one)
template <class T, bool KEPT, bool RES, int G, int VPT>
struct BwdCfg {
  static constexpr int B = kBlock<G>;
  static constexpr int kPerSm = B >= kBwdThreads ? 1 : kBwdThreads / B;
  static constexpr int kX = KEPT ? 8 : Slot8<T>::kBytes;  // bytes of x per vector
  static constexpr int kVec = Slot8<T>::kBytes * (RES ? 2 : 1) + kX;
  static constexpr int kStages = ring_stages(VPT * kVec, kPerSm * B);
  static constexpr int kSmem = kStages * VPT * kVec * B;
};

template <class T, bool KEPT, bool RES, int G, int VPT>
__global__ void __launch_bounds__(kBlock<G>, BwdCfg<T, KEPT, RES, G, VPT>::kPerSm) norm_bwd_kernel(const BwdArgs a) {
  using Cfg = BwdCfg<T, KEPT, RES, G, VPT>;
  constexpr int B = Cfg::B, R = B / G, D = Cfg::kStages;
  constexpr uint32_t kT = Slot8<T>::kBytes * B;  // bytes of one vector of every thread
  constexpr uint32_t kStage = Cfg::kVec * VPT * B;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) float sh[2][64];
  const uint32_t base = smem_u32(ring);
  const int t = threadIdx.x % G;
  const int cols = a.cols;
  const uint32_t step = gridDim.x * R, rows = (uint32_t)a.rows;
  const uint32_t row0 = blockIdx.x * R + threadIdx.x / G;
  bool in[VPT];  // vectors inside the row
#pragma unroll
  for (int i = 0; i < VPT; ++i) in[i] = (i * G + t) * 8 < cols;
  // where the row ahead and the present row's dx lie, moved on by a step per row
  const T* dy = static_cast<const T*>(a.dy) + (long long)row0 * a.ld_dy + t * 8;
  const T* x = KEPT ? nullptr : static_cast<const T*>(a.x) + (long long)row0 * a.ld_x + t * 8;
  const int8_t* xq = KEPT ? a.k.q + (long long)row0 * a.k.ld_q + t * 8 : nullptr;
  const T* dres = RES ? static_cast<const T*>(a.dres) + (long long)row0 * a.ld_dres + t * 8 : nullptr;
  const long long dy_step = (long long)step * a.ld_dy, x_step = (long long)step * (KEPT ? a.k.ld_q : a.ld_x);
  const long long res_step = (long long)step * a.ld_dres, dx_step = (long long)step * a.ld_dx;
  T* dx = static_cast<T*>(a.dx) + (long long)row0 * a.ld_dx + t * 8;
  auto move_on = [&]() {
    dy += dy_step;
    if constexpr (KEPT) xq += x_step;
    else x += x_step;
    if constexpr (RES) dres += res_step;
  };
  // a stage: VPT vectors of dy, then of dres, then of x
  auto g_slot = [&](int stage, int i) { return base + stage * kStage + i * kT + threadIdx.x * 16; };
  auto r_slot = [&](int stage, int i) { return base + stage * kStage + (VPT + i) * kT + threadIdx.x * 16; };
  auto x_slot = [&](int stage, int i) {
    return base + stage * kStage + (RES ? 2 : 1) * VPT * kT + i * (Cfg::kX * B) + threadIdx.x * (KEPT ? 8 : 16);
  };
  uint32_t row_ahead = row0;
  auto fetch = [&](int stage) {
    if (row_ahead < rows) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (in[i]) {
          Slot8<T>::fetch(g_slot(stage, i), B * 16, dy + i * G * 8);
          if constexpr (KEPT) cp_async8(x_slot(stage, i), xq + i * G * 8);
          else Slot8<T>::fetch(x_slot(stage, i), B * 16, x + i * G * 8);
          if constexpr (RES) Slot8<T>::fetch(r_slot(stage, i), B * 16, dres + i * G * 8);
        }
    }
    cp_async_commit();
    row_ahead += step;
    move_on();
  };
  // a row's statistics and its blocks' bytes come by plain loads into registers, two rows
  // ahead, each row's pair in registers of its own until its turn (passed along from row to row
  // they would be waited for at once)
  struct Small {
    float mean, rstd;
    uint32_t e[VPT];
  };
  const uint8_t* xe = KEPT ? a.k.e + (long long)row0 * a.k.ld_e + t / 4 : nullptr;
  const long long e_step = (long long)step * a.k.ld_e;
  uint32_t row_small = row0;
  auto fetch_small = [&]() {
    Small q;
    const bool ok = row_small < rows;
    q.mean = ok ? a.mean[row_small] : 0.0f;
    q.rstd = ok ? a.rstd[row_small] : 0.0f;
    if constexpr (KEPT) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) q.e[i] = (ok && in[i]) ? xe[i * (G / 4)] : 1u;
      xe += e_step;
    }
    row_small += step;
    return q;
  };
  if constexpr (D > 0) {
    // slots behind the last column hold zeros for good: dy = 0 there, so every term is 0
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (!in[i]) {
          Slot8<T>::zero(g_slot(d, i), B * 16);
          if constexpr (KEPT) sts_zero8(x_slot(d, i));
          else Slot8<T>::zero(x_slot(d, i), B * 16);
          if constexpr (RES) Slot8<T>::zero(r_slot(d, i), B * 16);
        }
#pragma unroll
    for (int d = 0; d < D - 1; ++d) fetch(d);
  }
  launch_dependents();  // the column reduction's blocks, as this kernel's end
  Small even = fetch_small(), odd = fetch_small();
  f2 w[VPT][4], dw[VPT][4], db[VPT][4];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * G + t) * 8;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[i][j] = dw[i][j] = db[i][j] = dup2(0.0f);
    if (c < cols) load_param8<T>(a.w, a.w_f32, c, w[i]);
  }
  uint32_t row = row0;
  int stage = 0;
  auto body = [&](Small& small, float* sums) {
    const bool live = row < rows;  // the same for all of a warp
    if constexpr (D > 0) {
      fetch(stage == 0 ? D - 1 : stage - 1);
      cp_async_wait<D - 1>();
    }
    const Small now = small;
    f2 u[VPT][4], h[VPT][4];
    f2 s0 = dup2(0.0f), s1 = dup2(0.0f);
    if (live) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if constexpr (D > 0) Slot8<T>::get(g_slot(stage, i), B * 16).get(u[i]);
        else load_vec(dy + i * G * 8, in[i]).get(u[i]);
        if constexpr (KEPT) {
          CkptVec8 k;
          if constexpr (D > 0) k.w = lds8(x_slot(stage, i));
          else k.w = in[i] ? *reinterpret_cast<const uint2*>(xq + i * G * 8) : make_uint2(0, 0);
          k.e = now.e[i];
          k.get(h[i]);
        } else {
          if constexpr (D > 0) Slot8<T>::get(x_slot(stage, i), B * 16).get(h[i]);
          else load_vec(x + i * G * 8, in[i]).get(h[i]);
        }
        // behind the last column (0 - mean) rstd could overflow, and dy = 0 times that be NaN
        const float rstd = in[i] ? now.rstd : 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[i][j] = mul2(add2(h[i][j], dup2(-now.mean)), dup2(rstd));
          dw[i][j] = fma2(u[i][j], h[i][j], dw[i][j]);
          db[i][j] = add2(db[i][j], u[i][j]);
          u[i][j] = mul2(u[i][j], w[i][j]);
          s0 = add2(s0, u[i][j]);
          s1 = fma2(u[i][j], h[i][j], s1);
        }
      }
    }
    float s[2] = {s0.x + s0.y, s1.x + s1.y};
    row_sum<G, 2>(s, sums);
    // rstd (u - mean(u) - h mean(u h))
    const f2 mu = dup2(-s[0] * a.inv_cols), mh = dup2(-s[1] * a.inv_cols);
    if (live) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        f2 o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = fma2(h[i][j], mh, add2(u[i][j], mu));
        if constexpr (RES) {
          f2 r[4];
          if constexpr (D > 0) Slot8<T>::get(r_slot(stage, i), B * 16).get(r);
          else load_vec(dres + i * G * 8, in[i]).get(r);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = fma2(o[j], dup2(now.rstd), r[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = mul2(o[j], dup2(now.rstd));
        }
        Vec8<T> p;
        p.set(o);
        if (in[i]) p.store(dx + i * G * 8);
      }
    }
    if constexpr (D > 0) stage = stage >= D - 1 ? 0 : stage + 1;
    else move_on();
    small = fetch_small();
    row += step;
    dx += dx_step;
  };
  for (uint32_t r0 = blockIdx.x * R; r0 < rows; r0 += step) {
    body(even, sh[0]);
    r0 += step;
    if (r0 >= rows) break;
    body(odd, sh[1]);
  }
  cp_async_wait<0>();
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
    __shared__ __align__(16) float acc[R][G * 8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<f2*>(&acc[threadIdx.x / G][t * 8 + 2 * j]) = which ? db[i][j] : dw[i][j];
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
// 32 columns per block, 32 warps over the parts, 4 loads in flight each; joined in a fixed
// order, so the sums do not depend on how blocks are scheduled.  blockIdx.y picks one of two
// sums whose parts lie one behind the other.  No __restrict__: the kernel before may still
// write `part` when this one starts.
__global__ void __launch_bounds__(1024) col_reduce_kernel(const float* part, int parts, int cols, float* out0,
                                                          float* out1) {
  __shared__ float sh[32][33];
  wait_for_previous();
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float* out = blockIdx.y == 0 ? out0 : out1;
  if (out == nullptr) return;
  const float* p = part + (long long)blockIdx.y * parts * cols + c;
  float s = 0.0f;
  if (c < cols) {
    int i = g;
    for (; i + 96 < parts; i += 128) {
      const float v0 = p[(long long)i * cols], v1 = p[(long long)(i + 32) * cols], v2 = p[(long long)(i + 64) * cols],
                  v3 = p[(long long)(i + 96) * cols];
      s += (v0 + v1) + (v2 + v3);
    }
    for (; i < parts; i += 32) s += p[(long long)i * cols];
  }
  sh[g][lane] = s;
  __syncthreads();
  // warp g sums column g of the strip: lane by lane, then by shuffles in a fixed tree
  s = warp_sum(sh[lane][g]);
  if (lane == 0 && blockIdx.x * 32 + g < cols) out[blockIdx.x * 32 + g] = s;
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
int walk_blocks(int rows, int rows_at_a_time, int per_sm, int sm_count) {
  return std::min((rows + rows_at_a_time - 1) / rows_at_a_time, per_sm * sm_count);
}
constexpr int kSizingSms = 160;  // at least the SMs of any sm_100 part, for workspace sizes

int bwd_blocks(int rows, int cols, int sms) {
  int n = 0;
#define MAO_CASE(G, V) n = walk_blocks(rows, kBlock<G> / G, kBlock<G> >= kBwdThreads ? 1 : kBwdThreads / kBlock<G>, sms);
  MAO_NORM_SIZES(MAO_CASE)
#undef MAO_CASE
  return n;
}

template <class T, bool KEEP, int G, int VPT>
mao_status fwd_one(const FwdArgs& a, int sms, cudaStream_t stream) {
  using Cfg = FwdCfg<T, G, VPT>;
  static std::atomic<bool> done[64];
  MAO_TRY(allow_smem(norm_kernel<T, KEEP, G, VPT>, Cfg::kSmem, done));
  const int grid = walk_blocks(a.rows, Cfg::B / G, Cfg::kPerSm, sms);
  norm_kernel<T, KEEP, G, VPT><<<grid, Cfg::B, Cfg::kSmem, stream>>>(a);
  return launched();
}

template <class T, bool KEEP>
mao_status fwd_sized(const FwdArgs& a, int sms, cudaStream_t stream) {
  const int cols = a.cols;
  LaunchScope ls(stream, MAO_K_LAYER_NORM, 0.0,
                 (double)a.rows * cols * (2.0 * sizeof(T) + (KEEP ? 1.0 + 1.0 / 32 : 0.0)));
#define MAO_CASE(G, V) return fwd_one<T, KEEP, G, V>(a, sms, stream);
  MAO_NORM_SIZES(MAO_CASE)
#undef MAO_CASE
}

template <class T>
mao_status fwd(const FwdArgs& a, int sms, cudaStream_t stream) {
  return a.k.q != nullptr ? fwd_sized<T, true>(a, sms, stream) : fwd_sized<T, false>(a, sms, stream);
}

template <class T, bool KEPT, bool RES, int G, int VPT>
mao_status bwd_one(const BwdArgs& a, int grid, cudaStream_t stream) {
  using Cfg = BwdCfg<T, KEPT, RES, G, VPT>;
  static std::atomic<bool> done[64];
  MAO_TRY(allow_smem(norm_bwd_kernel<T, KEPT, RES, G, VPT>, Cfg::kSmem, done));
  norm_bwd_kernel<T, KEPT, RES, G, VPT><<<grid, Cfg::B, Cfg::kSmem, stream>>>(a);
  return launched();
}

template <class T, bool KEPT, bool RES>
mao_status bwd_sized(const BwdArgs& a, int grid, cudaStream_t stream) {
  const int cols = a.cols;
  LaunchScope ls(stream, MAO_K_LAYER_NORM_BWD, 0.0,
                 (double)a.rows * cols * ((RES ? 3.0 : 2.0) * sizeof(T) + (KEPT ? 1.0 + 1.0 / 32 : sizeof(T))));
#define MAO_CASE(G, V) return bwd_one<T, KEPT, RES, G, V>(a, grid, stream);
  MAO_NORM_SIZES(MAO_CASE)
#undef MAO_CASE
}

template <class T>
mao_status bwd(const BwdArgs& a, bool kept, int grid, cudaStream_t stream) {
  if (kept) return a.dres ? bwd_sized<T, true, true>(a, grid, stream) : bwd_sized<T, true, false>(a, grid, stream);
  return a.dres ? bwd_sized<T, false, true>(a, grid, stream) : bwd_sized<T, false, false>(a, grid, stream);
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
  return sizeof(float) * 2 * (size_t)bwd_blocks(a->rows, a->cols, sms) * (size_t)a->cols;
}

// out0[col] = sum over parts of part[p * cols + col]; out1 likewise of the parts * cols values
// behind.  Either may be nullptr.
mao_status col_reduce_launch(const float* part, int parts, int cols, float* out0, float* out1, cudaStream_t stream) {
  LaunchScope ls(stream, MAO_K_COL_REDUCE, 0.0, 4.0 * (double)parts * cols * (out1 ? 2 : 1));
  return launch_dependent(col_reduce_kernel, dim3((cols + 31) / 32, out1 ? 2 : 1), 1024, 0, stream, part, parts, cols,
                          out0, out1);
}

}  // namespace

mao_status col_sum_launch(const float* part, int parts, int cols, float* out, cudaStream_t stream) {
  return col_reduce_launch(part, parts, cols, out, nullptr, stream);
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
  const int grid = bwd_blocks(a->rows, a->cols, dev->sm_count);
  mao_status st;
  switch (a->dtype) {
    case MAO_F32: st = bwd<float>(g, kept, grid, stream); break;
    case MAO_BF16: st = bwd<__nv_bfloat16>(g, kept, grid, stream); break;
    default: st = bwd<__half>(g, kept, grid, stream); break;
  }
  if (st != MAO_OK) return st;
  if (a->dw == nullptr && a->db == nullptr) return MAO_OK;
  return col_reduce_launch(g.part, grid, a->cols, a->dw, a->db, stream);
}
