// dz = dy act'(z), rounded to the activations' type for the two products that read it, with
// the column sums of the unrounded dz for the bias gradient in the same pass.
//
// The products' tensor-core operands have that type; a second plane with what the rounding leaves
// would double them.  Through GELU the rounding puts dW off by 1.7e-3 of its norm in bf16, 2.1e-4 in
// fp16 (3e-7 to 9e-7 without an activation).  The slopes come from approximate exponentials, off by
// about 1e-6: db is off by 3.4e-7 of its norm (8192 tokens).
//
// HBM-bound: dy 2 + z 2 (or 1 + 1/32 from a checkpoint) + dz 2 bytes per element.  A lane
// owns 16 columns, a block 512 columns of a chunk of rows, each warp every eighth row; a
// thread reads its next three rows ahead by cp.async.  Each chunk leaves one partial row of
// column sums, which the product kernel joins in order (no atomics: the same bits every run).
// Blocks behind those of this pass read the layer's input back from its checkpoint, so that
// one launch prepares both operands.
#include "act_bwd.h"
#include "ckpt8.cuh"

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
  int strips, blocks;  // column strips; blocks of this pass, the restore's come behind
  // x read back from its checkpoint for the product that follows (xr == nullptr: not asked for)
  CkptView xk;
  void* xr;
  long long ld_xr;
  Steps xs;
};

constexpr int kCols = 16;    // columns per lane
constexpr int kStages = 4;   // rows read ahead per thread, less one
constexpr int kThreads = 256;
constexpr int kStrip = 32 * kCols;  // columns per block

template <int ACT, bool KEPT>
constexpr int kSlot = 32 + (ACT == MAO_ACT_NONE ? 0 : (KEPT ? 16 : 32));  // ring bytes per thread and row

template <class T, int ACT, bool KEPT>
__global__ void __launch_bounds__(kThreads, 3) act_bwd_kernel(const ActArgs a) {
  constexpr bool HAS = ACT != MAO_ACT_NONE;
  constexpr uint32_t kPiece = kThreads * 16;
  extern __shared__ __align__(16) uint8_t ring[];
  launch_dependents();
  if ((int)blockIdx.x >= a.blocks) {
    restore_block<T, MAO_ACT_NONE>(a.xk, static_cast<T*>(a.xr), a.ld_xr, a.xs, (int)blockIdx.x - a.blocks);
    return;
  }
  const int chunk_id = (int)blockIdx.x / a.strips, strip = (int)blockIdx.x - chunk_id * a.strips;
  const uint32_t slot = smem_u32(ring) + threadIdx.x * 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // two vectors of 8 columns, 256 columns apart: neighbouring lanes read neighbouring 16 bytes
  const int c = strip * kStrip + lane * 8;
  const int halves = c >= a.cols ? 0 : (c + 256 < a.cols ? 2 : 1);  // vectors inside the row
  const long long r_end = min((long long)a.rows, ((long long)chunk_id + 1) * a.chunk);
  const long long r_begin = (long long)chunk_id * a.chunk + warp;
  const T* dy = static_cast<const T*>(a.dy);
  const T* z = static_cast<const T*>(a.z);
  auto fetch = [&](long long r, int stage) {
    const uint32_t dst = slot + stage * (kSlot<ACT, KEPT> * kThreads);
    const bool in = r < r_end;
    const T* p = dy + (in ? r : 0) * a.ld_dy + c;
    cp_async16(dst, in && halves > 0 ? p : dy, in && halves > 0);
    cp_async16(dst + kPiece, in && halves > 1 ? p + 256 : dy, in && halves > 1);
    if constexpr (HAS && KEPT) {
      const int8_t* q = a.k.q + (in ? r : 0) * a.k.ld_q + c;
      const uint32_t dk = dst + 2 * kPiece - threadIdx.x * 8;  // 8 bytes per thread and vector
      cp_async8(dk, in && halves > 0 ? q : a.k.q, in && halves > 0);
      cp_async8(dk + kPiece / 2, in && halves > 1 ? q + 256 : a.k.q, in && halves > 1);
    } else if constexpr (HAS) {
      const T* q = z + (in ? r : 0) * a.ld_z + c;
      cp_async16(dst + 2 * kPiece, in && halves > 0 ? q : z, in && halves > 0);
      cp_async16(dst + 3 * kPiece, in && halves > 1 ? q + 256 : z, in && halves > 1);
    }
    cp_async_commit();
  };
  struct Bytes {  // of the two vectors' checkpoint blocks
    uint32_t e[2];
  };
  auto fetch_e = [&](long long r) {
    Bytes b = {{1u, 1u}};
    if constexpr (HAS && KEPT) {
      const uint8_t* e = a.k.e + r * a.k.ld_e + (c >> 5);
      if (r < r_end && halves > 0) b.e[0] = e[0];
      if (r < r_end && halves > 1) b.e[1] = e[8];
    }
    return b;
  };
#pragma unroll
  for (int d = 0; d < kStages - 1; ++d) fetch(r_begin + 8 * d, d);
  // each in its own registers until its row's turn: passed along from row to row they would be
  // waited for at once
  Bytes e[kStages];
#pragma unroll
  for (int d = 0; d < kStages; ++d) e[d] = fetch_e(r_begin + 8 * d);
  f2 sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sum[j] = dup2(0.0f);
  for (long long r0 = r_begin; r0 < r_end; r0 += 8 * kStages) {
#pragma unroll
    for (int stage = 0; stage < kStages; ++stage) {
      const long long r = r0 + 8 * stage;
      if (r >= r_end) break;
      fetch(r + 8 * (kStages - 1), (stage + kStages - 1) % kStages);
      const Bytes now = e[stage];
      cp_async_wait<kStages - 1>();
      const uint32_t src = slot + stage * (kSlot<ACT, KEPT> * kThreads);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Vec8<T> g;
        g.w = lds16(src + h * kPiece);
        f2 d[4];
        g.get(d);
        if constexpr (HAS) {
          f2 f[4];
          if constexpr (KEPT) {
            CkptVec8 k;
            k.w = lds8(src + 2 * kPiece - threadIdx.x * 8 + h * (kPiece / 2));
            k.e = now.e[h];
            k.get(f);
          } else {
            Vec8<T> v;
            v.w = lds16(src + (2 + h) * kPiece);
            v.get(f);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = mul2(d[j], act_slope<ACT>(f[j]));
          Vec8<T> o;
          o.set(d);
          if (a.dz != nullptr && h < halves) o.store(static_cast<T*>(a.dz) + r * a.ld_dz + c + 256 * h);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[4 * h + j] = add2(sum[4 * h + j], d[j]);
      }
      e[stage] = fetch_e(r + 8 * kStages);
    }
  }
  cp_async_wait<0>();
  if (a.part == nullptr) return;
  // the warps' sums joined in warp order, through the ring's memory
  __syncthreads();
  float* sh = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int j = 0; j < 8; ++j) *reinterpret_cast<f2*>(sh + warp * kStrip + (j >> 2) * 256 + lane * 8 + 2 * (j & 3)) = sum[j];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kStrip / kThreads; ++i) {
    const int k = i * kThreads + threadIdx.x;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sh[w * kStrip + k];
    if (strip * kStrip + k < a.cols) a.part[(long long)chunk_id * a.cols + strip * kStrip + k] = s;
  }
}

template <class T, int ACT, bool KEPT>
mao_status run_one(const ActArgs& a, unsigned grid, cudaStream_t s) {
  constexpr int smem = kStages * kSlot<ACT, KEPT> * kThreads;  // at least the 16 KB of the joined sums
  static_assert(smem >= 8 * kStrip * (int)sizeof(float), "the joined sums use the ring's memory");
  static std::atomic<bool> done[64];
  MAO_TRY(allow_smem(act_bwd_kernel<T, ACT, KEPT>, smem, done));
  act_bwd_kernel<T, ACT, KEPT><<<grid, kThreads, smem, s>>>(a);
  return launched();
}

template <class T, bool KEPT>
mao_status run(const ActArgs& a, int act, unsigned grid, cudaStream_t s) {
  switch (act) {
    case MAO_ACT_NONE: return run_one<T, MAO_ACT_NONE, false>(a, grid, s);
    case MAO_ACT_RELU: return run_one<T, MAO_ACT_RELU, KEPT>(a, grid, s);
    case MAO_ACT_RELU2: return run_one<T, MAO_ACT_RELU2, KEPT>(a, grid, s);
    case MAO_ACT_GELU: return run_one<T, MAO_ACT_GELU, KEPT>(a, grid, s);
    case MAO_ACT_GELU_TANH: return run_one<T, MAO_ACT_GELU_TANH, KEPT>(a, grid, s);
    case MAO_ACT_SILU: return run_one<T, MAO_ACT_SILU, KEPT>(a, grid, s);
    default: return MAO_ERR_INVALID_ARG;
  }
}

}  // namespace

// Two full waves of the three blocks that an SM of a B200 holds, at least 32 rows each.
int act_bwd_chunk(int rows, int cols) {
  const int strips = (cols + kStrip - 1) / kStrip;
  const int want = std::max(1, 888 / strips);
  const int chunks = std::max(1, std::min(want, (rows + 31) / 32));
  return (rows + chunks - 1) / chunks;
}

mao_status act_bwd_launch(const ActBwd& b, int dtype, cudaStream_t stream) {
  ActArgs a;
  a.dy = b.dy, a.z = b.z, a.k = b.zk, a.dz = b.dz, a.part = b.part;
  a.ld_dy = b.ld_dy, a.ld_z = b.ld_z, a.ld_dz = b.ld_dz;
  a.rows = b.rows, a.cols = b.cols;
  a.chunk = act_bwd_chunk(b.rows, b.cols);
  a.strips = (b.cols + kStrip - 1) / kStrip;
  const bool sums = b.dz != nullptr || b.part != nullptr;
  a.blocks = sums ? a.strips * ((b.rows + a.chunk - 1) / a.chunk) : 0;
  a.xk = b.xk, a.xr = b.xr, a.ld_xr = b.x_cols;
  unsigned grid = (unsigned)a.blocks;
  if (b.xr != nullptr) {
    DeviceInfo* dev = nullptr;
    MAO_TRY(device_info(&dev));
    grid += steps_of(b.rows, b.x_cols / 8, dev->sm_count, &a.xs);
  }
  if (grid == 0) return MAO_OK;
  const bool kept = b.z == nullptr;
  const int act = sums ? b.act : MAO_ACT_NONE;
  const double z_bytes = act == MAO_ACT_NONE ? 0.0 : (kept ? 1.0 + 1.0 / 32 : 2.0);
  LaunchScope ls(stream, MAO_K_ACT_BWD, 0.0,
                 (sums ? (double)b.rows * b.cols * (2.0 + z_bytes + (b.dz ? 2.0 : 0.0)) : 0.0) +
                     (b.xr ? (double)b.rows * b.x_cols * (3.0 + 1.0 / 32) : 0.0));
  if (dtype == MAO_BF16)
    return kept ? run<__nv_bfloat16, true>(a, act, grid, stream) : run<__nv_bfloat16, false>(a, act, grid, stream);
  return kept ? run<__half, true>(a, act, grid, stream) : run<__half, false>(a, act, grid, stream);
}

}  // namespace mao
