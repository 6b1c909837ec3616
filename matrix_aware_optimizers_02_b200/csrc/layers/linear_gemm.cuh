// The trained layers' matrix products for sm_100a: D = A B^T with 16-bit operands (bf16 or
// fp16), fp32 accumulation in tensor memory, and the linear layer's epilogues.
//
//   forward    y  = act(x W^T + b) + res   A = x (K-major),      B = W (K-major)
//   dx         dx = dz W                   A = dz (K-major),     B = W (MN-major)
//   dW         dW = dz^T x                 A = dz (MN-major),    B = x (MN-major)
//
// One persistent kernel, one CTA per SM or one CTA pair per two SMs, each walking a list of work
// items (output tile, K slice) that the host's plan dealt it.  Warp roles (640 threads):
//   warp 0      TMA producer (one lane): a ring of 128-byte-swizzled A / B tiles;
//   warp 1      owner of the tensor memory and MMA issuer (one lane);
//   warps 4-19  epilogue, four per tensor-memory lane quarter, a quarter of the columns each.
// Two accumulators let an item's epilogue overlap the next item's MMAs.  The first four warps
// hand registers to the epilogue (32 against 112 a thread, 96 at launch: 128 * 32 + 512 * 112
// is 640 * 96); without that 4096 x 1536 -> 1536 took 36.9 instead of 32.8 us.  Sixteen epilogue
// warps hold the running sums of a 128 x 256 accumulator in 64 registers a thread; eight would
// need 128.
//
// Tiles.  PAIR: 256 x 256 per CTA pair (tcgen05.mma.cta_group::2); each CTA loads 128 rows of A
// and half of B's 256, for twice the MMA work of a one-CTA 128 x 128 tile's loads.  Either way a
// CTA takes in 32 KB per k-block at about 110 GB/s, the rate at which an SM's loads arrive, so
// the one-CTA tile is for products whose 256 x 256 tiles would leave SMs idle.  (256 x 128 pair
// tiles were measured and dropped: 24 KB per k-block took as long, no size gained.)
// Tiles that do not fill a whole round of the workers may be cut into K slices: each slice
// leaves its fp32 sums of the tile in the workspace, and a second kernel joins them in slice
// order and runs the same epilogue.
//
// The backward pass's two products run as one launch, the one with the longer K first, dealt
// so that the workers left over by its last round take more of the other (LinDeal).
// The two single-thread roles branch once per item to code of its majors: with majors as run-time
// values in the MMA loop 8192 x 4096 -> 14336 took 711 instead of 658 us.
//
// Order.  Tiles run in bands of kBandRows tile rows, column by column inside a band, so the
// tiles that are in flight together share few operand rows and columns in L2.
//
// Accuracy.  The tensor core's accumulation truncates: a sum over K terms of random sign is off by
// 1e-6 of its size for every 1024 of K, where fp32 with rounding stays below 1e-6, and one of terms
// of one sign by up to 7e-6.  So the sums leave tensor memory after a number of k-blocks, and the
// epilogue adds them in fp32 registers, rounded to nearest: after a few for an fp32 dW and for a
// forward product whose z is kept in 8 bits (where a sum's error decides which way a value rounds),
// after 128 for other results of 16 bits.  dW in fp32 is then off by 4.7e-7 (1024 tokens) to 7.7e-7
// (131072) of its size in the mean square for terms of random sign, by 6.4e-7 at most for one sign.
#pragma once

#include "gemm_tc.cuh"
#include "layer_math.cuh"

namespace mao {

// Where a bounded wait of these kernels records that it gave up; sticky until read.
static __device__ DevStatus g_layer_status;

constexpr int kBandRows = 8;
// k-blocks that a sum of nk of them spends in tensor memory at a time, in parts of one length
// (16 as 8 + 8 take the time of 12 + 4).  At most 12 for an fp32 dW.  For a kept z the same, and
// fewer for short K, where fp32's own error is smaller.  Error that values rounding the other way
// than the exact z's put in a kept z, in fp32 sums' own (2048 x K -> 2048, mean of six seeds), and
// the time of a product with SiLU and checkpoint, sustained:
//     K          12 blocks         8                 6
//     768   1.92   81 us     1.48   89 us     1.39   88 us    8192 x 768 -> 4096
//     1024  1.85   98        1.65   98        1.35  109       8192 x 1024 -> 4096
//     2048  1.44  295        1.19  318        1.01  350       8192 x 2048 -> 8192
//     4096  1.18  938        0.94  989                        8192 x 4096 -> 14336 (16: 1.40, 876)
// At 4096 parts of 11 give 1.11 in the time of 12.  K = 256 stays at 1.50 in one part.  The 8-bit
// steps themselves are off a hundred times as far.  4 blocks at K = 1024: 1.12, 118 us.
// Other 16-bit results: 128 (8192 terms).  Terms of one sign lose about a step of the result per
// truncated add: 8.7e-4 of it after 131072 in one part, where fp16's half step is 4.9e-4; 8192
// lose 6e-5.  K up to 8192 stays in one part.
inline int equal_parts(int nk, int most) {
  const int parts = (nk + most - 1) / most;
  return (nk + parts - 1) / parts;
}
inline int fold_blocks(int nk, bool kept) { return equal_parts(nk, !kept || nk > 32 ? 12 : (nk > 16 ? 8 : 6)); }
constexpr int kLongFold = 128;

// Epilogues of the backward kernel; the forward kernel has its own (bias, activation,
// residual, checkpoint of z).
enum LinKind : int {
  LIN_STORE = 0,   // out (16-bit) = acc
  LIN_GRAD32 = 1,  // out (fp32) = acc, or += acc
  LIN_FORWARD = 2,
};

struct LinEpilogue {
  void* out;
  const void* bias;
  const void* res;
  void* z;
  CkptView k;
  long long ld_out, ld_res, ld_z;
  int M, N;
  int kind;
  int act;
  int bias_f32;
  int accumulate;
};

struct LinProblem {
  CUtensorMap mapA, mapB;
  LinEpilogue e;
  float* part;       // [slice][sliced tile][BM][BN]: sums of the sliced tiles
  int a_mn;          // A's major, 0: K, 1: MN (B: K in the forward kernel, MN in the backward one)
  int tiles_m, tiles_n;
  int full;          // tiles [0, full) are whole items, the others come as `slices` items each
  int slices;
  int nk;            // k-blocks of 64
  int slice_blocks;  // k-blocks per slice
  int fold;          // k-blocks per accumulation in tensor memory
};

// Partial column sums joined on the side by the epilogue warps, before their first tile:
// out[c] = sum over p of part[p * cols + c].
struct LinColSum {
  const float* part;
  float* out;  // nullptr: none
  int parts, cols;
};

// Which worker does what.  List w has the first problem's items w, w + workers, ...; `extra`
// lists have one more of those than the others.  Of the last problem's `whole` items the other
// lists take `lead` each in turn, then all lists take theirs in turn (so that what runs at one
// time lies together in L2), `per_whole` in all for the others.  Its `cuts` items behind those
// (slices, or single tiles) go in turn to the others, at most `per_cut` each, and what is left
// in turn to the lists with an extra.
struct LinDeal {
  int workers;
  int first;  // items of the first of two problems, 0 where there is one
  int extra;
  int whole, per_whole, lead;
  int cuts, per_cut;
};

template <int NP>
struct LinParams {
  LinProblem p[NP];
  LinDeal deal;
  LinColSum sum;
};

template <int NP>
struct LinWalk {
  int w, step, phase, k;
  __host__ __device__ __forceinline__ LinWalk(int worker, int workers) : w(worker), step(workers), phase(NP > 1 ? 0 : 1), k(0) {}
  // the next item of this worker's lists; false: none left
  __host__ __device__ __forceinline__ bool next(const LinDeal& d, int& problem, int& item) {
    for (; w < d.workers; w += step, phase = (NP > 1 ? 0 : 1), k = 0) {
      if (NP > 1 && phase == 0) {
        item = w + k * d.workers;
        if (item < d.first) {
          ++k;
          problem = 0;
          return true;
        }
        phase = 1, k = 0;
      }
      const int others = d.workers - d.extra;
      const bool plain = w >= d.extra;
      if (phase == 1) {
        const int late = plain ? k - d.lead : k;  // rounds of all lists behind it
        item = late < 0 ? w - d.extra + k * others : others * d.lead + late * d.workers + w;
        if (item < d.whole && k < (plain ? d.per_whole : d.per_whole - d.lead)) {
          ++k;
          problem = NP - 1;
          return true;
        }
        phase = 2, k = 0;
      }
      item = plain ? w - d.extra + k * others : others * d.per_cut + w + k * d.extra;
      if (item < d.cuts && (!plain || k < d.per_cut)) {
        ++k;
        problem = NP - 1;
        item += d.whole;
        return true;
      }
    }
    return false;
  }
};

// ------------------------------------------------------------------ epilogue
template <int ACT>
__device__ __forceinline__ void act32(float* v) {
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const f2 r = act_value<ACT>(make_float2(v[j], v[j + 1]));
    v[j] = r.x, v[j + 1] = r.y;
  }
}

template <int ACT>
__device__ __forceinline__ void act8(f2 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = act_value<ACT>(v[j]);
}

__device__ __forceinline__ void ld_global_v8(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
// v += 16 consecutive 16-bit elements, a whole sector in one load
template <class T>
__device__ __forceinline__ void add16x16(const T* src, float* v) {
  uint32_t w[8];
  ld_global_v8(src, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const f2 f = Elem<T>::unpack(w[i]);
    v[2 * i] += f.x, v[2 * i + 1] += f.y;
  }
}

// 32 consecutive 16-bit elements of one row, `n` of them valid (a multiple of 8)
template <class T>
__device__ __forceinline__ void store16x32(T* dst, const float* v, int n) {
  uint32_t w[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = Elem<T>::pack(v[2 * j], v[2 * j + 1]);
  if (n >= 32 && aligned32(dst)) {
    st_global_v8(dst, w);
    st_global_v8(dst + 16, w + 8);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (8 * j < n) reinterpret_cast<uint4*>(dst)[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  }
}

// The epilogue of 32 consecutive columns [col, col + 32) of one row; v holds the sums.
// Columns come in eights (N is a multiple of 8).  With PAIRS a warp's columns come as pairs of
// such pieces: `second` says which, and `e_first` carries the first's checkpoint byte to the
// second, so that a lane writes two bytes at once (each lane's lie in a line of their own).
template <class T, bool FORWARD, bool PAIRS>
__device__ __forceinline__ void lin_epilogue(const LinEpilogue& e, int row, int col, float* v, bool second,
                                             uint32_t& e_first) {
  if (row >= e.M || col >= e.N) return;
  const int n = min(32, e.N - col);
  if constexpr (!FORWARD) {
    if (e.kind == LIN_STORE) {
      store16x32<T>(static_cast<T*>(e.out) + (long long)row * e.ld_out + col, v, n);
      return;
    }
    float* o = static_cast<float*>(e.out) + (long long)row * e.ld_out + col;
    if (e.accumulate) {
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        if (j < n) {
          const float4 a = *reinterpret_cast<const float4*>(o + j);
          v[j] += a.x, v[j + 1] += a.y, v[j + 2] += a.z, v[j + 3] += a.w;
        }
    }
    if (n == 32) {
      store_f32x32(o, v);
    } else {
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        if (j < n) *reinterpret_cast<float4*>(o + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
  } else {
    if (e.bias != nullptr) {
#pragma unroll
      for (int j = 0; j < 32; j += 8)
        if (j < n) {
          f2 b[4];
          load_param8<T>(e.bias, e.bias_f32, col + j, b);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j + 2 * i] += b[i].x, v[j + 2 * i + 1] += b[i].y;
        }
    }
    if (e.z != nullptr) store16x32<T>(static_cast<T*>(e.z) + (long long)row * e.ld_z + col, v, n);
    if (e.k.q != nullptr) {
      // this thread's 32 columns are one block of the checkpoint; columns behind the last
      // hold zeros (the operands' out-of-range rows load as zeros, and the bias skips them)
      float a = 0.0f;
#pragma unroll
      for (int j = 0; j < 32; j += 2) a = max_abs3(a, v[j], v[j + 1]);
      const uint32_t ex = ckpt_exponent(abs_bits(a));
      const float inv = ckpt_inverse(ex);
      const uint32_t mask = ex == 255u ? 0u : 0xffffffffu;
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = ckpt_q4(make_float2(v[4 * j], v[4 * j + 1]), make_float2(v[4 * j + 2], v[4 * j + 3]), inv, mask);
      int8_t* q = e.k.q + (long long)row * e.k.ld_q + col;
      if (aligned32(q)) {
        st_global_v8(q, w);
      } else {
        reinterpret_cast<uint4*>(q)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(q)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
      uint8_t* eb = e.k.e + (long long)row * e.k.ld_e + (col >> 5);
      if (!second) {
        e_first = ex;
        if (!PAIRS || col + 32 >= e.N) *eb = (uint8_t)ex;  // no second, or the row ends here
      } else if ((reinterpret_cast<uintptr_t>(eb - 1) & 1u) == 0) {
        *reinterpret_cast<uint16_t*>(eb - 1) = (uint16_t)(e_first | ex << 8);
      } else {
        eb[-1] = (uint8_t)e_first, eb[0] = (uint8_t)ex;
      }
    }
    switch (e.act) {
      case MAO_ACT_RELU: act32<MAO_ACT_RELU>(v); break;
      case MAO_ACT_RELU2: act32<MAO_ACT_RELU2>(v); break;
      case MAO_ACT_GELU: act32<MAO_ACT_GELU>(v); break;
      case MAO_ACT_GELU_TANH: act32<MAO_ACT_GELU_TANH>(v); break;
      case MAO_ACT_SILU: act32<MAO_ACT_SILU>(v); break;
      default: break;
    }
    if (e.res != nullptr) {
      const T* r = static_cast<const T*>(e.res) + (long long)row * e.ld_res + col;
      if (n == 32 && aligned32(r)) {
        add16x16(r, v);
        add16x16(r + 16, v + 16);
      } else {
#pragma unroll
        for (int j = 0; j < 32; j += 8)
          if (j < n) {
            Vec8<T> x;
            x.load(r + j);
            f2 f[4];
            x.get(f);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j + 2 * i] += f[i].x, v[j + 2 * i + 1] += f[i].y;
          }
      }
    }
    store16x32<T>(static_cast<T*>(e.out) + (long long)row * e.ld_out + col, v, n);
  }
}

// ------------------------------------------------------------------ kernel
template <bool PAIR>
struct LinCfg {
  static constexpr int BM = PAIR ? 256 : 128;  // tile rows (128 per CTA)
  static constexpr int BN = PAIR ? 256 : 128;  // tile columns
  static constexpr int BK = 64;
  static constexpr int A_TILE = 128 * 128;  // bytes: 128 rows of 64 elements per CTA
  static constexpr int B_TILE = 128 * 128;  // PAIR: half of B's rows per CTA
  static constexpr int STAGE_BYTES = A_TILE + B_TILE;
  // As deep as shared memory allows: the bytes in flight set the pace of products that the power
  // limit does not (4096^3: 118 us with 6 stages, 108 with 7).
  static constexpr int STAGES = (224 * 1024) / STAGE_BYTES;
  static constexpr int TMEM_COLS = 2 * BN;
  static constexpr int EPI_WARPS = 16;
  static constexpr int COLS = BN / 4;  // columns per epilogue warp
  static constexpr int EPI_FIRST = 4;  // first epilogue warp
  static constexpr int THREADS = 32 * (EPI_FIRST + EPI_WARPS);
  // what shared memory holds behind the stages; no static shared memory, so that the stages
  // start on a 1024-byte boundary without padding
  struct Shared {
    uint64_t full_bar[STAGES], empty_bar[STAGES];
    uint64_t tfull_bar[2], tempty_bar[2];
    uint64_t drain_bar;
    uint32_t tmem_base;
    int abort, prod_it, mma_it;
    float join[EPI_WARPS][33];
  };
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + (int)sizeof(Shared);
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of a CTA");
};

// Tile -> first row and column: bands of kBandRows tile rows, column by column.
__host__ __device__ __forceinline__ void lin_tile(int tile, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int band = tile / (kBandRows * tiles_n);
  const int first = band * kBandRows;
  const int rows = tiles_m - first < kBandRows ? tiles_m - first : kBandRows;
  const int r = tile - band * kBandRows * tiles_n;
  tn = r / rows;
  tm = first + r - tn * rows;
}

template <int N>
struct IntC {
  static constexpr int value = N;
};

struct LinItem {
  int m0, n0;    // first row / column of the tile
  int kb0, kb1;  // its k-blocks
  int part;      // index of its sums in the workspace, or -1: a whole tile
};

template <class Cfg>
__device__ __forceinline__ LinItem lin_item(const LinProblem& p, int item) {
  LinItem t;
  int tile = item, slice = 0;
  t.part = -1;
  t.kb0 = 0, t.kb1 = p.nk;
  if (item >= p.full && p.slices > 1) {
    const int tail = p.tiles_m * p.tiles_n - p.full;
    t.part = item - p.full;
    slice = t.part / tail;
    tile = p.full + t.part - slice * tail;
    t.kb0 = slice * p.slice_blocks;
    t.kb1 = min(p.nk, t.kb0 + p.slice_blocks);
  }
  int tm, tn;
  lin_tile(tile, p.tiles_m, p.tiles_n, tm, tn);
  t.m0 = tm * Cfg::BM;
  t.n0 = tn * Cfg::BN;
  return t;
}

// Inside each role's branch, so that the compiler knows which code has how many.
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 32;"); }
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 112;"); }

// One operand's share of a stage: 128 rows (K-major) or 128 columns of 64 K rows (MN-major).
template <bool PAIR, int MN_MAJOR>
__device__ __forceinline__ void lin_load(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, uint32_t bar_lead,
                                         int k0, int mn0) {
  if constexpr (!MN_MAJOR) {
    if constexpr (PAIR) tma_load_3d_pair(dst, map, bar_lead, k0, mn0, 0);
    else tma_load_3d(dst, map, bar, k0, mn0, 0);
  } else {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if constexpr (PAIR) tma_load_3d_pair(dst + c * 64 * 128, map, bar_lead, mn0 + c * 64, k0, 0);
      else tma_load_3d(dst + c * 64 * 128, map, bar, mn0 + c * 64, k0, 0);
    }
  }
}

template <class T, bool FORWARD, bool PAIR>
__device__ __forceinline__ void lin_body(const LinParams<FORWARD ? 1 : 2>& params) {
  constexpr int NP = FORWARD ? 1 : 2;
  using Cfg = LinCfg<PAIR>;
  constexpr int STAGES = Cfg::STAGES, BK = Cfg::BK;
  constexpr int B_MN = FORWARD ? 0 : 1;

  extern __shared__ __align__(1024) uint8_t smem[];
  typename Cfg::Shared& sh = *reinterpret_cast<typename Cfg::Shared*>(smem + STAGES * Cfg::STAGE_BYTES);
  uint64_t* const full_bar = sh.full_bar;
  uint64_t* const empty_bar = sh.empty_bar;
  uint64_t* const tfull_bar = sh.tfull_bar;
  uint64_t* const tempty_bar = sh.tempty_bar;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int worker = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int workers = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  DevStatus* status = &g_layer_status;
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzle's unit; the same for every CTA
    if (threadIdx.x == 0) report(status, MAO_ERR_ALIGN, 50);
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull_bar[a], 1);
      mbar_init(&tempty_bar[a], (PAIR ? 2 : 1) * 32 * Cfg::EPI_WARPS);
    }
    mbar_init(&sh.drain_bar, 1);
    sh.abort = 0;
    sh.prod_it = 0;
    sh.mma_it = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    if constexpr (PAIR) {
      tmem_alloc_pair(&sh.tmem_base, Cfg::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&sh.tmem_base, Cfg::TMEM_COLS);
      tmem_relinquish();
    }
  }
  if (warp == 0 && lane == 0) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      tma_prefetch_desc(&params.p[i].mapA);
      tma_prefetch_desc(&params.p[i].mapB);
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // both CTAs' barriers initialised before any remote arrival
  tc_fence_after();
  const uint32_t tmem_base = sh.tmem_base;
  volatile int* abort_flag = &sh.abort;
  launch_dependents();  // the joining kernel's blocks, as CTAs of this one end
  if constexpr (!FORWARD) wait_for_previous();  // the operands come from the kernel before

  if (warp == 0) {
    give_registers();
    if (lane == 0) {
      // -------------------------------------------------------------- producer
      int it = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      auto load_item = [&](auto a_mn, const LinProblem& p, const LinItem& t) {
        constexpr int A_MN = decltype(a_mn)::value;
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          if (!mbar_wait(&empty_bar[s], ph ^ 1, status, 51, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * Cfg::STAGE_BYTES;
          uint32_t lead = 0;
          if constexpr (PAIR) {
            if (leader) mbar_arrive_expect_tx(&full_bar[s], 2 * Cfg::STAGE_BYTES);
            lead = mapa_shared(smem_u32(&full_bar[s]), 0);
          } else {
            mbar_arrive_expect_tx(&full_bar[s], Cfg::STAGE_BYTES);
          }
          lin_load<PAIR, A_MN>(st, &p.mapA, &full_bar[s], lead, kb * BK, t.m0 + 128 * (int)rank);
          lin_load<PAIR, B_MN>(st + Cfg::A_TILE, &p.mapB, &full_bar[s], lead, kb * BK, t.n0 + 128 * (int)rank);
          if (++s == STAGES) s = 0, ph ^= 1;
        }
      };
      LinWalk<NP> walk(worker, workers);
      for (int which = 0, item = 0; ok && walk.next(params.deal, which, item);) {
        const LinProblem& p = params.p[which];
        const LinItem t = lin_item<Cfg>(p, item);
        if (!FORWARD && p.a_mn) load_item(IntC<1>{}, p, t);
        else load_item(IntC<0>{}, p, t);
      }
      sh.prod_it = it;
    }
  } else if (warp == 1) {
    give_registers();
    if (lane == 0 && leader) {
      // -------------------------------------------------------------- MMA issuer
      int it = 0, used = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      auto mma_item = [&](auto a_mn, const LinItem& t, int fold) {
        constexpr int A_MN = decltype(a_mn)::value;
        constexpr uint32_t IDESC = make_idesc(Elem<T>::kDtype == MAO_BF16 ? 1u : 0u, A_MN, B_MN, Cfg::BM, Cfg::BN);
        for (int c0 = t.kb0; c0 < t.kb1 && ok; c0 += fold) {
          const int c1 = min(t.kb1, c0 + fold);
          const int acc = used & 1;
          const uint32_t aph = (used >> 1) & 1;
          ++used;
          if (!mbar_wait(&tempty_bar[acc], aph ^ 1, status, 52, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * Cfg::BN;
          for (int kb = c0; kb < c1; ++kb, ++it) {
            if (!mbar_wait(&full_bar[s], ph, status, 53, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_base = smem_u32(smem + s * Cfg::STAGE_BYTES);
            const uint32_t b_base = a_base + Cfg::A_TILE;
#pragma unroll
            for (int k = 0; k < BK / 16; ++k) {
              const uint64_t ad = operand_desc<A_MN, 128, 2>(a_base, k), bd = operand_desc<B_MN, 128, 2>(b_base, k);
              const uint32_t accum = (kb > c0 || k > 0) ? 1u : 0u;
              if constexpr (PAIR) umma_f16_pair(d_tmem, ad, bd, IDESC, accum);
              else umma_f16(d_tmem, ad, bd, IDESC, accum);
            }
            if constexpr (PAIR) umma_commit_pair(&empty_bar[s], 0x3);
            else umma_commit(&empty_bar[s]);
            if (++s == STAGES) s = 0, ph ^= 1;
          }
          if (!ok) break;
          if constexpr (PAIR) umma_commit_pair(&tfull_bar[acc], 0x3);
          else umma_commit(&tfull_bar[acc]);
        }
      };
      LinWalk<NP> walk(worker, workers);
      for (int which = 0, item = 0; ok && walk.next(params.deal, which, item);) {
        const LinProblem& p = params.p[which];
        const LinItem t = lin_item<Cfg>(p, item);
        if (!FORWARD && p.a_mn) mma_item(IntC<1>{}, t, p.fold);
        else mma_item(IntC<0>{}, t, p.fold);
      }
      sh.mma_it = it;
      // every MMA issued here has finished before tensor memory is released
      if constexpr (PAIR) umma_commit_pair(&sh.drain_bar, 0x3);
      else umma_commit(&sh.drain_bar);
    }
  } else if (warp < Cfg::EPI_FIRST) {
    give_registers();
  } else {
    take_registers();
    // ---------------------------------------------------------------- epilogue
    constexpr int COLS = Cfg::COLS;
    const int q = warp & 3;                   // tensor-memory lane quarter this warp may read
    const int cb = ((warp - Cfg::EPI_FIRST) >> 2) * COLS;  // its first column
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + cb;
    uint32_t tempty_lead[2] = {0, 0};
    if constexpr (PAIR) {
      tempty_lead[0] = mapa_shared(smem_u32(&tempty_bar[0]), 0);
      tempty_lead[1] = mapa_shared(smem_u32(&tempty_bar[1]), 0);
    }
    if constexpr (!FORWARD) {
      // 32 columns at a time, the sixteen warps over the parts, joined in a fixed order
      const LinColSum& g = params.sum;
      if (g.out != nullptr) {
        for (int c0 = blockIdx.x * 32; c0 < g.cols; c0 += gridDim.x * 32) {
          const int c = c0 + lane, w = warp - Cfg::EPI_FIRST;
          float s = 0.0f;
          if (c < g.cols) {
            const float* src = g.part + c;
            int i = w;
            for (; i + 48 < g.parts; i += 64) {
              const float v0 = src[(long long)i * g.cols], v1 = src[(long long)(i + 16) * g.cols],
                          v2 = src[(long long)(i + 32) * g.cols], v3 = src[(long long)(i + 48) * g.cols];
              s += (v0 + v1) + (v2 + v3);
            }
            for (; i < g.parts; i += 16) s += src[(long long)i * g.cols];
          }
          sh.join[w][lane] = s;
          asm volatile("bar.sync 1, 512;" ::: "memory");
          if (w == 0 && c < g.cols) {
#pragma unroll
            for (int k = 1; k < Cfg::EPI_WARPS; ++k) s += sh.join[k][lane];
            g.out[c] = s;
          }
          asm volatile("bar.sync 1, 512;" ::: "memory");
        }
      }
    }
    int used = 0;
    bool ok = true;
    LinWalk<NP> walk(worker, workers);
    for (int which = 0, item = 0; ok && walk.next(params.deal, which, item);) {
      const LinProblem& p = params.p[which];
      const LinItem t = lin_item<Cfg>(p, item);
      const int row = t.m0 + 128 * (int)rank + q * 32 + lane;
      if constexpr (FORWARD) {
        // the residual's lines (128 bytes of this thread's row) on their way to L2 meanwhile
        if (p.e.res != nullptr && t.part < 0 && row < p.e.M && t.n0 + cb < p.e.N)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const T*>(p.e.res) + (long long)row * p.e.ld_res +
                                                        t.n0 + cb));
      }
      float run[COLS];
      for (int c0 = t.kb0; c0 < t.kb1; c0 += p.fold) {
        const int acc = used & 1;
        const bool w = mbar_wait(&tfull_bar[acc], (used >> 1) & 1, status, 54, abort_flag);
        ++used;
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool first = c0 == t.kb0;
#pragma unroll
        for (int ch = 0; ch < COLS / 32; ++ch) {
          uint32_t rr[32];
          tmem_ld_32x32b_x32(lane_base + acc * Cfg::BN + ch * 32, rr);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j)
            run[ch * 32 + j] = first ? __uint_as_float(rr[j]) : run[ch * 32 + j] + __uint_as_float(rr[j]);
        }
        tc_fence_before();
        if constexpr (PAIR) mbar_arrive_cluster_relaxed(tempty_lead[acc]);
        else mbar_arrive_relaxed(&tempty_bar[acc]);
      }
      if (!ok) break;
      // The chunks of 32 columns through one copy of the epilogue's code (unrolled, it would
      // be fetched anew for every chunk of a short product): the sums move down by a chunk.
      uint32_t e_first = 0;
#pragma unroll 1
      for (int ch = 0; ch < COLS / 32; ++ch) {
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = run[j];
#pragma unroll
        for (int j = 0; j + 32 < COLS; ++j) run[j] = run[j + 32];
        if (t.part >= 0) {
          // all of a sliced tile is stored, what lies behind the matrix too: zeros
          store_f32x32(p.part + ((long long)t.part * Cfg::BM + (row - t.m0)) * Cfg::BN + cb + ch * 32, v);
        } else {
          lin_epilogue<T, FORWARD, COLS == 64>(p.e, row, t.n0 + cb + ch * 32, v, ch & 1, e_first);
        }
      }
    }
  }

  // ------------------------------------------------------------------ teardown
  if (warp == 1 && lane == 0) mbar_wait(&sh.drain_bar, 0, status, 55, abort_flag, false);
  __syncthreads();
  if (leader && warp == 0 && lane == 0) {
    // after an early exit, let the loads in flight land before the CTA ends: the first
    // CTA's full barriers count both CTAs' bytes, and no producer runs more than STAGES
    // loads ahead of the MMAs
    const int last = max(sh.prod_it, sh.mma_it + (PAIR && *abort_flag ? STAGES : 0));
    for (int j = sh.mma_it; j < last; ++j)
      mbar_wait(&full_bar[j % STAGES], (j / STAGES) & 1, status, 56, abort_flag, false);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, Cfg::TMEM_COLS);
    else tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
  }
}

template <class T, bool FORWARD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(640, 1)
    lin_pair_kernel(const __grid_constant__ LinParams<FORWARD ? 1 : 2> p) {
  lin_body<T, FORWARD, true>(p);
}

template <class T, bool FORWARD>
__global__ void __launch_bounds__(640, 1) lin_kernel(const __grid_constant__ LinParams<FORWARD ? 1 : 2> p) {
  lin_body<T, FORWARD, false>(p);
}

// The same epilogue for 8 columns [col, col + 8) of one row, in a warp whose 4 neighbouring lanes
// hold the 32 columns of a block; `in` says whether they lie in the matrix.
template <class T, bool FORWARD>
__device__ __forceinline__ void lin_epilogue8(const LinEpilogue& e, int row, int col, f2 (&v)[4], bool in) {
  if constexpr (!FORWARD) {
    if (!in) return;
    if (e.kind == LIN_STORE) {
      Vec8<T> o;
      o.set(v);
      o.store(static_cast<T*>(e.out) + (long long)row * e.ld_out + col);
      return;
    }
    float* p = static_cast<float*>(e.out) + (long long)row * e.ld_out + col;
    Vec8<float> o;
    if (e.accumulate) {
      f2 was[4];
      o.load_keep(p);
      o.get(was);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = add2(v[j], was[j]);
    }
    o.set(v);
    o.store(p);
  } else {
    if (in && e.bias != nullptr) {
      f2 b[4];
      load_param8<T>(e.bias, e.bias_f32, col, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = add2(v[j], b[j]);
    }
    Vec8<T> o;
    if (in && e.z != nullptr) {
      o.set(v);
      o.store(static_cast<T*>(e.z) + (long long)row * e.ld_z + col);
    }
    if (e.k.q != nullptr) {
      // columns behind the last hold zeros, as in the product kernel
      Vec8<float> f;
      f.set(v);
      const uint32_t amax = f.block_max();
      if (row < e.M && (col & ~31) < e.N)
        ckpt_store8(e.k.q + (long long)row * e.k.ld_q + col,
                    (col & 31) ? nullptr : e.k.e + (long long)row * e.k.ld_e + (col >> 5), v, amax);
    }
    if (!in) return;
    switch (e.act) {
      case MAO_ACT_RELU: act8<MAO_ACT_RELU>(v); break;
      case MAO_ACT_RELU2: act8<MAO_ACT_RELU2>(v); break;
      case MAO_ACT_GELU: act8<MAO_ACT_GELU>(v); break;
      case MAO_ACT_GELU_TANH: act8<MAO_ACT_GELU_TANH>(v); break;
      case MAO_ACT_SILU: act8<MAO_ACT_SILU>(v); break;
      default: break;
    }
    if (e.res != nullptr) {
      f2 r[4];
      o.load(static_cast<const T*>(e.res) + (long long)row * e.ld_res + col);
      o.get(r);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = add2(v[j], r[j]);
    }
    o.set(v);
    o.store(static_cast<T*>(e.out) + (long long)row * e.ld_out + col);
  }
}

// Joins the slices of the sliced tiles in slice order and runs the epilogue.  A thread owns 8
// columns of a row, so a warp reads whole lines (with 32 columns a thread, as in the product
// kernel, 22 tiles of 3 slices took 8 us).  pieces: 8-column pieces of the first problem's
// sliced tiles; the second's follow.
struct LinJoin {
  LinEpilogue e;
  const float* part;
  int tiles_m, tiles_n, full, slices;
};
template <int NP>
struct LinJoins {
  LinJoin p[NP];
  int pieces;
};
constexpr int kJoinThreads = 256;
template <class T, bool FORWARD, int EDGE>
__global__ void __launch_bounds__(kJoinThreads) lin_join_kernel(const LinJoins<FORWARD ? 1 : 2> a) {
  constexpr int BM = EDGE, BN = EDGE;
  wait_for_previous();
  int i = blockIdx.x * kJoinThreads + threadIdx.x;
  const bool second = !FORWARD && i >= a.pieces;  // the same for a block: pieces is a multiple of its size
  if (second) i -= a.pieces;
  const LinJoin& p = a.p[second ? 1 : 0];
  const int sliced = p.tiles_m * p.tiles_n - p.full;
  const int tile = i / (BM * BN / 8);
  const int r = i - tile * (BM * BN / 8);
  int tm, tn;
  lin_tile(p.full + tile, p.tiles_m, p.tiles_n, tm, tn);
  const int row = tm * BM + r / (BN / 8), col = tn * BN + (r % (BN / 8)) * 8;
  const bool in = row < p.e.M && col < p.e.N;
  f2 v[4] = {dup2(0.0f), dup2(0.0f), dup2(0.0f), dup2(0.0f)};
  if (in) {
    const float* s = p.part + (long long)tile * BM * BN + r * 8;
    for (int k = 0; k < p.slices; ++k, s += (long long)sliced * BM * BN) {
      Vec8<float> x;
      x.load(s);
      f2 f[4];
      x.get(f);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = add2(v[j], f[j]);
    }
  }
  lin_epilogue8<T, FORWARD>(p.e, row, col, v, in);
}

}  // namespace mao
