// The linear layer and its gradient (mao_linear, mao_linear_backward): argument checks,
// the choice of tiles and K slices, and the launches.
#include "act_bwd.h"
#include "linear_gemm.cuh"
#include "mao_testing.h"

namespace mao {
namespace {

// ------------------------------------------------------------------ plan
enum LinTile : int { TILE_PAIR = 0, TILE_ONE = 1 };
constexpr int kTileEdge[2] = {256, 128};
constexpr int kPlanSms = 148;

struct Shape {
  long long M, N, K;
};
struct LinPlan {
  int tiles_m = 0, tiles_n = 0, nk = 0, full = 0, slices = 1, slice_blocks = 0;
  size_t part_bytes = 0;
  int items() const { return full + (tiles_m * tiles_n - full) * slices; }
};
struct LinPlans {
  int tile = TILE_ONE;
  LinPlan p[2];  // one product: p[0]
  LinDeal deal = {};
  size_t part_bytes() const { return p[0].part_bytes + p[1].part_bytes; }
};

// Sets a plan to `whole` unsliced tiles and the others in s slices; false if that makes none.
bool cut(LinPlan& p, int whole, int s, int tile_bytes) {
  p.full = whole;
  p.slices = s;
  p.slice_blocks = (p.nk + s - 1) / s;
  const long long rest = (long long)p.tiles_m * p.tiles_n - whole;
  p.part_bytes = s > 1 ? (size_t)s * (size_t)rest * tile_bytes : 0;
  return s == 1 || (rest > 0 && p.slice_blocks >= 4 && (p.nk + p.slice_blocks - 1) / p.slice_blocks == s);
}

// Tiles, K slices and the dealing of one product, or of two that share a launch (the longer K
// first), from their sizes alone (and so the same on every device and in the workspace
// query): of the candidates, the one whose longest list is estimated to end first.
bool search_plan(const Shape* q, int n, LinPlans* out) {
  // ns, fitted to products forced onto either tile, of 33 x 768 -> 2304 to 4001 x 6144 -> 1536,
  // whole and in 2 to 8 slices: a k-block of 64; set-up, first loads and last epilogue; and an
  // item's own share, in k-blocks.  E.g. 2048 x 768 -> 768: 10.5 us in 128 x 128 tiles, 14.6 in
  // 256 x 256; 4001 x 6144 -> 1536: 90 and 61 us; 512 x 4096 -> 4096: 27 and 27 us (in 2 slices)
  constexpr double kBlock[2] = {310.0, 285.0}, kFixed[2] = {7000.0, 7000.0};
  constexpr long long kItem[2] = {8, 4};
  constexpr double kJoin = 2500.0, kJoinBytes = 6000.0;  // the joining kernel; bytes per ns, written and read
  constexpr int kSlices[8] = {1, 2, 3, 4, 6, 8, 12, 16};
  double best = 1e300;
  for (int t = 0; t < 2; ++t) {
    const long long W = t == TILE_ONE ? kPlanSms : kPlanSms / 2;
    const int tile_bytes = 4 * kTileEdge[t] * kTileEdge[t];
    LinPlans c;
    c.tile = t;
    bool fits = true;
    for (int i = 0; i < n; ++i) {
      const long long tm = (q[i].M + kTileEdge[t] - 1) / kTileEdge[t], tn = (q[i].N + kTileEdge[t] - 1) / kTileEdge[t];
      fits = fits && tm * tn <= (1ll << 26);
      c.p[i].tiles_m = (int)tm, c.p[i].tiles_n = (int)tn;
      c.p[i].nk = (int)((q[i].K + 63) / 64);
    }
    if (!fits) continue;
    LinPlan& last = c.p[n - 1];
    const long long tiles0 = n > 1 ? (long long)c.p[0].tiles_m * c.p[0].tiles_n : 0;
    const long long tiles1 = (long long)last.tiles_m * last.tiles_n;
    for (int s0 : kSlices) {
      if (s0 > 1 && (n == 1 || tiles0 >= W)) break;  // the first is cut as a whole, where it is small
      if (n > 1 && !cut(c.p[0], s0 > 1 ? 0 : (int)tiles0, s0, tile_bytes)) continue;
      const long long first = tiles0 * s0, len0 = n > 1 ? c.p[0].slice_blocks + kItem[t] : 0;
      const long long extra = first % W, others = W - extra, base = first / W * len0;
      const long long len1 = last.nk + kItem[t];
      // whole items of the last problem per list, so that the lists end about together
      const long long total = first * len0 + tiles1 * len1;
      const long long y0 = std::max(0ll, (total / W - base) / len1), x0 = std::max(0ll, (total / W - base - len0) / len1);
      for (long long y = y0; y >= std::max(0ll, y0 - 1); --y) {
        for (long long x = extra > 0 ? x0 : 0; x >= std::max(0ll, x0 - 1) || x == 0; --x) {
          if (x > y) continue;
          const long long whole = std::min(tiles1, others * y + extra * x);
          const long long rest = tiles1 - whole;
          for (int s1 : kSlices) {
            if (s1 > 1 && rest == 0) break;
            if (!cut(last, s1 > 1 ? (int)whole : (int)tiles1, s1, tile_bytes)) continue;
            const long long cuts = rest * s1, len = last.slice_blocks + kItem[t];
            const long long most = (cuts + others - 1) / others;
            for (long long v = extra > 0 ? 0 : most; v <= std::min(most, 40ll) || extra == 0; ++v) {
              const long long u = extra > 0 ? (std::max(0ll, cuts - others * v) + extra - 1) / extra : 0;
              const long long longest = base + std::max(y * len1 + v * len, extra > 0 ? len0 + x * len1 + u * len : 0ll);
              const size_t bytes = c.part_bytes();
              const double cost = (double)longest * kBlock[t] + kFixed[t] +
                                  (bytes > 0 ? kJoin + 2.0 * (double)bytes / kJoinBytes : 0.0);
              if (cost < best) {
                best = cost;
                c.deal = LinDeal{(int)W, (int)first, (int)extra, (int)whole, (int)y, (int)(extra > 0 ? y - x : 0), (int)cuts, (int)v};
                *out = c;
              }
              if (extra == 0) break;
            }
          }
          if (x == 0) break;
        }
      }
    }
  }
  return best < 1e300;
}

// The search takes some tens of microseconds; a program calls with few sizes, so each thread
// keeps the plans of its latest ones.
bool plan_of(const Shape* q, int n, LinPlans* out) {
  struct Entry {
    int n = 0;
    Shape q[2] = {};
    LinPlans plans;
  };
  static thread_local Entry cache[32];
  unsigned long long h = (unsigned long long)n;
  for (int i = 0; i < n; ++i)
    h = (((h * 0x9E3779B97F4A7C15ull + (unsigned long long)q[i].M) * 0x9E3779B97F4A7C15ull + (unsigned long long)q[i].N) *
         0x9E3779B97F4A7C15ull) + (unsigned long long)q[i].K;
  Entry& e = cache[(h * 0x9E3779B97F4A7C15ull) >> 59];
  bool same = e.n == n;
  for (int i = 0; same && i < n; ++i) same = e.q[i].M == q[i].M && e.q[i].N == q[i].N && e.q[i].K == q[i].K;
  if (!same) {
    e.n = 0;
    if (!search_plan(q, n, &e.plans)) return false;
    for (int i = 0; i < n; ++i) e.q[i] = q[i];
    e.n = n;
  }
  *out = e.plans;
  return true;
}

// ------------------------------------------------------------------ launch
template <class T, bool FORWARD, bool PAIR>
mao_status launch_product(const LinParams<FORWARD ? 1 : 2>& p, int items, bool dependent, const DeviceInfo& dev,
                          cudaStream_t stream) {
  using Cfg = LinCfg<PAIR>;
  void (*kern)(LinParams<FORWARD ? 1 : 2>);
  if constexpr (PAIR) kern = lin_pair_kernel<T, FORWARD>;
  else kern = lin_kernel<T, FORWARD>;
  static std::atomic<bool> done[64];
  MAO_TRY(allow_smem(kern, Cfg::SMEM_BYTES, done));
  const int workers = std::min({items, p.deal.workers, PAIR ? dev.sm_count / 2 : dev.sm_count});
  const int grid = PAIR ? 2 * workers : workers;
  if (dependent) return launch_dependent(kern, dim3(grid), Cfg::THREADS, Cfg::SMEM_BYTES, stream, p);
  kern<<<grid, Cfg::THREADS, Cfg::SMEM_BYTES, stream>>>(p);
  return launched();
}

struct Operand {
  const void* p;
  long long inner, rows, ld;  // stored matrix: rows x inner
};

// K-major: boxes of 128 rows; MN-major: of 64 columns
mao_status encode(CUtensorMap* map, int dtype, const Operand& o, bool mn) {
  return encode_3d(map, dtype == MAO_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, o.p,
                   (uint64_t)o.inner, (uint64_t)o.rows, 1, (uint64_t)o.ld, (uint64_t)o.ld * o.rows, 64,
                   mn ? 64 : 128);
}

// One product of a launch: out = A B^T with the stored operands as described.
struct Product {
  Operand A, B;
  int a_mn;  // A's major
  LinEpilogue e;
  Shape shape() const { return Shape{e.M, e.N, a_mn ? A.rows : A.inner}; }
};

// One or two products in one launch, then the joining of their slices.  dependent: a kernel of
// this call comes before in the stream.
template <class T, bool FORWARD>
mao_status products(const Product* q, int n, const LinPlans& plans, const LinColSum& sum, float* part, int kernel_id,
                    double bytes, bool dependent, cudaStream_t stream) {
  constexpr int NP = FORWARD ? 1 : 2;
  DeviceInfo* dev = nullptr;
  MAO_TRY(device_info(&dev));
  LinParams<NP> a;
  LinJoins<NP> j;
  std::memset(&a, 0, sizeof(a));
  std::memset(&j, 0, sizeof(j));
  a.sum = sum;
  a.deal = plans.deal;
  double flops = 0.0;
  int items = 0, pieces = 0;
  for (int i = 0; i < n; ++i) {
    const LinPlan& c = plans.p[i];
    const int slot = i + NP - n;  // a single product of the backward pass is its kernel's last
    LinProblem& p = a.p[slot];
    MAO_TRY(encode(&p.mapA, Elem<T>::kDtype, q[i].A, q[i].a_mn));
    MAO_TRY(encode(&p.mapB, Elem<T>::kDtype, q[i].B, !FORWARD));
    p.e = q[i].e;
    p.part = part;
    part += c.part_bytes / sizeof(float);
    p.a_mn = q[i].a_mn;
    p.tiles_m = c.tiles_m, p.tiles_n = c.tiles_n;
    p.full = c.full, p.slices = c.slices;
    p.nk = c.nk, p.slice_blocks = c.slice_blocks;
    const bool kept = p.e.k.q != nullptr;
    p.fold = kept || p.e.kind == LIN_GRAD32 ? fold_blocks(c.nk, kept) : equal_parts(c.nk, kLongFold);
    items += c.items();
    const Shape s = q[i].shape();
    flops += 2.0 * (double)s.M * (double)s.N * (double)s.K;
    j.p[slot] = LinJoin{p.e, p.part, c.tiles_m, c.tiles_n, c.full, c.slices};
    if (c.slices > 1) {
      // a few rounds of tiles at most: far below 2^31 pieces, a multiple of a block's
      const int k = (c.tiles_m * c.tiles_n - c.full) * (kTileEdge[plans.tile] * kTileEdge[plans.tile] / 8);
      if (slot == 0) j.pieces = k;
      pieces += k;
    }
  }
  if (n < NP) a.p[0].mapA = a.p[NP - 1].mapA, a.p[0].mapB = a.p[NP - 1].mapB;  // prefetched, not used
  {
    LaunchScope ls(stream, kernel_id, flops, bytes);
    MAO_TRY(plans.tile == TILE_PAIR ? (launch_product<T, FORWARD, true>(a, items, dependent, *dev, stream))
                                    : (launch_product<T, FORWARD, false>(a, items, dependent, *dev, stream)));
  }
  if (pieces == 0) return MAO_OK;
  LaunchScope ls(stream, MAO_K_SLICE_REDUCE, 0.0, (double)plans.part_bytes());
  const dim3 grid(pieces / kJoinThreads);
  return plans.tile == TILE_PAIR
             ? launch_dependent(lin_join_kernel<T, FORWARD, 256>, grid, kJoinThreads, 0, stream, j)
             : launch_dependent(lin_join_kernel<T, FORWARD, 128>, grid, kJoinThreads, 0, stream, j);
}

LinEpilogue epilogue(void* out, long long ld, int M, int N, int kind) {
  LinEpilogue e;
  std::memset(&e, 0, sizeof(e));
  e.out = out, e.ld_out = ld, e.M = M, e.N = N, e.kind = kind;
  return e;
}

// ------------------------------------------------------------------ checks
mao_status check_sizes(int dtype, int rows, int n, int m) {
  if (!is16(dtype)) return MAO_ERR_DTYPE;
  MAO_TRY(check_dims(rows, n));
  MAO_TRY(check_dims(rows, m));
  return MAO_OK;
}

// an operand's extent must stay in a tensor map's strides (2^40 bytes)
mao_status check_extent(long long rows, long long ld) {
  return rows == 0 || ld <= ((1ll << 39) - 1) / rows ? MAO_OK : MAO_ERR_SHAPE;
}

mao_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MAO_OK;
  if (ws == nullptr || have < need) return MAO_ERR_WORKSPACE;
  return (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 ? MAO_OK : MAO_ERR_ALIGN;
}

struct BwdLayout {
  LinPlans plans;       // of the products asked for, the longer K first
  int products = 0;
  bool dx_first = false;
  int chunks = 0;       // partial rows of the bias gradient
  size_t dz = 0, x = 0, db = 0, part = 0, total = 0;
};

mao_status backward_layout(const mao_linear_backward_args* a, BwdLayout* L) {
  if (a == nullptr) return MAO_ERR_INVALID_ARG;
  MAO_TRY(check_sizes(a->dtype, a->rows, a->n, a->m));
  if (a->act < MAO_ACT_NONE || a->act > MAO_ACT_SILU) return MAO_ERR_INVALID_ARG;
  if (a->rows == 0) return MAO_OK;
  Carver cv;
  const size_t rows = (size_t)a->rows;
  if (a->act != MAO_ACT_NONE && (a->dx || a->dW)) L->dz = cv.take(2 * rows * a->m);
  if (a->dW && a->x == nullptr) L->x = cv.take(2 * rows * a->n);
  if (a->db) {
    const int chunk = act_bwd_chunk(a->rows, a->m);
    L->chunks = (a->rows + chunk - 1) / chunk;
    L->db = cv.take(sizeof(float) * (size_t)L->chunks * a->m);
  }
  const Shape dx{a->rows, a->n, a->m}, dw{a->m, a->n, a->rows};
  L->dx_first = a->dx && (!a->dW || a->m >= a->rows);
  Shape q[2];
  if (L->dx_first) q[L->products++] = dx;
  if (a->dW) q[L->products++] = dw;
  if (a->dx && !L->dx_first) q[L->products++] = dx;
  if (L->products > 0 && !plan_of(q, L->products, &L->plans)) return MAO_ERR_SHAPE;
  L->part = cv.take(L->plans.part_bytes());
  L->total = cv.total();
  return MAO_OK;
}

template <class T>
mao_status forward(const mao_linear_args* a, const LinPlans& plans, float* part, cudaStream_t stream) {
  LinEpilogue e = epilogue(a->y, a->ld_y, a->rows, a->m, LIN_FORWARD);
  e.bias = a->b, e.bias_f32 = a->b_dtype == MAO_F32;
  e.res = a->res, e.ld_res = a->ld_res;
  e.z = a->z, e.ld_z = a->ld_z;
  e.k = view(a->zc);
  e.act = a->act;
  const Product q{{a->x, a->n, a->rows, a->ld_x}, {a->W, a->n, a->m, a->n}, 0, e};
  const double r = a->rows, n = a->n, m = a->m;
  return products<T, true>(&q, 1, plans, LinColSum{}, part, MAO_K_LINEAR,
                           2.0 * (r * n + m * n + r * m) + (a->res ? 2.0 * r * m : 0.0) + (a->z ? 2.0 * r * m : 0.0) +
                               (a->zc.q ? r * m * (1.0 + 1.0 / 32) : 0.0),
                           false, stream);
}

// One elementwise launch (dz, the bias gradient's partial sums, x read back), then one launch
// for both products, which also joins the bias gradient.
template <class T>
mao_status backward(const mao_linear_backward_args* a, const BwdLayout& L, uint8_t* ws, cudaStream_t stream) {
  const bool has_act = a->act != MAO_ACT_NONE;
  ActBwd b = {};
  b.dy = a->dy, b.ld_dy = a->ld_dy;
  b.z = a->z, b.ld_z = a->ld_z, b.zk = view(a->zc);
  b.act = a->act;
  b.rows = a->rows, b.cols = a->m;
  if (has_act && L.products > 0) b.dz = ws + L.dz, b.ld_dz = a->m;
  if (a->db) b.part = reinterpret_cast<float*>(ws + L.db);
  if (a->dW && a->x == nullptr) b.xk = view(a->xc), b.xr = ws + L.x, b.x_cols = a->n;
  const bool prepared = b.dz || b.part || b.xr;
  if (prepared) MAO_TRY(act_bwd_launch(b, a->dtype, stream));
  const double r = a->rows, n = a->n, m = a->m;
  if (L.products == 0) {
    if (a->db) return col_sum_launch(b.part, L.chunks, a->m, a->db, stream);
    return MAO_OK;
  }
  const Operand Z = b.dz ? Operand{b.dz, a->m, a->rows, a->m} : Operand{a->dy, a->m, a->rows, a->ld_dy};
  const Operand X = b.xr ? Operand{b.xr, a->n, a->rows, a->n} : Operand{a->x, a->n, a->rows, a->ld_x};
  Product dx{Z, {a->W, a->n, a->m, a->n}, 0, epilogue(a->dx, a->ld_dx, a->rows, a->n, LIN_STORE)};
  Product dw{Z, X, 1, epilogue(a->dW, a->n, a->m, a->n, a->dw_dtype == MAO_F32 ? LIN_GRAD32 : LIN_STORE)};
  dw.e.accumulate = a->accumulate;
  Product q[2];
  int k = 0;
  if (L.dx_first) q[k++] = dx;
  if (a->dW) q[k++] = dw;
  if (a->dx && !L.dx_first) q[k++] = dx;
  const LinColSum sum{b.part, a->db, L.chunks, a->m};
  const double dw_bytes = (a->dw_dtype == MAO_F32 ? 4.0 : 2.0) * m * n;
  return products<T, false>(q, k, L.plans, sum, reinterpret_cast<float*>(ws + L.part),
                            k == 2 ? MAO_K_LINEAR_BWD : (a->dx ? MAO_K_LINEAR_DX : MAO_K_LINEAR_DW),
                            2.0 * r * m + (a->dx ? 2.0 * (m * n + r * n) : 0.0) + (a->dW ? 2.0 * r * n + dw_bytes : 0.0),
                            prepared, stream);
}

}  // namespace
}  // namespace mao

using namespace mao;

extern "C" mao_status mao_linear_workspace_size(const mao_linear_args* a, size_t* bytes) {
  if (a == nullptr || bytes == nullptr) return MAO_ERR_INVALID_ARG;
  MAO_TRY(check_sizes(a->dtype, a->rows, a->n, a->m));
  *bytes = 0;
  if (a->rows == 0) return MAO_OK;
  LinPlans plans;
  const Shape q{a->rows, a->m, a->n};
  if (!plan_of(&q, 1, &plans)) return MAO_ERR_SHAPE;
  *bytes = align_up(plans.part_bytes(), 256);
  return MAO_OK;
}

extern "C" mao_status mao_linear(const mao_linear_args* a, void* workspace, size_t ws_bytes, mao_stream_t stream_) {
  size_t need = 0;
  MAO_TRY(mao_linear_workspace_size(a, &need));
  if (a->act < MAO_ACT_NONE || a->act > MAO_ACT_SILU) return MAO_ERR_INVALID_ARG;
  if (a->W == nullptr) return MAO_ERR_INVALID_ARG;
  if (a->b != nullptr && a->b_dtype != MAO_F32 && a->b_dtype != a->dtype) return MAO_ERR_DTYPE;
  MAO_TRY(check_acts(a->x, a->rows, a->n, a->ld_x));
  MAO_TRY(check_acts(a->y, a->rows, a->m, a->ld_y));
  if (a->res != nullptr) MAO_TRY(check_acts(a->res, a->rows, a->m, a->ld_res));
  if (a->z != nullptr) MAO_TRY(check_acts(a->z, a->rows, a->m, a->ld_z));
  if (a->zc.q != nullptr) MAO_TRY(check_ckpt(a->zc, a->rows, a->m));
  if (!aligned16(a->W) || !aligned16(a->b)) return MAO_ERR_ALIGN;
  MAO_TRY(check_extent(a->rows, a->ld_x));
  MAO_TRY(check_extent(a->m, a->n));
  MAO_TRY(check_workspace(workspace, ws_bytes, need));
  DeviceInfo* dev = nullptr;
  MAO_TRY(device_info(&dev));
  if (a->rows == 0) return MAO_OK;
  LinPlans plans;
  const Shape q{a->rows, a->m, a->n};
  if (!plan_of(&q, 1, &plans)) return MAO_ERR_SHAPE;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  float* part = static_cast<float*>(workspace);
  return a->dtype == MAO_BF16 ? forward<__nv_bfloat16>(a, plans, part, stream) : forward<__half>(a, plans, part, stream);
}

extern "C" mao_status mao_linear_backward_workspace_size(const mao_linear_backward_args* a, size_t* bytes) {
  if (bytes == nullptr) return MAO_ERR_INVALID_ARG;
  BwdLayout L;
  MAO_TRY(backward_layout(a, &L));
  *bytes = L.total;
  return MAO_OK;
}

extern "C" mao_status mao_linear_backward(const mao_linear_backward_args* a, void* workspace, size_t ws_bytes,
                                          mao_stream_t stream_) {
  BwdLayout L;
  MAO_TRY(backward_layout(a, &L));
  MAO_TRY(check_acts(a->dy, a->rows, a->m, a->ld_dy));
  if (a->dW != nullptr) {
    if (a->dw_dtype != MAO_F32 && a->dw_dtype != a->dtype) return MAO_ERR_DTYPE;
    if (a->accumulate && a->dw_dtype != MAO_F32) return MAO_ERR_DTYPE;
    if (a->x == nullptr && a->xc.q != nullptr) MAO_TRY(check_ckpt(a->xc, a->rows, a->n));
    else MAO_TRY(check_acts(a->x, a->rows, a->n, a->ld_x));
    if (a->x != nullptr) MAO_TRY(check_extent(a->rows, a->ld_x));
  }
  if (a->act != MAO_ACT_NONE) {
    if (a->z == nullptr && a->zc.q != nullptr) MAO_TRY(check_ckpt(a->zc, a->rows, a->m));
    else MAO_TRY(check_acts(a->z, a->rows, a->m, a->ld_z));
  }
  if (a->dx != nullptr) {
    if (a->W == nullptr) return MAO_ERR_INVALID_ARG;
    MAO_TRY(check_acts(a->dx, a->rows, a->n, a->ld_dx));
  }
  if (!aligned16(a->W) || !aligned16(a->dW) || !aligned16(a->db)) return MAO_ERR_ALIGN;
  MAO_TRY(check_extent(a->rows, a->ld_dy));
  MAO_TRY(check_extent(a->rows, std::max(a->n, a->m)));
  MAO_TRY(check_extent(a->m, a->n));
  MAO_TRY(check_workspace(workspace, ws_bytes, L.total));
  DeviceInfo* dev = nullptr;
  MAO_TRY(device_info(&dev));
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (a->rows == 0) {
    if (a->dW && !a->accumulate)
      MAO_CUDA_TRY(cudaMemsetAsync(a->dW, 0, (size_t)elem_size(a->dw_dtype) * a->m * a->n, stream));
    if (a->db) MAO_CUDA_TRY(cudaMemsetAsync(a->db, 0, sizeof(float) * a->m, stream));
    return MAO_OK;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return a->dtype == MAO_BF16 ? backward<__nv_bfloat16>(a, L, ws, stream) : backward<__half>(a, L, ws, stream);
}

extern "C" mao_status mao_layer_status(mao_stream_t stream, int32_t* where) {
  DevStatus st;
  MAO_CUDA_TRY(cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)));
  MAO_CUDA_TRY(cudaMemcpyFromSymbol(&st, g_layer_status, sizeof(st)));
  if (where) *where = st.where;
  if (st.code != MAO_OK) {
    const DevStatus clear = {};
    MAO_CUDA_TRY(cudaMemcpyToSymbol(g_layer_status, &clear, sizeof(clear)));
  }
  return static_cast<mao_status>(st.code);
}

// ------------------------------------------------------------------ verification
namespace {
template <int NP>
void deal_out(const LinDeal& deal, int workers, uint8_t* dealt, const size_t (&from)[2], const size_t (&items)[2], size_t* stray) {
  for (int w = 0; w < workers; ++w) {
    LinWalk<NP> walk(w, workers);
    for (int which = 0, item = 0; walk.next(deal, which, item);) {
      if (item < 0 || (size_t)item >= items[which]) ++*stray;
      else if (dealt[from[which] + item] < 255) ++dealt[from[which] + item];
    }
  }
}
}  // namespace

extern "C" mao_status mao_test_linear_deal(const int64_t* sizes, int32_t products, int32_t backward, int32_t workers,
                                           int32_t* plan, uint8_t* dealt, size_t dealt_bytes) {
  if (sizes == nullptr || plan == nullptr || dealt == nullptr || workers < 1) return MAO_ERR_INVALID_ARG;
  if (products < 1 || products > (backward ? 2 : 1)) return MAO_ERR_INVALID_ARG;
  Shape q[2] = {};
  for (int i = 0; i < products; ++i) {
    q[i] = Shape{sizes[3 * i], sizes[3 * i + 1], sizes[3 * i + 2]};
    if (q[i].M < 1 || q[i].N < 1 || q[i].K < 1 || std::max({q[i].M, q[i].N, q[i].K}) > (1ll << 30)) return MAO_ERR_SHAPE;
  }
  LinPlans plans;
  if (!plan_of(q, products, &plans)) return MAO_ERR_SHAPE;
  plan[0] = kTileEdge[plans.tile];
  plan[1] = plans.deal.workers;
  size_t from[2] = {0, 0}, items[2] = {0, 0}, total = 0, stray = 0;
  for (int i = 0; i < products; ++i) {
    const LinPlan& c = plans.p[i];
    const int32_t put[6] = {c.tiles_m, c.tiles_n, c.nk, c.full, c.slices, c.slice_blocks};
    std::memcpy(plan + 2 + 6 * i, put, sizeof(put));
    const int slot = i + (backward ? 2 : 1) - products;  // as in products()
    from[slot] = total;
    items[slot] = (size_t)c.items();
    total += items[slot];
  }
  if (total > dealt_bytes) return MAO_ERR_WORKSPACE;
  std::memset(dealt, 0, total);
  if (backward) deal_out<2>(plans.deal, workers, dealt, from, items, &stray);
  else deal_out<1>(plans.deal, workers, dealt, from, items, &stray);
  return stray == 0 ? MAO_OK : MAO_ERR_UNSUPPORTED;
}

extern "C" mao_status mao_test_set_layer_status(int32_t code, int32_t where) {
  const DevStatus st = {code, where, 0, 0};
  MAO_CUDA_TRY(cudaMemcpyToSymbol(g_layer_status, &st, sizeof(st)));
  return MAO_OK;
}
