// The linear layer and its gradient (mao_linear, mao_linear_backward): argument checks,
// the choice of tiles and K slices, and the launches.
#include "act_bwd.h"
#include "linear_gemm.cuh"

namespace mao {
namespace {

// ------------------------------------------------------------------ plan
enum LinTile : int { TILE_PAIR256 = 0, TILE_PAIR128 = 1, TILE_ONE = 2 };
constexpr int kTileM[3] = {256, 256, 128}, kTileN[3] = {256, 128, 128};

struct LinPlan {
  int tile = TILE_ONE;
  int tiles_m = 0, tiles_n = 0, nk = 0, full = 0, slices = 1, slice_blocks = 0;
  int items = 0;
  size_t part_bytes = 0;
};

// Tiles and K slices of an M x N x K product, from its sizes alone (and so the same on
// every device and in the workspace query): the cheapest by estimated clocks.
constexpr int kPlanSms = 148;

bool plan_of(long long M, long long N, long long K, LinPlan* out) {
  // clocks of a k-block of 64, of the last epilogue, and of a join of the slices
  constexpr double kBlock[3] = {530.0, 400.0, 700.0}, kTail[3] = {5000.0, 4000.0, 4000.0};
  constexpr double kJoin = 7000.0, kJoinBytes = 2000.0;  // launch; bytes per clock
  const long long nk = (K + 63) / 64;
  double best = 1e300;
  for (int t = 0; t < 3; ++t) {
    const long long tm = (M + kTileM[t] - 1) / kTileM[t], tn = (N + kTileN[t] - 1) / kTileN[t], tiles = tm * tn;
    if (tiles > (1ll << 27)) continue;
    const long long workers = t == TILE_ONE ? kPlanSms : kPlanSms / 2;
    const long long waves = tiles / workers, rest = tiles - waves * workers;
    for (int s = 1; s <= 16; ++s) {
      const long long sb = (nk + s - 1) / s;
      if (s > 1 && (rest == 0 || sb < 4 || (nk + sb - 1) / sb != s)) break;
      const long long rounds = (rest * s + workers - 1) / workers;
      double cost = (double)(waves * nk + rounds * sb) * kBlock[t] + kTail[t];
      const double bytes = s > 1 ? 4.0 * s * (double)rest * kTileM[t] * kTileN[t] : 0.0;
      if (s > 1) cost += kJoin + 2.0 * bytes / kJoinBytes;
      if (cost < best) {
        best = cost;
        out->tile = t;
        out->tiles_m = (int)tm, out->tiles_n = (int)tn, out->nk = (int)nk;
        out->full = (int)(s > 1 ? tiles - rest : tiles);
        out->slices = s, out->slice_blocks = (int)sb;
        out->items = out->full + (int)(tiles - out->full) * s;
        out->part_bytes = (size_t)bytes;
      }
    }
  }
  return best < 1e300;
}

// ------------------------------------------------------------------ launch
template <class T, int KIND, int A_MN, int B_MN, bool PAIR, int BN>
mao_status launch_product(const LinParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  using Cfg = LinCfg<PAIR, BN>;
  void (*kern)(LinParams);
  if constexpr (PAIR) kern = lin_pair_kernel<T, KIND, A_MN, B_MN, BN>;
  else kern = lin_kernel<T, KIND, A_MN, B_MN>;
  static std::atomic<bool> done[64];
  MAO_TRY(allow_smem(kern, Cfg::SMEM_BYTES, done));
  const int workers = std::min(p.items, PAIR ? dev.sm_count / 2 : dev.sm_count);
  kern<<<PAIR ? 2 * workers : workers, Cfg::THREADS, Cfg::SMEM_BYTES, stream>>>(p);
  return launched();
}

struct Operand {
  const void* p;
  long long inner, rows, ld;  // stored matrix: rows x inner
};

// box_rows: the rows of a K-major tile that one CTA loads
mao_status encode(CUtensorMap* map, int dtype, const Operand& o, bool mn, int box_rows) {
  return encode_3d(map, dtype == MAO_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, o.p,
                   (uint64_t)o.inner, (uint64_t)o.rows, 1, (uint64_t)o.ld, (uint64_t)o.ld * o.rows, 64,
                   mn ? 64 : box_rows);
}

template <class T, int KIND, int A_MN, int B_MN>
mao_status product(const Operand& A, const Operand& B, const LinEpilogue& e, const LinPlan& plan, float* part,
                   int kernel_id, double bytes, cudaStream_t stream) {
  DeviceInfo* dev = nullptr;
  MAO_TRY(device_info(&dev));
  LinParams p;
  MAO_TRY(encode(&p.mapA, Elem<T>::kDtype, A, A_MN, 128));
  MAO_TRY(encode(&p.mapB, Elem<T>::kDtype, B, B_MN, plan.tile == TILE_PAIR128 ? 64 : 128));
  p.e = e;
  p.part = part;
  p.tiles_m = plan.tiles_m, p.tiles_n = plan.tiles_n;
  p.full = plan.full, p.slices = plan.slices, p.slice_blocks = plan.slice_blocks;
  p.nk = plan.nk, p.items = plan.items;
  const long long K = A_MN ? A.rows : A.inner;
  {
    LaunchScope ls(stream, kernel_id, 2.0 * e.M * (double)e.N * (double)K, bytes);
    switch (plan.tile) {
      case TILE_PAIR256: MAO_TRY((launch_product<T, KIND, A_MN, B_MN, true, 256>(p, *dev, stream))); break;
      case TILE_PAIR128: MAO_TRY((launch_product<T, KIND, A_MN, B_MN, true, 128>(p, *dev, stream))); break;
      default: MAO_TRY((launch_product<T, KIND, A_MN, B_MN, false, 128>(p, *dev, stream))); break;
    }
  }
  if (plan.slices == 1) return MAO_OK;
  const LinJoin j{e, part, plan.tiles_m, plan.tiles_n, plan.full, plan.slices};
  // at most one wave of tiles: far below 2^31 pieces
  const int pieces = (plan.tiles_m * plan.tiles_n - plan.full) * (kTileM[plan.tile] * kTileN[plan.tile] / 32);
  LaunchScope ls(stream, MAO_K_SLICE_REDUCE, 0.0, (double)plan.part_bytes);
  switch (plan.tile) {
    case TILE_PAIR256: lin_join_kernel<T, KIND, 256, 256><<<pieces / 128, 128, 0, stream>>>(j); break;
    case TILE_PAIR128: lin_join_kernel<T, KIND, 256, 128><<<pieces / 128, 128, 0, stream>>>(j); break;
    default: lin_join_kernel<T, KIND, 128, 128><<<pieces / 128, 128, 0, stream>>>(j); break;
  }
  return launched();
}

LinEpilogue epilogue(void* out, long long ld, int M, int N) {
  LinEpilogue e;
  std::memset(&e, 0, sizeof(e));
  e.out = out, e.ld_out = ld, e.M = M, e.N = N;
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
  LinPlan dx, dw;
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
    L->db = cv.take(sizeof(float) * (size_t)((a->rows + chunk - 1) / chunk) * a->m);
  }
  if (a->dx && !plan_of(a->rows, a->n, a->m, &L->dx)) return MAO_ERR_SHAPE;
  if (a->dW && !plan_of(a->m, a->n, a->rows, &L->dw)) return MAO_ERR_SHAPE;
  // one after the other on the stream: they share the slices' room
  L->part = cv.take(std::max(L->dx.part_bytes, L->dw.part_bytes));
  L->total = cv.total();
  return MAO_OK;
}

template <class T>
mao_status forward(const mao_linear_args* a, const LinPlan& plan, float* part, cudaStream_t stream) {
  LinEpilogue e = epilogue(a->y, a->ld_y, a->rows, a->m);
  e.bias = a->b, e.bias_f32 = a->b_dtype == MAO_F32;
  e.res = a->res, e.ld_res = a->ld_res;
  e.z = a->z, e.ld_z = a->ld_z;
  e.k = view(a->zc);
  e.act = a->act;
  const Operand x{a->x, a->n, a->rows, a->ld_x}, W{a->W, a->n, a->m, a->n};
  const double r = a->rows, n = a->n, m = a->m;
  return product<T, LIN_FORWARD, 0, 0>(x, W, e, plan, part, MAO_K_LINEAR,
                                       2.0 * (r * n + m * n + r * m) + (a->res ? 2.0 * r * m : 0.0) +
                                           (a->z ? 2.0 * r * m : 0.0) + (a->zc.q ? r * m * (1.0 + 1.0 / 32) : 0.0),
                                       stream);
}

template <class T>
mao_status backward(const mao_linear_backward_args* a, const BwdLayout& L, uint8_t* ws, cudaStream_t stream) {
  const bool has_act = a->act != MAO_ACT_NONE;
  const bool products = a->dx || a->dW;
  const void* dz = a->dy;
  long long ld_dz = a->ld_dy;
  if ((has_act && products) || a->db) {
    void* out = has_act && products ? ws + L.dz : nullptr;
    float* part = a->db ? reinterpret_cast<float*>(ws + L.db) : nullptr;
    MAO_TRY(act_bwd_launch(a->dy, a->ld_dy, a->z, a->ld_z, view(a->zc), a->z == nullptr, a->act, a->dtype, a->rows,
                           a->m, out, a->m, part, stream));
    if (out) dz = out, ld_dz = a->m;
    if (a->db) {
      const int chunk = act_bwd_chunk(a->rows, a->m);
      MAO_TRY(col_reduce_launch(part, (a->rows + chunk - 1) / chunk, a->m, a->db, nullptr, stream));
    }
  }
  float* part = reinterpret_cast<float*>(ws + L.part);
  const double r = a->rows, n = a->n, m = a->m;
  const Operand Z{dz, a->m, a->rows, ld_dz};
  if (a->dx) {
    const LinEpilogue e = epilogue(a->dx, a->ld_dx, a->rows, a->n);
    const Operand W{a->W, a->n, a->m, a->n};
    MAO_TRY((product<T, LIN_STORE, 0, 1>(Z, W, e, L.dx, part, MAO_K_LINEAR_DX, 2.0 * (r * n + m * n + r * m), stream)));
  }
  if (a->dW) {
    Operand X{a->x, a->n, a->rows, a->ld_x};
    if (a->x == nullptr) {
      MAO_TRY(restore_launch(view(a->xc), a->rows, a->n, MAO_ACT_NONE, ws + L.x, a->dtype, a->n, stream));
      X.p = ws + L.x, X.ld = a->n;
    }
    LinEpilogue e = epilogue(a->dW, a->n, a->m, a->n);
    e.accumulate = a->accumulate;
    if (a->dw_dtype == MAO_F32)
      return product<T, LIN_GRAD32, 1, 1>(Z, X, e, L.dw, part, MAO_K_LINEAR_DW, 2.0 * (r * n + r * m) + 4.0 * m * n, stream);
    return product<T, LIN_STORE, 1, 1>(Z, X, e, L.dw, part, MAO_K_LINEAR_DW, 2.0 * (r * n + r * m + m * n), stream);
  }
  return MAO_OK;
}

}  // namespace
}  // namespace mao

using namespace mao;

extern "C" mao_status mao_linear_workspace_size(const mao_linear_args* a, size_t* bytes) {
  if (a == nullptr || bytes == nullptr) return MAO_ERR_INVALID_ARG;
  MAO_TRY(check_sizes(a->dtype, a->rows, a->n, a->m));
  *bytes = 0;
  if (a->rows == 0) return MAO_OK;
  LinPlan plan;
  if (!plan_of(a->rows, a->m, a->n, &plan)) return MAO_ERR_SHAPE;
  *bytes = align_up(plan.part_bytes, 256);
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
  LinPlan plan;
  if (!plan_of(a->rows, a->m, a->n, &plan)) return MAO_ERR_SHAPE;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  float* part = static_cast<float*>(workspace);
  return a->dtype == MAO_BF16 ? forward<__nv_bfloat16>(a, plan, part, stream) : forward<__half>(a, plan, part, stream);
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
