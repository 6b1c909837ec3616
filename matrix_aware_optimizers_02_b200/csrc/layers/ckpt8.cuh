// Reading an 8-bit checkpoint back: the walk over its vectors and the pass itself, shared by
// the read-back kernels and the linear layer's backward pass.
#pragma once

#include <algorithm>

#include "layer_math.cuh"

namespace mao {

constexpr int kCkptThreads = 256;
constexpr int kCkptUnroll = 4;

// A thread's walk over vectors of 8: a block takes tiles of kCkptUnroll * kCkptThreads consecutive
// vectors, the grid's number of blocks apart, a thread kCkptUnroll of each, kCkptThreads apart.  One division at
// the start, then additions: (row, vector) moves by (dr, dv) inside a tile and by (tr, tv) to
// the next one (a division per vector made the read-back issue-bound: 133 instructions each).
struct Steps {
  long long total;  // vectors
  int rows, vpr, dr, dv, tr, tv;
};
struct Walk {
  long long row;
  int v;
  __device__ __forceinline__ Walk(const Steps& s, int block) {
    const uint32_t i = block * (kCkptThreads * kCkptUnroll) + threadIdx.x;  // below 2^31
    const uint32_t r = i / (uint32_t)s.vpr;
    row = r;
    v = (int)(i - r * (uint32_t)s.vpr);
  }
  __device__ __forceinline__ void move(int dr, int dv, int vpr) {
    row += dr;
    v += dv;
    if (v >= vpr) v -= vpr, ++row;
  }
};

// Block `block` of the pass's blocks.
template <class T, int ACT>
__device__ __forceinline__ void restore_block(const CkptView& k, T* __restrict__ y, long long ld_y, const Steps& st,
                                              int block) {
  Walk at(st, block);
  while (at.row < st.rows) {
    CkptVec8 v[kCkptUnroll];
    long long row[kCkptUnroll];
    int col[kCkptUnroll];
#pragma unroll
    for (int u = 0; u < kCkptUnroll; ++u) {
      row[u] = at.row;
      col[u] = at.v * 8;
      if (at.row < st.rows) v[u].load(k, at.row, col[u]);
      at.move(st.dr, st.dv, st.vpr);
    }
    at.move(st.tr, st.tv, st.vpr);
#pragma unroll
    for (int u = 0; u < kCkptUnroll; ++u) {
      if (row[u] >= st.rows) break;
      f2 f[4];
      v[u].get(f);
      Vec8<T> o;
      if constexpr (ACT == MAO_ACT_NONE) {
        o.set_exact(f);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = act_value<ACT, sizeof(T) == 4>(f[j]);
        o.set(f);
      }
      o.store(y + row[u] * ld_y + col[u]);
    }
  }
}

// One wave of blocks walks everything; never more blocks than vectors ask for.
inline unsigned steps_of(int rows, int vpr, int sms, Steps* s) {
  s->total = (long long)rows * vpr;
  s->rows = rows;
  s->vpr = vpr;
  const long long tile = kCkptThreads * kCkptUnroll;
  const long long grid = std::min<long long>((s->total + tile - 1) / tile, 8ll * sms);
  s->dr = kCkptThreads / vpr;
  s->dv = kCkptThreads % vpr;
  const long long rest = (grid - 1) * tile;  // a tile's kCkptUnroll moves have covered the first
  s->tr = (int)(rest / vpr);
  s->tv = (int)(rest % vpr);
  return (unsigned)grid;
}
}  // namespace mao
