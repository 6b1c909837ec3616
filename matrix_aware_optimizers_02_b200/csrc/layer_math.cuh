// Device-side arithmetic of the trained-layer operators: element types, activations
// and their derivatives, and the 8-bit checkpoint format (mao_ckpt8).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace mao {

// ------------------------------------------------------------------ element types
template <class T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kDtype = MAO_F32;
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kDtype = MAO_BF16;
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};
template <>
struct Elem<__half> {
  static constexpr int kDtype = MAO_F16;
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<__half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};

// 8 consecutive elements as they are stored: 16 bytes of a 16-bit type, 32 of fp32.
// A vector held in this form is half the registers of its fp32 values.
template <class T>
struct Vec8 {
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load_keep(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = Elem<T>::unpack(u[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    w = make_uint4(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]), Elem<T>::pack(v[4], v[5]),
                   Elem<T>::pack(v[6], v[7]));
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void load_keep(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *(reinterpret_cast<float4*>(p) + 1) = b;
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};

// 8 consecutive values of a parameter vector (weight or bias): fp32 or T
template <class T>
__device__ __forceinline__ void load_param8(const void* p, bool f32, long long i, float (&v)[8]) {
  if (f32) {
    Vec8<float> t;
    t.load_keep(static_cast<const float*>(p) + i);
    t.get(v);
  } else {
    Vec8<T> t;
    t.load_keep(static_cast<const T*>(p) + i);
    t.get(v);
  }
}

// ------------------------------------------------------------------ asynchronous loads
// A thread's own ring in shared memory: cp.async of 16 (or 8) bytes that only the issuing
// thread reads back, so no barrier orders them, only its own wait.  With ok false nothing is
// read and zeros are written.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the latest N groups of this thread have landed
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// One vector of 8 elements per thread in a ring slot: 16-byte pieces `stride` bytes apart
// (a block's threads side by side, so neighbouring lanes touch neighbouring banks).
template <class T>
struct Slot8 {
  static constexpr int kBytes = 8 * sizeof(T);
  static __device__ __forceinline__ void fetch(uint32_t dst, uint32_t stride, const T* src, bool ok) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) cp_async16(dst + i * stride, src + i * (16 / sizeof(T)), ok);
  }
  static __device__ __forceinline__ void get(uint32_t src, uint32_t stride, float (&v)[8]) {
    Vec8<T> t;
    uint4 w[kBytes / 16];
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) w[i] = lds16(src + i * stride);
    memcpy(&t, w, sizeof(t));
    t.get(v);
  }
};

// ------------------------------------------------------------------ activations
// sigmoid(z) = 1 / (1 + exp(-z)); exp(-z) = inf for z < -88 gives 0, as it should.
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// Phi(z) and phi(z), the normal distribution and its density, from one exponential:
//   Phi(-a) = erfc(a / sqrt 2) / 2 = exp(-a^2 / 2) t Q(t) / 2,   t = 1 / (1 + 0.38 a / sqrt 2),
// with Q the degree-6 polynomial whose largest relative error over 0 <= a / sqrt 2 <= 9.4 is
// least (a Lawson-weighted least-squares fit of exp(x^2) erfc(x) / t): 1.0e-6, relative, in
// the tail as well, against a half step of 4.9e-4 in fp16.  About 20 instructions where erff
// and expf take about 60: with erff the backward pass was bound by arithmetic (217 us for
// 8192 x 14336, 2.7 TB/s).
__device__ __forceinline__ void normal_cdf(float z, float& cdf, float& density) {
  const float a = fabsf(z);
  const float t = __fdividef(1.0f, fmaf(0.38f * 0.7071067811865476f, a, 1.0f));
  const float g = __expf(-0.5f * z * z);
  float q = -0.12500557059902176f;
  q = fmaf(q, t, 0.3344489817608761f);
  q = fmaf(q, t, -0.06744702421290848f);
  q = fmaf(q, t, 0.2458644792820478f);
  q = fmaf(q, t, 0.18144377612944992f);
  q = fmaf(q, t, 0.2163907947734426f);
  q = fmaf(q, t, 0.21430355427606323f);
  const float tail = 0.5f * q * t * g;
  cdf = z < 0.0f ? tail : 1.0f - tail;
  density = 0.3989422804014327f * g;
}

// EXACT: fp32 results (erff); otherwise results that are rounded to 16 bits.
template <int ACT, bool EXACT = false>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == MAO_ACT_RELU) {
    return z < 0.0f ? 0.0f : z;  // a NaN stays one
  } else if constexpr (ACT == MAO_ACT_RELU2) {
    const float r = z < 0.0f ? 0.0f : z;
    return r * r;
  } else if constexpr (ACT == MAO_ACT_GELU) {
    if constexpr (EXACT) {
      return 0.5f * z * (1.0f + erff(z * 0.7071067811865476f));
    } else {
      float c, d;
      normal_cdf(z, c, d);
      return z * c;
    }
  } else if constexpr (ACT == MAO_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = sigmoid(2 u), without the cancellation of 1 + tanh u at u << 0
    return z * sigmoid_f(2.0f * kGeluA * (z + kGeluB * z * z * z));
  } else if constexpr (ACT == MAO_ACT_SILU) {
    return z * sigmoid_f(z);
  } else {
    return z;
  }
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == MAO_ACT_RELU) {
    return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
  } else if constexpr (ACT == MAO_ACT_RELU2) {
    return 2.0f * (z < 0.0f ? 0.0f : z);
  } else if constexpr (ACT == MAO_ACT_GELU) {
    float c, d;
    normal_cdf(z, c, d);
    return fmaf(z, d, c);  // Phi(z) + z phi(z)
  } else if constexpr (ACT == MAO_ACT_GELU_TANH) {
    // d/dz z s(v(z)) with v = 2 sqrt(2/pi) (z + b z^3): s + z s (1 - s) v'
    const float s = sigmoid_f(2.0f * kGeluA * (z + kGeluB * z * z * z));
    return s + z * s * (1.0f - s) * (2.0f * kGeluA) * (1.0f + 3.0f * kGeluB * z * z);
  } else if constexpr (ACT == MAO_ACT_SILU) {
    const float s = sigmoid_f(z);
    return s + z * s * (1.0f - s);
  } else {
    return 1.0f;
  }
}

// ------------------------------------------------------------------ 8-bit checkpoints
// Bits of |x|: compares like |x| for finite values, with infinity and then NaN above.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The block byte for the largest magnitude's bits: floor(log2 a) + 127 is the exponent
// field, so e = max(field - 6, 1); 255 marks a block with a NaN or an infinity.
__device__ __forceinline__ uint32_t ckpt_exponent(uint32_t amax_bits) {
  const uint32_t f = amax_bits >> 23;
  return f == 255u ? 255u : (f > 7u ? f - 6u : 1u);
}
// 2^(127 - e), exact; 0 for a marked block, whose q are all 0.
__device__ __forceinline__ float ckpt_inverse(uint32_t e) {
  return e == 255u ? 0.0f : __uint_as_float((254u - e) << 23);
}
// 2^(e - 127); infinity for a marked block (0 * inf = NaN), 0 for e = 0.
__device__ __forceinline__ float ckpt_scale(uint32_t e) { return __uint_as_float(e << 23); }

// The byte of x / step.  Adding 1.5 * 2^23 leaves the whole number, rounded to nearest
// even, in the low mantissa bits.  A marked block has inv = 0: NaN * 0 and inf * 0 are NaN,
// which fminf / fmaxf turn into a limit, so it is set to 0 by the caller's mask.
__device__ __forceinline__ uint32_t ckpt_q(float x, float inv) {
  const float r = fminf(fmaxf(x * inv, -127.0f), 127.0f);
  return __float_as_uint(r + 12582912.0f) & 0xffu;
}
__device__ __forceinline__ uint32_t ckpt_q4(float a, float b, float c, float d, float inv, uint32_t mask) {
  const uint32_t lo = __byte_perm(ckpt_q(a, inv), ckpt_q(b, inv), 0x0040);
  const uint32_t hi = __byte_perm(ckpt_q(c, inv), ckpt_q(d, inv), 0x0040);
  return __byte_perm(lo, hi, 0x5410) & mask;
}
// four bytes of q to fp32: with the sign bit flipped a byte is q + 128, and 0x4B0000xx is
// the float 2^23 + xx
__device__ __forceinline__ void ckpt_unpack4(uint32_t w, float s, float* v) {
  const uint32_t u = w ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)) - 8388736.0f) * s;
}

// What a kernel needs of a checkpoint.
struct CkptView {
  int8_t* q;
  uint8_t* e;
  long long ld_q, ld_e;
};

// 8 consecutive values (columns c .. c+7 of a row, c a multiple of 8) in raw form.
struct CkptVec8 {
  uint2 w;
  uint32_t e;
  __device__ __forceinline__ void load(const CkptView& k, long long row, int c) {
    w = __ldcs(reinterpret_cast<const uint2*>(k.q + row * k.ld_q + c));
    e = k.e[row * k.ld_e + (c >> 5)];
  }
  __device__ __forceinline__ void zero() { w = make_uint2(0, 0), e = 1; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const float s = ckpt_scale(e);
    ckpt_unpack4(w.x, s, v);
    ckpt_unpack4(w.y, s, v + 4);
  }
};

// Writes 8 consecutive values' share of a block whose 32 columns are held by 4
// neighbouring lanes (8 each).  Every lane of the group calls this; lanes behind the last
// column pass zeros, which become the block's padding.
__device__ __forceinline__ void ckpt_store8(const CkptView& k, long long row, int c, const float (&v)[8],
                                            bool block_in_row) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, abs_bits(v[i]));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
  const uint32_t e = ckpt_exponent(a);
  const float inv = ckpt_inverse(e);
  const uint32_t mask = e == 255u ? 0u : 0xffffffffu;
  if (block_in_row) {
    uint2 w;
    w.x = ckpt_q4(v[0], v[1], v[2], v[3], inv, mask);
    w.y = ckpt_q4(v[4], v[5], v[6], v[7], inv, mask);
    *reinterpret_cast<uint2*>(k.q + row * k.ld_q + c) = w;
    if ((c & 31) == 0) k.e[row * k.ld_e + (c >> 5)] = (uint8_t)e;
  }
}

}  // namespace mao
