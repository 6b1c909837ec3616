// Device-side arithmetic of the trained-layer operators: element types, activations
// and their derivatives, and the 8-bit checkpoint format (mao_ckpt8).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace mao {

// ------------------------------------------------------------------ pairs
// Two fp32 values in a register pair: one fma / add / mul instruction for both (sm_100a),
// which halves the issue slots of the passes below; they were bound by them, not by HBM
// (layer norm 16384 x 4096 with checkpoint: 239 instructions per 8 elements, 70 % of the issue
// slots busy at 3.9 TB/s, before pairs and the packed checkpoint arithmetic).
using f2 = float2;
__device__ __forceinline__ unsigned long long bits2(f2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ f2 from2(unsigned long long r) {
  f2 a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
  return a;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return from2(r);
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return from2(r);
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return from2(r);
}
__device__ __forceinline__ f2 dup2(float a) { return make_float2(a, a); }

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
  static __device__ __forceinline__ f2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  // two fp32 values that bf16 holds exactly: their upper halves
  static __device__ __forceinline__ uint32_t pack_exact(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  }
};
template <>
struct Elem<__half> {
  static constexpr int kDtype = MAO_F16;
  static __device__ __forceinline__ f2 unpack(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  static __device__ __forceinline__ uint32_t pack_exact(float a, float b) { return pack(a, b); }
};

// Bits of |x|: compares like |x| for finite values, with infinity and then NaN above.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// max(|a|, |b|, |c|); a NaN in any of them gives a NaN
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_s16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.s16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t min_s16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.s16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// 8 consecutive elements as they are stored: 16 bytes of a 16-bit type, 32 of fp32.
// block_max(): largest magnitude over the 4 neighbouring lanes that hold a block of 32, as
// fp32 bits (the whole warp calls it).  16-bit types compare as packed integers.
template <class T>
struct Vec8 {
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load_keep(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = w; }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(f2 (&v)[4]) const {
    v[0] = Elem<T>::unpack(w.x), v[1] = Elem<T>::unpack(w.y), v[2] = Elem<T>::unpack(w.z), v[3] = Elem<T>::unpack(w.w);
  }
  __device__ __forceinline__ void set(const f2 (&v)[4]) {
    w = make_uint4(Elem<T>::pack(v[0].x, v[0].y), Elem<T>::pack(v[1].x, v[1].y), Elem<T>::pack(v[2].x, v[2].y),
                   Elem<T>::pack(v[3].x, v[3].y));
  }
  __device__ __forceinline__ void set_exact(const f2 (&v)[4]) {
    w = make_uint4(Elem<T>::pack_exact(v[0].x, v[0].y), Elem<T>::pack_exact(v[1].x, v[1].y),
                   Elem<T>::pack_exact(v[2].x, v[2].y), Elem<T>::pack_exact(v[3].x, v[3].y));
  }
  __device__ __forceinline__ uint32_t block_max() const {
    constexpr uint32_t k = 0x7fff7fffu;
    uint32_t m = max_u16x2(max_u16x2(w.x & k, w.y & k), max_u16x2(w.z & k, w.w & k));
    m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t h = max(m & 0xffffu, m >> 16);
    return abs_bits(Elem<T>::unpack(h).x);
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
  // a whole 32-byte sector per lane where the address allows (two 16-byte stores write each
  // sector in halves: 82 against 61 us for 16384 x 4096 read back)
  __device__ __forceinline__ void store(float* p) const {
    if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(a.x), "f"(a.y), "f"(a.z),
                   "f"(a.w), "f"(b.x), "f"(b.y), "f"(b.z), "f"(b.w)
                   : "memory");
    } else {
      *reinterpret_cast<float4*>(p) = a;
      *(reinterpret_cast<float4*>(p) + 1) = b;
    }
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(f2 (&v)[4]) const {
    v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w), v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void set(const f2 (&v)[4]) {
    a = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    b = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  }
  __device__ __forceinline__ void set_exact(const f2 (&v)[4]) { set(v); }
  __device__ __forceinline__ uint32_t block_max() const {
    float m = max_abs3(a.x, a.y, a.z);
    m = max_abs3(m, a.w, b.x);
    m = max_abs3(m, b.y, b.z);
    m = max_abs3(m, b.w, 0.0f);
    uint32_t u = abs_bits(m);
    u = max(u, __shfl_xor_sync(0xffffffffu, u, 1));
    return max(u, __shfl_xor_sync(0xffffffffu, u, 2));
  }
};

// 8 consecutive values of a parameter vector (weight or bias): fp32 or T
template <class T>
__device__ __forceinline__ void load_param8(const void* p, bool f32, long long i, f2 (&v)[4]) {
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

// ------------------------------------------------------------------ dependent launches
// A kernel launched as a programmatic dependent (launch_dependent in layer_host.h) may start
// while the kernel before it in the stream still runs: it waits here before it touches global
// memory, and with that for everything before, since every kernel of a chain waits.  The
// kernel before says when the dependents may be scheduled.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------------ asynchronous loads
// A thread's own ring in shared memory: cp.async of 16 (or 8) bytes that only the issuing
// thread reads back, so no barrier orders them, only its own wait.  With ok false nothing is
// read and zeros are written.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok = true) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool ok = true) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}
__device__ __forceinline__ void sts_zero8(uint32_t dst) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %1};" ::"r"(dst), "r"(0) : "memory");
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
  static __device__ __forceinline__ void fetch(uint32_t dst, uint32_t stride, const T* src) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) cp_async16(dst + i * stride, src + i * (16 / sizeof(T)));
  }
  static __device__ __forceinline__ void zero(uint32_t dst, uint32_t stride) {
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) sts_zero8(dst + i * stride), sts_zero8(dst + i * stride + 8);
  }
  static __device__ __forceinline__ Vec8<T> get(uint32_t src, uint32_t stride) {
    Vec8<T> t;
    uint4 w[kBytes / 16];
#pragma unroll
    for (int i = 0; i < kBytes / 16; ++i) w[i] = lds16(src + i * stride);
    memcpy(&t, w, sizeof(t));
    return t;
  }
};

// ------------------------------------------------------------------ activations
// Two values at a time.  sigmoid(z) = 1 / (1 + exp(-z)); exp(-z) = inf gives 0, as it should.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;
// 1 / (1 + 2^x), both lanes
__device__ __forceinline__ f2 inv_1p_exp2(f2 x) {
  const f2 d = add2(make_float2(exp2_fast(x.x), exp2_fast(x.y)), dup2(1.0f));
  return make_float2(rcp_fast(d.x), rcp_fast(d.y));
}

constexpr float kGeluA = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// Phi(z) and phi(z), the normal distribution and its density, from one exponential:
//   Phi(-a) = erfc(a / sqrt 2) / 2 = exp(-a^2 / 2) t Q(t) / 2,   t = 1 / (1 + 0.38 a / sqrt 2),
// with Q the degree-6 polynomial whose largest relative error over 0 <= a / sqrt 2 <= 9.4 is
// least (a Lawson-weighted least-squares fit of exp(x^2) erfc(x) / t): 1.0e-6, relative, in
// the tail as well, against a half step of 4.9e-4 in fp16.  About 12 instructions a value in
// pairs where erff and expf take about 60: with those the backward pass was bound by
// arithmetic (217 us for 8192 x 14336, 2.7 TB/s).
__device__ __forceinline__ void normal_cdf(f2 z, f2& cdf, f2& density) {
  const f2 a = make_float2(fabsf(z.x), fabsf(z.y));
  const f2 den = fma2(a, dup2(0.38f * 0.7071067811865476f), dup2(1.0f));
  const f2 t = make_float2(rcp_fast(den.x), rcp_fast(den.y));
  const f2 x = mul2(mul2(z, z), dup2(-0.5f * kLog2e));
  const f2 g = make_float2(exp2_fast(x.x), exp2_fast(x.y));
  // the coefficients of Q / 2
  f2 q = dup2(0.5f * -0.12500557059902176f);
  q = fma2(q, t, dup2(0.5f * 0.3344489817608761f));
  q = fma2(q, t, dup2(0.5f * -0.06744702421290848f));
  q = fma2(q, t, dup2(0.5f * 0.2458644792820478f));
  q = fma2(q, t, dup2(0.5f * 0.18144377612944992f));
  q = fma2(q, t, dup2(0.5f * 0.2163907947734426f));
  q = fma2(q, t, dup2(0.5f * 0.21430355427606323f));
  const f2 tail = mul2(mul2(q, t), g);
  const f2 rest = fma2(tail, dup2(-1.0f), dup2(1.0f));
  cdf = make_float2(z.x < 0.0f ? tail.x : rest.x, z.y < 0.0f ? tail.y : rest.y);
  density = mul2(g, dup2(0.3989422804014327f));
}

// 2^x's argument for gelu_tanh: (1 + tanh u) / 2 = 1 / (1 + exp(-2 u)), without the
// cancellation of 1 + tanh u at u << 0; -2 u log2(e) = z (c1 + c2 z^2)
__device__ __forceinline__ f2 gelu_tanh_arg(f2 z, f2 z2) {
  return mul2(z, fma2(z2, dup2(-2.0f * kLog2e * kGeluA * kGeluB), dup2(-2.0f * kLog2e * kGeluA)));
}
__device__ __forceinline__ f2 relu2v(f2 z) {  // a NaN stays one
  return make_float2(z.x < 0.0f ? 0.0f : z.x, z.y < 0.0f ? 0.0f : z.y);
}

// For fp32 results, each value to a few steps of itself in the tails too: no 1 + erf or 1 + tanh,
// which cancel where z << 0, and no flushed or approximate exponential.
//   sigmoid(v) = (v < 0 ? t : 1) / (1 + t),  t = exp(-|v|)
//   Phi(-a) = erfc(a / sqrt 2) / 2 = exp(-a^2 / 2) erfcx(a / sqrt 2) / 2, where z^2 is exact for the 8 bits of
//   a checkpoint's value and erfcx falls off like 1 / a, so that no rounding counts a^2 times
// Bound by these instructions: 16384 x 4096 read back to fp32 takes 61 us without an activation, 88 with
// silu, 96 with gelu_tanh, 158 with gelu (87 with 1 + erff, which is off by 4e-2 of the value at z = -5).
// A rounded reciprocal in place of the quotient took the same.
__device__ __forceinline__ float sigmoid32(float v) {
  const float t = expf(-fabsf(v));
  return (v < 0.0f ? t : 1.0f) / (1.0f + t);
}
template <int ACT>
__device__ __forceinline__ float act_value32(float z) {
  if constexpr (ACT == MAO_ACT_GELU) {
    const float a = fabsf(z);
    const float tail = 0.5f * expf(-0.5f * z * z) * erfcxf(a * 0.7071067811865476f);
    return z * (z < 0.0f ? tail : 1.0f - tail);
  } else if constexpr (ACT == MAO_ACT_GELU_TANH) {
    return z * sigmoid32(z * fmaf(z * z, 2.0f * kGeluA * kGeluB, 2.0f * kGeluA));
  } else {
    return z * sigmoid32(z);  // silu
  }
}

// EXACT: fp32 results; otherwise results that are rounded to 16 bits.
template <int ACT, bool EXACT = false>
__device__ __forceinline__ f2 act_value(f2 z) {
  if constexpr (EXACT && (ACT == MAO_ACT_GELU || ACT == MAO_ACT_GELU_TANH || ACT == MAO_ACT_SILU)) {
    return make_float2(act_value32<ACT>(z.x), act_value32<ACT>(z.y));
  } else if constexpr (ACT == MAO_ACT_RELU) {
    return relu2v(z);
  } else if constexpr (ACT == MAO_ACT_RELU2) {
    const f2 r = relu2v(z);
    return mul2(r, r);
  } else if constexpr (ACT == MAO_ACT_GELU) {
    f2 c, d;
    normal_cdf(z, c, d);
    return mul2(z, c);
  } else if constexpr (ACT == MAO_ACT_GELU_TANH) {
    return mul2(z, inv_1p_exp2(gelu_tanh_arg(z, mul2(z, z))));
  } else if constexpr (ACT == MAO_ACT_SILU) {
    return mul2(z, inv_1p_exp2(mul2(z, dup2(-kLog2e))));
  } else {
    return z;
  }
}

template <int ACT>
__device__ __forceinline__ f2 act_slope(f2 z) {
  if constexpr (ACT == MAO_ACT_RELU) {
    return make_float2(z.x > 0.0f ? 1.0f : (z.x <= 0.0f ? 0.0f : z.x), z.y > 0.0f ? 1.0f : (z.y <= 0.0f ? 0.0f : z.y));
  } else if constexpr (ACT == MAO_ACT_RELU2) {
    const f2 r = relu2v(z);
    return add2(r, r);
  } else if constexpr (ACT == MAO_ACT_GELU) {
    f2 c, d;
    normal_cdf(z, c, d);
    return fma2(z, d, c);  // Phi(z) + z phi(z)
  } else if constexpr (ACT == MAO_ACT_GELU_TANH) {
    // d/dz z s(v(z)) with v = 2 sqrt(2/pi) (z + b z^3): s + z s (1 - s) v'
    const f2 z2 = mul2(z, z);
    const f2 s = inv_1p_exp2(gelu_tanh_arg(z, z2));
    // z^2 held finite: where it is not, z s (1 - s) is 0, and 0 times an infinite v' would be NaN
    const f2 zz = make_float2(fminf(z2.x, 1e30f), fminf(z2.y, 1e30f));
    const f2 dv = fma2(zz, dup2(6.0f * kGeluA * kGeluB), dup2(2.0f * kGeluA));
    const f2 sp = fma2(mul2(s, s), dup2(-1.0f), s);
    return fma2(mul2(z, sp), dv, s);
  } else if constexpr (ACT == MAO_ACT_SILU) {
    const f2 s = inv_1p_exp2(mul2(z, dup2(-kLog2e)));
    return fma2(z, fma2(mul2(s, s), dup2(-1.0f), s), s);
  } else {
    return dup2(1.0f);
  }
}

// ------------------------------------------------------------------ 8-bit checkpoints
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
// 2^(e - 127); 0 for e = 0 (and infinity for a marked block, which ckpt_unpack4 turns into NaN).
__device__ __forceinline__ float ckpt_scale(uint32_t e) { return __uint_as_float(e << 23); }

// Four bytes of x / step.  x / step is exact; adding 1.5 * 2^23 in the same fma rounds it to
// the nearest whole number, ties to even, into the low mantissa bits.  Whole numbers of
// magnitude 128 (a magnitude that rounds up past 127.5 steps) are limited as 16-bit pairs.
// `mask` is 0 for a marked block, else all ones.
__device__ __forceinline__ uint32_t ckpt_q4(f2 a, f2 b, float inv, uint32_t mask) {
  const f2 magic = dup2(12582912.0f), i2 = dup2(inv);
  const f2 ra = fma2(a, i2, magic), rb = fma2(b, i2, magic);
  uint32_t lo = __byte_perm(__float_as_uint(ra.x), __float_as_uint(ra.y), 0x5410);
  uint32_t hi = __byte_perm(__float_as_uint(rb.x), __float_as_uint(rb.y), 0x5410);
  lo = min_s16x2(max_s16x2(lo, 0xff81ff81u), 0x007f007fu);
  hi = min_s16x2(max_s16x2(hi, 0xff81ff81u), 0x007f007fu);
  return __byte_perm(lo, hi, 0x6420) & mask;
}
// Four bytes of q to values.  With its sign bit flipped a byte is u = q + 128, and 0x4700uu00
// is the float 32768 + u; (32768 + u) s - 32896 s = q s in one fma, exactly (q s has 8 bits).
// 32896 s must stay finite: from s = 2^113 on the subtraction comes first.  A marked block is
// NaN whatever its q.
__device__ __forceinline__ void ckpt_unpack4(uint32_t w, uint32_t e, f2* v) {
  const float s = ckpt_scale(e);
  const uint32_t u = w ^ 0x80808080u;
  f2 a = make_float2(__uint_as_float(__byte_perm(u, 0x47000000u, 0x7404)),
                     __uint_as_float(__byte_perm(u, 0x47000000u, 0x7414)));
  f2 b = make_float2(__uint_as_float(__byte_perm(u, 0x47000000u, 0x7424)),
                     __uint_as_float(__byte_perm(u, 0x47000000u, 0x7434)));
  if (e < 240u) {
    const f2 c = dup2(-32896.0f * s);
    v[0] = fma2(a, dup2(s), c);
    v[1] = fma2(b, dup2(s), c);
  } else {
    const f2 f = dup2(e == 255u ? __uint_as_float(0x7fffffffu) : s);
    v[0] = mul2(add2(a, dup2(-32896.0f)), f);
    v[1] = mul2(add2(b, dup2(-32896.0f)), f);
  }
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
  __device__ __forceinline__ void get(f2 (&v)[4]) const {
    ckpt_unpack4(w.x, e, v);
    ckpt_unpack4(w.y, e, v + 2);
  }
};

// Writes 8 consecutive values' share of a block whose 32 columns are held by 4
// neighbouring lanes (8 each); amax: the block's largest magnitude (Vec8::block_max).  Lanes
// behind the last column pass zeros, which become the block's padding.
// q: where this lane's 8 bytes go; e: where the block's byte goes, for the block's first lane,
// else nullptr.
__device__ __forceinline__ void ckpt_store8(int8_t* q, uint8_t* e_out, const f2 (&v)[4], uint32_t amax) {
  const uint32_t e = ckpt_exponent(amax);
  const float inv = ckpt_inverse(e);
  const uint32_t mask = e == 255u ? 0u : 0xffffffffu;
  uint2 w;
  w.x = ckpt_q4(v[0], v[1], inv, mask);
  w.y = ckpt_q4(v[2], v[3], inv, mask);
  *reinterpret_cast<uint2*>(q) = w;
  if (e_out != nullptr) *e_out = (uint8_t)e;
}

}  // namespace mao
