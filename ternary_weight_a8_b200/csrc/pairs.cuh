// Activations in 16-byte chunks: unpacking, sums, maxima and 8-bit codes, in
// the packed two-wide fp32 instructions of sm_100a.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace bl {

// 16 bytes of activations: 8 bf16 or 4 fp32, handled as pairs of fp32 in the
// packed two-wide fp32 instructions (each half rounds as the scalar one does).
template <typename T>
constexpr int kPer = 16 / static_cast<int>(sizeof(T));
template <typename T>
constexpr int kPairs = kPer<T> / 2;

typedef unsigned long long f32x2;

__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void split2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

__device__ __forceinline__ f32x2 pair_of_bf16(uint32_t w) {  // exact
  return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t bf16_of_pair(f32x2 v) {
  float lo, hi;
  split2(v, lo, hi);
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

template <typename T>
__device__ __forceinline__ void to_pairs(const uint4& w, f32x2 (&p)[kPairs<T>]) {
  if constexpr (sizeof(T) == 2) {
    p[0] = pair_of_bf16(w.x);
    p[1] = pair_of_bf16(w.y);
    p[2] = pair_of_bf16(w.z);
    p[3] = pair_of_bf16(w.w);
  } else {
    p[0] = pack2(__uint_as_float(w.x), __uint_as_float(w.y));
    p[1] = pack2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
}

// The pairs rounded to T.
template <typename T>
__device__ __forceinline__ uint4 from_pairs(const f32x2 (&p)[kPairs<T>]) {
  if constexpr (sizeof(T) == 2) {
    return make_uint4(bf16_of_pair(p[0]), bf16_of_pair(p[1]), bf16_of_pair(p[2]), bf16_of_pair(p[3]));
  } else {
    float f[4];
    split2(p[0], f[0], f[1]);
    split2(p[1], f[2], f[3]);
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
}

// a + b in T.  For bf16 one rounding of the exact sum equals fp32's sum
// rounded once more: a sum that fp32 cannot hold has its smaller term below
// 2^-15 of the larger, far under half a bf16 step.
template <typename T>
__device__ __forceinline__ uint4 sum16(const uint4& a, const uint4& b) {
  if constexpr (sizeof(T) == 2) {
    auto add = [](uint32_t u, uint32_t v) {
      const __nv_bfloat162 h = __hadd2_rn(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                          *reinterpret_cast<const __nv_bfloat162*>(&v));
      return *reinterpret_cast<const uint32_t*>(&h);
    };
    return make_uint4(add(a.x, b.x), add(a.y, b.y), add(a.z, b.z), add(a.w, b.w));
  } else {
    f32x2 p[2], q[2];
    to_pairs<float>(a, p);
    to_pairs<float>(b, q);
    p[0] = add2(p[0], q[0]);
    p[1] = add2(p[1], q[1]);
    return from_pairs<float>(p);
  }
}

// The largest |value| of chunks, as its bits (of T; two 16-bit maxima for
// bf16): the order of the bits is that of the values, infinity above every
// number and NaN above infinity.
template <typename T>
__device__ __forceinline__ uint32_t absmax16(uint32_t m, const uint4& w) {
  if constexpr (sizeof(T) == 2) {
    m = __vmaxu2(m, __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu));
    return __vmaxu2(m, __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
  } else {
    m = max(m, max(w.x & 0x7fffffffu, w.y & 0x7fffffffu));
    return max(m, max(w.z & 0x7fffffffu, w.w & 0x7fffffffu));
  }
}
// As fp32 bits.
template <typename T>
__device__ __forceinline__ uint32_t absmax_bits(uint32_t m) {
  if constexpr (sizeof(T) == 2) return max(m & 0xffffu, m >> 16) << 16;
  return m;
}

// N fp32 values (the gains of a chunk, 16-byte aligned).  Plain loads: the
// kernel before may have written them, and every token reads them again, so
// they should stay in L1 (2048 x 2560 bf16 forward 11.2 us, 13.4 from L2).
// Volatile, so that none moves over a wait.
template <int P2>
__device__ __forceinline__ void load_pairs(const float* p, f32x2 (&f)[P2]) {
#pragma unroll
  for (int i = 0; i < P2 / 2; ++i) {
    float4 q;
    asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(q.x), "=f"(q.y), "=f"(q.z), "=f"(q.w) : "l"(p + 4 * i));
    f[2 * i] = pack2(q.x, q.y);
    f[2 * i + 1] = pack2(q.z, q.w);
  }
}

// Codes of a chunk of finite values, stored together; returns their sum.
// |v * s| <= 127 (1 + 2^-23), so no code needs clamping, and adding 1.5 * 2^23
// to the rounded product leaves rint of it (ties to even) in the sum's low bits.
// The sums are scalar: a packed sum of a packed product came out fused
// (-2.125 * 29.882353, -63.5 once rounded, gave -63), .rn on both or not.
template <typename T>
__device__ __forceinline__ int store_codes(const uint4& v, f32x2 s2, int8_t* dst) {
  constexpr float kMagic = 12582912.0f;
  f32x2 p[kPairs<T>];
  to_pairs<T>(v, p);
  uint32_t w[kPairs<T> / 2];
#pragma unroll
  for (int b = 0; b < kPairs<T> / 2; ++b) {
    float f[4];
    split2(mul2(p[2 * b], s2), f[0], f[1]);
    split2(mul2(p[2 * b + 1], s2), f[2], f[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __fadd_rn(f[e], kMagic);
    const uint32_t lo = __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x0040);
    w[b] = __byte_perm(lo, hi, 0x5410);
  }
  int sum = 0;
  if constexpr (sizeof(T) == 2) {
    sum = __dp4a(static_cast<int>(w[1]), 0x01010101, __dp4a(static_cast<int>(w[0]), 0x01010101, 0));
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    sum = __dp4a(static_cast<int>(w[0]), 0x01010101, 0);
    *reinterpret_cast<uint32_t*>(dst) = w[0];
  }
  return sum;
}

// The largest |value| of a chunk that is no NaN.
template <typename T>
__device__ __forceinline__ float absmax_any(const uint4& v) {
  f32x2 p[kPairs<T>];
  to_pairs<T>(v, p);
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < kPairs<T>; ++e) {
    float lo, hi;
    split2(p[e], lo, hi);
    m = fmaxf(m, fmaxf(fabsf(lo), fabsf(hi)));
  }
  return m;
}

// Codes for a token with infinities or NaN: NaN products (NaN * s, and
// infinity * 0, since an infinity makes s zero) give code 0.
template <typename T>
__device__ __forceinline__ int store_codes_any(const uint4& v, float s, int8_t* dst) {
  f32x2 p[kPairs<T>];
  to_pairs<T>(v, p);
  int sum = 0;
#pragma unroll
  for (int b = 0; b < kPairs<T>; ++b) {
    float f[2];
    split2(p[b], f[0], f[1]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int q = min(max(__float2int_rn(__fmul_rn(f[e], s)), -128), 127);
      dst[2 * b + e] = static_cast<int8_t>(q);
      sum += q;
    }
  }
  return sum;
}

}  // namespace bl
