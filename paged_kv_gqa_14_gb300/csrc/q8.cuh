// The 8-bit cache's value formats on the device: int8 (largest magnitude 127) and fp8 e4m3
// (largest 448), each with one power-of-two scale for a block of tokens and a kv head.
//
// A scale is a power of two, so a held value times its scale is a bf16 value exactly (int8 has
// seven significant bits, e4m3 four), and the smallest one that fits a block's largest
// magnitude does not depend on the order in which its tokens came.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace pkv {

// Biased fp32 exponent of the largest scale: its largest held value is finite in bf16.
template <int FMT>
__host__ __device__ constexpr int q8_max_exp() {
  return FMT == PKV_Q8_INT8 ? 254 - 6 : 254 - 8;
}

// Biased fp32 exponent of the smallest power of two >= amax / (largest held value), at least
// kQ8MinScaleExp and at most the one whose largest held value is finite in bf16 (magnitudes above
// that are held as it).  amax = 1.f 2^x fits (1.M 2^Q) 2^e iff x - Q < e, or x - Q = e and f <= M:
// adding (all ones - M) to the fraction bits carries into the exponent exactly when f > M.
template <int FMT>
__device__ __forceinline__ int q8_scale_exp(float amax) {
  constexpr unsigned M = FMT == PKV_Q8_INT8 ? 0x7E0000u : 0x600000u;  // 127 = 1.984375 2^6, 448 = 1.75 2^8
  constexpr int Q = FMT == PKV_Q8_INT8 ? 6 : 8;
  const int e = static_cast<int>((__float_as_uint(amax) + (0x7FFFFFu - M)) >> 23) - Q;
  return min(max(e, kQ8MinScaleExp), q8_max_exp<FMT>());
}

// 2^(e - 127) and its inverse for a biased exponent e in [1, 253].
__device__ __forceinline__ float q8_exp2(int e) { return __int_as_float(e << 23); }
__device__ __forceinline__ float q8_inv_exp2(int e) { return __int_as_float((254 - e) << 23); }

// Two values (already divided by the scale) as the format holds them, x0 in the low byte;
// rounding to nearest even, infinities to the largest value, NaN to 0 (int8) or NaN (e4m3).
template <int FMT>
__device__ __forceinline__ uint32_t q8_pack2(float x0, float x1) {
  if constexpr (FMT == PKV_Q8_INT8) {
    const int a = min(max(__float2int_rn(x0), -127), 127), b = min(max(__float2int_rn(x1), -127), 127);
    return (static_cast<uint32_t>(a) & 0xffu) | ((static_cast<uint32_t>(b) & 0xffu) << 8);
  } else {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
    return r;
  }
}

// The same of x0 inv and x1 inv, finite and within the format's largest: adding 1.5 2^23 rounds an int8 value to
// the nearest integer, ties to even, in the low bits of the sum.
template <int FMT>
__device__ __forceinline__ uint32_t q8_pack2_plain(float x0, float x1, float inv) {
  if constexpr (FMT == PKV_Q8_INT8) {
    const float a = fmaf(x0, inv, 12582912.f), b = fmaf(x1, inv, 12582912.f);
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040);
  } else {
    return q8_pack2<FMT>(x0 * inv, x1 * inv);
  }
}

// Four held values (bytes of w, lowest first) as f16 pairs, exactly.  int8: with the sign bit
// flipped a byte u is value + 128, and 0x6400 | u is the f16 number 1024 + u.
template <int FMT>
__device__ __forceinline__ void q8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == PKV_Q8_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0xE480), __ushort_as_half(0xE480));  // -1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 x = __hadd2(*reinterpret_cast<__half2*>(&a), off), y = __hadd2(*reinterpret_cast<__half2*>(&b), off);
    lo = *reinterpret_cast<uint32_t*>(&x);
    hi = *reinterpret_cast<uint32_t*>(&y);
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// The same, times a power of two s = 2^n (both halves of s2), n <= 5; n1152 holds -1152 s.  Exact
// while no result falls below f16's smallest step (n >= -24 for int8, n >= -15 for e4m3).
template <int FMT>
__device__ __forceinline__ void q8_to_f16_scaled(uint32_t w, uint32_t s2, uint32_t n1152, uint32_t& lo, uint32_t& hi) {
  const __half2 s = *reinterpret_cast<const __half2*>(&s2);
  __half2 x, y;
  if constexpr (FMT == PKV_Q8_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = *reinterpret_cast<const __half2*>(&n1152);
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    x = __hfma2(*reinterpret_cast<__half2*>(&a), s, off);  // (1024 + u) s - 1152 s, one exact rounding
    y = __hfma2(*reinterpret_cast<__half2*>(&b), s, off);
  } else {
    uint32_t a, b;
    q8_to_f16<FMT>(w, a, b);
    x = __hmul2(*reinterpret_cast<__half2*>(&a), s);
    y = __hmul2(*reinterpret_cast<__half2*>(&b), s);
  }
  lo = *reinterpret_cast<uint32_t*>(&x);
  hi = *reinterpret_cast<uint32_t*>(&y);
}

// 2^n and -1152 2^n as f16 pairs, n <= 5 (zero below f16's smallest step, n < -24).
__device__ __forceinline__ void q8_f16_pow2(int n, uint32_t& s2, uint32_t& n1152) {
  const uint32_t one = n >= -14 ? static_cast<uint32_t>(n + 15) << 10 : n >= -24 ? 1u << (n + 24) : 0u;
  const uint32_t off = n >= -24 ? (0xE480u + (static_cast<uint32_t>(n) << 10)) & 0xffffu : 0u;
  s2 = one | (one << 16);
  n1152 = off | (off << 16);
}

// The top bit of each of the four bytes of w that is an e4m3 NaN (all seven bits below its sign set).
__device__ __forceinline__ uint32_t e4m3_nan_bits(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// byte offset of 16-byte chunk c of token row r in a run of rows of D bytes under the TMA's swizzle:
// 128-byte rows xored within 8-row atoms, 64-byte rows xored with address bits 7-8
template <int D>
__device__ __forceinline__ uint32_t chunk8_off(int r, int c) {
  return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
// 16 bytes through L2 alone.
__device__ __forceinline__ void cp_async_l2(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival of this thread on `bar` once its cp.async so far have completed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// V and K enter their products as f16, held 2^(e - ref): a scale's distance from the reference is
// kept in [kQ8RefLow, kQ8RefHigh], where that is exact (1152 2^5 and 448 2^5 are f16 numbers).
constexpr int kQ8RefLow = -12, kQ8RefHigh = 5;
// A reference comes down to 2^-80 of the highest it has been under the same sums, however many moves that takes: in
// units of the highest they are below 2^48 (weights to 2^15.3, values below 448 2^5, 2^18 keys), so in units of the
// lowest below 2^128.  A block further down is rounded to the reference's units, or adds nothing.
constexpr int kQ8MaxDown = 80;
// Softmax weights are 2^(s - m + kQ8Lift) with s <= m + kQ8Slack: at most 2^15 (2^15.3 with the rounding of m in the
// prefill), f16 numbers.
constexpr float kQ8Lift = 7.f, kQ8Slack = 8.f;

// Four held values as fp32.
template <int FMT>
__device__ __forceinline__ void q8_to_f32(uint32_t w, float (&x)[4]) {
  if constexpr (FMT == PKV_Q8_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  } else {
    uint32_t lo, hi;
    q8_to_f16<FMT>(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
  }
}

}  // namespace pkv
