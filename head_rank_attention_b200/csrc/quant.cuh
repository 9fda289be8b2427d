// quant.cuh -- the 8-bit formats of the cached latent: nearest codes and their values.
//
// A block of tokens and 128 columns (one latent head) shares one fp32 scale s, and a code c
// stands for c * s.  Codes are the nearest ones to the exact quotient x / s, ties to even:
// int8 in [-127, 127], or e4m3 (3 mantissa bits, up to 448).  An fp32 quotient can round
// onto a tie that the exact one only comes near; quotients that do are decided by
// their exact side of it.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "paged_cache.h"
#include "sm100.cuh"

namespace hra {

template <CacheFormat F>
struct CodeTraits;
template <>
struct CodeTraits<kCacheInt8> {
  static constexpr float kTop = 127.f;
  // a tie k + 1/2 below 127.5 has at most 8 significant bits: 16 of fp32's 23 are zero
  static constexpr uint32_t kTieMask = 0xFFFFu;
};
template <>
struct CodeTraits<kCacheE4m3> {
  static constexpr float kTop = 448.f;
  // half way between neighbours of 4 significant bits: 5 bits, 19 of 23 are zero
  static constexpr uint32_t kTieMask = 0x7FFFFu;
};

// s of a block whose largest magnitude is amax: fl32(amax / top).  amax travels as the bits
// of |x| (their order is that of the values, with Inf and NaN above all numbers), so that a
// value that is no number shows in its block's scale.
template <CacheFormat F>
__device__ __forceinline__ float block_scale(uint32_t amax_bits) {
  return __fdiv_rn(__uint_as_float(amax_bits), CodeTraits<F>::kTop);
}

// A quotient of two numbers in fp64, moved to fp32 on its side of every tie.
template <CacheFormat F>
__device__ __forceinline__ float quotient_from_f64(double d) {
  float y = static_cast<float>(d);
  if ((__float_as_uint(y) & CodeTraits<F>::kTieMask) == 0 && static_cast<double>(y) != d && y != 0.f) {
    const bool up = (d > static_cast<double>(y)) == (y > 0.f);  // away from zero
    y = __uint_as_float(__float_as_uint(y) + (up ? 1u : ~0u));
  }
  return y;
}

// The code nearest to y, as its byte.
template <CacheFormat F>
__device__ __forceinline__ uint32_t to_code(float y) {
  if constexpr (F == kCacheInt8) {
    const int q = __float2int_rn(y);  // NaN gives 0
    return static_cast<uint32_t>(min(max(q, -127), 127)) & 0xFFu;
  } else {
    return __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
  }
}

template <CacheFormat F>
__device__ __forceinline__ float code_value(uint32_t byte) {
  if constexpr (F == kCacheInt8) {
    return static_cast<float>(static_cast<int>(static_cast<int8_t>(byte)));
  } else {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte), __NV_E4M3)));
  }
}

// A code under the block's old scale brought to its new one (the product of a code and an
// fp32 number is exact in fp64).
template <CacheFormat F>
__device__ __forceinline__ uint32_t rescale_code(uint32_t byte, float s_old, float s_new) {
  const double d = static_cast<double>(code_value<F>(byte)) * static_cast<double>(s_old) / static_cast<double>(s_new);
  return to_code<F>(quotient_from_f64<F>(d));
}

// Four values to their codes (lowest byte first), by quotients in fp64; s = 0 gives zeros.
template <CacheFormat F>
__device__ __forceinline__ uint32_t quantize4_exact(float4 x, float s) {
  uint32_t w = 0;
#pragma unroll 1
  for (int u = 0; u < 4; ++u) {
    const double d = static_cast<double>(u == 0 ? x.x : u == 1 ? x.y : u == 2 ? x.z : x.w) / static_cast<double>(s);
    w |= (s == 0.f ? 0u : to_code<F>(quotient_from_f64<F>(d))) << (8 * u);
  }
  return w;
}

// The same with fp32 arithmetic, for scales in [2^-90, 2^100] (quantize_fast_scale).
//
// kAnyScale: y = x * fl(1 / s) is within 1.5 units in the last place of Q = x / s; one correction by the
// residual, q = fl(y + fl(x - y s) * fl(1 / s)), rounds Q + d with |d| below 2^-21 units.  So q is within a
// unit of Q, and if q is no tie it lies on Q's side of every tie (a tie T is an fp32 number: Q < T < q
// would be more than a unit apart).  Where q is a tie (all of the tie's bits zero) the new residual
// x - q s, at most 0.6 units of q times s and so exact in an FMA, says by its sign on which side Q lies.
// Nothing here needs q to be the correctly rounded quotient.  In the range of scales above no residual
// of a quotient that matters (2^-10 and up) falls under fp32's smallest number.
//
// A scale that is fl32(amax / top) of a bf16 amax needs less.  With 8-bit significands X of x and A of
// amax, top x / amax is top X / A times a power of two, which is a tie or at least 2^-16 of itself
// away from every tie (int8; 2^-13 for e4m3), and x / s differs from it by the same factor 1 + d,
// |d| <= 2^-24, for the whole block.  If s is above amax / top every such tie is to be taken as
// just below, if under it as just above:
// kOwnScale: 1 / s is moved by 2^-20 to that side, and one multiplication does.
// kExactScale: s = amax / top exactly, ties are ties: the corrected quotient, which meets them.
// On sm_100 the difference is 6 instead of 20 instructions for four values, and ties are common: an
// x of amax / 2 is one (63.5).
enum QuantMode : int { kAnyScale, kExactScale, kOwnScale };
__device__ __forceinline__ bool quantize_fast_scale(float s) { return s >= 0x1p-90f && s <= 0x1p100f; }
// The mode of a run whose largest magnitude is amax, under the block's scale s, and the factor for it.
template <CacheFormat F>
__device__ __forceinline__ QuantMode quantize_mode(float amax, float s, float* r) {
  *r = 1.f / s;
  if (s != __fdiv_rn(amax, CodeTraits<F>::kTop)) return kAnyScale;
  const float over = fmaf(s, CodeTraits<F>::kTop, -amax);  // exact: a multiple of s's last bit
  if (over == 0.f) return kExactScale;
  *r *= over > 0.f ? 1.f - 0x1p-20f : 1.f + 0x1p-20f;
  return kOwnScale;
}

template <CacheFormat F, QuantMode MODE>
__device__ __forceinline__ uint32_t quantize4_fast(float4 x, float s, float r) {
  const float2 r2 = make_float2(r, r), ns2 = make_float2(-s, -s);
  const float2 xv[2] = {make_float2(x.x, x.y), make_float2(x.z, x.w)};
  float2 y[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    y[u] = mul2(xv[u], r2);
    if constexpr (MODE != kOwnScale) y[u] = fma2(fma2(y[u], ns2, xv[u]), r2, y[u]);
    if constexpr (MODE == kAnyScale) {
      auto decide = [&](float v, float q) {
        const float e = fmaf(-q, s, v);
        const bool tie = (__float_as_uint(q) & CodeTraits<F>::kTieMask) == 0 && e != 0.f && q != 0.f;
        return tie ? __uint_as_float(__float_as_uint(q) + ((e > 0.f) == (q > 0.f) ? 1u : ~0u)) : q;
      };
      y[u] = make_float2(decide(xv[u].x, y[u].x), decide(xv[u].y, y[u].y));
    }
  }
  if constexpr (F == kCacheInt8) {
    // y + 1.5 * 2^23 ends in the nearest integer, two's complement; |x| <= 127 s, and what y is off
    // by stays under a half
    const float2 big = make_float2(12582912.f, 12582912.f);
    const float2 a = add2(y[0], big), b = add2(y[1], big);
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
  } else {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[0].y), "f"(y[0].x));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[1].y), "f"(y[1].x));
    return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
  }
}

// Eight bf16 (four words) to eight codes.
__device__ __forceinline__ float4 bf16_to_f32x4(uint32_t lo, uint32_t hi) {
  return make_float4(__uint_as_float(lo << 16), __uint_as_float(lo & 0xFFFF0000u), __uint_as_float(hi << 16),
                     __uint_as_float(hi & 0xFFFF0000u));
}
template <CacheFormat F, QuantMode MODE>
__device__ __forceinline__ uint2 quantize8_fast(uint4 v, float s, float r) {
  return make_uint2(quantize4_fast<F, MODE>(bf16_to_f32x4(v.x, v.y), s, r),
                    quantize4_fast<F, MODE>(bf16_to_f32x4(v.z, v.w), s, r));
}
template <CacheFormat F>
__device__ __forceinline__ uint2 quantize8_exact(uint4 v, float s) {
  uint32_t w[2];
#pragma unroll 1
  for (int k = 0; k < 2; ++k) w[k] = quantize4_exact<F>(k == 0 ? bf16_to_f32x4(v.x, v.y) : bf16_to_f32x4(v.z, v.w), s);
  return make_uint2(w[0], w[1]);
}

// What four codes stand for under s, each fl32(code * s) rounded to bf16.
template <CacheFormat F>
__device__ __forceinline__ uint2 dequantize4(uint32_t w, float s) {
  float2 v[2];
  if constexpr (F == kCacheInt8) {
    // a byte under the exponent of 2^23: 2^23 + (code + 128)
    const uint32_t t = w ^ 0x80808080u;
    const float2 bias = make_float2(-8388736.f, -8388736.f);
    v[0] = add2(make_float2(__uint_as_float(__byte_perm(t, 0x4B000000u, 0x7440)), __uint_as_float(__byte_perm(t, 0x4B000000u, 0x7441))), bias);
    v[1] = add2(make_float2(__uint_as_float(__byte_perm(t, 0x4B000000u, 0x7442)), __uint_as_float(__byte_perm(t, 0x4B000000u, 0x7443))), bias);
  } else {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    v[0] = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    v[1] = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  }
  const float2 s2 = make_float2(s, s);
  v[0] = mul2(v[0], s2);
  v[1] = mul2(v[1], s2);
  return make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
}
template <CacheFormat F>
__device__ __forceinline__ uint4 dequantize8(uint2 c, float s) {
  const uint2 a = dequantize4<F>(c.x, s), b = dequantize4<F>(c.y, s);
  return make_uint4(a.x, a.y, b.x, b.y);
}

}  // namespace hra
