// quant.cuh -- the 8-bit formats of the cached latent: nearest codes and their values.
//
// A block of tokens and 128 columns (one latent head) shares one fp32 scale s, and a code c
// stands for c * s.  Codes are the nearest ones to the exact quotient x / s, ties to even:
// int8 in [-127, 127], or e4m3 (3 mantissa bits, up to 448).  An fp32 quotient can round
// onto a tie that the exact one only comes near, so code_quotient returns an fp32 number
// that lies on the exact quotient's side of every tie.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "paged_cache.h"

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

// fp32 y with x / s on its side of (or on) every tie of the format; s > 0.
template <CacheFormat F>
__device__ __forceinline__ float code_quotient(float x, float s) {
  const double d = static_cast<double>(x) / static_cast<double>(s);
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
  float y = static_cast<float>(d);
  if ((__float_as_uint(y) & CodeTraits<F>::kTieMask) == 0 && static_cast<double>(y) != d && y != 0.f) {
    const bool up = (d > static_cast<double>(y)) == (y > 0.f);
    y = __uint_as_float(__float_as_uint(y) + (up ? 1u : ~0u));
  }
  return to_code<F>(y);
}

}  // namespace hra
