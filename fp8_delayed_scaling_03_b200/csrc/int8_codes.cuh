// int8_codes.cuh -- 8-bit integer codes of a row from its largest magnitude:
// the chunk loads, maxima and casts of the row quantize and of the product
// that quantizes its few input rows itself.
//
//   amax = max_c |x[c]|,  scale = amax / 127,
//   q[c] = the integer nearest to 127 x[c] / amax (the exact quotient; ties to even)
//
// A row of zeros gets scale 1 and codes 0.  A row that holds a NaN or an
// infinity gets scale NaN and codes 0, so that every product with it is NaN.
// The maximum is taken over the absolute values' bit patterns, which order
// like the values and put infinities and NaN on top.
//
// The cast multiplies by 127 / amax in fp32: two roundings, at most 1.6e-5 off
// for |t| <= 127.  Only a value that close to the border of two codes can come
// out wrong, so for those (one in some 25,000) 254 |x| is compared with
// (2 k + 1) amax, which 64 bits hold exactly.  Codes therefore depend on the
// values alone, not on how the quotient is computed.
#pragma once

#include <type_traits>

#include "device.cuh"

namespace fp8lin {
namespace int8 {

constexpr int kChunk = 16;     // elements per 16-byte store of codes
constexpr float kBorder = 0.5f - 2e-5f;
constexpr float kTinyAmax = 1e-36f;   // 127 / kTinyAmax is below the largest float
constexpr float kUp = 1.2676506002282294e30f;  // 2^100

template <typename T>
struct Chunk {
  uint4 w[sizeof(T)];          // 16 elements: sizeof(T) x 16 bytes
};

template <typename T>
__device__ __forceinline__ float value(const Chunk<T>& c, int j) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(c.w);
  if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
  else if constexpr (std::is_same<T, __half>::value)
    return __half2float(__ushort_as_half(static_cast<unsigned short>(w[j >> 1] >> (16 * (j & 1)))));
  else return __uint_as_float((j & 1) ? (w[j >> 1] & 0xFFFF0000u) : (w[j >> 1] << 16));
}

// The chunk at column col of a row; elements past the row's end are zero.
template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int64_t col, int64_t cols, int vec_ok) {
  Chunk<T> c;
  if (vec_ok && col + kChunk <= cols) {
    const uint4* src = reinterpret_cast<const uint4*>(row + col);
    #pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) c.w[i] = __ldg(src + i);
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(c.w);
    if constexpr (sizeof(T) == 4) {
      #pragma unroll
      for (int j = 0; j < kChunk; ++j)
        w[j] = col + j < cols ? __float_as_uint(__ldg(reinterpret_cast<const float*>(row) + col + j)) : 0u;
    } else {
      #pragma unroll
      for (int j = 0; j < kChunk; j += 2) {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(row) + col + j;
        w[j >> 1] = (col + j < cols ? static_cast<uint32_t>(__ldg(h)) : 0u) |
                    (col + j + 1 < cols ? static_cast<uint32_t>(__ldg(h + 1)) << 16 : 0u);
      }
    }
  }
  return c;
}

template <typename T>
__device__ __forceinline__ uint32_t chunk_max(const Chunk<T>& c, uint32_t m) {
  #pragma unroll
  for (int j = 0; j < kChunk; ++j) m = max(m, __float_as_uint(value<T>(c, j)) & 0x7FFFFFFFu);
  return m;
}

// 16 codes.  kTiny: amax is so small that 127 / amax overflows; values and amax
// are then taken times 2^100, which is exact.
template <typename T, bool kTiny>
__device__ __forceinline__ uint4 cast_chunk(const Chunk<T>& c, float amax) {
  // t + 1.5 * 2^23 rounds t to the nearest integer (ties to even) and holds it
  // in its low bits, two's complement
  constexpr float kMagic = 12582912.0f;
  const float top = kTiny ? amax * kUp : amax;
  const float inv = __fdiv_rn(127.0f, top);
  auto scaled = [&](int j) { return kTiny ? value<T>(c, j) * kUp : value<T>(c, j); };
  uint32_t q[kChunk];
  bool near = false;
  #pragma unroll
  for (int j = 0; j < kChunk; ++j) {
    const float t = __fmul_rn(scaled(j), inv);
    const float m = __fadd_rn(t, kMagic);
    q[j] = __float_as_uint(m);
    near = near || fabsf(__fsub_rn(t, __fsub_rn(m, kMagic))) > kBorder;
  }
  if (near) {
    #pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const float v = scaled(j), t = __fmul_rn(v, inv);
      if (fabsf(t - rintf(t)) > kBorder) {
        // |t| is within 1.6e-5 of k + 0.5: which side 127 |v| / top lies on,
        // from two products that 64 bits hold exactly
        const int k = static_cast<int>(fabsf(t));
        const double lhs = 254.0 * static_cast<double>(fabsf(v)), rhs = static_cast<double>(2 * k + 1) * static_cast<double>(top);
        const int a = lhs > rhs || (lhs == rhs && (k & 1)) ? k + 1 : k;
        q[j] = static_cast<uint32_t>(v < 0.0f ? -a : a);
      }
    }
  }
  uint32_t w[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __byte_perm(__byte_perm(q[4 * i], q[4 * i + 1], 0x0040), __byte_perm(q[4 * i + 2], q[4 * i + 3], 0x0040), 0x5410);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The codes of a chunk of a row whose largest magnitude has the given bits.
template <typename T>
__device__ __forceinline__ uint4 codes(const Chunk<T>& c, uint32_t bits) {
  if (bits == 0u || bits >= 0x7F800000u) return make_uint4(0u, 0u, 0u, 0u);
  const float amax = __uint_as_float(bits);
  return amax < kTinyAmax ? cast_chunk<T, true>(c, amax) : cast_chunk<T, false>(c, amax);
}

// The scale of a row whose largest magnitude has the given bits.
__device__ __forceinline__ float row_scale(uint32_t bits) {
  if (bits >= 0x7F800000u) return __uint_as_float(0x7FFFFFFFu);
  return bits ? __fdiv_rn(__uint_as_float(bits), 127.0f) : 1.0f;
}

}  // namespace int8
}  // namespace fp8lin
