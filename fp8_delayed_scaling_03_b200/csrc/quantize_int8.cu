// quantize_int8.cu -- rows to 8-bit integers, each by its own largest magnitude.
//
//   amax = max_c |x[r, c]|,  scale[r] = amax / 127,
//   q[r, c] = the integer nearest to 127 x[r, c] / amax (the exact quotient; ties to even)
//
// A row of zeros gets scale 1 and codes 0.  A row that holds a NaN or an
// infinity gets scale NaN and codes 0, so that every product with it is NaN.
//
// One pass over HBM: a row's 16-element chunks stay in registers between the
// maximum and the cast (rows longer than 2 chunks x 512 threads read the rest
// a second time, from L2).  The maximum is taken over the absolute values' bit
// patterns, which order like the values and put infinities and NaN on top.
//
// The cast multiplies by 127 / amax in fp32: two roundings, at most 1.6e-5 off
// for |t| <= 127.  Only a value that close to the border of two codes can come
// out wrong, so for those (one in some 25,000) 254 |x| is compared with
// (2 k + 1) amax, which 64 bits hold exactly.  Codes therefore depend on the
// values alone, not on how the quotient is computed.
#include <type_traits>

#include "device.cuh"
#include "internal.h"
#include "launch.h"

namespace fp8lin {
namespace {

constexpr int kChunk = 16;     // elements per 16-byte store of codes
constexpr int kHeld = 2;       // chunks a thread keeps in registers
constexpr int kMaxThreads = 512;  // 128 registers a thread
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

// blockDim.y rows a block, blockDim.x threads a row (one warp when there is
// more than one row).
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) quantize_int8_kernel(const Int8QuantizeParams p) {
  __shared__ uint32_t warp_max[32];
  pdl_wait();
  pdl_trigger();
  const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = r < p.rows;
  const T* row = static_cast<const T*>(p.in) + (live ? r : 0) * p.ld_in;
  const int64_t chunks = live ? (p.cols + kChunk - 1) / kChunk : 0;
  const int64_t tid = threadIdx.x, step = blockDim.x;
  Chunk<T> held[kHeld];
  uint32_t bits = 0;
  #pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * step < chunks) held[i] = load_chunk<T>(row, (tid + i * step) * kChunk, p.cols, p.vec_ok);
  #pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * step < chunks) bits = chunk_max<T>(held[i], bits);
  for (int64_t c = tid + kHeld * step; c < chunks; c += step)
    bits = chunk_max<T>(load_chunk<T>(row, c * kChunk, p.cols, p.vec_ok), bits);
  bits = __reduce_max_sync(0xFFFFFFFFu, bits);
  if (blockDim.y == 1) {
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = bits;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    bits = __reduce_max_sync(0xFFFFFFFFu, lane < static_cast<int>(blockDim.x >> 5) ? warp_max[lane] : 0u);
  }
  if (live && tid == 0)
    p.scale[r] = bits >= 0x7F800000u ? __uint_as_float(0x7FFFFFFFu)
                                     : (bits ? __fdiv_rn(__uint_as_float(bits), 127.0f) : 1.0f);
  int8_t* out = p.out + (live ? r : 0) * p.ld_out;
  #pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * step < chunks)
      *reinterpret_cast<uint4*>(out + (tid + i * step) * kChunk) = codes<T>(held[i], bits);
  for (int64_t c = tid + kHeld * step; c < chunks; c += step)
    *reinterpret_cast<uint4*>(out + c * kChunk) =
        codes<T>(load_chunk<T>(row, c * kChunk, p.cols, p.vec_ok), bits);
}

}  // namespace

// Threads of a row: enough that a row fits the held chunks, at most kMaxThreads; rows
// of up to 1024 elements take one warp each, eight rows a block.
cudaError_t launch_quantize_int8(int in_dtype, const Int8QuantizeParams& p, cudaStream_t s) {
  const int64_t chunks = (p.cols + kChunk - 1) / kChunk;
  const int64_t want = (chunks + kHeld - 1) / kHeld;
  const unsigned threads = static_cast<unsigned>(want >= kMaxThreads ? kMaxThreads : (want + 31) / 32 * 32);
  const dim3 block(threads, threads == 32 ? 8u : 1u);
  const dim3 grid(static_cast<unsigned>((p.rows + block.y - 1) / block.y));
  if (in_dtype == kFP32) return launch_pdl(quantize_int8_kernel<float>, grid, block, 0, s, p);
  if (in_dtype == kFP16) return launch_pdl(quantize_int8_kernel<__half>, grid, block, 0, s, p);
  return launch_pdl(quantize_int8_kernel<__nv_bfloat16>, grid, block, 0, s, p);
}

}  // namespace fp8lin
