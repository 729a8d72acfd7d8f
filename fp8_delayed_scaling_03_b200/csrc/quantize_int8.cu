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
// Codes depend on the values alone, not on how the quotient is computed: see
// cast_chunk().
#include <type_traits>

#include "device.cuh"
#include "internal.h"
#include "launch.h"

namespace fp8lin {
namespace {

constexpr int kChunk = 16;     // elements per 16-byte store of codes
constexpr int kHeld = 2;       // chunks a thread keeps in registers
constexpr int kMaxThreads = 512;
constexpr float kBorder = 0.5f - 2e-5f;
constexpr float kTinyAmax = 1e-36f, kHugeAmax = 1e36f;   // between them 127 / amax and 127 amax are finite
constexpr float k2p100 = 1.2676506002282294e30f;

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
// (Plain loads: the read-only path does not promise to see what the kernel
// before wrote, and this one starts while that may still run.)
template <typename T>
__device__ __forceinline__ Chunk<T> load_chunk(const T* row, int64_t col, int64_t cols, int vec_ok) {
  Chunk<T> c;
  if (vec_ok && col + kChunk <= cols) {
    const uint4* src = reinterpret_cast<const uint4*>(row + col);
    #pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) c.w[i] = src[i];
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(c.w);
    if constexpr (sizeof(T) == 4) {
      #pragma unroll
      for (int j = 0; j < kChunk; ++j)
        w[j] = col + j < cols ? __float_as_uint(reinterpret_cast<const float*>(row)[col + j]) : 0u;
    } else {
      #pragma unroll
      for (int j = 0; j < kChunk; j += 2) {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(row) + col + j;
        w[j >> 1] = (col + j < cols ? static_cast<uint32_t>(h[0]) : 0u) |
                    (col + j + 1 < cols ? static_cast<uint32_t>(h[1]) << 16 : 0u);
      }
    }
  }
  return c;
}

// The running maximum of the absolute values' bit patterns: of 2-byte types
// two to a word.
template <typename T>
__device__ __forceinline__ uint32_t chunk_max(const Chunk<T>& c, uint32_t m) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(c.w);
  #pragma unroll
  for (int j = 0; j < 4 * static_cast<int>(sizeof(T)); ++j) {
    if constexpr (sizeof(T) == 2) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    else m = max(m, w[j] & 0x7FFFFFFFu);
  }
  return m;
}

// ... as the bit pattern of an fp32 value (infinities and NaN: that of
// infinity or above).
template <typename T>
__device__ __forceinline__ uint32_t max_bits(uint32_t m) {
  if constexpr (sizeof(T) == 4) return m;
  const uint32_t h = max(m & 0xFFFFu, m >> 16);
  if constexpr (std::is_same<T, __half>::value)
    return h >= 0x7C00u ? 0x7F800000u : __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
  else return h << 16;
}

// Two fp32 values in one register pair and the packed operations on them.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint2 bits2(uint64_t v) {
  uint2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(r.x), "=r"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// What the casts of one row share.  A row whose amax is so small that 127 /
// amax overflows is taken times 2^100, one so large that 127 amax does times
// 2^-100: exact for every value that can get another code than 0.
struct RowScale {
  float up, top, inv;          // 1, 2^100 or 2^-100; amax up; 127 / top
  bool zero;                   // all codes 0
};

__device__ __forceinline__ RowScale row_scale(uint32_t bits) {
  RowScale s;
  s.zero = bits == 0u || bits >= 0x7F800000u;
  const float amax = s.zero ? 1.0f : __uint_as_float(bits);
  s.up = amax < kTinyAmax ? k2p100 : (amax > kHugeAmax ? 1.0f / k2p100 : 1.0f);
  s.top = amax * s.up;
  s.inv = __fdiv_rn(127.0f, s.top);
  return s;
}

// The 16 codes of a chunk.  kScaled: s.up is not 1.
//
// m = the integer nearest to t = v inv, by adding and subtracting 1.5 * 2^23,
// whose sum holds it in its low bits, two's complement.  t is off by at most
// 1.6e-5, so m is wrong only next to the border of two codes:
//   2-byte inputs: 127 v and the remainder r = 127 v - m top are exact in
//     fp32, so |r| against top / 2 tells, and a tie goes to the even code.
//     Ties are common there (bf16 values and amax have 8 significant bits):
//     one in 225 to 460 (rows of 11008 to 1024 normal values), so every
//     element is corrected, without a branch (a branch an element took a third
//     longer).  The comparison adds m's lowest bit to r's pattern: above
//     top / 2, or equal to it and m odd.
//   fp32 inputs: only where t is within 2e-5 of a border, 254 |v| is compared
//     with (2 k + 1) top, which 64 bits hold exactly (one in some 25,000).
template <typename T, bool kScaled>
__device__ __forceinline__ uint4 cast_chunk(const Chunk<T>& c, const RowScale& s) {
  constexpr float kMagic = 12582912.0f;
  uint32_t q[kChunk];
  if constexpr (sizeof(T) == 2) {
    const uint64_t inv = f2(s.inv, s.inv), up = f2(s.up, s.up), magic = f2(kMagic, kMagic), minus = f2(-kMagic, -kMagic),
                   c127 = f2(127.0f, 127.0f), ntop = f2(-s.top, -s.top);
    const uint32_t half = __float_as_uint(0.5f * s.top);
    #pragma unroll
    for (int j = 0; j < kChunk; j += 2) {
      uint64_t v = f2(value<T>(c, j), value<T>(c, j + 1));
      if (kScaled) v = mul2(v, up);
      const uint64_t m = add2(mul2(v, inv), magic);
      const uint2 r = bits2(fma2(add2(m, minus), ntop, mul2(v, c127)));
      const uint2 b = bits2(m);
      auto code = [&](uint32_t mb, uint32_t rb) {
        const uint32_t a = rb + (mb & 1u);
        if (static_cast<int>(a) > static_cast<int>(half)) mb += 1u;   // r > 0
        if (a > (half | 0x80000000u)) mb -= 1u;                       // r < 0
        return mb;
      };
      q[j] = code(b.x, r.x);
      q[j + 1] = code(b.y, r.y);
    }
  } else {
    #pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const float v = kScaled ? value<T>(c, j) * s.up : value<T>(c, j), t = __fmul_rn(v, s.inv);
      const float m = __fadd_rn(t, kMagic);
      q[j] = __float_as_uint(m);
      if (fabsf(__fsub_rn(t, __fsub_rn(m, kMagic))) > kBorder) {
        const int k = static_cast<int>(fabsf(t));
        const double lhs = 254.0 * static_cast<double>(fabsf(v)), rhs = static_cast<double>(2 * k + 1) * static_cast<double>(s.top);
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

template <typename T>
__device__ __forceinline__ uint4 codes(const Chunk<T>& c, const RowScale& s) {
  if (s.zero) return make_uint4(0u, 0u, 0u, 0u);
  return s.up == 1.0f ? cast_chunk<T, false>(c, s) : cast_chunk<T, true>(c, s);
}

// blockDim.y rows a block, blockDim.x threads a row (one warp when there is
// more than one row).  40 registers for 2-byte inputs (57 left two blocks of
// 352 threads an SM: 4096 rows of 11008 took 43.7 us, 33.9 with 40), 64 for
// fp32, whose chunks take 32 (48 and fewer spill).
//
// Measured on a B200, inputs larger than L2: 8192 x 4096 bf16 23.0-23.9 us (4.2
// to 4.4 TB/s of the 6.5 TB/s a copy reaches), fp32 28.6-28.9 us (5.8).  bf16 is bound by
// instructions: some 11 an element, most of them the exact tie rule.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads, sizeof(T) == 2 ? 3 : 2) quantize_int8_kernel(const Int8QuantizeParams p) {
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
  bits = __reduce_max_sync(0xFFFFFFFFu, max_bits<T>(bits));
  if (blockDim.y == 1) {
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = bits;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    bits = __reduce_max_sync(0xFFFFFFFFu, lane < static_cast<int>(blockDim.x >> 5) ? warp_max[lane] : 0u);
  }
  if (live && tid == 0)
    p.scale[r] = bits >= 0x7F800000u ? __uint_as_float(0x7FFFFFFFu)
                                     : (bits ? __fdiv_rn(__uint_as_float(bits), 127.0f) : 1.0f);
  const RowScale rs = row_scale(bits);
  int8_t* out = p.out + (live ? r : 0) * p.ld_out;
  #pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * step < chunks)
      *reinterpret_cast<uint4*>(out + (tid + i * step) * kChunk) = codes<T>(held[i], rs);
  for (int64_t c = tid + kHeld * step; c < chunks; c += step)
    *reinterpret_cast<uint4*>(out + c * kChunk) =
        codes<T>(load_chunk<T>(row, c * kChunk, p.cols, p.vec_ok), rs);
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
