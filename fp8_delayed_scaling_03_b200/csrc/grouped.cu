// grouped.cu -- products of tokens with 8-bit weights that carry scales of
// their own: FP8 products grouped by expert with ragged sizes, and the 8-bit
// integer product with a scale per token and per channel.  sm_100a.
//
//   forward  Y[r, j]     = (sum_k X8[r, k] W8[e, j, k]) / (sx sw[e])    r in group e
//   dX       DX[r, k]    = (sum_j G8[r, j] W8[e, j, k]) / (sg sw[e])    r in group e
//   dW       DW[e, j, k] = (sum_{r in e} G8[r, j] X8[r, k]) / (sg sx)
//   int8     Y[i, j]     = (sum_k A[i, k] B[j, k]) sa[i] sb[j] + bias[j]
//
// One kernel runs all four.  Each output row is a "column" of the tile and its
// contiguous axis the "lane" axis:
//   * the operand whose index runs along the output's contiguous axis (the
//     weight's rows; X's columns for dW) is the M side of the MMA, 128 per
//     tile = the 128 TMEM lanes; the other one (the tokens; G's columns for
//     dW) is the N side, up to 256 per tile.  N may be any multiple of 16, so
//     a group's last tile costs only the tokens it has (rounded up to 16),
//     where tokens on the M side would always cost 128: what a ragged group
//     wastes is at most 15 columns of one tile, and a decoding step of a few
//     tokens streams the weights through a 16-column MMA;
//   * group sizes live on the device: each CTA scans the offsets into a
//     prefix of tile counts in shared memory and maps its persistent tile
//     indexes through a binary search.  Nothing is read back to the host;
//   * rows of a tile that belong to the next group are loaded and multiplied
//     like the others (rows past the buffer come back as zeros) and dropped
//     by the store, so no operand needs padding between groups;
//   * dW contracts over the rows of a group: a k-block may run past the
//     group's end.  Whole 32-row steps past it are not issued; the rows of
//     the last step past it are set to zero in both operands' shared memory
//     (in both, since an fp8 NaN of the next group times zero would be NaN).
// Roles as in gemm.cu: warp 0 lane 0 TMA producer, warp 1 MMA issuer, warps
// 2-9 epilogue over double-buffered TMEM accumulators, every wait bounded.
// The epilogue reads 16 lanes x 32 columns per tcgen05.ld.16x256b, whose
// register layout is the one stmatrix takes: stmatrix.trans turns the block
// over so that a token's 32 outputs are 64 contiguous bytes, which leave as
// 16-byte stores guarded by the group's end.
#include <algorithm>

#include "device.cuh"
#include "internal.h"
#include "launch.h"
#include "ring.cuh"

namespace fp8lin {
namespace {

constexpr int kLanes = 128;              // M side of a tile
constexpr int kKBlock = 128;             // bytes of the contraction per stage
constexpr int kStep = 32;                // contraction per MMA
constexpr int kThreads = 320;            // 10 warps: TMA, MMA, 8 epilogue
constexpr int kEpiWarps = 8;
constexpr int kSlab = 32 * 32 * 2;       // one staged 32 x 32 block of 2-byte outputs
constexpr int kLaneBytes = kLanes * kKBlock;
constexpr int kOperandBytes = 192 * 1024;
constexpr int kMaxStages = 10;
constexpr int kBarBytes = 256;
constexpr int kTmemCols = 512;           // two accumulators of up to 256 columns
constexpr int kRaster = 8;               // token tiles per raster group
constexpr int kSmem = kOperandBytes + kEpiWarps * kSlab + kBarBytes + 2 * (kMaxGroups + 1) * 4 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
static_assert((2 * kMaxStages + 5) * 8 + 8 <= kBarBytes, "barrier block");

__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Four 8 x 8 blocks of 2-byte values, each stored transposed: lane 8 j + c
// gives the address of column c of block j (16 bytes).
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// D(tmem) (+)= A(smem desc) x B(smem desc): 8-bit integers, int32 accumulate.
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <int OUT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (OUT == kFP16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

__device__ __forceinline__ float load_bias(const void* bias, int dtype, int j) {
  if (dtype == kFP32) return __ldg(static_cast<const float*>(bias) + j);
  const unsigned short b = __ldg(static_cast<const unsigned short*>(bias) + j);
  return dtype == kFP16 ? __half2float(__ushort_as_half(b)) : __uint_as_float(static_cast<uint32_t>(b) << 16);
}

// One tile: `cols` output rows from col0 (rows of the buffer, or of D_e for
// dW) by 128 lanes from lane0, contraction blocks [0, kb) from row/byte k0.
struct Tile {
  int e, col0, cols, lane0, kb, k0, kvalid;
};

template <bool kRaggedK>
__device__ __forceinline__ Tile tile_of(const GroupedParams& p, const int* bound, const int* first, int t) {
  Tile w;
  if constexpr (kRaggedK) {
    const int per = p.tiles_lane * p.tiles_col;
    w.e = t / per;
    t -= w.e * per;
    const int tl = t % p.tiles_lane, tc = t / p.tiles_lane;
    w.lane0 = tl * kLanes;
    w.col0 = tc * p.col_tile;
    w.cols = min(p.col_tile, p.ncol - w.col0);
    w.k0 = bound[w.e];
    w.kvalid = bound[w.e + 1] - w.k0;
    w.kb = (w.kvalid + kKBlock - 1) / kKBlock;
  } else {
    // the group whose tiles hold t: the largest e with first[e] <= t and tiles of its own
    int lo = 0, hi = p.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= t) lo = mid;
      else hi = mid;
    }
    w.e = lo;
    t -= first[lo];
    const int row0 = bound[lo], rows = bound[lo + 1] - row0;
    const int tiles_col = (rows + p.col_tile - 1) / p.col_tile;
    const int per = kRaster * p.tiles_lane;
    const int g = t / per;
    const int gc = min(kRaster, tiles_col - g * kRaster);
    t -= g * per;
    const int tc = g * kRaster + t % gc;
    w.lane0 = (t / gc) * kLanes;
    w.col0 = row0 + tc * p.col_tile;
    w.cols = min(p.col_tile, row0 + rows - w.col0);
    w.k0 = 0;
    w.kvalid = 0;
    w.kb = p.k_blocks;
  }
  return w;
}

// Group bounds (clamped to the buffer and made non-decreasing by a running
// maximum, so that no offset can lead outside it or let two groups share a
// row) and the index of each group's first tile.  One warp.
template <bool kRaggedK>
__device__ __forceinline__ void scan_groups(const GroupedParams& p, int* bound, int* first, int lane) {
  int top = 0, tiles = 0;
  if (!p.offsets) {
    if (lane == 0) {
      bound[0] = 0;
      bound[1] = p.rows;
      first[0] = 0;
      first[1] = kRaggedK ? p.tiles_lane * p.tiles_col : (p.rows + p.col_tile - 1) / p.col_tile * p.tiles_lane;
    }
    return;
  }
  auto offset = [&](int i) {
    const int64_t v = p.off64 ? static_cast<const int64_t*>(p.offsets)[i]
                              : static_cast<int64_t>(static_cast<const int*>(p.offsets)[i]);
    return static_cast<int>(min(max(v, static_cast<int64_t>(0)), static_cast<int64_t>(p.rows)));
  };
  top = offset(0);
  if (lane == 0) {
    bound[0] = top;
    first[0] = 0;
  }
  for (int e0 = 0; e0 < p.groups; e0 += 32) {
    const int e = e0 + lane;
    int end = e < p.groups ? offset(e + 1) : 0;
    #pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, end, d);
      if (lane >= d) end = max(end, o);
    }
    end = max(end, top);
    int begin = __shfl_up_sync(0xFFFFFFFFu, end, 1);
    if (lane == 0) begin = top;
    int n = 0;
    if (e < p.groups)
      n = kRaggedK ? p.tiles_lane * p.tiles_col : (end - begin + p.col_tile - 1) / p.col_tile * p.tiles_lane;
    #pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, n, d);
      if (lane >= d) n += o;
    }
    if (e < p.groups) {
      bound[e + 1] = end;
      first[e + 1] = tiles + n;
    }
    top = __shfl_sync(0xFFFFFFFFu, end, 31);
    tiles += __shfl_sync(0xFFFFFFFFu, n, 31);
  }
}

// kInt8: 8-bit integer operands with row and lane scales; else fp8 with one
// scale per tensor or group.  kRaggedK: the contraction is ragged (dW).
template <bool kInt8, bool kRaggedK, int OUT>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap t_lane, const __grid_constant__ CUtensorMap t_col,
                   const __grid_constant__ CUtensorMap t_col32, const __grid_constant__ GroupedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int col_bytes = max(p.col_tile, 32) * kKBlock;   // a 16-column tile keeps 32-row slots: 1024-byte aligned stages
  const int stage_bytes = kLaneBytes + col_bytes;
  uint8_t* s_epi = smem + kOperandBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_epi + kEpiWarps * kSlab);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* bound = reinterpret_cast<int*>(s_epi + kEpiWarps * kSlab + kBarBytes);
  int* first = bound + kMaxGroups + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nstages = p.stages;

  if (threadIdx.x == 64) {
    for (int s = 0; s < nstages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (p.k_blocks > 0) {  // an empty contraction has no maps
      prefetch_tmap(&t_lane);
      prefetch_tmap(&t_col);
      if (!kRaggedK) prefetch_tmap(&t_col32);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  // Offsets, operands and scales may be the previous kernel's output.
  pdl_wait();
  if (warp == 3) scan_groups<kRaggedK>(p, bound, first, lane);
  tc_fence_before();
  cta_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int tiles = first[p.groups];
  pdl_trigger();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int t = blockIdx.x; t < tiles && !*abort_flag; t += gridDim.x) {
        const Tile w = tile_of<kRaggedK>(p, bound, first, t);
        // columns loaded: the whole tile in one copy, or as many 32-row
        // copies as hold the group's remaining tokens
        const bool whole = kRaggedK || w.cols > p.col_tile - 32 || p.col_tile <= 32;
        const int boxes = kRaggedK ? (w.cols + 127) / 128 : (whole ? 1 : (w.cols + 31) / 32);
        const int bytes = kLaneBytes + (kRaggedK ? boxes * 128 * kKBlock : (whole ? p.col_tile : boxes * 32) * kKBlock);
        const int z = kRaggedK || p.lane_shared ? 0 : w.e;
        for (int kb = 0; kb < w.kb; ++kb, ++issued) {
          if (issued >= nstages && !mbar_wait(&empty[stage], phase ^ 1u, p.status, abort_flag)) break;
          uint8_t* s_lane = smem + stage * stage_bytes;
          uint8_t* s_col = s_lane + kLaneBytes;
          const int k = w.k0 + kb * kKBlock;
          mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(bytes));
          if (p.lane_mn) tma_load_3d(s_lane, &t_lane, &full[stage], w.lane0, k, z);
          else           tma_load_3d(s_lane, &t_lane, &full[stage], k, w.lane0, z);
          if constexpr (kRaggedK) {
            for (int b = 0; b < boxes; ++b)
              tma_load_3d(s_col + b * 128 * kKBlock, &t_col, &full[stage], w.col0 + b * 128, k, 0);
          } else if (whole) {
            tma_load_3d(s_col, &t_col, &full[stage], k, w.col0, 0);
          } else {
            for (int b = 0; b < boxes; ++b)
              tma_load_3d(s_col + b * 32 * kKBlock, &t_col32, &full[stage], k, w.col0 + b * 32, 0);
          }
          if (++stage == nstages) { stage = 0; phase ^= 1u; }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // dW runs the loop with the whole warp (its lanes clear the rows past a
    // group's end), lane 0 alone waits and issues; else lane 0 only.
    if (kRaggedK || lane == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, issued = false;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const Tile w = tile_of<kRaggedK>(p, bound, first, t);
        // N: the tile's columns, rounded up to 16; dW's column operand is
        // MN-major in chunks of 128, which it takes whole
        const int n = kRaggedK ? (w.cols + 127) / 128 * 128 : (w.cols + 15) / 16 * 16;
        const uint32_t idesc = p.idesc | static_cast<uint32_t>(n >> 3) << 17;
        if (lane == 0) ok = mbar_wait(&tempty[acc], acc_phase ^ 1u, p.status, abort_flag);
        if (kRaggedK) ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
        for (int kb = 0; kb < w.kb; ++kb) {
          if (lane == 0) ok = mbar_wait(&full[stage], phase, p.status, abort_flag);
          if (kRaggedK) ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
          if (!ok) break;
          tc_fence_after();
          uint8_t* s_lane = smem + stage * stage_bytes;
          int steps = kKBlock / kStep;
          if constexpr (kRaggedK) {
            const int valid = w.kvalid - kb * kKBlock;   // rows of this block inside the group
            if (valid < kKBlock) {
              steps = (valid + kStep - 1) / kStep;
              if (valid % kStep) {
                (void)mbar_try_wait(smem_u32(&full[stage]), phase);  // each lane acquires the copies' bytes
                // rows [valid, 32 steps) of the lane operand and of each 128-column chunk of the other:
                // 128 bytes a row, 16 per lane
                const int chunks = 1 + (w.cols + 127) / 128;
                const int words = (steps * kStep - valid) * (kKBlock / 16);
                for (int c = 0; c < chunks; ++c) {
                  uint4* row = reinterpret_cast<uint4*>(s_lane + c * 128 * kKBlock + valid * kKBlock);
                  for (int i = lane; i < words; i += 32) row[i] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
              }
            }
          }
          if (lane == 0) {
            const uint32_t a_base = smem_u32(s_lane), b_base = a_base + kLaneBytes;
            #pragma unroll
            for (int kk = 0; kk < kKBlock / kStep; ++kk) {
              if (kRaggedK && kk >= steps) break;
              // K-major: 32 bytes along the swizzled 128-byte row; MN-major: 32 rows of 128 bytes
              const uint64_t ad = !p.lane_mn ? smem_desc_sw128(a_base + kk * kStep, 16, 1024)
                                             : smem_desc_sw128(a_base + kk * kStep * 128, 128 * kKBlock, 1024);
              const uint64_t bd = !kRaggedK ? smem_desc_sw128(b_base + kk * kStep, 16, 1024)
                                            : smem_desc_sw128(b_base + kk * kStep * 128, 128 * kKBlock, 1024);
              const uint32_t accum = (kb | kk) ? 1u : 0u;
              if constexpr (kInt8) umma_i8(d_tmem, ad, bd, idesc, accum);
              else                 umma_f8f6f4(d_tmem, ad, bd, idesc, accum);
            }
            umma_commit(&empty[stage]);
          }
          if (kRaggedK) __syncwarp();
          if (++stage == nstages) { stage = 0; phase ^= 1u; }
        }
        if (lane == 0) {
          if (w.kb > 0) umma_commit(&tfull[acc]);
          else mbar_arrive(&tfull[acc]);  // empty contraction: nothing was issued
          issued = issued || w.kb > 0;
        }
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      // no MMA may still read shared memory or TMEM when the CTA tears down
      if (lane == 0 && issued) {
        umma_commit(drain);
        mbar_wait(drain, 0, nullptr, nullptr);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int ew = warp - 2;
    const int qd = warp & 3;          // TMEM lane quadrant of this warp
    const int half = ew >> 2;         // of the 32-column steps: 0 the even ones, 1 the odd ones
    if (blockIdx.x == 0 && threadIdx.x == 64) {
      for (int i = 0; i < 2; ++i) {
        if (p.side.copy_dst[i]) *p.side.copy_dst[i] = *p.side.copy_src[i];
        if (p.side.zero_dst[i]) *p.side.zero_dst[i] = 0.0f;
      }
    }
    if (blockIdx.x == 0 && ew == 2)
      for (int i = lane; i < p.sw_n; i += 32) p.sw_dst[i] = p.sw_src[i];
    if (blockIdx.x == 0 && ew == 1)
      for (int i = 0; i < p.nfin; ++i) ring_finalize_warp(p.fin[i], lane);
    const uint32_t slab = smem_u32(s_epi + ew * kSlab);
    const uint8_t* slab_ptr = s_epi + ew * kSlab;
    // stmatrix: this lane's 16 bytes of column (8 i + lane % 8), block lane / 8, 64-byte swizzle
    const uint32_t st_addr = slab + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) * 16);
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = blockIdx.x; t < tiles && !*abort_flag; t += gridDim.x) {
      const Tile w = tile_of<kRaggedK>(p, bound, first, t);
      const int n0 = w.lane0 + qd * 32;       // first output column of this warp
      const int steps = (w.cols + 31) / 32;
      // per-lane factors, fetched before the wait for the accumulator: this
      // thread's lanes are n0 + 8 j + lane / 4, j = 0..3
      float f[4], b[4];
      if constexpr (kInt8) {
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + 8 * j + (lane >> 2);
          f[j] = n < p.nlane && w.kb > 0 ? __ldg(p.scale_b + n) : 0.0f;
          b[j] = p.bias && n < p.nlane ? load_bias(p.bias, p.bias_dtype, n) : 0.0f;
        }
      } else {
        f[0] = w.kb > 0 ? 1.0f / (*p.scale_a * p.scale_b[w.e * p.scale_b_step]) : 0.0f;
      }
      // a warp leaves together: a lane that gave up must not strand the others
      // at the next warp barrier
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull[acc], acc_phase, p.status, abort_flag))) break;
      tc_fence_after();
      uint8_t* const d = static_cast<uint8_t*>(p.d) +
                         (static_cast<int64_t>(w.e) * p.stride_d + static_cast<int64_t>(w.col0) * p.ldd) * (OUT == kFP32 ? 4 : 2);
      if (half >= steps) {
        if (lane == 0) mbar_arrive(&tempty[acc]);
      }
      #pragma unroll 1
      for (int st = half; st < steps; st += 2) {
        uint32_t r[2][16];
        if (w.kb > 0) {
          __syncwarp();
          const uint32_t ta = tmem_base + (static_cast<uint32_t>(qd * 32) << 16) + static_cast<uint32_t>(acc * 256 + st * 32);
          tmem_ld_16x256b_x4(ta, r[0]);
          tmem_ld_16x256b_x4(ta + (16u << 16), r[1]);
          tmem_ld_wait();
        } else {  // empty contraction: the MMA never wrote this accumulator
          #pragma unroll
          for (int i = 0; i < 16; ++i) r[0][i] = r[1][i] = 0u;
        }
        if (st + 2 >= steps) {  // this warp's last read of the accumulator
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
        }
        const int c0 = st * 32;               // first column of this step within the tile
        const int live = min(32, w.cols - c0);
        // r[h][4 i + 2 b + u]: lane 16 h + 8 b + lane / 4, column 8 i + 2 (lane % 4) + u
        float v[2][16];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          float s[2] = {1.0f, 1.0f};
          if constexpr (kInt8) {
            #pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int c = 8 * i + 2 * (lane & 3) + u;
              s[u] = c < live && w.kb > 0 ? __ldg(p.scale_a + w.col0 + c0 + c) : 0.0f;
            }
          }
          #pragma unroll
          for (int h = 0; h < 2; ++h)
            #pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t x = r[h][4 * i + q];
              if constexpr (kInt8)
                v[h][4 * i + q] = __fadd_rn(__fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(x)), s[q & 1]), f[2 * h + (q >> 1)]),
                                            b[2 * h + (q >> 1)]);
              else
                v[h][4 * i + q] = __uint_as_float(x) * f[0];
            }
        }
        if constexpr (OUT == kFP32) {
          // eight lanes hold 8 consecutive floats of a row: 32-byte sectors, no staging
          float* df = reinterpret_cast<float*>(d);
          #pragma unroll
          for (int h = 0; h < 2; ++h)
            #pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int c = 8 * (i >> 2) + 2 * (lane & 3) + (i & 1);
              const int n = n0 + 16 * h + 8 * ((i >> 1) & 1) + (lane >> 2);
              if (c < live && n < p.nlane) df[static_cast<int64_t>(c0 + c) * p.ldd + n] = v[h][i];
            }
        } else {
          #pragma unroll
          for (int i = 0; i < 4; ++i)
            stmatrix_x4_trans(st_addr + i * 8 * 64, pack2<OUT>(v[0][4 * i], v[0][4 * i + 1]),
                              pack2<OUT>(v[0][4 * i + 2], v[0][4 * i + 3]), pack2<OUT>(v[1][4 * i], v[1][4 * i + 1]),
                              pack2<OUT>(v[1][4 * i + 2], v[1][4 * i + 3]));
          __syncwarp();
          unsigned short* dh = reinterpret_cast<unsigned short*>(d);
          if (p.vec_ok) {
            #pragma unroll
            for (int it = 0; it < 4; ++it) {
              const int c = it * 8 + (lane >> 2), q = lane & 3;
              const int n = n0 + q * 8;
              const uint4 o = *reinterpret_cast<const uint4*>(slab_ptr + c * 64 + ((q ^ ((c >> 1) & 3)) * 16));
              if (c < live && n < p.nlane) {
                unsigned short* dst = dh + static_cast<int64_t>(c0 + c) * p.ldd + n;
                if (n + 8 <= p.nlane) {
                  *reinterpret_cast<uint4*>(dst) = o;
                } else {
                  const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
                  #pragma unroll
                  for (int j = 0; j < 8; ++j)
                    if (n + j < p.nlane) dst[j] = static_cast<unsigned short>(ow[j >> 1] >> (16 * (j & 1)));
                }
              }
            }
          } else if (n0 + lane < p.nlane) {
            // rows that 16-byte stores cannot address: a lane per output column
            unsigned short* dst = dh + static_cast<int64_t>(c0) * p.ldd + n0 + lane;
            for (int c = 0; c < live; ++c)
              dst[static_cast<int64_t>(c) * p.ldd] = *reinterpret_cast<const unsigned short*>(
                  slab_ptr + c * 64 + (((lane >> 3) ^ ((c >> 1) & 3)) * 16) + (lane & 7) * 2);
          }
          __syncwarp();  // the next step overwrites the slab
        }
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }

  tc_fence_before();
  cta_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <bool kInt8, bool kRaggedK, int OUT>
cudaError_t launch_build(const CUtensorMap* maps, const GroupedParams& p, int grid, int dev, cudaStream_t s) {
  static bool configured[64] = {};
  auto kernel = grouped_kernel<kInt8, kRaggedK, OUT>;
  if (!configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), kSmem, s, maps[0], maps[1], maps[2], p);
}

}  // namespace

int grouped_stages(int col_tile) {
  return std::min(kMaxStages, kOperandBytes / (kLaneBytes + std::max(col_tile, 32) * kKBlock));
}

cudaError_t launch_grouped(const CUtensorMap* maps, const GroupedParams& p, bool int8, bool ragged_k, int out_dtype,
                           int64_t max_tiles, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = num_sms(dev);
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(sms, max_tiles)));
  if (!int8) return ragged_k ? launch_build<false, true, kBF16>(maps, p, grid, dev, s)
                             : launch_build<false, false, kBF16>(maps, p, grid, dev, s);
  if (out_dtype == kFP32) return launch_build<true, false, kFP32>(maps, p, grid, dev, s);
  if (out_dtype == kFP16) return launch_build<true, false, kFP16>(maps, p, grid, dev, s);
  return launch_build<true, false, kBF16>(maps, p, grid, dev, s);
}

}  // namespace fp8lin
