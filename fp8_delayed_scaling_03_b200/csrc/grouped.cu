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
//     (in both, since an fp8 NaN of the next group times zero would be NaN) by
//     a warp of its own, as the block lands.
// The stages of the operand ring take what shared memory the group tables (8
// bytes a group) leave: 192 KB up to 190 groups, a stage less beyond.
// Roles as in gemm.cu: warp 0 TMA producer, warp 1 MMA issuer, warps 2-9
// epilogue over double-buffered TMEM accumulators, every wait bounded.
// The epilogue reads 16 lanes x 32 columns per tcgen05.ld.16x256b, whose
// register layout is the one stmatrix takes: stmatrix.trans turns the block
// over so that a token's outputs are contiguous in a swizzled slab (64 lanes =
// 128 bytes, two warps), which leaves by a TMA store.  A block cut by its
// group's end (which TMA cannot clip: the next group's rows follow) leaves as
// 16-byte stores guarded by that end, and one of rows that TMA cannot address
// as 4-byte stores.
//
// Tiles.  Large products run on CTA pairs, 256 lanes x 256 columns: a CTA then
// loads 32 KB a k-block where a lone one of 128 x 256 loads 48 KB.  Few tokens
// run on single CTAs with narrow tiles, few tiles on clusters that split K, and
// dW of few rows a group, which its output bounds, on single CTAs
// (pick_grouped_tile in api.cu has the rule and its times).
//
// Measured on a B200 (graph replay; `of measured`: the copy bandwidth 6.53 TB/s
// and twice the cuBLAS bf16 burst rate, 3.34 PFLOP/s):
//   8192 rows in 8 equal groups, 11008 x 4096: forward 257-274 us (2.69-2.88
//     PFLOP/s, 0.81-0.86), dX 241-256 us (2.89-3.06, 0.86-0.92), dW 295-304 us
//     (2.43-2.50, 0.73-0.75); one group 256-267, 242-252 and 242-253 us.  Short
//     of power these are bound by the loads' latency against 192 KB of stages;
//     run without a pause the card's 1 kW limit holds them at 2.1-2.4 PFLOP/s,
//     where twice cuBLAS bf16's sustained rate is 2.8.
//     dW's 721 MB of output take 140 us at the 5.1 TB/s that the store path
//     reaches, and share the memory with the loads.
//   128 rows over 64 groups, 6912 x 1536: 91 us, 6.1 TB/s of weights (0.92).
//   4 rows over 8 groups, 4096 x 1024: 5.7 us, of which 3.2 us is what any
//     launch takes (offsets from L2 and their scan 0.8, first load 1.2, the
//     store's way out 0.6).
//   dW of one row over 22 groups, 10181 x 128: 14.8 us, 3.9 TB/s of output; 14
//     rows over 18 groups, 8317 x 1814 (rows of odd pitch): 156-166 us, 3.3-3.5
//     TB/s.
//   int8, 8192 x 11008 x 4096: 238-241 us (3.07-3.10 PFLOP/s): kind::i8 has
//     fp8's rate; fp32 out 253-256 us.
#include <algorithm>
#include <atomic>

#include "device.cuh"
#include "internal.h"
#include "launch.h"
#include "ring.cuh"

namespace fp8lin {
namespace {

constexpr int kLanes = 128;              // M side of a tile
constexpr int kKBlock = 128;             // bytes of the contraction per stage
constexpr int kStep = 32;                // contraction per MMA
constexpr int kEpiWarps = 8;
constexpr int kClearWarp = 2 + kEpiWarps; // dW: clears the rows of a group's last block past its end
constexpr int kThreads = 320;            // 10 warps: TMA, MMA, 8 epilogue
constexpr int kThreadsRaggedK = kThreads + 32;
constexpr int kSlab = 32 * 64 * 2;       // one staged block of 2-byte outputs: 32 columns x 64 lanes, two warps
constexpr int kSlabBytes = kEpiWarps / 2 * 2 * kSlab;  // two per two epilogue warps
constexpr int kLaneBytes = kLanes * kKBlock;
constexpr int kOperandBytes = 192 * 1024;
constexpr int kMaxStages = 10;
constexpr int kBarBytes = 512;
constexpr int kTmemCols = 512;           // two accumulators of up to 256 columns
constexpr int kRaster = 8;               // token tiles per raster group
// Shared memory: [operand stages][slabs][barriers][group bounds, first tiles].
constexpr int kSmemMax = 227 * 1024;
constexpr int kFixedSmem = 1024 + kSlabBytes + kBarBytes;
static_assert((4 * kMaxStages + 6) * 8 + 8 <= kBarBytes, "barrier block");

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

// Whether a phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ void umma_i8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on an mbarrier of either CTA of the pair without release: it tells
// that TMEM reads have completed (tcgen05.wait::ld before it), no memory is
// handed over.  A release at cluster scope would wait for the warp's output
// stores to be performed first.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Arrive on an mbarrier of either CTA of the pair, releasing at CTA scope: what
// it releases -- cleared rows of this CTA's shared memory -- is ordered before
// the MMA's reads by the proxy fence ahead of it, and is read by this SM's own
// tensor core.  (A release at cluster scope takes 1,100 cycles, a cluster-wide
// proxy fence another 1,050: together they stalled every tile of dW whose
// group ends inside a k-block, 415 us against 366 for 8192 rows in 8 uneven groups of 11008 x 4096.)
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// 16 bytes into the shared memory of a CTA of the cluster; their arrival is
// counted on its mbarrier.
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
      "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
      : "memory");
}

// Accumulators as register bits: int32 (exact) or fp32 sums.
template <bool kInt8>
__device__ __forceinline__ uint32_t add_sums(uint32_t a, uint32_t b) {
  return kInt8 ? a + b : __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}

// (a, b) = (x f, y f), one instruction.
__device__ __forceinline__ void mul_x2(float& a, float& b, float x, float y, float f) {
  asm("{\n\t.reg .b64 p, q;\n\t"
      "mov.b64 p, {%2, %3};\n\t"
      "mov.b64 q, {%4, %4};\n\t"
      "mul.rn.f32x2 p, p, q;\n\t"
      "mov.b64 {%0, %1}, p;\n\t}"
      : "=f"(a), "=f"(b)
      : "f"(x), "f"(y), "f"(f));
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
  // (plain loads: the read-only path does not promise to see what the kernel before wrote)
  if (dtype == kFP32) return static_cast<const float*>(bias)[j];
  const unsigned short b = static_cast<const unsigned short*>(bias)[j];
  return dtype == kFP16 ? __half2float(__ushort_as_half(b)) : __uint_as_float(static_cast<uint32_t>(b) << 16);
}

// One tile: `cols` output rows from col0 (rows of the buffer, or of D_e for
// dW) by 128 (a pair's: 256) lanes from lane0, contraction blocks [0, kb) from
// row/byte k0; kvalid rows of the group remain from k0 (dW).
struct Tile {
  int e, col0, cols, lane0, kb, k0, kvalid;
};

// The tile of index t of a product of tokens: the group whose tiles hold t,
// then groups of kRaster column tiles, lane tile by lane tile.
template <int kTileLanes>
__device__ __forceinline__ Tile token_tile(const GroupedParams& p, const int* bound, const int* first, int t) {
  Tile w;
  // the largest e with first[e] <= t and tiles of its own
  int lo = 0, hi = p.groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= t) lo = mid;
    else hi = mid;
  }
  w.e = lo;
  t -= first[lo];
  const int row0 = bound[lo], rows = bound[lo + 1] - row0;
  const int tiles_col = (rows + p.col_tile - 1) >> p.col_shift;
  int tc = 0, tl = t;
  if (tiles_col > 1) {   // (divisions are in the way of the first loads of a small launch)
    int base = 0;
    if (tiles_col > kRaster) {
      const int per = kRaster * p.tiles_lane, g = t / per;
      t -= g * per;
      base = g * kRaster;
    }
    const int gc = min(kRaster, tiles_col - base);
    tl = t / gc;
    tc = base + t - tl * gc;
  }
  w.lane0 = tl * kTileLanes;
  w.col0 = row0 + tc * p.col_tile;
  w.cols = min(p.col_tile, row0 + rows - w.col0);
  w.k0 = 0;
  w.kvalid = 0;
  w.kb = p.k_blocks;
  return w;
}

// The tiles unit, unit + units, ... of a launch, one after another.  A ragged
// contraction has the same tiles in every group, so its cursor is a mixed-radix
// counter (group, column tile, lane tile) that adds the digits of `units`:
// three divisions once, none per tile, which tiles of one or two k-blocks feel.
template <bool kRaggedK, int kTileLanes>
struct Cursor {
  int t, units;
  int e, tc, tl, de, dtc, dtl;   // kRaggedK
  __device__ __forceinline__ Cursor(const GroupedParams& p, int unit, int units_) : t(unit), units(units_) {
    if constexpr (kRaggedK) {
      const int per = p.tiles_lane * p.tiles_col;
      e = unit / per;
      tc = (unit - e * per) / p.tiles_lane;
      tl = unit - e * per - tc * p.tiles_lane;
      de = units / per;
      dtc = (units - de * per) / p.tiles_lane;
      dtl = units - de * per - dtc * p.tiles_lane;
    }
  }
  __device__ __forceinline__ void advance(const GroupedParams& p) {
    t += units;
    if constexpr (kRaggedK) {
      tl += dtl;
      int carry = tl >= p.tiles_lane;
      tl -= carry ? p.tiles_lane : 0;
      tc += dtc + carry;
      carry = tc >= p.tiles_col;
      tc -= carry ? p.tiles_col : 0;
      e += de + carry;
    }
  }
  __device__ __forceinline__ Tile tile(const GroupedParams& p, const int* bound, const int* first) const {
    if constexpr (kRaggedK) {
      Tile w;
      w.e = e;
      w.lane0 = tl * kTileLanes;
      w.col0 = tc * p.col_tile;
      w.cols = min(p.col_tile, p.ncol - w.col0);
      w.k0 = bound[e];
      w.kvalid = bound[e + 1] - w.k0;
      w.kb = (w.kvalid + kKBlock - 1) / kKBlock;
      return w;
    } else {
      return token_tile<kTileLanes>(p, bound, first, t);
    }
  }
};

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
      first[1] = kRaggedK ? p.tiles_lane * p.tiles_col : ((p.rows + p.col_tile - 1) >> p.col_shift) * p.tiles_lane;
    }
    return;
  }
  auto offset = [&](int i) {
    const int64_t v = p.off64 ? static_cast<int64_t>(__ldcg(static_cast<const long long*>(p.offsets) + i))
                              : static_cast<int64_t>(__ldcg(static_cast<const int*>(p.offsets) + i));
    return static_cast<int>(min(max(v, static_cast<int64_t>(0)), static_cast<int64_t>(p.rows)));
  };
  // (the loads of a round are issued before the round that precedes it is
  // scanned: one trip to L2 for up to 32 groups)
  int ahead = lane < p.groups ? offset(lane + 1) : 0;
  top = offset(0);
  if (lane == 0) {
    bound[0] = top;
    first[0] = 0;
  }
  for (int e0 = 0; e0 < p.groups; e0 += 32) {
    const int e = e0 + lane;
    int end = ahead;
    if (e + 32 < p.groups) ahead = offset(e + 33);
    const int live = min(32, p.groups - e0);
    if (e >= p.groups) end = 0;
    int begin = __shfl_up_sync(0xFFFFFFFFu, end, 1);
    if (lane == 0) begin = top;
    if (__any_sync(0xFFFFFFFFu, lane < live && end < begin)) {   // an offset falls: the running maximum
      for (int d = 1; d < live; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, end, d);
        if (lane >= d) end = max(end, o);
      }
      end = max(end, top);
      begin = __shfl_up_sync(0xFFFFFFFFu, end, 1);
      if (lane == 0) begin = top;
    }
    int n;   // tiles up to and with this group, of this round
    if constexpr (kRaggedK) {
      n = (min(lane, live - 1) + 1) * p.tiles_lane * p.tiles_col;
    } else {
      n = lane < live ? ((end - begin + p.col_tile - 1) >> p.col_shift) * p.tiles_lane : 0;
      for (int d = 1; d < live; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, n, d);
        if (lane >= d) n += o;
      }
    }
    if (e < p.groups) {
      bound[e + 1] = end;
      first[e + 1] = tiles + n;
    }
    top = __shfl_sync(0xFFFFFFFFu, end, live - 1);
    tiles += __shfl_sync(0xFFFFFFFFu, n, live - 1);
  }
}

// Clears rows [from, to) of this CTA's `chunks` operand chunks of 128 rows x
// 128 bytes (MN-major: a row is one index of the contraction).  One warp.
__device__ __forceinline__ void clear_rows(uint8_t* stage, int chunks, int from, int to, int lane) {
  const int words = (to - from) * (kKBlock / 16);
  for (int c = 0; c < chunks; ++c) {
    uint4* row = reinterpret_cast<uint4*>(stage + c * 128 * kKBlock + from * kKBlock);
    for (int i = lane; i < words; i += 32) row[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// kInt8: 8-bit integer operands with row and lane scales; else fp8 with one
// scale per tensor or group.  kRaggedK: the contraction is ragged (dW).
// kPair: a cluster of two CTAs runs tiles of 256 lanes with 2-SM MMAs: each CTA
// loads 128 lanes and half of the columns into its own shared memory, the even
// one issues, and each holds its 128 lanes' accumulators.
// kSplit: a cluster of p.split CTAs shares one tile per launch, each with a
// share of its k-blocks (few tiles, see pick_grouped_tile).
template <bool kInt8, bool kRaggedK, bool kPair, bool kSplit, int OUT>
__global__ void __launch_bounds__(kRaggedK ? kThreadsRaggedK : kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap t_lane, const __grid_constant__ CUtensorMap t_col,
                   const __grid_constant__ CUtensorMap t_lane32, const __grid_constant__ CUtensorMap t_col32,
                   const __grid_constant__ CUtensorMap t_d, const __grid_constant__ GroupedParams p) {
  static_assert(!kSplit || (!kPair && !kRaggedK), "split tiles are single-CTA tiles of tokens");
  constexpr int kTileLanes = kPair ? 2 * kLanes : kLanes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int cta_cols = kPair ? p.col_tile / 2 : p.col_tile;   // columns of a whole tile that this CTA loads
  const int col_bytes = max(cta_cols, 32) * kKBlock;   // a 16-column tile keeps 32-row slots: 1024-byte aligned stages
  const int stage_bytes = kLaneBytes + col_bytes;
  uint8_t* s_epi = smem + p.stages * stage_bytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_epi + kSlabBytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  // dW, one each per stage, for a group's last block that runs past its end:
  // its bytes landed in this CTA; every CTA's part is cleared (the issuer's CTA)
  uint64_t* landed = drain + 1;
  uint64_t* cleared = landed + kMaxStages;
  uint64_t* joined = cleared + kMaxStages;  // split tiles, rank 0: the other ranks' partial sums landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(joined + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* bound = reinterpret_cast<int*>(s_epi + kSlabBytes + kBarBytes);
  int* first = bound + p.groups + 1;
  // split tiles, rank 0: partial sums of ranks 1 .. split - 1 (16-byte aligned), each [32-column
  // step][epilogue warp][4 registers][lane] in the epilogue's register order
  uint8_t* partials = s_epi + kSlabBytes + kBarBytes + (2 * (p.groups + 1) * 4 + 15) / 16 * 16;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nstages = p.stages;
  const int rank = kPair ? static_cast<int>(cluster_rank()) : 0;      // place in the tile's geometry
  const int part = kSplit ? static_cast<int>(cluster_rank()) : 0;     // share of its k-blocks
  const int per_unit = kPair ? 2 : (kSplit ? p.split : 1);
  const int unit = static_cast<int>(blockIdx.x) / per_unit;
  const int units = static_cast<int>(gridDim.x) / per_unit;

  if (threadIdx.x == 64) {
    for (int s = 0; s < nstages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      if (kRaggedK) {
        mbar_init(&landed[s], 1);
        mbar_init(&cleared[s], kPair ? 2 : 1);
      }
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kPair ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(drain, 1);
    if (kSplit) mbar_init(joined, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (p.tma_store) prefetch_tmap(&t_d);
    if (p.k_blocks > 0) {  // an empty contraction has no maps
      prefetch_tmap(&t_lane);
      prefetch_tmap(&t_col);
      if (kRaggedK) prefetch_tmap(&t_lane32);
      if (kRaggedK || p.col_tile > 32) prefetch_tmap(&t_col32);
    }
  }
  if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(tmem_slot, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, kTmemCols);
      tmem_relinquish();
    }
  }
  // Offsets, operands and scales may be the previous kernel's output.  A
  // launch behind an independent product (dW behind dX) waits at its end
  // instead, see late_wait.
  if (!p.late_wait) pdl_wait();
  if (warp == 3) scan_groups<kRaggedK>(p, bound, first, lane);
  tc_fence_before();
  if constexpr (kPair || kSplit) cluster_sync();  // every CTA's barriers exist before another signals them
  else cta_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int tiles = first[p.groups];
  pdl_trigger();
  // the tile a role's cursor is at; of a split tile, this CTA's share of the k-blocks
  using Tiles = Cursor<kRaggedK, kTileLanes>;
  auto tile_at = [&](const Tiles& at) {
    Tile w = at.tile(p, bound, first);
    if constexpr (kSplit) {
      const int from = part * w.kb / p.split;
      w.kb = (part + 1) * w.kb / p.split - from;
      w.k0 = from * kKBlock;
    }
    return w;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // (the whole warp, converged, one elected lane issues: see the MMA issuer)
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    for (Tiles at(p, unit, units); at.t < tiles; at.advance(p)) {
      const Tile w = tile_at(at);
      // columns this CTA loads: its whole share of the tile in one copy, or
      // as many 32-row copies as hold its share of the remaining tokens
      const int share = kPair ? (w.cols + 31) / 32 * 16 : w.cols;
      const bool whole = kRaggedK || share > cta_cols - 32 || cta_cols <= 32;
      const int boxes = kRaggedK ? (kPair ? 1 : (w.cols + 127) / 128) : (whole ? 1 : (share + 31) / 32);
      const int bytes = kLaneBytes + (kRaggedK ? boxes * 128 : (whole ? cta_cols : boxes * 32)) * kKBlock;
      const int lane0 = w.lane0 + rank * kLanes;
      const int col0 = w.col0 + rank * (kRaggedK ? 128 : share);
      const int z = kRaggedK || p.lane_shared ? 0 : w.e;
      auto load = [&](int st, int kb) {
        uint8_t* s_lane = smem + st * stage_bytes;
        uint8_t* s_col = s_lane + kLaneBytes;
        const int k = w.k0 + kb * kKBlock;
        const int lane_x = p.lane_mn ? lane0 : k, lane_y = p.lane_mn ? k : lane0;
        if constexpr (kRaggedK) {
          const int valid = w.kvalid - kb * kKBlock;
          if (valid < kKBlock && valid % kStep != 0) {
            // The group's last block, to be cleared past its end: only the
            // 32-row steps that hold rows of the group, into this CTA's own
            // `landed` barrier; `full` just takes its turn.
            const int parts = (valid + kStep - 1) / kStep;
            if (rank == 0) mbar_arrive(&full[st]);
            mbar_arrive_expect_tx(&landed[st], static_cast<uint32_t>(parts * kStep * 128 * (1 + boxes)));
            for (int i = 0; i < parts; ++i) {
              tma_load_3d(s_lane + i * kStep * 128, &t_lane32, &landed[st], lane0, k + i * kStep, 0);
              for (int b = 0; b < boxes; ++b)
                tma_load_3d(s_col + b * 128 * kKBlock + i * kStep * 128, &t_col32, &landed[st], col0 + b * 128,
                            k + i * kStep, 0);
            }
            return;
          }
        }
        if constexpr (kPair) {
          // both CTAs' bytes are counted on the even CTA's full barrier
          const uint32_t bar = mapa_shared(smem_u32(&full[st]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(2 * bytes));
          tma_load_3d_pair(s_lane, &t_lane, bar, lane_x, lane_y, z);
          if constexpr (kRaggedK) {
            tma_load_3d_pair(s_col, &t_col, bar, col0, k, 0);
          } else if (whole) {
            tma_load_3d_pair(s_col, &t_col, bar, k, col0, 0);
          } else {
            for (int b = 0; b < boxes; ++b)
              tma_load_3d_pair(s_col + b * 32 * kKBlock, &t_col32, bar, k, col0 + b * 32, 0);
          }
        } else {
          mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(bytes));
          tma_load_3d(s_lane, &t_lane, &full[st], lane_x, lane_y, z);
          if constexpr (kRaggedK) {
            for (int b = 0; b < boxes; ++b)
              tma_load_3d(s_col + b * 128 * kKBlock, &t_col, &full[st], col0 + b * 128, k, 0);
          } else if (whole) {
            tma_load_3d(s_col, &t_col, &full[st], k, col0, 0);
          } else {
            for (int b = 0; b < boxes; ++b)
              tma_load_3d(s_col + b * 32 * kKBlock, &t_col32, &full[st], k, col0 + b * 32, 0);
          }
        }
      };
      bool ok = true;
      int kb = 0;
      while (kb < w.kb) {
        // two blocks at a time where both stages are free (the first nstages
        // loads find them so)
        const bool wrap = stage + 1 == nstages;
        const int stage1 = wrap ? 0 : stage + 1;
        const uint32_t phase1 = wrap ? phase ^ 1u : phase;
        const bool second = kb + 1 < w.kb && (issued + 1 < nstages || mbar_test(&empty[stage1], phase1 ^ 1u));
        ok = __all_sync(0xFFFFFFFFu, issued < nstages || mbar_await(&empty[stage], phase ^ 1u, p.status, abort_flag));
        if (!ok) break;
        const bool two = __all_sync(0xFFFFFFFFu, second);
        if (elect_one()) {
          load(stage, kb);
          if (two) load(stage1, kb + 1);
        }
        __syncwarp();
        issued = min(issued + (two ? 2 : 1), nstages);
        kb += two ? 2 : 1;
        stage = two ? stage1 : stage;
        phase = two ? phase1 : phase;
        if (++stage == nstages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop, converged, so that descriptors and loop
    // state stay in uniform registers; one elected lane issues.  (With lane 0
    // alone in the loop a k-block of four MMAs took 0.33 us to issue whatever
    // its columns, about as long as 256 columns take to compute.)
    const uint32_t step_k = p.lane_mn ? kStep * 128 >> 4 : kStep >> 4;   // descriptor units per 32 of the contraction
    constexpr uint32_t kColStep = kRaggedK ? kStep * 128 >> 4 : kStep >> 4;
    const uint32_t smem_base = smem_u32(smem);
    const uint64_t a_desc = p.lane_mn ? smem_desc_sw128(smem_base, 128 * kKBlock, 1024) : smem_desc_sw128(smem_base, 16, 1024);
    const uint64_t b_desc = kRaggedK ? smem_desc_sw128(smem_base + kLaneBytes, 128 * kKBlock, 1024)
                                     : smem_desc_sw128(smem_base + kLaneBytes, 16, 1024);
    const uint32_t stage_units = static_cast<uint32_t>(stage_bytes) >> 4;
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    uint32_t clear_phases = 0;   // one bit per stage
    bool ok = true, issued = false;
    // the next tile is looked up while the current one's first MMAs run, so
    // that the search is not in the way between two tiles
    Tile w{}, next{};
    Tiles at(p, unit, units);
    if (at.t < tiles) next = tile_at(at);
    while (at.t < tiles && ok) {
      w = next;
      at.advance(p);
      if (w.kb == 0 && at.t < tiles) next = tile_at(at);
      // N: the tile's columns, rounded up to 16 (a pair's: 32); dW's column
      // operand is MN-major in chunks of 128, which it takes whole
      const int n = kRaggedK ? (kPair ? 256 : (w.cols + 127) / 128 * 128)
                             : (kPair ? (w.cols + 31) / 32 * 32 : (w.cols + 15) / 16 * 16);
      const uint32_t idesc = p.idesc | static_cast<uint32_t>(n >> 3) << 17;
      ok = __all_sync(0xFFFFFFFFu, mbar_await(&tempty[acc], acc_phase ^ 1u, p.status, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * 256);
      // the MMAs of one k-block and the commit that frees its stage; one lane
      auto issue = [&](int st, int kb, int steps) {
        const uint64_t ad = a_desc + static_cast<uint32_t>(st) * stage_units;
        const uint64_t bd = b_desc + static_cast<uint32_t>(st) * stage_units;
        #pragma unroll
        for (int kk = 0; kk < kKBlock / kStep; ++kk) {
          if (kRaggedK && kk >= steps) break;
          const uint32_t accum = (kb | kk) ? 1u : 0u;
          if constexpr (kInt8) {
            if constexpr (kPair) umma_i8_pair(d_tmem, ad + kk * step_k, bd + kk * kColStep, idesc, accum);
            else                 umma_i8(d_tmem, ad + kk * step_k, bd + kk * kColStep, idesc, accum);
          } else {
            if constexpr (kPair) umma_f8f6f4_pair(d_tmem, ad + kk * step_k, bd + kk * kColStep, idesc, accum);
            else                 umma_f8f6f4(d_tmem, ad + kk * step_k, bd + kk * kColStep, idesc, accum);
          }
        }
        if constexpr (kPair) {
          const uint32_t e = smem_u32(&empty[st]);
          umma_commit_pair(e);
          umma_commit_pair(mapa_shared(e, 1));
        } else {
          umma_commit(&empty[st]);
        }
      };
      int kb = 0;
      while (kb < w.kb) {
        // Two blocks at a time where the second has landed too: waits, fences
        // and elections cost more issue time than the four MMAs between them.
        const int whole = kRaggedK ? w.kvalid / kKBlock : w.kb;   // blocks that need no clearing
        const bool wrap = stage + 1 == nstages;
        const int stage1 = wrap ? 0 : stage + 1;
        const uint32_t phase1 = wrap ? phase ^ 1u : phase;
        const bool second = kb + 1 < whole && mbar_test(&full[stage1], phase1);
        ok = __all_sync(0xFFFFFFFFu, mbar_await(&full[stage], phase, p.status, abort_flag));
        if (!ok) break;
        const bool two = __all_sync(0xFFFFFFFFu, second);
        int steps = kKBlock / kStep;
        if constexpr (kRaggedK) {
          if (kb >= whole) {   // the last block runs past the group's end
            const int valid = w.kvalid - kb * kKBlock;
            steps = (valid + kStep - 1) / kStep;
            if (valid % kStep) {
              ok = __all_sync(0xFFFFFFFFu,
                              mbar_await(&cleared[stage], (clear_phases >> stage) & 1u, p.status, abort_flag));
              if (!ok) break;
              clear_phases ^= 1u << stage;
            }
          }
        }
        tc_fence_after();
        if (elect_one()) {
          issue(stage, kb, steps);
          if (two) issue(stage1, kb + 1, kKBlock / kStep);
        }
        __syncwarp();
        issued = true;
        if (kb == 0 && at.t < tiles) next = tile_at(at);
        kb += two ? 2 : 1;
        stage = two ? stage1 : stage;
        phase = two ? phase1 : phase;
        if (++stage == nstages) { stage = 0; phase ^= 1u; }
      }
      if (elect_one()) {
        if constexpr (kPair) {
          const uint32_t f = smem_u32(&tfull[acc]);
          if (w.kb > 0) {
            umma_commit_pair(f);
            umma_commit_pair(mapa_shared(f, 1));
          } else {  // empty contraction: nothing was issued
            mbar_arrive_cluster(mapa_shared(f, 0));
            mbar_arrive_cluster(mapa_shared(f, 1));
          }
        } else {
          if (w.kb > 0) umma_commit(&tfull[acc]);
          else mbar_arrive(&tfull[acc]);
        }
      }
      __syncwarp();
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    // Given up: the other CTA's loads were waited for here alone, so it has to
    // know (settle_copies).
    if (kPair && !ok && elect_one()) st_cluster_u32(mapa_shared(smem_u32(const_cast<const int*>(abort_flag)), 1), 1u);
    // no MMA may still read shared memory or TMEM when the CTAs tear down
    if (issued && elect_one()) {
      if constexpr (kPair) umma_commit_pair(smem_u32(drain));
      else umma_commit(drain);
      mbar_await(drain, 0, nullptr, nullptr);
    }
  } else if (kRaggedK && warp == kClearWarp) {
    // ------------------------------------------------------------ clearing (dW)
    // The blocks that run past their group's end, as they land: their rows
    // past it become zeros in this CTA's operands, while the blocks before
    // them are multiplied.
    uint32_t phases = 0;   // one bit per stage
    int blocks = 0;        // k-blocks up to and with this tile's, less whole turns of the ring
    for (Tiles at(p, unit, units); at.t < tiles; at.advance(p)) {
      const Tile w = tile_at(at);
      blocks = (blocks + w.kb) % nstages;
      const int valid = w.kvalid - (w.kb - 1) * kKBlock;
      if (w.kb == 0 || valid % kStep == 0) continue;
      const int stage = blocks == 0 ? nstages - 1 : blocks - 1;
      if (!__all_sync(0xFFFFFFFFu, mbar_await(&landed[stage], (phases >> stage) & 1u, p.status, abort_flag))) break;
      phases ^= 1u << stage;
      clear_rows(smem + stage * stage_bytes, kPair ? 2 : 1 + (w.cols + 127) / 128, valid,
                 (valid + kStep - 1) / kStep * kStep, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair) mbar_arrive_remote(mapa_shared(smem_u32(&cleared[stage]), 0));
        else mbar_arrive(&cleared[stage]);
      }
    }
  } else if (warp >= 2) {
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
    // Two warps (64 lanes of the tile) share a slab of [32 columns][128 bytes],
    // 128-byte swizzle, so that a TMA store writes whole 128-byte lines: with a
    // warp's 64-byte rows alone the store engine bounded tiles of few k-blocks.
    const int duo = half * 2 + (qd >> 1);     // which two warps
    const bool issuer = (qd & 1) == 0;        // of the two: its lane 0 issues the stores
    uint8_t* const slabs = s_epi + duo * 2 * kSlab;
    const int chunk0 = (qd & 1) * 4;          // this warp's 16-byte chunks of a row: chunk0 .. chunk0 + 3
    // stmatrix: this lane's 16 bytes of column (8 i + lane % 8), block lane / 8
    const uint32_t st_off = (lane & 7) * 128 + (((chunk0 + (lane >> 3)) ^ (lane & 7)) * 16);
    int slab = 0;
    int held_e = -1;                          // fp8: the group whose factor is held
    float held_f = 0.0f;
    int acc = 0;
    uint32_t acc_phase = 0;
    auto hand_back = [&](int a) {  // this warp is done with accumulator a
      if (lane == 0) {
        if constexpr (kPair) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tempty[a]), 0));
        else mbar_arrive(&tempty[a]);
      }
    };
    for (Tiles at(p, unit, units); at.t < tiles; at.advance(p)) {
      const Tile w = tile_at(at);
      const int n0 = w.lane0 + rank * kLanes + qd * 32;       // first output column of this warp
      const int steps = (w.cols + 31) / 32;
      // per-lane factors, fetched before the wait for the accumulator: this
      // thread's lanes are n0 + 8 j + lane / 4, j = 0..3
      float f[4], b[4];
      if constexpr (kInt8) {
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = n0 + 8 * j + (lane >> 2);
          f[j] = n < p.nlane && p.k_blocks > 0 ? p.scale_b[n] : 0.0f;
          b[j] = p.bias && n < p.nlane ? load_bias(p.bias, p.bias_dtype, n) : 0.0f;
        }
      } else {
        if (w.e != held_e) {
          held_e = w.e;
          held_f = 1.0f / (__ldcg(p.scale_a) * __ldcg(p.scale_b + w.e * p.scale_b_step));
        }
        f[0] = (kRaggedK ? w.kb : p.k_blocks) > 0 ? held_f : 0.0f;
      }
      // The two warps of a slab leave together, here or below: one that gave up
      // alone, for a wait of its own or for the abort flag, would strand the
      // other at their next barrier.
      if (!duo_await(1 + duo, &tfull[acc], acc_phase, p.status, abort_flag)) break;
      tc_fence_after();
      if constexpr (kSplit) {
        if (part == 0) {
          if (ew == 0 && lane == 0)
            mbar_arrive_expect_tx(joined, static_cast<uint32_t>((p.split - 1) * steps * 32 * kLanes * 4));
          if (!duo_await(1 + duo, joined, 0, p.status, abort_flag)) break;
        }
      }
      uint8_t* const d = static_cast<uint8_t*>(p.d) +
                         (static_cast<int64_t>(w.e) * p.stride_d + static_cast<int64_t>(w.col0) * p.ldd) * (OUT == kFP32 ? 4 : 2);
      const uint32_t ta = tmem_base + (static_cast<uint32_t>(qd * 32) << 16) + static_cast<uint32_t>(acc * 256);
      uint32_t r[2][16];
      auto load_step = [&](int st) {   // asynchronous until tmem_ld_wait
        __syncwarp();
        tmem_ld_16x256b_x4(ta + st * 32, r[0]);
        tmem_ld_16x256b_x4(ta + (16u << 16) + st * 32, r[1]);
      };
      const bool have_k = w.kb > 0;
      if (half >= steps) {
        hand_back(acc);
      } else if (have_k) {
        load_step(half);
      } else {  // empty contraction: the MMA never wrote this accumulator
        #pragma unroll
        for (int i = 0; i < 16; ++i) r[0][i] = r[1][i] = 0u;
      }
      #pragma unroll 1
      for (int st = half; st < steps; st += 2) {
        if (have_k) tmem_ld_wait();
        if constexpr (kSplit) {
          // the other ranks' sums, from the same registers of their epilogue
          // threads, are added in rank order: the same result every time
          const int slot = (st * 4 + qd) * 8 * 512 + lane * 16;   // 8 x 16 bytes a thread, 512 bytes a warp
          if (part != 0) {
            const uint32_t to = mapa_shared(smem_u32(partials + (part - 1) * max(p.col_tile, 32) * kLanes * 4 + slot), 0);
            const uint32_t bar = mapa_shared(smem_u32(joined), 0);
            #pragma unroll
            for (int i = 0; i < 8; ++i)
              st_async_v4(to + i * 512, r[i >> 2][4 * (i & 3)], r[i >> 2][4 * (i & 3) + 1], r[i >> 2][4 * (i & 3) + 2],
                          r[i >> 2][4 * (i & 3) + 3], bar);
            if (st + 2 < steps && have_k) load_step(st + 2);
            continue;
          }
          for (int q = 1; q < p.split; ++q) {
            const uint8_t* from = partials + (q - 1) * max(p.col_tile, 32) * kLanes * 4 + slot;
            #pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 x = *reinterpret_cast<const uint4*>(from + i * 512);
              uint32_t* v = &r[i >> 2][4 * (i & 3)];
              v[0] = add_sums<kInt8>(v[0], x.x);
              v[1] = add_sums<kInt8>(v[1], x.y);
              v[2] = add_sums<kInt8>(v[2], x.z);
              v[3] = add_sums<kInt8>(v[3], x.w);
            }
          }
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
              s[u] = c < live && p.k_blocks > 0 ? p.scale_a[w.col0 + c0 + c] : 0.0f;
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
              else if (q & 1)   // two at a time: the same roundings
                mul_x2(v[h][4 * i + q - 1], v[h][4 * i + q], __uint_as_float(r[h][4 * i + q - 1]), __uint_as_float(x), f[0]);
            }
        }
        uint32_t o[16];   // the block's packed pairs, in stmatrix order
        if constexpr (OUT != kFP32) {
          #pragma unroll
          for (int i = 0; i < 4; ++i)
            #pragma unroll
            for (int j = 0; j < 4; ++j)
              o[4 * i + j] = pack2<OUT>(v[j >> 1][4 * i + 2 * (j & 1)], v[j >> 1][4 * i + 2 * (j & 1) + 1]);
        }
        if (st + 2 >= steps) {  // this warp's last read of the accumulator
          tc_fence_before();
          __syncwarp();
          hand_back(acc);
        } else if (have_k) {    // the next step's values arrive while this one is stored
          load_step(st + 2);
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
          uint8_t* const buf = slabs + slab * kSlab;
          const uint32_t st_addr = smem_u32(buf) + st_off;
          #pragma unroll
          for (int i = 0; i < 4; ++i)
            stmatrix_x4_trans(st_addr + i * 8 * 128, o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          unsigned short* dh = reinterpret_cast<unsigned short*>(d);
          if (p.tma_store && (kRaggedK || live == 32)) {
            // A whole block, or one that ends where D does (the copy clips it).
            // Past the barrier the other slab is free too: the store that read
            // it was waited for first.
            fence_proxy_async_smem();
            if (issuer && lane == 0) bulk_wait_read<0>();
            duo_sync(1 + duo);
            if (issuer && lane == 0) {
              if (n0 < p.nlane) tma_store_3d(&t_d, buf, n0, w.col0 + c0, kRaggedK ? w.e : 0);
              bulk_commit();
            }
          } else {
            // a block that ends with its group: guarded stores of this warp's part
            if (issuer && lane == 0) bulk_wait_read<0>();
            duo_sync(1 + duo);
            if (p.vec_ok) {
              const int q = lane & 3, n = n0 + q * 8, c1 = lane >> 2;
              unsigned short* dst = dh + static_cast<int64_t>(c0 + c1) * p.ldd + n;
              const int64_t pitch = 8 * p.ldd;
              const uint8_t* from = buf + c1 * 128 + (((chunk0 + q) ^ c1) * 16);   // columns c1, c1 + 8, ...
              if (n + 8 <= p.nlane) {
                #pragma unroll
                for (int it = 0; it < 4; ++it)
                  if (c1 + 8 * it < live) *reinterpret_cast<uint4*>(dst + it * pitch) = *reinterpret_cast<const uint4*>(from + it * 1024);
              } else {
                for (int it = 0; it < 4; ++it)
                  for (int j = 0; j < 8; ++j)
                    if (c1 + 8 * it < live && n + j < p.nlane)
                      dst[it * pitch + j] = *reinterpret_cast<const unsigned short*>(from + it * 1024 + j * 2);
              }
            } else {
              // Rows that 16-byte stores cannot address.  Each of the two
              // warps takes every other column, all 64 lanes of it, so that
              // its rows start alike -- at an even address or an odd one --
              // whatever the row pitch: 4-byte stores from the first even
              // address on, the two odd ends of all its rows in one more.
              const int nd = n0 - (qd & 1) * 32, left = p.nlane - nd;   // the slab's first lane, lanes from there
              unsigned short* const dst = dh + static_cast<int64_t>(c0 + (qd & 1)) * p.ldd + nd;
              const int64_t pitch = 2 * p.ldd;
              const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(dst) >> 1) & 1;
              const int row0 = qd & 1, rows = (live + 1 - row0) >> 1;   // this warp's columns: row0, row0 + 2, ...
              const int end = min(left, 64);
              auto at = [&](int c, int j) { return c * 128 + (((j >> 3) ^ (c & 7)) * 16) + (j & 7) * 2; };
              const int j = 2 * lane + shift, j1 = min(j + 1, 63);
              const bool pair = j + 1 < end;
              // the swizzle repeats every eight columns, this warp's four
              int off[4], off1[4];
              #pragma unroll
              for (int i = 0; i < 4; ++i) off[i] = at(2 * i + row0, j), off1[i] = at(2 * i + row0, j1);
              // all rows' pairs, then their stores: no store waits for a load
              // (eight rows at a time took 1.15 times as long)
              uint32_t x[16];
              if (shift) {
                #pragma unroll
                for (int i = 0; i < 16; ++i)
                  x[i] = static_cast<uint32_t>(*reinterpret_cast<const unsigned short*>(buf + off[i & 3] + (i >> 2) * 1024)) |
                         static_cast<uint32_t>(*reinterpret_cast<const unsigned short*>(buf + off1[i & 3] + (i >> 2) * 1024)) << 16;
              } else {
                #pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = *reinterpret_cast<const uint32_t*>(buf + off[i & 3] + (i >> 2) * 1024);
              }
              unsigned short* to = dst + j;
              if (rows == 16) {
                if (pair) {
                  #pragma unroll
                  for (int i = 0; i < 16; ++i, to += pitch) *reinterpret_cast<uint32_t*>(to) = x[i];
                }
              } else {
                #pragma unroll
                for (int i = 0; i < 16; ++i, to += pitch)
                  if (pair && i < rows) *reinterpret_cast<uint32_t*>(to) = x[i];
              }
              // the odd ends, a lane each: rows' first elements by lanes 0-15, their
              // last ones by lanes 16-31 (loaded before the stores they cost more than that hid)
              const int je = lane < 16 ? 0 : end - 1, row = lane & 15;
              const bool odd = lane < 16 ? shift != 0 : ((end - shift) & 1) != 0;
              if (odd && row < rows && end > (lane < 16 ? 0 : shift))
                dst[row * pitch + je] = *reinterpret_cast<const unsigned short*>(buf + at(2 * row + row0, je));
            }
            __syncwarp();
          }
          slab ^= 1;
        }
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    // the copies' global writes complete on their own; the CTA only has to
    // outlive their reads of its shared memory
    if (lane == 0) bulk_wait_read<0>();
  }

  if (p.late_wait) pdl_wait();
  tc_fence_before();
  if constexpr (kPair || kSplit) cluster_sync();  // no CTA leaves while another still signals or writes it
  else cta_sync();
  if (threadIdx.x == 0) settle_copies(abort_flag);
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if constexpr (kPair) tmem_dealloc_pair(tmem_base, kTmemCols);
    else tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <bool kInt8, bool kRaggedK, bool kPair, bool kSplit, int OUT>
cudaError_t launch_build(const CUtensorMap* maps, const GroupedParams& p, int64_t max_tiles, int dev, int sms,
                         cudaStream_t s) {
  static std::atomic<int> capacity[64];   // CTAs (pairs) that can be resident at once; 0: not yet configured
  auto kernel = grouped_kernel<kInt8, kRaggedK, kPair, kSplit, OUT>;
  const int per_unit = kPair ? 2 : (kSplit ? p.split : 1);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kRaggedK ? kThreadsRaggedK : kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(per_unit);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  if (!capacity[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e != cudaSuccess) return e;
    int fit = sms;
    if (kPair) {
      cfg.gridDim = dim3(2 * (sms / 2));
      cfg.dynamicSmemBytes = kSmemMax;
      cfg.attrs = attr + 1;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
      if (e != cudaSuccess) return e;
    }
    if (fit <= 0) return cudaErrorInvalidConfiguration;
    capacity[dev] = fit;
  }
  // a split launch has a cluster for every tile there can be: each runs one
  const int64_t units = kSplit ? max_tiles : std::min<int64_t>(capacity[dev].load(), max_tiles);
  cfg.gridDim = dim3(static_cast<unsigned>(std::max<int64_t>(1, units) * per_unit));
  cfg.dynamicSmemBytes = static_cast<size_t>(p.smem_bytes);
  cfg.attrs = attr;
  cfg.numAttrs = kPair || kSplit ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps[0], maps[1], maps[2], maps[3], maps[4], p);
}

template <bool kInt8, int OUT>
cudaError_t launch_tokens(const CUtensorMap* maps, const GroupedParams& p, bool pair, int64_t max_tiles, int dev,
                          int sms, cudaStream_t s) {
  if (pair) return launch_build<kInt8, false, true, false, OUT>(maps, p, max_tiles, dev, sms, s);
  if (p.split > 1) return launch_build<kInt8, false, false, true, OUT>(maps, p, max_tiles, dev, sms, s);
  return launch_build<kInt8, false, false, false, OUT>(maps, p, max_tiles, dev, sms, s);
}

}  // namespace

void grouped_smem(GroupedParams* p, bool pair) {
  const int cols = std::max(pair ? p->col_tile / 2 : p->col_tile, 32);
  const int stage = kLaneBytes + cols * kKBlock;
  int fixed = kFixedSmem + 2 * (p->groups + 1) * 4;
  if (p->split > 1) fixed += 16 + (p->split - 1) * std::max(p->col_tile, 32) * kLanes * 4;
  p->stages = std::min({kMaxStages, kOperandBytes / stage, (kSmemMax - fixed) / stage});
  p->smem_bytes = fixed + p->stages * stage;
}

cudaError_t launch_grouped(const CUtensorMap* maps, const GroupedParams& p, bool int8, bool ragged_k, bool pair,
                           int out_dtype, int64_t max_tiles, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int sms = num_sms(dev);
  if (sms <= 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (ragged_k)
    return pair ? launch_build<false, true, true, false, kBF16>(maps, p, max_tiles, dev, sms, s)
                : launch_build<false, true, false, false, kBF16>(maps, p, max_tiles, dev, sms, s);
  if (!int8) return launch_tokens<false, kBF16>(maps, p, pair, max_tiles, dev, sms, s);
  if (out_dtype == kFP32) return launch_tokens<true, kFP32>(maps, p, pair, max_tiles, dev, sms, s);
  if (out_dtype == kFP16) return launch_tokens<true, kFP16>(maps, p, pair, max_tiles, dev, sms, s);
  return launch_tokens<true, kBF16>(maps, p, pair, max_tiles, dev, sms, s);
}

}  // namespace fp8lin
