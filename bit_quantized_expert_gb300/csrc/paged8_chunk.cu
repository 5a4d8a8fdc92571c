// Attention of chunks of new tokens over the paged cache held in 8 bits (contract in include/gqa_paged8.h), on the
// fifth-generation tensor cores.
//
// Rows, row tiles, items, the split of the work, tensor memory and the order of the products are those of the 16-bit
// form (paged_chunk.cu).  What differs:
//
//   * Operands.  The tensor cores take e4m3 beside e4m3 alone, and queries and numerators need more bits than that, so codes
//     become fp16 on their way into shared memory: four warps (12 to 15) bring them there by asynchronous copies, a tile of
//     keys or of values ahead, convert them and store them in the operands' swizzle.
//   * Scales and pages.  One warp (11) reads them, up to four tiles ahead, and leaves in a ring what the others need of a tile:
//     where its blocks are, and each block's scale over a reference, by which its codes are multiplied as they are
//     converted.  The reference is for keys the tile's largest scale, for values the largest that the segment has met.  Both
//     are powers of two, and a code times 2^-15 or more is still an fp16 value, so nothing is rounded.  The softmax
//     sees one factor a tile, and O is in units of the values' reference.
//   * Wide tiles.  A reference may be a scale that only some of the rows see, and a factor below 2^-15 would take bits from what
//     the others see.  Codes of a tile with such a factor, or behind values so far apart that O in fp32 might lose them,
//     are left unscaled; the softmax goes on from there in a form of its own (far_tiles8), in which each
//     block's key scale multiplies its scores, its value scale the numerators, relative to the largest that the row itself
//     sees, and O is in units of that.
//   * Queries.  bf16 ones are scaled by a power of two a row so that fp16 holds them: by the softmax threads, a row each, in
//     shared memory before the item's first product.
//   * Values of masked tiles.  NaN ones are taken out of the operand once it is there, by warps 8 and 10, so that 0 * NaN does
//     not reach rows that do not see them; rows that do get their NaN back at the end.
//   * Registers.  184 a thread for the softmax, 64 for the issuing warpgroup, 80 for the converting one.
//
// What bounds it: the chain of a row tile, softmax, P V, next scores, as in the 16-bit form, whose softmax here shares its
// issue slots with the conversion (58 % of them are taken, the tensor pipe is active 64 % of the time, 75 % in the 16-bit
// form).  Measured in a graph: 2048 tokens at 32768 positions (16 / 2 heads of 128, bf16) 385 us, 1.47 PFLOP/s, 77 % of the
// dense rate (the 16-bit form of the same shape: 344); heads of 64 313; 34 sequences of single tokens and chunks (fp16)
// 80.2; 16 prompts 21.7; 4096 tokens with a window of 1024 69.8; 512 tokens of one prompt 19.3.  Where a wide tile is among the
// first: 2048 tokens 810 us (keys) and 1041 (values), the 34 sequences 138 and 172.
//
// Steps at 2048 tokens: 1131 us with codes through registers; 607 by asynchronous copies; 536 a block's codes at once; 505 by
// four warps of their own; 434 with scales that are powers of two and multiply the codes as they are converted, not scores
// and numerators in the softmax; 391 with NaN codes taken out by two other warps, scales read by a third, and short
// waits; 381 with the pages there as well (385 since wide tiles have a form of their own).  Not kept: codes brought by
// tensor map (1030 us by one warp, 620 by the converting ones), or through registers (spills); unrolled conversion (25 %
// more: its instructions displace the softmax's); NaN codes looked for in global memory ahead of the conversion (16
// prompts 22.4: four loads' latency a tile, where every tile is masked); a barrier of its own for a tile's places, so that
// its copies do not wait for its scales (16 prompts 21.0, 2048 tokens 389).
#include <cmath>
#include <cstring>

#include "paged8.cuh"
#include "paged_chunk.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;               // two softmax warpgroups, one for queries, scales and products, one for codes
constexpr int kScanWarps = 2;
constexpr int kConvertWarps = 4;
constexpr int kFirstConvert = 12;
// Registers a thread: 128 at launch; 2 * 184 + 64 + 80 = 4 * 128 after the split.
constexpr int kRegsSoftmax = 184, kRegsIssue = 64, kRegsConvert = 80;
static_assert(2 * kRegsSoftmax + kRegsIssue + kRegsConvert <= 4 * 128, "no more than at launch");
// Base-2 units by which the numerators' reference may lag behind the row's maximum, and by which it stands
// below the maximum that sets it: fp16's range from 2^15 down.
constexpr float kLazy = 6.f, kLift = 9.f;
// Base-2 units from which on a row's reference is taken off its scaled scores apart (far_tiles8).
constexpr float kFar = 65536.f;
constexpr int kInfos = 8;                   // slots for tiles' scales, a power of two
// The least factor that takes no bits from a code (the least code is 2^-9, the least fp16 value 2^-24), and the least ratio of a
// segment's value scales at which O moves to the larger unit without losing any (it has 2^9 and fp32's 2^-126).
constexpr float kLeastFactor = 0x1p-15f, kLeastRatio = 0x1p-64f;

template <int D>
struct Chunk8 {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kTN * 128;                  // 128 rows of 64 dims
  static constexpr int kTileBytes = kBoxes * kBoxBytes;        // a row tile of q, a tile of keys or of values
  // Ring: a segment of n tiles takes n + 1 stages, the i-th with the values of its tile i - 1 and the keys of tile i.
  static constexpr int kStages = 2;
  static constexpr int kStageBytes = 2 * kTileBytes;           // keys, then values
  static constexpr int kPartFloats = kItemRows * (D + 2);
  static constexpr int kRawBytes = kTN * D;                    // codes on their way, a tile of keys or of values
  // (The schedule's sums lie where the ring will be.)
  static constexpr int kSmem = 1024 + (2 + 2 * kStages) * kTileBytes + kSoftmaxWarps * kOutBytes + kRawBytes;
  static_assert((kPagedMaxSeqs + 1) * 4 <= kStages * kStageBytes, "sums fit");
};

// Waits for the phase of `parity`, the warp together; false: it gave up.  What a wait that runs out needs is elsewhere (walk):
// with the clock and the abort word looked at here, as in mbar_wait, the instructions of every wait are fetched beside the
// softmax's, and 2048 tokens at 32768 take 460 us in place of 404 (with a time limit given to the instruction itself 395 in
// place of 384).
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) {
  return mbar_wait_warp_tries(bar, parity, kWaitTries);
}

// What is known of a tile before its codes: the factors of its blocks as pairs of fp16 values, where the blocks start in the
// caches (-1: taken as zeros), the references that the factors are over, and whether it is its segment's last tile, or
// none (behind the share's last one).  In a wide tile the factors are 1, v_ref is negative, and the blocks' scales count, as
// their exponents of fp32.
constexpr uint32_t kLastTile = 1u, kNoTile = 2u;
struct __align__(16) TileInfo {
  uint32_t k_by[8], v_by[8];
  long long at[8];
  float k_ref, v_ref;
  uint32_t last;
  uint16_t exps[8];   // keys' in the low byte, values' in the high one
};

__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// N times `bytes` (16, or none: zeros) of global memory, `step` apart, into shared memory, 512 bytes apart, asynchronously.
// In one statement, so that every address has registers of its own: one that is stepped on waits until the copy before
// has left its queue (which took 190 cycles a copy behind the stores).
template <int N>
__device__ __forceinline__ void cp_async_pieces(uint32_t dst, const uint8_t* src, long long step, int bytes) {
  static_assert(N == 2 || N == 4, "pieces of a block");
  if constexpr (N == 4)
    asm volatile(
        "cp.async.cg.shared.global [%0], [%1], 16, %5;\n\tcp.async.cg.shared.global [%0+512], [%2], 16, %5;\n\t"
        "cp.async.cg.shared.global [%0+1024], [%3], 16, %5;\n\tcp.async.cg.shared.global [%0+1536], [%4], 16, %5;" ::"r"(dst),
        "l"(src), "l"(src + step), "l"(src + 2 * step), "l"(src + 3 * step), "r"(bytes)
        : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %3;\n\tcp.async.cg.shared.global [%0+512], [%2], 16, %3;" ::"r"(dst),
                 "l"(src), "l"(src + step), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A power of two of at most 1 as the factor of a pair of fp16 values.
__device__ __forceinline__ uint32_t factor(float by) { return pack16<true>(by, by); }
// The power of two with this exponent of fp32.
__device__ __forceinline__ float power(uint32_t exponent) { return __uint_as_float(exponent << 23); }

// This lane's codes of one block (16 bytes in each piece, 512 bytes apart at `in`) as fp16 values times `by` (factor) into the
// operand at `out`.
template <int D>
__device__ __forceinline__ void convert_block(uint32_t in, uint32_t out, uint32_t by) {
  constexpr int kRows = 512 / D, kPieces = 16 / kRows;
  uint32_t c[kPieces][4], h[kPieces][8];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) ld_shared4(in + k * 512, c[k][0], c[k][1], c[k][2], c[k][3]);
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) codes_to_half4(c[k][e], h[k][2 * e], h[k][2 * e + 1]);
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) h[k][e] = mul_half2(h[k][e], by);
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    // (rows 4 and 8 apart differ by one bit of the chunk in the swizzle, and not at all)
    const uint32_t to = (D == 128 && k & 1 ? out ^ 64u : out) + k * kRows * 128;
    st_shared16(to, h[k][0], h[k][1], h[k][2], h[k][3]);
    st_shared16(to ^ 16u, h[k][4], h[k][5], h[k][6], h[k][7]);
  }
}
// The first eight words of v to 8 consecutive columns of this thread's row.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// NaN for the dims d0 .. d0 + 15 in which a position that the row sees, in this segment's masked tiles, has a NaN code.
__device__ __noinline__ uint32_t nan_dims(const Paged8Args& a, const int32_t* table, TileRange r, int i0, int n, int p_lo,
                                          int p_hi, int p, int g, int d0) {
  uint32_t dims = 0;
  for (int i = i0; i < i0 + n; ++i) {
    const int j0 = r.tile(i) * kTN;
    if (tile_open<kTN>(a, j0, p_lo, p_hi)) continue;
    for (int j = j0; j < j0 + kTN; ++j) {
      if (!paged_sees(a, p, j)) continue;
      const int page = table[j >> a.page_shift];
      if (page < 0 || page >= a.num_pages) continue;
      const uint4 c = __ldcg(reinterpret_cast<const uint4*>(a.vc8 + page * a.page_stride + g * a.head_stride +
                                                            (j & ((1 << a.page_shift) - 1)) * a.row_stride + d0));
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      for (int e = 0; e < 16; ++e)
        if ((w[e / 4] >> (8 * (e % 4)) & 0x7Fu) == 0x7Fu) dims |= 1u << e;
    }
  }
  return dims;
}

// The least unit in which O of this thread's row, now in units of `unit`, stays below 2^60.  (What a row sees sets its unit in a
// wide tile, and the tiles before may have had a larger one for other rows' sake.)
template <int D>
__device__ __forceinline__ float least_unit(uint32_t tO, float unit) {
  float top = 0.f;
  __syncwarp();
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t v[16];
    tmem_ld16_wait(tO + c, v);
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(__uint_as_float(v[e])));
  }
  const int down = min(max(60 + 126 - (int)(__float_as_uint(top) >> 23), 0), 120);   // top < 2^(exponent - 126)
  return fmaxf(unit * power(127 - down), kLeastScale);
}
// Softmax of tiles i .. n - 1 of a segment (the first one's scores are there, masked) for a warp with a row beyond kFar, or from a
// wide tile on: scaled scores are rounded before the reference is taken off, a block at a time.  done < 0: a wait timed out.
// (v_ref: the row's unit of O.)
struct FarRow {
  float m, l, v_ref;
  int done, tiles;
};
template <int D>
__device__ __noinline__ FarRow far_tiles8(const Paged8Args& a, Item x, int i0, int i, int n, int p, uint32_t tS, uint32_t tO,
                                          uint32_t sfull, uint32_t pfull, const TileInfo* infos, float q_scale,
                                          FarRow row) {
  float m = row.m, l = row.l, v_ref = row.v_ref;
  int done = row.done, tiles = row.tiles;
  for (bool waited = true; i < n; ++i, waited = false) {
    if (!waited) {
      const int j0 = x.r.tile(i0 + i) * kTN;
      if (!wait_warp(sfull, done & 1)) return FarRow{m, l, v_ref, -1, tiles};
      ++done;
      ++tiles;
      tc_fence_after();
      if (!tile_open<kTN>(a, j0, x.p_lo, x.p_hi)) mask_scores(a, tS, p, j0);
    }
    const volatile TileInfo* ts = infos + ((tiles - 1) & (kInfos - 1));
    const float k = ts->k_ref * q_scale, v_tile = ts->v_ref;
    const bool wide = v_tile < 0.f;
    float v_new = v_tile;   // the unit of O
    if (wide) {
      v_new = i > 0 ? least_unit<D>(tO, v_ref) : kLeastScale;
#pragma unroll 1
      for (int blk = 0; blk < 8; ++blk) {
        const int j = x.r.tile(i0 + i) * kTN + 16 * blk;
        if (j <= p && (a.window == 0 || j + 15 > p - a.window || j < a.sinks)) v_new = fmaxf(v_new, power(ts->exps[blk] >> 8));
      }
    }
    auto k_of = [&](int blk) { return wide ? power(ts->exps[blk] & 0xFFu) * q_scale : k; };
    auto v_of = [&](int blk) { return wide ? power(ts->exps[blk] >> 8) / v_new : 1.f; };
    float mx = -INFINITY, by = 1.f, sum = 0.f;
    __syncwarp();
#pragma unroll 1
    for (int blk = 0; blk < 8; ++blk) {
      uint32_t v[16];
      float top = -INFINITY;
      tmem_ld16_wait(tS + 16 * blk, v);
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, __uint_as_float(v[e]));
      mx = fmaxf(mx, top * k_of(blk));
    }
    if (mx > m && (m == -INFINITY || mx - m > kLazy)) {
      by = ex2(m - mx);   // 0 if nothing was seen before
      m = mx;
      l *= by;
    }
    by *= v_ref / v_new;
    v_ref = v_new;
    const float ref = m == -INFINITY ? 0.f : m;
    __syncwarp();
    if (i > 0) rescale<D>(tO, by);
    // (numerators of a block take the place of scores that have been read)
#pragma unroll 1
    for (int blk = 0; blk < 8; ++blk) {
      const float k_blk = k_of(blk), v_blk = v_of(blk);
      uint32_t v[16];
      tmem_ld16_wait(tS + 16 * blk, v);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float p0 = ex2((__fmul_rn(__uint_as_float(v[e]), k_blk) - ref) + kLift);
        const float p1 = ex2((__fmul_rn(__uint_as_float(v[e + 1]), k_blk) - ref) + kLift);
        sum += p0 + p1;
        v[e / 2] = pack16<true>(p0 * v_blk, p1 * v_blk);
      }
      tmem_st8(tS + 8 * blk, v);
      if ((blk & 3) == 3) {
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(pfull + 8u * (blk / 4));
        __syncwarp();
      }
    }
    l += sum;
  }
  return FarRow{m, l, v_ref, done, tiles};
}

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads, 1)
    chunk8_kernel(const __grid_constant__ CUtensorMap q_map, const Paged8Args a, const ChunkSplit split) {
  using C = Chunk8<D>;
  extern __shared__ uint8_t sm_raw[];
  // barriers: stages (full, empty), q empty, per row tile q full, q converted, S full, P full (its first and its second
  // half), O full, O empty; scales (full, empty, a slot each); values clean (a stage each)
  __shared__ __align__(8) uint64_t bars[2 * C::kStages + 1 + 14 + 2 * kInfos + C::kStages];
  __shared__ __align__(16) TileInfo infos_s[kInfos];
  __shared__ uint32_t warp_s[kThreads / 32];
  __shared__ Share share_s;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  __shared__ int bad_s[4];   // segment + 1 whose values had NaN codes that a row sees
  const uint32_t raw = smem_u32(sm_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t sQ = base, sKV = base + 2 * C::kTileBytes;
  const uint32_t sOut = sKV + C::kStages * C::kStageBytes;
  const uint32_t sRaw = sOut + kSoftmaxWarps * kOutBytes;
  uint32_t* pre_s = reinterpret_cast<uint32_t*>(sm_raw + (sKV - raw));
  const uint32_t bar0 = smem_u32(bars);
  auto FULL = [&](int s) { return bar0 + 8u * s; };
  auto EMPTY = [&](int s) { return bar0 + 8u * (C::kStages + s); };
  constexpr int kB = 2 * C::kStages;
  const uint32_t QEMPTY = bar0 + 8u * kB;
  auto QFULL = [&](int t) { return bar0 + 8u * (kB + 1 + t); };
  auto QREADY = [&](int t) { return bar0 + 8u * (kB + 3 + t); };
  auto SFULL = [&](int t) { return bar0 + 8u * (kB + 5 + t); };
  auto PFULL = [&](int t, int part) { return bar0 + 8u * (kB + 7 + 2 * t + part); };
  auto OFULL = [&](int t) { return bar0 + 8u * (kB + 11 + t); };
  auto OEMPTY = [&](int t) { return bar0 + 8u * (kB + 13 + t); };
  auto INFO = [&](int s) { return bar0 + 8u * (kB + 15 + s); };
  auto INFOEMPTY = [&](int s) { return bar0 + 8u * (kB + 15 + kInfos + s); };
  auto CLEAN = [&](int s) { return bar0 + 8u * (kB + 15 + 2 * kInfos + s); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = (int)blockIdx.x;
  const int tpt = 128 / a.G, tokens = 2 * tpt;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(FULL(s), kConvertWarps);
      mbar_init(EMPTY(s), 1 + kScanWarps);
      mbar_init(CLEAN(s), kScanWarps);
    }
    mbar_init(QEMPTY, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(QFULL(t), 1);
      mbar_init(SFULL(t), 1);
      mbar_init(PFULL(t, 0), 4);
      mbar_init(PFULL(t, 1), 4);
      mbar_init(OFULL(t), 1);
      mbar_init(OEMPTY(t), 4);
      mbar_init(QREADY(t), 4);
    }
    for (int s = 0; s < kInfos; ++s) {
      mbar_init(INFO(s), 1);
      mbar_init(INFOEMPTY(s), kConvertWarps);
    }
    abort_s = 0;
    for (int i = 0; i < 4; ++i) bad_s[i] = 0;
    share_s.lo = share_s.hi = 0;
    mbar_fence_init();
    prefetch_tmap(&q_map);
  }
  if (warp == kSoftmaxWarps + 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();

  bool bad = false;
  find_share<kThreads>(a, tokens, pre_s, warp_s, &share_s, bad);
  if (bad && cta == 0) raise_flag(a.err, kErrBadPages);
  if (tid == 0) split.rec[cta].until = split.rec[cta].first = -1;
  // Lanes part ways in the schedule (and below, wherever a lane's own data decides).  Every such place ends in
  // __syncwarp before the warp's next collective instruction.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // Walks the segments of the share: body(b, s, g, item, i0, n, u) for tiles i0 .. i0 + n - 1 of an item,
  // the first of them unit u; stops when the body returns false.  (The others' waits then run out as well.)
  auto walk = [&](auto&& body) {
    uint32_t u = share_s.lo, at = share_s.at;
    const uint32_t hi = share_s.hi;
    int b = share_s.b, qt = share_s.qt;
    while (u < hi) {
      const SeqRows s = load_seq(a, b, bad);
      for (; u < hi && qt * tokens < s.n; ++qt) {
        const Item x = item_of(a, s, qt, tokens);
        const uint32_t units = (uint32_t)x.r.count + kItemUnits;
        for (int g = 0; g < a.Hkv && u < hi; ++g, at += units) {
          if (at + units <= u) continue;
          const int i0 = max((int)(u - at) - kItemUnits, 0), i1 = (int)min(hi - at, units) - kItemUnits;
          if (!body(b, s, g, x, i0, i1 - i0, u)) {   // a wait gave up
            abort_s = 1;
            return;
          }
          u = min(hi, at + units);
        }
      }
      qt = 0;
      ++b;
    }
  };
  // The page of block lane & 7 of tile i + lane / 8 of a segment, as the table has it (looked at by page_or_none, later,
  // so that nothing waits here), and -1 in the place of one whose block no row needs.
  auto read_page = [&](const int32_t* row, const Item& x, int i0, int n, int i, bool* need) {
    const int t = i0 + i + (lane >> 3);
    const int j = i + (lane >> 3) < n && t < x.r.count ? x.r.tile(t) * kTN + (lane & 7) * 16 : -1;
    *need = j >= 0 && j <= x.p_hi && (a.window == 0 || j + 15 > x.p_lo - a.window || j < a.sinks);
    int page = -1;
    if (*need) page = row[j >> a.page_shift];
    __syncwarp();
    return page;
  };
  auto page_or_none = [&](int page, bool need) {
    const bool ok = page >= 0 && page < a.num_pages;
    bad |= need && !ok;
    return ok ? page : -1;
  };

  if (warp >= kSoftmaxWarps && warp < kFirstConvert) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == kSoftmaxWarps || warp == kSoftmaxWarps + 2) {
      // ---- queries (warp 8), once the segment before has done its last scores; and values of masked tiles (both warps, two
      // positions a thread): NaN ones are taken out of the operand.  In the conversion itself, where all tiles come by, that
      // code took a quarter of its time without being run (2048 tokens at 32768: 522 in place of 407 us).
      // These warps see every stage, and a stage is free only with their word, so that they keep step with the ring.
      // Their word that a tile is done goes to its stage's own barrier: a stage is filled again only after both of them and
      // the product have left it.
      const int w = warp == kSoftmaxWarps ? 0 : 1;
      uint32_t at = 0, items = 0;
      int seg = 0;
      walk([&](int, const SeqRows& s, int g, const Item& x, int i0, int n, uint32_t) {
        if (w == 0) {
          if (items > 0 && !wait_warp(QEMPTY, (items - 1) & 1)) return false;
          ++items;
          if (lane == 0) {
            const uint32_t bytes = (uint32_t)(64 * 2 * a.G * tpt);
            for (int t = 0; t < (x.n > tpt ? 2 : 1); ++t) {
              mbar_arrive_expect_tx(QFULL(t), bytes * C::kBoxes);
              for (int bx = 0; bx < C::kBoxes; ++bx)
                tma_load_3d(sQ + t * C::kTileBytes + bx * C::kBoxBytes, &q_map, QFULL(t), bx * 64, g * a.G, s.row0 + x.t0 + t * tpt);
            }
          }
          __syncwarp();
        }
        for (int i = 0; i <= n; ++i, ++at) {
          const uint32_t st = at & 1;
          if (!wait_warp(FULL(st), (at >> 1) & 1)) return false;
          const int j0 = i > 0 ? x.r.tile(i0 + i - 1) * kTN : 0;
          if (i > 0 && !tile_open<kTN>(a, j0, x.p_lo, x.p_hi)) {
#pragma unroll 1
            for (int r = w * 32 + lane; r < kTN; r += kScanWarps * 32) {
              const uint32_t row = sKV + st * C::kStageBytes + C::kTileBytes + r * 128;
              uint32_t any = 0;
#pragma unroll 8
              for (int c = 0; c < 8 * C::kBoxes; ++c) {   // of 16 bytes; lanes start at different ones
                uint32_t w0, w1, w2, w3;
                ld_shared4(row + (c >> 3) * C::kBoxBytes + (((c + lane) & 7) << 4), w0, w1, w2, w3);
                any |= non_finite_bits<true>(w0) | non_finite_bits<true>(w1) | non_finite_bits<true>(w2) | non_finite_bits<true>(w3);
              }
              if (any & kSigns) {
#pragma unroll 1
                for (int c = 0; c < 8 * C::kBoxes; ++c) {
                  const uint32_t to = row + (c >> 3) * C::kBoxBytes + ((c & 7) << 4);
                  uint32_t v[4];
                  ld_shared4(to, v[0], v[1], v[2], v[3]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) v[e] &= ~(((non_finite_bits<true>(v[e]) & kSigns) >> 15) * 0xFFFFu);
                  st_shared16(to, v[0], v[1], v[2], v[3]);
                }
                const int j = j0 + r;
                if (j <= x.p_hi && (a.window == 0 || j > x.p_lo - a.window || j < a.sinks)) bad_s[seg & 3] = seg + 1;
                fence_proxy_async_smem();
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(CLEAN(st));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(EMPTY(st));
          __syncwarp();
        }
        ++seg;
        return true;
      });
    } else if (warp == kSoftmaxWarps + 1) {
      // ---- tensor-core instructions.  The whole warp takes every step, one elected lane issues (by predicate), and
      // row tile and ring stage are constants of the unrolled code.
      const uint32_t go = elect_one() ? 1u : 0u;
      constexpr uint32_t id_s = (1u << 4) | ((kTN >> 3) << 17) | ((128u >> 4) << 24);
      constexpr uint32_t id_o = (1u << 4) | (1u << 16) | (((uint32_t)D >> 3) << 17) | ((128u >> 4) << 24);
      constexpr uint32_t kTileUnits = C::kTileBytes >> 4, kBoxUnits = C::kBoxBytes >> 4;   // descriptors count 16 bytes
      const uint64_t dq = smem_desc_sw128(sQ), dk = smem_desc_sw128(sKV), dv = desc_values(sKV + C::kTileBytes, C::kBoxBytes);
      uint32_t at = 0, items = 0, cleans[2] = {0, 0}, seconds = 0, done0 = 0, done1 = 0, outs0 = 0, outs1 = 0;
      auto wait = [&](uint32_t bar, uint32_t phase) { return wait_warp(bar, phase & 1); };
      // S_t = Q_t K^T with the keys of stage ST
      auto scores = [&](auto t_c, auto st_c) {
        constexpr int t = decltype(t_c)::value, ST = decltype(st_c)::value;
#pragma unroll
        for (int box = 0; box < C::kBoxes; ++box)
          tc_mma4_ss(go, t * 128, dq + (t * kTileUnits + box * kBoxUnits), dk + (ST * 2 * kTileUnits + box * kBoxUnits), id_s,
                     box != 0);
        tc_commit_if(go, SFULL(t));
      };
      // O_t (+)= P_t V, P in two halves, with the values of stage ST; then the next tile's scores
      auto turn = [&](auto t_c, auto st_c, uint32_t done, bool first, bool more) {
        constexpr int t = decltype(t_c)::value, ST = decltype(st_c)::value;
        const uint64_t v = dv + ST * 2 * kTileUnits;
        if (!wait(PFULL(t, 0), done)) return false;
        tc_fence_after();
        tc_mma4_ts(go, kTmemO + t * 128, t * 128, v, id_o, !first);
        if (!wait(PFULL(t, 1), done)) return false;
        tc_fence_after();
        tc_mma4_ts(go, kTmemO + t * 128, t * 128 + 32, v + (8192u >> 4), id_o, 1u);
        if (more) scores(t_c, st_c);
        else tc_commit_if(go, OFULL(t));
        return true;
      };
      using Zero = std::integral_constant<int, 0>;
      using One = std::integral_constant<int, 1>;
      // body(stage as a constant) for the stage of a tile
      static_assert(C::kStages == 2, "a tile's stage is its parity");
      auto at_stage = [&](uint32_t tile, auto&& body) { return tile & 1 ? body(One{}) : body(Zero{}); };
      walk([&](int, const SeqRows&, int, const Item& x, int i0, int n_any, uint32_t) {
        const int n = __shfl_sync(0xFFFFFFFFu, n_any, 0);
        const bool two = __shfl_sync(0xFFFFFFFFu, (int)(x.n > tpt), 0) != 0;
        if (!wait(FP16 ? QFULL(0) : QREADY(0), items++)) return false;
        if (two && !wait(FP16 ? QFULL(1) : QREADY(1), seconds++)) return false;
        if (!at_stage(at, [&](auto st_c) {
              constexpr int ST = decltype(st_c)::value;
              if (!wait(FULL(ST), at >> 1)) return false;
              tc_fence_after();
              scores(Zero{}, st_c);
              if (two) scores(One{}, st_c);
              tc_commit_if(go, EMPTY(ST));
              if (n == 1) tc_commit_if(go, QEMPTY);
              return true;
            }))
          return false;
        ++at;
        for (int i = 0; i < n; ++i, ++at) {
          const bool more = i + 1 < n, closed = !tile_open<kTN>(a, x.r.tile(i0 + i) * kTN, x.p_lo, x.p_hi);
          if (!at_stage(at, [&](auto st_c) {   // the tile's values, the next one's keys
                constexpr int ST = decltype(st_c)::value;
                if (!wait(FULL(ST), at >> 1)) return false;
                if (closed && !wait(CLEAN(ST), cleans[ST]++)) return false;
                // (the second row tile's result too, where this item has none: bad_s is a short ring)
                if (i == 0 && outs0 > 0 && !wait(OEMPTY(0), outs0 - 1)) return false;
                if (i == 0 && outs1 > 0 && !wait(OEMPTY(1), outs1 - 1)) return false;
                if (!turn(Zero{}, st_c, done0++, i == 0, more)) return false;
                if (two) {
                  if (!turn(One{}, st_c, done1++, i == 0, more)) return false;
                }
                tc_commit_if(go, EMPTY(ST));
                if (i + 2 == n) tc_commit_if(go, QEMPTY);
                return true;
              }))
            return false;
        }
        ++outs0;
        outs1 += two;
        return true;
      });
    } else {
      // ---- scales of blocks, four tiles at a time, read two tiles ahead.  A block that no row needs, or whose
      // page is bad, has the least scale.
      uint32_t tiles = 0;
      bool ended = true;
      bad = false;
      // The slot was last used eight tiles ago.  Once the values of four tiles ago have been converted, the products of six
      // tiles ago are done, and with them the softmax of those before, which had its references from there.
      auto next_info = [&]() -> TileInfo* {
        if (tiles >= 4 && !wait_warp(INFOEMPTY((tiles - 4) & (kInfos - 1)), ((tiles - 4) / kInfos) & 1)) {
          ended = false;
          return nullptr;
        }
        return infos_s + (tiles & (kInfos - 1));
      };
      walk([&](int b, const SeqRows&, int g, const Item& x, int i0, int n, uint32_t) {
        const int32_t* row = a.table + (size_t)b * a.max_pages;
        const int my_off = ((lane & 7) * 16) & ((1 << a.page_shift) - 1);   // of the block in its page
        bool need;
        int pg_ahead = read_page(row, x, i0, n, 0, &need);
        float ks_ahead = kLeastScale, vs_ahead = kLeastScale, k_ref = 1.f, v_ref = kLeastScale, v_last = kLeastScale;
        float v_least = kMostScale;   // the segment's least value scale
        long long from_ahead = -1, from = -1;
        uint32_t k_by = 0u, v_by = 0u, exps = 0u;
        auto read_scales = [&]() {
          const int page = page_or_none(pg_ahead, need), index = scale_index(max(page, 0), a.Hkv, g, a.page_shift, my_off);
          ks_ahead = vs_ahead = kLeastScale;
          from_ahead = -1;
          if (page >= 0) {
            from_ahead = page * a.page_stride + g * a.head_stride + my_off * a.row_stride;
            ks_ahead = a.ks[index];
            vs_ahead = a.vs[index];
          }
          __syncwarp();
        };
        read_scales();
        for (int i = 0; i < n; ++i, ++tiles) {
          if ((i & 3) == 0) {
            const float ks = scale_ok(ks_ahead) ? ks_ahead : kLeastScale, vs = scale_ok(vs_ahead) ? vs_ahead : kLeastScale;
            bad |= !scale_ok(ks_ahead) || !scale_ok(vs_ahead);
            __syncwarp();
            from = from_ahead;
            k_ref = ks;
            float top = vs, least = from >= 0 ? vs : kMostScale;
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) {
              k_ref = fmaxf(k_ref, __shfl_xor_sync(0xFFFFFFFFu, k_ref, off));
              top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
              least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, off));
            }
            v_ref = v_last;   // of this lane's tile: the largest so far
            float v_low = v_least;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const float y = __shfl_sync(0xFFFFFFFFu, top, 8 * t), z = __shfl_sync(0xFFFFFFFFu, least, 8 * t);
              v_last = fmaxf(v_last, y);
              v_least = fminf(v_least, z);
              if (t <= lane >> 3) {
                v_ref = fmaxf(v_ref, y);
                v_low = fminf(v_low, z);
              }
            }
            // (blocks that are taken as zeros lose nothing)
            const bool lost = (from >= 0 && (ks < k_ref * kLeastFactor || vs < v_ref * kLeastFactor)) || v_low < v_ref * kLeastRatio;
            const bool wide = (__ballot_sync(0xFFFFFFFFu, lost) >> (lane & 24) & 0xFFu) != 0u;
            k_by = factor(wide ? 1.f : ks / k_ref);
            v_by = factor(wide ? 1.f : vs / v_ref);
            v_ref = wide ? -v_ref : v_ref;
            exps = __float_as_uint(ks) >> 23 | __float_as_uint(vs) >> 23 << 8;
            pg_ahead = read_page(row, x, i0, n, i + 4, &need);
          }
          if ((i & 3) == 2) read_scales();
          TileInfo* to = next_info();
          if (to == nullptr) return false;
          if (lane >> 3 == (i & 3)) {
            to->k_by[lane & 7] = k_by;
            to->v_by[lane & 7] = v_by;
            to->at[lane & 7] = from;
            to->exps[lane & 7] = (uint16_t)exps;
            if ((lane & 7) == 0) {
              to->last = i + 1 == n ? kLastTile : 0u;
              to->k_ref = k_ref;
              to->v_ref = v_ref;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(INFO(tiles & (kInfos - 1)));
          __syncwarp();
        }
        return true;
      });
      if (ended) {
        TileInfo* to = next_info();
        if (to != nullptr) {
          if (lane < 8) to->at[lane] = -1;
          if (lane == 0) to->last = kNoTile;
          __syncwarp();
          if (lane == 0) mbar_arrive(INFO(tiles & (kInfos - 1)));
        } else {
          abort_s = 1;
        }
      }
      if (bad) raise_flag(a.err, kErrBadPages);
    }
  } else if (warp >= kFirstConvert) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
    // ---- codes into operands: a warp has 32 of the tile's positions, two blocks; a lane has 16 bytes of a row, and the
    // warp kRows rows (a piece) at a time.
    constexpr int kRows = 512 / D, kPerBlock = 16 / kRows;
    const int w = warp - kFirstConvert;
    // A lane's dims 16 q .. and its row of a piece; eight lanes in a row have two rows of one box of 64 dims, so that what
    // they store lies in different banks.  Pieces come by asynchronous copies, each lane's own 16 bytes by itself, so that
    // nothing but its own count of copies stands between them and their use.
    const int q = D == 128 ? (lane & 3) | (lane >> 4) << 2 : lane & 3, rr = D == 128 ? (lane >> 2) & 3 : lane >> 2;
    const uint32_t mine = sRaw + w * 32 * D + lane * 16;
    const uint32_t line = (q >> 2) * C::kBoxBytes + (w * 32 + rr) * 128 + ((((2 * q) & 7) ^ rr) << 4);
    const long long step = kRows * a.row_stride, lane_off = rr * a.row_stride + q * 16;
    const uint32_t infos = smem_u32(infos_s);
    long long from0 = -1, from1 = -1;   // this warp's two blocks of the tile whose copies go out
    uint32_t last = kNoTile;            // of the tile that is converted
    auto read_info = [&](uint32_t tile) {
      const uint32_t info = infos + (tile & (kInfos - 1)) * (uint32_t)sizeof(TileInfo);
      uint32_t word;
      asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(from0), "=l"(from1) : "r"(info + 64 + w * 16) : "memory");
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(word) : "r"(info + 136) : "memory");
      return word;
    };
    // A block of a cache on its way to its place, which this lane has read: one group of copies.
    auto fetch = [&](const uint8_t* cache, long long from, int blk) {
      const bool go = from >= 0;
      cp_async_pieces<kPerBlock>(mine + blk * kPerBlock * 512, go ? cache + from + lane_off : cache, go ? step : 0, go ? 16 : 0);
      cp_async_commit();
    };
    // Keys and values of one tile after another, whatever segment it is of.  A stage has the values of a tile and the
    // keys of the next one, or only one of them at a segment's ends.  By the same instructions, a block a turn (what is
    // unrolled is fetched anew each time, beside the softmax's instructions, and that takes longer than it does); behind
    // keys come the values of their tile, behind values the keys of the next.
    uint32_t at = 0, tile = 0, kv = 0;
    bool fresh = true, ok = wait_warp(INFO(0), 0);
    if (ok) last = read_info(0);
#pragma unroll 1
    for (int blk = 0; blk < 2; ++blk) fetch(a.kc8, blk == 0 ? from0 : from1, blk);
    while (last != kNoTile) {
      const uint32_t st = at & 1;
      if (fresh && at >= C::kStages && !wait_warp(EMPTY(st), (at / C::kStages - 1) & 1)) {
        ok = false;
        break;
      }
      uint32_t to = sKV + st * C::kStageBytes + kv * C::kTileBytes + line, in = mine;
      uint32_t by0, by1, next = last;
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                   : "=r"(by0), "=r"(by1)
                   : "r"(infos + (tile & (kInfos - 1)) * (uint32_t)sizeof(TileInfo) + kv * 32 + w * 8)
                   : "memory");
      if (kv != 0) {
        if (!wait_warp(INFO((tile + 1) & (kInfos - 1)), ((tile + 1) / kInfos) & 1)) {
          ok = false;
          break;
        }
        next = read_info(tile + 1);
      }
#pragma unroll 1
      for (int blk = 0; blk < 2; ++blk) {
        cp_async_wait<1>();   // the older of two blocks
        convert_block<D>(in, to, blk == 0 ? by0 : by1);
        fetch(kv != 0 ? a.kc8 : a.vc8, blk == 0 ? from0 : from1, blk);
        to += 16 * 128;
        in += kPerBlock * 512;
      }
      fresh = kv == 0 || last != 0u;
      if (fresh) {
        fence_proxy_async_smem();
        ++at;
      }
      __syncwarp();
      if (lane == 0) {
        if (fresh) mbar_arrive(FULL(st));
        if (kv != 0) mbar_arrive(INFOEMPTY(tile & (kInfos - 1)));
      }
      __syncwarp();
      tile += kv;
      last = next;
      kv ^= 1u;
    }
    if (!ok) abort_s = 1;
  } else {
    // ---- softmax: row `r` of row tile `t`
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, r = (warp & 3) * 32 + lane, tok = r / a.G, head = r - tok * a.G;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = t * 128 + lanes, tO = kTmemO + t * 128 + lanes;
    int seg = 0, done = 0, outs = 0, tiles = 0;   // segments, own tiles, items and all tiles so far
    walk([&](int b, const SeqRows& s, int g, const Item& x, int i0, int n, uint32_t u) {
      const int nt = x.n > tpt ? 2 : 1;
      if (t >= nt) {
        ++seg;
        tiles += n;
        return true;
      }
      const bool live = tok < tpt && t * tpt + tok < x.n;
      const int p = live ? x.p_lo + t * tpt + tok : -1;      // a row that is no token sees nothing
      float q_scale = a.qk_scale;
      if (!FP16) {
        // bf16 times the power of two that brings the row's largest to 2^14 .. 2^15: exact down to 2^-24, and so within 2^-39 of the
        // largest, or 2^-105.  (At most 2^80, so that a scale of the scores is never 0, which would undo a mask.)
        if (!wait_warp(QFULL(t), outs & 1)) return false;
        const uint32_t line = sQ + t * C::kTileBytes + r * 128;
        uint32_t w[D / 2];
#pragma unroll
        for (int e = 0; e < D / 8; ++e)
          ld_shared4(line + (e >> 3) * C::kBoxBytes + (((e & 7) ^ (r & 7)) << 4), w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < D / 2; ++e) top = max(top, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
        const int E = (int)(top >> 7), e2 = E == 255 ? 0 : min(max(E - 141, -80), 60);
        const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
        q_scale *= __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
        for (int e = 0; e < D / 2; ++e) {
          const float2 f = unpack16<false>(w[e]);
          w[e] = pack16<true>(f.x * down, f.y * down);
        }
#pragma unroll
        for (int e = 0; e < D / 8; ++e)
          st_shared16(line + (e >> 3) * C::kBoxBytes + (((e & 7) ^ (r & 7)) << 4), w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(QREADY(t));
        __syncwarp();
      }
      float m = -INFINITY, negm = 0.f, l = 0.f, v_ref = kLeastScale;   // negm = kLift - m (0 while nothing is seen)
      for (int i = 0; i < n; ++i) {
        const int j0 = x.r.tile(i0 + i) * kTN;
        const bool open = tile_open<kTN>(a, j0, x.p_lo, x.p_hi);
        if (!wait_warp(SFULL(t), done & 1)) return false;
        ++done;
        tc_fence_after();
        const volatile TileInfo* ts = infos_s + (tiles & (kInfos - 1));
        ++tiles;
        if (!open) mask_scores(a, tS, p, j0);
        uint32_t sr[128];
        tmem_ld128(tS, sr);
        const float k = ts->k_ref * q_scale, v_new = ts->v_ref;
        float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
          mx0 = max3(mx0, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
          mx1 = max3(mx1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
          mx2 = max3(mx2, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
          mx3 = max3(mx3, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
        }
        const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * k;
        // The reference moves if the new maximum is well above it (or is the first).  (A wide tile, whose v_ref is negative and
        // whose scores are not what they seem here, comes by the same condition.)
        const bool move = mx > m && (m == -INFINITY || mx - m > kLazy);
        if (__any_sync(0xFFFFFFFFu, move || v_new != v_ref)) {
          if (__any_sync(0xFFFFFFFFu, v_new < 0.f || (move && p >= 0 && fabsf(mx) > kFar))) {   // from here on in another way
            const FarRow row = far_tiles8<D>(a, x, i0, i, n, p, tS, tO, SFULL(t), PFULL(t, 0), infos_s, q_scale,
                                             FarRow{m, l, v_ref, done, tiles});
            if (row.done < 0) return false;
            m = row.m;
            l = row.l;
            v_ref = row.v_ref;
            done = row.done;
            tiles = row.tiles;
            negm = kLift - m;
            break;
          }
          float by = v_ref / v_new;
          v_ref = v_new;
          if (move) {
            const float alpha = m == -INFINITY ? 0.f : ex2(m - mx);
            m = mx;
            negm = kLift - mx;
            l *= alpha;
            by *= alpha;
          }
          __syncwarp();
          if (i > 0) rescale<D>(tO, by);
        }
        const uint64_t scale2 = pair2(k, k), negm2 = pair2(negm, negm);
        uint64_t sum0 = 0, sum1 = 0;   // two fp32 sums each
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float2 x0 = unpair2(fma2(pair2(__uint_as_float(sr[c + e]), __uint_as_float(sr[c + e + 1])), scale2, negm2));
            const float2 x1 = unpair2(fma2(pair2(__uint_as_float(sr[c + e + 2]), __uint_as_float(sr[c + e + 3])), scale2, negm2));
            const float p0 = ex2(x0.x), p1 = ex2(x0.y), p2 = ex2(x1.x), p3 = ex2(x1.y);
            sum0 = add2(sum0, pair2(p0, p1));
            sum1 = add2(sum1, pair2(p2, p3));
            pk[e / 2] = pack16<true>(p0, p1);
            pk[e / 2 + 1] = pack16<true>(p2, p3);
          }
          tmem_st16(tS + c / 2, pk);
          if (c == 32 || c == 96) {   // half of P is there: its part of the product can start
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(PFULL(t, c / 64));
            __syncwarp();
          }
        }
        const float2 s0 = unpair2(sum0), s1 = unpair2(sum1);
        l += (s0.x + s0.y) + (s1.x + s1.y);
      }
      // ---- the item's result, or this share's part of it
      const int my_seg = seg++;
      if (!wait_warp(OFULL(t), outs & 1)) return false;
      ++outs;
      tc_fence_after();
      const bool whole = i0 == 0 && n == x.r.count;
      if (*(volatile int*)&bad_s[my_seg & 3] == my_seg + 1) {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t v[16];
          tmem_ld16_wait(tO + c, v);
          const uint32_t nan =
              live ? nan_dims(a, a.table + (size_t)b * a.max_pages, x.r, i0, n, x.p_lo, x.p_hi, p, g, c) : 0u;
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = nan & (1u << e) ? 0x7FC00000u : v[e];
          tmem_st16(tO + c, v);
          tmem_wait_st();
        }
      }
      __syncwarp();
      // (O of a row that sees nothing is 0: its tiles are masked.)
      const float inv = whole ? (p < 0 ? 0.f : v_ref / l) : v_ref;
      // Rows of the result are stored by four lanes each: lane 4 i + j stores bytes 16 j of rows i, i + 8, ...
      unsigned long long to[4];
      {
        const unsigned long long orow =
            live ? reinterpret_cast<unsigned long long>(a.o + (long long)(s.row0 + x.t0 + t * tpt + tok) * a.o_stride +
                                                        (long long)(g * a.G + head) * D)
                 : 0ull;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          to[k] = __shfl_sync(0xFFFFFFFFu, orow, k * 8 + (lane >> 2));
          if (to[k] != 0) to[k] += (lane & 3) * 16;
        }
      }
      float* part = split.part + ((size_t)cta * 2 + (i0 == 0 ? 1 : 0)) * C::kPartFloats + 4 * (t * 128 + r);
      const uint32_t out = sOut + warp * kOutBytes;
      const uint64_t inv2 = pair2(inv, inv);
      uint32_t not_finite = 0;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        tmem_ld32(tO + c, v);
        if (whole) {
#pragma unroll
          for (int e = 0; e < 16; e += 2) {   // pairs 2 e, 2 e + 2 become words e, e + 1
            const uint64_t f0 = mul2(pair2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), inv2);
            const uint64_t f1 = mul2(pair2(__uint_as_float(v[2 * e + 2]), __uint_as_float(v[2 * e + 3])), inv2);
            const float2 y0 = unpair2(f0), y1 = unpair2(f1);
            v[e] = pack16<FP16>(y0.x, y0.y);
            v[e + 1] = pack16<FP16>(y1.x, y1.y);
            not_finite |= non_finite_bits<FP16>(v[e]) | non_finite_bits<FP16>(v[e + 1]);
          }
          // 64 bytes a row through shared memory (16-byte pieces XOR-ed against bank conflicts), so that a store
          // touches 8 rows, not 32.
#pragma unroll
          for (int e = 0; e < 4; ++e)
            st_shared16(out + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4), v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          __syncwarp();
          uint4 w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int rr = k * 8 + (lane >> 2);
            ld_shared4(out + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4), w[k].x, w[k].y, w[k].z, w[k].w);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (to[k] != 0) *reinterpret_cast<uint4*>(to[k] + 2 * c) = w[k];
        } else if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(part + (c + e) * kItemRows) =
                make_float4(__uint_as_float(v[e]) * inv, __uint_as_float(v[e + 1]) * inv, __uint_as_float(v[e + 2]) * inv,
                            __uint_as_float(v[e + 3]) * inv);
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(OEMPTY(t));
      if (live && (not_finite & kSigns)) raise_flag(a.err, kErrNonFinite);
      if (!whole) {
        if (live) {
          float* stats = part + D * kItemRows - 3 * (t * 128 + r);
          stats[0] = m == -INFINITY ? kUnseen : -negm;
          stats[kItemRows] = l;
        }
        if (i0 + n < x.r.count && tid == 0) {   // the item goes on: who begins it, and who ends it
          const uint32_t first = i0 == 0 ? u : u - kItemUnits - i0, end = first + x.r.count + kItemUnits;
          const uint32_t total = share_s.total;
          const int ctas = share_s.ctas;
          auto cut_at = [&](int c) { return snap(share_start(total, c, ctas), first, end, kItemUnits, share_s.slack); };
          int c = share_of(i0 == 0 ? end - 1 : first, total, ctas);
          if (i0 == 0) {
            while (c > cta + 1 && cut_at(c) >= end) --c;
            split.rec[cta] = SplitRecord{s.row0 + x.t0, g, x.n, x.p_lo, c, cta};
          } else {
            while (c + 1 < cta && cut_at(c + 1) <= first) ++c;
            split.rec[cta].first = c;
          }
        }
      }
      __syncwarp();
      return true;
    });
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // After a timeout, copies and products still in flight finish before the CTA gives up its memory.
  if (warp == kSoftmaxWarps + 1 && *(volatile int*)&abort_s) {
    if (lane == 0) raise_flag(a.err, kErrWaitTimeout);
    const long long c0 = clock64();
    while (clock64() - c0 < 4000000ll) {
    }
    __syncwarp();
  }
  if (warp == kSoftmaxWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem_slot, 512);
  }
}

template <int D, bool FP16>
cudaError_t launch(const CUtensorMap& q_map, const Paged8Args& a, const ChunkSplit& split, int ctas, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(chunk8_kernel<D, FP16>), Chunk8<D>::kSmem, &ready);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Chunk8<D>::kSmem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, chunk8_kernel<D, FP16>, q_map, a, split);
  return e == cudaSuccess ? launch_paged_chunk_join(a, D, split, ctas, st) : e;
}

}  // namespace

cudaError_t launch_paged8_chunk(const gqa_paged_dims& d, const Paged8Args& a, void* scratch, int ctas, cudaStream_t st) {
  CUtensorMap q_map;
  std::memset(&q_map, 0, sizeof(q_map));
  if (!encode_queries(&q_map, a.q, d)) return cudaErrorInvalidValue;
  const int D = d.head_dim;
  const ChunkSplit split = paged_chunk_split(D, scratch, ctas);
  if (D == 128) return a.fp16 ? launch<128, true>(q_map, a, split, ctas, st) : launch<128, false>(q_map, a, split, ctas, st);
  return a.fp16 ? launch<64, true>(q_map, a, split, ctas, st) : launch<64, false>(q_map, a, split, ctas, st);
}

}  // namespace moe
