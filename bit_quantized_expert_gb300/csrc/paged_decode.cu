// Single-token attention over the paged cache (contract in include/gqa_paged.h): every sequence has at most
// one new token, so the work is one pass over the visible cache, bound by HBM.
//
//   * the cache is walked in tiles of 64 positions; an item is one key/value head of one sequence, and all
//     its query heads (up to eight) share the tile, so a cached byte is read once;
//   * the tiles of all items, in order, are cut into equal shares, one per CTA and one CTA per SM: one long
//     sequence is spread over every SM and a batch of very different lengths is balanced by construction
//     (see paged.cuh); a share may hold the end of one item, several whole ones and the start of another;
//   * four warps copy the tile's pages by tensor map into a ring (a page of the table is a box of
//     16 to 64 rows), 32 page numbers at a time read ahead by their lanes; eight consumer warps take tiles
//     in turn (four warps a tile, 16 positions a warp) with m16n8k16 products: S = Q K^T with the heads as
//     the 16-row operand (rows 8..15 zero), then O += P V with rows 0..7 the rounded numerators and rows
//     8..15 their rounding remainders, so P keeps about twice the type's bits;
//   * all rows stand at one position and see the same set, so positions that they do not see are cut out
//     of the value operand itself: whatever lies there, non-finite values included, has no effect;
//   * running max, sum and O stay in registers; at an item's end the eight warps are joined in shared
//     memory in a fixed order (one barrier an item: two joining buffers, every thread weighs for
//     itself), and the result goes to o, or, for an item that other CTAs share, to a partial that a
//     second launch joins in order.
//
// Measured (16 query and 2 key/value heads of 128, in a graph, no cache in L2): 64 sequences of 1 to 32768 positions, 139
// MB, 28.7 us (4.8 TB/s), of which ~5 us are fixed steps: launch, schedule, first copies, joins; one sequence of 32768,
// 33.6 MB, 14.0 us (10.5 with its cache in L2); 64 sequences with heads of 64, 69.5 MB, 18.2 us.  tcgen05
// would not help: eight heads fill an eighth of its 64-row tiles, and bytes bound the rest.
#include <cmath>
#include <type_traits>

#include "paged.cuh"

namespace moe {
namespace {

constexpr int kTN = 64;                        // positions per tile
constexpr int kWarps = 8;                      // consumer warps: two groups of four, alternate tiles
constexpr int kCopyWarps = 4;
constexpr int kThreads = (kWarps + kCopyWarps) * 32;
constexpr int kRows = 8;                       // query heads per key/value head, at most
constexpr int kItemUnits = 3;                  // what an item costs beside its tiles, in tiles (~3500 cycles)
constexpr int kSlack = 1;                      // tiles that a cut moves to reach an item's end
// Base-2 units by which numerators stand above e^(s - max): fp16 keeps 2^-25 at best, so they use its range
// from 2^15 down, or a long cache of small ones would be summed as nothing.  (All parts of an item are
// scaled alike, so the joins do not see it.)  bf16 has fp32's range.
template <bool FP16>
constexpr float kLift = FP16 ? 15.f : 0.f;

template <int D>
struct Dec {
  static constexpr int kBoxes = D / 64;                  // 64-dim boxes of a row
  static constexpr int kBoxBytes = kTN * 128;
  static constexpr int kStageBytes = 2 * kBoxes * kBoxBytes;
  static constexpr int kStages = 128 * 1024 / kStageBytes;
  static constexpr int kOStride = D + 8;                 // padded row of the joining buffer (floats)
  static constexpr int kJoinFloats = kWarps * kRows * kOStride;
  static constexpr int kJoinBytes = 2 * kJoinFloats * 4; // two buffers: an item's is read while the next one's is written
  static constexpr int kPartFloats = kRows * D + 2 * kRows;
  static size_t smem(int B) { return 1024 + (size_t)kStages * kStageBytes + kJoinBytes + ((size_t)B + 1) * 4; }
};

template <bool FP16>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  if (FP16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr)
               : "memory");
}

// Byte offset of 16-byte chunk `chunk` (8 dims) of row `pos` in a tile of 64-dim boxes written by the
// tensor map's 128-byte swizzle.
__device__ __forceinline__ uint32_t swz(int pos, int chunk) {
  return (uint32_t)((chunk >> 3) * (kTN * 128) + pos * 128 + (((chunk & 7) ^ (pos & 7)) << 4));
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ PagedMaps maps, const PagedArgs a, const DecodeSplit split) {
  using C = Dec<D>;
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages];
  __shared__ __align__(16) float ml_s[2][kRows][2][kWarps];   // per buffer and row: the warps' max, then sum
  __shared__ uint32_t warp_s[kThreads / 32];
  __shared__ int abort_s;
  const uint32_t raw = smem_u32(sm_raw), base = (raw + 1023u) & ~1023u;
  float* join_s = reinterpret_cast<float*>(sm_raw + (base - raw) + C::kStages * C::kStageBytes);
  uint32_t* pre_s = reinterpret_cast<uint32_t*>(sm_raw + (base - raw) + C::kStages * C::kStageBytes + C::kJoinBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = (int)blockIdx.x;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), kCopyWarps);
      mbar_init(smem_u32(&empty[s]), 4);
    }
    abort_s = 0;
    mbar_fence_init();
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's share: units lo .. hi - 1 of (sequence, head, tile); pre_s: units before each sequence
  bool bad = false;
  auto cost = [&](int b) {
    const SeqRows s = load_seq(a, b, bad);
    return s.n == 0 ? 0ull : (unsigned long long)(visible_tiles<kTN>(a, s.p0, s.p0).count + kItemUnits) * a.Hkv;
  };
  bool over;
  uint32_t total = scan_sequences<kThreads>(a.B, pre_s, warp_s, &over, cost);
  if (over) {   // refused: nothing is computed
    bad = true;
    total = 0;
  }
  if (bad && cta == 0) raise_flag(a.err, kErrBadPages);
  const int ctas = (int)min(gridDim.x, total);   // every share holds a tile
  if (tid == 0) split.rec[cta].until = -1;
  if (cta >= ctas) return;
  // Its two cuts, by the even lanes and the odd ones of every warp.
  uint32_t lo, hi;
  int b_first;   // the sequence that holds unit lo
  {
    uint32_t x = share_start(total, cta + (lane & 1), ctas);
    const int b = find_sequence(pre_s, a.B, x);
    if (x < total) {
      const uint32_t units = (pre_s[b + 1] - pre_s[b]) / a.Hkv, first = x - (x - pre_s[b]) % units;
      x = snap(x, first, first + units, kItemUnits, kSlack);
    }
    __syncwarp();
    lo = __shfl_sync(0xFFFFFFFFu, x, 0);
    hi = __shfl_sync(0xFFFFFFFFu, x, 1);
    b_first = __shfl_sync(0xFFFFFFFFu, b, 0);
  }

  if (warp >= kWarps) {
    // ---- copies: every warp takes a quarter of a tile's boxes, since the copies of a warp's lanes are issued
    // one by one (75 to 120 cycles each: 16 of them, the boxes of pages of 16, took as long as a tile's
    // stream from memory).
    const int pw = warp - kWarps;
    const int ppt_shift = max(0, 6 - a.page_shift), ppt = 1 << ppt_shift;   // pages of a tile
    const int box_rows = min(kTN, 1 << a.page_shift);
    const int copies = ppt * 2 * C::kBoxes;                    // (page, keys or values, 64-dim box)
    const int c0 = copies * pw / kCopyWarps, mine = copies * (pw + 1) / kCopyWarps - c0;
    const int sub = (c0 + lane) / (2 * C::kBoxes), kv = ((c0 + lane) / C::kBoxes) & 1, box = (c0 + lane) % C::kBoxes;
    const int batch = 32 >> ppt_shift;                         // tiles whose page numbers the lanes hold
    int b = b_first, issued = 0;
    bool stop = false;
    bad = false;
    for (uint32_t u = lo; u < hi && !stop; ++b) {
      if (pre_s[b + 1] <= u) continue;
      const SeqRows s = load_seq(a, b, bad);
      const TileRange r = visible_tiles<kTN>(a, s.p0, s.p0);
      const int32_t* row = a.table + (size_t)b * a.max_pages;
      const uint32_t end = min(pre_s[b + 1], hi);
      while (u < end && !stop) {
        const uint32_t units = r.count + kItemUnits, g = (u - pre_s[b]) / units, first = pre_s[b] + g * units;
        const int i0 = max((int)(u - first) - kItemUnits, 0), n = (int)min(end - first, units) - kItemUnits - i0;
        // Page numbers of a batch of tiles, one a lane, read one batch ahead; a page that the token does not need
        // is not read, and takes, like a bad one, a number out of the map's range, which reads as zeros.
        int pg = 0, ahead = 0;
        bool need = false;
        auto read_ahead = [&](int i) {
          const int t = i0 + i + (lane >> ppt_shift);
          const int ip = t < r.count ? ((r.tile(t) * kTN) >> a.page_shift) + (lane & (ppt - 1)) : 0;
          need = (lane >> ppt_shift) < n - i && t < r.count && ip < a.max_pages && page_needed(a, ip, s.p0, s.p0);
          if (need) ahead = row[ip];
        };
        read_ahead(0);
        for (int i = 0; i < n; ++i) {
          const int in = i & (batch - 1);
          if (in == 0) {
            const bool ok = ahead >= 0 && ahead < a.num_pages;
            pg = need && ok ? ahead : a.num_pages;
            bad |= need && !ok;
            read_ahead(i + batch);
          }
          const int st = issued % C::kStages;
          if (issued >= C::kStages &&
              !mbar_wait_warp(smem_u32(&empty[st]), ((issued / C::kStages) - 1) & 1, &abort_s, a.err)) {
            stop = true;
            break;
          }
          const uint32_t bar = smem_u32(&full[st]);
          const int off = (r.tile(i0 + i) * kTN) & ((1 << a.page_shift) - 1);   // 64 in the second half of a page of 128
          if (lane == 0) mbar_arrive_expect_tx(bar, mine * box_rows * 128);
          __syncwarp();
          const int p = __shfl_sync(0xFFFFFFFFu, pg, (in * ppt + sub) & 31);
          if (lane < mine)
            tma_load_4d(base + st * C::kStageBytes + (kv * C::kBoxes + box) * C::kBoxBytes + sub * box_rows * 128,
                        kv ? &maps.v : &maps.k, bar, box * 64, off, (int)g, p);
          __syncwarp();
          ++issued;
        }
        u = min(end, first + units);
      }
    }
    if (bad) raise_flag(a.err, kErrBadPages);
    // After a timeout, copies still in flight land before the CTA exits.
    if (stop && lane == 0) {
      const long long t0 = clock64();
      while (clock64() - t0 < 4000000ll) {
      }
    }
    return;
  }

  // ---- consumers.  Every warp walks every segment; after a timeout the waits fail at once and the walk
  // goes on without data, so that the barriers still match.
  const int wg = warp >> 2, wq = warp & 3;
  const int r = lane >> 2, c2 = (lane & 3) * 2;
  const int lrow = lane & 7, lmat = lane >> 3;
  const int kpos = wq * 16 + 8 * (lmat >> 1) + lrow;   // key row this lane addresses
  const int vpos = wq * 16 + 8 * (lmat & 1) + lrow;    // value row this lane addresses

  // The segment at unit u: tiles i0 .. i0 + n - 1 of head g of sequence b (n = 0: the share is done).
  struct Segment {
    int g, i0, n, p0, row0;
    uint32_t first, end;   // the item's first unit and the unit past its last
    TileRange r;
  };
  uint32_t u = lo;
  int b = b_first;
  auto next_segment = [&]() {
    Segment x;
    x.n = 0;
    if (u >= hi) return x;
    while (pre_s[b + 1] <= u) ++b;
    const SeqRows s = load_seq(a, b, bad);
    x.r = visible_tiles<kTN>(a, s.p0, s.p0);
    x.p0 = s.p0;
    x.row0 = s.row0;
    const uint32_t units = x.r.count + kItemUnits;
    x.g = (int)((u - pre_s[b]) / units);
    x.first = pre_s[b] + x.g * units;
    x.end = x.first + units;
    x.i0 = max((int)(u - x.first) - kItemUnits, 0);
    x.n = (int)min(hi - x.first, units) - kItemUnits - x.i0;
    u = min(hi, x.end);
    return x;
  };
  // The heads as the 16-row operand.  Rows past the group's heads repeat its first one: every row has sums of its own,
  // and theirs are not stored, so no value needs a look before the products do.
  uint32_t qa[D / 16][2];
  auto load_queries = [&](const Segment& x) {
    const uint32_t* qh = reinterpret_cast<const uint32_t*>(
        a.q + (x.n > 0 ? x.row0 * a.q_stride + (long long)(x.g * a.G + (r < a.G ? r : 0)) * D : 0) + c2);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qa[kk][0] = qh[8 * kk];
      qa[kk][1] = qh[8 * kk + 4];
    }
  };

  int it = 0, buf = 0;   // tiles of the share so far, joining buffer
  Segment x = next_segment();
  load_queries(x);
  while (x.n > 0) {
    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m_run = kUnseen, l_run = 0.f;
    for (int i = (it ^ wg) & 1; i < x.n; i += 2) {   // tile it + i of the share goes to group (it + i) & 1
      const int st = (it + i) % C::kStages;
      if (mbar_wait_warp(smem_u32(&full[st]), ((it + i) / C::kStages) & 1, &abort_s, a.err)) {
        const uint32_t sk = base + st * C::kStageBytes, sv = sk + C::kBoxes * C::kBoxBytes;
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          uint32_t b0, b1, b2, b3;
          ldsm4(sk + swz(kpos, 2 * kk + (lmat & 1)), b0, b1, b2, b3);
          mma16<FP16>(sc[0], qa[kk][0], 0u, qa[kk][1], 0u, b0, b1);
          mma16<FP16>(sc[1], qa[kk][0], 0u, qa[kk][1], 0u, b2, b3);
        }
        const int j0 = x.r.tile(x.i0 + i) * kTN;
        uint32_t keep0 = 0xFFFFFFFFu, keep1 = 0xFFFFFFFFu;   // value pairs that the token sees
        float s2[2][2] = {{sc[0][0] * a.qk_scale, sc[0][1] * a.qk_scale}, {sc[1][0] * a.qk_scale, sc[1][1] * a.qk_scale}};
        const bool open = tile_open<kTN>(a, j0, x.p0, x.p0);
        if (!open) {
          const int j = j0 + wq * 16 + c2;
          const bool v00 = paged_sees(a, x.p0, j), v01 = paged_sees(a, x.p0, j + 1);
          const bool v10 = paged_sees(a, x.p0, j + 8), v11 = paged_sees(a, x.p0, j + 9);
          s2[0][0] = v00 ? s2[0][0] : -INFINITY;
          s2[0][1] = v01 ? s2[0][1] : -INFINITY;
          s2[1][0] = v10 ? s2[1][0] : -INFINITY;
          s2[1][1] = v11 ? s2[1][1] : -INFINITY;
          keep0 = (v00 ? 0xFFFFu : 0u) | (v01 ? 0xFFFF0000u : 0u);
          keep1 = (v10 ? 0xFFFFu : 0u) | (v11 ? 0xFFFF0000u : 0u);
        }
        float mx = fmaxf(fmaxf(s2[0][0], s2[0][1]), fmaxf(s2[1][0], s2[1][1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        const float m_new = fmaxf(m_run, mx);
        const float alpha = ex2(m_run - m_new);
        m_run = m_new;
        float p[2][2];   // (lifted after the difference: a maximum of 2^24 or more less the lift would be rounded by up to 16)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) p[j][e] = ex2((s2[j][e] - m_new) + kLift<FP16>);
        l_run = l_run * alpha + ((p[0][0] + p[0][1]) + (p[1][0] + p[1][1]));
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][0] *= alpha;
          o[j][1] *= alpha;
          o[j][2] *= alpha;
          o[j][3] *= alpha;
        }
        const uint32_t a0 = pack16<FP16>(p[0][0], p[0][1]), a2 = pack16<FP16>(p[1][0], p[1][1]);
        const float2 t0 = unpack16<FP16>(a0), t2 = unpack16<FP16>(a2);
        const uint32_t a1 = pack16<FP16>(p[0][0] - t0.x, p[0][1] - t0.y);
        const uint32_t a3 = pack16<FP16>(p[1][0] - t2.x, p[1][1] - t2.y);
#pragma unroll
        for (int jj = 0; jj < D / 16; ++jj) {
          uint32_t b0, b1, b2, b3;
          ldsm4_t(sv + swz(vpos, 2 * jj + (lmat >> 1)), b0, b1, b2, b3);
          if (!open) {
            b0 &= keep0;
            b1 &= keep1;
            b2 &= keep0;
            b3 &= keep1;
          }
          mma16<FP16>(o[2 * jj], a0, a1, a2, a3, b0, b1);
          mma16<FP16>(o[2 * jj + 1], a0, a1, a2, a3, b2, b3);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
    }
    it += x.n;

    // ---- join the eight warps in order; the next segment's queries are on their way meanwhile
    l_run += __shfl_xor_sync(0xFFFFFFFFu, l_run, 1);
    l_run += __shfl_xor_sync(0xFFFFFFFFu, l_run, 2);
    if ((lane & 3) == 0) {
      ml_s[buf][r][0][warp] = m_run;
      ml_s[buf][r][1][warp] = l_run;
    }
    float* ow = join_s + buf * C::kJoinFloats + (warp * kRows + r) * C::kOStride + c2;
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
      *reinterpret_cast<float2*>(ow + 8 * j) = make_float2(o[j][0] + o[j][2], o[j][1] + o[j][3]);
    const Segment now = x;
    x = next_segment();
    load_queries(x);
    __syncwarp();
    consumers_sync();
    const bool whole = now.i0 == 0 && now.n == now.r.count;
    float* part = split.part + ((size_t)cta * 2 + (now.i0 == 0 ? 1 : 0)) * C::kPartFloats;
    for (int e = tid; e < a.G * (D / 4); e += kWarps * 32) {
      const int row = e / (D / 4), dim = (e % (D / 4)) * 4;
      float mw[kWarps], lw[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; w += 4) {
        const float4 m4 = *reinterpret_cast<const float4*>(&ml_s[buf][row][0][w]);
        const float4 l4 = *reinterpret_cast<const float4*>(&ml_s[buf][row][1][w]);
        mw[w] = m4.x, mw[w + 1] = m4.y, mw[w + 2] = m4.z, mw[w + 3] = m4.w;
        lw[w] = l4.x, lw[w + 1] = l4.y, lw[w + 2] = l4.z, lw[w + 3] = l4.w;
      }
      float M = mw[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) M = fmaxf(M, mw[w]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 v =
            *reinterpret_cast<const float4*>(join_s + buf * C::kJoinFloats + (w * kRows + row) * C::kOStride + dim);
        const float sw = ex2(mw[w] - M);
        acc.x += v.x * sw;
        acc.y += v.y * sw;
        acc.z += v.z * sw;
        acc.w += v.w * sw;
        L += lw[w] * sw;
      }
      if (whole) {
        const float inv = now.p0 < 0 ? 0.f : 1.f / L;
        const float4 v = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (!isfinite(v.x) || !isfinite(v.y) || !isfinite(v.z) || !isfinite(v.w)) raise_flag(a.err, kErrNonFinite);
        *reinterpret_cast<uint2*>(a.o + now.row0 * a.o_stride + (long long)(now.g * a.G + row) * D + dim) =
            make_uint2(pack16<FP16>(v.x, v.y), pack16<FP16>(v.z, v.w));
      } else {
        *reinterpret_cast<float4*>(part + row * D + dim) = acc;
        if (dim == 0) {
          part[kRows * D + row] = M;
          part[kRows * D + kRows + row] = L;
        }
      }
    }
    if (now.i0 == 0 && !whole && tid == 0) {
      // the last CTA with a part: the one whose share holds the item's last unit
      int c = share_of(now.end - 1, total, ctas);
      while (c > cta + 1 && snap(share_start(total, c, ctas), now.first, now.end, kItemUnits, kSlack) >= now.end) --c;
      split.rec[cta] = SplitRecord{now.row0, now.g, 1, now.p0, c, cta};
    }
    __syncwarp();   // lanes part above; the next tiles' products are collective
    buf ^= 1;
  }
}

// Joins the parts of one split item (blockIdx.x: the CTA that began it) for one query head (blockIdx.y).
// Warp w takes parts w, w + 4, ...; the four warps are then joined in order.
// A warp has BATCH of its parts in flight at once, or FEW where no warp has more (0: never looked at).  Here 8.  Over an 8-bit
// cache, whose items take half as long, 10 and 2: one sequence's 76 parts a head come in two round trips, and an item of few
// parts does not go through the sums of many (32768 positions 12.95 -> 12.55 us, windows 14.1 -> 13.9; with 20 in flight,
// whose registers leave room for half as many blocks, 64 ragged take 22.7 in place of 21.9).
constexpr int kJoinWarps = 4;

template <int D, bool FP16, int BATCH, int FEW>
__global__ void __launch_bounds__(kJoinWarps * 32) decode_join_kernel(const PagedArgs a, const DecodeSplit split) {
  using C = Dec<D>;
  constexpr int E = D / 32;
  __shared__ float mw_s[kJoinWarps], lw_s[kJoinWarps];
  __shared__ float red[kJoinWarps][D];
  pdl_wait();
  pdl_launch_dependents();
  const int first = (int)blockIdx.x, row = (int)blockIdx.y;
  const SplitRecord rec = load_record(split.rec + first);
  if (rec.until < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int parts = rec.until - first + 1;
  float m = kUnseen, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  auto turn = [&](auto batch_c, int i0) {
    constexpr int N = decltype(batch_c)::value;
    float mb[N], lb[N], ob[N][E];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = i0 + i * kJoinWarps;
      mb[i] = kUnseen;
      lb[i] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) ob[i][e] = 0.f;
      if (c < parts) {
        const float* p = split.part + ((size_t)(first + c) * 2 + (c == 0 ? 1 : 0)) * C::kPartFloats;
        mb[i] = __ldcg(p + kRows * D + row);
        lb[i] = __ldcg(p + kRows * D + kRows + row);
#pragma unroll
        for (int e = 0; e < E; ++e) ob[i][e] = __ldcg(p + row * D + e * 32 + lane);
      }
    }
    float mx = m;
#pragma unroll
    for (int i = 0; i < N; ++i) mx = fmaxf(mx, mb[i]);
    const float sc = exp2f(m - mx);
    l *= sc;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= sc;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float w = exp2f(mb[i] - mx);
      l += lb[i] * w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += ob[i][e] * w;
    }
    m = mx;
  };
  if (FEW > 0 && parts <= kJoinWarps * FEW) {
    if (warp < parts) turn(std::integral_constant<int, FEW == 0 ? 1 : FEW>{}, warp);
  } else {
#pragma unroll 1
    for (int i0 = warp; i0 < parts; i0 += kJoinWarps * BATCH) turn(std::integral_constant<int, BATCH>{}, i0);
  }
  if (lane == 0) {
    mw_s[warp] = m;
    lw_s[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) red[warp][e * 32 + lane] = acc[e];
  __syncthreads();
  for (int d = threadIdx.x * 2; d < D; d += kJoinWarps * 64) {
    float M = mw_s[0], L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) M = fmaxf(M, mw_s[w]);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float sw = exp2f(mw_s[w] - M);
      L += lw_s[w] * sw;
      x += red[w][d] * sw;
      y += red[w][d + 1] * sw;
    }
    x /= L;
    y /= L;
    const uint32_t w = pack16<FP16>(x, y);
    const float2 back = unpack16<FP16>(w);   // (over an 8-bit cache a finite sum may be past fp16)
    if (!isfinite(back.x) || !isfinite(back.y)) raise_flag(a.err, kErrNonFinite);
    *reinterpret_cast<uint32_t*>(a.o + rec.row * a.o_stride + (long long)(rec.g * a.G + row) * D + d) = w;
  }
}

template <int D, bool FP16>
cudaError_t launch(const PagedMaps& maps, const PagedArgs& a, const DecodeSplit& split, int ctas, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(decode_kernel<D, FP16>), (int)Dec<D>::smem(kPagedMaxSeqs), &ready);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Dec<D>::smem(a.B);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, decode_kernel<D, FP16>, maps, a, split);
  return e == cudaSuccess ? launch_paged_decode_join(a, D, split, ctas, false, st) : e;
}

}  // namespace

size_t paged_decode_scratch(int D, int ctas) {
  return (size_t)ctas * (2 * (kRows * D + 2 * kRows) * sizeof(float) + sizeof(SplitRecord));
}

DecodeSplit paged_decode_split(int D, void* scratch, int ctas) {
  DecodeSplit split;
  split.part = static_cast<float*>(scratch);
  split.rec = reinterpret_cast<SplitRecord*>(split.part + (size_t)ctas * 2 * (kRows * D + 2 * kRows));
  return split;
}

namespace {
template <int BATCH, int FEW>
cudaError_t launch_join(const PagedArgs& a, int D, const DecodeSplit& split, int ctas, cudaStream_t st) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, a.G);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (D == 128)
    return a.fp16 ? cudaLaunchKernelEx(&cfg, decode_join_kernel<128, true, BATCH, FEW>, a, split)
                  : cudaLaunchKernelEx(&cfg, decode_join_kernel<128, false, BATCH, FEW>, a, split);
  return a.fp16 ? cudaLaunchKernelEx(&cfg, decode_join_kernel<64, true, BATCH, FEW>, a, split)
                : cudaLaunchKernelEx(&cfg, decode_join_kernel<64, false, BATCH, FEW>, a, split);
}

}  // namespace

cudaError_t launch_paged_decode_join(const PagedArgs& a, int D, const DecodeSplit& split, int ctas, bool wide, cudaStream_t st) {
  return wide ? launch_join<10, 2>(a, D, split, ctas, st)
              : launch_join<8, 0>(a, D, split, ctas, st);
}

cudaError_t launch_paged_decode(const PagedMaps& maps, const PagedArgs& a, int D, void* scratch, int ctas, cudaStream_t st) {
  const DecodeSplit split = paged_decode_split(D, scratch, ctas);
  if (D == 128) return a.fp16 ? launch<128, true>(maps, a, split, ctas, st) : launch<128, false>(maps, a, split, ctas, st);
  return a.fp16 ? launch<64, true>(maps, a, split, ctas, st) : launch<64, false>(maps, a, split, ctas, st);
}

}  // namespace moe
