// Single-token attention over the paged cache held in 8 bits (contract in include/gqa_paged8.h): one pass over the
// visible codes, bound by HBM.
//
//   * work split, items, shares and the joining launch are those of the 16-bit form (paged_decode.cu): tiles of 64
//     positions of one key/value head, all its query heads (up to eight) together, equal shares of tiles, one a CTA;
//   * three warps copy the tile's pages by tensor map into a ring of 128 KB (a page is one box of keys and one of values); a
//     fourth reads the tile's eight scales, page numbers two and scales one batch of four tiles ahead, into the
//     ring's stage;
//   * eight consumer warps, two a tile, 32 positions each.  Codes become fp16, exactly, in registers (one conversion for
//     two of them), and both products are m16n8k16 in fp16 with the heads as the 16-row operand.  Which dims meet in
//     one step of Q K^T is free as long as queries and keys agree: a lane takes 16 bytes of a key's row at once
//     (one shared load, no ldmatrix), whose every four are one step.  Values come transposed by ldmatrix in pairs of dims, so
//     even and odd dims of 16 go to two tiles of O, and a lane ends with four dims in a row;
//   * queries are scaled by a power of two a row so that fp16 holds them; a block's key scale multiplies its scores.  Its
//     value scale multiplies its numerators, relative to the largest that the warp has met (O is kept in units
//     of that), so that all of fp16's range serves the numerators, rounded ones in rows 0..7 and their remainders
//     in rows 8..15 of the operand.
//   * the warps' results of a segment lie in one of two buffers; a warp joins them only when its tiles of the next segment
//     are done, so that none waits for a slower one before the share's end.
//
// Measured in a graph, 16 / 2 heads of 128: one sequence of 32768 positions (fp16) 12.2 us, of which 2.5 are its bytes and the
// rest is a chain: the dependency wait 0.7, the schedule 1.4, the first tile's way 0.9, tiles 2.4, the join within a CTA 1.2,
// the second launch and its join 4; 64 ragged ones (up to 32768, 69.6 MB) 21.7 us, 3.2 TB/s, 47 % of the copy rate (20.9 in
// pages of 64); 32 of them with a window of 4096 13.2; 64 ragged ones with heads of 64 18.4 (16.6 in pages of 64).  While
// tiles run, a warp's own chain bounds it (conversion, product, maximum, exponential, product): two warps a scheduler
// fill 43 % of the issue slots.  Twelve consumer warps of 152 registers, three a scheduler, were slower (26.7), and so were
// rings of 96 or 160 KB with one joining buffer (23.3).
// Steps: 32768 positions 13.8 -> 13.0 and 64 ragged ones 22.5 -> 21.7 with four independent products side by side (one
// waits ~30 cycles for the one before); 32768 positions 13.0 -> 12.5 with the schedule of up to 32 sequences without
// barriers and joins of many parts in fewer round trips; windows 13.9 -> 13.2, 64 ragged in pages of 64 22.1 -> 20.9
// without a barrier at a segment's end.  kItemUnits of 2, 3, 4, 5 at the latter: 25.1, 22.2, 20.9, 21.1.
#include <cmath>
#include <cstring>

#include "paged8.cuh"

namespace moe {
namespace {

constexpr int kTN = 64;                        // positions per tile
constexpr int kWarps = 8;                      // consumer warps: four groups of two, tiles in turn
constexpr int kGroups = 4;
constexpr int kCopyWarps = 3;                  // (12 warps in all: a thirteenth would leave 128 registers a thread, not 168)
constexpr int kThreads = (kWarps + kCopyWarps + 1) * 32;
constexpr int kRows = 8;                       // query heads per key/value head, at most
constexpr int kItemUnits = 4;                  // what an item costs beside its tiles, in tiles
constexpr int kSlack = 1;                      // tiles that a cut moves to reach an item's end
constexpr float kLift = 15.f;                  // base-2 units of the largest numerator, which uses fp16's range from there down
constexpr float kLower = 0x1p-15f;             // 2^-kLift

template <int D>
struct Dec8 {
  static constexpr int kTileBytes = kTN * D;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = 128 * 1024 / kStageBytes;
  static constexpr int kOStride = D + 16;                // padded row of the joining buffer (floats)
  static constexpr int kJoinFloats = kWarps * kRows * kOStride;
  static constexpr int kJoinBytes = 2 * kJoinFloats * 4; // two buffers: an item's is read while the next one's is written
  static constexpr int kPartFloats = kRows * D + 2 * kRows;
  static size_t smem(int B) { return 1024 + (size_t)kStages * kStageBytes + kJoinBytes + ((size_t)B + 1) * 4; }
  // Byte offset of 16-byte chunk `chunk` of row `pos` in a tile written under the tensor map's swizzle (of 128 bytes, or of 64).
  static __device__ __forceinline__ uint32_t at(int pos, int chunk) {
    return D == 128 ? (uint32_t)(pos * 128 + ((chunk ^ (pos & 7)) << 4)) : (uint32_t)(pos * 64 + ((chunk ^ ((pos >> 1) & 3)) << 4));
  }
};

__device__ __forceinline__ void mma_half(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// A segment whose warps' results lie in a joining buffer.
struct Told {
  int g, i0, n, count, p0, row0;
  uint32_t first, end;
};

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads, 1)
    decode8_kernel(const __grid_constant__ PagedMaps maps, const Paged8Args a, const DecodeSplit split) {
  using C = Dec8<D>;
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t full[C::kStages], empty[C::kStages], told[2], joined[2];
  __shared__ __align__(16) float scale_s[C::kStages][8];      // of the stage's blocks: keys, values
  __shared__ __align__(16) float ml_s[2][kRows][2][kWarps];   // per buffer and row: the warps' max, then sum
  __shared__ uint32_t warp_s[kThreads / 32];
  __shared__ Told told_s[2];
  __shared__ int abort_s;
  const uint32_t raw = smem_u32(sm_raw), base = (raw + 1023u) & ~1023u;
  float* join_s = reinterpret_cast<float*>(sm_raw + (base - raw) + C::kStages * C::kStageBytes);
  uint32_t* pre_s = reinterpret_cast<uint32_t*>(sm_raw + (base - raw) + C::kStages * C::kStageBytes + C::kJoinBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = (int)blockIdx.x;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&full[s]), kCopyWarps + 1);
      mbar_init(smem_u32(&empty[s]), kWarps / kGroups);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&told[i]), kWarps);
      mbar_init(smem_u32(&joined[i]), kWarps);
    }
    abort_s = 0;
    mbar_fence_init();
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
  }
  __syncthreads();   // the barriers are there (before the calls before are done)
  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's share: units lo .. hi - 1 of (sequence, head, tile); pre_s: units before each sequence
  bool bad = false;
  auto cost = [&](int b) {
    const SeqRows s = load_seq(a, b, bad);
    return s.n == 0 ? 0ull : (unsigned long long)(visible_tiles<kTN>(a, s.p0, s.p0).count + kItemUnits) * a.Hkv;
  };
  bool over;
  uint32_t total = scan_sequences8<kThreads>(a.B, pre_s, warp_s, &over, cost);
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
    // Producers walk the share's segments: body(sequence, its rows, tiles, head, first tile, tiles) until it returns false.
    bool stop = false;
    bad = false;
    auto walk = [&](auto&& body) {
      int b = b_first;
      for (uint32_t u = lo; u < hi && !stop; ++b) {
        if (pre_s[b + 1] <= u) continue;
        const SeqRows s = load_seq(a, b, bad);
        const TileRange r = visible_tiles<kTN>(a, s.p0, s.p0);
        const uint32_t end = min(pre_s[b + 1], hi);
        while (u < end && !stop) {
          const uint32_t units = r.count + kItemUnits, g = (u - pre_s[b]) / units, first = pre_s[b] + g * units;
          const int i0 = max((int)(u - first) - kItemUnits, 0), n = (int)min(end - first, units) - kItemUnits - i0;
          body(b, s, r, (int)g, i0, n);
          u = min(end, first + units);
        }
      }
    };
    int issued = 0;
    // The next stage of the ring, once it is free.
    auto next_stage = [&](int* st) {
      *st = issued % C::kStages;
      if (issued >= C::kStages && !mbar_wait_warp(smem_u32(&empty[*st]), ((issued / C::kStages) - 1) & 1, &abort_s, a.err)) {
        stop = true;
        return false;
      }
      ++issued;
      return true;
    };
    if (warp < kWarps + kCopyWarps) {
      // ---- copies: every warp takes a third of a tile's boxes
      const int pw = warp - kWarps;
      const int ppt_shift = max(0, 6 - a.page_shift), ppt = 1 << ppt_shift;   // pages of a tile
      const int box_rows = min(kTN, 1 << a.page_shift);
      const int copies = ppt * 2;                                // (page, keys or values)
      const int c0 = copies * pw / kCopyWarps, mine = copies * (pw + 1) / kCopyWarps - c0;
      const int sub = (c0 + lane) >> 1, kv = (c0 + lane) & 1;
      const int batch = 32 >> ppt_shift;                         // tiles whose page numbers the lanes hold
      walk([&](int b, const SeqRows& s, const TileRange& r, int g, int i0, int n) {
        const int32_t* row = a.table + (size_t)b * a.max_pages;
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
          int st;
          if (!next_stage(&st)) break;
          const uint32_t bar = smem_u32(&full[st]);
          const int off = (r.tile(i0 + i) * kTN) & ((1 << a.page_shift) - 1);   // 64 in the second half of a page of 128
          if (lane == 0) mbar_arrive_expect_tx(bar, mine * box_rows * D);
          __syncwarp();
          const int p = __shfl_sync(0xFFFFFFFFu, pg, (in * ppt + sub) & 31);
          if (lane < mine)
            tma_load_4d(base + st * C::kStageBytes + kv * C::kTileBytes + sub * box_rows * D, kv ? &maps.v : &maps.k, bar, 0,
                        off, g, p);
          __syncwarp();
        }
      });
    } else {
      // ---- scales: lane 8 t + 4 kv + block of batches of four tiles
      const int lt = lane >> 3, kv = (lane >> 2) & 1, blk = lane & 3;
      const float* scales = kv ? a.vs : a.ks;
      walk([&](int b, const SeqRows& s, const TileRange& r, int g, int i0, int n) {
        const int32_t* row = a.table + (size_t)b * a.max_pages;
        // The block's first position in the batch of tiles from i on, or -1 if the token sees none of it.
        auto block_at = [&](int i) {
          const int t = i0 + i + lt;
          if (i + lt >= n || t >= r.count) return -1;
          const int j = r.tile(t) * kTN + blk * 16;
          return j <= s.p0 && (a.window == 0 || j + 15 > s.p0 - a.window || j < a.sinks) ? j : -1;
        };
        auto page_of = [&](int i) {
          const int j = block_at(i);
          return j < 0 ? -1 : row[j >> a.page_shift];
        };
        auto scale_of = [&](int i, int page) {
          const int j = block_at(i);
          if (j < 0 || page < 0 || page >= a.num_pages) return kLeastScale;   // (a bad page: the copies say so)
          return scales[scale_index(page, a.Hkv, g, a.page_shift, j & ((1 << a.page_shift) - 1))];
        };
        int page = page_of(0);
        float ahead = scale_of(0, page), now = 0.f;
        page = page_of(4);
        for (int i = 0; i < n; ++i) {
          if ((i & 3) == 0) {
            now = ahead;
            if (!scale_ok(now)) {
              bad = true;
              now = kLeastScale;
            }
            ahead = scale_of(i + 4, page);
            page = page_of(i + 8);
          }
          __syncwarp();
          int st;
          if (!next_stage(&st)) break;
          if (lt == (i & 3)) scale_s[st][lane & 7] = now;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&full[st]));
          __syncwarp();
        }
      });
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
  const int group = warp >> 1, half = (warp & 1) * 32;   // its tiles' positions half .. half + 31
  const int r = lane >> 2, c = lane & 3;
  const int vpos = half + (lane >> 3) * 8 + (lane & 7);  // value row this lane addresses

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
  // The heads as the 16-row operand; rows past the group's heads repeat its first one: every row has sums of its own,
  // and theirs are not stored.  A lane's dims: D / 4 in a row from c * D / 4 on, four to a step.
  uint32_t qa[D / 8];
  float q_scale;   // of this lane's row: of the scores in base-2 units
  auto load_queries = [&](const Segment& x) {
    const uint4* qh = reinterpret_cast<const uint4*>(
        a.q + (x.n > 0 ? x.row0 * a.q_stride + (long long)(x.g * a.G + (r < a.G ? r : 0)) * D : 0) + c * (D / 4));
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const uint4 w = qh[e];
      qa[4 * e] = w.x;
      qa[4 * e + 1] = w.y;
      qa[4 * e + 2] = w.z;
      qa[4 * e + 3] = w.w;
    }
  };
  auto convert_queries = [&]() {
    q_scale = a.qk_scale;
    if (FP16) return;
    // bf16 times the power of two that brings the row's largest to 2^14 .. 2^15: exact down to 2^-24, and so within 2^-39 of the
    // largest, or 2^-105.
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < D / 8; ++e) top = max(top, max(qa[e] & 0x7FFFu, (qa[e] >> 16) & 0x7FFFu));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const int E = (int)(top >> 7), e2 = E == 255 ? 0 : min(max(E - 141, -80), 60);
    const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
    q_scale *= __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
    for (int e = 0; e < D / 8; ++e) {
      const float2 f = unpack16<false>(qa[e]);
      qa[e] = pack16<true>(f.x * down, f.y * down);
    }
  };

  // Joins the eight warps' results of the s-th segment in order.  Every warp comes here only when its tiles of the next
  // segment are done, so that none waits for a slower one but behind the share's last segment.
  auto join = [&](int s) {
    const int buf = s & 1;
    mbar_wait_warp(smem_u32(&told[buf]), (s >> 1) & 1, &abort_s, a.err);
    const Told now = told_s[buf];
    const bool whole = now.i0 == 0 && now.n == now.count;
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
        const uint2 w = make_uint2(pack16<FP16>(v.x, v.y), pack16<FP16>(v.z, v.w));
        const float2 w0 = unpack16<FP16>(w.x), w1 = unpack16<FP16>(w.y);
        if (!isfinite(w0.x) || !isfinite(w0.y) || !isfinite(w1.x) || !isfinite(w1.y)) raise_flag(a.err, kErrNonFinite);
        *reinterpret_cast<uint2*>(a.o + now.row0 * a.o_stride + (long long)(now.g * a.G + row) * D + dim) = w;
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
      int c2 = share_of(now.end - 1, total, ctas);
      while (c2 > cta + 1 && snap(share_start(total, c2, ctas), now.first, now.end, kItemUnits, kSlack) >= now.end) --c2;
      split.rec[cta] = SplitRecord{now.row0, now.g, 1, now.p0, c2, cta};
    }
    __syncwarp();   // lanes part above; the next tiles' products are collective
    if (lane == 0) mbar_arrive(smem_u32(&joined[buf]));
    __syncwarp();
  };

  int it = 0, segs = 0;   // tiles and segments of the share so far
  Segment x = next_segment();
  load_queries(x);
  while (x.n > 0) {
    convert_queries();
    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    float m_run = kUnseen, l_run = 0.f, v_ref = kLeastScale;   // O is in units of v_ref
    for (int i = (group - it) & (kGroups - 1); i < x.n; i += kGroups) {   // tile it + i of the share goes to group (it + i) & 3
      const int st = (it + i) % C::kStages;
      if (mbar_wait_warp(smem_u32(&full[st]), ((it + i) / C::kStages) & 1, &abort_s, a.err)) {
        const uint32_t sk = base + st * C::kStageBytes, sv = sk + C::kTileBytes;
        // (four independent products beside one another: one alone waits ~30 cycles for the one before it)
        float sc[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
        for (int s = 0; s < D / 64; ++s) {
          uint32_t w[4][4];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint4 v = ld_shared16(sk + C::at(half + 8 * t + r, c * (D / 64) + s));
            w[t][0] = v.x, w[t][1] = v.y, w[t][2] = v.z, w[t][3] = v.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              uint32_t b0, b1;
              codes_to_half4(w[t][e], b0, b1);
              mma_half(sc[t], qa[8 * s + 2 * e], 0u, qa[8 * s + 2 * e + 1], 0u, b0, b1);
            }
        }
        const float2 ks = *reinterpret_cast<const float2*>(&scale_s[st][half >> 4]);
        const float2 vs = *reinterpret_cast<const float2*>(&scale_s[st][4 + (half >> 4)]);
        const float k0 = ks.x * q_scale, k1 = ks.y * q_scale;
        const int j0 = x.r.tile(x.i0 + i) * kTN;
        const bool open = tile_open<kTN>(a, j0, x.p0, x.p0);
        uint32_t keep[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};   // value pairs that the token sees
        float s2[4][2];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          s2[t][0] = sc[t][0] * (t < 2 ? k0 : k1);
          s2[t][1] = sc[t][1] * (t < 2 ? k0 : k1);
        }
        if (!open) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int j = j0 + half + 8 * t + 2 * c;
            const bool v0 = paged_sees(a, x.p0, j), v1 = paged_sees(a, x.p0, j + 1);
            s2[t][0] = v0 ? s2[t][0] : -INFINITY;
            s2[t][1] = v1 ? s2[t][1] : -INFINITY;
            keep[t] = (v0 ? 0xFFFFu : 0u) | (v1 ? 0xFFFF0000u : 0u);
          }
        }
        float mx = fmaxf(fmaxf(fmaxf(s2[0][0], s2[0][1]), fmaxf(s2[1][0], s2[1][1])),
                         fmaxf(fmaxf(s2[2][0], s2[2][1]), fmaxf(s2[3][0], s2[3][1])));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        const float m_new = fmaxf(m_run, mx), v_new = fmaxf(v_ref, fmaxf(vs.x, vs.y));
        if (__any_sync(0xFFFFFFFFu, m_new != m_run || v_new != v_ref)) {
          const float alpha = ex2(m_run - m_new), by = alpha * (v_ref / v_new);
          m_run = m_new;
          v_ref = v_new;
          l_run *= alpha;
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            o[j][0] *= by;
            o[j][1] *= by;
            o[j][2] *= by;
            o[j][3] *= by;
          }
        }
        const float v0 = vs.x / v_ref, v1 = vs.y / v_ref;   // at most 1
        uint32_t hi2[4], lo2[4];
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          // (lifted after the difference: a maximum of 2^24 or more less the lift would be rounded by up to 16)
          float p0 = ex2((s2[t][0] - m_run) + kLift), p1 = ex2((s2[t][1] - m_run) + kLift);
          sum += p0 + p1;
          p0 *= t < 2 ? v0 : v1;
          p1 *= t < 2 ? v0 : v1;
          hi2[t] = pack16<true>(p0, p1);
          const float2 h = unpack16<true>(hi2[t]);
          lo2[t] = pack16<true>(p0 - h.x, p1 - h.y);
        }
        l_run += sum;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          uint32_t w[4], even[4], odd[4];
          ldsm4_t(sv + C::at(vpos, j), w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            codes_to_half4(__byte_perm(w[t], 0u, 0x3120), even[t], odd[t]);
            if (!open) {
              even[t] &= keep[t];
              odd[t] &= keep[t];
            }
          }
          mma_half(o[2 * j], hi2[0], lo2[0], hi2[1], lo2[1], even[0], even[1]);
          mma_half(o[2 * j + 1], hi2[0], lo2[0], hi2[1], lo2[1], odd[0], odd[1]);
          mma_half(o[2 * j], hi2[2], lo2[2], hi2[3], lo2[3], even[2], even[3]);
          mma_half(o[2 * j + 1], hi2[2], lo2[2], hi2[3], lo2[3], odd[2], odd[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
    }
    it += x.n;

    // ---- this warp's result, for the join (the buffer has been read, two segments ago); the next segment's queries are on
    // their way meanwhile
    const int buf = segs & 1;
    if (segs >= 2) mbar_wait_warp(smem_u32(&joined[buf]), ((segs >> 1) - 1) & 1, &abort_s, a.err);
    l_run += __shfl_xor_sync(0xFFFFFFFFu, l_run, 1);
    l_run += __shfl_xor_sync(0xFFFFFFFFu, l_run, 2);
    if (c == 0) {
      ml_s[buf][r][0][warp] = m_run;
      ml_s[buf][r][1][warp] = l_run * kLower;
    }
    const float unit = v_ref * kLower;
    float* ow = join_s + buf * C::kJoinFloats + (warp * kRows + r) * C::kOStride + 4 * c;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)   // (even dims, then odd ones)
      *reinterpret_cast<float4*>(ow + 16 * j) =
          make_float4((o[2 * j][0] + o[2 * j][2]) * unit, (o[2 * j + 1][0] + o[2 * j + 1][2]) * unit,
                      (o[2 * j][1] + o[2 * j][3]) * unit, (o[2 * j + 1][1] + o[2 * j + 1][3]) * unit);
    if (tid == 0) told_s[buf] = Told{x.g, x.i0, x.n, x.r.count, x.p0, x.row0, x.first, x.end};
    x = next_segment();
    load_queries(x);
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&told[buf]));
    __syncwarp();
    if (segs > 0) join(segs - 1);
    ++segs;
  }
  if (segs > 0) join(segs - 1);
}

template <int D, bool FP16>
cudaError_t launch(const PagedMaps& maps, const Paged8Args& a, const DecodeSplit& split, int ctas, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(decode8_kernel<D, FP16>), (int)Dec8<D>::smem(kPagedMaxSeqs), &ready);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Dec8<D>::smem(a.B);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, decode8_kernel<D, FP16>, maps, a, split);
  return e == cudaSuccess ? launch_paged_decode_join(a, D, split, ctas, true, st) : e;
}

}  // namespace

cudaError_t launch_paged8_decode(const gqa_paged_dims& d, const Paged8Args& a, void* scratch, int ctas, cudaStream_t st) {
  PagedMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (!encode_pages8(&maps.k, a.kc8, d, kTN) || !encode_pages8(&maps.v, a.vc8, d, kTN)) return cudaErrorInvalidValue;
  const int D = d.head_dim;
  const DecodeSplit split = paged_decode_split(D, scratch, ctas);
  if (D == 128) return a.fp16 ? launch<128, true>(maps, a, split, ctas, st) : launch<128, false>(maps, a, split, ctas, st);
  return a.fp16 ? launch<64, true>(maps, a, split, ctas, st) : launch<64, false>(maps, a, split, ctas, st);
}

}  // namespace moe
