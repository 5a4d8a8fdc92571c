// The paged key/value cache as the kernels see it: the arguments of one call and the checked reads
// of the tables that live on the GPU (contracts in include/gqa_paged.h).
#pragma once

#include <atomic>
#include <cfloat>

#include "../../include/gqa_paged.h"
#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr uint32_t kErrBadPages = 16u;   // a length, page or slot out of range

constexpr int kPagedMaxSeqs = 4096;

struct PagedArgs {
  const uint16_t* q;        // [T, Hq, D]
  const uint16_t* kc;       // [num_pages, Hkv, page_size, D]
  const uint16_t* vc;
  const int32_t* table;     // [B, max_pages]
  const int32_t* q_start;   // [B + 1]
  const int32_t* kv_len;    // [B]
  uint16_t* o;              // [T, Hq, D]
  uint32_t* err;
  int Hq, Hkv, G;
  int page_shift, num_pages, max_pages;
  int B, T, max_new;
  int window, sinks;
  int fp16;
  long long q_stride, o_stride, page_stride, head_stride, row_stride;
  float qk_scale;           // log2(e) / sqrt(D): scores in base-2 units
};

// Everything that an earlier call may have written (tables, lengths, slots, queries, keys and values) is read by ordinary
// loads, after pdl_wait: a launch waits there for the calls before it, but its CTAs may be resident while those still
// write, and the read-only path (__ldg) is for data that no one changes while the kernel runs.

// One sequence's rows and length, cut to what the buffers hold.  A sequence whose rows do not lie in
// the buffers has none.
struct SeqRows {
  int row0, n;   // its rows of q and o
  int p0;        // position of its first row (negative: the row sees nothing)
  int L;         // positions in the cache
};

__device__ __forceinline__ SeqRows load_seq(const PagedArgs& a, int b, bool& bad) {
  const int r0 = a.q_start[b], r1 = a.q_start[b + 1], len = a.kv_len[b];
  const bool rows_ok = r0 >= 0 && r1 >= r0 && r1 <= a.T;
  SeqRows s;
  s.row0 = rows_ok ? r0 : 0;
  s.n = rows_ok ? r1 - r0 : 0;
  s.L = min(max(len, 0), a.max_pages << a.page_shift);
  s.p0 = s.L - s.n;
  if (!rows_ok || s.L != len || s.n > a.max_new) bad = true;
  s.n = min(s.n, a.max_new);
  return s;
}

// Positions, windows and their differences stay within 32 bits: a row of the block table spans at most 2^30
// positions, and a window that no position can pass is taken as none.
// Whether the token at position p sees position j.
__device__ __forceinline__ bool paged_sees(const PagedArgs& a, int p, int j) {
  return j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
}

// The cache tiles of TN positions that rows at positions p_lo .. p_hi see: tiles 0 .. head - 1 hold the
// leading positions that stay visible, the others follow `skip` tiles later.  At least one tile, so
// that rows that see nothing are still written.
struct TileRange {
  int count, head, skip;
  __device__ __forceinline__ int tile(int i) const { return i < head ? i : i + skip; }
};

template <int TN>
__device__ __forceinline__ TileRange visible_tiles(const PagedArgs& a, int p_lo, int p_hi) {
  constexpr int kShift = TN == 64 ? 6 : 7;
  static_assert(TN == 1 << kShift, "tile");
  TileRange r;
  r.head = r.skip = 0;
  r.count = p_hi < 0 ? 1 : (p_hi >> kShift) + 1;
  if (a.window > 0 && p_hi >= 0) {
    const int first = max(0, p_lo - a.window + 1) >> kShift;         // first tile of the window
    const int head = (min(a.sinks, p_hi + 1) + TN - 1) >> kShift;
    if (head < first) {
      r.head = head;
      r.skip = first - head;
      r.count -= r.skip;
    }
  }
  return r;
}

// Whether rows at positions p_lo .. p_hi see any position of page `ip`.
__device__ __forceinline__ bool page_needed(const PagedArgs& a, int ip, int p_lo, int p_hi) {
  const int j0 = ip << a.page_shift, j1 = j0 + (1 << a.page_shift) - 1;
  return j0 <= p_hi && (a.window == 0 || j1 > p_lo - a.window || j0 < a.sinks);
}

// The maximum of no scores: the lowest finite value, since a visible score may be any finite one, and since two of it
// differ by 0 (of infinities the difference, a weight's exponent, is none).  The sum beside it is 0.
constexpr float kUnseen = -FLT_MAX;

// Whether every row at positions p_lo .. p_hi sees every position j0 .. j0 + TN - 1.
template <int TN>
__device__ __forceinline__ bool tile_open(const PagedArgs& a, int j0, int p_lo, int p_hi) {
  return j0 + TN - 1 <= p_lo && (a.window == 0 || j0 > p_hi - a.window || j0 + TN <= a.sinks);
}

// ------------------------------------------------------------------------------------------
// Split of the work over the CTAs.  The cache tiles of all items (an item is a block of query rows of
// one key/value head), in order, each item's behind a few units that stand for its start and end, are cut
// into equal consecutive shares, one a CTA.  An item that lies in several shares leaves one partial result
// (unnormalised O, max and sum per row) in each, joined by a second launch in order.  A CTA has at most
// two partials: slot 0 of an item that began before it, slot 1 of one that goes on after it.
// ------------------------------------------------------------------------------------------
constexpr int kPagedMaxCtas = 160;   // one CTA per SM, of 152

// What the joining launch needs of a CTA whose last item goes on in later CTAs.
struct SplitRecord {
  int32_t row, g, rows;   // first row of o, head group, tokens of the item
  int32_t p_lo;           // position of the item's first token
  int32_t until;          // the last CTA with a part of the item that begins here (< 0: none goes on)
  int32_t first;          // the CTA where the item that goes on begins: this one, or (chunk form) an earlier one
};

// (From L2: the launch that wrote it may have ended just now.)
__device__ __forceinline__ SplitRecord load_record(const SplitRecord* r) {
  return SplitRecord{__ldcg(&r->row), __ldcg(&r->g), __ldcg(&r->rows), __ldcg(&r->p_lo), __ldcg(&r->until), __ldcg(&r->first)};
}

// The schedule is made by every CTA for itself, by a block of NT threads together: it stands before all work, and
// its time is a chain of latencies (34 sequences mixed: 4,300 cycles; by one warp without barriers, 6,700).

// Exclusive sums over the block; `over`: the total passes 32 bits (and the sums mean nothing).
template <int NT>
__device__ __forceinline__ uint32_t exclusive_scan(unsigned long long mine, uint32_t* warp_s, uint32_t* sum, bool* over) {
  static_assert(NT % 32 == 0 && NT <= 512, "one warp scans the warps' sums, 16 lanes wide");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = (uint32_t)mine;
  bool carry = (mine >> 32) != 0;   // sums only grow, so none is wrong unless some addition carries
  __syncwarp();                     // the lanes' runs differ in length
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, inc, off);
    if (lane >= off) {
      inc += x;
      carry |= inc < x;
    }
  }
  if (lane == 31) warp_s[warp] = inc;
  __syncthreads();
  uint32_t w = lane < NT / 32 ? warp_s[lane] : 0u;
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) {
    const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, w, off);
    if (lane >= off) {
      w += x;
      carry |= lane < 16 && w < x;
    }
  }
  *sum = __shfl_sync(0xFFFFFFFFu, w, 15);
  const uint32_t before = __shfl_sync(0xFFFFFFFFu, w, (warp + 15) & 15);
  *over = __syncthreads_or(carry) != 0;   // (warp_s may be written again after it)
  return (warp == 0 ? 0u : before) + inc - (uint32_t)mine;
}

// Sums of cost(b) over the sequences before each, into pre_s[0 .. B], by the block; returns the total.
template <int NT, class Cost>
__device__ __forceinline__ uint32_t scan_sequences(int B, uint32_t* pre_s, uint32_t* warp_s, bool* over, Cost cost) {
  const int tid = threadIdx.x, per = (B + NT - 1) / NT, b0 = min(tid * per, B), b1 = min(b0 + per, B);
  unsigned long long mine = 0;
  uint32_t sum;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    pre_s[b] = (uint32_t)mine;
    mine += cost(b);
  }
  const uint32_t before = exclusive_scan<NT>(mine, warp_s, &sum, over);
#pragma unroll 1
  for (int b = b0; b < b1; ++b) pre_s[b] += before;
  if (tid == 0) pre_s[B] = sum;
  __syncwarp();
  __syncthreads();
  return sum;
}

// The last sequence b with pre_s[b] <= x (x < pre_s[B]).
__device__ __forceinline__ int find_sequence(const uint32_t* pre_s, int B, uint32_t x) {
  int lo = 0, hi = B - 1;
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre_s[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// A cut of the order within the item of units s .. e - 1 (`own` of them its start and end, then its tiles),
// moved to an end of the item that is within `slack` tiles.  What remains between has tiles on both sides.
__device__ __forceinline__ uint32_t snap(uint32_t x, uint32_t s, uint32_t e, uint32_t own, uint32_t slack) {
  const uint32_t down = x - s, up = e - x;
  if (down <= own + slack && down <= own + up) return s;
  return up <= slack ? e : x;
}

// Where the c-th of n equal shares of `total` units begins: the first shares take one of those left over.
__device__ __forceinline__ uint32_t share_start(uint32_t total, int c, int n) {
  const uint32_t q = total / n;
  return q * c + min((uint32_t)c, total - q * n);
}

// The share that holds unit `pos`.
__device__ __forceinline__ int share_of(uint32_t pos, uint32_t total, int n) {
  const uint32_t q = total / n, more = total - q * n, wide = (q + 1) * more;   // `more` shares of q + 1, then of q
  return (int)(pos < wide ? pos / (q + 1) : more + (pos - wide) / q);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
      "%5}], [%6];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

struct PagedMaps {
  CUtensorMap k, v;   // {D, page_size, Hkv, num_pages}, box {64, min(page_size, rows of a tile), 1, 1}, 128-byte swizzle
  CUtensorMap q;      // chunk form: {D, Hq, T}, box {64, G, tokens of a tile}
};

// 2^x.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values rounded to a pair of the 16-bit type (lo in the low half), and back.
template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if (FP16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool FP16>
__device__ __forceinline__ float2 unpack16(uint32_t x) {
  if (FP16) return __half22float2(*reinterpret_cast<const __half2*>(&x));
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
}

// Lets `kernel` use `bytes` of shared memory on the current device, once for each of the first 64 (bits of `ready`;
// racing first calls set the same value).
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>* ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (ready->load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// ------------------------------------------------------------------------------------------
// The two forms and their joining launch
// ------------------------------------------------------------------------------------------
size_t paged_decode_scratch(int D, int ctas);      // bytes of partials and records
size_t paged_chunk_scratch(int D, int ctas);
cudaError_t launch_paged_chunk(const PagedMaps& maps, const PagedArgs& a, int D, void* scratch, int ctas, cudaStream_t st);
cudaError_t launch_paged_decode(const PagedMaps& maps, const PagedArgs& a, int D, void* scratch, int ctas, cudaStream_t st);

}  // namespace moe
