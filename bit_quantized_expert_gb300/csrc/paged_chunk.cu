// Attention of chunks of new tokens over the paged cache (contract in include/gqa_paged.h), on the
// fifth-generation tensor cores.
//
//   * Rows.  The G query heads of a key/value head share its cache, so a 128-row operand tile holds
//     floor(128 / G) tokens, each with its G heads (row = token * G + head): one tensor-map box of q.  An
//     item is two such tiles of one key/value head of one sequence, and walks the cache tiles (128
//     positions) that its rows see.
//   * Work split.  Shares of the cache tiles of all items, one per SM (paged.cuh).
//   * Roles.  Warps 0..3 and 4..7: softmax of the first and second row tile, one row a thread; warp 8:
//     copies; warp 9: tensor-core instructions; warps 10 and 11: the values of masked tiles.  (Registers are
//     moved to the softmax by warpgroups.)  While one row tile's softmax runs, the other's
//     products do:  S0 = Q0 K^T | S1 = Q1 K^T, then per cache tile  O0 += P0 V, S0 = Q0 K'^T,
//     O1 += P1 V, S1 = Q1 K'^T.
//   * S and O stay in tensor memory (128 columns of fp32 a tile each).  P replaces S there, in 16 bits,
//     as the A operand of the second product; V is read as it lies (positions by dims) through a
//     descriptor whose major axis is the output's.
//   * The running maximum that scales the numerators moves only when the new one is above it by kLazy
//     base-2 units: O is rescaled in a few tiles, not in all.
//   * Only tiles that some row does not wholly see are masked.  In those, the value tile is also
//     searched for non-finite values, since 0 times one of them is not 0: they are taken out, and the rows that do
//     see them get them back at the end.
//
// Bound by the softmax's chain: a cache tile of a row tile takes ~1,400 cycles of softmax (512 of them exponentials, at
// 32 a cycle and SM), then P V and the next scores, ~2,800 in all where both row tiles' products are 2,048.
// At 128 dims tensor memory is full, so the next scores cannot start before P is consumed; at 64 there is room, but an
// order that used it (two barriers more a tile) was slower (297 against 276 us behind 32768 positions).  Measured (16 query and 2
// key/value heads of 128, in a graph, no inputs in L2): 2048 tokens behind 32768 positions 341 us at best (1.66 PFLOP/s),
// 357 in the middle, with the clock that the power limit leaves; tensor pipe 74.6 % active; a prompt of 512 16.4 us; 4096
// tokens with a window of 1024 57.9 us; 2048 tokens behind 32768 positions with heads of 64 271 us.
#include <cmath>
#include <type_traits>

#include "paged.cuh"

namespace moe {
namespace {

constexpr int kTN = 128;                    // positions per cache tile
constexpr int kThreads = 384;               // two softmax warpgroups, one for copies and products
constexpr int kSoftmaxWarps = 8;
constexpr int kScanWarps = 2;
// Registers a thread: 168 at launch; 2 * 200 + 104 = 3 * 168 after the split.
constexpr int kRegsSoftmax = 200, kRegsOther = 104;
constexpr int kItemRows = 256;              // two row tiles
constexpr uint32_t kTmemO = 256;            // columns: S0 0, S1 128, O0 256, O1 384 (all 512 are allocated: base 0)
constexpr int kOutBytes = 32 * 64;          // a warp's staging of its 32 rows of o, 32 dims at a time
constexpr int kItemUnits = 2;               // what an item costs beside its tiles, in tiles (~5,000 cycles)
// Base-2 units by which the numerators' reference may lag behind the row's maximum, and by which it stands
// below the maximum that sets it: fp16 numerators use its range from 2^15 down, since it keeps 2^-25 at best and a
// long cache of small ones would be summed as nothing.  bf16 has fp32's range, and lags more: of 14 units and 6,
// 2048 tokens at 32768 take 364 and 374 us.
template <bool FP16>
constexpr float kLazy = FP16 ? 6.f : 14.f;
template <bool FP16>
constexpr float kLift = FP16 ? 9.f : 0.f;
// Base-2 units from which on a row's reference is taken off its scores before they are scaled (far_tiles).  Nearer ones
// are scaled and shifted in one fma, by a shift that is the scaled reference rounded: off by at most 2^-8 units here, but
// from 2^24 units on by as much as fp16 numerators have room for (2^16 at the top), from 2^31 on by all of bf16's range.
constexpr float kFar = 65536.f;

template <int D>
struct Chunk {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kTN * 128;                  // 128 rows of 64 dims
  static constexpr int kTileBytes = kBoxes * kBoxBytes;        // a row tile of q, a tile of keys or of values
  // Ring: a segment of n tiles takes n + 1 stages, the i-th with the values of its tile i - 1 and the keys
  // of tile i, which are used one after the other, so that one wait and one release serve both.
  static constexpr int kStages = 2;
  static constexpr int kStageBytes = 2 * kTileBytes;           // keys, then values
  static constexpr int kPartFloats = kItemRows * (D + 2);      // O by four columns of all rows, then max, then sum
  static size_t smem(int B) {
    return 1024 + (size_t)(2 + 2 * kStages) * kTileBytes + kSoftmaxWarps * kOutBytes + ((size_t)B + 1) * 4;
  }
};

struct ChunkSplit {
  float* part;         // [ctas][2][kPartFloats]
  SplitRecord* rec;    // [ctas]
};

// One row block: tokens t0 .. t0 + n - 1 of a sequence, at positions p_lo .. p_hi; it is an item for each
// key/value head.
struct Item {
  int t0, n, p_lo, p_hi;
  TileRange r;
};

__device__ __forceinline__ Item item_of(const PagedArgs& a, const SeqRows& s, int qt, int tokens) {
  Item x;
  x.t0 = qt * tokens;
  x.n = min(tokens, s.n - x.t0);
  x.p_lo = s.p0 + x.t0;
  x.p_hi = x.p_lo + x.n - 1;
  x.r = visible_tiles<kTN>(a, x.p_lo, x.p_hi);
  return x;
}

// A CTA's share: units lo .. hi - 1 of (sequence, row block, head, cache tile), an item's tiles standing behind
// kItemUnits units for its start and end, and the row block that holds
// unit lo (or ends just before it), which begins at unit `at`.
struct Share {
  uint32_t lo, hi, at, total, slack;
  int b, qt, ctas;
};

// Finds this CTA's share, by the block together: row blocks per sequence are scanned into pre_s[0 .. B], then
// their costs (units times heads), a run of consecutive row blocks a thread; the threads whose runs hold the
// two cuts walk theirs once more.  Leaves the share empty if there is nothing to do, or (bad) 2^32 units or more.
__device__ __forceinline__ void find_share(const PagedArgs& a, int tokens, uint32_t* pre_s, uint32_t* warp_s,
                                           Share* share_s, bool& bad) {
  const int tid = threadIdx.x, cta = (int)blockIdx.x;
  bool over;
  const uint32_t blocks = scan_sequences<kThreads>(a.B, pre_s, warp_s, &over, [&](int b) {
    return (uint32_t)(load_seq(a, b, bad).n + tokens - 1) / (uint32_t)tokens;
  });
  if (over) {
    bad = true;
    return;
  }
  const uint32_t per = (blocks + kThreads - 1) / kThreads;
  const uint32_t i0 = min(tid * per, blocks), i1 = min(i0 + per, blocks);
  // body(b, qt, units of an item) for the row blocks i0 .. i1 - 1
  auto run = [&](auto&& body) {
    if (i0 >= i1) return;
    uint32_t i = i0;
#pragma unroll 1
    for (int b = find_sequence(pre_s, a.B, i0); i < i1; ++b) {
      const SeqRows s = load_seq(a, b, bad);
#pragma unroll 1
      for (; i < i1 && i < pre_s[b + 1]; ++i) {
        const int qt = (int)(i - pre_s[b]);
        body(b, qt, (uint32_t)item_of(a, s, qt, tokens).r.count + kItemUnits);
      }
    }
  };
  unsigned long long mine = 0;
  int b_last = 0, qt_last = 0;
  uint32_t units_last = 0;
  run([&](int b, int qt, uint32_t units) {
    mine += (unsigned long long)units * a.Hkv;
    b_last = b;
    qt_last = qt;
    units_last = units;
  });
  uint32_t total;
  uint32_t at = exclusive_scan<kThreads>(mine, warp_s, &total, &over);
  if (over) bad = true;
  if (over || total == 0) return;
  const int ctas = (int)min(gridDim.x, total);   // no more shares than units
  if (cta >= ctas) return;
  const uint32_t lo = share_start(total, cta, ctas), hi = share_start(total, cta + 1, ctas);
  // A part costs a result written, read and joined: more than two tiles of imbalance.
  const uint32_t slack = max(2u, (total / ctas) >> 5);
  if (tid == 0) {
    share_s->total = total;
    share_s->ctas = ctas;
    share_s->slack = slack;
    if (hi == total) share_s->hi = total;
  }
  const uint32_t end = at + (uint32_t)mine;
  if ((lo < at || lo >= end) && (hi < at || hi >= end)) return;
  auto cut = [&](int b, int qt, uint32_t units) {
    const uint32_t past = at + units * a.Hkv;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const uint32_t x = side == 0 ? lo : hi;
      if (x < at || x >= past) continue;
      const uint32_t first = x - (x - at) % units, to = x == first ? x : snap(x, first, first + units, kItemUnits, slack);
      if (side == 0) {
        share_s->lo = to;
        share_s->at = at;
        share_s->b = b;
        share_s->qt = qt;
      } else {
        share_s->hi = to;
      }
    }
    at = past;
  };
  if (i1 - i0 == 1) cut(b_last, qt_last, units_last);   // most schedules: nothing to walk again
  else run(cut);
}

// Four products of one 64-wide piece of the inner axis, in one statement: every descriptor is in a register
// before the first, so that the issuing warp, which shares its scheduler with softmax warps, waits for one
// slot a product and not for its descriptor arithmetic.  The whole warp comes here together; the lane with
// `go` set issues, by predicate and not by branch, so that the warp never parts.
// D[tmem] (+)= A[smem] B[smem]^T, both K-major in the 128-byte swizzle: 32 bytes a step.
__device__ __forceinline__ void tc_mma4_ss(uint32_t go, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\tsetp.ne.b32 p, %10, 0;\n\tsetp.ne.b32 t, %11, 0;\n\tsetp.ne.b32 e, %12, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %5, %9, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %2, %6, %9, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %3, %7, %9, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %4, %8, %9, t;\n\t}" ::"r"(d),
      "l"(a), "l"(a + 2u), "l"(a + 4u), "l"(a + 6u), "l"(b), "l"(b + 2u), "l"(b + 4u), "l"(b + 6u), "r"(idesc), "r"(acc),
      "r"(1u), "r"(go)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: A 16-bit pairs in tensor memory (8 columns a step), B as desc_values (2048
// bytes a step).
__device__ __forceinline__ void tc_mma4_ts(uint32_t go, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\tsetp.ne.b32 p, %10, 0;\n\tsetp.ne.b32 t, %11, 0;\n\tsetp.ne.b32 e, %12, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %5, %9, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %6, %9, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %7, %9, t;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %8, %9, t;\n\t}" ::"r"(d),
      "r"(a), "r"(a + 8u), "r"(a + 16u), "r"(a + 24u), "l"(b), "l"(b + 128u), "l"(b + 256u), "l"(b + 384u), "r"(idesc),
      "r"(acc), "r"(1u), "r"(go)
      : "memory");
}
// tc_commit by the lane with `go` set.
__device__ __forceinline__ void tc_commit_if(uint32_t go, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(go)
      : "memory");
}

// Descriptor of a value tile as the B operand with the output dims as its major axis: rows of 64 dims
// (128 B, swizzled), positions 128 B apart, eight of them to the next group of 1024 B, the next 64 dims
// kBoxBytes away.
__device__ __forceinline__ uint64_t desc_values(uint32_t saddr, uint32_t box_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(box_bytes >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

#define R16(v, o)                                                                                                  \
  "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]),      \
      "=r"(v[o + 7]), "=r"(v[o + 8]), "=r"(v[o + 9]), "=r"(v[o + 10]), "=r"(v[o + 11]), "=r"(v[o + 12]),           \
      "=r"(v[o + 13]), "=r"(v[o + 14]), "=r"(v[o + 15])

// 32 consecutive columns of this thread's row.
__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t (&r)[32]) {
  asm volatile(
      "{\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t}"
      : R16(r, 0), R16(r, 16)
      : "r"(t)
      : "memory");
}

// All 128 columns of S: four loads and one wait in one statement.
__device__ __forceinline__ void tmem_ld128(uint32_t t, uint32_t (&r)[128]) {
  asm volatile(
      "{\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,"
      "%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%129];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,"
      "%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95}, [%130];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,"
      "%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%131];\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t}"
      : R16(r, 0), R16(r, 16), R16(r, 32), R16(r, 48), R16(r, 64), R16(r, 80), R16(r, 96), R16(r, 112)
      : "r"(t), "r"(t + 32u), "r"(t + 64u), "r"(t + 96u)
      : "memory");
}
#undef R16

#define I16(v, o)                                                                                                  \
  "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]),             \
      "r"(v[o + 7]), "r"(v[o + 8]), "r"(v[o + 9]), "r"(v[o + 10]), "r"(v[o + 11]), "r"(v[o + 12]), "r"(v[o + 13]), \
      "r"(v[o + 14]), "r"(v[o + 15])
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      I16(v, 0)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      I16(v, 0), I16(v, 16)
      : "memory");
}
#undef I16
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void ld_shared4(uint32_t at, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(at) : "memory");
}
// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Pairs of fp32 values in one register pair.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 unpair2(uint64_t v) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// The lowest n bits (n any integer).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// Bit 15 of each half of w that holds a non-finite value (an exponent of ones, which one more carries into
// the sign's place).
template <bool FP16>
__device__ __forceinline__ uint32_t non_finite_bits(uint32_t w) {
  return FP16 ? (w & 0x7C007C00u) + 0x04000400u : (w & 0x7F807F80u) + 0x00800080u;
}
constexpr uint32_t kSigns = 0x80008000u;

// 0xFFFF in each half of w that holds a non-finite value.
template <bool FP16>
__device__ __forceinline__ uint32_t non_finite16(uint32_t w) {
  const uint32_t mask = FP16 ? 0x7C007C00u : 0x7F807F80u;
  return __vcmpeq2(w & mask, mask);
}

// What the rows that see non-finite values add to dims d0 .. d0 + 15 of their result: the sum of those
// values over the positions that the row sees in this segment's masked tiles.
template <bool FP16>
__device__ __noinline__ void add_non_finite(const PagedArgs& a, const int32_t* table, TileRange r, int i0, int n, int p_lo,
                                            int p_hi, int p, int g, int d0, float* acc) {
  for (int i = i0; i < i0 + n; ++i) {
    const int j0 = r.tile(i) * kTN;
    if (tile_open<kTN>(a, j0, p_lo, p_hi)) continue;
    for (int j = j0; j < j0 + kTN; ++j) {
      if (!paged_sees(a, p, j)) continue;
      const int page = table[j >> a.page_shift];
      if (page < 0 || page >= a.num_pages) continue;
      const uint16_t* v = a.vc + page * a.page_stride + g * a.head_stride + (j & ((1 << a.page_shift) - 1)) * a.row_stride + d0;
      for (int e = 0; e < 16; e += 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(v + e), bad = non_finite16<FP16>(w);
        const float2 x = unpack16<FP16>(w);
        if (bad & 0xFFFFu) acc[e] += x.x;
        if (bad >> 16) acc[e + 1] += x.y;
      }
    }
  }
}

// A row's scores of the tile at position j0 that the token at position p does not see become -infinity.  Masked where
// they lie, 32 positions at a time, before they are loaded: visible is j <= p, and j > p - window or j < sinks.  (A short
// loop: unrolled over the loaded scores the masks were ~6 KB of instructions that every masked tile fetched anew, 1,000
// to 2,600 cycles.)
__device__ __forceinline__ void mask_scores(const PagedArgs& a, uint32_t tS, int p, int j0) {
  auto seen = [&](int j) {
    const uint32_t see = low_bits(p + 1 - j);
    return a.window > 0 ? see & (~low_bits(p - a.window + 1 - j) | low_bits(a.sinks - j)) : see;
  };
  uint32_t words = 0;   // those that some row of the warp does not wholly see: few, as its rows are few tokens
#pragma unroll
  for (int w = 0; w < 4; ++w) words |= __all_sync(0xFFFFFFFFu, seen(j0 + 32 * w) == 0xFFFFFFFFu) ? 0u : 1u << w;
#pragma unroll 1
  while (words != 0) {
    const int c = 32 * (__ffs(words) - 1);
    words &= words - 1;
    const uint32_t see = seen(j0 + c);
    uint32_t v[32] = {};
    if (__any_sync(0xFFFFFFFFu, see != 0u)) tmem_ld32(tS + c, v);
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = see & (1u << e) ? v[e] : 0xFF800000u;
    tmem_st32(tS + c, v);
  }
  tmem_wait_st();
}

// O of this thread's row times `by`.
template <int D>
__device__ __forceinline__ void rescale(uint32_t tO, float by) {
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t v[16];
    tmem_ld16_wait(tO + c, v);
#pragma unroll
    for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * by);
    tmem_st16(tO + c, v);
  }
}

// Softmax of tiles i .. n - 1 of a segment (the first one's scores are there, masked) for a warp with a row beyond kFar:
// numerators 2^((s - m) scale + kLift), 32 scores at a time.  Apart from the other tiles' loop: with the subtraction on a
// path of its own in there, 2048 tokens at 32768 took 348 us and at 64 dims 277, so 339 and 270.  done < 0: a wait timed out.
struct FarRow {
  float m, l;
  int done;
};
template <int D, bool FP16>
__device__ __noinline__ FarRow far_tiles(const PagedArgs& a, Item x, int i0, int i, int n, int p, uint32_t tS, uint32_t tO,
                                         uint32_t sfull, int done, uint32_t pfull, volatile int* abort_s, float m, float l) {
  for (bool waited = true; i < n; ++i, waited = false) {
    if (!waited) {
      const int j0 = x.r.tile(i0 + i) * kTN;
      if (!mbar_wait_warp(sfull, done & 1, abort_s, a.err)) return FarRow{m, l, -1};
      ++done;
      tc_fence_after();
      if (!tile_open<kTN>(a, j0, x.p_lo, x.p_hi)) mask_scores(a, tS, p, j0);
    }
    float mx = -INFINITY, alpha = 1.f, sum = 0.f;
    __syncwarp();
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      uint32_t v[32];
      tmem_ld32(tS + c, v);
#pragma unroll
      for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(v[e]));
    }
    if (mx > m && (m == -INFINITY || (mx - m) * a.qk_scale > kLazy<FP16>)) {
      alpha = ex2((m - mx) * a.qk_scale);   // 0 if nothing was seen before
      m = mx;
      l *= alpha;
    }
    const float ref = m == -INFINITY ? 0.f : m;
    __syncwarp();
    if (i > 0) rescale<D>(tO, alpha);
    // (numerators of 32 scores take the place of the 16 before them, which have been read)
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      uint32_t v[32], pk[16];
      tmem_ld32(tS + c, v);
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const float p0 = ex2(fmaf(__uint_as_float(v[e]) - ref, a.qk_scale, kLift<FP16>));
        const float p1 = ex2(fmaf(__uint_as_float(v[e + 1]) - ref, a.qk_scale, kLift<FP16>));
        sum += p0 + p1;
        pk[e / 2] = pack16<FP16>(p0, p1);
      }
      tmem_st16(tS + c / 2, pk);
      if (c == 32 || c == 96) {
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(pfull + 8u * (c / 64));
        __syncwarp();
      }
    }
    l += sum;
  }
  return FarRow{m, l, done};
}

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ PagedMaps maps, const PagedArgs a, const ChunkSplit split) {
  using C = Chunk<D>;
  extern __shared__ uint8_t sm_raw[];
  // barriers: stages (full, empty), q (full, empty), per row tile S full, P
  // full (its first and its second half), O full, O empty; values clean (a stage each)
  __shared__ __align__(8) uint64_t bars[3 * C::kStages + 2 + 8 + 2];
  __shared__ uint32_t warp_s[kThreads / 32];
  __shared__ Share share_s;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  __shared__ int bad_s[4];   // segment + 1 whose values had non-finite ones that a row sees
  const uint32_t raw = smem_u32(sm_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t sQ = base, sKV = base + 2 * C::kTileBytes;
  const uint32_t sOut = sKV + C::kStages * C::kStageBytes;
  uint32_t* pre_s = reinterpret_cast<uint32_t*>(sm_raw + (sOut - raw) + kSoftmaxWarps * kOutBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto FULL = [&](int s) { return bar0 + 8u * s; };
  auto EMPTY = [&](int s) { return bar0 + 8u * (C::kStages + s); };
  constexpr int kB = 2 * C::kStages;
  const uint32_t QFULL = bar0 + 8u * kB, QEMPTY = QFULL + 8u;
  auto SFULL = [&](int t) { return bar0 + 8u * (kB + 2 + t); };
  auto PFULL = [&](int t, int part) { return bar0 + 8u * (kB + 4 + 2 * t + part); };
  auto OFULL = [&](int t) { return bar0 + 8u * (kB + 8 + t); };
  auto OEMPTY = [&](int t) { return bar0 + 8u * (kB + 10 + t); };
  auto CLEAN = [&](int s) { return bar0 + 8u * (kB + 12 + s); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = (int)blockIdx.x;
  const int tpt = 128 / a.G, tokens = 2 * tpt;

  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), 1 + kScanWarps);
      mbar_init(CLEAN(s), kScanWarps);
    }
    mbar_init(QFULL, 1);
    mbar_init(QEMPTY, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(SFULL(t), 1);
      mbar_init(PFULL(t, 0), 4);
      mbar_init(PFULL(t, 1), 4);
      mbar_init(OFULL(t), 1);
      mbar_init(OEMPTY(t), 4);
    }
    abort_s = 0;
    for (int i = 0; i < 4; ++i) bad_s[i] = 0;
    share_s.lo = share_s.hi = 0;
    mbar_fence_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
  }
  if (warp == kSoftmaxWarps + 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();

  bool bad = false;
  find_share(a, tokens, pre_s, warp_s, &share_s, bad);
  if (bad && cta == 0) raise_flag(a.err, kErrBadPages);
  if (tid == 0) split.rec[cta].until = split.rec[cta].first = -1;
  // Lanes part ways in the schedule (and below, wherever a lane's own data decides).  Every such place ends in
  // __syncwarp before the warp's next collective instruction (barriers, tensor-memory loads and stores): those
  // assume a converged warp, which a join of branches alone does not promise.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // Walks the segments of the share: body(b, s, g, item, i0, n, u) for tiles i0 .. i0 + n - 1 of an item,
  // the first of them unit u; stops when the body returns false.
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
          if (!body(b, s, g, x, i0, i1 - i0, u)) return;
          u = min(hi, at + units);
        }
      }
      qt = 0;
      ++b;
    }
  };

  if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kSoftmaxWarps) {
      // ---- copies
      const int ppt_shift = 7 - a.page_shift, ppt = 1 << ppt_shift, box_rows = 1 << a.page_shift;   // pages of a tile
      const int batch = 32 >> ppt_shift;                              // tiles whose page numbers the lanes hold
      int at = 0, items = 0;   // ring stages and segments so far
      bad = false;
      walk([&](int b, const SeqRows& s, int g, const Item& x, int i0, int n, uint32_t) {
        const bool two = x.n > tpt;
        const int32_t* row = a.table + (size_t)b * a.max_pages;
        const int sub = lane / C::kBoxes, box = lane % C::kBoxes;   // one copy a lane: (page of the tile, 64-dim box)
        // Page numbers of a batch of tiles, one a lane, read one batch ahead; a page that no row needs is not
        // read, and takes, like a bad one, a number out of the map's range, which reads as zeros.
        int pg = 0, ahead = 0;
        bool need = false;
        auto read_ahead = [&](int i) {
          const int t = i0 + i + (lane >> ppt_shift);
          const int ip = t < x.r.count ? (x.r.tile(t) << ppt_shift) + (lane & (ppt - 1)) : 0;
          need = (lane >> ppt_shift) < n - i && t < x.r.count && ip < a.max_pages && page_needed(a, ip, x.p_lo, x.p_hi);
          if (need) ahead = row[ip];
        };
        read_ahead(0);
        for (int i = 0; i <= n; ++i, ++at) {
          // stage `at`: values of tile i - 1 (whose pages are at hand), then keys of tile i
          const int st = at & 1;
          if (at >= C::kStages && !mbar_wait_warp(EMPTY(st), (at / C::kStages - 1) & 1, &abort_s, a.err)) return false;
          if (lane == 0) mbar_arrive_expect_tx(FULL(st), i == 0 || i == n ? C::kTileBytes : 2 * C::kTileBytes);
          __syncwarp();
          auto copy = [&](const CUtensorMap* map, int half, int in) {
            const int p = __shfl_sync(0xFFFFFFFFu, pg, (in * ppt + sub) & 31);
            if (lane < ppt * C::kBoxes)
              tma_load_4d(sKV + st * C::kStageBytes + half * C::kTileBytes + box * C::kBoxBytes + sub * box_rows * 128, map,
                          FULL(st), box * 64, 0, g, p);
            __syncwarp();
          };
          if (i > 0) copy(&maps.v, 1, (i - 1) & (batch - 1));
          if (i < n) {
            const int in = i & (batch - 1);
            if (in == 0) {
              const bool ok = ahead >= 0 && ahead < a.num_pages;
              pg = need && ok ? ahead : a.num_pages;
              bad |= need && !ok;
              read_ahead(i + batch);
            }
            copy(&maps.k, 0, in);
          }
          if (i == 0) {   // the queries, once the segment before has done its last scores
            if (items > 0 && !mbar_wait_warp(QEMPTY, (items - 1) & 1, &abort_s, a.err)) return false;
            ++items;
            if (lane == 0) {
              const uint32_t bytes = (uint32_t)(64 * 2 * a.G * tpt);
              mbar_arrive_expect_tx(QFULL, bytes * C::kBoxes * (two ? 2 : 1));
              for (int t = 0; t < (two ? 2 : 1); ++t)
                for (int bx = 0; bx < C::kBoxes; ++bx)
                  tma_load_3d(sQ + t * C::kTileBytes + bx * C::kBoxBytes, &maps.q, QFULL, bx * 64, g * a.G,
                              s.row0 + x.t0 + t * tpt);
            }
            __syncwarp();
          }
        }
        return true;
      });
      if (bad) raise_flag(a.err, kErrBadPages);
    } else if (warp == kSoftmaxWarps + 1) {
      // ---- tensor-core instructions.  The whole warp takes every step, one elected lane issues (by predicate), and
      // row tile and ring stage are constants of the unrolled code: descriptors and addresses then sit in uniform
      // registers, and a product costs one issue slot beside the two softmax warps of this scheduler.  (A
      // single lane's walk with computed descriptors took twice as long per product under that load.)
      const uint32_t go = elect_one() ? 1u : 0u;
      constexpr uint32_t fmt = FP16 ? 0u : ((1u << 7) | (1u << 10));
      constexpr uint32_t id_s = (1u << 4) | fmt | ((kTN >> 3) << 17) | ((128u >> 4) << 24);
      constexpr uint32_t id_o = (1u << 4) | fmt | (1u << 16) | (((uint32_t)D >> 3) << 17) | ((128u >> 4) << 24);
      constexpr uint32_t kTileUnits = C::kTileBytes >> 4, kBoxUnits = C::kBoxBytes >> 4;   // descriptors count 16 bytes
      const uint64_t dq = smem_desc_sw128(sQ), dk = smem_desc_sw128(sKV), dv = desc_values(sKV + C::kTileBytes, C::kBoxBytes);
      uint32_t at = 0, items = 0, cleans[2] = {0, 0}, done0 = 0, done1 = 0, outs0 = 0, outs1 = 0;
      auto wait = [&](uint32_t bar, uint32_t phase) { return mbar_wait_warp(bar, phase & 1, &abort_s, a.err); };
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
        if (!wait(QFULL, items++)) return false;
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
          const bool more = i + 1 < n;
          const bool closed = !tile_open<kTN>(a, x.r.tile(i0 + i) * kTN, x.p_lo, x.p_hi);
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
      // ---- values of masked tiles: non-finite ones are taken out, two positions a thread.  (Beside the softmax,
      // which would spend 700 cycles of its chain on it, twice: one row tile's product would also wait for the other's.)
      // These warps see every stage, and a stage is free only with their word, so that they keep step with the ring.
      // Their word that a tile is done goes to its stage's own barrier: a stage is filled again only after both of them and the
      // product have left it, so neither can speak twice there before the other has spoken, nor twice before the product's
      // warp has looked.  (One barrier for all tiles would count a quick warp's two tiles as both warps' first.)
      uint32_t at = 0;
      int seg = 0;
      walk([&](int, const SeqRows&, int, const Item& x, int i0, int n, uint32_t) {
        for (int i = 0; i <= n; ++i, ++at) {
          const uint32_t st = at & 1;
          if (!mbar_wait_warp(FULL(st), (at >> 1) & 1, &abort_s, a.err)) return false;
          const int j0 = i > 0 ? x.r.tile(i0 + i - 1) * kTN : 0;
          if (i > 0 && !tile_open<kTN>(a, j0, x.p_lo, x.p_hi)) {
  #pragma unroll 1
            for (int r = (warp - kSoftmaxWarps - 2) * 32 + lane; r < kTN; r += kScanWarps * 32) {
              const uint32_t row = sKV + st * C::kStageBytes + C::kTileBytes + r * 128;
              uint32_t any = 0;
  #pragma unroll 8
              for (int c = 0; c < 8 * C::kBoxes; ++c) {   // of 16 bytes; lanes start at different ones
                uint32_t w0, w1, w2, w3;
                ld_shared4(row + (c >> 3) * C::kBoxBytes + (((c + lane) & 7) << 4), w0, w1, w2, w3);
                any |= non_finite_bits<FP16>(w0) | non_finite_bits<FP16>(w1) | non_finite_bits<FP16>(w2) |
                       non_finite_bits<FP16>(w3);
              }
              if (any & kSigns) {
  #pragma unroll 1
                for (int c = 0; c < 8 * C::kBoxes; ++c) {
                  const uint32_t to = row + (c >> 3) * C::kBoxBytes + ((c & 7) << 4);
                  uint32_t w0, w1, w2, w3;
                  ld_shared4(to, w0, w1, w2, w3);
                  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(w0 & ~non_finite16<FP16>(w0)),
                               "r"(w1 & ~non_finite16<FP16>(w1)), "r"(w2 & ~non_finite16<FP16>(w2)),
                               "r"(w3 & ~non_finite16<FP16>(w3))
                               : "memory");
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
    }
  } else {
    // ---- softmax: row `r` of row tile `t`
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, r = (warp & 3) * 32 + lane, tok = r / a.G, head = r - tok * a.G;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = t * 128 + lanes, tO = kTmemO + t * 128 + lanes;
    int seg = 0, done = 0, outs = 0;   // segments, own tiles and items so far
    walk([&](int b, const SeqRows& s, int g, const Item& x, int i0, int n, uint32_t u) {
      const int nt = x.n > tpt ? 2 : 1;
      if (t >= nt) {
        ++seg;
        return true;
      }
      const bool live = tok < tpt && t * tpt + tok < x.n;
      const int p = live ? x.p_lo + t * tpt + tok : -1;      // a row that is no token sees nothing
      float m = -INFINITY, negm = 0.f, l = 0.f;              // negm = kLift - m in base-2 units (0 while nothing is seen)
      for (int i = 0; i < n; ++i) {
        const int j0 = x.r.tile(i0 + i) * kTN;
        const bool open = tile_open<kTN>(a, j0, x.p_lo, x.p_hi);
        if (!mbar_wait_warp(SFULL(t), done & 1, &abort_s, a.err)) return false;
        ++done;
        tc_fence_after();
        if (!open) mask_scores(a, tS, p, j0);
        uint32_t sr[128];
        tmem_ld128(tS, sr);
        float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
        for (int c = 0; c < 128; c += 8) {
          mx0 = max3(mx0, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
          mx1 = max3(mx1, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
          mx2 = max3(mx2, __uint_as_float(sr[c + 4]), __uint_as_float(sr[c + 5]));
          mx3 = max3(mx3, __uint_as_float(sr[c + 6]), __uint_as_float(sr[c + 7]));
        }
        const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
        // The reference moves if the new maximum is well above it (or is the first).
        const bool move = mx > m && (m == -INFINITY || (mx - m) * a.qk_scale > kLazy<FP16>);
        if (__any_sync(0xFFFFFFFFu, move)) {
          if (__any_sync(0xFFFFFFFFu, move && p >= 0 && fabsf(mx) * a.qk_scale > kFar)) {   // the tiles from here on in another way
            const FarRow row = far_tiles<D, FP16>(a, x, i0, i, n, p, tS, tO, SFULL(t), done, PFULL(t, 0), &abort_s, m, l);
            if (row.done < 0) return false;
            m = row.m;
            l = row.l;
            done = row.done;
            negm = kLift<FP16> - m * a.qk_scale;
            break;
          }
          float alpha = 1.f;
          if (move) {
            const float nn = kLift<FP16> - mx * a.qk_scale;
            alpha = m == -INFINITY ? 0.f : ex2(nn - negm);
            m = mx;
            negm = nn;
            l *= alpha;
          }
          __syncwarp();
          if (i > 0) rescale<D>(tO, alpha);
        }
        const uint64_t scale2 = pair2(a.qk_scale, a.qk_scale), negm2 = pair2(negm, negm);
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
            pk[e / 2] = pack16<FP16>(p0, p1);
            pk[e / 2 + 1] = pack16<FP16>(p2, p3);
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
      if (!mbar_wait_warp(OFULL(t), outs & 1, &abort_s, a.err)) return false;
      ++outs;
      tc_fence_after();
      const bool whole = i0 == 0 && n == x.r.count;
      if (*(volatile int*)&bad_s[my_seg & 3] == my_seg + 1) {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t v[16];
          float extra[16];
          tmem_ld16_wait(tO + c, v);
#pragma unroll
          for (int e = 0; e < 16; ++e) extra[e] = 0.f;
          if (live) add_non_finite<FP16>(a, a.table + (size_t)b * a.max_pages, x.r, i0, n, x.p_lo, x.p_hi, p, g, c, extra);
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + extra[e]);
          tmem_st16(tO + c, v);
          tmem_wait_st();
        }
      }
      __syncwarp();
      // (O of a row that sees nothing is 0: its tiles are masked.)
      const float inv = p < 0 ? 0.f : 1.f / l;
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
      uint64_t check0 = 0, check1 = 0;   // 0 unless a result is not finite: the sums of 0 times every one
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        tmem_ld32(tO + c, v);
        if (whole) {
#pragma unroll
          for (int e = 0; e < 16; e += 2) {   // pairs 2 e, 2 e + 2 become words e, e + 1
            const uint64_t f0 = mul2(pair2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), inv2);
            const uint64_t f1 = mul2(pair2(__uint_as_float(v[2 * e + 2]), __uint_as_float(v[2 * e + 3])), inv2);
            check0 = fma2(f0, 0ull, check0);
            check1 = fma2(f1, 0ull, check1);
            const float2 y0 = unpair2(f0), y1 = unpair2(f1);
            v[e] = pack16<FP16>(y0.x, y0.y);
            v[e + 1] = pack16<FP16>(y1.x, y1.y);
          }
          // 64 bytes a row through shared memory (16-byte pieces XOR-ed against bank conflicts), so that a store
          // touches 8 rows, not 32.
#pragma unroll
          for (int e = 0; e < 4; ++e)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(out + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)),
                         "r"(v[4 * e]), "r"(v[4 * e + 1]), "r"(v[4 * e + 2]), "r"(v[4 * e + 3])
                         : "memory");
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
            *reinterpret_cast<uint4*>(part + (c + e) * kItemRows) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(OEMPTY(t));
      const float2 checks = unpair2(add2(check0, check1));
      if (live && !(checks.x + checks.y == 0.f)) raise_flag(a.err, kErrNonFinite);
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
  // After a timeout, copies and products still in flight finish before the CTA gives up its memory.
  if (tid == 0 && *(volatile int*)&abort_s) {
    const long long c0 = clock64();
    while (clock64() - c0 < 4000000ll) {
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem_slot, 512);
  }
}

// Joins the parts of the split items, a row a lane.  Few parts, which is most items: block y of the CTA that began the
// item takes rows 32 y .. 32 y + 31, a warp a quarter of the dims, all parts in order.  Many (one sequence's few
// rows are cut into as many parts as there are SMs for its heads): the blocks of all its CTAs but the last share
// the pairs of 32 rows and an eighth of the dims, a warp takes every fourth part, and the warps' results are
// joined in order through shared memory.  Bound by latency (a launch, the record, the parts from L2), so what
// counts is loads in flight (119 registers: with at most 64, a prompt of 2048 took 40 us, not 31): 2 us of a graph where
// nothing is split, 3 where a window chunk's 64 cuts are.  8 tokens behind 32768 positions, 76 parts a head: 25 us in
// all (22 with the cache in L2, and joined as few 73).  `Many` begins at 6: at 4, 512 tokens behind 8192 take 45 us, not
// 40; at 10, 256 take 30, not 29.
constexpr int kJoinWarps = 4;
constexpr int kJoinMany = 6;   // parts

template <int D, bool FP16>
__global__ void __launch_bounds__(kJoinWarps * 32) chunk_join_kernel(const PagedArgs a, const ChunkSplit split) {
  using C = Chunk<D>;
  constexpr int kFewDims = D / 4, kManyDims = D / 8;
  __shared__ float acc_s[kJoinWarps][kManyDims][32], m_s[kJoinWarps][32], l_s[kJoinWarps][32];
  pdl_wait();
  pdl_launch_dependents();
  SplitRecord rec = load_record(split.rec + blockIdx.x);
  const int first = rec.first;
  if (first < 0) return;
  if (first != (int)blockIdx.x) rec = load_record(split.rec + first);
  const int n = rec.until - first + 1;
  if (first != (int)blockIdx.x && n < kJoinMany) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tpt = 128 / a.G;
  auto part = [&](int c) { return split.part + ((size_t)c * 2 + (c == first ? 1 : 0)) * C::kPartFloats; };

  // Parts c0, c0 + S, ... of a row's N dims from d on: K at a time, everything of them in flight at once.
  float M, L;
  auto sum_parts = [&](auto n_c, auto k_c, float* acc, int c0, int S, int d, int slot) {
    constexpr int N = decltype(n_c)::value, K = decltype(k_c)::value;
    M = kUnseen;
    L = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.f;
    for (int c = c0; c <= rec.until; c += K * S) {
      // (a part past the last is read as the first and weighs nothing: loads without branches)
      float m[K], l[K];
      float4 o[K][N / 4];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float* p = part(c + k * S <= rec.until ? c + k * S : c);
        m[k] = __ldcg(p + D * kItemRows + slot);
        l[k] = __ldcg(p + (D + 1) * kItemRows + slot);
#pragma unroll
        for (int e = 0; e < N / 4; ++e) o[k][e] = __ldcg(reinterpret_cast<const float4*>(p + (d + 4 * e) * kItemRows) + slot);
      }
#pragma unroll
      for (int k = 1; k < K; ++k)
        if (c + k * S > rec.until) {
          m[k] = kUnseen;
          l[k] = 0.f;
#pragma unroll
          for (int e = 0; e < N / 4; ++e) o[k][e] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      float top = M;
#pragma unroll
      for (int k = 0; k < K; ++k) top = fmaxf(top, m[k]);
      const float w = exp2f(M - top);
      M = top;
      L *= w;
#pragma unroll
      for (int e = 0; e < N; ++e) acc[e] *= w;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float x = exp2f(m[k] - top);
        L += l[k] * x;
#pragma unroll
        for (int e = 0; e < N / 4; ++e) {
          acc[4 * e] += o[k][e].x * x;
          acc[4 * e + 1] += o[k][e].y * x;
          acc[4 * e + 2] += o[k][e].z * x;
          acc[4 * e + 3] += o[k][e].w * x;
        }
      }
    }
  };
  // The row's result for N dims from d on, of unnormalised values `v` and their sum.
  auto store = [&](auto n_c, const float* v, float sum, int d, int slot) {
    constexpr int N = decltype(n_c)::value;
    const int t = slot >> 7, r = slot & 127, tok = r / a.G;
    const float inv = rec.p_lo + t * tpt + tok < 0 ? 0.f : 1.f / sum;   // a row before position 0 sees nothing
    bool nonfinite = false;
    uint32_t w[N / 2];
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float x = v[e] * inv, y = v[e + 1] * inv;
      nonfinite |= !isfinite(x) || !isfinite(y);
      w[e / 2] = pack16<FP16>(x, y);
    }
    if (nonfinite) raise_flag(a.err, kErrNonFinite);
    uint16_t* o = a.o + (long long)(rec.row + t * tpt + tok) * a.o_stride + (long long)(rec.g * a.G + r % a.G) * D + d;
    if constexpr (N >= 8) {
#pragma unroll
      for (int e = 0; e < N / 8; ++e)
        *reinterpret_cast<uint4*>(o + 8 * e) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
    } else {
#pragma unroll
      for (int e = 0; e < N / 2; ++e) *reinterpret_cast<uint32_t*>(o + 2 * e) = w[e];
    }
  };
  auto is_live = [&](int slot) {
    const int t = slot >> 7, tok = (slot & 127) / a.G;
    return tok < tpt && t * tpt + tok < rec.rows;
  };

  using Two = std::integral_constant<int, 2>;
  using Four = std::integral_constant<int, 4>;
  if (n < kJoinMany) {
    using Dims = std::integral_constant<int, kFewDims>;
    const int slot = (int)blockIdx.y * 32 + lane;
    if (!is_live(slot)) return;
    float acc[kFewDims];
    sum_parts(Dims{}, Two{}, acc, first, 1, warp * kFewDims, slot);
    store(Dims{}, acc, L, warp * kFewDims, slot);
    return;
  }
  using Dims = std::integral_constant<int, kManyDims>;
  const int slots = rec.rows <= tpt ? rec.rows * a.G : 128 + (rec.rows - tpt) * a.G;   // up to the last token's
  const int blocks = (n - 1) * (int)gridDim.y;
  for (int x = ((int)blockIdx.x - first) * (int)gridDim.y + (int)blockIdx.y; x < (slots + 31) / 32 * 8; x += blocks) {
    const int slot = (x >> 3) * 32 + lane, d = (x & 7) * kManyDims;
    const bool live = is_live(slot);
    if (live) {
      float acc[kManyDims];
      sum_parts(Dims{}, Four{}, acc, first + warp, kJoinWarps, d, slot);
#pragma unroll
      for (int e = 0; e < kManyDims; ++e) acc_s[warp][e][lane] = acc[e];
      m_s[warp][lane] = M;
      l_s[warp][lane] = L;
    }
    __syncwarp();
    __syncthreads();
    if (live) {
      constexpr int N = kManyDims / kJoinWarps;   // this warp's dims
      float top = m_s[0][lane], sum = 0.f, y[N];
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = 0.f;
#pragma unroll
      for (int k = 1; k < kJoinWarps; ++k) top = fmaxf(top, m_s[k][lane]);
#pragma unroll
      for (int k = 0; k < kJoinWarps; ++k) {
        const float w = exp2f(m_s[k][lane] - top);
        sum += l_s[k][lane] * w;
#pragma unroll
        for (int e = 0; e < N; ++e) y[e] += acc_s[k][warp * N + e][lane] * w;
      }
      store(std::integral_constant<int, N>{}, y, sum, d + warp * N, slot);
    }
    __syncwarp();
    __syncthreads();   // before acc_s is written again
  }
}

template <int D, bool FP16>
cudaError_t launch(const PagedMaps& maps, const PagedArgs& a, const ChunkSplit& split, int ctas, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(chunk_kernel<D, FP16>), (int)Chunk<D>::smem(kPagedMaxSeqs), &ready);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Chunk<D>::smem(a.B);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, chunk_kernel<D, FP16>, maps, a, split);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(ctas, kItemRows / 32);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<D, FP16>, a, split);
}

}  // namespace

size_t paged_chunk_scratch(int D, int ctas) {
  return (size_t)ctas * (2 * (size_t)kItemRows * (D + 2) * sizeof(float) + sizeof(SplitRecord));
}

cudaError_t launch_paged_chunk(const PagedMaps& maps, const PagedArgs& a, int D, void* scratch, int ctas, cudaStream_t st) {
  ChunkSplit split;
  split.part = static_cast<float*>(scratch);
  split.rec = reinterpret_cast<SplitRecord*>(split.part + (size_t)ctas * 2 * kItemRows * (D + 2));
  if (D == 128) return a.fp16 ? launch<128, true>(maps, a, split, ctas, st) : launch<128, false>(maps, a, split, ctas, st);
  return a.fp16 ? launch<64, true>(maps, a, split, ctas, st) : launch<64, false>(maps, a, split, ctas, st);
}

}  // namespace moe
