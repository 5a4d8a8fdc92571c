// What the chunk forms of the paged attention share: rows and row tiles, the split of the work, tensor-core and
// tensor-memory helpers, masks (paged_chunk.cu says how they are used).
#pragma once

#include <type_traits>

#include "paged.cuh"

namespace moe {
namespace {

constexpr int kTN = 128;                    // positions per cache tile
constexpr int kSoftmaxWarps = 8;
constexpr int kItemRows = 256;              // two row tiles
constexpr uint32_t kTmemO = 256;            // columns: S0 0, S1 128, O0 256, O1 384 (all 512 are allocated: base 0)
constexpr int kOutBytes = 32 * 64;          // a warp's staging of its 32 rows of o, 32 dims at a time
constexpr int kItemUnits = 2;               // what an item costs beside its tiles, in tiles (~5,000 cycles)

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
template <int NT>
__device__ __forceinline__ void find_share(const PagedArgs& a, int tokens, uint32_t* pre_s, uint32_t* warp_s,
                                           Share* share_s, bool& bad) {
  const int tid = threadIdx.x, cta = (int)blockIdx.x;
  bool over;
  const uint32_t blocks = scan_sequences<NT>(a.B, pre_s, warp_s, &over, [&](int b) {
    return (uint32_t)(load_seq(a, b, bad).n + tokens - 1) / (uint32_t)tokens;
  });
  if (over) {
    bad = true;
    return;
  }
  const uint32_t per = (blocks + NT - 1) / NT;
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
  uint32_t at = exclusive_scan<NT>(mine, warp_s, &total, &over);
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

}  // namespace
}  // namespace moe
