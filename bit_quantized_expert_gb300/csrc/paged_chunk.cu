// Attention of chunks of new tokens over the paged cache (contract in include/gqa_paged.h), on the
// fifth-generation tensor cores.
//
//   * Rows.  The G query heads of a key/value head share its cache, so a 128-row operand tile holds
//     floor(128 / G) tokens, each with its G heads (row = token * G + head): one tensor-map box of q.  An
//     item is two such tiles of one key/value head of one sequence, and walks the cache tiles (128
//     positions) that its rows see.
//   * Work split.  Shares of the cache tiles of all items, one per SM (paged.cuh).
//   * Roles.  Warps 0..3 and 4..7: softmax of the first and second row tile, one row a thread; warp 8:
//     copies; warp 9: tensor-core instructions; warps 10 and 11 fill the warpgroup (registers are moved to
//     the softmax by warpgroups).  While one row tile's softmax runs, the other's
//     products do:  S0 = Q0 K^T | S1 = Q1 K^T, then per cache tile  O0 += P0 V, S0 = Q0 K'^T,
//     O1 += P1 V, S1 = Q1 K'^T.
//   * S and O stay in tensor memory (128 columns of fp32 a tile each).  P replaces S there, in 16 bits,
//     as the A operand of the second product; V is read as it lies (positions by dims) through a
//     descriptor whose major axis is the output's.
//   * The running maximum that scales the numerators moves only when the new one is above it by 8 in
//     base-2 units: p stays below 2^8, nothing overflows, and O is rescaled in a few tiles, not in all.
//   * Only tiles that some row does not wholly see are masked.  In those, the value tile is also
//     searched for non-finite values, since 0 times one of them is not 0: they are taken out, and the rows that do
//     see them get them back at the end.
#include <cmath>

#include "paged.cuh"

namespace moe {
namespace {

constexpr int kTN = 128;                    // positions per cache tile
constexpr int kThreads = 384;              // two softmax warpgroups, one for copies and products
// Registers a thread: 168 at launch; 2 * 208 + 88 = 3 * 168 after the split.
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
constexpr int kItemRows = 256;              // two row tiles
constexpr uint32_t kTmemO = 256;            // columns: S0 0, S1 128, O0 256, O1 384
constexpr float kLazy = 8.f;                // base-2 units the running maximum may lag behind

template <int D>
struct Chunk {
  static constexpr int kBoxes = D / 64;
  static constexpr int kBoxBytes = kTN * 128;                  // 128 rows of 64 dims
  static constexpr int kTileBytes = kBoxes * kBoxBytes;        // a row tile of q, a tile of keys or of values
  static constexpr int kSlots = 4 * 32768 / kTileBytes;        // ring of key and value tiles
  static constexpr int kPartFloats = kItemRows * (D + 2);      // O by columns, then max, then sum
  static size_t smem(int B) { return 1024 + (size_t)(2 + kSlots) * kTileBytes + ((size_t)B + 1) * 8; }
};

struct ChunkSplit {
  float* part;         // [ctas][2][kPartFloats]
  SplitRecord* rec;    // [ctas]
};

// One item: tokens t0 .. t0 + n - 1 of a sequence, at positions p_lo .. p_hi.
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

// D[tmem] (+)= A[tmem] B[smem]: A K-major 16-bit pairs in tensor memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
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

// 32 consecutive columns of this thread's row; valid only after tmem_wait_ld, which ties them.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "{\n\ttcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;\n\t}"
      : R16(r, 0), R16(r, 16)
      : "r"(taddr)
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 0xFFFF in each half of w that holds a non-finite value.
template <bool FP16>
__device__ __forceinline__ uint32_t non_finite16(uint32_t w) {
  const uint32_t mask = FP16 ? 0x7C007C00u : 0x7F807F80u;
  return __vcmpeq2(w & mask, mask);
}

// What the rows that see non-finite values add to dims d0 .. d0 + 31 of their result: the sum of those
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
      for (int e = 0; e < 32; e += 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(v + e), bad = non_finite16<FP16>(w);
        const float2 x = unpack16<FP16>(w);
        if (bad & 0xFFFFu) acc[e] += x.x;
        if (bad >> 16) acc[e + 1] += x.y;
      }
    }
  }
}

template <int D, bool FP16>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ PagedMaps maps, const PagedArgs a, const ChunkSplit split) {
  using C = Chunk<D>;
  extern __shared__ uint8_t sm_raw[];
  // barriers: key/value slots (full, empty), q (full, empty), per row tile S full, P full, O full, O empty; second
  // half of the values clean
  __shared__ __align__(8) uint64_t bars[2 * C::kSlots + 2 + 8 + 1];
  __shared__ unsigned long long warp_s[kThreads / 32];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  __shared__ int bad_s[4];   // segment + 1 whose values had non-finite ones that a row sees
  const uint32_t raw = smem_u32(sm_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t sQ = base, sKV = base + 2 * C::kTileBytes;
  unsigned long long* pre_s =
      reinterpret_cast<unsigned long long*>(sm_raw + (base - raw) + (2 + C::kSlots) * C::kTileBytes);
  const uint32_t bar0 = smem_u32(bars);
  auto FULL = [&](int s) { return bar0 + 8u * s; };
  auto EMPTY = [&](int s) { return bar0 + 8u * (C::kSlots + s); };
  constexpr int kB = 2 * C::kSlots;
  const uint32_t QFULL = bar0 + 8u * kB, QEMPTY = QFULL + 8u, CLEAN = bar0 + 8u * (kB + 10);
  auto SFULL = [&](int t) { return bar0 + 8u * (kB + 2 + t); };
  auto PFULL = [&](int t) { return bar0 + 8u * (kB + 4 + t); };
  auto OFULL = [&](int t) { return bar0 + 8u * (kB + 6 + t); };
  auto OEMPTY = [&](int t) { return bar0 + 8u * (kB + 8 + t); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = (int)blockIdx.x;
  const int tpt = 128 / a.G, tokens = 2 * tpt;

  if (tid == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), 1);
    }
    mbar_init(QFULL, 1);
    mbar_init(QEMPTY, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(SFULL(t), 1);
      mbar_init(PFULL(t), 4);
      mbar_init(OFULL(t), 1);
      mbar_init(OEMPTY(t), 4);
    }
    mbar_init(CLEAN, 4);
    abort_s = 0;
    for (int i = 0; i < 4; ++i) bad_s[i] = 0;
    mbar_fence_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's share: units lo .. hi - 1 of (sequence, head, row block, cache tile)
  bool bad = false;
  scan_sequences<kThreads>(a.B, pre_s, warp_s, [&](int b) {
    const SeqRows s = load_seq(a, b, bad);
    unsigned long long sum = 0;
    for (int qt = 0; qt * tokens < s.n; ++qt) sum += item_of(a, s, qt, tokens).r.count;
    return sum * a.Hkv;
  });
  if (bad && cta == 0) raise_flag(a.err, kErrBadPages);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const unsigned long long total = pre_s[a.B];
  const int ctas = (int)min((unsigned long long)gridDim.x, total);   // every share holds a tile
  if (tid == 0) split.rec[cta].until = -1;
  const bool active = cta < ctas;
  const unsigned long long lo = active ? total * cta / ctas : 0, hi = active ? total * (cta + 1) / ctas : 0;

  // Walks the segments of the share: body(b, s, g, item, i0, n, u) for tiles i0 .. i0 + n - 1 of an item,
  // the first of them unit u; stops when the body returns false.
  auto walk = [&](auto&& body) {
    unsigned long long u = lo;
    for (int b = active ? find_sequence(pre_s, a.B, lo) : 0; u < hi; ++b) {
      if (pre_s[b + 1] <= u) continue;
      const SeqRows s = load_seq(a, b, bad);
      const unsigned long long per_head = (pre_s[b + 1] - pre_s[b]) / a.Hkv;
      int g = (int)((u - pre_s[b]) / per_head);
      unsigned long long at = pre_s[b] + g * per_head;   // first unit of the item being looked at
      int qt = 0;
      while (u < hi && g < a.Hkv) {
        const Item x = item_of(a, s, qt, tokens);
        if (at + x.r.count > u) {
          const int i0 = (int)(u - at), n = (int)min((unsigned long long)(x.r.count - i0), hi - u);
          if (!body(b, s, g, x, i0, n, u)) return;
          u += n;
        }
        at += x.r.count;
        if (++qt * tokens >= s.n) {
          qt = 0;
          ++g;
        }
      }
    }
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == 8) {
    // ---- copies
    const int ppt = max(1, kTN >> a.page_shift), box_rows = min(kTN, 1 << a.page_shift);
    const int batch = 32 / ppt;                              // tiles whose page numbers the lanes hold
    int it = 0, items = 0;
    bool stop = false;
    bad = false;
    walk([&](int b, const SeqRows& s, int g, const Item& x, int i0, int n, unsigned long long) {
      const bool two = x.n > tpt;
      if (items > 0 && !mbar_wait_warp(QEMPTY, (items - 1) & 1, &abort_s, a.err)) {
        stop = true;
        return false;
      }
      if (lane == 0) {
        const uint32_t bytes = (uint32_t)(64 * 2 * a.G * tpt);
        mbar_arrive_expect_tx(QFULL, bytes * C::kBoxes * (two ? 2 : 1));
        for (int t = 0; t < (two ? 2 : 1); ++t)
          for (int box = 0; box < C::kBoxes; ++box)
            tma_load_3d(sQ + t * C::kTileBytes + box * C::kBoxBytes, &maps.q, QFULL, box * 64, g * a.G,
                        s.row0 + x.t0 + t * tpt);
      }
      ++items;
      const int32_t* row = a.table + (size_t)b * a.max_pages;
      int pg = 0;
      for (int i = 0; i < n; ++i, ++it) {
        const int in = i % batch;
        if (in == 0) {
          const int t = i0 + i + lane / ppt;
          pg = a.num_pages;                                  // out of the map's range: zeros
          if (t < x.r.count && lane / ppt < n - i) {
            const int ip = ((x.r.tile(t) * kTN) >> a.page_shift) + lane % ppt;
            if (ip < a.max_pages && page_needed(a, ip, x.p_lo, x.p_hi)) {
              const int p = __ldg(row + ip);
              if (p >= 0 && p < a.num_pages) pg = p;
              else bad = true;
            }
          }
        }
        const int sub = lane / C::kBoxes, box = lane % C::kBoxes;   // one copy a lane: (page of the tile, 64-dim box)
        const int p = __shfl_sync(0xFFFFFFFFu, pg, (in * ppt + sub) & 31);
        for (int kv = 0; kv < 2; ++kv) {
          const int seq = 2 * it + kv, sl = seq % C::kSlots;
          if (seq >= C::kSlots && !mbar_wait_warp(EMPTY(sl), ((seq / C::kSlots) - 1) & 1, &abort_s, a.err)) {
            stop = true;
            return false;
          }
          if (lane == 0) mbar_arrive_expect_tx(FULL(sl), C::kTileBytes);
          __syncwarp();
          if (lane < ppt * C::kBoxes)
            tma_load_4d(sKV + sl * C::kTileBytes + box * C::kBoxBytes + sub * box_rows * 128, kv ? &maps.v : &maps.k,
                        FULL(sl), box * 64, 0, g, p);
        }
      }
      return true;
    });
    if (bad) raise_flag(a.err, kErrBadPages);
    (void)stop;
    } else if (warp == 9) {
    // ---- tensor-core instructions
    if (lane == 0) {
      const uint32_t fmt = FP16 ? 0u : ((1u << 7) | (1u << 10));
      const uint32_t id_s = (1u << 4) | fmt | ((kTN >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t id_o = (1u << 4) | fmt | (1u << 16) | (((uint32_t)D >> 3) << 17) | ((128u >> 4) << 24);
      int it = 0, items = 0, cleans = 0, done[2] = {0, 0}, outs[2] = {0, 0};   // P tiles and items so far, per row tile
      auto wait = [&](uint32_t bar, int phase) { return mbar_wait(bar, phase & 1, &abort_s, a.err); };
      auto scores = [&](int t, int tile) {   // S_t = Q_t K^T
        const int sl = (2 * tile) % C::kSlots;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kBoxBytes + (kk & 3) * 32;
          tc_mma_f16(tmem + t * 128, smem_desc_sw128(sQ + t * C::kTileBytes + off),
                     smem_desc_sw128(sKV + sl * C::kTileBytes + off), id_s, kk != 0);
        }
        tc_commit(SFULL(t));
      };
      walk([&](int, const SeqRows&, int, const Item& x, int i0, int n, unsigned long long) {
        const int nt = x.n > tpt ? 2 : 1;
        if (!wait(QFULL, items) || !wait(FULL((2 * it) % C::kSlots), 2 * it / C::kSlots)) return false;
        tc_fence_after();
        for (int t = 0; t < nt; ++t) scores(t, it);
        tc_commit(EMPTY((2 * it) % C::kSlots));
        if (n == 1) tc_commit(QEMPTY);
        for (int i = 0; i < n; ++i, ++it) {
          const bool more = i + 1 < n;
          const int sv = (2 * it + 1) % C::kSlots;
          if (more && !wait(FULL((2 * it + 2) % C::kSlots), (2 * it + 2) / C::kSlots)) return false;
          if (!wait(FULL(sv), (2 * it + 1) / C::kSlots)) return false;
          if (nt == 2 && C::kBoxes == 2 && !tile_open<kTN>(a, x.r.tile(i0 + i) * kTN, x.p_lo, x.p_hi) &&
              !wait(CLEAN, cleans++))
            return false;
          for (int t = 0; t < nt; ++t) {
            if (i == 0 && outs[t] > 0 && !wait(OEMPTY(t), outs[t] - 1)) return false;
            if (!wait(PFULL(t), done[t])) return false;
            ++done[t];
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kTN / 16; ++kk)
              tc_mma_ts(tmem + kTmemO + t * 128, tmem + t * 128 + kk * 8,
                        desc_values(sKV + sv * C::kTileBytes + kk * 2048, C::kBoxBytes), id_o, (i | kk) != 0);
            if (t == nt - 1) tc_commit(EMPTY(sv));
            if (more) {
              scores(t, it + 1);
              if (t == nt - 1) {
                tc_commit(EMPTY((2 * it + 2) % C::kSlots));
                if (i + 2 == n) tc_commit(QEMPTY);
              }
            } else {
              tc_commit(OFULL(t));
            }
          }
        }
        ++items;
        for (int t = 0; t < nt; ++t) ++outs[t];
        return true;
      });
    }
    }
  } else {
    // ---- softmax: row `r` of row tile `t`
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, r = (warp & 3) * 32 + lane, tok = r / a.G, head = r % a.G;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + t * 128 + lanes, tO = tmem + kTmemO + t * 128 + lanes;
    int it = 0, seg = 0, done = 0, outs = 0;
    walk([&](int b, const SeqRows& s, int g, const Item& x, int i0, int n, unsigned long long u) {
      const bool mine = t == 0 || x.n > tpt;
      const bool live = mine && tok < tpt && t * tpt + tok < x.n;
      const int p = live ? x.p_lo + t * tpt + tok : -1;      // a row that is no token sees nothing
      float m = -INFINITY, negm = 0.f, l = 0.f;              // negm = -m in base-2 units (0 while nothing is seen)
      if (!mine) {
        it += n;
        ++seg;
        return true;
      }
      for (int i = 0; i < n; ++i, ++it) {
        const int j0 = x.r.tile(i0 + i) * kTN;
        const bool open = tile_open<kTN>(a, j0, x.p_lo, x.p_hi);
        if (!mbar_wait_warp(SFULL(t), done & 1, &abort_s, a.err)) return false;
        ++done;
        tc_fence_after();
        if (!open && (t == 0 || C::kBoxes == 2)) {
          // Take non-finite values out of this thread's position of the value tile: its 64-dim box t, or all
          // of it where the other row tile's warps have no rows.
          const int seq = 2 * it + 1, sl = seq % C::kSlots;
          if (!mbar_wait_warp(FULL(sl), (seq / C::kSlots) & 1, &abort_s, a.err)) return false;
          const bool both = x.n > tpt && C::kBoxes == 2;
          bool found = false;
          for (int box = both ? t : 0; box < (both ? t + 1 : C::kBoxes); ++box) {
            const uint32_t rowaddr = sKV + sl * C::kTileBytes + box * C::kBoxBytes + r * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint32_t at = rowaddr + (((c + lane) & 7) << 4);
              uint32_t w0, w1, w2, w3;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w0), "=r"(w1), "=r"(w2), "=r"(w3)
                           : "r"(at)
                           : "memory");
              const uint32_t b0 = non_finite16<FP16>(w0), b1 = non_finite16<FP16>(w1), b2 = non_finite16<FP16>(w2),
                             b3 = non_finite16<FP16>(w3);
              if ((b0 | b1 | b2 | b3) != 0u) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w0 & ~b0), "r"(w1 & ~b1),
                             "r"(w2 & ~b2), "r"(w3 & ~b3)
                             : "memory");
                found = true;
              }
            }
          }
          if (found) {
            const int j = j0 + r;
            if (j <= x.p_hi && (a.window == 0 || j > x.p_lo - a.window || j < a.sinks)) bad_s[seg & 3] = seg + 1;
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (t == 1 && lane == 0) mbar_arrive(CLEAN);
        }
        uint32_t sr[128];
        tmem_ld128(tS, sr);
        if (!open) {
          const int c_hi = p - j0;
          if (a.window == 0) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c > c_hi) sr[c] = 0xFF800000u;
          } else {
            const int c_lo = p - a.window - j0, c_s = a.sinks - j0;
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c > c_hi || (c <= c_lo && c >= c_s)) sr[c] = 0xFF800000u;
          }
        }
        float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
        for (int c = 0; c < 128; c += 4) {
          mx0 = fmaxf(mx0, __uint_as_float(sr[c]));
          mx1 = fmaxf(mx1, __uint_as_float(sr[c + 1]));
          mx2 = fmaxf(mx2, __uint_as_float(sr[c + 2]));
          mx3 = fmaxf(mx3, __uint_as_float(sr[c + 3]));
        }
        const float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
        // Move the reference if the new maximum is well above it (or is the first).
        const bool move = mx > m && (m == -INFINITY || (mx - m) * a.qk_scale > kLazy);
        float alpha = 1.f;
        if (move) {
          const float nn = -(mx * a.qk_scale);
          alpha = m == -INFINITY ? 0.f : ex2(nn - negm);
          m = mx;
          negm = nn;
          l *= alpha;
        }
        if (i > 0 && __any_sync(0xFFFFFFFFu, move)) {
          for (int c = 0; c < D; c += 32) {
            uint32_t v[32];
            tmem_ld32(tO + c, v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
            tmem_st32(tO + c, v);
          }
        }
        float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float p0 = ex2(fmaf(__uint_as_float(sr[c + e]), a.qk_scale, negm));
            const float p1 = ex2(fmaf(__uint_as_float(sr[c + e + 1]), a.qk_scale, negm));
            const float p2 = ex2(fmaf(__uint_as_float(sr[c + e + 2]), a.qk_scale, negm));
            const float p3 = ex2(fmaf(__uint_as_float(sr[c + e + 3]), a.qk_scale, negm));
            l0 += p0;
            l1 += p1;
            l2 += p2;
            l3 += p3;
            pk[e / 2] = pack16<FP16>(p0, p1);
            pk[e / 2 + 1] = pack16<FP16>(p2, p3);
          }
          tmem_st16(tS + c / 2, pk);
        }
        l += (l0 + l1) + (l2 + l3);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(PFULL(t));
      }
      // ---- the item's result, or this share's part of it
      const int my_seg = seg++;
      if (!mbar_wait_warp(OFULL(t), outs & 1, &abort_s, a.err)) return false;
      ++outs;
      tc_fence_after();
      const bool whole = i0 == 0 && n == x.r.count;
      const bool hurt = *(volatile int*)&bad_s[my_seg & 3] == my_seg + 1;
      const float inv = p < 0 ? 0.f : 1.f / l;
      uint16_t* orow = a.o + (long long)(s.row0 + x.t0 + t * tpt + tok) * a.o_stride + (long long)(g * a.G + head) * D;
      float* part = split.part + ((size_t)cta * 2 + (i0 == 0 ? 1 : 0)) * C::kPartFloats;
      bool nonfinite = false;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        tmem_ld32(tO + c, v);
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = p < 0 ? 0.f : __uint_as_float(v[e]);
        if (hurt && live) {
          float extra[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) extra[e] = 0.f;
          add_non_finite<FP16>(a, a.table + (size_t)b * a.max_pages, x.r, i0, n, x.p_lo, x.p_hi, p, g, c, extra);
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] += extra[e];
        }
        if (whole) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float f0 = f[e] * inv, f1 = f[e + 1] * inv;
            nonfinite |= !isfinite(f0) || !isfinite(f1);
            w[e / 2] = pack16<FP16>(f0, f1);
          }
          if (live) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(orow + c + 8 * e) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
          }
        } else if (live) {
#pragma unroll
          for (int e = 0; e < 32; ++e) part[(c + e) * kItemRows + t * 128 + r] = f[e];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(OEMPTY(t));
      if (live && whole && nonfinite) raise_flag(a.err, kErrNonFinite);
      if (!whole) {
        if (live) {
          part[D * kItemRows + t * 128 + r] = m == -INFINITY ? -1e30f : -negm;
          part[(D + 1) * kItemRows + t * 128 + r] = l;
        }
        if (i0 == 0 && tid == 0)
          split.rec[cta] = SplitRecord{s.row0 + x.t0, g, x.n, share_of(u + x.r.count - 1, total, ctas), x.p_lo};
      }
      return true;
    });
  }
  // After a timeout, copies and products still in flight finish before the CTA gives up its memory.
  if (tid == 0 && *(volatile int*)&abort_s) {
    const long long c0 = clock64();
    while (clock64() - c0 < 4000000ll) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of one split item (blockIdx.x: the CTA that began it) for 32 of its rows (blockIdx.y), in
// order; a warp takes a quarter of the dims, a lane a row.
template <int D, bool FP16>
__global__ void __launch_bounds__(128) chunk_join_kernel(const PagedArgs a, const ChunkSplit split) {
  using C = Chunk<D>;
  constexpr int E = D / 4;
  pdl_wait();
  pdl_launch_dependents();
  const int first = (int)blockIdx.x;
  const SplitRecord rec = split.rec[first];
  if (rec.until < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = (int)blockIdx.y * 32 + lane;
  const int tpt = 128 / a.G, t = slot >> 7, r = slot & 127, tok = r / a.G;
  if (tok >= tpt || t * tpt + tok >= rec.rows) return;
  auto part = [&](int c) { return split.part + ((size_t)c * 2 + (c == first ? 1 : 0)) * C::kPartFloats; };
  float M = -1e30f, L = 0.f, acc[E];
  for (int c = first; c <= rec.until; ++c) M = fmaxf(M, __ldcg(part(c) + D * kItemRows + slot));
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int c = first; c <= rec.until; ++c) {
    const float* pc = part(c);
    const float w = exp2f(__ldcg(pc + D * kItemRows + slot) - M);
    L += __ldcg(pc + (D + 1) * kItemRows + slot) * w;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += __ldcg(pc + (warp * E + e) * kItemRows + slot) * w;
  }
  bool nonfinite = false;
  uint32_t w[E / 2];
  const float inv = rec.p_lo + t * tpt + tok < 0 ? 0.f : 1.f / L;   // a row before position 0 sees nothing
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float x = acc[e] * inv, y = acc[e + 1] * inv;
    nonfinite |= !isfinite(x) || !isfinite(y);
    w[e / 2] = pack16<FP16>(x, y);
  }
  if (nonfinite) raise_flag(a.err, kErrNonFinite);
  uint16_t* orow = a.o + (long long)(rec.row + t * tpt + tok) * a.o_stride + (long long)(rec.g * a.G + r % a.G) * D + warp * E;
#pragma unroll
  for (int e = 0; e < E / 8; ++e)
    *reinterpret_cast<uint4*>(orow + 8 * e) = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
}

template <int D, bool FP16>
cudaError_t launch(const PagedMaps& maps, const PagedArgs& a, const ChunkSplit& split, int ctas, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(chunk_kernel<D, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Chunk<D>::smem(kPagedMaxSeqs));
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
  cfg.blockDim = dim3(128);
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
