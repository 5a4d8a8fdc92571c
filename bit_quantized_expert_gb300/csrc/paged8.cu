// Paged key/value cache in 8 bits: the append, the read, and the C ABI of its calls (contracts in
// include/gqa_paged8.h).
//
//   append8_kernel  a warp takes the 16 positions of one block of one head, keys or values: the largest new value
//                   gives the scale (a power of two, found from the bits of that value, so that quantising is
//                   exact but for the codes' own rounding), then all rows of the block are written.  No two warps
//                   have a block in common, so a scale and the codes under it change together.
//   read8_kernel    the same walk, codes times scale into 16-bit rows.
// Every CTA scans the sequences' block counts for itself, so that a warp finds its block by a search in shared memory.
//
// Measured in a graph (2 heads of 128).  Append: 64 single tokens 3.4 us, the latency of a launch and four dependent
// loads (schedule, page beside the rows, scale, old codes where the scale grows); 8 prompts (17.6 MB) 7.3 us.
// Read: 300 positions 2.4 us; 8 sequences of up to 32768 (37.8 MB) 9.0 us, 4.2 TB/s, 62 % of the copy rate.
// Steps at 8 prompts: 10.2; 8.0 with held codes read only where the scale grows; 7.7 with the rows on their way before the
// page is known; 7.3 with CTAs of 128 threads.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "paged8.cuh"

namespace moe {
namespace {

// Threads of a CTA.  Few sequences: 128, as many CTAs as an SM holds (append of 64 tokens 3.4 us, 8 prompts 7.3; with 256 threads
// 3.6 and 7.7).  Every CTA scans the sequences, so for many of them there are few and wide ones, in one wave.  Narrow against
// wide CTAs, in a graph, us:
//                       append                                       read
//   200 sequences       1 token 3.9 / 4.5, 500 39.2 / 42.0           up to 64 4.6 / 4.7, 500 27.1 / 29.6
//   300                 1 token 4.1 / 4.7, 32 10.0 / 9.6, 500 57.0 / 59.5      1 3.2 / 3.2, 32 6.4 / 6.6, 500 39.7 / 43.0
//   400                 1 token 5.9 / 4.7
//   1000                100 49.2 / 45.0                              100 38.2 / 29.5
//   1024                1 token 12.1 / 7.8                           up to 64 19.5 / 9.4
//   4000                20 245 / 53                                  20 224 / 32
//   4096                1 token 234 / 27
// So the sides meet between 200 and 400 sequences, whatever their rows; between 257 and there the rule costs up to 14 %.
constexpr int kNarrow = 128, kWide = 512;
constexpr int kManySeqs = 256;
constexpr int kNarrowThreads = 1024;   // of an SM, keys and values each, at most

// Arguments of the append and of the read: `k`, `v` are rows of 16-bit values.
struct WalkArgs : PagedArgs {
  uint16_t *k, *v;
  uint8_t *kc8, *vc8;
  float *ks, *vs;
  long long k_stride, v_stride;
};

// The blocks of 16 positions that hold a sequence's rows: first .. first + n - 1 (block -1 and below: before position 0).
struct Blocks {
  int first, n;
};
__device__ __forceinline__ Blocks blocks_of(const SeqRows& s, bool from_zero) {
  if (s.n == 0 || (from_zero && s.p0 + s.n <= 0)) return Blocks{0, 0};
  const int first = (from_zero ? max(s.p0, 0) : s.p0) >> kBlock8Shift;
  return Blocks{first, ((s.p0 + s.n - 1) >> kBlock8Shift) - first + 1};
}

// One block of one head: page number as the table has it, and offsets o0 .. o1 - 1 that rows row0 .. have.
struct Unit {
  int g, page, off, row0, o0, o1;
};

// body(unit, page) for every block, a warp each; page() gives the page's number, -1 for none; blockIdx.y: keys or values.
template <int NT, bool FROM_ZERO, class Body>
__device__ __forceinline__ void walk_blocks(const WalkArgs& a, uint32_t* pre_s, uint32_t* warp_s, Body&& body) {
  bool bad = false, over;
  const uint32_t total = scan_sequences8<NT>(a.B, pre_s, warp_s, &over, [&](int b) {
    return (unsigned long long)blocks_of(load_seq(a, b, bad), FROM_ZERO).n * a.Hkv;
  });
  if (over) bad = true;   // (cannot be: T * Hq and B * Hkv are below 2^31)
  const uint32_t warps = gridDim.x * (NT / 32);
  for (uint32_t u = blockIdx.x * (NT / 32) + (threadIdx.x >> 5); !over && u < total; u += warps) {
    const int b = find_sequence(pre_s, a.B, u);
    const SeqRows s = load_seq(a, b, bad);
    const uint32_t at = u - pre_s[b], block = at / a.Hkv;
    const int j0 = (blocks_of(s, FROM_ZERO).first + (int)block) << kBlock8Shift;   // its first position
    Unit x;
    x.g = (int)(at - block * a.Hkv);
    x.o0 = max((FROM_ZERO ? max(s.p0, 0) : s.p0) - j0, 0);
    x.o1 = min(s.p0 + s.n - j0, 1 << kBlock8Shift);
    x.row0 = s.row0 + (j0 - s.p0);   // the row that offset 0 would have
    x.page = j0 >= 0 ? a.table[(size_t)b * a.max_pages + (j0 >> a.page_shift)] : -1;
    x.off = j0 & ((1 << a.page_shift) - 1);
    body(x, [&]() {   // the number is looked at here, not before: what does not depend on it goes first
      const bool ok = x.page >= 0 && x.page < a.num_pages;
      bad |= !ok && j0 >= 0;
      return ok ? x.page : -1;
    });
    __syncwarp();
  }
  if (bad) raise_flag(a.err, kErrBadPages);
}

// A lane has 8 dims (16 bytes of a row, 8 codes) of every (256 / D)-th row.
template <int D, bool FP16, int NT>
__global__ void __launch_bounds__(NT, NT == kNarrow ? 5 : 1) append8_kernel(const WalkArgs a) {
  constexpr int kLanes = D / 8, kStep = 32 / kLanes, kTurns = 16 / kStep;
  extern __shared__ uint32_t pre_s[];
  __shared__ uint32_t warp_s[NT / 32];
  pdl_wait();
  pdl_launch_dependents();
  const bool values = blockIdx.y != 0;
  const uint16_t* src = values ? a.v : a.k;
  uint8_t* dst = values ? a.vc8 : a.kc8;
  float* scales = values ? a.vs : a.ks;
  const long long stride = values ? a.v_stride : a.k_stride;
  const int lane = threadIdx.x & 31, r0 = lane / kLanes, dim = (lane % kLanes) * 8;
  walk_blocks<NT, true>(a, pre_s, warp_s, [&](const Unit& u, auto&& page_of) {
    // The new rows, all in flight together, beside the page's number.  (What the block holds before them is read only where
    // the scale grows.)
    uint4 x[kTurns];
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int o = r0 + i * kStep;
      x[i] = make_uint4(0, 0, 0, 0);
      if (o >= u.o0 && o < u.o1)
        x[i] = __ldcg(reinterpret_cast<const uint4*>(src + (long long)(u.row0 + o) * stride + u.g * D + dim));
    }
    const int page = page_of();
    if (page < 0) return;
    uint8_t* to = dst + page * a.page_stride + u.g * a.head_stride + (u.off + r0) * a.row_stride + dim;
    float* scale = scales + scale_index(page, a.Hkv, u.g, a.page_shift, u.off);
    float was = u.o0 > 0 ? *scale : kLeastScale;
    if (!scale_ok(was)) {
      raise_flag(a.err, kErrBadPages);
      was = kLeastScale;
    }
    uint32_t top = 0;   // bits of the largest magnitude (as fp32, whose order is that of its bits)
    bool lost = false;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack16<FP16>(w[e]);
        const uint32_t m0 = __float_as_uint(fabsf(f.x)), m1 = __float_as_uint(fabsf(f.y));
        constexpr uint32_t kMost = (127u + 60u + 8u) << 23 | 0x600000u;   // 448 * 2^60
        lost |= m0 > kMost || m1 > kMost;
        top = max(top, max(m0 > kMost ? 0u : m0, m1 > kMost ? 0u : m1));
      }
    }
    __syncwarp();
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    // top = 1.m * 2^(E - 127) <= 448 * 2^e = 1.75 * 2^(8 + e) from e = E - 135 on, or one more where 1.m > 1.75
    const int e = min(max((int)(top >> 23) - 135 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), -60), 60);
    const float s = fmaxf(__uint_as_float((uint32_t)(e + 127) << 23), was);
    const float inv = 1.f / s, ratio = was / s;   // exact
    auto code = [&](float v) { return fabsf(v) <= 448.f * kMostScale ? v * inv : __uint_as_float(0x7FC00000u); };
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int o = r0 + i * kStep;
      if (o < u.o0 || o >= u.o1) continue;
      const float2 f0 = unpack16<FP16>(x[i].x), f1 = unpack16<FP16>(x[i].y), f2 = unpack16<FP16>(x[i].z),
                   f3 = unpack16<FP16>(x[i].w);
      *reinterpret_cast<uint2*>(to + (long long)i * kStep * a.row_stride) =
          make_uint2(to_codes4(code(f0.x), code(f0.y), code(f1.x), code(f1.y)),
                     to_codes4(code(f2.x), code(f2.y), code(f3.x), code(f3.y)));
    }
    if (u.o0 > 0 && ratio != 1.f) {   // codes in the scale before, to codes in the new one
      uint2 old[kTurns];
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        old[i] = make_uint2(0, 0);
        if (r0 + i * kStep < u.o0) old[i] = __ldcg(reinterpret_cast<const uint2*>(to + (long long)i * kStep * a.row_stride));
      }
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        if (r0 + i * kStep >= u.o0) continue;
        uint32_t h[4];
        codes_to_half4(old[i].x, h[0], h[1]);
        codes_to_half4(old[i].y, h[2], h[3]);
        const float2 f0 = unpack16<true>(h[0]), f1 = unpack16<true>(h[1]), f2 = unpack16<true>(h[2]), f3 = unpack16<true>(h[3]);
        *reinterpret_cast<uint2*>(to + (long long)i * kStep * a.row_stride) =
            make_uint2(to_codes4(f0.x * ratio, f0.y * ratio, f1.x * ratio, f1.y * ratio),
                       to_codes4(f2.x * ratio, f2.y * ratio, f3.x * ratio, f3.y * ratio));
      }
    }
    if (lane == 0) *scale = s;
    if (lost) raise_flag(a.err, kErrNonFinite);
  });
}

template <int D, bool FP16, int NT>
__global__ void __launch_bounds__(NT) read8_kernel(const WalkArgs a) {
  constexpr int kLanes = D / 8, kStep = 32 / kLanes, kTurns = 16 / kStep;
  extern __shared__ uint32_t pre_s[];
  __shared__ uint32_t warp_s[NT / 32];
  pdl_wait();
  pdl_launch_dependents();
  const bool values = blockIdx.y != 0;
  const uint8_t* src = values ? a.vc8 : a.kc8;
  uint16_t* dst = values ? a.v : a.k;
  const float* scales = values ? a.vs : a.ks;
  const long long stride = values ? a.v_stride : a.k_stride;
  const int lane = threadIdx.x & 31, r0 = lane / kLanes, dim = (lane % kLanes) * 8;
  walk_blocks<NT, false>(a, pre_s, warp_s, [&](const Unit& u, auto&& page_of) {
    const int page = page_of();
    uint2 x[kTurns];
    float s = 0.f;
    if (page >= 0) s = scales[scale_index(page, a.Hkv, u.g, a.page_shift, u.off)];
    const uint8_t* from = src + page * a.page_stride + u.g * a.head_stride + (u.off + r0) * a.row_stride + dim;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int o = r0 + i * kStep;
      x[i] = make_uint2(0, 0);
      if (page >= 0 && o >= u.o0 && o < u.o1)
        x[i] = __ldcg(reinterpret_cast<const uint2*>(from + (long long)i * kStep * a.row_stride));
    }
    if (page >= 0 && !scale_ok(s)) {
      raise_flag(a.err, kErrBadPages);
      s = kLeastScale;
    }
    auto pair = [&](uint32_t h) {
      const float2 f = unpack16<true>(h);
      float y0 = f.x * s, y1 = f.y * s;
      if (FP16) {   // (comparisons, so that NaN stays)
        y0 = y0 > 65504.f ? 65504.f : y0 < -65504.f ? -65504.f : y0;
        y1 = y1 > 65504.f ? 65504.f : y1 < -65504.f ? -65504.f : y1;
      }
      return pack16<FP16>(y0, y1);
    };
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int o = r0 + i * kStep;
      if (o < u.o0 || o >= u.o1) continue;
      uint32_t h[4];
      codes_to_half4(x[i].x, h[0], h[1]);
      codes_to_half4(x[i].y, h[2], h[3]);
      *reinterpret_cast<uint4*>(dst + (long long)(u.row0 + o) * stride + u.g * D + dim) =
          make_uint4(pair(h[0]), pair(h[1]), pair(h[2]), pair(h[3]));
    }
  });
}

// The dims rules of gqa_paged.h, and the caches' strides in bytes on 16-byte boundaries.
int check_paged8_dims(const gqa_paged_dims* in, gqa_paged_dims* d) {
  const int st = check_paged_dims(in, d);
  if (st != MOE_OK) return st;
  return d->page_stride % 16 != 0 || d->head_stride % 16 != 0 || d->row_stride % 16 != 0 ? MOE_ERR_MISALIGNED : MOE_OK;
}

template <class Args>
void fill(Args* a, const gqa_paged_dims& d, const int32_t* block_table, const int32_t* q_start, const int32_t* kv_len,
          void* workspace) {
  std::memset(a, 0, sizeof(*a));
  static_cast<PagedArgs&>(*a) = paged_args(d);
  a->table = block_table;
  a->q_start = q_start;
  a->kv_len = kv_len;
  a->err = static_cast<uint32_t*>(workspace);
}

template <template <int, bool, int> class K, int NT>
cudaError_t launch_walk(const WalkArgs& a, int D, int sms, cudaStream_t st) {
  // At most this many blocks: a sequence's rows touch two more than a sixteenth of them, and one each.
  const long long blocks = std::min((long long)a.T, (long long)a.T / 16 + 2ll * std::min(a.B, a.T)) * a.Hkv;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int most = NT == kNarrow ? sms * (kNarrowThreads / NT) : K<64, false, NT>::wide_ctas(sms);
  cfg.gridDim = dim3((unsigned)std::min((blocks + NT / 32 - 1) / (NT / 32), (long long)most), 2);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = ((size_t)a.B + 1) * 4;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (D == 128)
    return a.fp16 ? cudaLaunchKernelEx(&cfg, K<128, true, NT>::fn, a) : cudaLaunchKernelEx(&cfg, K<128, false, NT>::fn, a);
  return a.fp16 ? cudaLaunchKernelEx(&cfg, K<64, true, NT>::fn, a) : cudaLaunchKernelEx(&cfg, K<64, false, NT>::fn, a);
}
template <template <int, bool, int> class K>
cudaError_t launch_walk(const WalkArgs& a, int D, int sms, cudaStream_t st) {
  return a.B <= kManySeqs ? launch_walk<K, kNarrow>(a, D, sms, st) : launch_walk<K, kWide>(a, D, sms, st);
}
template <int D, bool FP16, int NT>
struct Append8 {
  static constexpr auto fn = append8_kernel<D, FP16, NT>;
  static int wide_ctas(int sms) { return sms / 2; }
};
template <int D, bool FP16, int NT>
struct Read8 {
  static constexpr auto fn = read8_kernel<D, FP16, NT>;
  static int wide_ctas(int sms) { return sms; }
};

}  // namespace

// One cache as the tensor maps see it; boxes of `rows` positions of one page and head.
bool encode_pages8(CUtensorMap* m, const uint8_t* cache, const gqa_paged_dims& d, int rows) {
  EncodeTiledFn f = encode_fn();
  if (f == nullptr) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d.head_dim, (cuuint64_t)d.page_size, (cuuint64_t)d.n_kv_heads,
                              (cuuint64_t)d.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)d.row_stride, (cuuint64_t)d.head_stride, (cuuint64_t)d.page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)d.head_dim, (cuuint32_t)(rows < d.page_size ? rows : d.page_size), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(cache), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, d.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe

using namespace moe;

extern "C" size_t gqa_paged8_workspace_bytes(const gqa_paged_dims* dims) {
  gqa_paged_dims d;
  return check_paged8_dims(dims, &d) == MOE_OK ? gqa_paged_workspace_bytes(dims) : 0;
}

extern "C" moe_status gqa_paged8_append(const gqa_paged_dims* dims, const uint16_t* k, const uint16_t* v,
                                        const int32_t* block_table, const int32_t* q_start, const int32_t* kv_len,
                                        uint8_t* k_cache, uint8_t* v_cache, float* k_scale, float* v_scale, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  gqa_paged_dims d;
  int st = check_paged8_dims(dims, &d);
  if (st != MOE_OK) return (moe_status)st;
  if (d.n_seqs == 0 || d.n_tokens == 0) return MOE_OK;
  if ((st = check_pointers({block_table, q_start, kv_len}, {k, v, k_cache, v_cache, k_scale, v_scale, workspace})) != MOE_OK)
    return (moe_status)st;
  if (workspace_bytes < gqa_paged_workspace_bytes(dims)) return MOE_ERR_WORKSPACE;
  if (k_cache == v_cache || k_scale == v_scale) return MOE_ERR_INVALID_ARG;   // (both would be written)
  int sms = 0;
  if (device_sms(&sms) != MOE_OK) return MOE_ERR_CUDA;
  WalkArgs a;
  fill(&a, d, block_table, q_start, kv_len, workspace);
  a.k = const_cast<uint16_t*>(k);
  a.v = const_cast<uint16_t*>(v);
  a.kc8 = k_cache;
  a.vc8 = v_cache;
  a.ks = k_scale;
  a.vs = v_scale;
  a.k_stride = d.k_stride;
  a.v_stride = d.v_stride;
  return launch_walk<Append8>(a, d.head_dim, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status gqa_paged8_read(const gqa_paged_dims* dims, const uint8_t* k_cache, const uint8_t* v_cache,
                                      const float* k_scale, const float* v_scale, const int32_t* block_table,
                                      const int32_t* q_start, const int32_t* kv_len, uint16_t* k, uint16_t* v,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  gqa_paged_dims d;
  int st = check_paged8_dims(dims, &d);
  if (st != MOE_OK) return (moe_status)st;
  if (d.n_seqs == 0 || d.n_tokens == 0) return MOE_OK;
  if ((st = check_pointers({block_table, q_start, kv_len}, {k, v, k_cache, v_cache, k_scale, v_scale, workspace})) != MOE_OK)
    return (moe_status)st;
  if (workspace_bytes < gqa_paged_workspace_bytes(dims)) return MOE_ERR_WORKSPACE;
  if (k == v) return MOE_ERR_INVALID_ARG;   // (both would be written)
  int sms = 0;
  if (device_sms(&sms) != MOE_OK) return MOE_ERR_CUDA;
  WalkArgs a;
  fill(&a, d, block_table, q_start, kv_len, workspace);
  a.k = k;
  a.v = v;
  a.kc8 = const_cast<uint8_t*>(k_cache);
  a.vc8 = const_cast<uint8_t*>(v_cache);
  a.ks = const_cast<float*>(k_scale);
  a.vs = const_cast<float*>(v_scale);
  a.k_stride = d.k_stride;
  a.v_stride = d.v_stride;
  return launch_walk<Read8>(a, d.head_dim, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status gqa_paged8_attention(const gqa_paged_dims* dims, const uint16_t* q, const uint8_t* k_cache,
                                           const uint8_t* v_cache, const float* k_scale, const float* v_scale,
                                           const int32_t* block_table, const int32_t* q_start, const int32_t* kv_len,
                                           uint16_t* o, void* workspace, size_t workspace_bytes, void* stream) {
  gqa_paged_dims d;
  int st = check_paged8_dims(dims, &d);
  if (st != MOE_OK) return (moe_status)st;
  if (d.n_seqs == 0 || d.n_tokens == 0) return MOE_OK;
  if ((st = check_pointers({block_table, q_start, kv_len}, {q, k_cache, v_cache, k_scale, v_scale, o, workspace})) != MOE_OK)
    return (moe_status)st;
  if (workspace_bytes < gqa_paged_workspace_bytes(dims)) return MOE_ERR_WORKSPACE;
  Paged8Args a;
  fill(&a, d, block_table, q_start, kv_len, workspace);
  a.q = q;
  a.o = o;
  a.kc8 = k_cache;
  a.vc8 = v_cache;
  a.ks = k_scale;
  a.vs = v_scale;
  int sms = 0;
  if (device_sms(&sms) != MOE_OK) return MOE_ERR_CUDA;
  const auto launch = d.max_new == 1 ? launch_paged8_decode : launch_paged8_chunk;
  return launch(d, a, static_cast<uint8_t*>(workspace) + kWsHeadBytes, std::min(sms, kPagedMaxCtas),
                static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
