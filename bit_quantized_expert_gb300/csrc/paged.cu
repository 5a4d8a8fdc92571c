// Paged key/value cache: the plan (block tables and slot maps), the append, and the C ABI of the three
// calls (contracts in include/gqa_paged.h).
//
//   plan_kernel    one cluster of eight CTAs.  Every CTA scans the sequences' new and fresh-page counts
//                  into shared memory (at most 4096 of each), then the cluster writes the table entries
//                  (one warp a sequence) and the token rows (one thread a row, its sequence by binary
//                  search) together.  Bound by latency: in a graph 4.3 us for 64 single tokens, 7.7 for
//                  1024 sequences with 96 chunks, 8.3 for 4096 single tokens.  (64 and 4096 single tokens and 8
//                  prompts of 1024 when the cluster's size was chosen: by one CTA 3.8, 19.3 and 9.9 us, by four
//                  3.8, 8.6 and 4.9, by eight 3.8, 7.6 and 4.2.)
//   append_kernel  16 bytes a thread, head rows contiguous on both sides.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <utility>

#include "paged.cuh"

namespace moe {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;   // the portable cluster size
constexpr int kPlanSeqsPerThread = kPagedMaxSeqs / kPlanThreads;

struct PlanArgs {
  const int32_t *ctx_len, *new_len, *free_pages, *n_free;
  int32_t *table, *q_start, *kv_len, *positions, *slots, *n_free_out;
  uint32_t* err;
  int B, T, page_shift, num_pages, max_pages, free_capacity;
};

// Lengths of one sequence, cut to the block-table row.
struct PlanSeq {
  int ctx, n;        // cached and new positions (as given, negatives as 0)
  int old, held;     // pages before and after
  int kv;            // length after the step
};

__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs& a, int ctx, int n, bool& bad) {
  PlanSeq s;
  const long long cap = (long long)a.max_pages << a.page_shift;
  const int round = (1 << a.page_shift) - 1;
  if (ctx < 0 || n < 0 || (long long)max(ctx, 0) + max(n, 0) > cap) bad = true;
  s.ctx = (int)min((long long)max(ctx, 0), cap);
  s.n = max(n, 0);
  s.kv = (int)min((long long)s.ctx + s.n, cap);
  s.old = (int)(((long long)s.ctx + round) >> a.page_shift);
  s.held = (int)(((long long)s.kv + round) >> a.page_shift);
  return s;
}

__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const PlanArgs a) {
  extern __shared__ long long plan_smem[];
  long long* start_s = plan_smem;            // [B + 1] rows before each sequence
  long long* base_s = plan_smem + a.B + 1;   // [B + 1] fresh pages before each sequence
  __shared__ long long warp_s[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = (int)blockIdx.x, ctas = (int)gridDim.x;
  bool bad = false;
  pdl_wait();
  pdl_launch_dependents();

  // Exclusive sums over the sequences, four consecutive ones a thread, in 64 bits: the lengths are
  // unchecked, so their sum may pass 32.
  long long rows = 0, fresh = 0;
  int nr[kPlanSeqsPerThread], fr[kPlanSeqsPerThread];
#pragma unroll
  for (int i = 0; i < kPlanSeqsPerThread; ++i) {
    const int b = tid * kPlanSeqsPerThread + i;
    nr[i] = fr[i] = 0;
    if (b < a.B) {
      const PlanSeq s = plan_seq(a, a.ctx_len[b], a.new_len[b], bad);
      nr[i] = s.n;
      fr[i] = s.held - s.old;
    }
    rows += nr[i];
    fresh += fr[i];
  }
  long long ir = rows, jf = fresh;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long r = __shfl_up_sync(0xFFFFFFFFu, ir, off), f = __shfl_up_sync(0xFFFFFFFFu, jf, off);
    if (lane >= off) {
      ir += r;
      jf += f;
    }
  }
  if (lane == 31) {
    warp_s[0][warp] = ir;
    warp_s[1][warp] = jf;
  }
  __syncthreads();
  if (warp == 0) {
    long long r = warp_s[0][lane], f = warp_s[1][lane];
    const long long r0 = r, f0 = f;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long x = __shfl_up_sync(0xFFFFFFFFu, r, off), y = __shfl_up_sync(0xFFFFFFFFu, f, off);
      if (lane >= off) {
        r += x;
        f += y;
      }
    }
    warp_s[0][lane] = r - r0;
    warp_s[1][lane] = f - f0;
  }
  __syncthreads();
  {
    long long r = warp_s[0][warp] + ir - rows, f = warp_s[1][warp] + jf - fresh;
#pragma unroll
    for (int i = 0; i < kPlanSeqsPerThread; ++i) {
      const int b = tid * kPlanSeqsPerThread + i;
      if (b <= a.B) {
        start_s[b] = r;
        base_s[b] = f;
      }
      r += nr[i];
      f += fr[i];
    }
    if (a.B == kPagedMaxSeqs && tid == kPlanThreads - 1) {
      start_s[a.B] = r;
      base_s[a.B] = f;
    }
  }
  const int n_free_raw = __ldcg(a.n_free);
  const int n_free = min(max(n_free_raw, 0), a.free_capacity);
  if (n_free != n_free_raw) bad = true;
  // Every CTA has read n_free (which n_free_out may be) before one of them writes n_free_out.
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  __syncthreads();

  const long long total = start_s[a.B], taken = base_s[a.B];
  if (total > a.T || taken > n_free) bad = true;
  if (cta == 0 && tid == 0) *a.n_free_out = (int)max(0ll, n_free - taken);

  // The m-th fresh page, or -1.
  auto fresh_page = [&](long long m) {
    if (m >= n_free) return -1;
    const int p = a.free_pages[n_free - 1 - m];
    if (p >= 0 && p < a.num_pages) return p;
    bad = true;
    return -1;
  };

  for (int b = tid + cta * kPlanThreads; b <= a.B; b += ctas * kPlanThreads) {
    a.q_start[b] = (int)min(start_s[b], (long long)a.T);
    if (b < a.B) {
      const PlanSeq s = plan_seq(a, a.ctx_len[b], a.new_len[b], bad);
      a.kv_len[b] = s.kv;
    }
  }
  const int warps = kPlanThreads / 32;
  for (int b = cta * warps + warp; b < a.B; b += ctas * warps) {
    const long long m0 = base_s[b];
    const int cnt = (int)(base_s[b + 1] - m0);
    if (cnt == 0) continue;
    const PlanSeq s = plan_seq(a, a.ctx_len[b], a.new_len[b], bad);
    int32_t* row = a.table + (size_t)b * a.max_pages + s.old;
    for (int i = lane; i < cnt; i += 32) row[i] = fresh_page(m0 + i);
  }
  const int rows_used = (int)min(total, (long long)a.T);
  for (int t = cta * kPlanThreads + tid; t < rows_used; t += ctas * kPlanThreads) {
    int lo = 0, hi = a.B - 1;   // the last sequence whose first row is at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start_s[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    const int b = lo;
    const PlanSeq s = plan_seq(a, a.ctx_len[b], a.new_len[b], bad);
    const long long pos = (long long)s.ctx + (t - start_s[b]);
    if (a.positions != nullptr) a.positions[t] = (int)min(pos, (long long)INT_MAX);
    int page = -1;
    if (pos < s.kv) {
      const int ip = (int)(pos >> a.page_shift);
      if (ip >= s.old) {
        page = fresh_page(base_s[b] + (ip - s.old));
      } else {
        page = __ldcg(a.table + (size_t)b * a.max_pages + ip);   // a held page: no CTA writes its entry
        if (page < 0 || page >= a.num_pages) {
          bad = true;
          page = -1;
        }
      }
    }
    a.slots[t] = page < 0 ? -1 : (page << a.page_shift) + (int)(pos & ((1 << a.page_shift) - 1));
  }
  if (bad) raise_flag(a.err, kErrBadPages);
}

struct AppendArgs {
  const uint16_t *k, *v;
  const int32_t *slots, *q_start;
  uint16_t *kc, *vc;
  uint32_t* err;
  int Hkv, B, T, page_shift, num_pages;
  int unit_shift;   // log2 of the 16-byte units of a head row (8 or 16)
  long long k_stride, v_stride, page_stride, head_stride, row_stride;
};

constexpr int kAppendThreads = 256;
constexpr int kAppendBatch = 4;

// The keys or the values (blockIdx.y), units of 16 bytes numbered by (token, head, unit of the row) in Index;
// four units a thread and turn, their slots and their data loaded together, so that one round trip to
// memory lies between the start and the stores.  8 prompts of up to 4096 tokens, 23.5 MB both ways, take 6.2 us in a
// graph where keys and values come from memory (3.8 TB/s, the launch and that round trip among them), 4.2 where they lie
// in L2, as behind a projection (with 2, 8 or 16 CTAs an SM in place of 4: 5.3, 5.8, 6.4).
template <class Index>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const bool values = blockIdx.y != 0;
  const uint16_t* src = values ? a.v : a.k;
  uint16_t* dst = values ? a.vc : a.kc;
  const long long stride = values ? a.v_stride : a.k_stride;
  const Index per = (Index)a.Hkv << a.unit_shift, n = (Index)a.T * per;
  const int rows = min(max(a.q_start[a.B], 0), a.T);
  const Index step = (Index)gridDim.x * kAppendThreads;
  for (Index i0 = (Index)blockIdx.x * kAppendThreads + threadIdx.x; i0 < n; i0 += step * kAppendBatch) {
    int t[kAppendBatch], r[kAppendBatch], slot[kAppendBatch];
    uint4 x[kAppendBatch];
#pragma unroll
    for (int j = 0; j < kAppendBatch; ++j) {
      const Index i = i0 + j * step;
      t[j] = i < n ? (int)(i / per) : a.T;
      r[j] = i < n ? (int)(i - (Index)t[j] * per) : 0;
      if (t[j] < rows) {
        slot[j] = a.slots[t[j]];
        x[j] = __ldcg(reinterpret_cast<const uint4*>(src + t[j] * stride) + r[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kAppendBatch; ++j) {
      if (t[j] >= rows) continue;
      const int page = slot[j] >> a.page_shift, off = slot[j] & ((1 << a.page_shift) - 1);
      if (slot[j] < 0 || page >= a.num_pages) {
        if (slot[j] != -1) raise_flag(a.err, kErrBadPages);
        continue;
      }
      const int h = r[j] >> a.unit_shift, u = r[j] & ((1 << a.unit_shift) - 1);
      *(reinterpret_cast<uint4*>(dst + page * a.page_stride + h * a.head_stride + off * a.row_stride) + u) = x[j];
    }
  }
}

// int32 arrays of one call, by address and entries.
struct Ints {
  const int32_t* p;
  long long n;
};
bool overlap(const Ints& x, const Ints& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return x.n > 0 && y.n > 0 && a < b + (uintptr_t)y.n * 4 && b < a + (uintptr_t)x.n * 4;
}

}  // namespace

// The dims rules, and the dims with every default filled in.
int check_paged_dims(const gqa_paged_dims* in, gqa_paged_dims* out) {
  if (in == nullptr) return MOE_ERR_INVALID_ARG;
  gqa_paged_dims d = *in;
  if (d.n_heads < 1 || d.n_kv_heads < 1 || d.n_heads % d.n_kv_heads != 0) return MOE_ERR_INVALID_ARG;
  if (d.page_size < 1 || d.num_pages < 1 || d.max_pages < 1 || d.n_seqs < 0 || d.n_tokens < 0 || d.max_new < 0 ||
      d.window < 0 || d.sinks < 0 || (d.dtype != GQA_PAGED_BF16 && d.dtype != GQA_PAGED_FP16))
    return MOE_ERR_INVALID_ARG;
  if ((d.head_dim != 64 && d.head_dim != 128) || d.n_heads / d.n_kv_heads > 8 || d.n_seqs > kPagedMaxSeqs)
    return MOE_ERR_UNSUPPORTED;
  if (d.page_size != 16 && d.page_size != 32 && d.page_size != 64 && d.page_size != 128) return MOE_ERR_UNSUPPORTED;
  const long long lim = 1ll << 31;
  if ((long long)d.num_pages * d.page_size >= lim || (long long)d.num_pages * d.page_size * d.n_kv_heads >= lim ||
      (long long)d.max_pages * d.page_size > lim / 2 || (long long)d.n_tokens * d.n_heads >= lim ||
      (long long)d.n_seqs * d.n_kv_heads >= lim)
    return MOE_ERR_UNSUPPORTED;
  const long long D = d.head_dim;
  if (d.max_new == 0) d.max_new = d.n_tokens;
  if (d.q_stride == 0) d.q_stride = d.n_heads * D;
  if (d.o_stride == 0) d.o_stride = d.n_heads * D;
  if (d.k_stride == 0) d.k_stride = d.n_kv_heads * D;
  if (d.v_stride == 0) d.v_stride = d.n_kv_heads * D;
  if (d.page_stride == 0) d.page_stride = (long long)d.n_kv_heads * d.page_size * D;
  if (d.head_stride == 0) d.head_stride = d.page_size * D;
  if (d.row_stride == 0) d.row_stride = D;
  // A stride over an extent of one is never stepped: any legal value serves.
  if (d.n_tokens <= 1) d.q_stride = d.o_stride = d.n_heads * D, d.k_stride = d.v_stride = d.n_kv_heads * D;
  if (d.n_kv_heads == 1) d.head_stride = D;
  if (d.num_pages == 1) d.page_stride = std::max(d.page_size * d.row_stride, d.n_kv_heads * d.head_stride);
  const long long s[7] = {d.q_stride, d.o_stride, d.k_stride, d.v_stride, d.page_stride, d.head_stride, d.row_stride};
  const long long least[7] = {d.n_heads * D, d.n_heads * D, d.n_kv_heads * D, d.n_kv_heads * D, D, D, D};
  for (int i = 0; i < 7; ++i) {
    if (s[i] < least[i]) return MOE_ERR_INVALID_ARG;
    if (s[i] >= (1ll << 39)) return MOE_ERR_UNSUPPORTED;
  }
  for (int i = 0; i < 7; ++i)
    if (s[i] % 8 != 0) return MOE_ERR_MISALIGNED;
  // No two elements of a cache at one address: in order of stride, each axis steps over the one below.
  std::pair<long long, long long> ax[3] = {
      {d.page_stride, d.num_pages}, {d.head_stride, d.n_kv_heads}, {d.row_stride, d.page_size}};
  std::sort(ax, ax + 3);
  long long span = D;   // elements from the first to past the last of the axes below
  for (const auto& x : ax) {
    if (x.second == 1) continue;
    if (x.first < span) return MOE_ERR_INVALID_ARG;
    span += x.first * (x.second - 1);
  }
  *out = d;
  return MOE_OK;
}

PagedArgs paged_args(const gqa_paged_dims& d) {
  PagedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.Hq = d.n_heads;
  a.Hkv = d.n_kv_heads;
  a.G = d.n_heads / d.n_kv_heads;
  a.page_shift = log2_of(d.page_size);
  a.num_pages = d.num_pages;
  a.max_pages = d.max_pages;
  a.B = d.n_seqs;
  a.T = d.n_tokens;
  a.max_new = std::min(d.max_new, d.n_tokens);
  // A window that no position can pass is none (and keeps p - window within 32 bits).
  a.window = d.window >= (d.max_pages << a.page_shift) ? 0 : d.window;
  a.sinks = d.sinks;
  a.fp16 = d.dtype == GQA_PAGED_FP16;
  a.q_stride = d.q_stride;
  a.o_stride = d.o_stride;
  a.page_stride = d.page_stride;
  a.head_stride = d.head_stride;
  a.row_stride = d.row_stride;
  a.qk_scale = (float)(1.4426950408889634 / std::sqrt((double)d.head_dim));
  return a;
}

int device_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

namespace {

// One cache as the tensor maps see it; boxes of `rows` positions of one page and head.
bool encode_pages(CUtensorMap* m, const uint16_t* cache, const gqa_paged_dims& d, int rows) {
  EncodeTiledFn f = encode_fn();
  if (f == nullptr) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d.head_dim, (cuuint64_t)d.page_size, (cuuint64_t)d.n_kv_heads,
                              (cuuint64_t)d.num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)d.row_stride * 2, (cuuint64_t)d.head_stride * 2,
                                 (cuuint64_t)d.page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)std::min(rows, d.page_size), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return f(m, d.dtype == GQA_PAGED_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
           const_cast<uint16_t*>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// The queries in boxes of one row tile: the G heads of a group for floor(128 / G) tokens.
bool encode_queries(CUtensorMap* m, const uint16_t* q, const gqa_paged_dims& d) {
  EncodeTiledFn f = encode_fn();
  if (f == nullptr) return false;
  const int G = d.n_heads / d.n_kv_heads;
  const cuuint64_t dims[3] = {(cuuint64_t)d.head_dim, (cuuint64_t)d.n_heads, (cuuint64_t)d.n_tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d.head_dim * 2, (cuuint64_t)d.q_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(128 / G)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return f(m, d.dtype == GQA_PAGED_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
           const_cast<uint16_t*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace moe

using namespace moe;

extern "C" size_t gqa_paged_workspace_bytes(const gqa_paged_dims* dims) {
  gqa_paged_dims d;
  if (check_paged_dims(dims, &d) != MOE_OK) return 0;
  return kWsHeadBytes + (d.max_new == 1 ? paged_decode_scratch(d.head_dim, kPagedMaxCtas)
                                        : paged_chunk_scratch(d.head_dim, kPagedMaxCtas));
}

extern "C" moe_status gqa_paged_plan(const gqa_paged_dims* dims, const int32_t* ctx_len, const int32_t* new_len,
                                     const int32_t* free_pages, int32_t free_capacity, const int32_t* n_free,
                                     int32_t* block_table, int32_t* q_start, int32_t* kv_len, int32_t* positions,
                                     int32_t* slots, int32_t* n_free_out, void* workspace, size_t workspace_bytes,
                                     void* stream) {
  gqa_paged_dims d;
  int st = check_paged_dims(dims, &d);
  if (st != MOE_OK) return (moe_status)st;
  if (d.n_seqs == 0) return MOE_OK;
  if (free_capacity < 0 || (free_capacity > 0 && free_pages == nullptr)) return MOE_ERR_INVALID_ARG;
  if (d.n_tokens > 0 && slots == nullptr) return MOE_ERR_INVALID_ARG;
  if ((st = check_pointers({ctx_len, new_len, n_free, block_table, q_start, kv_len, n_free_out}, {workspace})) != MOE_OK)
    return (moe_status)st;
  if (misaligned(slots, 4) || misaligned(positions, 4) || misaligned(free_pages, 4)) return MOE_ERR_MISALIGNED;
  if (workspace_bytes < gqa_paged_workspace_bytes(dims)) return MOE_ERR_WORKSPACE;
  // The CTAs read the inputs, the table's held entries too, while others write the outputs.
  const Ints in[4] = {{n_free, 1}, {ctx_len, d.n_seqs}, {new_len, d.n_seqs}, {free_pages, free_capacity}};
  const Ints out[6] = {{n_free_out, 1},         {block_table, (long long)d.n_seqs * d.max_pages},
                       {q_start, d.n_seqs + 1}, {kv_len, d.n_seqs},
                       {slots, d.n_tokens},     {positions, positions == nullptr ? 0 : d.n_tokens}};
  for (int i = 0; i < 6; ++i) {
    for (int j = 0; j < 4; ++j)
      if (overlap(out[i], in[j]) && !(i == 0 && j == 0 && n_free_out == n_free)) return MOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return MOE_ERR_INVALID_ARG;
  }
  PlanArgs a = {ctx_len,    new_len, free_pages, n_free,     block_table,
                q_start,    kv_len,  positions,  slots,      n_free_out,
                static_cast<uint32_t*>(workspace), d.n_seqs, d.n_tokens, log2_of(d.page_size), d.num_pages, d.max_pages,
                free_capacity};
  const size_t smem = 2 * ((size_t)d.n_seqs + 1) * sizeof(long long);
  static std::atomic<uint64_t> ready{0};
  if (allow_smem(reinterpret_cast<const void*>(plan_kernel), 2 * (kPagedMaxSeqs + 1) * (int)sizeof(long long), &ready) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kPlanCtas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, plan_kernel, a) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status gqa_paged_append(const gqa_paged_dims* dims, const uint16_t* k, const uint16_t* v,
                                       const int32_t* slots, const int32_t* q_start, uint16_t* k_cache,
                                       uint16_t* v_cache, void* workspace, size_t workspace_bytes, void* stream) {
  gqa_paged_dims d;
  int st = check_paged_dims(dims, &d);
  if (st != MOE_OK) return (moe_status)st;
  if (d.n_seqs == 0 || d.n_tokens == 0) return MOE_OK;
  if ((st = check_pointers({slots, q_start}, {k, v, k_cache, v_cache, workspace})) != MOE_OK) return (moe_status)st;
  if (workspace_bytes < gqa_paged_workspace_bytes(dims)) return MOE_ERR_WORKSPACE;
  int sms = 0;
  if (device_sms(&sms) != MOE_OK) return MOE_ERR_CUDA;
  AppendArgs a = {k, v, slots, q_start, k_cache, v_cache, static_cast<uint32_t*>(workspace), d.n_kv_heads, d.n_seqs,
                  d.n_tokens, log2_of(d.page_size), d.num_pages, log2_of(d.head_dim / 8), d.k_stride, d.v_stride, d.page_stride,
                  d.head_stride, d.row_stride};
  const long long units = ((long long)d.n_tokens * d.n_kv_heads) << a.unit_shift;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min((units + kAppendThreads - 1) / kAppendThreads, (long long)sms * 4), 2);
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = at;
  cfg.numAttrs = 1;
  // 32-bit unit numbers unless the last turn's could pass them.
  const bool wide = units + (long long)cfg.gridDim.x * kAppendThreads * kAppendBatch >= (1ll << 32);
  const cudaError_t e = wide ? cudaLaunchKernelEx(&cfg, append_kernel<unsigned long long>, a)
                             : cudaLaunchKernelEx(&cfg, append_kernel<uint32_t>, a);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" moe_status gqa_paged_attention(const gqa_paged_dims* dims, const uint16_t* q, const uint16_t* k_cache,
                                          const uint16_t* v_cache, const int32_t* block_table, const int32_t* q_start,
                                          const int32_t* kv_len, uint16_t* o, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  gqa_paged_dims d;
  int st = check_paged_dims(dims, &d);
  if (st != MOE_OK) return (moe_status)st;
  if (d.n_seqs == 0 || d.n_tokens == 0) return MOE_OK;
  if ((st = check_pointers({block_table, q_start, kv_len}, {q, k_cache, v_cache, o, workspace})) != MOE_OK)
    return (moe_status)st;
  if (workspace_bytes < gqa_paged_workspace_bytes(dims)) return MOE_ERR_WORKSPACE;
  PagedArgs a = paged_args(d);
  a.q = q;
  a.kc = k_cache;
  a.vc = v_cache;
  a.table = block_table;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.o = o;
  a.err = static_cast<uint32_t*>(workspace);
  const bool single = d.max_new == 1;
  const int tile = single ? 64 : 128;   // positions of a cache tile
  int sms = 0;
  PagedMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  if (device_sms(&sms) != MOE_OK || !encode_pages(&maps.k, k_cache, d, tile) || !encode_pages(&maps.v, v_cache, d, tile) ||
      (!single && !encode_queries(&maps.q, q, d)))
    return MOE_ERR_CUDA;
  void* scratch = static_cast<uint8_t*>(workspace) + kWsHeadBytes;
  const int ctas = std::min(sms, kPagedMaxCtas);
  const auto launch = single ? launch_paged_decode : launch_paged_chunk;
  return launch(maps, a, d.head_dim, scratch, ctas, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                                     : MOE_ERR_CUDA;
}
