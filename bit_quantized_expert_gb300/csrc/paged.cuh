// The paged key/value cache as the kernels see it: the arguments of one call and the checked reads
// of the tables that live on the GPU (contracts in include/gqa_paged.h).
#pragma once

#include "../../include/gqa_paged.h"
#include "common.cuh"
#include "kernels.h"

namespace moe {

constexpr uint32_t kErrBadPages = 16u;   // a length, page or slot out of range

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

// One sequence's rows and length, cut to what the buffers hold.  A sequence whose rows do not lie in
// the buffers has none.
struct SeqRows {
  int row0, n;   // its rows of q and o
  int p0;        // position of its first row (negative: the row sees nothing)
  int L;         // positions in the cache
};

__device__ __forceinline__ SeqRows load_seq(const PagedArgs& a, int b, bool& bad) {
  const int r0 = __ldg(a.q_start + b), r1 = __ldg(a.q_start + b + 1), len = __ldg(a.kv_len + b);
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

// Whether the token at position p sees position j.
__device__ __forceinline__ bool paged_sees(const PagedArgs& a, int p, int j) {
  return j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
}

}  // namespace moe
