// The paged cache held in 8 bits as the kernels see it (contract in include/gqa_paged8.h): its arguments, the
// conversions of e4m3 codes, and the scales of its blocks.
#pragma once

#include "../../include/gqa_paged8.h"
#include "paged.cuh"

namespace moe {

constexpr int kBlock8Shift = 4;               // positions of a scale, as a power of two
constexpr float kLeastScale = 0x1p-60f, kMostScale = 0x1p60f;

// (kc and vc of PagedArgs are not used; its cache strides are bytes.)
struct Paged8Args : PagedArgs {
  const uint8_t *kc8, *vc8;   // [num_pages, Hkv, page_size, D]
  const float *ks, *vs;       // [num_pages, Hkv, page_size / 16]
};

// A power of two in the scales' range.
__device__ __forceinline__ bool scale_ok(float s) {
  return s >= kLeastScale && s <= kMostScale && (__float_as_uint(s) & 0x7FFFFFu) == 0;
}

// Index of the scale of the block at offset `off` of a page.  Fits: num_pages * page_size * Hkv < 2^31.
__device__ __forceinline__ int scale_index(int page, int Hkv, int g, int page_shift, int off) {
  return ((page * Hkv + g) << (page_shift - kBlock8Shift)) + (off >> kBlock8Shift);
}

// Two codes (low byte first) as a pair of fp16 values, exact.
__device__ __forceinline__ uint32_t codes_to_half2(uint16_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(two));
  return d;
}
// Four codes as two such pairs.
__device__ __forceinline__ void codes_to_half4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
// Four fp32 values as codes, rounded to nearest even (a NaN becomes 0x7F).
__device__ __forceinline__ uint32_t to_codes4(float x0, float x1, float x2, float x3) {
  uint32_t d;
  asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(d)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return d;
}

// scan_sequences for the block, or for up to 32 sequences by every warp for itself, one a lane, without a barrier (all write
// the same sums): 0.15 to 0.2 us of a call.
template <int NT, class Cost>
__device__ __forceinline__ uint32_t scan_sequences8(int B, uint32_t* pre_s, uint32_t* warp_s, bool* over, Cost cost) {
  if (B > 32) return scan_sequences<NT>(B, pre_s, warp_s, over, cost);
  const int lane = threadIdx.x & 31;
  const unsigned long long mine = lane < B ? cost(lane) : 0;
  uint32_t sum = (uint32_t)mine;
  bool carry = mine >> 32 != 0;
  __syncwarp();
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, sum, off);
    if (lane >= off) {
      sum += x;
      carry |= sum < x;
    }
  }
  if (lane < B) pre_s[lane + 1] = sum;
  if (lane == 0) pre_s[0] = 0;
  sum = __shfl_sync(0xFFFFFFFFu, sum, 31);
  *over = __any_sync(0xFFFFFFFFu, carry);
  __syncwarp();
  return sum;
}

// One cache as the tensor maps see it; boxes of `rows` positions of one page and head.
bool encode_pages8(CUtensorMap* m, const uint8_t* cache, const gqa_paged_dims& d, int rows);
cudaError_t launch_paged8_decode(const gqa_paged_dims& d, const Paged8Args& a, void* scratch, int ctas, cudaStream_t st);
cudaError_t launch_paged8_chunk(const gqa_paged_dims& d, const Paged8Args& a, void* scratch, int ctas, cudaStream_t st);

}  // namespace moe
