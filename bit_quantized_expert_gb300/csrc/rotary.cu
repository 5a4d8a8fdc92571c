// Rotary positions of queries and keys (contract in include/gqa_rotary.h).
//
//   rotary_kernel  a CTA takes a few tokens.  Angles are turns in 64-bit fixed point: the position times the
//                  frequency wraps at whole turns by itself (two 32-bit multiplications; fp64, which positions past
//                  2^16 would need otherwise, has a sixty-fourth of the rate here), and the upper 32 bits are the
//                  angle in fp32.  A token's cosines and sines are made once, by as many threads as it has pairs,
//                  into shared memory, while the rows of all its heads are on their way into registers.
//
// Measured (16 query and 2 key heads of 128, in a graph): 64 tokens, half pairs, 2.0 us, the latency of a launch, a load, sines
// and a store; 8192 tokens, 96 of the dims in neighbouring pairs, 75.5 MB from and to memory, 16.4 us (4.6 TB/s, 68 % of the copy
// rate).  Steps there: 21.8 at first; 19.4 with as many tokens a CTA as fill its turns; 17.7 with quotients by a
// multiplication and without a wait for n_rows; 16.4 with two units in flight a thread and eight CTAs an SM, not four and four.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/gqa_paged.h"
#include "../../include/gqa_rotary.h"
#include "paged.cuh"

namespace moe {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotBatch = 2;       // units of a thread in flight
constexpr int kRotMaxPairs = 128;
constexpr int kRotMaxTokens = 8;   // of a CTA

struct RotaryArgs {
  const uint16_t *q, *k;
  const int32_t *positions, *n_rows;
  const unsigned long long* turns;
  uint16_t *qo, *ko;
  long long q_stride, k_stride, qo_stride, ko_stride;
  float amplitude;
  int Hq, heads, D, T, pairs;   // heads of q and of both, pairs of a head
  int tokens;                   // of a CTA
  int units, turned;            // of a head, and those that hold pairs
  uint32_t by_token, by_head;   // ceil(2^32 / d) for a token's and a head's units (0: numbers too large for it)
};

// i / d, for i * d < 2^32 by a multiplication (the quotient's excess, i * (m d - 2^32) / 2^32 d, stays below 1 / d).
__device__ __forceinline__ int quotient(int i, int d, uint32_t m) {
  return m != 0 ? (int)__umulhi((uint32_t)i, m) : i / d;
}

template <int V>
struct Words;
template <>
struct Words<8> {
  using type = uint4;
};
template <>
struct Words<4> {
  using type = uint2;
};
template <>
struct Words<2> {
  using type = uint32_t;
};
template <>
struct Words<1> {
  using type = uint16_t;
};

// V values of the 16-bit type, and V fp32 values back.
template <int V, bool FP16>
__device__ __forceinline__ void widen(const typename Words<V>::type& w, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = unpack16<FP16>(w).x;
  } else {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(&w);
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 f = unpack16<FP16>(p[e / 2]);
      x[e] = f.x;
      x[e + 1] = f.y;
    }
  }
}
template <int V, bool FP16>
__device__ __forceinline__ typename Words<V>::type narrow(const float (&x)[V]) {
  typename Words<V>::type w;
  if constexpr (V == 1) {
    w = (uint16_t)pack16<FP16>(x[0], 0.f);
  } else {
    uint32_t* p = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int e = 0; e < V; e += 2) p[e / 2] = pack16<FP16>(x[e], x[e + 1]);
  }
  return w;
}

// HALF: a unit is V firsts of pairs and their V seconds, or V dims that are copied.  Otherwise (V = 8): 8 dims, the
// pairs among them below rot_dim turned.  MANY: eight CTAs an SM, for what counts there is loads in flight (four where a
// unit is two loads of 16 bytes: 16.8 us in place of 20.7); few tokens are a matter of one chain, which the registers that
// this leaves would lengthen.
template <bool HALF, int V, bool FP16, bool MANY>
__global__ void __launch_bounds__(kRotThreads, MANY ? (HALF && V == 8 ? 4 : 8) : 1) rotary_kernel(const RotaryArgs a) {
  using W = typename Words<V>::type;
  __shared__ float2 turn_s[kRotMaxTokens * kRotMaxPairs];   // amplitude times (cosine, sine)
  pdl_wait();
  pdl_launch_dependents();
  // (Rows past n_rows are loaded as well, and not stored: nothing waits for that number before the loads.)
  const int t0 = (int)blockIdx.x * a.tokens, n = min(a.tokens, a.T - t0);
  const int rows = a.n_rows != nullptr ? *a.n_rows - t0 : n;
  const int per = a.heads * a.units, total = n * per;
  for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < total; i0 += kRotThreads * kRotBatch) {
    W x[kRotBatch], y[kRotBatch];
    uint16_t* to[kRotBatch];
    int tok[kRotBatch], unit[kRotBatch];
#pragma unroll
    for (int j = 0; j < kRotBatch; ++j) {
      const int i = i0 + j * kRotThreads;
      to[j] = nullptr;
      if (i < total) {
        tok[j] = quotient(i, per, a.by_token);
        const int r = i - tok[j] * per, h = quotient(r, a.units, a.by_head);
        unit[j] = r - h * a.units;
        const bool key = h >= a.Hq;
        const int head = key ? h - a.Hq : h;
        const uint16_t* from = (key ? a.k + (t0 + tok[j]) * a.k_stride : a.q + (t0 + tok[j]) * a.q_stride) + head * a.D;
        to[j] = (key ? a.ko + (t0 + tok[j]) * a.ko_stride : a.qo + (t0 + tok[j]) * a.qo_stride) + head * a.D;
        const int d = (HALF && unit[j] >= a.turned ? unit[j] + a.turned : unit[j]) * V;
        to[j] += d;
        x[j] = __ldcg(reinterpret_cast<const W*>(from + d));
        if (HALF && unit[j] < a.turned) y[j] = __ldcg(reinterpret_cast<const W*>(from + d + a.pairs));
      }
    }
    if (i0 == (int)threadIdx.x) {   // the first turn of every thread
      for (int i = threadIdx.x; i < n * a.pairs; i += kRotThreads) {
        const int t = i / a.pairs, p = i - t * a.pairs;
        const unsigned long long phase = (unsigned long long)(long long)a.positions[t0 + t] * a.turns[p];
        float s, c;
        sincospif((float)(int)(phase >> 32) * 0x1p-31f, &s, &c);
        turn_s[t * a.pairs + p] = make_float2(c * a.amplitude, s * a.amplitude);
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kRotBatch; ++j) {
      if (to[j] == nullptr || tok[j] >= rows) continue;
      if constexpr (HALF) {
        if (unit[j] < a.turned) {
          float u[V], v[V];
          widen<V, FP16>(x[j], u);
          widen<V, FP16>(y[j], v);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float2 w = turn_s[tok[j] * a.pairs + unit[j] * V + e];
            const float f = u[e] * w.x - v[e] * w.y;
            v[e] = u[e] * w.y + v[e] * w.x;
            u[e] = f;
          }
          *reinterpret_cast<W*>(to[j]) = narrow<V, FP16>(u);
          *reinterpret_cast<W*>(to[j] + a.pairs) = narrow<V, FP16>(v);
        } else {
          *reinterpret_cast<W*>(to[j]) = x[j];
        }
      } else {
        uint32_t* w32 = reinterpret_cast<uint32_t*>(&x[j]);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          const int p = unit[j] * (V / 2) + e;
          if (p >= a.pairs) continue;
          const float2 w = turn_s[tok[j] * a.pairs + p], f = unpack16<FP16>(w32[e]);
          w32[e] = pack16<FP16>(f.x * w.x - f.y * w.y, f.x * w.y + f.y * w.x);
        }
        *reinterpret_cast<W*>(to[j]) = x[j];
      }
    }
  }
}

// Rows of one tensor: `n` of `width` elements, `stride` apart.
struct RowSet {
  const uint16_t* p;
  long long n, width, stride;
};

// Whether two sets of rows share an element.  Sets whose strides differ are taken as blocks of memory.
bool share(const RowSet& x, const RowSet& y) {
  const long long xb = (long long)(reinterpret_cast<uintptr_t>(x.p) / 2), yb = (long long)(reinterpret_cast<uintptr_t>(y.p) / 2);
  const long long xe = xb + (x.n - 1) * x.stride + x.width, ye = yb + (y.n - 1) * y.stride + y.width;
  if (xe <= yb || ye <= xb) return false;
  if (x.stride != y.stride) return true;
  const long long off = ((yb - xb) % x.stride + x.stride) % x.stride;   // of y's rows behind x's, modulo a stride
  return off < x.width || off + y.width > x.stride;
}

template <bool HALF, int V>
cudaError_t launch(const cudaLaunchConfig_t& cfg, const RotaryArgs& a, bool fp16) {
  if (a.tokens == 1)
    return fp16 ? cudaLaunchKernelEx(&cfg, rotary_kernel<HALF, V, true, false>, a)
                : cudaLaunchKernelEx(&cfg, rotary_kernel<HALF, V, false, false>, a);
  return fp16 ? cudaLaunchKernelEx(&cfg, rotary_kernel<HALF, V, true, true>, a)
              : cudaLaunchKernelEx(&cfg, rotary_kernel<HALF, V, false, true>, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status gqa_rotary_table(const gqa_rotary_scaling* s, uint64_t* turns) {
  if (s == nullptr || turns == nullptr) return MOE_ERR_INVALID_ARG;
  const int rot = s->rot_dim;
  if (rot < 2 || rot % 2 != 0 || s->kind < GQA_ROTARY_PLAIN || s->kind > GQA_ROTARY_BY_PARTS) return MOE_ERR_INVALID_ARG;
  if (!(s->base >= 1.0) || !std::isfinite(s->base) || !(s->factor >= 1.0) || !std::isfinite(s->factor) ||
      (s->kind == GQA_ROTARY_PLAIN && s->factor != 1.0))
    return MOE_ERR_INVALID_ARG;
  if (s->kind == GQA_ROTARY_BY_PARTS && (!(s->original > 0.0) || !std::isfinite(s->original) || !(s->low >= 0.0) ||
                                         !(s->high > s->low) || !std::isfinite(s->high)))
    return MOE_ERR_INVALID_ARG;
  if (rot > 2 * kRotMaxPairs || (s->kind == GQA_ROTARY_BASE && rot == 2)) return MOE_ERR_UNSUPPORTED;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  const double base = s->kind == GQA_ROTARY_BASE ? s->base * std::pow(s->factor, (double)rot / (rot - 2)) : s->base;
  if (!std::isfinite(base)) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < rot / 2; ++i) {
    double w = std::pow(base, -2.0 * i / rot);
    if (s->kind == GQA_ROTARY_LINEAR) w /= s->factor;
    if (s->kind == GQA_ROTARY_BY_PARTS) {
      const double g = std::min(std::max((s->original * w / kTwoPi - s->low) / (s->high - s->low), 0.0), 1.0);
      w = g * w + (1.0 - g) * (w / s->factor);
    }
    turns[i] = (uint64_t)(w / kTwoPi * 18446744073709551616.0 + 0.5);   // w <= 1: below a sixth of a turn
  }
  return MOE_OK;
}

extern "C" moe_status gqa_rotary(const gqa_rotary_dims* dims, const uint16_t* q, const uint16_t* k, const int32_t* positions,
                                 const uint64_t* turns, const int32_t* n_rows, uint16_t* q_out, uint16_t* k_out,
                                 void* stream) {
  if (dims == nullptr) return MOE_ERR_INVALID_ARG;
  gqa_rotary_dims d = *dims;
  if (d.n_heads < 0 || d.n_kv_heads < 0 || (d.n_heads == 0 && d.n_kv_heads == 0) || d.head_dim < 1 || d.rot_dim < 2 ||
      d.rot_dim % 2 != 0 || d.rot_dim > d.head_dim || d.n_tokens < 0 ||
      (d.pairs != GQA_ROTARY_HALF && d.pairs != GQA_ROTARY_INTERLEAVED) ||
      (d.dtype != GQA_PAGED_BF16 && d.dtype != GQA_PAGED_FP16) || !std::isfinite(d.amplitude))
    return MOE_ERR_INVALID_ARG;
  const long long heads = (long long)d.n_heads + d.n_kv_heads, lim = 1ll << 31;
  if (d.head_dim % 8 != 0 || d.head_dim > 2 * kRotMaxPairs || heads * d.head_dim > (1 << 26) ||
      d.n_tokens * heads >= lim)
    return MOE_ERR_UNSUPPORTED;
  const long long qw = (long long)d.n_heads * d.head_dim, kw = (long long)d.n_kv_heads * d.head_dim;
  int64_t* strides[4] = {&d.q_stride, &d.q_out_stride, &d.k_stride, &d.k_out_stride};
  for (int i = 0; i < 4; ++i) {
    const long long least = i < 2 ? qw : kw;
    // (over one row, or none, a stride is never stepped)
    if (*strides[i] == 0 || d.n_tokens <= 1 || least == 0) *strides[i] = least;
    if (*strides[i] < least) return MOE_ERR_INVALID_ARG;
    if (*strides[i] >= (1ll << 39)) return MOE_ERR_UNSUPPORTED;
    if (*strides[i] % 8 != 0) return MOE_ERR_MISALIGNED;
  }
  if (d.n_tokens == 0) return MOE_OK;
  if (positions == nullptr || turns == nullptr || (qw > 0 && (q == nullptr || q_out == nullptr)) ||
      (kw > 0 && (k == nullptr || k_out == nullptr)))
    return MOE_ERR_INVALID_ARG;
  auto off = [](const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; };
  if (off(positions, 4) || off(n_rows, 4) || off(turns, 16) || (qw > 0 && (off(q, 16) || off(q_out, 16))) ||
      (kw > 0 && (off(k, 16) || off(k_out, 16))))
    return MOE_ERR_MISALIGNED;
  const RowSet qi = {q, d.n_tokens, qw, d.q_stride}, qo = {q_out, d.n_tokens, qw, d.q_out_stride};
  const RowSet ki = {k, d.n_tokens, kw, d.k_stride}, ko = {k_out, d.n_tokens, kw, d.k_out_stride};
  const bool q_in_place = q == q_out && d.q_stride == d.q_out_stride, k_in_place = k == k_out && d.k_stride == d.k_out_stride;
  if ((qw > 0 && !q_in_place && share(qi, qo)) || (kw > 0 && !k_in_place && share(ki, ko)) ||
      (qw > 0 && kw > 0 && (share(qi, ko) || share(ki, qo) || share(qo, ko))))
    return MOE_ERR_INVALID_ARG;

  RotaryArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q;
  a.k = k;
  a.positions = positions;
  a.n_rows = n_rows;
  a.turns = reinterpret_cast<const unsigned long long*>(turns);
  a.qo = q_out;
  a.ko = k_out;
  a.q_stride = d.q_stride;
  a.k_stride = d.k_stride;
  a.qo_stride = d.q_out_stride;
  a.ko_stride = d.k_out_stride;
  a.amplitude = d.amplitude;
  a.Hq = d.n_heads;
  a.heads = (int)heads;
  a.D = d.head_dim;
  a.T = d.n_tokens;
  a.pairs = d.rot_dim / 2;
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  // Wide heads' dims that stay need no copy where both tensors are turned in place.
  const bool copy = (qw > 0 && !q_in_place) || (kw > 0 && !k_in_place);
  const bool half = d.pairs == GQA_ROTARY_HALF;
  const int V = half ? (a.pairs % 8 == 0 ? 8 : a.pairs % 4 == 0 ? 4 : a.pairs % 2 == 0 ? 2 : 1) : 8;
  a.turned = half ? a.pairs / V : (d.rot_dim + 7) / 8;
  // (units of a CTA: at most 2^29, so that its counters stay within 32 bits)
  a.units = a.turned + (copy ? (half ? (d.head_dim - d.rot_dim) / V : d.head_dim / 8 - a.turned) : 0);
  // Tokens of a CTA: one while there are few, then as many as fill its turns best.
  const int per = a.heads * a.units, turn = kRotThreads * kRotBatch;
  a.tokens = 1;
  if (d.n_tokens > 4 * sms) {
    double best = 0.0;
    for (int n = 2; n <= kRotMaxTokens; ++n) {
      const double used = (double)n * per / ((((long long)n * per + turn - 1) / turn) * turn);
      if (used > best + 0.02) best = used, a.tokens = n;
    }
  }
  if ((long long)a.tokens * per * per < (1ll << 32) && per > 1 && a.units > 1) {
    a.by_token = (uint32_t)(((1ull << 32) + per - 1) / per);
    a.by_head = (uint32_t)(((1ull << 32) + a.units - 1) / a.units);
  }
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((d.n_tokens + a.tokens - 1) / a.tokens));
  cfg.blockDim = dim3(kRotThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const bool fp16 = d.dtype == GQA_PAGED_FP16;
  cudaError_t e;
  if (!half) e = launch<false, 8>(cfg, a, fp16);
  else if (V == 8) e = launch<true, 8>(cfg, a, fp16);
  else if (V == 4) e = launch<true, 4>(cfg, a, fp16);
  else if (V == 2) e = launch<true, 2>(cfg, a, fp16);
  else e = launch<true, 1>(cfg, a, fp16);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
