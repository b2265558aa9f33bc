// Device code shared by the attention kernels over the 4-bit cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace pq {
namespace ptx {

// Float32 from the shared memory of a block of the cluster.
template <int N>
__device__ __forceinline__ void ld_cluster(float (&v)[N], uint32_t cluster_addr) {
  static_assert(N == 2 || N == 4, "8 or 16 bytes");
  if constexpr (N == 4)
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(cluster_addr)
                 : "memory");
  else
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "r"(cluster_addr) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}

}  // namespace ptx

constexpr float kLog2e = 1.4426950408889634f;

// Partial results of one chunk of a context, per (token, query head): the un-normalised output [HD], then the
// reference exponent (log2) that output and sum are relative to, and the sum.
struct Partials {
  float* o;       // [chunk][T * heads_q][HD]
  float2* ml;     // [chunk][T * heads_q]
  int chunks;     // 1: no partials, the output is written directly
  int chunk_len;  // tokens of a chunk
  int sms;        // the device's
  int cluster;    // masked calls: a tile's chunks are a cluster, which joins them over its shared memory (o and ml are not used)
};

// The sum beside a row's first piece where a masked call's walk was not cut: its output is written already.
constexpr float kRowDone = -1.0f;

// Sequence b's new tokens, the first and how many: rows of the call, whatever q_start holds.
__device__ __forceinline__ void new_tokens(const int32_t* q_start, int T, int b, int& q0, int& qlen) {
  q0 = min(max(q_start[b], 0), T);
  qlen = max(0, min(max(q_start[b + 1], 0), T) - q0);
}

// Bits of the 32 tokens from `first` on that lie in [lo, hi].
__device__ __forceinline__ uint32_t token_bits32(int first, int lo, int hi) {
  const int a = lo - first, b = hi - first;
  const uint32_t upto = b < 0 ? 0u : b >= 31 ? ~0u : (2u << b) - 1;
  const uint32_t from = a <= 0 ? ~0u : a > 31 ? 0u : ~0u << a;
  return upto & from;
}

// The row's part of a tree: bits j0 .. j0 + 63 of its list, 0 outside it (j0 may be negative).
__device__ __forceinline__ uint64_t tree_bits(const uint32_t* list, int words, int j0) {
  const int k = j0 >> 5;                                 // floor
  uint32_t w[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) w[i] = k + i >= 0 && k + i < words ? __ldg(list + k + i) : 0u;
  const uint32_t lo = __funnelshift_r(w[0], w[1], j0 & 31), hi = __funnelshift_r(w[1], w[2], j0 & 31);
  return (uint64_t)hi << 32 | lo;
}

// How far behind the first of `qlen` new tokens a drafted one lies: its list holds its ancestors and itself (an empty one: 0).
__device__ __forceinline__ int tree_depth(const uint32_t* list, int words, int qlen) {
  int n = 0;
  for (int w = 0; w < words && 32 * w < qlen; ++w)
    n += __popc(__ldg(list + w) & (qlen - 32 * w >= 32 ? 0xffffffffu : (1u << (qlen - 32 * w)) - 1));
  return max(n, 1) - 1;
}

// (x & mask) ^ flip in one instruction (of two constants the compiler would make two).
__device__ __forceinline__ uint32_t and_xor(uint32_t x, uint32_t mask, uint32_t flip) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(y) : "r"(x), "r"(mask), "r"(flip));
  return y;
}

__device__ __forceinline__ uint32_t hsub2_bits(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Nibbles k and k + 4 of a word (k = 0..3) -> fp16 pairs, exactly: the codes for even k (1024 + code + 8 under 0x6400,
// less 1032) and 16 times the codes for odd k, whose bits stay four places up in the mantissa (less 1152): one shift
// a word instead of three.  The factor is taken out of the other operand (queries) or of the result (outputs).
__device__ __forceinline__ void code_pairs(uint32_t x, uint32_t (&y)[4]) {
  const uint32_t z = x >> 8;
  y[0] = hsub2_bits(and_xor(x, 0x000F000Fu, 0x64086408u), 0x64086408u);
  y[1] = hsub2_bits(and_xor(x, 0x00F000F0u, 0x64806480u), 0x64806480u);
  y[2] = hsub2_bits(and_xor(z, 0x000F000Fu, 0x64086408u), 0x64086408u);
  y[3] = hsub2_bits(and_xor(z, 0x00F000F0u, 0x64806480u), 0x64806480u);
}
constexpr float kOddNibble = 0.0625f;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// 2^x; results below the smallest normal number become 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A value scale as far as it counts toward the largest one: not if it is infinite (NaN drops out of fmaxf).
__device__ __forceinline__ float finite_or_0(float x) {
  const float y = fabsf(x);
  return y < 3.0e38f ? y : 0.0f;
}

// An exponent e with x < 2^e (x >= 0), within -100..126; 0 for x = 0.  Scores taken relative to (largest score + e)
// make probability times value scale at most 1, which fp16 holds; output and sum carry the same factor, so it
// leaves with their quotient.
__device__ __forceinline__ float scale_exponent(float x) {
  const int e = (int)(__float_as_uint(x) >> 23) - 126;
  return x == 0.0f ? 0.0f : (float)max(-100, min(126, e));
}

// The same for one token's value scale, of either sign and finite or not, within -80..126: what its score is raised by for
// the row's reference.  The lower end keeps a probability whose value is (next to) nothing below 2^80.
__device__ __forceinline__ float value_exponent(float scale) {
  return fmaxf(-80.0f, (float)min(126, (int)(__float_as_uint(finite_or_0(scale)) >> 23) - 126));
}
// A sum of probabilities from which the reference is raised although their products with the value scales are small.
constexpr float kSumTop = 1e28f;

// Queries enter the products as fp16, a row's below 2^15: exact down to 2^-25 of the row's largest channel (the odd ones
// carry a factor of 1/16).
constexpr float kQueryExp = 15.0f;

// One query row's output from its un-normalised float32 sums: lane l of the warp holds channels E l .. E l + E - 1
// (E = HD / 32).  Divides by the sum of the probabilities (none: 0), rotates back, stores bf16.
template <int HD>
__device__ __forceinline__ void finish_row(float (&o)[HD / 32], float l, int rotate, uint16_t* dst, int lane) {
  constexpr int E = HD / 32;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (rotate) {
    if constexpr (E == 4) {
      const float p0 = o[0] + o[1], p1 = o[0] - o[1], p2 = o[2] + o[3], p3 = o[2] - o[3];
      o[0] = p0 + p2, o[1] = p1 + p3, o[2] = p0 - p2, o[3] = p1 - p3;
    } else {
      const float p0 = o[0] + o[1], p1 = o[0] - o[1];
      o[0] = p0, o[1] = p1;
    }
#pragma unroll
    for (int b = 1; b < 32; b <<= 1)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float p = __shfl_xor_sync(0xffffffffu, o[i], b);
        o[i] = (lane & b) ? p - o[i] : o[i] + p;
      }
  }
  const float f = rotate ? inv * (HD == 128 ? 0.08838834764831845f : 0.125f) : inv;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(dst + 4 * lane) = make_uint2(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f));
  else
    *reinterpret_cast<uint32_t*>(dst + 2 * lane) = pack_bf16(o[0] * f, o[1] * f);
}

}  // namespace pq
