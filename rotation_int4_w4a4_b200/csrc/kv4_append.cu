// One pass from a projection's queries, keys and values to attention's operands (sm_100a).
// Per token and head, in float32:
//   1. queries and keys: x <- (x r) w, r = 1 / sqrt(mean x^2 + eps)           (if norm weights are given)
//   2. queries and keys: the first rope_dim channels turned by the position's angles, pairs (i, i + rope_dim / 2)
//      or (2i, 2i + 1): (a, b) -> (a cos - b sin, b cos + a sin)              (if a table is given)
//   3. y = x H / sqrt(hd)                                                     (if the cache is rotated)
//   4. queries: bf16(y).  Keys, values: scale = max|y| / 7, code = RNE(y / scale), two codes a byte, into the
//      token's slot of the paged cache.
// (OSTQuant page: Hadamard on Q and K after the position rotation, one rotation per head for V; RRS page,
// set-up of the experiments: the cache quantised in groups of 128, here the head.)
//
// Bytes bound it: every input is read and every output written once (4 bytes a query channel, 2.5 + 4/hd a key or
// value channel), all else stays in registers.  A head is hd / 4 lanes of 4 channels: the norm's sum and the head's
// maximum are shuffle trees over those lanes, the rotation's partner and the Hadamard stages beyond 4 channels are
// shuffles too, so nothing goes through shared memory.
//
// A code sits next to a rounding border now and then, so the arithmetic is pinned: products and sums are rounded one by
// one (no contraction into FMAs), sums are taken over neighbours first, and the factor of each head is
// 7 * (1 / max).  The same formula written out in float32 gives the same codes bit for bit.
#include <cuda_bf16.h>

#include <cstdint>

#include "internal.h"
#include "kv4.h"
#include "ptx.cuh"
#include "rows.cuh"

namespace pq {
namespace {

constexpr int AP_WARPS = 8;
// Heads whose maximum is below this are taken as zero (7 / max would overflow float32).
constexpr float kKv4Tiny = 1e-36f;

__device__ __forceinline__ float4 ap_load4(const uint16_t* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}

__device__ __forceinline__ uint2 ap_bf16x4(const float (&v)[4]) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// A warp takes 32 / LANES heads of one token; HD = 4 LANES.
template <int LANES>
__global__ void __launch_bounds__(32 * AP_WARPS) kv4_append_kernel(const Kv4AppendArgs a) {
  constexpr int HD = 4 * LANES;
  constexpr int HPW = 32 / LANES;                       // heads per warp
  const int lane = threadIdx.x & 31;
  const int l = lane & (LANES - 1);                     // lane within the head
  const int e0 = 4 * l;                                 // its first channel
  const int heads = a.heads_q + 2 * a.cache.heads;
  const int groups = (heads + HPW - 1) / HPW;           // warps per token
  const int64_t warp = (int64_t)blockIdx.x * AP_WARPS + (threadIdx.x >> 5);
  const int64_t t = warp / groups;
  if (t >= a.T) return;                                 // whole warps
  const int head = (int)(warp - t * groups) * HPW + lane / LANES;
  const bool live = head < heads;
  const int kind = head < a.heads_q ? 0 : head < a.heads_q + a.cache.heads ? 1 : 2;   // query, key, value
  const int h = kind == 0 ? head : kind == 1 ? head - a.heads_q : head - a.heads_q - a.cache.heads;

  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (live) {
    const uint16_t* src = kind == 0 ? a.Q + t * a.ldq : kind == 1 ? a.K + t * a.ldk : a.V + t * a.ldv;
    const float4 x = ap_load4(src + h * HD + e0);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  }
  const uint16_t* norm = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
  if (a.q_norm || a.k_norm) {
    float s = __fadd_rn(__fadd_rn(__fmul_rn(v[0], v[0]), __fmul_rn(v[1], v[1])),
                        __fadd_rn(__fmul_rn(v[2], v[2]), __fmul_rn(v[3], v[3])));
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
    if (live && norm) {
      const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(s, 1.0f / HD), a.eps)));
      const float4 w = ap_load4(norm + e0);
      v[0] = __fmul_rn(__fmul_rn(v[0], r), w.x);
      v[1] = __fmul_rn(__fmul_rn(v[1], r), w.y);
      v[2] = __fmul_rn(__fmul_rn(v[2], r), w.z);
      v[3] = __fmul_rn(__fmul_rn(v[3], r), w.w);
    }
  }
  bool bad = false;
  if (a.rope) {
    const int pos = a.positions[t];
    bad = pos < 0 || pos >= a.rope_rows;
    const int half = a.rope_dim / 2;
    const float* row = a.rope + (int64_t)(bad ? 0 : pos) * a.rope_dim;
    const bool turns = live && kind < 2 && e0 < a.rope_dim;
    if (a.interleaved) {
      if (turns) {
        const float2 c = *reinterpret_cast<const float2*>(row + e0 / 2);
        const float2 s = *reinterpret_cast<const float2*>(row + half + e0 / 2);
        const float x0 = v[0], x1 = v[1], x2 = v[2], x3 = v[3];
        v[0] = __fsub_rn(__fmul_rn(x0, c.x), __fmul_rn(x1, s.x));
        v[1] = __fadd_rn(__fmul_rn(x1, c.x), __fmul_rn(x0, s.x));
        v[2] = __fsub_rn(__fmul_rn(x2, c.y), __fmul_rn(x3, s.y));
        v[3] = __fadd_rn(__fmul_rn(x3, c.y), __fmul_rn(x2, s.y));
      }
    } else {
      // the partner channels are half / 4 lanes away
      const bool first = e0 < half;
      const int from = lane + (first ? half / 4 : -(half / 4));
      float o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __shfl_sync(0xffffffffu, v[i], from & 31);
      if (turns) {
        const int e = first ? e0 : e0 - half;
        const float4 c = *reinterpret_cast<const float4*>(row + e);
        const float4 s = *reinterpret_cast<const float4*>(row + half + e);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __fmul_rn(v[i], cc[i]), q = __fmul_rn(o[i], ss[i]);
          v[i] = first ? __fsub_rn(p, q) : __fadd_rn(p, q);
        }
      }
    }
  }
  const bool rotate = kind < 2 ? a.cache.rotate_k != 0 : a.cache.rotate_v != 0;
  if (a.cache.rotate_k || a.cache.rotate_v) {
    float y[4];
    {
      const float p0 = v[0] + v[1], p1 = v[0] - v[1], p2 = v[2] + v[3], p3 = v[2] - v[3];
      y[0] = p0 + p2, y[1] = p1 + p3, y[2] = p0 - p2, y[3] = p1 - p3;
    }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = __shfl_xor_sync(0xffffffffu, y[i], o);
        y[i] = (l & o) ? p - y[i] : y[i] + p;
      }
    if (rotate) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = y[i];
    }
  }
  float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (bad && lane == 0) atomicOr(a.status, PQ_DEV_BAD_INDEX);
  if (!live) return;
  // 1 / sqrt(hd), and that over 7
  constexpr float kNorm = HD == 128 ? (float)0.08838834764831845 : 0.125f;
  constexpr float kStep = (float)(1.0 / (7.0 * (HD == 128 ? 11.313708498984761 : 8.0)));
  if (kind == 0) {
    if (rotate) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __fmul_rn(v[i], kNorm);
    }
    if (bad) v[0] = v[1] = v[2] = v[3] = 0.0f;
    *reinterpret_cast<uint2*>(a.Q_out + (t * a.heads_q + h) * (int64_t)HD + e0) = ap_bf16x4(v);
    return;
  }
  const int64_t slot = a.slots[t];
  if (slot < 0 || bad) return;
  const int64_t page = slot >> a.cache.page_shift;
  if (page >= a.cache.pages) {
    if (l == 0) atomicOr(a.status, PQ_DEV_BAD_INDEX);
    return;
  }
  const int64_t in_page = slot & ((1 << a.cache.page_shift) - 1);
  const int64_t at = (((page * a.cache.heads + h) << a.cache.page_shift) + in_page);
  const bool zero = !(m >= kKv4Tiny);
  const float inv = zero ? 0.0f : __fmul_rn(__frcp_rn(m), 7.0f);
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(__fadd_rn(__fmul_rn(v[i], inv), kRowRoundMagic)) & 15u;
  const uint16_t packed = (uint16_t)(b[0] | (b[1] << 4) | (b[2] << 8) | (b[3] << 12));
  uint8_t* codes = kind == 1 ? a.cache.k_codes : a.cache.v_codes;
  *reinterpret_cast<uint16_t*>(codes + at * (HD / 2) + 2 * l) = packed;
  if (l == 0) {
    float* scales = kind == 1 ? a.cache.k_scales : a.cache.v_scales;
    scales[at] = zero ? 0.0f : __fmul_rn(m, rotate ? kStep : (float)(1.0 / 7.0));
  }
}

// Cached rows back as bf16(code * scale), in the cache's own basis; rows without a slot become 0.  One thread a
// 4-byte piece (8 channels).
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4View c, const int64_t* __restrict__ slots, int64_t T,
                                                       uint16_t* __restrict__ K_out, uint16_t* __restrict__ V_out,
                                                       unsigned int* status) {
  const int words = c.head_dim / 8;
  const int64_t per_token = 2 * (int64_t)c.heads * words;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t t = i / per_token;
  if (t >= T) return;
  const int r = (int)(i - t * per_token);
  const int kv = r >= c.heads * words;
  const int h = (r - kv * c.heads * words) / words, w = r % words;
  uint16_t* out = kv ? V_out : K_out;
  const int64_t slot = slots[t];
  const int64_t page = slot >> c.page_shift;
  uint4 y = make_uint4(0u, 0u, 0u, 0u);
  if (slot >= 0 && page < c.pages) {
    const int64_t at = ((page * c.heads + h) << c.page_shift) + (slot & ((1 << c.page_shift) - 1));
    const uint32_t x = reinterpret_cast<const uint32_t*>((kv ? c.v_codes : c.k_codes))[at * words + w];
    const float s = (kv ? c.v_scales : c.k_scales)[at];
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float lo = (float)((int)(x << (28 - 8 * k)) >> 28) * s, hi = (float)((int)(x << (24 - 8 * k)) >> 28) * s;
      const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
      o[k] = *reinterpret_cast<const uint32_t*>(&p);
    }
    y = make_uint4(o[0], o[1], o[2], o[3]);
  } else if (slot >= 0) {
    atomicOr(status, PQ_DEV_BAD_INDEX);
  }
  *reinterpret_cast<uint4*>(out + (t * c.heads + h) * (int64_t)c.head_dim + 8 * w) = y;
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t stream) {
  const int heads = a.heads_q + 2 * a.cache.heads;
  const int hpw = a.cache.head_dim == 128 ? 1 : 2;
  const int64_t warps = a.T * ((heads + hpw - 1) / hpw);
  const unsigned grid = (unsigned)((warps + AP_WARPS - 1) / AP_WARPS);
  if (a.cache.head_dim == 128) kv4_append_kernel<32><<<grid, 32 * AP_WARPS, 0, stream>>>(a);
  else kv4_append_kernel<16><<<grid, 32 * AP_WARPS, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4View& c, const int64_t* slots, int64_t T, uint16_t* K_out, uint16_t* V_out,
                            unsigned int* status, cudaStream_t stream) {
  const int64_t n = T * 2 * c.heads * (c.head_dim / 8);
  kv4_read_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(c, slots, T, K_out, V_out, status);
  return cudaGetLastError();
}

}  // namespace pq
