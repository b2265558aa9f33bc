// One pass from a projection's queries, keys and values to attention's operands (sm_100a).
// Per token and head, in float32:
//   1. queries and keys: x <- (x r) w, r = 1 / sqrt(mean x^2 + eps)           (if norm weights are given)
//   2. queries and keys: the first rope_dim channels turned by the position's angles, pairs (i, i + rope_dim / 2)
//      or (2i, 2i + 1): (a, b) -> (a cos - b sin, b cos + a sin)              (if a table is given)
//   3. y = x H / sqrt(hd)                                                     (if the cache is rotated)
//   4. queries: bf16(y).  Keys, values: scale = max|y| / 7, code = RNE(y / scale), two codes a byte, into the
//      token's slot of the paged cache (a maximum that is infinite or NaN: scale NaN, codes 0).
// (OSTQuant page: Hadamard on Q and K after the position rotation, one rotation per head for V; RRS page,
// set-up of the experiments: the cache quantised in groups of 128, here the head.)
//
// Bytes bound it: every input is read and every output written once (4 bytes a query channel, 2.5 + 4/hd a key or
// value channel), all else stays in registers.  A head is spread over a few lanes: the norm's sum and the head's
// maximum are shuffle trees over those lanes, the rotation's partner and the Hadamard stages beyond a lane's channels
// are shuffles too, so nothing goes through shared memory.
//
// A code sits next to a rounding border now and then, so the arithmetic is pinned: products and sums are rounded one by
// one (no contraction into FMAs), sums are taken over neighbours first, and the factor of each head is
// 7 * (1 / max).  The same formula written out in float32 gives the same codes bit for bit.
#include <cuda_bf16.h>

#include <cstdint>

#include "internal.h"
#include "kv4.h"
#include "nan_max.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace pq {
namespace {

// Heads whose maximum is below this are taken as zero (7 / max would overflow float32).
constexpr float kKv4Tiny = 1e-36f;

// bf16 channels of a lane: 4 consecutive (8-byte aligned), or 8 of the head's first half and the same 8 of its second.
template <int HD, int E, bool WIDE>
__device__ __forceinline__ void ap_load(float (&v)[E], const uint16_t* head, int e0) {
#pragma unroll
  for (int c = 0; c < E; c += 8) {
    const uint16_t* p = head + e0 + c * (HD / 16);      // c = 8: HD / 2 further on
    if constexpr (WIDE) {
      row_bf16x8(__ldg(reinterpret_cast<const uint4*>(p)), v + c);
    } else {
#pragma unroll
      for (int k = 0; k < (E < 8 ? E : 8); k += 4) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p + k));
        v[c + k] = __uint_as_float(w.x << 16), v[c + k + 1] = __uint_as_float(w.x & 0xFFFF0000u);
        v[c + k + 2] = __uint_as_float(w.y << 16), v[c + k + 3] = __uint_as_float(w.y & 0xFFFF0000u);
      }
    }
  }
}

__device__ __forceinline__ uint32_t ap_bf16x2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Products of pairs, each rounded on its own (mul.rn: as __fmul_rn).
__device__ __forceinline__ void ap_mul2(float& a, float& b, float c, float d) {
  ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(a, b), ptx::f2_pack(c, d)), a, b);
}

// (a, b) -> (a cos - b sin, b cos + a sin) of N channel pairs.
template <int N>
__device__ __forceinline__ void ap_turn(float* a, float* b, const float* cos, const float* sin) {
#pragma unroll
  for (int c = 0; c < N; c += 4) {
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(cos + c)), s4 = __ldg(reinterpret_cast<const float4*>(sin + c));
    const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {                         // (scalar: a packed product and sum may become one packed FMA)
      const float x = a[c + k], y = b[c + k];
      a[c + k] = __fsub_rn(__fmul_rn(x, cc[k]), __fmul_rn(y, ss[k]));
      b[c + k] = __fadd_rn(__fmul_rn(y, cc[k]), __fmul_rn(x, ss[k]));
    }
  }
}

// A head is LANES lanes of E channels, a warp takes 32 / LANES heads of one kind (queries, keys or values) of one token,
// a block one token's warps (blockIdx.x; more than 16 warps: blockIdx.y too).
// E = 16: 8 channels of each half of the head.  The pairs of a position rotation of the whole head then meet inside a
// thread, loads and stores cover 128 contiguous bytes of a head, and shuffles and reductions are shared by four times
// the channels (8192 tokens of 32 + 8 + 8 heads of 128: 66 us, 3.0 TB/s of the copy's 6.55, the L1 pipe that carries loads,
// stores and shuffles bounding it, 24 bytes of spills a thread among them; 95 us with 4 channels a lane everywhere).
// E = 4: any layout of the rotation (halves that do not fall on multiples of 8 channels, or cross the middle).
template <int HD, int E, bool WIDE>
__global__ void __launch_bounds__(512, 3) kv4_append_kernel(const Kv4AppendArgs a) {
  constexpr int LANES = HD / E;
  constexpr int HPW = 32 / LANES;                       // heads per warp
  constexpr bool SPLIT = E == 16;
  const int lane = threadIdx.x & 31;
  const int l = lane & (LANES - 1);                     // lane within the head
  const int e0 = (SPLIT ? 8 : 4) * l;                   // its first channel
  const int heads = a.cache.heads;
  const int wq = (a.heads_q + HPW - 1) / HPW, wk = (heads + HPW - 1) / HPW;   // warps a token for queries; keys or values
  const int64_t t = blockIdx.x;
  const int64_t slot = a.slots[t];
  const int pos = a.rope ? a.positions[t] : 0;
  int w = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (w >= wq + 2 * wk) return;                         // whole warps
  const int kind = w < wq ? 0 : w < wq + wk ? 1 : 2;    // query, key, value
  w -= kind == 0 ? 0 : kind == 1 ? wq : wq + wk;
  const int h = w * HPW + lane / LANES;
  const bool live = h < (kind == 0 ? a.heads_q : heads);

  float v[E];
  {
    const uint16_t* src = kind == 0 ? a.Q + t * a.ldq : kind == 1 ? a.K + t * a.ldk : a.V + t * a.ldv;
    ap_load<HD, E, WIDE>(v, src + (live ? h : 0) * HD, e0);
  }
  const uint16_t* norm = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
  if (norm) {                                           // the same for the whole warp
    // sum of squares, neighbours first: the thread's channels, the lanes, then the head's halves
    float s[E];
#pragma unroll
    for (int c = 0; c < E; c += 2) {
      s[c] = v[c], s[c + 1] = v[c + 1];
      ap_mul2(s[c], s[c + 1], v[c], v[c + 1]);
    }
#pragma unroll
    for (int o = 1; o < (SPLIT ? 8 : 4); o <<= 1)
#pragma unroll
      for (int c = 0; c < E; c += 2 * o) s[c] = __fadd_rn(s[c], s[c + o]);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
      s[0] = __fadd_rn(s[0], __shfl_xor_sync(0xffffffffu, s[0], o));
      if constexpr (SPLIT) s[8] = __fadd_rn(s[8], __shfl_xor_sync(0xffffffffu, s[8], o));
    }
    if constexpr (SPLIT) s[0] = __fadd_rn(s[0], s[8]);
    const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(s[0], 1.0f / HD), a.eps)));
    float g[E];
    ap_load<HD, E, WIDE>(g, norm, e0);
#pragma unroll
    for (int c = 0; c < E; c += 2) {
      ap_mul2(v[c], v[c + 1], r, r);
      ap_mul2(v[c], v[c + 1], g[c], g[c + 1]);
    }
  }
  bool bad = false;
  if (a.rope) {
    bad = pos < 0 || pos >= a.rope_rows;
    if (kind < 2) {
      const int half = a.rope_dim / 2;
      const float* row = a.rope + (int64_t)(bad ? 0 : pos) * a.rope_dim;
      if (a.interleaved) {
#pragma unroll
        for (int c = 0; c < E; c += 4) {
          const int e = e0 + (c >= 8 ? HD / 2 + c - 8 : c);
          if (e < a.rope_dim) {
            const float2 cs = __ldg(reinterpret_cast<const float2*>(row + e / 2));
            const float2 sn = __ldg(reinterpret_cast<const float2*>(row + half + e / 2));
            const float x0 = v[c], x1 = v[c + 1], x2 = v[c + 2], x3 = v[c + 3];
            v[c] = __fsub_rn(__fmul_rn(x0, cs.x), __fmul_rn(x1, sn.x));
            v[c + 1] = __fadd_rn(__fmul_rn(x1, cs.x), __fmul_rn(x0, sn.x));
            v[c + 2] = __fsub_rn(__fmul_rn(x2, cs.y), __fmul_rn(x3, sn.y));
            v[c + 3] = __fadd_rn(__fmul_rn(x3, cs.y), __fmul_rn(x2, sn.y));
          }
        }
      } else if (SPLIT && half == HD / 2) {
        ap_turn<(SPLIT ? 8 : 0)>(v, v + (SPLIT ? 8 : 0), row + e0, row + half + e0);
      } else {
        // the partner channels are some lanes away (SPLIT: in the head's first half, which holds all that turn)
        constexpr int N = SPLIT ? 8 : 4;
        const bool first = e0 < half, turns = e0 < a.rope_dim;
        const int from = (lane + (first ? half / N : -(half / N))) & 31;
        float o[N];
#pragma unroll
        for (int c = 0; c < N; ++c) o[c] = __shfl_sync(0xffffffffu, v[c], from);
        if (turns) {
          if (first) {
            ap_turn<N>(v, o, row + e0, row + half + e0);
          } else {
            ap_turn<N>(o, v, row + e0 - half, row + e0);
          }
        }
      }
    }
  }
  const bool rotate = kind < 2 ? a.cache.rotate_k != 0 : a.cache.rotate_v != 0;
  if (rotate) {
    // Hadamard butterflies, neighbours first: within 8 (or 4) channels, across the lanes, across the head's halves
    constexpr int N = SPLIT ? 8 : 4;
#pragma unroll
    for (int c = 0; c < E; c += 2) {
      const float x = v[c], y = v[c + 1];
      v[c] = x + y;
      v[c + 1] = x - y;
    }
#pragma unroll
    for (int o = 2; o < N; o <<= 1)
#pragma unroll
      for (int c = 0; c < E; c += 2)
        if ((c & o) == 0) {
          const uint64_t x = ptx::f2_pack(v[c], v[c + 1]), y = ptx::f2_pack(v[c + o], v[c + o + 1]);
          ptx::f2_unpack(ptx::f2_add(x, y), v[c], v[c + 1]);
          ptx::f2_unpack(ptx::f2_sub(x, y), v[c + o], v[c + o + 1]);
        }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
      // the upper lane of a pair keeps the difference: partner - own
      const float sign = (l & o) ? -1.0f : 1.0f;
#pragma unroll
      for (int c = 0; c < E; c += 2) {
        const uint64_t p = ptx::f2_pack(__shfl_xor_sync(0xffffffffu, v[c], o), __shfl_xor_sync(0xffffffffu, v[c + 1], o));
        ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(v[c], v[c + 1]), ptx::f2_pack(sign, sign), p), v[c], v[c + 1]);
      }
    }
    if constexpr (SPLIT) {
#pragma unroll
      for (int c = 0; c < 8; c += 2) {
        const uint64_t x = ptx::f2_pack(v[c], v[c + 1]), y = ptx::f2_pack(v[c + 8], v[c + 9]);
        ptx::f2_unpack(ptx::f2_add(x, y), v[c], v[c + 1]);
        ptx::f2_unpack(ptx::f2_sub(x, y), v[c + 8], v[c + 9]);
      }
    }
  }
  if (bad && lane == 0) atomicOr(a.status, PQ_DEV_BAD_INDEX);
  // 1 / sqrt(hd), and that over 7
  constexpr float kNorm = HD == 128 ? (float)0.08838834764831845 : 0.125f;
  constexpr float kStep = (float)(1.0 / (7.0 * (HD == 128 ? 11.313708498984761 : 8.0)));
  if (kind == 0) {
    if (!live) return;
    const float f = rotate ? kNorm : 1.0f;
    uint16_t* dst = a.Q_out + (t * a.heads_q + h) * (int64_t)HD + e0;
    uint32_t y[E / 2];
#pragma unroll
    for (int c = 0; c < E; c += 2) {
      ap_mul2(v[c], v[c + 1], f, f);
      y[c / 2] = bad ? 0u : ap_bf16x2(v[c], v[c + 1]);
    }
    if constexpr (SPLIT) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<uint4*>(dst + HD / 2) = make_uint4(y[4], y[5], y[6], y[7]);
    } else {
      *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
    }
    return;
  }
  float m = 0.0f;
#pragma unroll
  for (int c = 0; c < E; c += 2) m = max3_nan(m, fabsf(v[c]), fabsf(v[c + 1]));
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!live) return;
  if (slot < 0 || bad) return;
  const int64_t page = slot >> a.cache.page_shift;
  if (page >= a.cache.pages) {
    if (l == 0) atomicOr(a.status, PQ_DEV_BAD_INDEX);
    return;
  }
  const int64_t in_page = slot & ((1 << a.cache.page_shift) - 1);
  const int64_t at = (((page * heads + h) << a.cache.page_shift) + in_page);
  const bool some = m >= kKv4Tiny && m < INFINITY;
  const float inv = some ? __fmul_rn(__frcp_rn(m), 7.0f) : 0.0f;
  uint8_t* codes = (kind == 1 ? a.cache.k_codes : a.cache.v_codes) + at * (HD / 2) + e0 / 2;
  uint32_t packed[E / 4];
#pragma unroll
  for (int c = 0; c < E; c += 4) {
    uint32_t b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) b[k] = __float_as_uint(__fadd_rn(__fmul_rn(v[c + k], inv), kRowRoundMagic));
    packed[c / 4] = some ? (b[0] & 15u) | ((b[1] & 15u) << 4) | ((b[2] & 15u) << 8) | ((b[3] & 15u) << 12) : 0u;
  }
  if constexpr (SPLIT) {
    *reinterpret_cast<uint32_t*>(codes) = packed[0] | (packed[1] << 16);
    *reinterpret_cast<uint32_t*>(codes + HD / 4) = packed[2] | (packed[3] << 16);
  } else {
    *reinterpret_cast<uint16_t*>(codes) = (uint16_t)packed[0];
  }
  if (l == 0) {
    float* scales = kind == 1 ? a.cache.k_scales : a.cache.v_scales;
    scales[at] = some ? __fmul_rn(m, rotate ? kStep : (float)(1.0 / 7.0)) : m < kKv4Tiny ? 0.0f : NAN;
  }
}

// Cached rows back as bf16(code * scale), in the cache's own basis; rows without a slot become 0.  A block a token, a
// thread a 4-byte piece (8 channels).
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4View c, const int64_t* __restrict__ slots,
                                                       uint16_t* __restrict__ K_out, uint16_t* __restrict__ V_out,
                                                       unsigned int* status) {
  const int64_t t = blockIdx.x;
  const int wshift = c.head_dim == 128 ? 4 : 3;          // words a head, log2
  const int per = c.heads << wshift;
  const int64_t slot = __ldg(slots + t);
  const int64_t page = slot >> c.page_shift;
  const bool in = slot >= 0 && page < c.pages;
  if (slot >= 0 && !in && threadIdx.x == 0) atomicOr(status, PQ_DEV_BAD_INDEX);
  for (int r = threadIdx.x; r < 2 * per; r += blockDim.x) {
    const bool kv = r >= per;
    const int p = kv ? r - per : r;
    const int h = p >> wshift;
    uint4 y = make_uint4(0u, 0u, 0u, 0u);
    if (in) {
      const int64_t at = ((page * c.heads + h) << c.page_shift) + (slot & ((1 << c.page_shift) - 1));
      const uint32_t x = reinterpret_cast<const uint32_t*>((kv ? c.v_codes : c.k_codes))[(at << wshift) + (p & ((1 << wshift) - 1))];
      const float s = (kv ? c.v_scales : c.k_scales)[at];
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        o[k] = ap_bf16x2((float)((int)(x << (28 - 8 * k)) >> 28) * s, (float)((int)(x << (24 - 8 * k)) >> 28) * s);
      y = make_uint4(o[0], o[1], o[2], o[3]);
    }
    *reinterpret_cast<uint4*>((kv ? V_out : K_out) + (t * per + p) * 8) = y;
  }
}

template <int HD, int E, bool WIDE>
cudaError_t launch_append(const Kv4AppendArgs& a, cudaStream_t stream) {
  constexpr int HPW = 32 / (HD / E);
  const int warps = (a.heads_q + HPW - 1) / HPW + 2 * ((a.cache.heads + HPW - 1) / HPW);
  const int rounds = (warps + 15) / 16, block = (warps + rounds - 1) / rounds;
  kv4_append_kernel<HD, E, WIDE><<<dim3((unsigned)a.T, (unsigned)rounds), 32 * block, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t stream) {
  const int hd = a.cache.head_dim;
  const bool wide = hd == 128;
  // Rotations of the whole head, of 8-channel groups within its first half, or of neighbours suit 16 channels a lane.
  if (!a.rope || a.interleaved || a.rope_dim == hd || (a.rope_dim % 16 == 0 && a.rope_dim <= hd / 2)) {
    const bool vec = aligned16(a.Q) && aligned16(a.K) && aligned16(a.V) && a.ldq % 8 == 0 && a.ldk % 8 == 0 && a.ldv % 8 == 0 &&
                     aligned16(a.q_norm) && aligned16(a.k_norm);
    if (vec) return wide ? launch_append<128, 16, true>(a, stream) : launch_append<64, 16, true>(a, stream);
    return wide ? launch_append<128, 16, false>(a, stream) : launch_append<64, 16, false>(a, stream);
  }
  return wide ? launch_append<128, 4, false>(a, stream) : launch_append<64, 4, false>(a, stream);
}

cudaError_t launch_kv4_read(const Kv4View& c, const int64_t* slots, int64_t T, uint16_t* K_out, uint16_t* V_out,
                            unsigned int* status, cudaStream_t stream) {
  const int per = 2 * c.heads * (c.head_dim / 8);
  const int threads = per >= 256 ? 256 : (per + 31) / 32 * 32;
  kv4_read_kernel<<<(unsigned)T, threads, 0, stream>>>(c, slots, K_out, V_out, status);
  return cudaGetLastError();
}

}  // namespace pq
