// A unit of the 4-bit floating-point quantisation: 16 rows x 128 channels (or 256 for blocks of 256) of bf16 in one warp's
// registers, rotated, to E2M1 codes and block scales (sm_100a).  Shared by the kernel for rows (quant_fp4.cu) and the product
// that quantises its few tokens itself (fp4.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "nan_max.cuh"
#include "ptx.cuh"

namespace pq {

constexpr int QF_ROWS = 16;                 // rows a warp takes
constexpr int QF_PIECE = 512;               // bytes of a piece of scales
// mx: blocks whose maximum is below this count as zero, so that 1 / scale stays a normal float32.
constexpr float kFp4TinyBlock = 7.888609052210118e-31f;     // 2^-100

__device__ __forceinline__ void mma_m16n8k16_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight float32 -> eight E2M1 codes (nearest, ties to even, +-6 at most), the first in the lowest nibble.
__device__ __forceinline__ uint32_t fp4_e2m1x8(const float* v) {
  uint32_t r;
  asm("{ .reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d}; }"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Scale bytes of two blocks from their largest magnitudes (the second's in the high byte), and what their channels are
// multiplied with (0: codes 0).  unit: the rotation's 1 / sqrt(g); nv: top = unit / (6 factor) and unit is unit / factor.
// The conversions run on the unit that makes the codes, the busiest one, so two blocks share them.
template <bool NV>
__device__ __forceinline__ uint32_t fp4_block_scales(float m0, float m1, float unit, float top, float& f0, float& f1) {
  if constexpr (NV) {
    uint16_t b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(m1 * top), "f"(m0 * top));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(b));
    const float2 s = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const bool ok0 = m0 < INFINITY, ok1 = m1 < INFINITY;   // otherwise E4M3's NaN
    f0 = ok0 && s.x > 0.0f ? __fdividef(unit, s.x) : 0.0f;
    f1 = ok1 && s.y > 0.0f ? __fdividef(unit, s.y) : 0.0f;
    return (ok0 ? b & 0xFFu : 0x7Fu) | (ok1 ? b & 0xFF00u : 0x7F00u);
  } else {
    uint32_t bytes = 0u;
    auto one = [&](float m, float& f, int shift) {
      m *= unit;
      const uint32_t e = __float_as_uint(m) >> 23;       // scale 2^(e - 129), its byte e - 2
      const bool fine = m >= kFp4TinyBlock && m < INFINITY;
      f = fine ? unit * __uint_as_float((256u - e) << 23) : 0.0f;
      bytes |= (fine ? e - 2u : m < kFp4TinyBlock ? 0u : 0xFFu) << shift;   // E8M0's NaN
    };
    one(m0, f0, 0);
    one(m1, f1, 8);
    return bytes;
  }
}

// 16 channels (32 bytes) of a row: one load where they begin on 32 bytes, otherwise two.
__device__ __forceinline__ void fp4_load16(uint32_t (&w)[8], const uint16_t* p, bool in, bool aligned32) {
  if (!in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0u;
  } else if (aligned32) {
    asm("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
        : "l"(p));
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

// What a call multiplies its sums with: nv: the rotation's 1 / sqrt(g) over the tensor's factor, and that over 6; mx: 1 / sqrt(g).
struct Fp4Scaling {
  float unit, top;
  static Fp4Scaling of(int g, bool nv, float factor) {
    const double turn = g == 0 ? 1.0 : 1.0 / std::sqrt((double)g);
    return Fp4Scaling{(float)(nv ? turn / (double)factor : turn), (float)(turn / (6.0 * (double)factor))};
  }
};

// G: 0, 64, 128 or 256.  Lane 4 g + t holds channels 64 s + 16 t .. + 15 of rows g and g + 8 (s = 0 .. SPANS - 1).
template <int G, bool NV>
struct Fp4Unit {
  static constexpr int SPANS = G == 256 ? 4 : 2;         // of 64 channels
  static constexpr int WORDS = NV ? SPANS : SPANS / 2;   // of four scale bytes a row
  uint32_t x[SPANS][2][8];

  // The lane's part of the +-1 matrix: row k <-> index bits (k & 1, k >> 3, lane (k >> 1) & 3), column n of half nn <-> (n & 1,
  // nn, n >> 1).
  static __device__ __forceinline__ void signs(uint32_t (&b)[2][2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nn = 0; nn < 2; ++nn)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const int col = (g & 1) | (nn << 1) | ((g >> 1) << 2);
        b[nn][hi] = 0x3F803F80u | ((__popc(((hi << 1) | (t << 2)) & col) & 1) << 15) |
                    ((uint32_t)(__popc((1 | (hi << 1) | (t << 2)) & col) & 1) << 31);
      }
  }

  // Rows r0 .. r0 + 15 from channel c0 on (the unit's first); what lies outside is 0.
  __device__ __forceinline__ void load(const uint16_t* X, int64_t ldx, int rows, int D, int r0, int c0, bool aligned32) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = c0 + 16 * (lane & 3);
#pragma unroll
    for (int s = 0; s < SPANS; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = r0 + g + 8 * h;
        fp4_load16(x[s][h], X + (int64_t)r * ldx + c + 64 * s, r < rows && c + 64 * s < D, aligned32);
      }
  }

  // The rotated sums of the rows (h = 0, 1: row g + 8 h), channels in their order; x is free again.
  __device__ __forceinline__ void rotate(const uint32_t (&b)[2][2], float (&v)[2][SPANS][16]) const {
    if constexpr (G == 0) {
#pragma unroll
      for (int s = 0; s < SPANS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[h][s][2 * i] = __uint_as_float(x[s][h][i] << 16);
            v[h][s][2 * i + 1] = __uint_as_float(x[s][h][i] & 0xFFFF0000u);
          }
    } else {
#pragma unroll
      for (int s = 0; s < SPANS; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int nn = 0; nn < 2; ++nn) {
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_m16n8k16_bf16(c, x[s][0][2 * j], x[s][1][2 * j], x[s][0][2 * j + 1], x[s][1][2 * j + 1], b[nn][0], b[nn][1]);
            v[0][s][4 * j + 2 * nn] = c[0], v[0][s][4 * j + 2 * nn + 1] = c[1];
            v[1][s][4 * j + 2 * nn] = c[2], v[1][s][4 * j + 2 * nn + 1] = c[3];
          }
    }
  }

  // Codes and scales of rotate's sums, which it finishes: put(h, s, q): the 16 codes of span s; put_scales(h, k, word): scale
  // word k of the row, from every lane of the row's four.
  template <typename Put, typename PutScales>
  static __device__ __forceinline__ void quantise(float (&v)[2][SPANS][16], Fp4Scaling sc, Put put, PutScales put_scales) {
    const int t = threadIdx.x & 3;
    if constexpr (G != 0) {
      // Index bits 2 and 3 within the span, 6 and 7 across spans; two neighbours an instruction.
      auto turn = [](float* a, float* c) {
        const uint64_t p = ptx::f2_pack(a[0], a[1]), q = ptx::f2_pack(c[0], c[1]);
        ptx::f2_unpack(ptx::f2_add(p, q), a[0], a[1]);
        ptx::f2_unpack(ptx::f2_sub(p, q), c[0], c[1]);
      };
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int s = 0; s < SPANS; ++s)
#pragma unroll
          for (int d = 4; d < 16; d <<= 1)
#pragma unroll
            for (int i = 0; i < 16; i += 2)
              if ((i & d) == 0) turn(v[h][s] + i, v[h][s] + i + d);
#pragma unroll
        for (int d = 1; d < G / 64; d <<= 1)
#pragma unroll
          for (int s = 0; s < SPANS; ++s)
            if ((s & d) == 0) {
#pragma unroll
              for (int i = 0; i < 16; i += 2) turn(v[h][s] + i, v[h][s + d] + i);
            }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t word[WORDS];
#pragma unroll
      for (int s2 = 0; s2 < SPANS; s2 += 2) {
        float m[2], f[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float* y = v[h][s2 + k];
          float a = max3_nan(fabsf(y[0]), fabsf(y[1]), fabsf(y[2])), b = max3_nan(fabsf(y[3]), fabsf(y[4]), fabsf(y[5]));
          a = max3_nan(a, fabsf(y[6]), fabsf(y[7]));
          b = max3_nan(b, fabsf(y[8]), fabsf(y[9]));
          a = max3_nan(a, fabsf(y[10]), fabsf(y[11]));
          b = max3_nan(b, fabsf(y[12]), fabsf(y[13]));
          m[k] = max_nan(max3_nan(a, fabsf(y[14]), fabsf(y[15])), b);
          if constexpr (!NV) m[k] = max_nan(m[k], __shfl_xor_sync(0xffffffffu, m[k], 1));
        }
        const uint32_t bytes = fp4_block_scales<NV>(m[0], m[1], sc.unit, sc.top, f[0], f[1]);
        if constexpr (NV) {
          word[s2] = (bytes & 0xFFu) << (8 * t);
          word[s2 + 1] = (bytes >> 8) << (8 * t);
        } else {                                         // the first span's two blocks, then the second's
          word[s2 / 2] = ((bytes & 0xFFu) | (bytes & 0xFF00u) << 8) << (8 * (t >> 1));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float* y = v[h][s2 + k];
          const uint64_t f2 = ptx::f2_pack(f[k], f[k]);
#pragma unroll
          for (int i = 0; i < 16; i += 2) ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(y[i], y[i + 1]), f2), y[i], y[i + 1]);
          // times 0 an infinity or a NaN is not 0: the codes are chosen, not computed
          const uint32_t keep = f[k] != 0.0f ? 0xffffffffu : 0u;
          put(h, s2 + k, make_uint2(fp4_e2m1x8(y) & keep, fp4_e2m1x8(y + 8) & keep));
        }
      }
#pragma unroll
      for (int k = 0; k < WORDS; ++k) {
        if constexpr (NV) word[k] |= __shfl_xor_sync(0xffffffffu, word[k], 1);
        word[k] |= __shfl_xor_sync(0xffffffffu, word[k], 2);
        put_scales(h, k, word[k]);
      }
    }
  }
};

}  // namespace pq
