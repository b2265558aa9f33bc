// Rows of bf16 -> E2M1 codes with one scale a block of channels (sm_100a):
//   y = x H_g / sqrt(g) per block of g channels (g = 64, 128 or 256; g = 0: y = x), then per block of
//   mx: 32 channels, scale = 2^(floor(log2 max|y|) - 2), codes = E2M1(y / scale)
//   nv: 16 channels, scale = E4M3(max|y| / (6 factor)), codes = E2M1(y / (scale factor))
// and the scales in the order in which the product's tensor memory takes them (pieces of 128 rows x 4 blocks).
//
// A block of channels needs nothing from the rest of its row, so the kernel streams: 2 bytes an element in, 0.5 and a
// scale's share out, HBM its floor.  What stands in the way is the rotation.  Here a warp takes 16 rows and 4 of the
// log2(g) butterfly stages are one matrix instruction (m16n8k16, bf16 x +-1, exact products, float32 sums): lane t of
// a row's four holds 16 consecutive channels of every 64, of which the matrix turns index bits 0, 1 (within 4 channels)
// and 4, 5 (the lane), the operands' order being free; bits 2, 3, 6 and 7 are additions within the thread.  No value
// crosses lanes but a block's maximum (mx: one shuffle) and the scale bytes of a word.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "internal.h"
#include "nan_max.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace pq {
namespace {

constexpr int QF_WARPS = 8;
constexpr int QF_ROWS = 16;                 // rows a warp takes
constexpr int PIECE = 512;                  // bytes of a piece of scales
// mx: blocks whose maximum is below this count as zero, so that 1 / scale stays a normal float32.
constexpr float kTinyBlock = 7.888609052210118e-31f;     // 2^-100

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight float32 -> eight E2M1 codes (nearest, ties to even, +-6 at most), the first in the lowest nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
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
__device__ __forceinline__ uint32_t block_scales(float m0, float m1, float unit, float top, float& f0, float& f1) {
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
      const bool fine = m >= kTinyBlock && m < INFINITY;
      f = fine ? unit * __uint_as_float((256u - e) << 23) : 0.0f;
      bytes |= (fine ? e - 2u : m < kTinyBlock ? 0u : 0xFFu) << shift;   // E8M0's NaN
    };
    one(m0, f0, 0);
    one(m1, f1, 8);
    return bytes;
  }
}

// 16 channels (32 bytes) of a row: one load where they begin on 32 bytes, otherwise two.
__device__ __forceinline__ void load16(uint32_t (&w)[8], const uint16_t* p, bool in, bool aligned32) {
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

// G: 0, 64, 128 or 256.  A warp's unit is 16 rows x 128 channels (G = 256: 256); a block's warps take row_warps units one
// below the other and QF_WARPS / row_warps side by side.  Blocks go through the units in turn, the loads of the next one
// under the arithmetic of this one.
template <int G, bool NV>
__global__ void __launch_bounds__(32 * QF_WARPS, G == 256 ? 1 : 2) quant_fp4_kernel(
    const uint16_t* __restrict__ X, int rows, int64_t ldx, int D, int units, int col_blocks, int blocks, int row_warps,
    int aligned32, float unit, float top, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int NS = G == 256 ? 4 : 2;                   // spans of 64 channels
  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int row_warp = warp % row_warps, col_warp = warp / row_warps, col_warps = QF_WARPS / row_warps;
  const int pieces = NV ? (D + 63) / 64 : (D + 127) / 128;   // scale words a row

  // The +-1 matrix: row k <-> index bits (k & 1, k >> 3, lane (k >> 1) & 3), column n of half nn <-> (n & 1, nn, n >> 1).
  uint32_t b[2][2];
#pragma unroll
  for (int nn = 0; nn < 2; ++nn)
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int col = (g & 1) | (nn << 1) | ((g >> 1) << 2);
      b[nn][hi] = 0x3F803F80u | ((__popc(((hi << 1) | (t << 2)) & col) & 1) << 15) |
                  ((uint32_t)(__popc((1 | (hi << 1) | (t << 2)) & col) & 1) << 31);
    }

  uint32_t x[NS][2][8];
  int br = (int)blockIdx.x / col_blocks, bc = (int)blockIdx.x % col_blocks;
  const int step_r = (int)gridDim.x / col_blocks, step_c = (int)gridDim.x % col_blocks;
  auto load = [&]() {                                    // this thread's channels: c0 + 64 s .. + 15
    const int r0 = (br * row_warps + row_warp) * QF_ROWS, c0 = (bc * col_warps + col_warp) * 64 * NS + 16 * t;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = r0 + g + 8 * h;
        load16(x[s][h], X + (int64_t)r * ldx + c0 + 64 * s, r < rows && c0 + 64 * s < D, aligned32 != 0);
      }
  };
  load();
  for (int at = blockIdx.x; at < blocks; at += gridDim.x) {
    const int u = bc * col_warps + col_warp, r0 = (br * row_warps + row_warp) * QF_ROWS;
    const int c0 = u * 64 * NS + 16 * t;
    float v[2][NS][16];
    if constexpr (G == 0) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[h][s][2 * i] = __uint_as_float(x[s][h][i] << 16);
            v[h][s][2 * i + 1] = __uint_as_float(x[s][h][i] & 0xFFFF0000u);
          }
    } else {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int nn = 0; nn < 2; ++nn) {
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_bf16(c, x[s][0][2 * j], x[s][1][2 * j], x[s][0][2 * j + 1], x[s][1][2 * j + 1], b[nn][0], b[nn][1]);
            v[0][s][4 * j + 2 * nn] = c[0], v[0][s][4 * j + 2 * nn + 1] = c[1];
            v[1][s][4 * j + 2 * nn] = c[2], v[1][s][4 * j + 2 * nn + 1] = c[3];
          }
    }
    br += step_r, bc += step_c;
    if (bc >= col_blocks) bc -= col_blocks, ++br;
    if (at + (int)gridDim.x < blocks) load();
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
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int d = 4; d < 16; d <<= 1)
#pragma unroll
            for (int i = 0; i < 16; i += 2)
              if ((i & d) == 0) turn(v[h][s] + i, v[h][s] + i + d);
#pragma unroll
        for (int d = 1; d < G / 64; d <<= 1)
#pragma unroll
          for (int s = 0; s < NS; ++s)
            if ((s & d) == 0) {
#pragma unroll
              for (int i = 0; i < 16; i += 2) turn(v[h][s] + i, v[h][s + d] + i);
            }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + g + 8 * h;
      const bool live = r < rows;
      uint8_t* const row_codes = codes + (int64_t)r * (D / 2);
      uint32_t word[NV ? NS : NS / 2];
#pragma unroll
      for (int s2 = 0; s2 < NS; s2 += 2) {
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
        const uint32_t bytes = block_scales<NV>(m[0], m[1], unit, top, f[0], f[1]);
        if constexpr (NV) {
          word[s2] = (bytes & 0xFFu) << (8 * t);
          word[s2 + 1] = (bytes >> 8) << (8 * t);
        } else {                                         // the first span's two blocks, then the second's
          word[s2 / 2] = ((bytes & 0xFFu) | (bytes & 0xFF00u) << 8) << (8 * (t >> 1));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int s = s2 + k;
          float* y = v[h][s];
          const uint64_t f2 = ptx::f2_pack(f[k], f[k]);
#pragma unroll
          for (int i = 0; i < 16; i += 2) ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(y[i], y[i + 1]), f2), y[i], y[i + 1]);
          // times 0 an infinity or a NaN is not 0: the codes are chosen, not computed
          const uint32_t keep = f[k] != 0.0f ? 0xffffffffu : 0u;
          const uint2 q = make_uint2(e2m1x8(y) & keep, e2m1x8(y + 8) & keep);
          if (live && c0 + 64 * s < D) *reinterpret_cast<uint2*>(row_codes + (c0 + 64 * s) / 2) = q;
        }
      }
      uint8_t* const place = scales + (int64_t)(r >> 7) * pieces * PIECE + (r & 31) * 16 + ((r >> 5) & 3) * 4;
#pragma unroll
      for (int k = 0; k < (NV ? NS : NS / 2); ++k) {
        if constexpr (NV) word[k] |= __shfl_xor_sync(0xffffffffu, word[k], 1);
        word[k] |= __shfl_xor_sync(0xffffffffu, word[k], 2);
        const int piece = u * (NV ? NS : NS / 2) + k;
        if (t == 0 && live && piece < pieces) *reinterpret_cast<uint32_t*>(place + (int64_t)piece * PIECE) = word[k];
      }
    }
  }
}

template <int G, bool NV>
cudaError_t launch_fp4(const void* X, int64_t rows, int D, int64_t ldx, float factor, uint8_t* codes, uint8_t* scales,
                       cudaStream_t stream) {
  constexpr int width = G == 256 ? 256 : 128;
  const int units = (D + width - 1) / width;
  const int tiles = (int)((rows + QF_ROWS - 1) / QF_ROWS);
  int row_warps = 1;                                     // few rows: a block's warps take other channels instead
  while (row_warps < QF_WARPS && row_warps < tiles) row_warps *= 2;
  const int col_blocks = (units + QF_WARPS / row_warps - 1) / (QF_WARPS / row_warps);
  const int64_t blocks = (int64_t)col_blocks * ((tiles + row_warps - 1) / row_warps);
  if (blocks >= ((int64_t)1 << 30)) return cudaErrorInvalidConfiguration;
  const int fit = device_sm_count() * (G == 256 ? 1 : 2);
  const int aligned32 = (reinterpret_cast<uintptr_t>(X) & 31) == 0 && ldx % 16 == 0;
  const double turn = G == 0 ? 1.0 : 1.0 / std::sqrt((double)G);
  const float unit = (float)(NV ? turn / (double)factor : turn), top = (float)(turn / (6.0 * (double)factor));
  quant_fp4_kernel<G, NV><<<(unsigned)std::min<int64_t>(blocks, fit), 32 * QF_WARPS, 0, stream>>>(
      static_cast<const uint16_t*>(X), (int)rows, ldx, D, units, col_blocks, (int)blocks, row_warps, aligned32, unit, top, codes,
      scales);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_fp4(const void* X, int64_t rows, int D, int64_t ldx, int g, bool nv, float factor, uint8_t* codes,
                             uint8_t* scales, cudaStream_t stream) {
#define PQ_CASE(G) (nv ? launch_fp4<G, true>(X, rows, D, ldx, factor, codes, scales, stream) \
                       : launch_fp4<G, false>(X, rows, D, ldx, factor, codes, scales, stream))
  switch (g) {
    case 64: return PQ_CASE(64);
    case 128: return PQ_CASE(128);
    case 256: return PQ_CASE(256);
    default: return PQ_CASE(0);
  }
#undef PQ_CASE
}

}  // namespace pq
