// Rows of bf16 -> signed 8-bit codes with one symmetric scale a row (sm_100a):
//   y = x H_g / sqrt(g) per block of g channels (g = 64, 128 or 256; g = 0: y = x),
//   scale = max|y| / 127, codes = RNE(y / scale) in -127..127; scale NaN and codes 0 if max|y| is infinite or NaN.
// The row scale of the RRS page's set-up (per-token activation quantisation) at 8 bits (ParoQuant
// page §4.1 keeps in 8 bits what 4 bits lose); weights take the same pass, one scale an output channel.
//
// The scale needs the whole row before the first code, so a row stays in registers between its one
// read and its one write: 3 bytes move per element (2 in, 1 out) and HBM bounds the kernel, the
// shuffles next.  A thread holds 4 pieces of 8 channels (8 for the longest rows).  For a rotation it
// takes every (g / 32)-th piece of one block of g channels, so that 5 of the log2(g) butterfly stages
// run inside the thread (8 channels, 4 pieces) and only 1 to 3 across lanes: with a piece from each
// of 4 blocks a thread, the 3 to 5 stages across lanes bounded the kernel (8192 x 14336 at g = 128:
// 105 us; so 85, 4.2 TB/s of the copy's 6.55).  The factor 1/sqrt(g) goes into the scale: the codes do not depend on it.
// Without a rotation 8192 x 4096 takes 17.3 us, 5.8 TB/s.  Rows of more than 32768 channels do not fit the registers (300
// to 500 bytes a thread spill): 2048 x 40960 at g = 128 takes 114 us, 2.2 TB/s.
#include <cuda_bf16.h>

#include <cstdint>

#include "internal.h"
#include "nan_max.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace pq {
namespace {

constexpr int Q8_SLOTS = 4;           // 8-channel pieces a thread holds for rows up to 32 * 1024 channels
constexpr int Q8_SLOTS_LONG = 8;      // for longer rows
constexpr int Q8_BLOCK = 256;         // threads a block gets by stacking short rows
// Rows whose maximum is below this are taken as zero: 127 / max would overflow float32.
constexpr float kQ8Tiny = 1e-36f;

// (a, b) -> (a + b, a - b) of two neighbouring channels at once.
__device__ __forceinline__ void butterfly(float* a, float* b) {
  const uint64_t x = ptx::f2_pack(a[0], a[1]), y = ptx::f2_pack(b[0], b[1]);
  ptx::f2_unpack(ptx::f2_add(x, y), a[0], a[1]);
  ptx::f2_unpack(ptx::f2_sub(x, y), b[0], b[1]);
}

template <int G, int SLOTS>
__global__ void __launch_bounds__(1024) quant_rows8_kernel(const uint16_t* __restrict__ X, int64_t rows, int64_t ldx,
                                                           int D, int tpr, float scale_mult,
                                                           int8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ float red[2][32];
  ptx::griddep_launch_dependents();
  const int per_block = blockDim.x / tpr;
  const int sub = threadIdx.x / tpr;                       // row within the block's group of rows
  const int t = threadIdx.x - sub * tpr;
  const int lane = threadIdx.x & 31;
  const int pieces = D / 8;
  // Piece s of this thread: of its block of channels (LPG lanes each), or spread over the row.
  constexpr int LPG = G > 0 ? G / 32 : 1;
  auto piece = [&](int s) {
    return G > 0 ? (t / LPG) * (4 * LPG) + t % LPG + LPG * (s & 3) + (s >> 2) * 4 * tpr : t + s * tpr;
  };
  uint4 raw[SLOTS];
  auto load = [&](int64_t row) {
    const uint4* src = reinterpret_cast<const uint4*>(X + (row < rows ? row : 0) * ldx);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int c = piece(s);
      raw[s] = row < rows && c < pieces ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  const int64_t stride = (int64_t)gridDim.x * per_block;
  int64_t row = (int64_t)blockIdx.x * per_block + sub;
  load(row);
  // The block's rows, the loads of the next ones under the arithmetic of these (all threads take the same rounds).
  for (int64_t first = (int64_t)blockIdx.x * per_block, round = 0; first < rows; first += stride, row += stride, ++round) {
    const bool live = row < rows;
    float v[SLOTS][8];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) row_bf16x8(raw[s], v[s]);
    if (first + stride < rows) load(row + stride);
    float m = 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      if (G > 0) {                                         // stages within 8 channels, then across the block's lanes
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float a = v[s][i], b = v[s][i + 1];
          v[s][i] = a + b;
          v[s][i + 1] = a - b;
        }
#pragma unroll
        for (int h = 2; h < 8; h <<= 1)
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            if ((i & h) == 0) butterfly(v[s] + i, v[s] + i + h);
#pragma unroll
        for (int l = 1; l < LPG; l <<= 1) {
          const float sign = (lane & l) ? -1.0f : 1.0f;    // the upper lane keeps partner - own
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const uint64_t o = ptx::f2_pack(__shfl_xor_sync(0xffffffffu, v[s][i], l), __shfl_xor_sync(0xffffffffu, v[s][i + 1], l));
            ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(v[s][i], v[s][i + 1]), ptx::f2_pack(sign, sign), o), v[s][i], v[s][i + 1]);
          }
        }
      }
    }
    if (G > 0) {                                           // across the thread's pieces of the block
#pragma unroll
      for (int u = 0; u < SLOTS; u += 4)
#pragma unroll
        for (int h = 1; h < 4; h <<= 1)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            if ((s & h) == 0) {
#pragma unroll
              for (int i = 0; i < 8; i += 2) butterfly(v[u + s] + i, v[u + s + h] + i);
            }
    }
    // NaN stays in the maximum: a row that holds one must not come out as numbers
    float m2 = 0.0f;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        m = max3_nan(m, fabsf(v[s][i]), fabsf(v[s][i + 1]));
        m2 = max3_nan(m2, fabsf(v[s][i + 2]), fabsf(v[s][i + 3]));
      }
    m = max_nan(m, m2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (tpr > 32) {                                        // the same for the whole block
      // two buffers: a round's maxima are read before the round after next overwrites them
      float* buf = red[round & 1];
      if (lane == 0) buf[threadIdx.x >> 5] = m;
      __syncthreads();
      m = lane < tpr / 32 ? buf[sub * (tpr / 32) + lane] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if (!live) continue;
    const float inv = m >= kQ8Tiny && m < INFINITY ? 127.0f / m : 0.0f;
    if (t == 0) scales[row] = inv != 0.0f ? m * scale_mult : m < kQ8Tiny ? 0.0f : NAN;
    uint2* dst = reinterpret_cast<uint2*>(codes + row * D);
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
      const int c = piece(s);
      if (c >= pieces) continue;
      if (inv == 0.0f) {
        dst[c] = make_uint2(0u, 0u);
        continue;
      }
      uint32_t b[8];                                        // codes in the low bytes (1.5 * 2^23 added)
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(fmaf(v[s][i], inv, kRowRoundMagic));
      dst[c] = make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                          __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
    }
  }
}

template <int G>
cudaError_t launch_g(const void* X, int64_t rows, int D, int64_t ldx, int8_t* codes, float* scales,
                     cudaStream_t stream) {
  const int pieces = D / 8;
  const int slots = pieces <= 1024 * Q8_SLOTS ? Q8_SLOTS : Q8_SLOTS_LONG;
  const int tpr = (pieces + 32 * slots - 1) / (32 * slots) * 32;
  const int per_block = tpr < Q8_BLOCK ? Q8_BLOCK / tpr : 1;
  // blocks that run at once: 64 registers a thread
  const int64_t fit = (int64_t)device_sm_count() * (1024 / (tpr * per_block) > 0 ? 1024 / (tpr * per_block) : 1);
  const int64_t want = (rows + per_block - 1) / per_block;
  const unsigned grid = (unsigned)(want < fit ? want : fit);
  const float mult = (float)(1.0 / (127.0 * (G == 0 ? 1.0 : G == 64 ? 8.0 : G == 256 ? 16.0 : 11.313708498984761)));
  const uint16_t* x = static_cast<const uint16_t*>(X);
  if (slots == Q8_SLOTS)
    quant_rows8_kernel<G, Q8_SLOTS><<<grid, tpr * per_block, 0, stream>>>(x, rows, ldx, D, tpr, mult, codes, scales);
  else
    quant_rows8_kernel<G, Q8_SLOTS_LONG><<<grid, tpr * per_block, 0, stream>>>(x, rows, ldx, D, tpr, mult, codes, scales);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quant_rows8(const void* X, int64_t rows, int D, int64_t ldx, int g, int8_t* codes, float* scales,
                               cudaStream_t stream) {
  switch (g) {
    case 64: return launch_g<64>(X, rows, D, ldx, codes, scales, stream);
    case 128: return launch_g<128>(X, rows, D, ldx, codes, scales, stream);
    case 256: return launch_g<256>(X, rows, D, ldx, codes, scales, stream);
    default: return launch_g<0>(X, rows, D, ldx, codes, scales, stream);
  }
}

}  // namespace pq
