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
// crosses lanes but a block's maximum (mx: one shuffle) and the scale bytes of a word (the 8-bit rows, whose butterflies go
// through shuffles, take 85 us for what is 49 here).
// 8192 x 14336, g = 128: 48.6 us nv, 47.7 mx (6.2 TB/s, 95% of the copy), g = 256 55.  Issue 67%: the floats'
// conversion to E2M1 and the scales share a slow pipe, so two blocks' scales are converted by one instruction.
#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "quant_fp4.cuh"

namespace pq {
namespace {

constexpr int QF_WARPS = 8;

// A warp's unit is 16 rows x 128 channels (G = 256: 256); a block's warps take row_warps units one below the other and QF_WARPS /
// row_warps side by side.  Blocks go through the units in turn, the loads of the next one under the arithmetic of this one.
template <int G, bool NV>
__global__ void __launch_bounds__(32 * QF_WARPS, G == 256 ? 1 : 2) quant_fp4_kernel(
    const uint16_t* __restrict__ X, int rows, int64_t ldx, int D, int col_blocks, int blocks, int row_warps, int aligned32,
    Fp4Scaling sc, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  using Unit = Fp4Unit<G, NV>;
  constexpr int WIDTH = 64 * Unit::SPANS;
  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int row_warp = warp % row_warps, col_warp = warp / row_warps, col_warps = QF_WARPS / row_warps;
  const int pieces = NV ? (D + 63) / 64 : (D + 127) / 128;   // scale words a row
  uint32_t b[2][2];
  Unit::signs(b);

  Unit x;
  int br = (int)blockIdx.x / col_blocks, bc = (int)blockIdx.x % col_blocks;
  const int step_r = (int)gridDim.x / col_blocks, step_c = (int)gridDim.x % col_blocks;
  auto load = [&]() {
    x.load(X, ldx, rows, D, (br * row_warps + row_warp) * QF_ROWS, (bc * col_warps + col_warp) * WIDTH, aligned32 != 0);
  };
  load();
  for (int at = blockIdx.x; at < blocks; at += gridDim.x) {
    const int u = bc * col_warps + col_warp, r0 = (br * row_warps + row_warp) * QF_ROWS, c0 = u * WIDTH + 16 * t;
    float v[2][Unit::SPANS][16];
    x.rotate(b, v);
    br += step_r, bc += step_c;
    if (bc >= col_blocks) bc -= col_blocks, ++br;
    if (at + (int)gridDim.x < blocks) load();
    Unit::quantise(
        v, sc,
        [&](int h, int s, uint2 q) {
          const int r = r0 + g + 8 * h;
          if (r < rows && c0 + 64 * s < D) *reinterpret_cast<uint2*>(codes + (int64_t)r * (D / 2) + (c0 + 64 * s) / 2) = q;
        },
        [&](int h, int k, uint32_t word) {
          const int r = r0 + g + 8 * h, piece = u * Unit::WORDS + k;
          if (t == 0 && r < rows && piece < pieces)
            *reinterpret_cast<uint32_t*>(scales + ((int64_t)(r >> 7) * pieces + piece) * QF_PIECE + (r & 31) * 16 + ((r >> 5) & 3) * 4) = word;
        });
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
  quant_fp4_kernel<G, NV><<<(unsigned)std::min<int64_t>(blocks, fit), 32 * QF_WARPS, 0, stream>>>(
      static_cast<const uint16_t*>(X), (int)rows, ldx, D, col_blocks, (int)blocks, row_warps, aligned32, Fp4Scaling::of(G, NV, factor), codes,
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
