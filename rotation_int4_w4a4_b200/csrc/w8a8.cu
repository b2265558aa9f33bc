// W8A8 GEMM with one scale per token and one per output channel (sm_100a):
//   Y[t][n] = fl(d sa[t] sw[n]),  d = sum_k qa[t][k] qw[n][k]  (exact in int32 for D <= 65536).
#include <cuda_bf16.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace pq {
namespace {

// 64 tokens x 64 channels per block of 256 threads, 64 codes of K at a time in shared memory;
// a thread forms 4 x 4 outputs with __dp4a.
constexpr int TB = 64;

__global__ void __launch_bounds__(256) w8a8_dp4a_kernel(const int8_t* __restrict__ A, const float* __restrict__ sa,
                                                        const int8_t* __restrict__ W, const float* __restrict__ sw,
                                                        void* __restrict__ Y, int64_t T, int64_t N, int D,
                                                        int out_bf16) {
  __shared__ int as[TB][TB / 4 + 1], ws[TB][TB / 4 + 1];
  const int64_t t0 = (int64_t)blockIdx.y * TB, n0 = (int64_t)blockIdx.x * TB;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  ptx::griddep_wait();
  for (int k0 = 0; k0 < D; k0 += TB) {
    const int r = threadIdx.x >> 2, c = threadIdx.x & 3;      // row, 16-byte piece
    const bool in = k0 + 16 * c < D;
    const int4 a = in && t0 + r < T ? *reinterpret_cast<const int4*>(A + (t0 + r) * D + k0 + 16 * c) : make_int4(0, 0, 0, 0);
    const int4 w = in && n0 + r < N ? *reinterpret_cast<const int4*>(W + (n0 + r) * D + k0 + 16 * c) : make_int4(0, 0, 0, 0);
    __syncthreads();
    as[r][4 * c] = a.x, as[r][4 * c + 1] = a.y, as[r][4 * c + 2] = a.z, as[r][4 * c + 3] = a.w;
    ws[r][4 * c] = w.x, ws[r][4 * c + 1] = w.y, ws[r][4 * c + 2] = w.z, ws[r][4 * c + 3] = w.w;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TB / 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(as[ty + 16 * i][k], ws[tx + 16 * j][k], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = t0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (t >= T || n >= N) continue;
      const float y = (float)acc[i][j] * sa[t] * sw[n];
      if (out_bf16) static_cast<__nv_bfloat16*>(Y)[t * N + n] = __float2bfloat16_rn(y);
      else static_cast<float*>(Y)[t * N + n] = y;
    }
}

}  // namespace

pq_status w8a8_launch(const int8_t* codes_A, const float* scales_A, const int8_t* codes_W, const float* scales_W,
                      int64_t T, int64_t N, int64_t D, void* Y, pq_out_dtype out_dtype, cudaStream_t stream,
                      bool pdl) {
  (void)pdl;
  const dim3 grid((unsigned)((N + TB - 1) / TB), (unsigned)((T + TB - 1) / TB), 1);
  w8a8_dp4a_kernel<<<grid, 256, 0, stream>>>(codes_A, scales_A, codes_W, scales_W, Y, T, N, (int)D,
                                             out_dtype == PQ_OUT_BF16 ? 1 : 0);
  return cuda_fail(cudaGetLastError(), "w8a8_dp4a_kernel launch");
}

}  // namespace pq
