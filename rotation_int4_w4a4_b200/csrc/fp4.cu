// Product of E2M1 codes with one scale a block of channels on tcgen05 tensor cores (sm_100a):
//   Y[t][n] = alpha sum_b sa[t][b] sw[n][b] sum_(k in b) qa[t][k] qw[n][k]
// mx: blocks of 32 channels, E8M0 scales; nv: blocks of 16, E4M3 scales.  The tensor cores multiply the scales in
// themselves (kind::mxf4, kind::mxf4nvf4; float32 accumulator), so there is no arithmetic a block outside them.
//
// Weights are MMA operand A (output channels = tensor-memory lanes), tokens operand B, both as they lie in memory: packed
// K-major rows, 128 bytes = 256 codes a step, by TMA into the 128-byte-swizzled operand layout, zero-filled past the last
// row and the last code.  Scales lie in pieces of 128 rows x 4 blocks (512 bytes), which tcgen05.cp puts into tensor
// memory as they are; a piece serves one instruction of 64 codes (nv) or two (mx).  Rows past the end have whatever scales
// the buffer holds there: they reach their own outputs only, which nobody stores.
//
// fp4_tile_kernel: tiles of 128 channels x NP tokens (16 to 128), the reduction cut into ranges over the 1 to 8 CTAs of a
//   cluster, each with its own part of the weights in flight.  The CTAs leave their float32 partial tiles in shared memory,
//   meet, and each adds one slice of the tokens in the order of the ranges: one launch, no workspace, the same bits each
//   time.
//   warp 0: TMA producer; warp 1: tensor memory, scale copies and MMA issue; warps 2..5: epilogue.
//
// Every mbarrier wait is bounded; a timeout sets the library's status word, the CTA drains what it has in flight, meets
// its cluster, frees tensor memory and returns.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace pq {
namespace {

constexpr int KB = 128;                 // bytes of a K step a row = a swizzle row: 256 codes
constexpr int PIECE = 512;              // bytes of a piece of scales
constexpr uint64_t kWaitNs = 2000000000ull;

// Scale pieces of 128 rows in a K step.
template <bool NV> constexpr int kPieces = NV ? 4 : 2;

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, int* abort_flag, unsigned int* status) {
  if (ptx::mbar_wait_bounded(bar, parity, abort_flag, kWaitNs)) return true;
  *abort_flag = 1;
  atomicOr(status, PQ_DEV_TIMEOUT);
  return false;
}

// One lane polls for the warp.
__device__ __forceinline__ bool warp_wait_or_abort(uint64_t* bar, uint32_t parity, int* abort_flag,
                                                   unsigned int* status) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait_or_abort(bar, parity, abort_flag, status) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

// While draining: bounded in time only.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  int never = 0;
  (void)ptx::mbar_wait_bounded(bar, parity, &never, kWaitNs);
}

__device__ __forceinline__ void store_y(void* Y, int64_t idx, float y, int out_bf16) {
  if (out_bf16) static_cast<__nv_bfloat16*>(Y)[idx] = __float2bfloat16_rn(y);
  else static_cast<float*>(Y)[idx] = y;
}

// ------------------------------------------------------------------------------------ tile kernel
constexpr int TM = 128;                 // weight rows per tile
constexpr int T_THREADS = 192;

// NP: token columns of a tile.  DEEP: stages for one CTA per SM (about 220 KB in flight), otherwise for two.
template <int NP, bool NV, bool DEEP> struct TileGeom {
  static constexpr int SF = kPieces<NV> * PIECE;          // scale bytes of 128 rows a step
  static constexpr uint32_t TX = (TM + NP) * KB + 2 * SF;
  static constexpr int STAGES = ((DEEP ? 227 : 113) * 1024 - 2048) / (int)TX;
  // Tensor memory: the accumulator, then each stage's scales, 4 columns a piece (its own, so that no copy overwrites
  // scales that an earlier instruction may still read).
  static constexpr uint32_t STAGE_COLS = 2 * 4 * kPieces<NV>;
  static constexpr uint32_t USED = NP + STAGES * STAGE_COLS;
  static constexpr uint32_t COLS = USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
  static_assert(USED <= 512 && (DEEP || COLS <= 256), "tensor memory");
  static_assert(STAGES >= 2, "stages");
};

template <int NP, bool NV, bool DEEP> struct __align__(1024) TileSmem {
  using Geom = TileGeom<NP, NV, DEEP>;
  uint8_t a[Geom::STAGES][TM * KB];
  uint8_t b[Geom::STAGES][NP * KB];
  uint8_t sa[Geom::STAGES][Geom::SF], sb[Geom::STAGES][Geom::SF];
  uint64_t full[Geom::STAGES], empty[Geom::STAGES];
  uint64_t acc_full;
  uint32_t tmem_slot;
  int abort_flag;
};

// Token column c of the cluster's R partial tiles (float32 [token][128 channels] at the same offset in each), 4 channels a
// lane, added in the order of the ranges.
template <int R>
__device__ __forceinline__ void add_ranges(float (&d)[4], uint32_t base, int c, int lane) {
  int4 v[R];
#pragma unroll
  for (int p = 0; p < R; ++p) v[p] = ptx::ld_cluster_v4(ptx::mapa_shared(base + 16u * (uint32_t)(c * (TM / 4) + lane), (uint32_t)p));
#pragma unroll
  for (int p = 0; p < R; ++p) {
    d[0] += __int_as_float(v[p].x), d[1] += __int_as_float(v[p].y);
    d[2] += __int_as_float(v[p].z), d[3] += __int_as_float(v[p].w);
  }
}

// Grid: x = tile * split + range (the cluster), tiles channel-fastest.  tmSW, tmSA: the scale pieces as rows of 256 bytes;
// pieces: 512-byte pieces of 128 rows of a tensor.  codes64: 64-code products of the whole reduction.
template <int NP, bool NV, bool DEEP>
__global__ void __launch_bounds__(T_THREADS) fp4_tile_kernel(
    const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmSW,
    const __grid_constant__ CUtensorMap tmSA, float alpha, void* __restrict__ Y, int T, int N, int steps, int codes64,
    int pieces, int m_tiles, int split, int out_bf16, int pdl, unsigned int* status) {
  using Geom = TileGeom<NP, NV, DEEP>;
  constexpr int STAGES = Geom::STAGES;
  extern __shared__ unsigned char smem_raw[];
  TileSmem<NP, NV, DEEP>& S =
      *reinterpret_cast<TileSmem<NP, NV, DEEP>*>(smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u));
  static_assert(sizeof(S.a) + sizeof(S.b) >= sizeof(float) * TM * NP, "partial tile overlays the stages");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = (int)blockIdx.x / split, rank = (int)blockIdx.x % split;
  const int m0 = (tile % m_tiles) * TM, t0 = (tile / m_tiles) * NP;   // NP < 128: one tile of tokens (t0 = 0)
  const int per = (steps + split - 1) / split;
  const int k0 = min(steps, rank * per), k1 = min(steps, k0 + per);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(&S.full[s], 1);
      ptx::mbar_init(&S.empty[s], 1);
    }
    ptx::mbar_init(&S.acc_full, 1);
    S.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmSW);
    ptx::prefetch_tmap(&tmSA);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&S.tmem_slot, Geom::COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = S.tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      const int sw0 = (m0 / 128) * pieces * 2, sa0 = (t0 / 128) * pieces * 2;
      auto weights = [&](int s, int kb) {
        ptx::mbar_arrive_expect_tx(&S.full[s], Geom::TX);
        ptx::tma_load_2d(S.a[s], &tmW, &S.full[s], kb * KB, m0);
        ptx::tma_load_2d(S.sa[s], &tmSW, &S.full[s], 0, sw0 + kb * kPieces<NV> * 2);
      };
      auto tokens = [&](int s, int kb) {
        ptx::tma_load_2d(S.b[s], &tmA, &S.full[s], kb * KB, t0);
        ptx::tma_load_2d(S.sb[s], &tmSA, &S.full[s], 0, sa0 + kb * kPieces<NV> * 2);
      };
      // The first ring of weights is requested before the wait for the kernel that writes the token codes.
      const int head = min(STAGES, k1 - k0);
      for (int i = 0; i < head; ++i) weights(i, k0 + i);
      if (pdl) ptx::griddep_wait();
      for (int i = 0; i < head; ++i) tokens(i, k0 + i);
      int step = head;
      for (int kb = k0 + head; kb < k1; ++kb, ++step) {
        const int s = step % STAGES;
        if (!wait_or_abort(&S.empty[s], ((uint32_t)(step / STAGES) & 1u) ^ 1u, &S.abort_flag, status)) break;
        weights(s, kb);
        tokens(s, kb);
      }
      // Every load has landed and every stage's release has arrived before the CTA may exit.
      for (int j = (step > STAGES ? step - STAGES : 0); j < step; ++j) {
        drain_wait(&S.full[j % STAGES], (uint32_t)(j / STAGES) & 1u);
        drain_wait(&S.empty[j % STAGES], (uint32_t)(j / STAGES) & 1u);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      for (int kb = k0, step = 0; kb < k1; ++kb, ++step) {
        const int s = step % STAGES;
        if (!wait_or_abort(&S.full[s], (uint32_t)(step / STAGES) & 1u, &S.abort_flag, status)) break;
        ptx::tc_fence_after();
        const uint32_t sa = tmem + NP + (uint32_t)s * Geom::STAGE_COLS, sb = sa + 4 * kPieces<NV>;
        const int live = min(4, codes64 - 4 * kb);        // 64-code products that are not all padding
#pragma unroll
        for (int p = 0; p < kPieces<NV>; ++p) {
          ptx::tmem_copy_scales<false>(sa + 4 * p, ptx::smem_desc_rows16(ptx::smem_addr(S.sa[s]) + PIECE * p));
          ptx::tmem_copy_scales<false>(sb + 4 * p, ptx::smem_desc_rows16(ptx::smem_addr(S.sb[s]) + PIECE * p));
        }
        const uint32_t a0 = ptx::smem_addr(S.a[s]), b0 = ptx::smem_addr(S.b[s]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          constexpr uint32_t id0 = ptx::idesc_e2m1(!NV, TM, NP, 0), id1 = ptx::idesc_e2m1(!NV, TM, NP, NV ? 0 : 2);
          const uint32_t col = 4 * (NV ? k : k / 2);
          if (k < live)
            ptx::umma_e2m1<NV, false>(tmem, ptx::smem_desc_sw128(a0 + 32 * k), ptx::smem_desc_sw128(b0 + 32 * k),
                                      k & 1 ? id1 : id0, sa + col, sb + col, step > 0 || k > 0 ? 1u : 0u);
        }
        ptx::umma_commit(&S.empty[s]);
      }
      ptx::umma_commit(&S.acc_full);
      drain_wait(&S.acc_full, 0);
    }
  } else {
    if (pdl) ptx::griddep_wait();                         // Y may still be read by what ran before
    const int sub = warp & 3;
    const int n = m0 + 32 * sub + lane;
    const bool some = k1 > k0;                            // an empty range contributes zeros
    bool ok = true;
    if (some) ok = warp_wait_or_abort(&S.acc_full, 0, &S.abort_flag, status);
    ptx::tc_fence_after();
    const uint32_t col0 = tmem + ((uint32_t)(32 * sub) << 16);
    float* part = reinterpret_cast<float*>(S.a);          // [token][128 channels], over the finished stages
    // Rolled: it runs once a CTA.
#pragma unroll 1
    for (int c = 0; c < NP; c += 16) {
      uint32_t r[16];
      if (some && ok) {
        ptx::tmem_ld32x16(col0 + c, r);
        ptx::tmem_ld_wait(r);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = 0u;
      }
      if (split > 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * TM + 32 * sub + lane] = __uint_as_float(r[i]);
      } else if (n < N) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = t0 + c + i;
          if (t < T) store_y(Y, (int64_t)t * N + n, alpha * __uint_as_float(r[i]), out_bf16);
        }
      }
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  if (split > 1) {
    ptx::cluster_sync();                                  // every partial tile is written
    // This CTA adds token columns rank, rank + split, ... over the cluster; a warp takes one column, a lane 4 channels of
    // it, with the reads of all the cluster's tiles (and of two columns) in flight at once.
    const uint32_t mine = ptx::smem_addr(S.a);
    constexpr int W = T_THREADS / 32;
    const int n = m0 + 4 * lane;
    const int columns = min(NP, T - t0);
    for (int c0 = rank + split * warp; c0 < columns; c0 += 2 * split * W) {
      float d[2][4] = {};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = c0 + u * split * W;
        if (c < columns) {
          if (split == 2) add_ranges<2>(d[u], mine, c, lane);
          else if (split == 4) add_ranges<4>(d[u], mine, c, lane);
          else add_ranges<8>(d[u], mine, c, lane);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = c0 + u * split * W;
        if (c < columns) {
          const int64_t at = (int64_t)(t0 + c) * N + n;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (n + k < N) store_y(Y, at + k, alpha * d[u][k], out_bf16);
        }
      }
    }
    ptx::cluster_sync();                                  // nobody leaves while its tile is read
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, Geom::COLS);
  }
}

// ----------------------------------------------------------------------------------------- launch
struct Fp4Maps {
  CUtensorMap w, a, sw, sa;
};

pq_status make_maps(Fp4Maps* m, const uint8_t* codes_A, const uint8_t* scales_A, const uint8_t* codes_W,
                    const uint8_t* scales_W, int64_t T, int64_t N, int64_t D, int64_t pieces, int pieces_step, int a_rows) {
  const auto scale_map = [&](CUtensorMap* map, const uint8_t* base, int64_t rows) {
    return make_u8_tile_map(map, base, (rows + 127) / 128 * pieces * 2, 256, 256, 2 * pieces_step, /*swizzle128=*/false);
  };
  cudaError_t e = make_u8_tile_map(&m->w, codes_W, N, D / 2, KB, TM, /*swizzle128=*/true);
  if (e == cudaSuccess) e = make_u8_tile_map(&m->a, codes_A, T, D / 2, KB, a_rows, /*swizzle128=*/true);
  if (e == cudaSuccess) e = scale_map(&m->sw, scales_W, N);
  if (e == cudaSuccess) e = scale_map(&m->sa, scales_A, T);
  return cuda_fail(e, "4-bit operand tensor map");
}

struct Fp4Call {
  float alpha;
  void* Y;
  int T, N, steps, codes64, pieces, bf16;
  bool pdl;
  unsigned int* status;
  cudaStream_t stream;
};

template <int NP, bool NV, bool DEEP>
pq_status launch_tile(const Fp4Maps& m, const Fp4Call& c, int m_tiles, int64_t tiles, int split) {
  constexpr size_t smem = sizeof(TileSmem<NP, NV, DEEP>) + 1024;
  static_assert((DEEP ? 1 : 2) * smem <= 232448, "shared memory exceeds 227 KB an SM");
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = set_kernel_attributes(reinterpret_cast<const void*>(fp4_tile_kernel<NP, NV, DEEP>), (int)smem, done);
  if (e != cudaSuccess) return cuda_fail(e, "fp4_tile_kernel attributes");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split), 1, 1);
  cfg.blockDim = dim3(T_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = c.pdl ? 2 : 1;
  return cuda_fail(cudaLaunchKernelEx(&cfg, fp4_tile_kernel<NP, NV, DEEP>, m.w, m.a, m.sw, m.sa, c.alpha, c.Y, c.T, c.N, c.steps,
                                      c.codes64, c.pieces, m_tiles, split, c.bf16, c.pdl ? 1 : 0, c.status),
                   "fp4_tile_kernel launch");
}

template <bool NV>
pq_status run(const uint8_t* codes_A, const uint8_t* scales_A, const uint8_t* codes_W, const uint8_t* scales_W, int64_t T,
              int64_t N, int64_t D, Fp4Call c) {
  const int sms = device_sm_count();
  const int np = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
  const int64_t m_tiles = (N + TM - 1) / TM, tiles = m_tiles * ((T + np - 1) / np);
  if (tiles >= ((int64_t)1 << 31)) { set_error("too many output tiles"); return PQ_ERR_INVALID_ARG; }
  // Ranges of the reduction: as long as every CTA still has an SM of its own and keeps some steps.
  int split = 1;
  while (split < 8 && tiles * split * 2 <= sms && c.steps >= 4 * split) split *= 2;
  Fp4Maps m;
  const pq_status st = make_maps(&m, codes_A, scales_A, codes_W, scales_W, T, N, D, c.pieces, kPieces<NV>, np);
  if (st != PQ_OK) return st;
#define PQ_TILE_CASE(NP)                                                                   \
  (tiles * split <= sms ? launch_tile<NP, NV, true>(m, c, (int)m_tiles, tiles, split) \
                        : launch_tile<NP, NV, false>(m, c, (int)m_tiles, tiles, split))
  return np == 16 ? PQ_TILE_CASE(16) : np == 32 ? PQ_TILE_CASE(32) : np == 64 ? PQ_TILE_CASE(64) : PQ_TILE_CASE(128);
#undef PQ_TILE_CASE
}

}  // namespace

pq_status fp4_launch(const uint8_t* codes_A, const uint8_t* scales_A, const uint8_t* codes_W, const uint8_t* scales_W,
                     int64_t T, int64_t N, int64_t D, bool nv, float alpha, void* Y, pq_out_dtype out_dtype,
                     cudaStream_t stream, bool pdl) {
  unsigned int* status = nullptr;
  const cudaError_t e = gemm_status_address(&status);
  if (e != cudaSuccess) return cuda_fail(e, "status word");
  const Fp4Call c = {alpha, Y, (int)T, (int)N, (int)((D + 2 * KB - 1) / (2 * KB)), (int)((D + 63) / 64),
                     (int)(nv ? (D + 63) / 64 : (D + 127) / 128), out_dtype == PQ_OUT_BF16 ? 1 : 0, pdl, status, stream};
  return nv ? run<true>(codes_A, scales_A, codes_W, scales_W, T, N, D, c)
            : run<false>(codes_A, scales_A, codes_W, scales_W, T, N, D, c);
}

}  // namespace pq
