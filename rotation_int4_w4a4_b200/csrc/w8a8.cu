// W8A8 GEMM with one scale per token and one per output channel on tcgen05 tensor cores (sm_100a):
//   Y[t][n] = fl(fl(fl(d) sa[t]) sw[n]),  d = sum_k qa[t][k] qw[n][k]
// d is exact: int8 products summed in int32 (D <= 65536, so |d| <= 2^30).  Integer sums do not depend on their order,
// so neither the split of the reduction nor the tile changes a bit of the result.
//
// Both kernels take weights as MMA operand A (output channels = tensor-memory lanes) and tokens as operand B, both as
// they lie in memory: K-major rows of 128 bytes by TMA into the 128-byte-swizzled operand layout, zero-filled past
// the last row and the last code.  A warp's store of one token then covers 32 consecutive channels.
//
// w8a8_pair_kernel (many output tiles): persistent, one CTA per SM, clusters of two CTAs that share every MMA
//   (cta_group::2, M256 N256 K32; each SM loads 128 weight rows and 128 tokens per 128-code step).  The whole
//   reduction of a 256 x 256 tile runs in one accumulator, and there are two (512 columns of tensor memory), so the
//   epilogue of a tile overlaps the next tile's reduction.  Tensor-bound.
//   warp 0: TMA producer; warp 1: tensor memory, MMA issue (even CTA); warps 4..11: epilogue, two a lane quarter.
//
// w8a8_tile_kernel (few tiles: decode batches, short prompts, narrow layers): tiles of 128 channels x NP tokens (16 to
//   128), the reduction cut into ranges over the 1 to 8 CTAs of a cluster, each with its own part of the weights in
//   flight: at these sizes streaming the weights is the work, and it takes every SM's loads to fill HBM.  The CTAs
//   leave their int32 partial tiles in shared memory, meet, and each adds one slice of the tokens over the cluster's
//   shared memory: one launch, no workspace.
//   warp 0: TMA producer; warp 1: tensor memory, MMA issue; warps 2..5: epilogue.
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

constexpr int KB = 128;                 // codes per K step = bytes of a swizzle row
constexpr uint64_t kWaitNs = 2000000000ull;

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

__device__ __forceinline__ void store_y(void* Y, int64_t idx, int d, float sa, float sw, int out_bf16) {
  const float y = (float)d * sa * sw;
  if (out_bf16) static_cast<__nv_bfloat16*>(Y)[idx] = __float2bfloat16_rn(y);
  else static_cast<float*>(Y)[idx] = y;
}

// ------------------------------------------------------------------------------------ pair kernel
constexpr int PM = 128;                 // weight rows per CTA
constexpr int PN = 256;                 // tokens per tile
constexpr int PN_HALF = PN / 2;         // tokens each CTA stages
constexpr int P_STAGES = 6;
constexpr int P_THREADS = 384;
constexpr int P_EPI_WARP0 = 4;
constexpr int P_EPI_COLS = PN / 2;      // tokens per epilogue warp
constexpr uint32_t P_TX = 2 * (PM + PN_HALF) * KB;   // both CTAs' bytes, on the even CTA's barrier

struct __align__(1024) PairSmem {
  uint8_t a[P_STAGES][PM * KB];
  uint8_t b[P_STAGES][PN_HALF * KB];
  uint64_t full[P_STAGES], empty[P_STAGES];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t mma_done, pair_done;
  uint32_t tmem_slot;
  int abort_flag;
};
constexpr size_t kPairSmem = sizeof(PairSmem) + 1024;
static_assert(kPairSmem <= 232448, "shared memory exceeds 227 KB");

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P_THREADS, 1) w8a8_pair_kernel(
    const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, const float* __restrict__ scales_A,
    const float* __restrict__ scales_W, void* __restrict__ Y, int T, int N, int steps, int m_tiles, int tiles,
    int out_bf16, unsigned int* status) {
  extern __shared__ unsigned char smem_raw[];
  PairSmem& S = *reinterpret_cast<PairSmem*>(smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)ptx::cluster_ctarank();
  const int first = (int)(blockIdx.x >> 1), stride = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < P_STAGES; ++s) {
      ptx::mbar_init(&S.full[s], 1);
      ptx::mbar_init(&S.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&S.acc_full[b], 1);
      ptx::mbar_init(&S.acc_empty[b], 2 * 8);            // both CTAs' epilogue warps
    }
    ptx::mbar_init(&S.mma_done, 1);
    ptx::mbar_init(&S.pair_done, 1);
    S.abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmA);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(&S.tmem_slot, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = S.tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full0 = ptx::mapa_shared(ptx::smem_addr(&S.full[0]), 0);
      int step = 0;
      bool ok = true;
      for (int u = first; u < tiles && ok; u += stride) {
        const int m0 = (u % m_tiles) * 2 * PM + PM * rank, n0 = (u / m_tiles) * PN + PN_HALF * rank;
        for (int kb = 0; kb < steps; ++kb, ++step) {
          const int s = step % P_STAGES;
          if (!wait_or_abort(&S.empty[s], ((uint32_t)(step / P_STAGES) & 1u) ^ 1u, &S.abort_flag, status)) { ok = false; break; }
          if (rank == 0) ptx::mbar_arrive_expect_tx(&S.full[s], P_TX);
          ptx::tma_load_2d_pair(S.a[s], &tmW, full0 + 8u * s, kb * KB, m0);
          ptx::tma_load_2d_pair(S.b[s], &tmA, full0 + 8u * s, kb * KB, n0);
        }
      }
      // Every load issued has landed and every release aimed at this CTA has arrived before it may exit.
      const int j0 = step > P_STAGES ? step - P_STAGES : 0;
      if (rank == 0)
        for (int j = j0; j < step; ++j) drain_wait(&S.full[j % P_STAGES], (uint32_t)(j / P_STAGES) & 1u);
      for (int j = j0; j < step; ++j) drain_wait(&S.empty[j % P_STAGES], (uint32_t)(j / P_STAGES) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = ptx::idesc_s8_s32(2 * PM, PN);
      int step = 0, tile = 0;
      bool ok = true;
      for (int u = first; u < tiles && ok; u += stride, ++tile) {
        const int b = tile & 1;
        if (!wait_or_abort(&S.acc_empty[b], ((uint32_t)(tile >> 1) & 1u) ^ 1u, &S.abort_flag, status)) { ok = false; break; }
        ptx::tc_fence_after();
        const uint32_t d = tmem + (uint32_t)b * PN;
        for (int kb = 0; kb < steps; ++kb, ++step) {
          const int s = step % P_STAGES;
          if (!wait_or_abort(&S.full[s], (uint32_t)(step / P_STAGES) & 1u, &S.abort_flag, status)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t a0 = ptx::smem_addr(S.a[s]), b0 = ptx::smem_addr(S.b[s]);
#pragma unroll
          for (int k = 0; k < KB / 32; ++k)
            ptx::umma_s8_pair(d, ptx::smem_desc_sw128(a0 + 32 * k), ptx::smem_desc_sw128(b0 + 32 * k), idesc,
                              kb > 0 || k > 0 ? 1u : 0u);
          ptx::umma_commit_pair(&S.empty[s], 0x3);
        }
        if (!ok) break;
        ptx::umma_commit_pair(&S.acc_full[b], 0x3);
      }
      ptx::umma_commit_pair(&S.mma_done, 0x1);
      drain_wait(&S.mma_done, 0);
      for (int j = (tile > 2 ? tile - 2 : 0); j < tile; ++j) drain_wait(&S.acc_empty[j & 1], (uint32_t)(j >> 1) & 1u);
    }
  } else if (warp >= P_EPI_WARP0) {
    // Lane quarter warp % 4 (channels), token half of the tile.
    const int ew = warp - P_EPI_WARP0;
    const int sub = warp & 3, half = ew >> 2;
    const uint32_t acc_empty0 = ptx::mapa_shared(ptx::smem_addr(&S.acc_empty[0]), 0);
    int tile = 0;
    for (int u = first; u < tiles; u += stride, ++tile) {
      const int b = tile & 1;
      const int n = (u % m_tiles) * 2 * PM + PM * rank + 32 * sub + lane;       // this thread's channel
      const int t0 = (u / m_tiles) * PN + P_EPI_COLS * half;
      const float sw = n < N ? __ldg(scales_W + n) : 0.0f;
      // The token scales of this half, 4 a lane; the epilogue shuffles them out.
      float sa_l[P_EPI_COLS / 32];
#pragma unroll
      for (int i = 0; i < P_EPI_COLS / 32; ++i) sa_l[i] = t0 + 32 * i + lane < T ? __ldg(scales_A + t0 + 32 * i + lane) : 0.0f;
      if (!warp_wait_or_abort(&S.acc_full[b], (uint32_t)(tile >> 1) & 1u, &S.abort_flag, status)) break;
      ptx::tc_fence_after();
      const uint32_t col0 = tmem + ((uint32_t)(32 * sub) << 16) + (uint32_t)(b * PN + half * P_EPI_COLS);
#pragma unroll 1
      for (int c = 0; c < P_EPI_COLS / 32; ++c) {
        uint32_t r[32];
        ptx::tmem_ld32(col0 + 32 * c, r);
        ptx::tmem_ld_wait(r);
        if (c == P_EPI_COLS / 32 - 1) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_remote(acc_empty0 + 8u * b);
        }
        const float sa_c = c == 0 ? sa_l[0] : c == 1 ? sa_l[1] : c == 2 ? sa_l[2] : sa_l[3];
        const int t = t0 + 32 * c;
        const int live = min(32, T - t);
        const int64_t base = (int64_t)t * N + n;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float sa = __shfl_sync(0xffffffffu, sa_c, i);
          if (i < live && n < N) store_y(Y, base + (int64_t)i * N, (int)r[i], sa, sw, out_bf16);
        }
      }
    }
  }

  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  // Neither CTA leaves while its peer may still arrive on its barriers or read its tiles.
  if (threadIdx.x == 0) {
    ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_addr(&S.pair_done), (uint32_t)rank ^ 1u));
    int never = 0;
    if (!ptx::mbar_wait_bounded_cl(&S.pair_done, 0, &never, kWaitNs)) atomicOr(status, PQ_DEV_TIMEOUT);
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------------------------ tile kernel
constexpr int TM = 128;                 // weight rows per tile
constexpr int T_THREADS = 192;

// NP: token columns of a tile.  DEEP: stages for one CTA per SM (about 200 KB in flight), otherwise for two.
template <int NP, bool DEEP> struct TileGeom {
  static constexpr int SHALLOW = NP == 16 ? 6 : NP == 32 ? 5 : NP == 64 ? 4 : 3;
  static constexpr int STAGES = DEEP ? 2 * SHALLOW : SHALLOW;
  static constexpr uint32_t TX = (TM + NP) * KB;
  static constexpr uint32_t COLS = NP < 32 ? 32 : NP;
};

template <int NP, bool DEEP> struct __align__(1024) TileSmem {
  uint8_t a[TileGeom<NP, DEEP>::STAGES][TM * KB];
  uint8_t b[TileGeom<NP, DEEP>::STAGES][NP * KB];
  uint64_t full[TileGeom<NP, DEEP>::STAGES], empty[TileGeom<NP, DEEP>::STAGES];
  uint64_t acc_full;
  uint32_t tmem_slot;
  int abort_flag;
};

// Token column c of the cluster's R partial tiles (int32 [token][128 channels] at the same offset in each), 4 channels a
// lane.
template <int R>
__device__ __forceinline__ void add_ranges(int4& d, uint32_t base, int c, int lane) {
  int4 v[R];
#pragma unroll
  for (int p = 0; p < R; ++p) v[p] = ptx::ld_cluster_v4(ptx::mapa_shared(base + 16u * (uint32_t)(c * (TM / 4) + lane), (uint32_t)p));
#pragma unroll
  for (int p = 0; p < R; ++p) d.x += v[p].x, d.y += v[p].y, d.z += v[p].z, d.w += v[p].w;
}

// Grid: x = tile * split + range (the cluster), tiles channel-fastest.
template <int NP, bool DEEP>
__global__ void __launch_bounds__(T_THREADS) w8a8_tile_kernel(
    const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, const float* __restrict__ scales_A,
    const float* __restrict__ scales_W, void* __restrict__ Y, int T, int N, int steps, int m_tiles, int split,
    int out_bf16, int pdl, unsigned int* status) {
  using Geom = TileGeom<NP, DEEP>;
  constexpr int STAGES = Geom::STAGES;
  extern __shared__ unsigned char smem_raw[];
  TileSmem<NP, DEEP>& S = *reinterpret_cast<TileSmem<NP, DEEP>*>(smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u));
  static_assert(sizeof(S.a) + sizeof(S.b) >= sizeof(int) * TM * NP, "partial tile overlays the stages");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tile = (int)blockIdx.x / split, rank = (int)blockIdx.x % split;
  const int m0 = (tile % m_tiles) * TM, t0 = (tile / m_tiles) * NP;
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
      // The first ring of weights is requested before the wait for the kernel that writes the token codes.
      const int head = min(STAGES, k1 - k0);
      for (int i = 0; i < head; ++i) {
        ptx::mbar_arrive_expect_tx(&S.full[i], Geom::TX);
        ptx::tma_load_2d(S.a[i], &tmW, &S.full[i], (k0 + i) * KB, m0);
      }
      if (pdl) ptx::griddep_wait();
      for (int i = 0; i < head; ++i) ptx::tma_load_2d(S.b[i], &tmA, &S.full[i], (k0 + i) * KB, t0);
      int step = head;
      for (int kb = k0 + head; kb < k1; ++kb, ++step) {
        const int s = step % STAGES;
        if (!wait_or_abort(&S.empty[s], ((uint32_t)(step / STAGES) & 1u) ^ 1u, &S.abort_flag, status)) break;
        ptx::mbar_arrive_expect_tx(&S.full[s], Geom::TX);
        ptx::tma_load_2d(S.a[s], &tmW, &S.full[s], kb * KB, m0);
        ptx::tma_load_2d(S.b[s], &tmA, &S.full[s], kb * KB, t0);
      }
      // Every load has landed and every stage's release has arrived before the CTA may exit.
      for (int j = (step > STAGES ? step - STAGES : 0); j < step; ++j) {
        drain_wait(&S.full[j % STAGES], (uint32_t)(j / STAGES) & 1u);
        drain_wait(&S.empty[j % STAGES], (uint32_t)(j / STAGES) & 1u);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = ptx::idesc_s8_s32(TM, NP);
      for (int kb = k0, step = 0; kb < k1; ++kb, ++step) {
        const int s = step % STAGES;
        if (!wait_or_abort(&S.full[s], (uint32_t)(step / STAGES) & 1u, &S.abort_flag, status)) break;
        ptx::tc_fence_after();
        const uint32_t a0 = ptx::smem_addr(S.a[s]), b0 = ptx::smem_addr(S.b[s]);
#pragma unroll
        for (int k = 0; k < KB / 32; ++k)
          ptx::umma_s8(tmem, ptx::smem_desc_sw128(a0 + 32 * k), ptx::smem_desc_sw128(b0 + 32 * k), idesc,
                       step > 0 || k > 0 ? 1u : 0u);
        ptx::umma_commit(&S.empty[s]);
      }
      ptx::umma_commit(&S.acc_full);
      drain_wait(&S.acc_full, 0);
    }
  } else {
    if (pdl) ptx::griddep_wait();
    const int sub = warp & 3;
    const int n = m0 + 32 * sub + lane;
    const bool some = k1 > k0;                            // an empty range contributes zeros
    bool ok = true;
    if (some) ok = warp_wait_or_abort(&S.acc_full, 0, &S.abort_flag, status);
    ptx::tc_fence_after();
    const uint32_t col0 = tmem + ((uint32_t)(32 * sub) << 16);
    int* part = reinterpret_cast<int*>(S.a);              // [token][128 channels], over the finished stages
    const float sw = n < N ? __ldg(scales_W + n) : 0.0f;
    // Rolled: this runs once a CTA, and unrolled over 128 columns it was bound by the fetch of its own code (391 x 1003 x
    // 4176: 9 of 26 thousand cycles).
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
        for (int i = 0; i < 16; ++i) part[(c + i) * TM + 32 * sub + lane] = (int)r[i];
      } else if (n < N) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int t = t0 + c + i;
          if (t < T) store_y(Y, (int64_t)t * N + n, (int)r[i], __ldg(scales_A + t), sw, out_bf16);
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
    if (pdl) ptx::griddep_wait();
    const uint32_t mine = ptx::smem_addr(S.a);
    constexpr int W = T_THREADS / 32;
    const int n = m0 + 4 * lane;
    float sw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) sw[k] = n + k < N ? __ldg(scales_W + n + k) : 0.0f;
    const int columns = min(NP, T - t0);
    for (int c0 = rank + split * warp; c0 < columns; c0 += 2 * split * W) {
      int4 d[2] = {make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0)};
      float sa[2] = {0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = c0 + u * split * W;
        if (c < columns) {
          sa[u] = __ldg(scales_A + t0 + c);
          if (split == 2) add_ranges<2>(d[u], mine, c, lane);
          else if (split == 4) add_ranges<4>(d[u], mine, c, lane);
          else add_ranges<8>(d[u], mine, c, lane);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = c0 + u * split * W;
        if (c < columns) {
          const int v[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
          const int64_t at = (int64_t)(t0 + c) * N + n;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (n + k < N) store_y(Y, at + k, v[k], sa[u], sw[k], out_bf16);
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
pq_status operand_map(CUtensorMap* map, const int8_t* base, int64_t rows, int64_t D, int box_rows) {
  const cudaError_t e = make_u8_tile_map(map, base, rows, D, KB, box_rows, /*swizzle128=*/true);
  return cuda_fail(e, "8-bit operand tensor map");
}

void pdl_attribute(cudaLaunchAttribute* a) {
  a->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a->val.programmaticStreamSerializationAllowed = 1;
}

template <int NP, bool DEEP>
pq_status launch_tile(const CUtensorMap& tmW, const CUtensorMap& tmA, const float* scales_A, const float* scales_W,
                      void* Y, int T, int N, int steps, int m_tiles, int64_t tiles, int split, int bf16, bool pdl,
                      unsigned int* status, cudaStream_t stream) {
  constexpr size_t smem = sizeof(TileSmem<NP, DEEP>) + 1024;
  static_assert((DEEP ? 1 : 2) * smem <= 232448, "shared memory exceeds 227 KB an SM");
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = set_kernel_attributes(reinterpret_cast<const void*>(w8a8_tile_kernel<NP, DEEP>), (int)smem, done);
  if (e != cudaSuccess) return cuda_fail(e, "w8a8_tile_kernel attributes");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * split), 1, 1);
  cfg.blockDim = dim3(T_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  pdl_attribute(&attr[1]);
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cuda_fail(cudaLaunchKernelEx(&cfg, w8a8_tile_kernel<NP, DEEP>, tmW, tmA, scales_A, scales_W, Y, T, N, steps, m_tiles,
                                      split, bf16, pdl ? 1 : 0, status),
                   "w8a8_tile_kernel launch");
}

}  // namespace

pq_status w8a8_launch(const int8_t* codes_A, const float* scales_A, const int8_t* codes_W, const float* scales_W,
                      int64_t T, int64_t N, int64_t D, void* Y, pq_out_dtype out_dtype, cudaStream_t stream,
                      bool pdl) {
  unsigned int* status = nullptr;
  cudaError_t e = gemm_status_address(&status);
  if (e != cudaSuccess) return cuda_fail(e, "status word");
  const int sms = device_sm_count();
  const int steps = (int)((D + KB - 1) / KB);
  const int bf16 = out_dtype == PQ_OUT_BF16 ? 1 : 0;
  const int64_t pair_m = (N + 2 * PM - 1) / (2 * PM), pair_tiles = pair_m * ((T + PN - 1) / PN);
  CUtensorMap tmW, tmA;
  // The pair kernel reads half the operand bytes a product but needs 256 x 256 tiles for most SM pairs (us, pair against
  // tile): 512 tokens, N = 14336, D = 4096 (112 tiles) 39 : 53; N = 8192 (64) 24.7 : 28.7; N = 5120 (40) 28.8 : 28.7 with the
  // quantisation; D = 14336, N = 4096 (32) 57 : 53.
  if (T > 128 && pair_tiles * 4 >= 3 * (sms / 2)) {
    if (pair_tiles >= ((int64_t)1 << 30)) { set_error("too many output tiles"); return PQ_ERR_INVALID_ARG; }
    pq_status st = operand_map(&tmW, codes_W, N, D, PM);
    if (st == PQ_OK) st = operand_map(&tmA, codes_A, T, D, PN_HALF);
    if (st != PQ_OK) return st;
    static std::atomic<bool> done[kMaxDevices];
    e = set_kernel_attributes(reinterpret_cast<const void*>(w8a8_pair_kernel), (int)kPairSmem, done);
    if (e != cudaSuccess) return cuda_fail(e, "w8a8_pair_kernel attributes");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(pair_tiles, sms / 2)), 1, 1);
    cfg.blockDim = dim3(P_THREADS, 1, 1);
    cfg.dynamicSmemBytes = kPairSmem;
    cfg.stream = stream;
    // Not a programmatic dependent: its CTAs fill an SM and would wait there for the quantisation, with nothing to load
    // meanwhile but the first weights (measured with a plain wait at the start, in a graph, so against one after the other:
    // 8192 x 4096 x 14336 413 : 416 us, 4096 x 4096 x 4096 105 : 106, 512 x 14336 x 4096 40 : 41).
    return cuda_fail(cudaLaunchKernelEx(&cfg, w8a8_pair_kernel, tmW, tmA, scales_A, scales_W, Y, (int)T, (int)N, steps,
                                        (int)pair_m, (int)pair_tiles, bf16, status),
                     "w8a8_pair_kernel launch");
  }
  const int np = T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128;
  const int64_t m_tiles = (N + TM - 1) / TM, tiles = m_tiles * ((T + np - 1) / np);
  // Ranges of the reduction: as long as every CTA still has an SM of its own and keeps some steps.  (Two CTAs an SM, with
  // half the stages each, streamed no faster, and as a dependent they waited for SMs: 64 tokens, N = D = 4096, 8 ranges:
  // 20.7 us behind the quantisation; 4: 14.5.)
  int split = 1;
  while (split < 8 && tiles * split * 2 <= sms && steps >= 4 * split) split *= 2;
  pq_status st = operand_map(&tmW, codes_W, N, D, TM);
  if (st == PQ_OK) st = operand_map(&tmA, codes_A, T, D, np);
  if (st != PQ_OK) return st;
#define PQ_TILE_CASE(NP)                                                                                                  \
  (tiles * split <= sms                                                                                                    \
       ? launch_tile<NP, true>(tmW, tmA, scales_A, scales_W, Y, (int)T, (int)N, steps, (int)m_tiles, tiles, split, bf16, pdl, \
                               status, stream)                                                                            \
       : launch_tile<NP, false>(tmW, tmA, scales_A, scales_W, Y, (int)T, (int)N, steps, (int)m_tiles, tiles, split, bf16,   \
                                pdl, status, stream))
  return np == 16 ? PQ_TILE_CASE(16) : np == 32 ? PQ_TILE_CASE(32) : np == 64 ? PQ_TILE_CASE(64) : PQ_TILE_CASE(128);
#undef PQ_TILE_CASE
}

}  // namespace pq
