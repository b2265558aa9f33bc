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
// fp4_pair_kernel (many tokens): persistent, one CTA per SM, clusters of two CTAs that share every MMA (cta_group::2, M256 N256
//   K64).  Here tokens are operand A and weights B, so that a thread of the epilogue has 16 channels of one token side by side
//   and stores them whole.  Scales of 256 columns are wanted in both CTAs, those of 128 rows in each its own.  Tensor memory
//   holds two accumulators of 256 columns only if they share some (128): the scales take the rest.  The epilogue reads the
//   shared columns first and hands them over, and the next tile's reduction runs under what is left of it.
//   warp 0: TMA producer; warp 1: tensor memory, scale copies and MMA issue (even CTA); warps 4..11: epilogue, two a lane
//   quarter.
//
// Issue bounds the pair kernel before the tensor cores do: a step is 12 scale copies, 4 products and a commit.  From a branch
// on the lane's number they took 1660 cycles (8192 x 4096 x 14336: 361 us; operands move to uniform registers one by one),
// from an elected lane with a warp's waits 800 (178 us), with the elected lane walking the steps alone 660 (167 us, 5.8
// PFLOP/s); the four products take 550.  A warp of its own for the copies costs more in barriers than it saves (185 us), and
// copies a half step ahead of their products twice as much (326 us: they wait for the products before them).  In a row of such
// calls the 1000 W limit lowers the clock, and the same product takes 175 to 200 us.
// The tile kernel is bound by the weights' bytes and the latencies of one launch: 64 tokens through 14336 x 4096 (33 MB from HBM) take
// 10.4 us, 3.2 TB/s, of which a launch that only starts, waits once for memory and ends is 4.
//
// Every mbarrier wait is bounded; a timeout sets the library's status word, the CTA drains what it has in flight, meets
// its cluster, frees tensor memory and returns.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "ptx_fp4.cuh"
#include "quant_fp4.cuh"

namespace pq {
namespace {

constexpr int KB = 128;                 // bytes of a K step a row = a swizzle row: 256 codes
constexpr int PIECE = QF_PIECE;         // bytes of a piece of scales
constexpr uint64_t kWaitNs = 2000000000ull;

// Scale pieces of 128 rows in a K step.
template <bool NV> constexpr int kPieces = NV ? 4 : 2;

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, int* abort_flag, unsigned int* status) {
  if (ptx::mbar_wait_bounded(bar, parity, abort_flag, kWaitNs, 100)) return true;
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

// Every lane polls, and an elected one acts: its operands stay in uniform registers.
__device__ __forceinline__ bool issue_wait(uint64_t* bar, uint32_t parity, int* abort_flag, unsigned int* status) {
  if (__all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, parity, abort_flag, kWaitNs, 100))) return true;
  if ((threadIdx.x & 31) == 0) {
    *abort_flag = 1;
    atomicOr(status, PQ_DEV_TIMEOUT);
  }
  __syncwarp();
  return false;
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

// ------------------------------------------------------------------------------------ pair kernel
constexpr int PM = 128;                 // tokens per CTA
constexpr int PN = 256;                 // channels per tile
constexpr int PN_HALF = PN / 2;         // channels each CTA stages
constexpr int P_STAGES = 5;
constexpr int P_THREADS = 384;
constexpr int P_EPI_WARP0 = 4;

template <bool NV> struct PairGeom {
  static constexpr int SF = kPieces<NV> * PIECE;                        // scale bytes of 128 rows a step
  static constexpr uint32_t TX = 2 * ((PM + PN_HALF) * KB + 3 * SF);    // both CTAs' bytes, on the even CTA's barrier
  static constexpr uint32_t ACC1 = PN / 2;                              // the second accumulator's first column
  static constexpr uint32_t SF_COL = ACC1 + PN;                         // buffers of scales, a step's each
  static constexpr uint32_t SF_COLS = kPieces<NV> * 12;                 // of them 4 a piece for A, then 8 for B
  static constexpr int SF_BUFS = 128 / SF_COLS;
};

template <bool NV> struct __align__(1024) PairSmem {
  uint8_t a[P_STAGES][PM * KB];
  uint8_t b[P_STAGES][PN_HALF * KB];
  uint8_t out[8][32 * 128];             // an epilogue warp's outputs on their way to memory: 32 tokens x 128 bytes, swizzled
  uint8_t sa[P_STAGES][PairGeom<NV>::SF];
  uint8_t sb[P_STAGES][2][PairGeom<NV>::SF];
  uint64_t full[P_STAGES], empty[P_STAGES];
  uint64_t acc_full, acc_empty;         // a phase a tile
  uint64_t mma_done, pair_done;
  uint32_t tmem_slot;
  int abort_flag;
};

// Tiles in strips of P_STRIP tiles of tokens, channel tiles within a strip: the tiles that run at once read few operands.
constexpr int P_STRIP = 8;
__device__ __forceinline__ void tile_place(int u, int m_tiles, int n_tiles, int& m, int& n) {
  const int strip = u / (P_STRIP * n_tiles), in = u % (P_STRIP * n_tiles);
  const int height = min(P_STRIP, m_tiles - strip * P_STRIP);
  m = strip * P_STRIP + in % height;
  n = in / height;
}

template <bool NV>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P_THREADS, 1) fp4_pair_kernel(
    const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmSW,
    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmY, float alpha, void* __restrict__ Y, int T,
    int N, int steps, int codes64, int pieces, int m_tiles, int n_tiles, int out_bf16, int bulk, int pdl, unsigned int* status) {
  using Geom = PairGeom<NV>;
  extern __shared__ unsigned char smem_raw[];
  PairSmem<NV>& S = *reinterpret_cast<PairSmem<NV>*>(smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)ptx::cluster_ctarank();
  const int first = (int)(blockIdx.x >> 1), stride = (int)(gridDim.x >> 1);
  const int tiles = m_tiles * n_tiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P_STAGES; ++s) {
      ptx::mbar_init(&S.full[s], 1);
      ptx::mbar_init(&S.empty[s], 1);
    }
    ptx::mbar_init(&S.acc_full, 1);
    ptx::mbar_init(&S.acc_empty, 2 * 8);                   // both CTAs' epilogue warps
    ptx::mbar_init(&S.mma_done, 1);
    ptx::mbar_init(&S.pair_done, 1);
    S.abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmSW);
    ptx::prefetch_tmap(&tmSA);
    ptx::prefetch_tmap(&tmY);
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
    const uint32_t full0 = ptx::mapa_shared(ptx::smem_addr(&S.full[0]), 0);
    if (pdl) ptx::griddep_wait();                          // for the kernel that writes the token codes
    int step = 0;
    bool ok = true;
    for (int u = first; u < tiles && ok; u += stride) {
      int m, n;
      tile_place(u, m_tiles, n_tiles, m, n);
      const int m0 = m * 2 * PM + PM * rank, n0 = n * PN;
      const int sa0 = (m0 / 128) * pieces * 2, sb0 = (n0 / 128) * pieces * 2;
      for (int kb = 0; kb < steps; ++kb, ++step) {
        const int s = step % P_STAGES, sk = kb * kPieces<NV> * 2;
        if (!(ok = issue_wait(&S.empty[s], ((uint32_t)(step / P_STAGES) & 1u) ^ 1u, &S.abort_flag, status))) break;
        if (ptx::elect_one()) {
          if (rank == 0) ptx::mbar_arrive_expect_tx(&S.full[s], Geom::TX);
          ptx::tma_load_2d_pair(S.a[s], &tmA, full0 + 8u * s, kb * KB, m0);
          ptx::tma_load_2d_pair(S.b[s], &tmW, full0 + 8u * s, kb * KB, n0 + PN_HALF * rank);
          ptx::tma_load_2d_pair(S.sa[s], &tmSA, full0 + 8u * s, 0, sa0 + sk);
          ptx::tma_load_2d_pair(S.sb[s][0], &tmSW, full0 + 8u * s, 0, sb0 + sk);
          ptx::tma_load_2d_pair(S.sb[s][1], &tmSW, full0 + 8u * s, 0, sb0 + 2 * pieces + sk);
        }
        __syncwarp();
      }
    }
    // Every load issued has landed and every release aimed at this CTA has arrived before it may exit.
    if (lane == 0) {
      const int j0 = step > P_STAGES ? step - P_STAGES : 0;
      if (rank == 0)
        for (int j = j0; j < step; ++j) drain_wait(&S.full[j % P_STAGES], (uint32_t)(j / P_STAGES) & 1u);
      for (int j = j0; j < step; ++j) drain_wait(&S.empty[j % P_STAGES], (uint32_t)(j / P_STAGES) & 1u);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      constexpr uint32_t id0 = ptx::idesc_e2m1(!NV, 2 * PM, PN, 0), id1 = ptx::idesc_e2m1(!NV, 2 * PM, PN, NV ? 0 : 2);
      // Descriptors of the first stage; an offset of b bytes adds b / 16 to the address field.
      const uint64_t da = ptx::smem_desc_sw128(ptx::smem_addr(S.a[0])), db = ptx::smem_desc_sw128(ptx::smem_addr(S.b[0]));
      const uint64_t dsa = ptx::smem_desc_rows16(ptx::smem_addr(S.sa[0])), dsb = ptx::smem_desc_rows16(ptx::smem_addr(S.sb[0]));
      // One elected lane for the whole walk.
      if (ptx::elect_one()) {
        int tile = 0, s = 0, b = 0;                        // stage and buffer of scales of the step
        uint32_t turn = 0;                                 // how often the ring has gone round, its low bit
        int ps = 0;                                        // stage and turn of the step that last read the buffer
        uint32_t pturn = 0;
        int step = 0;
        bool ok = true;
        for (int u = first; u < tiles && ok; u += stride, ++tile) {
          if (tile > 0 && !(ok = wait_or_abort(&S.acc_empty, (uint32_t)(tile - 1) & 1u, &S.abort_flag, status))) break;
          ptx::tc_fence_after();
          const uint32_t d = tmem + (tile & 1 ? Geom::ACC1 : 0u);
          for (int kb = 0; kb < steps; ++kb, ++step) {
            if (Geom::SF_BUFS < P_STAGES) {                // otherwise the stage's own round trip says so
              if (step >= Geom::SF_BUFS) {
                if (!(ok = wait_or_abort(&S.empty[ps], pturn, &S.abort_flag, status))) break;
                if (++ps == P_STAGES) ps = 0, pturn ^= 1u;
              }
            }
            if (!(ok = wait_or_abort(&S.full[s], turn, &S.abort_flag, status))) break;
            ptx::tc_fence_after();
            const uint32_t sa = tmem + Geom::SF_COL + (uint32_t)b * Geom::SF_COLS, sb = sa + 4 * kPieces<NV>;
            const uint64_t a0 = da + (uint64_t)(s * (PM * KB / 16)), b0 = db + (uint64_t)(s * (PN_HALF * KB / 16));
            const uint64_t sa0 = dsa + (uint64_t)(s * (Geom::SF / 16)), sb0 = dsb + (uint64_t)(s * (2 * Geom::SF / 16));
            const int live = min(4, codes64 - 4 * kb);     // 64-code products that are not all padding
#pragma unroll
            for (int p = 0; p < kPieces<NV>; ++p) {
              ptx::tmem_copy_scales<true>(sa + 4 * p, sa0 + PIECE / 16 * p);
              ptx::tmem_copy_scales<true>(sb + 8 * p, sb0 + PIECE / 16 * p);
              ptx::tmem_copy_scales<true>(sb + 8 * p + 4, sb0 + (Geom::SF + PIECE * p) / 16);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int p = NV ? k : k / 2;
              if (k < live)
                ptx::umma_e2m1<NV, true>(d, a0 + 2 * k, b0 + 2 * k, k & 1 ? id1 : id0, sa + 4 * p, sb + 8 * p,
                                         kb > 0 || k > 0 ? 1u : 0u);
            }
            ptx::umma_commit_pair(&S.empty[s], 0x3);
            if (++s == P_STAGES) s = 0, turn ^= 1u;
            if (++b == Geom::SF_BUFS) b = 0;
          }
          if (!ok) break;
          ptx::umma_commit_pair(&S.acc_full, 0x3);
        }
        ptx::umma_commit_pair(&S.mma_done, 0x1);
        drain_wait(&S.mma_done, 0);
        if (tile > 0) drain_wait(&S.acc_empty, (uint32_t)(tile - 1) & 1u);
      }
      __syncwarp();
    }
  } else if (warp >= P_EPI_WARP0) {
    // Lane quarter warp % 4 (tokens); 64 of the columns that the accumulators share, then 64 of the others.  Outputs leave by
    // TMA, through 4 KB of shared memory a warp (stored from the registers, a token a lane, they took 32 cycles an
    // instruction).
    const int ew = warp - P_EPI_WARP0, sub = warp & 3, half = ew >> 2;
    const uint32_t acc_empty0 = ptx::mapa_shared(ptx::smem_addr(&S.acc_empty), 0);
    const uint32_t lanes = tmem + ((uint32_t)(32 * sub) << 16);
    uint8_t* const out = S.out[ew];
    const uint32_t line = ptx::smem_addr(out) + 128u * lane, turn = (uint32_t)(lane & 7);
    int tile = 0;
    for (int u = first; u < tiles; u += stride, ++tile) {
      int m, n;
      tile_place(u, m_tiles, n_tiles, m, n);
      const int row0 = m * 2 * PM + PM * rank + 32 * sub, n0 = n * PN;
      const uint32_t acc = lanes + (tile & 1 ? Geom::ACC1 : 0u);
      auto put = [&](const uint32_t* r, int ch) {          // 64 channels from ch of this lane's token
        if (row0 >= T || ch >= N) return;                  // the whole warp
        if (bulk) {
          // bf16: one box of 64 channels; float32: two of 32
          for (int b = 0; b < (out_bf16 ? 1 : 2); ++b) {
            if (ch + 32 * b >= N) break;
            if (lane == 0) ptx::bulk_wait_read();          // the box before has left
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 8; ++c) {                  // 16 bytes
              uint32_t w[4];
              if (out_bf16) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const __nv_bfloat162 p = __floats2bfloat162_rn(alpha * __uint_as_float(r[8 * c + 2 * i]), alpha * __uint_as_float(r[8 * c + 2 * i + 1]));
                  w[i] = *reinterpret_cast<const uint32_t*>(&p);
                }
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(alpha * __uint_as_float(b ? r[32 + 4 * c + i] : r[4 * c + i]));
              }
              ptx::sts_v4(line + ((c ^ turn) << 4), w[0], w[1], w[2], w[3]);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              ptx::tma_store_2d(&tmY, out, ch + 32 * b, row0);
              ptx::bulk_commit();
            }
            __syncwarp();
          }
        } else {                                           // rows of Y that begin anywhere: 16 channels of two tokens at a time, by element
          // (6872 x 12291 x 2304 to bf16 111 us, where TMA takes 88 for 12288; a whole token's 64 channels by aligned words, a token
          // at a time, 140)
          float (*f)[17] = reinterpret_cast<float(*)[17]>(out);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) f[lane][i] = alpha * __uint_as_float(r[16 * q + i]);
            __syncwarp();
            const int64_t at = (int64_t)(row0 + (lane >> 4)) * N + ch + 16 * q + (lane & 15);
            const int live = ch + 16 * q + (lane & 15) < N ? T - row0 - (lane >> 4) : 0;
            if (out_bf16) {
              __nv_bfloat16* const y = static_cast<__nv_bfloat16*>(Y) + at;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (2 * i < live) y[(int64_t)(2 * i) * N] = __float2bfloat16_rn(f[2 * i + (lane >> 4)][lane & 15]);
            } else {
              float* const y = static_cast<float*>(Y) + at;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (2 * i < live) y[(int64_t)(2 * i) * N] = f[2 * i + (lane >> 4)][lane & 15];
            }
          }
          __syncwarp();
        }
      };
      if (!warp_wait_or_abort(&S.acc_full, (uint32_t)tile & 1u, &S.abort_flag, status)) break;
      ptx::tc_fence_after();
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        // columns of the tile: the shared ones are the first accumulator's last 128 and the second's first
        const int col = (part == (tile & 1) ? PN / 2 : 0) + 64 * half;
        uint32_t r[64];
        ptx::tmem_ld32(acc + col, reinterpret_cast<uint32_t(&)[32]>(r[0]));
        ptx::tmem_ld32(acc + col + 32, reinterpret_cast<uint32_t(&)[32]>(r[32]));
        ptx::tmem_ld_wait(reinterpret_cast<uint32_t(&)[32]>(r[0]));
        ptx::tmem_ld_wait(reinterpret_cast<uint32_t(&)[32]>(r[32]));
        if (part == 0) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_remote(acc_empty0);
        }
        put(r, n0 + col);
        __syncwarp();
      }
    }
    if (lane == 0) ptx::bulk_wait();                       // every box is in memory
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

// NP: token columns of a tile.  DEEP: stages for one CTA per SM (about 220 KB in flight), otherwise for two: where there are
// more CTAs than SMs (us, deep against two; 64 tokens, D 4096: 14336 channels, 112 tiles, 9.2 : 9.6; 28672, 224, 16.4 : 10.7; 16
// tokens, 65536, 512, 36.6 : 30.8).
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

// The quantisation that a product of up to 16 tokens does itself: rows of bf16 in, codes and scales out as well.
struct Fp4Fuse {
  const uint16_t* X;
  int64_t ldx;
  int D, aligned32;
  Fp4Scaling sc;
  uint8_t *codes, *scales;
};

// Grid: x = tile * split + range (the cluster), tiles channel-fastest.  tmSW, tmSA: the scale pieces as rows of 256 bytes;
// pieces: 512-byte pieces of 128 rows of a tensor.  codes64: 64-code products of the whole reduction.
// G >= 0 (NP = 16): the tokens come as bf16 rows, which the epilogue's warps rotate in blocks of G and quantise into the
// operand's place while the weights are on their way, every tile for itself (a range of 1024 channels is 8 units for 4
// warps); the first tile's blocks write the codes and scales out too.
template <int NP, bool NV, bool DEEP, int G>
__global__ void __launch_bounds__(T_THREADS) fp4_tile_kernel(
    const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmSW,
    const __grid_constant__ CUtensorMap tmSA, const Fp4Fuse fuse, float alpha, void* __restrict__ Y, int T, int N, int steps,
    int codes64, int pieces, int m_tiles, int split, int out_bf16, int pdl, unsigned int* status) {
  constexpr bool FUSED = G >= 0;
  constexpr int UNITS = G == 256 ? 1 : 2;                 // units of quantisation a step, a warp each
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
      ptx::mbar_init(&S.full[s], FUSED ? 1 + UNITS : 1);
      ptx::mbar_init(&S.empty[s], 1);
    }
    ptx::mbar_init(&S.acc_full, 1);
    S.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmSW);
    if (!FUSED) {
      ptx::prefetch_tmap(&tmA);
      ptx::prefetch_tmap(&tmSA);
    }
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
        ptx::mbar_arrive_expect_tx(&S.full[s], FUSED ? TM * KB + Geom::SF : Geom::TX);
        ptx::tma_load_2d(S.a[s], &tmW, &S.full[s], kb * KB, m0);
        ptx::tma_load_2d(S.sa[s], &tmSW, &S.full[s], 0, sw0 + kb * kPieces<NV> * 2);
      };
      auto tokens = [&](int s, int kb) {
        if (FUSED) return;
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
    // One elected lane for the whole walk.
    if (ptx::elect_one()) {
      constexpr uint32_t id0 = ptx::idesc_e2m1(!NV, TM, NP, 0), id1 = ptx::idesc_e2m1(!NV, TM, NP, NV ? 0 : 2);
      const uint64_t da = ptx::smem_desc_sw128(ptx::smem_addr(S.a[0])), db = ptx::smem_desc_sw128(ptx::smem_addr(S.b[0]));
      const uint64_t dsa = ptx::smem_desc_rows16(ptx::smem_addr(S.sa[0])), dsb = ptx::smem_desc_rows16(ptx::smem_addr(S.sb[0]));
      int s = 0;
      uint32_t turn = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (!wait_or_abort(&S.full[s], turn, &S.abort_flag, status)) break;
        ptx::tc_fence_after();
        const uint32_t sa = tmem + NP + (uint32_t)s * Geom::STAGE_COLS, sb = sa + 4 * kPieces<NV>;
        const uint64_t a0 = da + (uint64_t)(s * (TM * KB / 16)), b0 = db + (uint64_t)(s * (NP * KB / 16));
        const uint64_t sa0 = dsa + (uint64_t)(s * (Geom::SF / 16)), sb0 = dsb + (uint64_t)(s * (Geom::SF / 16));
        const int live = min(4, codes64 - 4 * kb);        // 64-code products that are not all padding
#pragma unroll
        for (int p = 0; p < kPieces<NV>; ++p) {
          ptx::tmem_copy_scales<false>(sa + 4 * p, sa0 + PIECE / 16 * p);
          ptx::tmem_copy_scales<false>(sb + 4 * p, sb0 + PIECE / 16 * p);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t col = 4 * (NV ? k : k / 2);
          if (k < live)
            ptx::umma_e2m1<NV, false>(tmem, a0 + 2 * k, b0 + 2 * k, k & 1 ? id1 : id0, sa + col, sb + col,
                                      kb > k0 || k > 0 ? 1u : 0u);
        }
        ptx::umma_commit(&S.empty[s]);
        if (++s == STAGES) s = 0, turn ^= 1u;
      }
      ptx::umma_commit(&S.acc_full);
      drain_wait(&S.acc_full, 0);
    }
    __syncwarp();
  } else {
    if constexpr (FUSED) {
      using Unit = Fp4Unit<G, NV>;
      constexpr int WIDTH = 64 * Unit::SPANS;
      const int g = lane >> 2, t = lane & 3;
      uint32_t b[2][2];
      Unit::signs(b);
      Unit x;
      // unit i of the range: half i % UNITS of step i / UNITS; the four warps take them in turn
      const int units = (k1 - k0) * UNITS;
      auto load = [&](int i) { x.load(fuse.X, fuse.ldx, T, fuse.D, 0, (k0 * UNITS + i) * WIDTH, fuse.aligned32 != 0); };
      const int i0 = warp - 2;
      if (i0 < units) load(i0);
      for (int i = i0; i < units; i += 4) {
        const int step = i / UNITS, half = i % UNITS, s = step % STAGES, u = k0 * UNITS + i;
        float v[2][Unit::SPANS][16];
        x.rotate(b, v);
        if (i + 4 < units) load(i + 4);
        if (step >= STAGES && !warp_wait_or_abort(&S.empty[s], ((uint32_t)(step / STAGES) & 1u) ^ 1u, &S.abort_flag, status)) break;
        const bool out = m0 == 0;
        Unit::quantise(
            v, fuse.sc,
            [&](int h, int sp, uint2 q) {                 // 16 codes, half of a 16-byte piece of the swizzled row
              const int r = g + 8 * h, c = u * WIDTH + 64 * sp + 16 * t, piece = 2 * (half * Unit::SPANS + sp) + (t >> 1);
              *reinterpret_cast<uint2*>(S.b[s] + r * KB + ((piece ^ (r & 7)) << 4) + (t & 1) * 8) = q;
              if (out && r < T && c < fuse.D) *reinterpret_cast<uint2*>(fuse.codes + (int64_t)r * (fuse.D / 2) + c / 2) = q;
            },
            [&](int h, int k, uint32_t word) {
              const int r = g + 8 * h, piece = half * Unit::WORDS + k, at = u * Unit::WORDS + k;
              if (t == 0) *reinterpret_cast<uint32_t*>(S.sb[s] + piece * PIECE + r * 16) = word;
              if (t == 0 && out && r < T && at < pieces) *reinterpret_cast<uint32_t*>(fuse.scales + at * PIECE + r * 16) = word;
            });
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&S.full[s]);
      }
    }
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
  CUtensorMap w, a, sw, sa, y;
};

pq_status make_maps(Fp4Maps* m, const uint8_t* codes_A, const uint8_t* scales_A, const uint8_t* codes_W,
                    const uint8_t* scales_W, int64_t T, int64_t N, int64_t D, int64_t pieces, int pieces_step, int a_rows,
                    bool weights_only = false) {
  const auto scale_map = [&](CUtensorMap* map, const uint8_t* base, int64_t rows) {
    return make_u8_tile_map(map, base, (rows + 127) / 128 * pieces * 2, 256, 256, 2 * pieces_step, /*swizzle128=*/false);
  };
  cudaError_t e = make_u8_tile_map(&m->w, codes_W, N, D / 2, KB, TM, /*swizzle128=*/true);
  if (e == cudaSuccess) e = scale_map(&m->sw, scales_W, N);
  if (weights_only) {
    m->a = m->w, m->sa = m->sw;         // not used
    return cuda_fail(e, "4-bit operand tensor map");
  }
  if (e == cudaSuccess) e = make_u8_tile_map(&m->a, codes_A, T, D / 2, KB, a_rows, /*swizzle128=*/true);
  if (e == cudaSuccess) e = scale_map(&m->sa, scales_A, T);
  return cuda_fail(e, "4-bit operand tensor map");
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Y as dense rows: boxes of 128 bytes x 32 rows, 128-byte swizzle; the row stride has to be a multiple of 16 bytes.
cudaError_t make_out_map(CUtensorMap* map, void* base, int64_t rows, int64_t inner, bool bf16) {
  static const EncodeTiled enc = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q);
    return reinterpret_cast<EncodeTiled>(e == cudaSuccess && q == cudaDriverEntryPointSuccess ? p : nullptr);
  }();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)inner * (bf16 ? 2 : 4)};
  cuuint32_t box[2] = {bf16 ? 64u : 32u, 32u};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims, strides, box,
                   estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

struct Fp4Call {
  float alpha;
  void* Y;
  int T, N, steps, codes64, pieces, bf16;
  bool pdl;
  unsigned int* status;
  cudaStream_t stream;
  int g;                                // -1: the token codes are in hand
  Fp4Fuse fuse;
};

template <int NP, bool NV, bool DEEP, int G = -1>
pq_status launch_tile(const Fp4Maps& m, const Fp4Call& c, int m_tiles, int64_t tiles, int split) {
  constexpr size_t smem = sizeof(TileSmem<NP, NV, DEEP>) + 1024;
  static_assert((DEEP ? 1 : 2) * smem <= 232448, "shared memory exceeds 227 KB an SM");
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = set_kernel_attributes(reinterpret_cast<const void*>(fp4_tile_kernel<NP, NV, DEEP, G>), (int)smem, done);
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
  return cuda_fail(cudaLaunchKernelEx(&cfg, fp4_tile_kernel<NP, NV, DEEP, G>, m.w, m.a, m.sw, m.sa, c.fuse, c.alpha, c.Y, c.T, c.N,
                                      c.steps, c.codes64, c.pieces, m_tiles, split, c.bf16, c.pdl ? 1 : 0, c.status),
                   "fp4_tile_kernel launch");
}

template <bool NV>
pq_status launch_pair(Fp4Maps& m, const Fp4Call& c, int m_tiles, int n_tiles, int sms) {
  // Rows of Y that begin on 16 bytes leave by TMA.
  const bool bulk = c.N % (c.bf16 ? 8 : 4) == 0;
  m.y = m.a;
  if (bulk) {
    const cudaError_t e = make_out_map(&m.y, c.Y, c.T, c.N, c.bf16 != 0);
    if (e != cudaSuccess) return cuda_fail(e, "output tensor map");
  }
  constexpr size_t smem = sizeof(PairSmem<NV>) + 1024;
  static_assert(smem <= 232448, "shared memory exceeds 227 KB");
  static std::atomic<bool> done[kMaxDevices];
  const cudaError_t e = set_kernel_attributes(reinterpret_cast<const void*>(fp4_pair_kernel<NV>), (int)smem, done);
  if (e != cudaSuccess) return cuda_fail(e, "fp4_pair_kernel attributes");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>((int64_t)m_tiles * n_tiles, sms / 2)), 1, 1);
  cfg.blockDim = dim3(P_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = c.pdl ? 1 : 0;
  return cuda_fail(cudaLaunchKernelEx(&cfg, fp4_pair_kernel<NV>, m.w, m.a, m.sw, m.sa, m.y, c.alpha, c.Y, c.T, c.N, c.steps, c.codes64,
                                      c.pieces, m_tiles, n_tiles, c.bf16, bulk ? 1 : 0, c.pdl ? 1 : 0, c.status),
                   "fp4_pair_kernel launch");
}

int tile_tokens(int64_t T) { return T <= 16 ? 16 : T <= 32 ? 32 : T <= 64 ? 64 : 128; }

// K steps of the tile kernel's reduction, and the ranges it is cut into (figures: us on the device).
// It is cut by twos as long as every CTA still has an SM of its own and keeps two steps.  Uncut, and by 2, 4 and 8 at most: 1 token,
// N x D 4096 x 4096 7.4, 6.8, 5.8, 5.8; 4096 x 14336 18.9, 12.0, 8.9, 8.9; 16 tokens, 1024 x 14336 18.6, 11.9, 7.9, 6.4; 391
// tokens, 1003 x 4192 13.3, 11.5, 9.2, 9.2.
// Where it is cut and the tokens are up to 16, whose join is short, it is cut on, to two CTAs an SM, as long as each keeps four
// steps and all clusters run at once.  Two CTAs an SM : one, nv, weights from HBM:
//   taken       1 token 8192 x 8192 10.0 : 11.0, 5120 x 5120 7.3 : 8.6; 16 tokens 10.3 : 11.3, 7.7 : 8.7
//   two steps   1 token 4096 x 4096, with the quantisation 7.2 : 7.0; 16 tokens 7.6 : 7.2
//   more tokens 64, 5120 x 5120 9.4 : 9.7, but 4096 x 8192 10.7 : 9.7, 4096 x 14336 12.4 : 11.3; 128, 4096 x 8192 13.3 : 11.0
//   uncut       16 tokens 14336 x 4096 10.2 : 9.9
//   at once     a 25th of the places stays empty beside clusters of 4: 1 token, 71 tiles, 9088 x 4096 8.1 : 8.9, 72 tiles, 9216
//               10.8 : 8.9; an eighth beside those of 8: 32 tiles, 4096 x 8192 7.9 : 8.5, 36 tiles, 4608 11.5 : 8.2
int fp4_ranges(int64_t T, int64_t N, int64_t D, int* split) {
  const int np = tile_tokens(T), sms = device_sm_count(), steps = (int)((D + 2 * KB - 1) / (2 * KB));
  const int64_t tiles = (N + TM - 1) / TM * ((T + np - 1) / np);
  *split = 1;
  while (*split < 8 && tiles * *split * 2 <= sms && steps >= 4 * *split) *split *= 2;
  while (T <= 16 && *split > 1 && *split < 8 && tiles * *split * 2 <= (*split == 2 ? 48 * sms / 25 : 7 * sms / 4) && steps >= 8 * *split)
    *split *= 2;
  return steps;
}

template <bool NV>
pq_status run(const uint8_t* codes_A, const uint8_t* scales_A, const uint8_t* codes_W, const uint8_t* scales_W, int64_t T,
              int64_t N, int64_t D, Fp4Call c) {
  const int sms = device_sm_count();
  const int np = tile_tokens(T);
  const int64_t m_tiles = (N + TM - 1) / TM, tiles = m_tiles * ((T + np - 1) / np);
  const int64_t pair_m = (T + 2 * PM - 1) / (2 * PM), pair_n = (N + PN - 1) / PN;
  // Pairs of CTAs from 129 tokens on, unless so few tiles of 128 x 128 that each may have its reduction cut over several SMs (us on
  // the device, nv, pairs against tiles).  256 tokens, N x D 4096 x 4096 10.6 : 10.6, 4096 x 14336 22.0 : 16.7; past that border
  // 6144 x 256 6.3 : 6.8, 5120 x 14336 22.2 : 23.4, 14336 x 4096 11.3 : 14.0; 1024 tokens 4096 x 4096 11.5 : 14.6, 4096 x 14336 24.4 : 31.9.
  if (T > 128 && 2 * tiles > sms) {
    if (pair_m * pair_n >= ((int64_t)1 << 30)) { set_error("too many output tiles"); return PQ_ERR_INVALID_ARG; }
    Fp4Maps m;
    const pq_status st = make_maps(&m, codes_A, scales_A, codes_W, scales_W, T, N, D, c.pieces, kPieces<NV>, PM);
    if (st != PQ_OK) return st;
    return launch_pair<NV>(m, c, (int)pair_m, (int)pair_n, sms);
  }
  if (tiles >= ((int64_t)1 << 31)) { set_error("too many output tiles"); return PQ_ERR_INVALID_ARG; }
  int split = 1;
  fp4_ranges(T, N, D, &split);
  Fp4Maps m;
  const pq_status st = make_maps(&m, codes_A, scales_A, codes_W, scales_W, T, N, D, c.pieces, kPieces<NV>, np, c.g >= 0);
  if (st != PQ_OK) return st;
  // One CTA an SM where all clusters run at once so: those of 4 leave an eighth of the SMs empty, those of 8 a fifth (us, one CTA an
  // SM, in two waves, against two; 1 token, 2048 x 14336, 16 clusters of 8, 11.8 : 6.9; 4608 x 4096, 36 of 4, 9.6 : 6.1; 64 tokens,
  // 2048 x 8192 12.7 : 8.7; 391 tokens, 1003 x 4192, 32 of 4, which fit, 9.4 : 9.7).
  const bool deep = tiles * split <= (split == 8 ? 13 * sms / 16 : split == 4 ? 7 * sms / 8 : sms);
  if (c.g >= 0) {
#define PQ_FUSED_CASE(G)                                                                     \
  (deep ? launch_tile<16, NV, true, G>(m, c, (int)m_tiles, tiles, split)                     \
        : launch_tile<16, NV, false, G>(m, c, (int)m_tiles, tiles, split))
    return c.g == 0 ? PQ_FUSED_CASE(0) : c.g == 64 ? PQ_FUSED_CASE(64) : c.g == 128 ? PQ_FUSED_CASE(128) : PQ_FUSED_CASE(256);
#undef PQ_FUSED_CASE
  }
#define PQ_TILE_CASE(NP)                                                                   \
  (deep ? launch_tile<NP, NV, true>(m, c, (int)m_tiles, tiles, split)                      \
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
                     (int)(nv ? (D + 63) / 64 : (D + 127) / 128), out_dtype == PQ_OUT_BF16 ? 1 : 0, pdl, status, stream, -1, {}};
  return nv ? run<true>(codes_A, scales_A, codes_W, scales_W, T, N, D, c)
            : run<false>(codes_A, scales_A, codes_W, scales_W, T, N, D, c);
}

pq_status fp4_linear_launch(const void* X, int64_t T, int64_t D, int64_t ldx, int g, bool nv, float factor, uint8_t* codes_A,
                            uint8_t* scales_A, const uint8_t* codes_W, const uint8_t* scales_W, int64_t N, float alpha, void* Y,
                            pq_out_dtype out_dtype, cudaStream_t stream) {
  // Up to 16 tokens one kernel does both, where no block has more than 4 steps of them to quantise and an SM has one block (us on the
  // device, one kernel against two; one token).  4096 x 4096, 4 steps a block: 7.0 : 7.1 with weights from HBM, 6.7 : 6.3 from L2, and
  // 3 less of the host for the second launch; at worst 4608 x 4096, the same, 8.0 : 7.3; 2048 x 2048, 2 steps: 5.0 : 5.7; 6144 x 4096, 4 steps and two blocks an SM: 8.2 : 7.6; 14336 x 4096, 16 steps: 12.9 :
  // 8.8; 4096 x 14336, 14 steps: 13.9 : 10.3.
  int split = 1;
  const int steps = fp4_ranges(T, N, D, &split);
  if (T > kFp4FusedT || steps > 4 * split || (N + TM - 1) / TM * split > device_sm_count()) {
    const pq_status st = cuda_fail(launch_quant_fp4(X, T, (int)D, ldx, g, nv, factor, codes_A, scales_A, stream),
                                   "pq_fp4_linear quantisation launch");
    if (st != PQ_OK) return st;
    return fp4_launch(codes_A, scales_A, codes_W, scales_W, T, N, D, nv, alpha, Y, out_dtype, stream, /*pdl=*/true);
  }
  unsigned int* status = nullptr;
  const cudaError_t e = gemm_status_address(&status);
  if (e != cudaSuccess) return cuda_fail(e, "status word");
  const int aligned32 = (reinterpret_cast<uintptr_t>(X) & 31) == 0 && ldx % 16 == 0;
  const Fp4Call c = {alpha, Y, (int)T, (int)N, (int)((D + 2 * KB - 1) / (2 * KB)), (int)((D + 63) / 64),
                     (int)(nv ? (D + 63) / 64 : (D + 127) / 128), out_dtype == PQ_OUT_BF16 ? 1 : 0, /*pdl=*/false, status, stream, g,
                     {static_cast<const uint16_t*>(X), ldx, (int)D, aligned32, Fp4Scaling::of(g, nv, factor), codes_A, scales_A}};
  return nv ? run<true>(codes_A, scales_A, codes_W, scales_W, T, N, D, c)
            : run<false>(codes_A, scales_A, codes_W, scales_W, T, N, D, c);
}

}  // namespace pq
