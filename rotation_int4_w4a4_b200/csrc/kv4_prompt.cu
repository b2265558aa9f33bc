// Attention over the paged 4-bit cache for many query rows a sequence (prompts and long chunks) on tcgen05 tensor
// cores, sm_100a.  The mathematics is that of the few-row kernel (kv4_attention.cu): per row
//   s_t = scale (q . kc_t) ks_t,  o = sum_t softmax(s)_t vs_t vc_t,  codes exact, all sums float32.
//
// The query rows of one key/value head (row = new token x head of the group) come in tiles of 128 = the lanes of tensor
// memory; a CTA takes two tiles (256 rows) and walks the cached tokens 128 at a time:
//   S_i = Q_i K^T   (bf16, M128 N128)       into 128 columns of tensor memory, i = 0, 1
//   P_i = softmax numerators times vs, fp16, written over S_i's columns
//   O_i += P_i V    (fp16, A from tensor memory, M128 N head_dim) into head_dim more columns
// While the tensor cores work for one tile, the other's softmax runs; both tiles share each 128 keys and values, so a
// code is unpacked once per 256 rows.  The tensor cores and the exponentials (16 a clock and SM) are about evenly
// loaded: 2 x 128 x 128 x head_dim multiply-adds against 128 x 128 exponentials a tile and step.
//   warps 0..3, 4..7   softmax of tile 0, 1: a thread owns a row: its scores from tensor memory, maximum, exponentials,
//                      P back; O is rescaled in tensor memory only when the row's reference grows by more than 2^8
//                      (P stays below 2^8, which fp16 holds); at the end its output row.
//   warps 8..11        producers: 128 tokens' codes from the pages, unpacked to bf16 keys and fp16 values in the
//                      swizzled operand layout, two stages each; their scales beside them.
//   warp 12            tensor memory and MMA issue.
// Channels sit in the operands in the order 0 4 1 5 2 6 3 7 of each 8 (the order in which nibbles come out of a word);
// queries are staged in the same order and the output is read back through it.
// Keys are rows of 128 bytes, K-major; values lie the same way and enter as an MN-major operand.
//
// Few rows over a long context leave SMs idle: the context is then cut into chunks whose partial results a second
// kernel joins (kv4_attention.cu).
//
// Every mbarrier wait is bounded; a timeout sets the library's status word, the CTA drains, frees tensor memory and
// returns.
#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "kv4.h"
#include "kv4_device.cuh"
#include "ptx.cuh"

namespace pq {
namespace {

constexpr int PT = 128;                  // rows per tile and tokens per step
constexpr int PR_THREADS = 512;
constexpr int PR_STAGES = 2;             // key and value stages
constexpr int SC_RING = 4;               // scale stages: a step's scales outlive its keys by at most one step
constexpr uint64_t kPrWaitNs = 2000000000ull;
constexpr uint32_t S_COL = 0, O_COL = 256;               // tensor memory: S_i at 128 i, O_i at 256 + 128 i
constexpr float kLazy = 8.0f;            // log2 growth of the reference that is let pass
constexpr uint32_t PR_REG_LAUNCH = 128, PR_REG_SOFT = 184, PR_REG_PROD = 96, PR_REG_CTRL = 48;
static_assert(256 * PR_REG_SOFT + 128 * PR_REG_PROD + 128 * PR_REG_CTRL <= PR_THREADS * PR_REG_LAUNCH,
              "setmaxnreg shares exceed the launch allocation");

// kind::f16 with a float32 accumulator: A and B types at bits 7 and 10 (0 fp16, 1 bf16), B MN-major at bit 16.
__host__ __device__ constexpr uint32_t idesc_f16(int bf16, int b_mn_major, int N) {
  return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)b_mn_major << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(PT >> 4) << 24);
}

template <int HD>
struct __align__(1024) PromptSmem {
  static constexpr int KBLK = HD / 64;                   // 128-byte blocks of a row
  uint8_t q[2][KBLK][PT * 128];
  uint8_t k[PR_STAGES][KBLK][PT * 128];
  uint8_t v[PR_STAGES][KBLK][PT * 128];
  float ks[SC_RING][PT], vs[SC_RING][PT];                // ks already times scale * log2(e)
  uint32_t valid[SC_RING][4];                            // which tokens exist, a bit each
  float vmax[SC_RING][4];                                // largest value scale of each 32
  uint64_t q_full;
  uint64_t k_full[PR_STAGES], k_empty[PR_STAGES], v_full[PR_STAGES], v_empty[PR_STAGES];
  uint64_t sc_full[SC_RING];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t mma_done;
  uint32_t tmem_slot;
  int abort_flag;
};

__device__ __forceinline__ bool pr_wait(uint64_t* bar, uint32_t parity, int* abort_flag, unsigned int* status) {
  if (ptx::mbar_wait_bounded(bar, parity, abort_flag, kPrWaitNs)) return true;
  *abort_flag = 1;
  atomicOr(status, PQ_DEV_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool pr_warp_wait(uint64_t* bar, uint32_t parity, int* abort_flag, unsigned int* status) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = pr_wait(bar, parity, abort_flag, status) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

// The work of a block: sequence, key/value head, first row of its 256, chunk of the context.
struct Work {
  int b, kvh, r0, chunk;
  int q0, qlen, rows, n;
};

// Tiles are numbered through the sequences; those of one sequence from its last rows (the longest) to its first.
// Returns false when the block has no tile.  Called by whole warps.
__device__ __forceinline__ bool find_work(const Kv4AttnArgs& a, const Partials& part, Work& w) {
  const int lane = threadIdx.x & 31;
  const int heads = a.cache.heads, group = a.heads_q / heads;
  int tile = (int)(blockIdx.x / (heads * part.chunks));
  const int rest = (int)(blockIdx.x % (heads * part.chunks));
  w.kvh = rest % heads;
  w.chunk = rest / heads;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    int q0 = 0, qlen = 0;
    if (b < a.B) {
      q0 = max(0, a.q_start[b]);
      qlen = max(0, min((int)a.T, a.q_start[b + 1]) - q0);
    }
    const int tiles = (qlen * group + 2 * PT - 1) / (2 * PT);
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, tile < upto);
    if (hit) {
      const int src = __ffs(hit) - 1;
      w.b = b0 + src;
      w.q0 = __shfl_sync(0xffffffffu, q0, src);
      w.qlen = __shfl_sync(0xffffffffu, qlen, src);
      w.r0 = (__shfl_sync(0xffffffffu, upto, src) - 1 - tile) * 2 * PT;
      w.rows = w.qlen * group;
      return true;
    }
    tile -= __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// Unnormalised Walsh-Hadamard transform of a head in registers, Sylvester order.
template <int N>
__device__ __forceinline__ void fwht(float (&v)[N]) {
#pragma unroll
  for (int h = 1; h < N; h <<= 1)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & h) == 0) {
        const float x = v[i], y = v[i + h];
        v[i] = x + y;
        v[i + h] = x - y;
      }
}

// Swizzled place of 16-byte chunk c of row r in a block of 128-byte rows.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

template <int HD>
__global__ void __launch_bounds__(PR_THREADS, 1) kv4_prompt_kernel(const Kv4AttnArgs a, const Partials part) {
  using Smem = PromptSmem<HD>;
  constexpr int HB = HD / 2;
  extern __shared__ unsigned char smem_raw[];
  Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  Work w;
  if (!find_work(a, part, w)) return;                    // the whole block agrees
  const int group = a.heads_q / a.cache.heads;
  const int ps = a.cache.page_shift;
  int n = max(0, a.seq_lens[w.b]);
  if (n > (int64_t)a.table_width << ps) {
    n = (int)((int64_t)a.table_width << ps);
    if (threadIdx.x == 0) atomicOr(a.status, PQ_DEV_BAD_INDEX);
  }
  const int last_row = min(w.rows, w.r0 + 2 * PT) - 1;
  const int p_first = n - w.qlen + w.r0 / group, p_last = n - w.qlen + last_row / group;
  const int lo = a.window > 0 ? max(0, p_first - a.window + 1) : 0;
  const int hi = min(n, p_last + 1);
  const int c_lo = part.chunks > 1 ? max(lo, w.chunk * part.chunk_len) : lo;
  const int c_hi = part.chunks > 1 && w.chunk < part.chunks - 1 ? min(hi, (w.chunk + 1) * part.chunk_len) : hi;
  const int j0 = c_lo / PT;
  const int steps = c_hi > c_lo ? (c_hi + PT - 1) / PT - j0 : 0;
  const int tiles = w.rows - w.r0 > PT ? 2 : 1;          // row tiles that hold rows

  if (threadIdx.x == 0) {
    ptx::mbar_init(&S.q_full, 8);
    for (int s = 0; s < PR_STAGES; ++s) {
      ptx::mbar_init(&S.k_full[s], 4);
      ptx::mbar_init(&S.k_empty[s], 1);
      ptx::mbar_init(&S.v_full[s], 4);
      ptx::mbar_init(&S.v_empty[s], 1);
    }
    for (int s = 0; s < SC_RING; ++s) ptx::mbar_init(&S.sc_full[s], 4);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&S.s_full[i], 1);
      ptx::mbar_init(&S.p_full[i], 4);
      ptx::mbar_init(&S.o_full[i], 1);
    }
    ptx::mbar_init(&S.mma_done, 1);
    S.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 12) {
    ptx::tmem_alloc(&S.tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = S.tmem_slot;

  if (warp < 8) {
    // ------------------------------------------------------------------------------- softmax
    ptx::setmaxnreg_inc<PR_REG_SOFT>();
    const int i = warp >> 2;                             // row tile
    const int row = (warp & 3) * 32 + lane;              // lane of tensor memory
    const int r = w.r0 + PT * i + row;
    const bool live = r < w.rows;
    const int rr = min(r, w.rows - 1);
    const int64_t token = w.q0 + rr / group;
    const int head = w.kvh * group + rr % group;
    {
      const uint4* src = reinterpret_cast<const uint4*>(a.Q + token * a.ldq + head * HD);
#pragma unroll
      for (int c = 0; c < HD / 8; ++c) {
        const uint4 x = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
        // channels 0 4 | 1 5 | 2 6 | 3 7
        const uint4 y = make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                                   __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632));
        *reinterpret_cast<uint4*>(S.q[i][c / 8] + sw128(row, c % 8)) = y;
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.q_full);
    }
    const int pos = n - w.qlen + rr / group;
    const int row_hi = min(pos, c_hi - 1), row_lo = a.window > 0 ? max(pos - a.window + 1, c_lo) : c_lo;
    // whole tiles: every row of this warp's tile sees every token
    const int t_first = n - w.qlen + min(w.rows - 1, w.r0 + PT * i) / group;
    const int t_last = n - w.qlen + min(w.rows - 1, w.r0 + PT * i + PT - 1) / group;
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_col = lane_base + S_COL + 128 * i, o_col = lane_base + O_COL + 128 * i;
    float m = -INFINITY, l = 0.0f;
    bool ok = i < tiles;
    for (int j = 0; j < steps && ok; ++j) {
      const int sc = j % SC_RING;
      ok = pr_warp_wait(&S.sc_full[sc], (uint32_t)(j / SC_RING) & 1u, &S.abort_flag, a.status) &&
           pr_warp_wait(&S.s_full[i], (uint32_t)j & 1u, &S.abort_flag, a.status);
      if (!ok) break;
      ptx::tc_fence_after();
      const int tok0 = (j0 + j) * PT;
      const uint4 valid = *reinterpret_cast<const uint4*>(S.valid[sc]);
      const bool whole = (valid.x & valid.y & valid.z & valid.w) == 0xffffffffu && tok0 >= c_lo && tok0 + PT <= c_hi &&
                         tok0 + PT - 1 <= t_first && (a.window <= 0 || tok0 > t_last - a.window);
      uint64_t x[PT / 2];                                // scores in pairs, log2 domain
      {
        uint32_t* xr = reinterpret_cast<uint32_t*>(x);
#pragma unroll
        for (int c = 0; c < 4; ++c) ptx::tmem_ld32(s_col + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(xr + 32 * c));
        ptx::tmem_ld_wait();
      }
      float mx = -INFINITY, vm;
      const float4* ks4 = reinterpret_cast<const float4*>(S.ks[sc]);
      const float4* vs4 = reinterpret_cast<const float4*>(S.vs[sc]);
#pragma unroll
      for (int c = 0; c < PT / 4; ++c) {
        const float4 k = ks4[c];
        x[2 * c] = ptx::f2_mul(x[2 * c], ptx::f2_pack(k.x, k.y));
        x[2 * c + 1] = ptx::f2_mul(x[2 * c + 1], ptx::f2_pack(k.z, k.w));
      }
      if (whole) {
        const float4 v4 = *reinterpret_cast<const float4*>(S.vmax[sc]);
        vm = fmaxf(fmaxf(v4.x, v4.y), fmaxf(v4.z, v4.w));
      } else {
        vm = 0.0f;
#pragma unroll
        for (int c = 0; c < PT / 4; ++c) {
          const float4 v4 = vs4[c];
          const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
          const uint32_t bits = (c < 8 ? valid.x : c < 16 ? valid.y : c < 24 ? valid.z : valid.w) >> (4 * (c & 7));
          float e[4];
          ptx::f2_unpack(x[2 * c], e[0], e[1]);
          ptx::f2_unpack(x[2 * c + 1], e[2], e[3]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tok = tok0 + 4 * c + k;
            const bool seen = ((bits >> k) & 1u) && tok >= row_lo && tok <= row_hi;
            e[k] = seen ? e[k] : -INFINITY;
            if (seen) vm = fmaxf(vm, finite_or_0(vv[k]));
          }
          x[2 * c] = ptx::f2_pack(e[0], e[1]);
          x[2 * c + 1] = ptx::f2_pack(e[2], e[3]);
        }
      }
      {
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int c = 0; c < PT / 2; ++c) {
          float e0, e1;
          ptx::f2_unpack(x[c], e0, e1);
          m0 = fmaxf(m0, e0);
          m1 = fmaxf(m1, e1);
        }
        mx = fmaxf(m0, m1);
      }
      // the reference: largest score plus the exponent of the largest value scale
      const float cand = mx + scale_exponent(vm);
      const bool grow = cand > m + kLazy || (m == -INFINITY && cand > m);
      if (__any_sync(0xffffffffu, grow)) {
        const float m_new = grow ? cand : m;
        const float f = m_new == -INFINITY ? 1.0f : ex2(m - m_new);
        m = m_new;
        l *= f;
        if (j > 0) {
          ok = pr_warp_wait(&S.o_full[i], (uint32_t)(j - 1) & 1u, &S.abort_flag, a.status);
          if (!ok) break;
          ptx::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < HD; c += 16) {
            uint32_t o[16];
            ptx::tmem_ld32x16(o_col + c, o);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            ptx::tmem_st32x16(o_col + c, o);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      const uint64_t ref2 = ptx::f2_pack(-ref, -ref);
      uint64_t sum0 = 0ull, sum1 = 0ull;
#pragma unroll
      for (int c = 0; c < PT / 32; ++c) {                // 32 tokens -> 16 columns of P
        uint32_t p[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 v4 = vs4[8 * c + k];
          float e[4];
          ptx::f2_unpack(ptx::f2_add(x[16 * c + 2 * k], ref2), e[0], e[1]);
          ptx::f2_unpack(ptx::f2_add(x[16 * c + 2 * k + 1], ref2), e[2], e[3]);
          const uint64_t p0 = ptx::f2_pack(ex2(e[0]), ex2(e[1])), p1 = ptx::f2_pack(ex2(e[2]), ex2(e[3]));
          sum0 = ptx::f2_add(sum0, p0);
          sum1 = ptx::f2_add(sum1, p1);
          float y[4];
          ptx::f2_unpack(ptx::f2_mul(p0, ptx::f2_pack(v4.x, v4.y)), y[0], y[1]);
          ptx::f2_unpack(ptx::f2_mul(p1, ptx::f2_pack(v4.z, v4.w)), y[2], y[3]);
          if (!whole) {                                  // a hidden token's value scale may be anything
#pragma unroll
            for (int q = 0; q < 4; ++q) y[q] = e[q] == -INFINITY ? 0.0f : y[q];
          }
          p[2 * k] = pack_f16(y[0], y[1]);
          p[2 * k + 1] = pack_f16(y[2], y[3]);
        }
        ptx::tmem_st32x16(s_col + 16 * c, p);
      }
      float a0, a1, a2, a3;
      ptx::f2_unpack(sum0, a0, a1);
      ptx::f2_unpack(sum1, a2, a3);
      l += (a0 + a1) + (a2 + a3);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.p_full[i]);
    }
    // ---- the row's output
    if (i < tiles) {
      float o[HD];
      if (ok && steps > 0) ok = pr_warp_wait(&S.o_full[i], (uint32_t)(steps - 1) & 1u, &S.abort_flag, a.status);
      if (ok && steps > 0) {
        ptx::tc_fence_after();
        uint32_t* od = reinterpret_cast<uint32_t*>(o);
#pragma unroll
        for (int c = 0; c < HD / 32; ++c) ptx::tmem_ld32(o_col + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(od + 32 * c));
        ptx::tmem_ld_wait();
        ptx::tc_fence_before();
      } else {
#pragma unroll
        for (int c = 0; c < HD; ++c) o[c] = 0.0f;
      }
      if (live) {
        // operand order -> channel order: place 2k of each 8 holds channel k, 2k + 1 holds k + 4
#pragma unroll
        for (int c = 0; c < HD; c += 8) {
          const float t1 = o[c + 1], t2 = o[c + 2], t3 = o[c + 3], t4 = o[c + 4], t5 = o[c + 5], t6 = o[c + 6];
          o[c + 1] = t2, o[c + 2] = t4, o[c + 3] = t6, o[c + 4] = t1, o[c + 5] = t3, o[c + 6] = t5;
        }
        if (part.chunks > 1) {
          const int64_t at = ((int64_t)w.chunk * a.T + token) * a.heads_q + head;
          part.ml[at] = make_float2(m, l);
          if (m != -INFINITY || l != 0.0f) {
            float4* dst = reinterpret_cast<float4*>(part.o + at * HD);
#pragma unroll
            for (int c = 0; c < HD / 4; ++c) dst[c] = make_float4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
        } else {
          float f = l == 0.0f ? 0.0f : 1.0f / l;
          if (a.cache.rotate_v) {
            fwht(o);
            f *= HD == 128 ? 0.08838834764831845f : 0.125f;
          }
          uint4* dst = reinterpret_cast<uint4*>(a.O + token * a.ldo + head * HD);
#pragma unroll
          for (int c = 0; c < HD / 8; ++c)
            dst[c] = make_uint4(pack_bf16(o[8 * c] * f, o[8 * c + 1] * f), pack_bf16(o[8 * c + 2] * f, o[8 * c + 3] * f),
                                pack_bf16(o[8 * c + 4] * f, o[8 * c + 5] * f), pack_bf16(o[8 * c + 6] * f, o[8 * c + 7] * f));
        }
      }
    }
  } else if (warp < 12) {
    // ----------------------------------------------------------------------------- producers
    ptx::setmaxnreg_dec<PR_REG_PROD>();
    const int t = threadIdx.x - 256;                     // token of the step
    const int wq = warp - 8;
    const int32_t* table = a.table + w.b * a.table_stride;
    const float c_log2 = a.scale * kLog2e;
    uint4 kx[HB / 16], vx[HB / 16];
    float ks = 0.0f, vs = 0.0f;
    bool valid = false;
    auto load = [&](int j) {
      const int tok = (j0 + j) * PT + t;
      valid = false;
      int64_t at = 0;
      if (tok < n) {
        const int page = table[tok >> ps];
        if (page < 0 || page >= a.cache.pages) atomicOr(a.status, PQ_DEV_BAD_INDEX);
        else {
          valid = true;
          at = (((int64_t)page * a.cache.heads + w.kvh) << ps) + (tok & ((1 << ps) - 1));
        }
      }
#pragma unroll
      for (int c = 0; c < HB / 16; ++c) {
        kx[c] = valid ? __ldg(reinterpret_cast<const uint4*>(a.cache.k_codes + at * HB) + c) : make_uint4(0u, 0u, 0u, 0u);
        vx[c] = valid ? __ldg(reinterpret_cast<const uint4*>(a.cache.v_codes + at * HB) + c) : make_uint4(0u, 0u, 0u, 0u);
      }
      ks = valid ? __ldg(a.cache.k_scales + at) * c_log2 : 0.0f;
      vs = valid ? __ldg(a.cache.v_scales + at) : 0.0f;
    };
    if (steps > 0) load(0);
    for (int j = 0; j < steps; ++j) {
      const int s = j % PR_STAGES, sc = j % SC_RING;
      const uint32_t reuse = ((uint32_t)(j / PR_STAGES) & 1u) ^ 1u;
      if (!pr_warp_wait(&S.k_empty[s], reuse, &S.abort_flag, a.status)) break;
      S.ks[sc][t] = ks;
      S.vs[sc][t] = vs;
      const uint32_t bits = __ballot_sync(0xffffffffu, valid);
      float vm = finite_or_0(vs);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
      if (lane == 0) {
        S.valid[sc][wq] = bits;
        S.vmax[sc][wq] = vm;
      }
#pragma unroll
      for (int c = 0; c < HB / 16; ++c) {
        const uint32_t x[4] = {kx[c].x, kx[c].y, kx[c].z, kx[c].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {                    // a word: 8 channels, one 16-byte chunk
          const int ch = 4 * c + q;
          *reinterpret_cast<uint4*>(S.k[s][ch / 8] + sw128(t, ch % 8)) =
              make_uint4(code_pair_bf16(x[q], 0), code_pair_bf16(x[q], 4), code_pair_bf16(x[q], 8), code_pair_bf16(x[q], 12));
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(&S.sc_full[sc]);
        ptx::mbar_arrive(&S.k_full[s]);
      }
      if (!pr_warp_wait(&S.v_empty[s], reuse, &S.abort_flag, a.status)) break;
#pragma unroll
      for (int c = 0; c < HB / 16; ++c) {
        const uint32_t x[4] = {vx[c].x, vx[c].y, vx[c].z, vx[c].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int ch = 4 * c + q;
          *reinterpret_cast<uint4*>(S.v[s][ch / 8] + sw128(t, ch % 8)) =
              make_uint4(code_pair(x[q], 0), code_pair(x[q], 4), code_pair(x[q], 8), code_pair(x[q], 12));
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.v_full[s]);
      if (j + 1 < steps) load(j + 1);
    }
  } else {
    ptx::setmaxnreg_dec<PR_REG_CTRL>();
    if (warp == 12 && lane == 0 && steps > 0) {
      // ------------------------------------------------------------------------- MMA issue
      constexpr uint32_t id_s = idesc_f16(1, 0, PT), id_o = idesc_f16(0, 1, HD);
      auto mma_s = [&](int i, int s) {
        const uint32_t q0 = ptx::smem_addr(S.q[i][0]), k0 = ptx::smem_addr(S.k[s][0]);
#pragma unroll
        for (int k = 0; k < HD / 16; ++k) {
          const uint32_t off = (uint32_t)((k / 4) * PT * 128 + 32 * (k % 4));
          ptx::umma_f16(tmem + S_COL + 128 * i, ptx::smem_desc_sw128(q0 + off), ptx::smem_desc_sw128(k0 + off), id_s,
                        k > 0 ? 1u : 0u);
        }
        ptx::umma_commit(&S.s_full[i]);
      };
      auto mma_o = [&](int i, int s, bool first) {
        const uint32_t v0 = ptx::smem_addr(S.v[s][0]);
#pragma unroll
        for (int k = 0; k < PT / 16; ++k)
          ptx::umma_f16_ts(tmem + O_COL + 128 * i, tmem + S_COL + 128 * i + 8 * k,
                           ptx::smem_desc_sw128_mn(v0 + 2048 * k, PT * 128), id_o, first && k == 0 ? 0u : 1u);
        ptx::umma_commit(&S.o_full[i]);
      };
      bool ok = pr_wait(&S.q_full, 0, &S.abort_flag, a.status) && pr_wait(&S.k_full[0], 0, &S.abort_flag, a.status);
      if (ok) {
        ptx::tc_fence_after();
        for (int i = 0; i < tiles; ++i) mma_s(i, 0);
        ptx::umma_commit(&S.k_empty[0]);
      }
      for (int j = 0; j < steps && ok; ++j) {
        const int s = j % PR_STAGES, s1 = (j + 1) % PR_STAGES;
        const bool more = j + 1 < steps;
        if (!(ok = pr_wait(&S.v_full[s], (uint32_t)(j / PR_STAGES) & 1u, &S.abort_flag, a.status))) break;
        if (more && !(ok = pr_wait(&S.k_full[s1], (uint32_t)((j + 1) / PR_STAGES) & 1u, &S.abort_flag, a.status))) break;
        for (int i = 0; i < tiles; ++i) {
          if (!(ok = pr_wait(&S.p_full[i], (uint32_t)j & 1u, &S.abort_flag, a.status))) break;
          ptx::tc_fence_after();
          mma_o(i, s, j == 0);
          // MMAs of one thread run in order: S_i is overwritten after its probabilities have been read
          if (more) mma_s(i, s1);
        }
        if (!ok) break;
        ptx::umma_commit(&S.v_empty[s]);
        if (more) ptx::umma_commit(&S.k_empty[s1]);
      }
      ptx::umma_commit(&S.mma_done);
      int never = 0;
      (void)ptx::mbar_wait_bounded(&S.mma_done, 0, &never, kPrWaitNs);
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

template <int HD>
pq_status launch_prompt(const Kv4AttnArgs& a, const Partials& part, int64_t tiles, cudaStream_t stream) {
  constexpr size_t smem = sizeof(PromptSmem<HD>) + 1024;
  static_assert(smem <= 232448, "shared memory exceeds 227 KB");
  static std::atomic<bool> done[kMaxDevices];
  cudaError_t e = set_kernel_attributes(reinterpret_cast<const void*>(kv4_prompt_kernel<HD>), (int)smem, done);
  if (e != cudaSuccess) return cuda_fail(e, "kv4_prompt_kernel attributes");
  // The warp roles re-divide the launch's registers, which works only if it was compiled with exactly that many.
  static std::atomic<int> regs{-1};
  if (regs.load(std::memory_order_relaxed) < 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kv4_prompt_kernel<HD>);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes(prompt)");
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != (int)PR_REG_LAUNCH) {
    set_error("kv4_prompt_kernel compiled with %d registers per thread, %u expected", regs.load(), PR_REG_LAUNCH);
    return PQ_ERR_CUDA;
  }
  const int64_t grid = tiles * a.cache.heads * part.chunks;
  if (grid >= ((int64_t)1 << 31)) { set_error("too many query tiles for one call"); return PQ_ERR_INVALID_ARG; }
  kv4_prompt_kernel<HD><<<(unsigned)grid, PR_THREADS, smem, stream>>>(a, part);
  return cuda_fail(cudaGetLastError(), "kv4_prompt_kernel launch");
}

}  // namespace

int64_t kv4_prompt_tiles(const Kv4AttnArgs& a) {
  const int64_t group = a.heads_q / a.cache.heads;
  return (a.T * group + 2 * PT - 1) / (2 * PT) + a.B;
}

pq_status launch_kv4_prompt(const Kv4AttnArgs& a, const Partials& part, cudaStream_t stream) {
  const int64_t tiles = kv4_prompt_tiles(a);
  return a.cache.head_dim == 128 ? launch_prompt<128>(a, part, tiles, stream) : launch_prompt<64>(a, part, tiles, stream);
}

}  // namespace pq
