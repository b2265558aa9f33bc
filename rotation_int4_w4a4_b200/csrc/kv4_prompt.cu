// Attention over the paged 4-bit cache for many query rows a sequence (prompts and long chunks) on tcgen05 tensor
// cores, sm_100a.  The mathematics is that of the few-row kernel (kv4_attention.cu): per row
//   s_t = scale (q . kc_t) ks_t,  o = sum_t softmax(s)_t vs_t vc_t,  all sums float32.
//
// The query rows of one key/value head (row = new token x head of the group) come in tiles of 128 = the lanes of tensor
// memory; a CTA takes two tiles (256 rows, i = 0, 1) and walks the cached tokens 128 at a time, staged once for both,
// in halves of 64:
//   S_i = Q_i K^T   (fp16, M128 N64)        into 64 columns of tensor memory, two buffers a tile
//   P_i = softmax numerators, fp16, written over S_i's columns
//   O_i += P_i V    (A from tensor memory, M128 N head_dim) into head_dim more columns
// The scores of the next half are computed before the probabilities of this one are awaited, so a tile's softmax finds
// them ready: with one buffer of 128 it waited for the products of every step (5000 of 9000 cycles, measured).  The
// tensor cores and the exponentials (16 a clock and SM) are about evenly loaded: 2 x 128 x 128 x head_dim multiply-adds
// against 128 x 128 exponentials a tile and step.
//   warps 0, 1         MMA issue for tile 0, 1 (0: tensor memory).  The oldest warps: the others' waiting polls must
//                      not take their issue slots.
//   warps 4..7, 8..11  softmax of tile 0, 1: a thread owns a row: its scores from tensor memory, exponentials, P back;
//                      the reference they are taken against moves, and O is rescaled in tensor memory, only when a
//                      row's P would outgrow fp16; at the end its output row.
//   warps 12..15       producers: 128 tokens' codes from the pages, unpacked to fp16 keys and values in the swizzled
//                      operand layout, two stages each; their scales beside them.
// Spills in a half step cost much: the operands leave so little of the L1 cache that they come back from L2 (with the next
// half's scores loaded ahead, 400 bytes spilled: 655 us instead of 564).  The compiler reports 40 bytes of stores and 84 of
// loads (heads of 64: 28 and 56); which code they belong to is not known.
// 4096 of 8192 tokens, 32 + 8 heads of 128: 505 us, 51% of the library's bf16 rate; a half step takes 2300 cycles, of which
// the matrix instructions need 1400 and the exponentials 1000: the chain scores -> exponentials -> P -> product -> next
// scores bounds it, with 10% of the SMs' time idle behind the last blocks.
//
// Where the scales go.  Of 32 tokens that every row of the block sees and whose scales are of a size (kScaleSpread), keys
// and values come with their scales multiplied in, as fp16 relative to a power of two for each 32 tokens (a key: one
// rounding of code * scale; a value: the scale's and the product's; half a step is 2^-11, an eighth of a bf16 cache's).
// With the scales left to the softmax, every thread would read two scales a token from shared memory, a broadcast that
// costs four times its bytes: measured, 3800 of 6200 shared-memory cycles a step.  Where scales differ by more, or some row
// must not see a token (the diagonal, a window's edge, the ends of a sequence), the 32 keep the bare codes, exact, and the
// scales in the softmax, where a hidden token's can be left out whatever it holds: a row's result must not depend on it,
// not even in its last bit.
// Queries become fp16 relative to their row's largest channel (exact but for channels below 2^-25 of it).
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
constexpr int PR_SOFT0 = 4, PR_PROD0 = 12;               // first softmax and producer warps; 0 and 1 issue MMAs
constexpr int HT = PT / 2;               // tokens of a half step
constexpr int PR_STAGES = 2;             // key and value stages
constexpr int SC_RING = 4;               // scale stages: a step's scales outlive its keys by at most one step
constexpr uint64_t kPrWaitNs = 2000000000ull;
constexpr uint32_t S_COL = 0, O_COL = 256;               // tensor memory: S_i at 128 i + 64 (half & 1), O_i at 256 + 128 i
constexpr float kTop = 32768.0f;         // sum of 64 probabilities (fp16 holds 65504) from which it is taken elsewhere
// Scales are multiplied into the operands of 32 tokens whose key scales (0 aside) lie within this factor, and their value
// scales (0 counts: such a token's score must not set the reference).  The reference of such a step is its largest score plus
// the exponent of its largest value scale, which may belong to another token: the largest product is then up to 2^6 below 1
// and keeps 18 of fp16's 24 places below it.  Within the factor every operand is a normal fp16 number (of scales above 2^-100).
// 4096 of 8192 tokens: 478 us with every step so, 482 where the first 64 tokens differ by more, 696 where all do.
constexpr float kScaleSpread = 64.0f;
// kind::f16 on fp16 operands (types 0 at bits 7 and 10) with a float32 accumulator, B MN-major at bit 16.
__host__ __device__ constexpr uint32_t idesc_f16(int b_mn_major, int N) {
  return (1u << 4) | ((uint32_t)b_mn_major << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(PT >> 4) << 24);
}

template <int HD>
struct __align__(1024) PromptSmem {
  static constexpr int KBLK = HD / 64;                   // 128-byte blocks of a row
  uint8_t q[2][KBLK][PT * 128];
  uint8_t k[PR_STAGES][KBLK][PT * 128];
  uint8_t v[PR_STAGES][KBLK][PT * 128];
  // What multiplies a token's score, and its probability: its scales, or (scales multiplied in) its group's powers of 2.
  float ks[SC_RING][PT], vs[SC_RING][PT];
  float ve[SC_RING][PT];                                 // value_exponent of vs
  uint32_t valid[SC_RING][4];                            // which tokens exist, a bit each
  int scaled[SC_RING][4];                                // the 32 tokens' scales are in the operands
  float k_pow[SC_RING][4], v_exp[SC_RING][4];            // 2^e of each 32 keys, e of each 32 values
  uint64_t q_full;
  uint64_t k_full[PR_STAGES], k_empty[PR_STAGES], v_full[PR_STAGES], v_empty[PR_STAGES];
  uint64_t sc_full[SC_RING];
  uint64_t s_full[2][2], p_full[2][2], o_full[2][2];     // [tile][half step & 1]
  uint64_t mma_done;
  uint32_t tmem_slot;
  int abort_flag;
};

// spins: polls before the waiting warp sleeps between them.  Softmax and MMA issue poll (a sleeping warp comes back
// late); the producers, two stages ahead, sleep: their polls would take issue slots from the others.
constexpr int kSpin = 200;
__device__ __forceinline__ bool pr_warp_wait(uint64_t* bar, uint32_t parity, int* abort_flag, unsigned int* status,
                                             int spins = kSpin) {
  // the whole warp polls: an elected lane's answer would have to travel to the others first (4096 of 8192 tokens: 533 us
  // that way, 496 this way)
  if (__all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, parity, abort_flag, kPrWaitNs, spins))) return true;
  if ((threadIdx.x & 31) == 0) {
    *abort_flag = 1;
    atomicOr(status, PQ_DEV_TIMEOUT);
  }
  __syncwarp();
  return false;
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
    if (b < a.B) new_tokens(a.q_start, (int)a.T, b, q0, qlen);
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

// Pairs through one butterfly: (x + y, x - y).
__device__ __forceinline__ void butterfly2(uint64_t& x, uint64_t& y) {
  const uint64_t s = ptx::f2_add(x, y);
  y = ptx::f2_sub(x, y);
  x = s;
}

// Swizzled place of 16-byte chunk c of row r in a block of 128-byte rows.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// Largest of 32 raw scores.
__device__ __forceinline__ float chunk_max(const uint32_t (&r)[32]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int k = 0; k < 16; ++k)
    m[k % 4] = ptx::max3(m[k % 4], __uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// 2^(c s + off) of 32 scores: 16 registers of fp16 pairs, and their sum.
__device__ __forceinline__ float chunk_exp(const uint32_t (&r)[32], float c, float off, uint32_t (&p)[16]) {
  const uint64_t c2 = ptx::f2_pack(c, c), off2 = ptx::f2_pack(off, off);
  uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    float e0, e1;
    ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])), c2, off2), e0, e1);
    e0 = ex2(e0);
    e1 = ex2(e1);
    sum[k & 3] = ptx::f2_add(sum[k & 3], ptx::f2_pack(e0, e1));
    p[k] = pack_f16(e0, e1);
  }
  float a0, a1;
  ptx::f2_unpack(ptx::f2_add(ptx::f2_add(sum[0], sum[1]), ptx::f2_add(sum[2], sum[3])), a0, a1);
  return a0 + a1;
}

// Bits of the 64 tokens from `first` on that lie in [lo, hi].
__device__ __forceinline__ uint64_t token_bits(int first, int lo, int hi) {
  const int a = lo - first, b = hi - first;
  const uint64_t upto = b < 0 ? 0ull : b >= 63 ? ~0ull : (2ull << b) - 1;
  const uint64_t from = a <= 0 ? ~0ull : a > 63 ? 0ull : ~0ull << a;
  return upto & from;
}

// The same with the scales of 32 tokens (log2 units), of which the row sees some (a bit each): the largest score
// plus exponent of the value scale.  What a hidden token holds is selected away, never multiplied by 0.
__device__ __forceinline__ float chunk_top(const uint32_t (&r)[32], uint32_t seen, const float4* ks, const float4* ve, float c) {
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float4 k4 = ks[k], v4 = ve[k];
    const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, vv[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (seen & (1u << (4 * k + q))) top = fmaxf(top, fmaf(__uint_as_float(r[4 * k + q]), kk[q] * c, vv[q]));
  }
  return top;
}

// chunk_exp with the scales: probabilities times value scales in p; top: the largest magnitude of those so far.
__device__ __forceinline__ float chunk_exp_masked(const uint32_t (&r)[32], uint32_t seen, const float4* ks, const float4* vs,
                                                  float c, float off, uint32_t (&p)[16], float& top) {
  const uint64_t c2 = ptx::f2_pack(c, c), off2 = ptx::f2_pack(off, off);
  uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float4 k4 = ks[k], v4 = vs[k];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int t = 4 * k + 2 * q;
      const uint64_t f = ptx::f2_mul(q ? ptx::f2_pack(k4.z, k4.w) : ptx::f2_pack(k4.x, k4.y), c2);
      float e0, e1, y0, y1;
      ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(r[t]), __uint_as_float(r[t + 1])), f, off2), e0, e1);
      const bool s0 = seen & (1u << t), s1 = seen & (2u << t);
      e0 = s0 ? ex2(e0) : 0.0f;
      e1 = s1 ? ex2(e1) : 0.0f;
      sum[q] = ptx::f2_add(sum[q], ptx::f2_pack(e0, e1));
      y0 = e0 * (s0 ? (q ? v4.z : v4.x) : 0.0f);
      y1 = e1 * (s1 ? (q ? v4.w : v4.y) : 0.0f);
      top = ptx::max3(top, fabsf(y0), fabsf(y1));
      p[t / 2] = pack_f16(y0, y1);
    }
  }
  float a0, a1;
  ptx::f2_unpack(ptx::f2_add(sum[0], sum[1]), a0, a1);
  return a0 + a1;
}

// Columns of tensor memory hold channels in the operands' order: place 2k of each 8 channel k, 2k + 1 channel k + 4 (odd
// k: 16 times too large on the keys' side, which the queries undo, and on the values' side, undone here).
__device__ __forceinline__ void load_channels(float (&o)[32], uint32_t col) {
  uint32_t x[32];
  ptx::tmem_ld32(col, x);
  ptx::tmem_ld_wait(x);
#pragma unroll
  for (int c = 0; c < 32; c += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = k & 1 ? kOddNibble : 1.0f;
      o[c + k] = __uint_as_float(x[c + 2 * k]) * f;
      o[c + k + 4] = __uint_as_float(x[c + 2 * k + 1]) * f;
    }
}

// Unnormalised Walsh-Hadamard transform (Sylvester order) of a row's HD columns: the stages within 32 channels go back
// to tensor memory, those across them follow 16 columns of each 32 at a time; put(c, v) takes channels c .. c + 15 of
// the 32-channel block b.  Two columns an instruction (channels k and k + 4) but for the stage between them.
template <int HD, typename Put>
__device__ __forceinline__ void rotate_row(uint32_t col, Put put) {
  constexpr int N32 = HD / 32;
  const uint64_t up = ptx::f2_pack(kOddNibble, kOddNibble), down = ptx::f2_pack(-kOddNibble, -kOddNibble);
#pragma unroll 1
  for (int c = 0; c < HD; c += 32) {
    uint32_t x[32];
    uint64_t v[16];
    ptx::tmem_ld32(col + c, x);
    ptx::tmem_ld_wait(x);
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = ptx::f2_pack(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
#pragma unroll
    for (int k = 0; k < 16; k += 2) {                    // channels k, k + 1; the odd one's factor goes in
      const uint64_t y = v[k + 1];
      v[k + 1] = ptx::f2_fma(y, down, v[k]);
      v[k] = ptx::f2_fma(y, up, v[k]);
    }
#pragma unroll
    for (int h = 2; h < 16; h <<= 1) {                   // channels 2, 8, 16 apart
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if ((k & h) == 0) butterfly2(v[k], v[k + h]);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {                       // 4 apart
      float a, b;
      ptx::f2_unpack(v[k], a, b);
      x[2 * k] = __float_as_uint(a + b);
      x[2 * k + 1] = __float_as_uint(a - b);
    }
    ptx::tmem_st32x16(col + c, reinterpret_cast<const uint32_t(&)[16]>(x[0]));
    ptx::tmem_st32x16(col + c + 16, reinterpret_cast<const uint32_t(&)[16]>(x[16]));
  }
  ptx::tmem_st_wait();
#pragma unroll 1
  for (int c = 0; c < 32; c += 16) {
    uint32_t x[N32][16];
    uint64_t v[N32][8];
#pragma unroll
    for (int b = 0; b < N32; ++b) ptx::tmem_ld32x16(col + 32 * b + c, x[b]);
#pragma unroll
    for (int b = 0; b < N32; ++b) {
      ptx::tmem_ld_wait(x[b]);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[b][k] = ptx::f2_pack(__uint_as_float(x[b][2 * k]), __uint_as_float(x[b][2 * k + 1]));
    }
#pragma unroll
    for (int h = 1; h < N32; h <<= 1)
#pragma unroll
      for (int b = 0; b < N32; ++b)
        if ((b & h) == 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) butterfly2(v[b][k], v[b + h][k]);
        }
#pragma unroll
    for (int b = 0; b < N32; ++b)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float y[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) ptx::f2_unpack(v[b][4 * g + k], y[k], y[k + 4]);
        put(4 * b + c / 8 + g, y);
      }
  }
}
__device__ __forceinline__ uint4 bf16x8(const float* o, float f) {
  return make_uint4(pack_bf16(o[0] * f, o[1] * f), pack_bf16(o[2] * f, o[3] * f), pack_bf16(o[4] * f, o[5] * f),
                    pack_bf16(o[6] * f, o[7] * f));
}

// Whether every row of the block sees all of the 32 tokens from tok0 on: known from the lengths alone.
struct Interior {
  int c_lo, c_hi, p_first, p_last, window;
  __device__ __forceinline__ bool operator()(int tok0) const {
    return tok0 >= c_lo && tok0 + 32 <= c_hi && tok0 + 31 <= p_first && (window <= 0 || tok0 > p_last - window);
  }
};

template <int HD>
__global__ void __launch_bounds__(PR_THREADS, 1) kv4_prompt_kernel(const Kv4AttnArgs a, const Partials part) {
  using Smem = PromptSmem<HD>;
  constexpr int HB = HD / 2;
  extern __shared__ unsigned char smem_raw[];
  // an offset, not an address: the compiler keeps seeing shared memory
  Smem& S = *reinterpret_cast<Smem*>(smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  ptx::griddep_launch_dependents();                      // the kernel that joins chunks waits for this one
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
  const Interior interior{c_lo, c_hi, p_first, p_last, a.window};

  if (threadIdx.x == 32) {
    ptx::mbar_init(&S.q_full, 8);
    for (int s = 0; s < PR_STAGES; ++s) {
      ptx::mbar_init(&S.k_full[s], 4);
      ptx::mbar_init(&S.k_empty[s], tiles);
      ptx::mbar_init(&S.v_full[s], 4);
      ptx::mbar_init(&S.v_empty[s], tiles);
    }
    for (int s = 0; s < SC_RING; ++s) ptx::mbar_init(&S.sc_full[s], 4);
    for (int i = 0; i < 2; ++i) {
      for (int b = 0; b < 2; ++b) {
        ptx::mbar_init(&S.s_full[i][b], 1);
        ptx::mbar_init(&S.p_full[i][b], 4);
        ptx::mbar_init(&S.o_full[i][b], 1);
      }
    }
    ptx::mbar_init(&S.mma_done, tiles);
    S.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 0) {
    ptx::tmem_alloc(&S.tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = S.tmem_slot;

  if (warp >= PR_SOFT0 && warp < PR_PROD0) {
    // ------------------------------------------------------------------------------- softmax
    const int i = (warp - PR_SOFT0) >> 2;                // row tile
    const int row = (warp & 3) * 32 + lane;              // lane of tensor memory
    const int r = w.r0 + PT * i + row;
    const bool live = r < w.rows;
    const int rr = min(r, w.rows - 1);
    const int head = w.kvh * group + rr % group;
    // Rows come from and go to memory RPI at a time, LPR lanes a row (a row a lane touches 32 lines an instruction), and
    // pass through shared memory, where a thread reaches its own.  Loops stay rolled: code that runs once is bound by
    // its fetch.
    constexpr int LPR = HD / 8, RPI = 32 / LPR;
    const int io_row = (warp & 3) * 32 + lane / LPR, io_chunk = lane % LPR;
    auto place = [&](int r_, int c) { return reinterpret_cast<uint4*>(S.q[i][c / 8] + sw128(r_, c % 8)); };
    // body(row of the tile, token, query head) over the warp's rows that exist.  Rows of the tile are few: dividing by the
    // group is a multiplication by its reciprocal (rows + group below 2^16).
    const int tile_tok = (w.r0 + PT * i) / group, tile_off = (w.r0 + PT * i) % group;
    const uint32_t inv_group = group == 1 ? 0u : 0xffffffffu / (uint32_t)group + 1u;
    auto each_row = [&](auto body) {
#pragma unroll 4
      for (int k = 0; k < LPR; ++k) {
        const int to = io_row + RPI * k, x = to + tile_off;
        const int t = group == 1 ? x : (int)__umulhi((uint32_t)x, inv_group);
        if (w.r0 + PT * i + to < w.rows) body(to, (int64_t)w.q0 + tile_tok + t, w.kvh * group + x - t * group);
      }
    };
    float c_row;                                         // raw scores to log2 units, but for the keys' power of two
    {
      each_row([&](int to, int64_t t, int hq) {
        ptx::cp_async16(place(to, io_chunk), reinterpret_cast<const uint4*>(a.Q + t * a.ldq + hq * HD) + io_chunk, 16);
      });
      ptx::cp_async_wait_all();
      __syncwarp();
      // largest magnitude, two channels an instruction; infinities and NaN do not count (the rare second pass)
      uint32_t mw = 0u;
#pragma unroll 4
      for (int c = 0; c < HD / 8; ++c) {
        const uint4 x = *place(row, c);
        mw = __vimax3_u16x2(mw, x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu);
        mw = __vimax3_u16x2(mw, x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu);
      }
      float mq = __uint_as_float(max(mw << 16, mw & 0xFFFF0000u));
      if (!(mq < INFINITY)) {
        mq = 0.0f;
#pragma unroll 1
        for (int c = 0; c < HD; ++c)
          mq = fmaxf(mq, finite_or_0(__uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(place(row, c / 8))[c % 8] << 16)));
      }
      const float eq = scale_exponent(live ? mq : 0.0f);
      const float up = ex2(kQueryExp - eq), f = a.scale < 0.0f ? -up : up, f16 = f * kOddNibble;
      c_row = fabsf(a.scale) * kLog2e * ex2(eq - kQueryExp);
      // channels 0 4 | 1 5 | 2 6 | 3 7; the keys' odd channels come 16 times too large
#pragma unroll 4
      for (int c = 0; c < HD / 8; ++c) {
        uint4 x = *place(row, c);
        if (!live) x = make_uint4(0u, 0u, 0u, 0u);
        auto even = [&](uint32_t lo, uint32_t hi) { return pack_f16(__uint_as_float(lo << 16) * f, __uint_as_float(hi << 16) * f); };
        auto odd = [&](uint32_t lo, uint32_t hi) {
          return pack_f16(__uint_as_float(lo & 0xFFFF0000u) * f16, __uint_as_float(hi & 0xFFFF0000u) * f16);
        };
        *place(row, c) = make_uint4(even(x.x, x.z), odd(x.x, x.z), even(x.y, x.w), odd(x.y, x.w));
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.q_full);
    }
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const uint32_t s_col = lane_base + S_COL + 128 * i, o_col = lane_base + O_COL + 128 * i;
    float m = -INFINITY, l = 0.0f;
    bool ok = i < tiles;
    for (int h = 0; h < 2 * steps && ok; ++h) {            // half steps
      const int j = h >> 1, sc = j % SC_RING, t0 = HT * (h & 1);
      const uint32_t s_buf = s_col + t0;
      if (t0 == 0) ok = pr_warp_wait(&S.sc_full[sc], (uint32_t)(j / SC_RING) & 1u, &S.abort_flag, a.status);
      ok = ok && pr_warp_wait(&S.s_full[i][h & 1], (uint32_t)j & 1u, &S.abort_flag, a.status);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint4 valid = *reinterpret_cast<const uint4*>(S.valid[sc]);
      const uint32_t va = t0 ? valid.z : valid.x, vb = t0 ? valid.w : valid.y;
      // Raises rows' references to cand (largest score plus exponent of a value scale), in the sum and in O.
      auto raise = [&](bool grow, float cand) {
        const float m_new = grow ? cand : m;
        const float f = m_new == -INFINITY ? 1.0f : ex2(m - m_new);
        m = m_new;
        l *= f;
        if (h == 0) return true;
        if (!pr_warp_wait(&S.o_full[i][(h - 1) & 1], (uint32_t)((h - 1) >> 1) & 1u, &S.abort_flag, a.status)) return false;
        ptx::tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < HD; c += 16) {
          uint32_t o[16];
          ptx::tmem_ld32x16(o_col + c, o);
          ptx::tmem_ld_wait(o);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
          ptx::tmem_st32x16(o_col + c, o);
        }
        return true;
      };
      // The maximum is not taken first: the reference of the halves before serves until a row's probabilities outgrow
      // it, and only then (and at first) is the maximum found, the reference raised and the half done again.
      uint32_t pa[16], pb[16];
      if ((va & vb) == 0xffffffffu && (S.scaled[sc][2 * (h & 1)] & S.scaled[sc][2 * (h & 1) + 1]) != 0) {
        bool over = m == -INFINITY;
        float2 kp = *reinterpret_cast<const float2*>(&S.k_pow[sc][2 * (h & 1)]);
        const float2 v2 = *reinterpret_cast<const float2*>(&S.v_exp[sc][2 * (h & 1)]);
        kp.x *= c_row, kp.y *= c_row;
        float sum0, sum1;
        for (int pass = 0;; ++pass) {
          uint32_t xa[32], xb[32];                       // the scores of the half's two groups of 32 tokens
          ptx::tmem_ld32(s_buf, xa);
          ptx::tmem_ld32(s_buf + 32, xb);
          ptx::tmem_ld_wait(xa);
          ptx::tmem_ld_wait(xb);
          if (__any_sync(0xffffffffu, over)) {
            const float cand = fmaxf(fmaf(chunk_max(xa), kp.x, v2.x), fmaf(chunk_max(xb), kp.y, v2.y));
            if (!(ok = raise(over && cand > m, cand))) break;
          }
          const float ref = m == -INFINITY ? 0.0f : m;
          sum0 = chunk_exp(xa, kp.x, v2.x - ref, pa);
          sum1 = chunk_exp(xb, kp.y, v2.y - ref, pb);
          over = sum0 + sum1 > kTop;
          if (pass == 1 || !__any_sync(0xffffffffu, over)) break;
        }
        if (!ok) break;
        // each sum without its values' power of two
        l = fmaf(sum0, ex2(-v2.x), fmaf(sum1, ex2(-v2.y), l));
      } else {
        const int pos = n - w.qlen + rr / group;
        const uint64_t bits = token_bits((j0 + j) * PT + t0, a.window > 0 ? max(pos - a.window + 1, c_lo) : c_lo, min(pos, c_hi - 1));
        const uint32_t sa = (uint32_t)bits & va, sb = (uint32_t)(bits >> 32) & vb;
        const float4* ks = reinterpret_cast<const float4*>(S.ks[sc]) + t0 / 4;
        const float4* vs = reinterpret_cast<const float4*>(S.vs[sc]) + t0 / 4;
        float sum = 0.0f;
        bool over = m == -INFINITY && (sa | sb) != 0u;
        for (int pass = 0;; ++pass) {
          uint32_t x[32];
          if (__any_sync(0xffffffffu, over)) {
            float cand = -INFINITY;
#pragma unroll 1
            for (int g = 0; g < 2; ++g) {
              ptx::tmem_ld32(s_buf + 32 * g, x);
              ptx::tmem_ld_wait(x);
              cand = fmaxf(cand, chunk_top(x, g ? sb : sa, ks + 8 * g, reinterpret_cast<const float4*>(S.ve[sc]) + t0 / 4 + 8 * g, c_row));
            }
            if (!(ok = raise(over && cand > m, cand))) break;
          }
          const float ref = m == -INFINITY ? 0.0f : m;
          float top = 0.0f;
          ptx::tmem_ld32(s_buf, x);
          ptx::tmem_ld_wait(x);
          sum = chunk_exp_masked(x, sa, ks, vs, c_row, -ref, pa, top);
          ptx::tmem_ld32(s_buf + 32, x);
          ptx::tmem_ld_wait(x);
          sum += chunk_exp_masked(x, sb, ks + 8, vs + 8, c_row, -ref, pb, top);
          over = top > kTop || sum > kSumTop;
          if (pass == 1 || !__any_sync(0xffffffffu, over)) break;
        }
        if (!ok) break;
        l += sum;
      }
      ptx::tmem_st32x16(s_buf, pa);
      ptx::tmem_st32x16(s_buf + 16, pb);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.p_full[i][h & 1]);
    }
    // ---- the row's output, 32 channels at a time
    if (i < tiles) {
      if (ok && steps > 0) ok = pr_warp_wait(&S.o_full[i][1], (uint32_t)(steps - 1) & 1u, &S.abort_flag, a.status);
      ptx::tc_fence_after();
      const bool some = ok && steps > 0;
      // The queries' place (their products are done) takes each row's output, HD / 8 chunks of 16 bytes; rows leave from
      // there whole.  A warp touches its own rows only.
      auto stage = [&](int c, uint4 x) { *place(row, c) = x; };
      auto flush = [&](auto dst_of) {                    // dst_of(token, head): where the row goes
        __syncwarp();
        each_row([&](int from, int64_t t, int hq) { reinterpret_cast<uint4*>(dst_of(t, hq))[io_chunk] = *place(from, io_chunk); });
        __syncwarp();
      };
      if (part.chunks > 1) {
        const int64_t token = w.q0 + rr / group, first = (int64_t)w.chunk * a.T;
        if (live) part.ml[(first + token) * a.heads_q + head] = make_float2(some ? m : -INFINITY, some ? l : 0.0f);
        if (some) {
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {         // HD / 2 channels in float32 fill the place
#pragma unroll 1
            for (int c = 0; c < HD / 2; c += 32) {
              float o[32];
              load_channels(o, o_col + half * (HD / 2) + c);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                stage(c / 4 + k, make_uint4(__float_as_uint(o[4 * k]), __float_as_uint(o[4 * k + 1]), __float_as_uint(o[4 * k + 2]),
                                            __float_as_uint(o[4 * k + 3])));
            }
            flush([&](int64_t t, int hq) { return part.o + ((first + t) * a.heads_q + hq) * HD + half * (HD / 2); });
          }
        }
      } else {
        const float f = l == 0.0f ? 0.0f : 1.0f / l;
        if (!some) {
#pragma unroll 1
          for (int c = 0; c < HD / 8; ++c) stage(c, make_uint4(0u, 0u, 0u, 0u));
        } else if (!a.cache.rotate_v) {
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            float o[32];
            load_channels(o, o_col + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) stage(c / 8 + k, bf16x8(o + 8 * k, f));
          }
        } else {                                         // x H / sqrt(head_dim)
          const float fr = f * (HD == 128 ? 0.08838834764831845f : 0.125f);
          rotate_row<HD>(o_col, [&](int c, const float* y) { stage(c, bf16x8(y, fr)); });
        }
        flush([&](int64_t t, int hq) { return a.O + t * a.ldo + (int64_t)hq * HD; });
      }
      ptx::tc_fence_before();
    }
  } else if (warp >= PR_PROD0) {
    // ----------------------------------------------------------------------------- producers
    const int t = threadIdx.x - 32 * PR_PROD0;           // token of the step
    const int wq = warp - PR_PROD0;
    const int32_t* table = a.table + w.b * a.table_stride;
    uint4 kx[HB / 16], vx[HB / 16];
    float ks, vs;
    int64_t at = -1, at_next = -1;                       // cache row of the token (-1: none), one step ahead
    auto locate = [&](int j) {
      const int tok = (j0 + j) * PT + t;
      at_next = -1;
      if (tok >= c_lo && tok < c_hi && j < steps) {
        const int page = table[tok >> ps];
        if (page < 0 || page >= a.cache.pages) atomicOr(a.status, PQ_DEV_BAD_INDEX);
        else at_next = (((int64_t)page * a.cache.heads + w.kvh) << ps) + (tok & ((1 << ps) - 1));
      }
    };
    auto load = [&](uint4 (&x)[HB / 16], float& sc, const uint8_t* codes, const float* scales, int64_t r) {
#pragma unroll
      for (int c = 0; c < HB / 16; ++c)
        x[c] = r >= 0 ? __ldg(reinterpret_cast<const uint4*>(codes + r * HB) + c) : make_uint4(0u, 0u, 0u, 0u);
      sc = r >= 0 ? __ldg(scales + r) : 0.0f;
    };
    locate(0);
    at = at_next;
    load(kx, ks, a.cache.k_codes, a.cache.k_scales, at);
    load(vx, vs, a.cache.v_codes, a.cache.v_scales, at);
    locate(1);
    for (int j = 0; j < steps; ++j) {
      const int s = j % PR_STAGES, sc = j % SC_RING;
      const uint32_t reuse = ((uint32_t)(j / PR_STAGES) & 1u) ^ 1u;
      if (!pr_warp_wait(&S.k_empty[s], reuse, &S.abort_flag, a.status, 0)) break;
      const uint32_t bits = __ballot_sync(0xffffffffu, at >= 0);
      const float km = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(finite_or_0(ks))));
      const float vm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(finite_or_0(vs))));
      const float k1 = finite_or_0(ks);
      const float k_least = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(k1 == 0.0f ? INFINITY : k1)));
      const float v_least = __uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(finite_or_0(vs))));
      const bool scaled = interior((j0 + j) * PT + 32 * wq) && km <= kScaleSpread * k_least && vm < kScaleSpread * v_least;
      const float ke = scale_exponent(km), ve = scale_exponent(vm);
      S.ks[sc][t] = scaled ? ex2(ke) : ks;
      S.vs[sc][t] = scaled ? ex2(ve) : vs;
      S.ve[sc][t] = scaled ? ve + 1.0f : value_exponent(vs);
      if (lane == 0) {
        S.scaled[sc][wq] = scaled ? 1 : 0;
        S.valid[sc][wq] = bits;
        S.k_pow[sc][wq] = ex2(ke);
        S.v_exp[sc][wq] = ve;
      }
      // code * scale in one rounding: scale as fp16 high and low parts, code * low below the fused multiply-add
      const float kn = ks * ex2(-ke);
      const __half2 k_hi = __float2half2_rn(kn), k_lo = __float2half2_rn(kn - __low2float(k_hi));
      const __half2 v_hi = __float2half2_rn(vs * ex2(-ve));
#pragma unroll
      for (int c = 0; c < HB / 16; ++c) {
        const uint32_t x[4] = {kx[c].x, kx[c].y, kx[c].z, kx[c].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {                    // a word: 8 channels, one 16-byte chunk
          const int ch = 4 * c + q;
          uint32_t y[4];
          code_pairs(x[q], y);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (scaled) {
              const __half2 code = *reinterpret_cast<const __half2*>(&y[k]);
              const __half2 z = __hfma2(code, k_hi, __hmul2(code, k_lo));
              y[k] = *reinterpret_cast<const uint32_t*>(&z);
            }
          }
          *reinterpret_cast<uint4*>(S.k[s][ch / 8] + sw128(t, ch % 8)) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(&S.sc_full[sc]);
        ptx::mbar_arrive(&S.k_full[s]);
      }
      // the next step's keys, under this step's values (and the other way round below)
      load(kx, ks, a.cache.k_codes, a.cache.k_scales, at_next);
      if (!pr_warp_wait(&S.v_empty[s], reuse, &S.abort_flag, a.status, 0)) break;
#pragma unroll
      for (int c = 0; c < HB / 16; ++c) {
        const uint32_t x[4] = {vx[c].x, vx[c].y, vx[c].z, vx[c].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int ch = 4 * c + q;
          uint32_t y[4];
          code_pairs(x[q], y);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (scaled) {
              const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&y[k]), v_hi);
              y[k] = *reinterpret_cast<const uint32_t*>(&z);
            }
          }
          *reinterpret_cast<uint4*>(S.v[s][ch / 8] + sw128(t, ch % 8)) = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&S.v_full[s]);
      load(vx, vs, a.cache.v_codes, a.cache.v_scales, at_next);
      at = at_next;
      locate(j + 2);
    }
  } else {
    const int i = warp;                                  // row tile
    if (i < tiles && steps > 0) {
      // ------------------------------------------------------------------------- MMA issue
      // The whole warp walks the half steps and one elected lane issues: descriptors stay in uniform registers.
      constexpr uint32_t id_s = idesc_f16(0, HT), id_o = idesc_f16(1, HD);
      // Descriptors of the operands' first tiles; an offset of b bytes adds b / 16 to the address field.
      constexpr uint64_t kTile = Smem::KBLK * PT * 128 / 16, kBlock = PT * 128 / 16, kHalf = HT * 128 / 16;
      const uint64_t dq = ptx::smem_desc_sw128(ptx::smem_addr(S.q[i][0]));
      const uint64_t dk = ptx::smem_desc_sw128(ptx::smem_addr(S.k[0][0]));
      const uint64_t dv = ptx::smem_desc_sw128_mn(ptx::smem_addr(S.v[0][0]), PT * 128);
      const uint32_t s_col = tmem + S_COL + 128 * i, o_col = tmem + O_COL + 128 * i;
      auto wait = [&](uint64_t* bar, uint32_t parity) { return pr_warp_wait(bar, parity, &S.abort_flag, a.status); };
      // Scores of half step h; its second half is the last to read the keys' stage.
      auto scores = [&](int h) {
        const int j = h >> 1, st = j % PR_STAGES;
        const uint64_t k0 = dk + (uint64_t)st * kTile + (uint64_t)(h & 1) * kHalf;
        const uint32_t d = s_col + HT * (h & 1);
        if (ptx::elect_one()) {
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint64_t off = (uint64_t)(k / 4) * kBlock + 2 * (k % 4);
            ptx::umma_f16(d, dq + off, k0 + off, id_s, k > 0 ? 1u : 0u);
          }
          ptx::umma_commit(&S.s_full[i][h & 1]);
          if (h & 1) ptx::umma_commit(&S.k_empty[st]);
        }
        __syncwarp();
      };
      bool ok = wait(&S.q_full, 0) && wait(&S.k_full[0], 0);
      if (ok) {
        ptx::tc_fence_after();
        scores(0);
      }
      for (int h = 0; h < 2 * steps && ok; ++h) {
        const int j = h >> 1, st = j % PR_STAGES;
        if (h + 1 < 2 * steps) {
          // MMAs of one thread run in order: the buffer's last probabilities have been read by then
          if (h & 1) {
            const int j1 = j + 1;
            if (!(ok = wait(&S.k_full[j1 % PR_STAGES], (uint32_t)(j1 / PR_STAGES) & 1u))) break;
            ptx::tc_fence_after();
          }
          scores(h + 1);
        }
        if ((h & 1) == 0 && !(ok = wait(&S.v_full[st], (uint32_t)(j / PR_STAGES) & 1u))) break;
        if (!(ok = wait(&S.p_full[i][h & 1], (uint32_t)j & 1u))) break;
        ptx::tc_fence_after();
        const uint64_t v0 = dv + (uint64_t)st * kTile + (uint64_t)(h & 1) * kHalf;
        const uint32_t p = s_col + HT * (h & 1);
        if (ptx::elect_one()) {
#pragma unroll
          for (int k = 0; k < HT / 16; ++k)
            ptx::umma_f16_ts(o_col, p + 8 * k, v0 + 128 * k, id_o, h == 0 && k == 0 ? 0u : 1u);
          ptx::umma_commit(&S.o_full[i][h & 1]);
          if (h & 1) ptx::umma_commit(&S.v_empty[st]);
        }
        __syncwarp();
      }
      if (ptx::elect_one()) ptx::umma_commit(&S.mma_done);
      __syncwarp();
      if (lane == 0) {
        int never = 0;
        (void)ptx::mbar_wait_bounded(&S.mma_done, 0, &never, kPrWaitNs);
      }
    }
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
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
  const int64_t grid = tiles * a.cache.heads * part.chunks;
  if (grid >= ((int64_t)1 << 31)) { set_error("too many query tiles for one call"); return PQ_ERR_INVALID_ARG; }
  kv4_prompt_kernel<HD><<<(unsigned)grid, PR_THREADS, smem, stream>>>(a, part);
  return cuda_fail(cudaGetLastError(), "kv4_prompt_kernel launch");
}

}  // namespace

int64_t kv4_prompt_tiles(const Kv4AttnArgs& a) {
  const int64_t group = a.heads_q / a.cache.heads;
  return (a.T * group + (2 * PT - 1) * (int64_t)a.B) / (2 * PT);   // a sequence's last tile may hold a single row
}

pq_status launch_kv4_prompt(const Kv4AttnArgs& a, const Partials& part, cudaStream_t stream) {
  const int64_t tiles = kv4_prompt_tiles(a);
  return a.cache.head_dim == 128 ? launch_prompt<128>(a, part, tiles, stream) : launch_prompt<64>(a, part, tiles, stream);
}

}  // namespace pq
