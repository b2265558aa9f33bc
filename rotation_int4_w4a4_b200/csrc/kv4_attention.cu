// Attention over the paged 4-bit cache for a few query rows a sequence (decode; sm_100a), and what chooses between this
// kernel and the one for prompts.
//
// Per query row (token at position p, query head) and cached token t of its key/value head, t <= p (and t > p - window):
//   s_t = scale (q . kc_t) ks_t,  P = softmax(s),  o = sum_t P_t vs_t vc_t   (then o H / sqrt(hd) for rotated values)
// kc, vc: 4-bit codes, ks, vs: their scales.  The codes are exact in fp16, so the products run on the tensor cores on
// the codes themselves; ks multiplies the finished dot product and vs the probability, both in float32.
//
// The cache is read once for all query rows of a key/value head (the group's heads x the sequence's new tokens), 64
// bytes a token for keys and as much for values.  Bytes are the floor.  Above it lie the instructions (about 650 for 32
// tokens of a head of 128), but no pipe is full: ALU 58%, issue 55%, DRAM 47%; a quarter of a warp's time is fixed latencies,
// a fifth its own issue, an eighth each memory, a busy pipe and other warps' turns.  The same time with all pages in L2, and
// with 16 warps an SM.  256 users of 4096 tokens: 287 us, 61% of the copy's bandwidth; 64 of up to 8192: 74; one of 65536: 33
// (call by call).
// A warp owns blocks of 32 tokens:
//   - keys are the A operand (16 tokens x 16 channels), the query rows the 8-column B operand: a thread's 16-byte
//     load of one token is its share of the A operands of all 8 channel steps, because the channels of a dot product
//     may be taken in any order as long as the queries follow the same one (set up once).  No shared memory.
//   - the scores come out tokens x rows and stay in the warp's registers;
//   - probabilities go back in as B operand (movmatrix transposes 8 x 8 of them) against the values as A operand
//     (16 channels x 16 tokens): two tokens' words are byte-permuted together, then masked.
//   - keys: nibble ^ 8 = code + 8 alone in an fp16 is (code + 8) 2^-24, below the normal range but exact, and four
//     places up 16 times that: one mask a pair of codes and one shift a word.  The offset 8 leaves with the query's sum
//     (the accumulator starts at -8 sum(q)), the factors with the queries, which become fp16 scaled below 2^15 (exact
//     down to 2^-25 of a row's largest) and with the scores' float32 factor.
//   - values become fp16: nibble ^ 8 under 0x6400 is 1024 + (code + 8), and 1032 is subtracted from the operand
//     itself, exactly, since a long sum of probabilities times 1032 would drown the result.
//   - the loads of the next block are issued as soon as this block's registers are free (168 a thread): 52 KB an SM in
//     flight.
// The second product takes P_t vs_t as fp16.  Both are relative to a reference (a score plus the exponent of a value
// scale) that a row keeps until its products outgrow fp16; only then, and at first, are the block's maximum score and
// value scale reduced over the warp.  Rounding a product costs half a step of fp16, 2^-11, an eighth of what bf16 would.
// Sums and the output are float32.
//
// A block's warps join their maxima, sums and outputs through shared memory.  The tokens of all sequences and heads are
// cut into equal shares, one for each block that runs at once (64 users of 0 to 8192 tokens: 74 us; chunks of fixed length,
// of which short sequences leave some empty: 89); a second kernel joins the float32 partial results.
//
// MASKED instances take sinks (under a window a row also sees the first tokens) and trees of drafted tokens (a list of bits says
// which of the new tokens a row sees).  They walk steps of 128 tokens: those with sinks, then the window's; the gap is not read.
// The tokens that a row sees of 32 are one word, made where some token may be hidden: a row of the cache is read once for all
// of a tree's rows.  64 users of 0 to 8192 tokens under a window of 1024 with 4 sinks: 35 us; one token over 65536 the same 13
// (of which 9 are a launch, the first loads and the output); 8 drafts over 1029 tokens 11.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "kv4.h"
#include "kv4_device.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace pq {
namespace {

constexpr int AT_WARPS = 4;
constexpr int AT_BLOCK = 32;            // tokens a warp takes at a time
constexpr int AT_TILES = AT_BLOCK / 16;
// Up to so many query rows a key/value head and sequence this kernel takes the call, beyond them the one of kv4_prompt.cu,
// whose tiles have 128 rows (us, this against that; 8 key/value heads of 128, the same for 1, 4 and 8 heads of queries on
// each).  64 sequences over 2048 tokens: 32 rows 137 : 162, 48 rows 192 : 162.  16 over 300: 32 rows 14 : 18, 48 rows 25 : 18.
// Where that kernel's tiles are few it comes later: 8 over 2048, 64 rows 42 : 51, 96 rows 56 : 37; one over 8192, 64 rows
// 29 : 29; one over 1024, 96 rows 19 : 24.
constexpr int64_t kPromptRows = 32;
constexpr float kRowsTop = 16384.0f;    // a product of probability and value scale from which the reference is raised (fp16: 65504)
// A nibble alone in the low bits of an fp16 is n 2^-24, below the normal range (matrix instructions take those at full
// value); four places up it is 16 times that.
constexpr float kCodeUnit = 5.9604644775390625e-8f;      // 2^-24

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t a0, const uint32_t a1, const uint32_t a2,
                                        const uint32_t a3, const uint32_t b0, const uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&x)[W], const uint8_t* p) {
  if constexpr (W == 4) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else if constexpr (W == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    x[0] = v.x, x[1] = v.y;
  } else {
    x[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
}

// Work cut into equal shares.  An item is one row tile of one sequence and key/value head; its length is the steps of 128
// tokens (a block's four warps, 32 each) of its sequence.  Items lie end to end (sequence, head, row tile) and each block
// takes the same number of steps of that line, so lengths that differ cost nothing.  A block whose share ends inside an
// item leaves a partial result: slot 2 c + 1 of block c for an item that begins there, 2 c for one that began before.
struct Shares {
  float* o;       // [2 blocks][R][HD], un-normalised
  float2* ml;     // [2 blocks][R]: reference exponent and sum
  int4* begun;    // [blocks]: sequence, head, row tile and last block of the item in slot 2 c + 1 (sequence -1: none)
  int blocks;     // 0: an item a block, no shares
};
constexpr int AT_STEP = AT_BLOCK * AT_WARPS;
constexpr int AT_SEQS = 1024;           // sequences whose lengths a block can add up
constexpr int AT_MIN_STEPS = 2;         // a share's least length
// Steps that an item's beginning and end cost, ahead of its own on the line (64 users, us: 0 steps 95, 1 85, 3 69, 6 73).
constexpr int AT_LEAD = 3;

struct Span {
  int q0, qlen, n, lo;                  // first token, new tokens, cached tokens, first token that any row's window holds
  int steps;
  int sink_steps;                       // MASKED: steps with sinks in front of the window's; the walk skips what lies between
};
template <bool MASKED>
__device__ __forceinline__ Span span_of(const Kv4AttnArgs& a, int b, bool report) {
  Span s;
  new_tokens(a.q_start, (int)a.T, b, s.q0, s.qlen);
  s.n = max(0, a.seq_lens[b]);
  const int64_t cap = (int64_t)a.table_width << a.cache.page_shift;
  if (s.n > cap) {
    s.n = (int)cap;
    if (report) atomicOr(a.status, PQ_DEV_BAD_INDEX);
  }
  s.lo = a.window > 0 ? max(0, s.n - s.qlen - a.window + 1) : 0;
  s.steps = max(1, (s.n + AT_STEP - 1) / AT_STEP - s.lo / AT_STEP);
  s.sink_steps = 0;
  if constexpr (MASKED) {
    s.sink_steps = min((min(a.sinks, s.n) + AT_STEP - 1) / AT_STEP, s.lo / AT_STEP);
    s.steps += s.sink_steps;
  }
  return s;
}

// MASKED: with sinks, or a tree of drafted tokens.
template <int HD, int NT, bool MASKED>
__global__ void __launch_bounds__(32 * AT_WARPS, NT == 1 ? 3 : 2) kv4_rows_kernel(const Kv4AttnArgs a, const Shares shares,
                                                                int row_tiles, int cluster) {
  constexpr int R = 8 * NT;              // query rows per tile
  constexpr int KS = HD / 16;            // channel steps of the first product = channel tiles of the second
  constexpr int KW = HD / 32;            // words of a token's key a thread holds
  constexpr int VW = HD / 64;            // words of a token's value a thread holds
  constexpr int HB = HD / 2;             // bytes a token
  __shared__ float sm_o[AT_WARPS][R][HD];
  __shared__ float sm_m[AT_WARPS][R], sm_l[AT_WARPS][R];

  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int group = a.heads_q / a.cache.heads;
  const int ps = a.cache.page_shift;
  // MASKED: an item may be cut over the blocks of a cluster, which join their results over its shared memory.
  const int rank = MASKED && cluster > 1 ? (int)ptx::cluster_ctarank() : 0;
  const float c_log2 = a.scale * kLog2e;
  // Shares: where each sequence's items begin on the line, and this block's part of it.
  __shared__ int64_t sm_first[AT_SEQS + 1];
  __shared__ int64_t sm_sum[AT_WARPS];
  __shared__ int64_t sm_share;
  // What a block remembers of an item while it walks the tokens; two, since a warp may be done with one before the others.
  struct Item { int64_t next; int b, kvh, rt, step0, step1, steps, q0, rows; };
  __shared__ Item sm_item[2];
  if (shares.blocks) {
    const int per = (a.B + 32 * AT_WARPS - 1) / (32 * AT_WARPS), b0 = threadIdx.x * per;
    auto length = [&](int b) {
      if (b >= a.B) return (int64_t)0;
      const Span s = span_of<MASKED>(a, b, false);
      return s.qlen <= 0 ? (int64_t)0 : (int64_t)(AT_LEAD + s.steps) * a.cache.heads * (((int64_t)s.qlen * group + R - 1) / R);
    };
    int64_t mine = 0;
    for (int k = 0; k < per; ++k) mine += length(b0 + k);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) sm_sum[warp] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < AT_WARPS; ++w) {
      if (w < warp) upto += sm_sum[w];
      total += sm_sum[w];
    }
    int64_t at = upto - mine;
    for (int k = 0; k < per; ++k)
      if (b0 + k < a.B) {
        sm_first[b0 + k] = at;
        if (per > 1) at += length(b0 + k);
      }
    if (threadIdx.x == 0) {
      sm_first[a.B] = total;
      shares.begun[blockIdx.x] = make_int4(-1, 0, 0, 0);
      sm_share = max((int64_t)AT_MIN_STEPS, (total + shares.blocks - 1) / shares.blocks);
      sm_item[1].next = sm_share * blockIdx.x;
    }
    __syncthreads();
  }

  for (int done = 0;; ++done) {
    // ---- the next item, or the share's part of one
    int b, kvh, rt, step0, step1;
    int64_t line = 0, end = 0;
    if (shares.blocks) {
      line = sm_item[(done & 1) ^ 1].next;
      end = min(sm_share * (blockIdx.x + 1), sm_first[a.B]);
      if (line >= end) break;
      int l = 0, h = a.B - 1;                            // the last sequence that begins at or before line
      while (l < h) {
        const int mid = (l + h + 1) / 2;
        if (sm_first[mid] <= line) l = mid; else h = mid - 1;
      }
      b = l;
    } else {
      b = blockIdx.z;
    }
    const Span sp = span_of<MASKED>(a, b, threadIdx.x == 0);
    const int qlen = sp.qlen, n = sp.n, rows = qlen * group;
    if (shares.blocks) {
      const int tiles = (rows + R - 1) / R, length = AT_LEAD + sp.steps;
      const int64_t off = line - sm_first[b];
      const int item = (int)(off / length);
      kvh = item / tiles;
      rt = item % tiles;
      const int from = (int)(off - (int64_t)item * length), to = (int)min((int64_t)length, from + (end - line));
      line += to - from;
      step0 = max(0, from - AT_LEAD);
      step1 = to - AT_LEAD;
      if (step1 <= 0) break;                             // the share ends in the lead: the next block begins the item
    } else {
      kvh = blockIdx.y;
      rt = (MASKED && cluster > 1 ? blockIdx.x / cluster : blockIdx.x) + done * row_tiles;
      if ((int64_t)rt * R >= rows) break;                // the whole cluster agrees
      step0 = 0;
      step1 = sp.steps;
      if (MASKED && cluster > 1) {
        const int per = (sp.steps + cluster - 1) / cluster;
        step0 = min(sp.steps, rank * per);
        step1 = min(sp.steps, step0 + per);
      }
    }
    if (threadIdx.x == 0) sm_item[done & 1] = Item{line, b, kvh, rt, step0, step1, sp.steps, sp.q0, rows};
    const int32_t* table = a.table + b * a.table_stride;
    const int r0 = rt * R;
    // positions of the tile's first and last row, and the tokens the tile sees
    int p_first = n - qlen + r0 / group, p_last = n - qlen + min(rows - 1, r0 + R - 1) / group;
    int lo = a.window > 0 ? max(0, p_first - a.window + 1) : 0;
    int hi = min(n, p_last + 1);
    const bool tree = MASKED && a.tree != nullptr;
    if (tree) lo = sp.lo, hi = n, p_first = n - qlen - 1, p_last = n - 1;   // every row sees up to p_first; none is behind p_last
    const int t_first = sp.lo / AT_STEP * AT_STEP;
    // MASKED walks steps, not tokens: those of the sinks, then those from t_first on.
    const int c_lo = MASKED ? step0 * AT_STEP : max(lo, t_first + step0 * AT_STEP);
    const int c_hi = MASKED ? step1 * AT_STEP : step1 == sp.steps ? hi : min(hi, t_first + step1 * AT_STEP);
    const int sink_end = sp.sink_steps * AT_STEP, gap = t_first - sink_end;
    auto token_of = [&](int at) { return MASKED ? at + (at >= sink_end ? gap : 0) : at; };

    // ---- query operands: B fragment of step (w, h): channels (d, d + 4), (d + 1, d + 5), d = 8 (KW t + w) + 2 h
    uint32_t qb[NT][KS][2];
    // For this thread's two columns: -8 * sum of the query (the codes' offset), and raw scores to log2 units, but for the
    // keys' scales.
    float bq[NT][2];
    uint64_t cq[NT];
    int pos[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + 8 * nt + g;
      uint32_t x[KW][4];
      if (r < rows) {
        const uint16_t* src = a.Q + (int64_t)(sp.q0 + r / group) * a.ldq + (kvh * group + r % group) * HD + 8 * KW * t;
#pragma unroll
        for (int w = 0; w < KW; ++w) load_words<4>(x[w], reinterpret_cast<const uint8_t*>(src + 8 * w));
      } else {
#pragma unroll
        for (int w = 0; w < KW; ++w) x[w][0] = x[w][1] = x[w][2] = x[w][3] = 0u;
      }
      float sum = 0.0f, mq = 0.0f;
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mq = ptx::max3(mq, finite_or_0(__uint_as_float(x[w][k] << 16)), finite_or_0(__uint_as_float(x[w][k] & 0xFFFF0000u)));
      mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, 1));
      mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, 2));
      const float eq = scale_exponent(mq), f = ex2(kQueryExp - eq);
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[2 * k] = __uint_as_float(x[w][k] << 16) * f;
          v[2 * k + 1] = __uint_as_float(x[w][k] & 0xFFFF0000u) * f;
          sum += v[2 * k] + v[2 * k + 1];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          qb[nt][2 * w + h][0] = pack_f16(v[2 * h], v[2 * h + 4]);
          qb[nt][2 * w + h][1] = pack_f16(v[2 * h + 1] * kOddNibble, v[2 * h + 5] * kOddNibble);
        }
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      float c2[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        bq[nt][e] = -8.0f * kCodeUnit * __shfl_sync(0xffffffffu, sum, 4 * (2 * t + e));
        c2[e] = c_log2 * ex2(__shfl_sync(0xffffffffu, eq, 4 * (2 * t + e)) + (24.0f - kQueryExp));
        pos[nt][e] = n - qlen + min(rows - 1, r0 + 8 * nt + 2 * t + e) / group;
        if (tree && a.window > 0) {
          const int row = pos[nt][e] - (n - qlen);
          pos[nt][e] = n - qlen + tree_depth(a.tree + (int64_t)(sp.q0 + row) * a.tree_words, a.tree_words, qlen);
        }
      }
      cq[nt] = ptx::f2_pack(c2[0], c2[1]);
    }

    float o[NT][KS][4];
    float m[NT][2], l[NT][2];            // reference exponent and sum
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int j = 0; j < KS; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.0f;
    }

    // ---- the warp's blocks of 32 tokens
    uint32_t kx[AT_TILES][2][KW], vx[AT_TILES][4][VW];
    float ks[AT_TILES][2], vs[AT_TILES][2];
    int lim[AT_TILES];                   // tokens of the 16-token tile that exist
    bool all;                            // every token of the block does
    uint32_t base[AT_TILES];             // cache row of the tile's first token (a cache has fewer than 2^32)
    const uint8_t* const kp = a.cache.k_codes + (HB * g + 4 * KW * t);   // this thread's part of a tile
    const uint8_t* const vp = a.cache.v_codes + (HB * 2 * t + 4 * VW * g);
    const float *const ksp = a.cache.k_scales + g, *const vsp = a.cache.v_scales + g;
    int page_of[AT_TILES];               // pages of the block to be located next: read a block ahead
    auto look_up = [&](int tok0) {
#pragma unroll
      for (int i = 0; i < AT_TILES; ++i) page_of[i] = tok0 + 16 * i < n ? __ldg(table + ((tok0 + 16 * i) >> ps)) : 0;
    };
    // Pieces in front of token `from` are not looked at: a window's older pages may be anyone's by now.
    auto locate = [&](int tok0, int from) {
      // MASKED: of the sinks and from lo on
      all = tok0 + AT_BLOCK <= n && (tok0 + 16 > from || (MASKED && tok0 + 16 < a.sinks));
#pragma unroll
      for (int i = 0; i < AT_TILES; ++i) {
        const int tok = tok0 + 16 * i;
        int k = tok + 16 > from || (MASKED && tok < a.sinks) ? min(16, n - tok) : 0;
        uint32_t at = 0;
        if (k > 0) {
          const int page = page_of[i];
          if (page < 0 || page >= a.cache.pages) {
            k = 0;
            all = false;
            if (lane == 0) atomicOr(a.status, PQ_DEV_BAD_INDEX);
          } else {
            at = (((uint32_t)page * (uint32_t)a.cache.heads + kvh) << ps) + (tok & ((1 << ps) - 1));
          }
        }
        lim[i] = k;
        base[i] = at;
      }
    };
    // Loads of a block whose tokens all exist carry no predicates.
    auto load_k = [&]() {
      if (all) {
#pragma unroll
        for (int i = 0; i < AT_TILES; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            load_words<KW>(kx[i][h], kp + (uint64_t)base[i] * HB + HB * 8 * h);
            ks[i][h] = __ldg(ksp + base[i] + 8 * h);
          }
      } else {
#pragma unroll
        for (int i = 0; i < AT_TILES; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool in = g + 8 * h < lim[i];
            // codes of a token that does not exist are never used: the cache's first bytes stand in
            load_words<KW>(kx[i][h], in ? kp + (uint64_t)base[i] * HB + HB * 8 * h : a.cache.k_codes);
            ks[i][h] = in ? __ldg(ksp + base[i] + 8 * h) : 0.0f;
          }
      }
    };
    auto load_v = [&](uint32_t (&vx)[AT_TILES][4][VW], float (&vs)[AT_TILES][2]) {
      if (all) {
#pragma unroll
        for (int i = 0; i < AT_TILES; ++i) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            load_words<VW>(vx[i][k], vp + (uint64_t)base[i] * HB + HB * ((k & 1) + 8 * (k >> 1)));
#pragma unroll
          for (int h = 0; h < 2; ++h) vs[i][h] = __ldg(vsp + base[i] + 8 * h);
        }
      } else {
#pragma unroll
        for (int i = 0; i < AT_TILES; ++i) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tok = (k & 1) + 8 * (k >> 1);
            const bool in = 2 * t + tok < lim[i];
            load_words<VW>(vx[i][k], in ? vp + (uint64_t)base[i] * HB + HB * tok : a.cache.v_codes);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) vs[i][h] = g + 8 * h < lim[i] ? __ldg(vsp + base[i] + 8 * h) : 0.0f;
        }
      }
    };

    const int first = (c_lo & ~(AT_BLOCK - 1)) + AT_BLOCK * warp;
    auto inside = [&](int at) { return at < c_hi && (!MASKED || token_of(at) < hi); };
    if (inside(first)) {
      look_up(token_of(first));
      locate(token_of(first), MASKED ? lo : c_lo);
      load_k();
      load_v(vx, vs);
      look_up(token_of(first + AT_BLOCK * AT_WARPS));
    }
    for (int at = first; inside(at); at += AT_BLOCK * AT_WARPS) {
      const int tok0 = token_of(at);
      const bool whole = MASKED ? all && tok0 + AT_BLOCK <= hi && tok0 + AT_BLOCK - 1 <= p_first &&
                                      (a.window <= 0 || tok0 > p_last - a.window || tok0 + AT_BLOCK <= a.sinks)
                                : all && tok0 >= c_lo && tok0 + AT_BLOCK <= c_hi && tok0 + AT_BLOCK - 1 <= p_first &&
                                      (a.window <= 0 || tok0 > p_last - a.window);
      float s[AT_TILES][NT][4];
#pragma unroll
      for (int i = 0; i < AT_TILES; ++i) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[i][nt][0] = s[i][nt][2] = bq[nt][0], s[i][nt][1] = s[i][nt][3] = bq[nt][1];
#pragma unroll
        for (int w = 0; w < KW; ++w)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x0 = kx[i][0][w] >> (8 * h), x1 = kx[i][1][w] >> (8 * h);
            const uint32_t a0 = and_xor(x0, 0x000F000Fu, 0x00080008u), a2 = and_xor(x0, 0x00F000F0u, 0x00800080u);
            const uint32_t a1 = and_xor(x1, 0x000F000Fu, 0x00080008u), a3 = and_xor(x1, 0x00F000F0u, 0x00800080u);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_f16(s[i][nt], a0, a1, a2, a3, qb[nt][2 * w + h][0], qb[nt][2 * w + h][1]);
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(s[i][nt][2 * h], s[i][nt][2 * h + 1]),
                                       ptx::f2_mul(ptx::f2_pack(ks[i][h], ks[i][h]), cq[nt])),
                           s[i][nt][2 * h], s[i][nt][2 * h + 1]);
      }
      if (MASKED && !whole) {
        // The tokens of the block that each of the thread's rows sees, a bit each: of the tokens in front of the new ones, and of
        // the new ones up to the row or by its list.
        const int old = n - qlen;
        uint32_t exist = 0u;
#pragma unroll
        for (int i = 0; i < AT_TILES; ++i) exist |= ((1u << max(0, lim[i])) - 1) << (16 * i);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int last = tree ? old - 1 : min(pos[nt][e], hi - 1);
            uint32_t sees = token_bits32(tok0, a.window > 0 ? max(0, pos[nt][e] - a.window + 1) : 0, last) |
                            token_bits32(tok0, 0, min(a.sinks - 1, last));
            if (tree && tok0 + AT_BLOCK > old) {
              const int row = min(rows - 1, r0 + 8 * nt + 2 * t + e) / group;
              const uint32_t mine = (uint32_t)tree_bits(a.tree + (int64_t)(sp.q0 + row) * a.tree_words, a.tree_words, tok0 - old);
              sees |= tok0 >= old ? mine : mine & (~0u << (old - tok0));
            }
            sees = (sees & exist) >> g;
#pragma unroll
            for (int i = 0; i < AT_TILES; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                if (!((sees >> (16 * i + 8 * h)) & 1u)) s[i][nt][2 * h + e] = -INFINITY;
          }
      }
      if (!MASKED && !whole) {
#pragma unroll
        for (int i = 0; i < AT_TILES; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int tok = tok0 + 16 * i + 8 * h + g;
            const bool in = 8 * h + g < lim[i] && tok >= c_lo && tok < c_hi;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!(in && tok <= pos[nt][e] && (a.window <= 0 || tok > pos[nt][e] - a.window)))
                  s[i][nt][2 * h + e] = -INFINITY;
          }
      }
      // the next block's keys and values
      const int next = at + AT_BLOCK * AT_WARPS;
      uint32_t vn[AT_TILES][4][VW];
      float vsn[AT_TILES][2];
      if (inside(next)) {
        locate(token_of(next), MASKED ? lo : next);
        load_k();
        load_v(vn, vsn);
        look_up(token_of(next + AT_BLOCK * AT_WARPS));
      }
      uint32_t pb[AT_TILES][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        bool over = m[nt][0] == -INFINITY || m[nt][1] == -INFINITY;
        float sum[2];
        for (int pass = 0;; ++pass) {
          if (__any_sync(0xffffffffu, over)) {
            // Raise the references of the rows that need it (not of their neighbours in the tile, whose results must not
            // depend on them) to this block's largest score plus exponent of the value scale, over the tokens that the row
            // sees: their largest product is then 1/2 to 1.
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = -INFINITY, most = 0.0f;
              const float ref = m[nt][e] == -INFINITY ? 0.0f : m[nt][e];
#pragma unroll
              for (int i = 0; i < AT_TILES; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float z = s[i][nt][2 * h + e];
                  if (z != -INFINITY) {
                    const float p = ex2(z - ref);
                    x = fmaxf(x, z + value_exponent(vs[i][h]));
                    most = ptx::max3(most, fabsf(p * vs[i][h]), p * (kRowsTop / kSumTop * (4 * AT_BLOCK)));
                  }
                }
#pragma unroll
              for (int b = 4; b < 32; b <<= 1) {
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, b));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, b));
              }
              x = m[nt][e] == -INFINITY || most > kRowsTop ? fmaxf(m[nt][e], x) : m[nt][e];
              alpha[e] = x == -INFINITY ? 1.0f : ex2(m[nt][e] - x);
              m[nt][e] = x;
            }
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              o[nt][j][0] *= alpha[0];
              o[nt][j][1] *= alpha[1];
              o[nt][j][2] *= alpha[0];
              o[nt][j][3] *= alpha[1];
            }
            l[nt][0] *= alpha[0];
            l[nt][1] *= alpha[1];
          }
          const float r0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0], r1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
          sum[0] = sum[1] = 0.0f;
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < AT_TILES; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float s0 = s[i][nt][2 * h], s1 = s[i][nt][2 * h + 1];
              const float p0 = ex2(s0 - r0), p1 = ex2(s1 - r1);
              sum[0] += p0;
              sum[1] += p1;
              // a hidden token's value scale may be anything: select, do not multiply
              const float w0 = whole || s0 != -INFINITY ? p0 * vs[i][h] : 0.0f;
              const float w1 = whole || s1 != -INFINITY ? p1 * vs[i][h] : 0.0f;
              top = ptx::max3(top, fabsf(w0), fabsf(w1));
              pb[i][nt][h] = pack_f16(w0, w1);
            }
          over = top > kRowsTop || fmaxf(sum[0], sum[1]) > kSumTop;
          if (pass == 1 || !__any_sync(0xffffffffu, over)) break;
        }
        l[nt][0] += sum[0];
        l[nt][1] += sum[1];
#pragma unroll
        for (int i = 0; i < AT_TILES; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) pb[i][nt][h] = movmatrix_trans(pb[i][nt][h]);
      }
#pragma unroll
      for (int i = 0; i < AT_TILES; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // words of tokens 2t and 2t + 1 (and + 8), their low or high 16 bits side by side
          uint32_t y[VW][2][4];
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            code_pairs(__byte_perm(vx[i][0][w], vx[i][1][w], half ? 0x7632 : 0x5410), y[w][0]);
            code_pairs(__byte_perm(vx[i][2][w], vx[i][3][w], half ? 0x7632 : 0x5410), y[w][1]);
          }
          if constexpr (VW == 2) {
            // channel tile j: rows g <-> channel 16 g + j, rows g + 8 <-> 16 g + 8 + j
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j = 4 * half + k;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o[nt][j], y[0][0][k], y[1][0][k], y[0][1][k], y[1][1][k], pb[i][nt][0], pb[i][nt][1]);
            }
          } else {
            // channel tile j: rows g <-> channel 8 g + 2 j, rows g + 8 <-> 8 g + 2 j + 1
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int j = 2 * half + k;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o[nt][j], y[0][0][2 * k], y[0][0][2 * k + 1], y[0][1][2 * k], y[0][1][2 * k + 1], pb[i][nt][0], pb[i][nt][1]);
            }
          }
        }
#pragma unroll
      for (int i = 0; i < AT_TILES; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int w = 0; w < VW; ++w) vx[i][k][w] = vn[i][k][w];
        vs[i][0] = vsn[i][0], vs[i][1] = vsn[i][1];
      }
    }

    // ---- join the block's warps
    __syncthreads();                     // the previous row tile's reads are done
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const int r = 8 * nt + 2 * t + e;
        if (g == 0) {
          sm_m[warp][r] = m[nt][e];
          sm_l[warp][r] = x;
        }
        // odd nibbles' channels come 16 times too large
        if constexpr (VW == 2) {
#pragma unroll
          for (int j = 1; j < KS; j += 2) {
            o[nt][j][e] *= kOddNibble;
            o[nt][j][2 + e] *= kOddNibble;
          }
        } else {
#pragma unroll
          for (int j = 0; j < KS; ++j) o[nt][j][2 + e] *= kOddNibble;
        }
        float* dst = &sm_o[warp][r][(HD / 8) * g];
        if constexpr (VW == 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 8; j += 4)
              *reinterpret_cast<float4*>(dst + 8 * h + j) =
                  make_float4(o[nt][j][2 * h + e], o[nt][j + 1][2 * h + e], o[nt][j + 2][2 * h + e], o[nt][j + 3][2 * h + e]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; j += 2)
            *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(o[nt][j][e], o[nt][j][2 + e], o[nt][j + 1][e], o[nt][j + 1][2 + e]);
        }
      }
    __syncthreads();
    const Item& it = sm_item[done & 1];
    const bool entire = it.step0 == 0 && it.step1 == it.steps;
    for (int r = warp; r < R && it.rt * R + r < it.rows; r += AT_WARPS) {
      constexpr int E = HD / 32;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) mx = fmaxf(mx, sm_m[w][r]);
      const float mu = mx == -INFINITY ? 0.0f : mx;
      float sum = 0.0f, y[E];
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) {
        const float f = ex2(sm_m[w][r] - mu);
        sum = fmaf(sm_l[w][r], f, sum);
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = fmaf(sm_o[w][r][E * lane + i], f, y[i]);
      }
      const int at = it.rt * R + r;
      const int64_t token = it.q0 + at / group;
      const int head = it.kvh * group + at % group;
      if (MASKED && cluster > 1) {                       // the block's result, in place of its first warp's
        __syncwarp();
#pragma unroll
        for (int i = 0; i < E; ++i) sm_o[0][r][E * lane + i] = y[i];
        if (lane == 0) sm_m[0][r] = mx, sm_l[0][r] = sum;
      } else if (entire) {
        finish_row<HD>(y, sum, a.cache.rotate_v, a.O + token * a.ldo + head * HD, lane);
      } else {
        const int64_t row = (int64_t)(2 * blockIdx.x + (it.step0 == 0)) * R + r;
        if (lane == 0) shares.ml[row] = make_float2(mx, sum);
        if (mx != -INFINITY || sum != 0.0f) {
#pragma unroll
          for (int i = 0; i < E; ++i) shares.o[row * HD + E * lane + i] = y[i];
        }
      }
    }
    if (MASKED && cluster > 1) {
      ptx::cluster_sync();                               // every block's rows are in its shared memory
      constexpr int E = HD / 32;
      for (int r = rank + cluster * warp; r < R && it.rt * R + r < it.rows; r += cluster * AT_WARPS) {
        const uint32_t m_at = ptx::smem_addr(&sm_m[0][r]), l_at = ptx::smem_addr(&sm_l[0][r]), o_at = ptx::smem_addr(&sm_o[0][r][E * lane]);
        float mb = -INFINITY, lb = 0.0f;                 // a block a lane
        if (lane < cluster) {
          mb = ptx::ld_cluster_f32(ptx::mapa_shared(m_at, (uint32_t)lane));
          lb = ptx::ld_cluster_f32(ptx::mapa_shared(l_at, (uint32_t)lane));
        }
        float v[KV4_CLUSTER][E];
#pragma unroll
        for (int c = 0; c < KV4_CLUSTER; ++c) ptx::ld_cluster<E>(v[c], ptx::mapa_shared(o_at, (uint32_t)min(c, cluster - 1)));
        float mx = mb;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mu = mx == -INFINITY ? 0.0f : mx;
        // a block that saw nothing counts for nothing; one whose scores are all NaN keeps its NaN
        const float f = mb == -INFINITY ? (lb == 0.0f ? 0.0f : 1.0f) : ex2(mb - mu);
        float sum = 0.0f, y[E];
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = 0.0f;
#pragma unroll
        for (int c = 0; c < KV4_CLUSTER; ++c) {
          if (c >= cluster) break;
          const float fc = __shfl_sync(0xffffffffu, f, c);
          sum = fmaf(__shfl_sync(0xffffffffu, lb, c), fc, sum);
#pragma unroll
          for (int i = 0; i < E; ++i) y[i] = fmaf(v[c][i], fc, y[i]);
        }
        const int at = it.rt * R + r;
        finish_row<HD>(y, sum, a.cache.rotate_v, a.O + (it.q0 + at / group) * a.ldo + (it.kvh * group + at % group) * HD, lane);
      }
      ptx::cluster_sync();                               // nobody leaves, or goes on, while its rows are read
    }
    if (threadIdx.x == 0 && it.step0 == 0 && !entire && !(MASKED && cluster > 1))
      shares.begun[blockIdx.x] = make_int4(it.b, it.kvh, it.rt, (int)((it.next + (it.steps - it.step1) - 1) / sm_share));
  }
}

// Joins a query row's partial results: a warp does (parts = 1), or a block, whose warps take every eighth piece each and
// the first joins theirs.  at(k): piece k's row in ml_of and o_of.
constexpr int JN_WARPS = 8;
template <int HD, int parts, typename At>
__device__ __forceinline__ void join_row(const float2* ml_of, const float* o_of, int pieces, At at, int rotate, uint16_t* dst) {
  __shared__ float sm_o[JN_WARPS * HD];
  __shared__ float2 sm_ml[JN_WARPS];
  const int part = parts == 1 ? 0 : threadIdx.x >> 5;
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  float mx = -INFINITY;
  for (int c = part + parts * lane; c < pieces; c += 32 * parts) mx = fmaxf(mx, ml_of[at(c)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float mu = mx == -INFINITY ? 0.0f : mx;
  float sum = 0.0f, y[E];
#pragma unroll
  for (int i = 0; i < E; ++i) y[i] = 0.0f;
  for (int c0 = part; c0 < pieces; c0 += 32 * parts) {   // 32 pieces a turn: a lane takes each one's factor
    const int mine = c0 + parts * lane;
    float f = -1.0f;                                     // nothing seen and no output written: not to be read
    if (mine < pieces) {
      const float2 ml = ml_of[at(mine)];
      if (ml.x != -INFINITY || ml.y != 0.0f) {
        f = ex2(ml.x - mu);
        sum = fmaf(ml.y, f, sum);
      }
    }
    const int turn = min(32, (pieces - c0 + parts - 1) / parts);
#pragma unroll 8
    for (int k = 0; k < turn; ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k);
      float x[E];
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = o_of[at(c0 + parts * k) * HD + E * lane + i];
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = fk != -1.0f ? fmaf(x[i], fk, y[i]) : y[i];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if constexpr (parts == 1) {
    finish_row<HD>(y, sum, rotate, dst, lane);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) sm_o[part * HD + E * lane + i] = y[i];
    if (lane == 0) sm_ml[part] = make_float2(mx, sum);
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int w = 1; w < parts; ++w) mx = fmaxf(mx, sm_ml[w].x);
      const float all = mx == -INFINITY ? 0.0f : mx;
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < E; ++i) y[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < parts; ++w) {
        const float2 ml = sm_ml[w];
        const float f = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : ex2(ml.x - all);
        sum = fmaf(ml.y, f, sum);
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = fmaf(sm_o[w * HD + E * lane + i], f, y[i]);
      }
      finish_row<HD>(y, sum, rotate, dst, lane);
    }
  }
}

// The chunks of the prompt kernel, a warp or a block a row.  Rows of tokens outside every sequence stay as they were.  Both
// joining kernels are launched as programmatic dependents of the kernel that writes the pieces.
template <int HD>
__global__ void __launch_bounds__(32 * JN_WARPS) kv4_join_kernel(const Kv4AttnArgs a, const Partials part, int warp_a_row) {
  const int64_t total = a.T * a.heads_q;
  const int64_t row = warp_a_row ? (int64_t)blockIdx.x * JN_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  const int64_t token = row / a.heads_q;
  ptx::griddep_wait();
  if (token < a.q_start[0] || token >= min((int64_t)a.q_start[a.B], a.T)) return;   // the whole block, or warp
  if ((a.tree || a.sinks > 0) && part.ml[row].y == kRowDone) return;
  auto at = [&](int k) { return k * total + row; };
  uint16_t* dst = a.O + token * a.ldo + (row - token * a.heads_q) * HD;
  if (warp_a_row) join_row<HD, 1>(part.ml, part.o, part.chunks, at, a.cache.rotate_v, dst);
  else join_row<HD, JN_WARPS>(part.ml, part.o, part.chunks, at, a.cache.rotate_v, dst);
}

// The shares: blocks (x, y) look at `per` blocks' slots from x per on, for items that begin in one and go on in the next
// ones.  Few items have many pieces: a block a row (y, y + gridDim.y ..); many have few: a warp a row.
template <int HD, int R>
__global__ void __launch_bounds__(32 * JN_WARPS) kv4_join_shares_kernel(const Kv4AttnArgs a, const Shares shares, int per,
                                                                        int warp_a_row) {
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, group = a.heads_q / a.cache.heads;
  const int first = blockIdx.x * per, last = min(first + per, shares.blocks);
  for (int c0 = first; c0 < last; c0 += 32) {
    const int mine = c0 + lane;
    uint32_t begun = __ballot_sync(0xffffffffu, mine < last && shares.begun[min(mine, last - 1)].x >= 0);
    for (; begun; begun &= begun - 1) {
      const int c = c0 + __ffs(begun) - 1;
      const int4 item = shares.begun[c];                 // sequence, head, row tile, last block
      const Span sp = span_of<false>(a, item.x, false);   // where its rows are
      const int rows = min(R, sp.qlen * group - item.z * R), pieces = item.w - c + 1;
      auto join = [&](int r, auto parts) {
        const int at = item.z * R + r;
        const int64_t token = sp.q0 + at / group;
        const int head = item.y * group + at % group;
        join_row<HD, decltype(parts)::value>(shares.ml, shares.o, pieces,
                                             [&](int k) { return (int64_t)(2 * (c + k) + (k == 0)) * R + r; },
                                             a.cache.rotate_v, a.O + token * a.ldo + head * HD);
      };
      if (warp_a_row) {
        for (int r = blockIdx.y * JN_WARPS + (threadIdx.x >> 5); r < rows; r += gridDim.y * JN_WARPS)
          join(r, std::integral_constant<int, 1>());
      } else {
        for (int r = blockIdx.y; r < rows; r += gridDim.y) {
          join(r, std::integral_constant<int, JN_WARPS>());
          __syncthreads();
        }
      }
    }
  }
}

cudaError_t launch_join(const void* kernel, dim3 grid, void** args, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * JN_WARPS, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

template <int HD, int NT>
cudaError_t launch_rows(const Kv4AttnArgs& a, const Shares& shares, int row_tiles, int64_t max_rows, int cluster,
                        cudaStream_t stream) {
  const dim3 grid = shares.blocks ? dim3((unsigned)shares.blocks)
                                  : dim3((unsigned)(row_tiles * cluster), (unsigned)a.cache.heads, (unsigned)a.B);
  if (cluster > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(32 * AT_WARPS, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_rows_kernel<HD, NT, true>, a, shares, row_tiles, cluster);
  }
  if (kv4_masked(a)) kv4_rows_kernel<HD, NT, true><<<grid, 32 * AT_WARPS, 0, stream>>>(a, shares, row_tiles, 1);
  else kv4_rows_kernel<HD, NT, false><<<grid, 32 * AT_WARPS, 0, stream>>>(a, shares, row_tiles, 1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !shares.blocks) return e;
  // Joining blocks: a few for each item, if those are fewer than shares.
  const int64_t items = std::max<int64_t>(1, std::min<int64_t>(4 * (int64_t)a.B * a.cache.heads * row_tiles, shares.blocks));
  const int64_t rows = std::max<int64_t>(1, std::min<int64_t>(max_rows, 8 * NT));
  int per = (int)((shares.blocks + items - 1) / items), warp_a_row = items == shares.blocks;
  void* args[] = {const_cast<Kv4AttnArgs*>(&a), const_cast<Shares*>(&shares), &per, &warp_a_row};
  return launch_join(reinterpret_cast<const void*>(kv4_join_shares_kernel<HD, 8 * NT>),
                     dim3((unsigned)((shares.blocks + per - 1) / per), (unsigned)(warp_a_row ? (rows + JN_WARPS - 1) / JN_WARPS : rows)),
                     args, stream);
}

}  // namespace

// The rules for masked calls below were found on 8 key/value heads of 128.  Tried with and without each on these, on 8 heads of 64 and
// on 4, 2 (of 128 and 64) and 1, 750 calls in all: none costs 5% but the uncut windows of 2048 on places that are half to two thirds full (there).
pq_status kv4_attention_run(const Kv4AttnArgs& a, int64_t max_q, int64_t max_len, cudaStream_t stream) {
  // What a masked call walks of a sequence: its window and its sinks, in steps of 128.
  if (kv4_masked(a) && a.window > 0) max_len = std::min<int64_t>(max_len, (int64_t)a.window + max_q + a.sinks + 256);
  const int group = a.heads_q / a.cache.heads;
  const int64_t max_rows = max_q * group;
  const int sms = device_sm_count();
  const int64_t walk = (max_len + AT_STEP - 1) / AT_STEP;
  // Masked calls that leave blocks idle.  (1) They keep to tiles of 8 rows, whose blocks are quicker (us, 8 against 16; 8 key/value
  // heads of 128, 32 rows each).  One sequence over 1029 tokens 11.4 : 14.9, 8100 19.5 : 20.2; two over 2048 14.2 : 16.2, 4300
  // 23.3 : 20.6; four over 1029 14.9 : 17.2, 2048 19.2 : 19.2, 3000 25.6 : 22.1; 16 over 130 17.2 : 12.7.
  const int64_t eights = a.B * a.cache.heads * ((max_rows + 7) / 8);
  const bool narrow = kv4_masked(a) && 2 * eights <= 3 * sms && eights * walk <= 2048;
  // (2) They stay here with more rows, a step of 128 tokens an SM for each of 8 tiles (us, this against the prompts' kernel; 8 heads).
  // One sequence over 300 tokens, 128 rows 9.2 : 14.6; 1029, 64 rows 12.4 : 14.1, 128 rows 14.7 : 15.4; 2048, 64 rows 14.0 :
  // 14.4, 80 rows 15.6 : 14.6; 8192, 36 rows 23.6 : 21.9.  Two over 1029, 64 rows 14.7 : 15.9, 80 rows 17.1 : 16.7.  Four over
  // 300, 64 rows 12.5 : 15.2; 1029, 64 rows 19.0 : 18.8.  Eight over 300, 48 rows 13.9 : 15.4, 80 rows 24.9 : 15.9.
  const bool stay = kv4_masked(a) && max_rows <= 128 && eights <= 3 * sms && eights * walk <= 8 * sms;
  const bool prompt = max_rows > kPromptRows && !stay;
  const int nt = max_rows > 8 && !narrow ? 2 : 1;
  const bool wide = a.cache.head_dim == 128;
  // Float32 workspace for partial results: [rows][head_dim] outputs, [rows] references and sums, then `extra` bytes.
  void* ws = nullptr;
  auto workspace = [&](size_t rows, size_t extra, float** o, float2** ml) {
    const size_t bytes = rows * (a.cache.head_dim * sizeof(float) + sizeof(float2)) + extra;
    cudaMemPool_t pool = nullptr;
    // A device's first call makes the pool, which a thread that captures may do in relaxed mode only (it is no work on a stream).
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return cuda_fail(e, "capture mode");
    e = scratch_pool(&pool);
    const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return cuda_fail(e, "scratch memory pool");
    if (back != cudaSuccess) return cuda_fail(back, "capture mode");
    e = cudaMallocFromPoolAsync(&ws, bytes, pool, stream);
    if (e != cudaSuccess) {
      set_error("cudaMallocFromPoolAsync(%zu bytes of attention workspace): %s", bytes, cudaGetErrorString(e));
      return PQ_ERR_ALLOC;
    }
    *o = static_cast<float*>(ws);
    *ml = reinterpret_cast<float2*>(*o + rows * a.cache.head_dim);
    return PQ_OK;
  };
  pq_status st = PQ_OK;
  if (prompt) {
    // One block an SM: chunks only where the tiles (of 256 rows; a sequence's last one half full on average) leave SMs idle,
    // at least two steps of 128 tokens each (400 rows over 1500 tokens: 31 us; 35 with four, 42 uncut; 64 rows over 8192: 32
    // with four or fewer, 39 with eight).
    int64_t tiles = a.B == 1 ? kv4_prompt_tiles(a) : std::max<int64_t>((a.T * group + 128 * (int64_t)a.B) / 256, 1);
    // Sequences of up to 256 rows have a tile each.  (Masked calls alone: the others' parts, and so their bits, stay.)
    if (kv4_masked(a) && max_rows <= 256) tiles = a.B;
    const int64_t want = sms / (tiles * a.cache.heads);
    Partials part = {};
    part.sms = sms;
    part.chunks = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, (max_len + 255) / 256), 256));
    if (kv4_masked(a)) {
      // A masked walk is cut into equal parts by its own length (us on the device, uncut and by the number of parts at most).
      // Of several sequences the longest keeps one SM busy: 16 of 0 to 8192 tokens, 61 drafts on 32 + 8 heads of 128: 168; 2
      // parts 137, 3 112, 4 111, 6 127, 8 140 in the sequences' order, longest first 2 107, 3 96, 5 109.  Not where the walks are short:
      // chunks of up to 801 under a window of 700: 29; 34, 33, 39.  Short walks of few tiles go down to a step a part: 5 sequences under a window of 512, 25 drafts: 23; 4 parts
      // 17.1, 8 14.7.
      const int64_t steps = (max_len + 127) / 128, share = std::max<int64_t>(16, tiles * a.cache.heads * steps / (2 * sms));
      if (a.B > 1 && steps >= 32) part.chunks = std::max<int>(part.chunks, (int)std::min<int64_t>((steps + share - 1) / share, 16));
      if (steps <= 8) part.chunks = (int)std::max<int64_t>(1, std::min<int64_t>(want, steps));
      // Few tiles: the chunks of a tile as a cluster, which joins them over its shared memory, where all clusters run at once (a
      // GPC holds two of eight) and a block has no more than 28 rows to join (us, cluster against two kernels; 8 key/value heads
      // of 128).  64 rows over 400 tokens 15.7 : 19.4, 2048 15.5 : 21.7; 128 over 2048 20.4 : 21.4; 256 over 1029 20.5 : 20.4; 256
      // over 400, in two, 26.7 : 17.8.  The host saves 4 us of a second launch and the workspace.
      const int64_t items = tiles * a.cache.heads;
      const int64_t c = std::min<int64_t>(std::min<int64_t>(2 * items <= sms ? std::max<int64_t>(3 * sms / 4 / items, 2) : 1, steps), KV4_CLUSTER);
      const int64_t rows = std::min<int64_t>(max_rows, 256);
      if (c > 1 && (rows <= 28 * c || c == KV4_CLUSTER) && (steps + c - 1) / c <= (steps + part.chunks - 1) / part.chunks + 2)
        part.chunks = (int)c, part.cluster = 1;
      else if (steps - (steps + part.chunks - 1) / part.chunks < 2)
        part.chunks = 1;                                 // a step saved pays for no second kernel: 8 sequences over 300, uncut 15.9 : 17.2
    }
    if (!part.cluster && a.T * a.heads_q >= ((int64_t)1 << 31)) part.chunks = 1;  // the joining kernel takes a block a row
    part.chunk_len = (int)(((max_len + part.chunks - 1) / part.chunks + 127) / 128 * 128);
    if (part.chunks > 1 && !part.cluster) st = workspace((size_t)part.chunks * a.T * a.heads_q, 0, &part.o, &part.ml);
    if (st == PQ_OK) st = launch_kv4_prompt(a, part, stream);
    if (st == PQ_OK && part.chunks > 1 && !part.cluster) {
      int warp_a_row = part.chunks < 2 * JN_WARPS;
      const int64_t rows = a.T * a.heads_q;
      void* args[] = {const_cast<Kv4AttnArgs*>(&a), &part, &warp_a_row};
      st = cuda_fail(launch_join(wide ? reinterpret_cast<const void*>(kv4_join_kernel<128>) : reinterpret_cast<const void*>(kv4_join_kernel<64>),
                                 dim3((unsigned)(warp_a_row ? (rows + JN_WARPS - 1) / JN_WARPS : rows)), args, stream),
                     "kv4_join_kernel launch");
    }
  } else {
    // Up to 640 tokens one block an item, otherwise as many shares as blocks run at once: a second kernel and its workspace
    // cost more than shares of short sequences save (us on the device, one block against shares; 8 key/value heads of 128).
    // One sequence: 512 tokens 8.8 : 14.8, 1024 12.3 : 13.8, 1536 15.7 : 12.4, 2048 19.4 : 12.5.  64 of up to: 512 tokens
    // 15.3 : 21.0, 1024 24.5 : 27.1, 2048 35.5 : 35.2.  (Call by call the host adds 1 to 2 us to the shares.)
    // The sides meet between 1000 and 2000 tokens, so calls from 641 to there take up to 5 us longer than they need.
    const int row_tiles = (int)std::min<int64_t>((max_rows + 8 * nt - 1) / (8 * nt), 4096);
    Shares shares = {};
    // Masked calls of few items cut each over a cluster, whose blocks join over its shared memory, as long as all run at once:
    // no second kernel, no workspace (us, cluster against uncut or shares; 8 key/value heads of 128, one sequence, 8 rows each).
    // 260 tokens 9.0 : 8.5, 400 8.3 : 9.6, 1029 9.0 : 13.9, 3000 10.7 : 12.8, 4300 12.2 : 12.5, 6000 13.3 : 12.9.  Equal shares
    // use blocks that a cluster leaves idle: worth it from about 4 steps a block that they save.
    int cluster = 1;
    if (kv4_masked(a) && walk >= 4) {
      const int64_t items = (int64_t)a.B * a.cache.heads * row_tiles, fit = (nt == 1 ? 3 : 2) * (int64_t)sms;
      // Clusters of 4 and 8 fill no GPC: 7/8 of the places hold them (51 clusters of 8, in two waves, 23.0; 48: 14.2).
      while (cluster < KV4_CLUSTER && 2 * cluster <= walk && items * cluster * 2 <= (cluster == 1 ? fit : fit * 7 / 8)) cluster *= 2;
      if (walk > 8 * cluster || walk * (fit - items * cluster) > 4 * cluster * fit) cluster = 1;
    }
    // Under a window walks differ little: a block an item, as long as all run at once and none is long (us, uncut against shares;
    // 8 key/value heads, windows of 512, 1024, 2048 and 4096).  32 sequences 14.8 : 20.2, 20.9 : 25.5, 35.7 : 35.9, 61.9 : 54.4; 48 of
    // them 17.7 : 24.1, 26.0 : 32.5, 42.3 : 47.4, 71.9 : 73.2; 64, more than run at once, 29.9 : 30.4, 45.1 : 39.2, 71.4 : 59.0.
    // 16, which leave places empty, under 2048 23.6 : 21.3.
    const bool uncut = kv4_masked(a) && a.window > 0 && walk <= 20 &&
                       (int64_t)a.B * a.cache.heads * row_tiles <= (nt == 1 ? 3 : 2) * (int64_t)sms;
    if (cluster == 1 && !uncut && max_len > 640 && a.B <= AT_SEQS) {
      shares.blocks = (nt == 1 ? 3 : 2) * sms;
      const size_t rows = (size_t)shares.blocks * 2 * 8 * nt;
      st = workspace(rows, shares.blocks * sizeof(int4), &shares.o, &shares.ml);
      shares.begun = reinterpret_cast<int4*>(shares.ml + rows);
    }
    if (st == PQ_OK)
      st = cuda_fail(wide ? (nt == 1 ? launch_rows<128, 1>(a, shares, row_tiles, max_rows, cluster, stream) : launch_rows<128, 2>(a, shares, row_tiles, max_rows, cluster, stream))
                          : (nt == 1 ? launch_rows<64, 1>(a, shares, row_tiles, max_rows, cluster, stream) : launch_rows<64, 2>(a, shares, row_tiles, max_rows, cluster, stream)),
                     "kv4_rows_kernel launch");
  }
  if (ws) {
    const cudaError_t e = cudaFreeAsync(ws, stream);
    if (st == PQ_OK && e != cudaSuccess) return cuda_fail(e, "cudaFreeAsync(attention workspace)");
  }
  return st;
}

}  // namespace pq
