// Argument checks and dispatch of the 8-bit product and of the 4-bit key/value cache.
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "kv4.h"

using namespace pq;

namespace {

constexpr int64_t kMaxD8 = 65536;               // 2^7 * 2^7 * D stays below 2^31
constexpr int64_t kMaxRows = (int64_t)1 << 24;  // rows of one call (keeps every grid within its limits)
constexpr int64_t kMaxTokens = (int64_t)1 << 30;  // tokens of a sequence (positions, and sums of two, stay within int32)

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

pq_status check_quant8(const void* X, int64_t T, int64_t D, int64_t ldx, int g, const int8_t* codes,
                       const float* scales) {
  if (!X || !codes || !scales) { set_error("X, codes and scales must be non-NULL"); return PQ_ERR_INVALID_ARG; }
  if (g != 0 && g != 64 && g != 128 && g != 256) {
    set_error("g=%d: rows are rotated in blocks of 64, 128 or 256 (or not, g = 0)", g);
    return PQ_ERR_UNSUPPORTED;
  }
  if (T < 1 || T > kMaxRows) { set_error("T=%lld must be in 1..2^24", (long long)T); return PQ_ERR_INVALID_ARG; }
  if (D < 16 || D > kMaxD8 || D % 16 != 0 || (g && D % g != 0)) {
    set_error("D=%lld must be in 16..65536, a multiple of 16 and of g=%d", (long long)D, g);
    return PQ_ERR_INVALID_ARG;
  }
  if (ldx < D || ldx % 8 != 0) {
    set_error("ldx=%lld must be >= D=%lld and a multiple of 8", (long long)ldx, (long long)D);
    return PQ_ERR_INVALID_ARG;
  }
  if (!aligned16(X) || !aligned16(codes) || !aligned16(scales)) {
    set_error("device pointers must be 16-byte aligned");
    return PQ_ERR_INVALID_ARG;
  }
  return PQ_OK;
}

pq_status check_gemm8(const int8_t* codes_A, const float* scales_A, const int8_t* codes_W, const float* scales_W,
                      int64_t T, int64_t N, int64_t D, const void* Y, pq_out_dtype out_dtype) {
  if (!codes_A || !scales_A || !codes_W || !scales_W || !Y) {
    set_error("all tensor pointers must be non-NULL");
    return PQ_ERR_INVALID_ARG;
  }
  if (T < 1 || N < 1 || T > kMaxRows || N > kMaxRows) {
    set_error("T=%lld and N=%lld must be in 1..2^24", (long long)T, (long long)N);
    return PQ_ERR_INVALID_ARG;
  }
  if (D < 16 || D > kMaxD8 || D % 16 != 0) {
    set_error("D=%lld must be in 16..65536 and a multiple of 16", (long long)D);
    return PQ_ERR_INVALID_ARG;
  }
  if (out_dtype != PQ_OUT_F32 && out_dtype != PQ_OUT_BF16) { set_error("bad out_dtype"); return PQ_ERR_INVALID_ARG; }
  if (!aligned16(codes_A) || !aligned16(scales_A) || !aligned16(codes_W) || !aligned16(scales_W) || !aligned16(Y)) {
    set_error("device pointers must be 16-byte aligned");
    return PQ_ERR_INVALID_ARG;
  }
  return PQ_OK;
}

pq_status check_cache(const pq_kv4_cache* c, Kv4View* v) {
  if (!c) { set_error("cache is NULL"); return PQ_ERR_INVALID_ARG; }
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) {
    set_error("the cache's four buffers must be non-NULL");
    return PQ_ERR_INVALID_ARG;
  }
  if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales)) {
    set_error("the cache's buffers must be 16-byte aligned");
    return PQ_ERR_INVALID_ARG;
  }
  if (c->head_dim != 64 && c->head_dim != 128) {
    set_error("head_dim=%d: the cache holds heads of 64 or 128", c->head_dim);
    return PQ_ERR_UNSUPPORTED;
  }
  int shift = 4;
  while (shift <= 8 && (1 << shift) != c->page_size) ++shift;
  if (shift > 8) {
    set_error("page_size=%d must be 16, 32, 64, 128 or 256", c->page_size);
    return PQ_ERR_UNSUPPORTED;
  }
  if (c->heads < 1 || c->heads > 1024) { set_error("heads=%d must be in 1..1024", c->heads); return PQ_ERR_INVALID_ARG; }
  if (c->pages < 1 || c->pages >= ((int64_t)1 << 31)) {
    set_error("pages=%lld must be in 1..2^31-1", (long long)c->pages);
    return PQ_ERR_INVALID_ARG;
  }
  if (c->pages * c->heads >= ((int64_t)1 << 32) / c->page_size) {
    set_error("pages * heads * page_size must be below 2^32");
    return PQ_ERR_INVALID_ARG;
  }
  if (c->flags & ~(PQ_KV4_ROTATE_K | PQ_KV4_ROTATE_V)) { set_error("unknown cache flags 0x%x", c->flags); return PQ_ERR_INVALID_ARG; }
  *v = Kv4View{c->k_codes, c->k_scales, c->v_codes, c->v_scales, c->pages, shift, c->heads, c->head_dim,
               (c->flags & PQ_KV4_ROTATE_K) ? 1 : 0, (c->flags & PQ_KV4_ROTATE_V) ? 1 : 0};
  return PQ_OK;
}

pq_status check_heads(int heads_q, int heads) {
  if (heads_q < 1 || heads_q > 4096 || heads_q % heads != 0) {
    set_error("heads_q=%d must be in 1..4096 and a multiple of the cache's %d heads", heads_q, heads);
    return PQ_ERR_INVALID_ARG;
  }
  return PQ_OK;
}

pq_status check_rows(const char* what, const void* p, int64_t ld, int64_t need, int64_t ld_mult, uintptr_t align) {
  if (!p) { set_error("%s is NULL", what); return PQ_ERR_INVALID_ARG; }
  if (ld < need || ld % ld_mult != 0) {
    set_error("%s: row stride %lld must be >= %lld and a multiple of %lld", what, (long long)ld, (long long)need,
              (long long)ld_mult);
    return PQ_ERR_INVALID_ARG;
  }
  if (!aligned(p, align)) { set_error("%s must be %d-byte aligned", what, (int)align); return PQ_ERR_INVALID_ARG; }
  return PQ_OK;
}

}  // namespace

extern "C" pq_status pq_quant_rows8(const void* X, int64_t T, int64_t D, int64_t ldx, int g, int8_t* codes,
                                    float* scales, void* stream) {
  clear_error();
  const pq_status st = check_quant8(X, T, D, ldx, g, codes, scales);
  if (st != PQ_OK) return st;
  return cuda_fail(launch_quant_rows8(X, T, (int)D, ldx, g, codes, scales, reinterpret_cast<cudaStream_t>(stream)),
                   "pq_quant_rows8 launch");
}

extern "C" pq_status pq_w8a8_gemm(const int8_t* codes_A, const float* scales_A, const int8_t* codes_W,
                                  const float* scales_W, int64_t T, int64_t N, int64_t D, void* Y,
                                  pq_out_dtype out_dtype, void* stream) {
  clear_error();
  const pq_status st = check_gemm8(codes_A, scales_A, codes_W, scales_W, T, N, D, Y, out_dtype);
  if (st != PQ_OK) return st;
  return w8a8_launch(codes_A, scales_A, codes_W, scales_W, T, N, D, Y, out_dtype,
                     reinterpret_cast<cudaStream_t>(stream), /*pdl=*/false);
}

extern "C" pq_status pq_w8a8_linear(const void* X, int64_t T, int64_t D, int64_t ldx, int g, int8_t* codes_A,
                                    float* scales_A, const int8_t* codes_W, const float* scales_W, int64_t N, void* Y,
                                    pq_out_dtype out_dtype, void* stream) {
  clear_error();
  pq_status st = check_quant8(X, T, D, ldx, g, codes_A, scales_A);
  if (st != PQ_OK) return st;
  st = check_gemm8(codes_A, scales_A, codes_W, scales_W, T, N, D, Y, out_dtype);
  if (st != PQ_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = cuda_fail(launch_quant_rows8(X, T, (int)D, ldx, g, codes_A, scales_A, s), "pq_w8a8_linear quantisation launch");
  if (st != PQ_OK) return st;
  return w8a8_launch(codes_A, scales_A, codes_W, scales_W, T, N, D, Y, out_dtype, s, /*pdl=*/true);
}

extern "C" pq_status pq_kv4_append(const pq_kv4_cache* cache, const void* Q, int64_t ldq, const void* K, int64_t ldk,
                                   const void* V, int64_t ldv, int64_t T, int heads_q, const void* q_norm,
                                   const void* k_norm, float eps, const float* rope, int64_t rope_rows, int rope_dim,
                                   const int32_t* positions, const int64_t* slots, uint32_t flags, void* Q_out,
                                   void* stream) {
  clear_error();
  Kv4AppendArgs a = {};
  pq_status st = check_cache(cache, &a.cache);
  if (st == PQ_OK) st = check_heads(heads_q, a.cache.heads);
  if (st != PQ_OK) return st;
  const int64_t hd = a.cache.head_dim;
  st = check_rows("Q", Q, ldq, heads_q * hd, 4, 8);
  if (st == PQ_OK) st = check_rows("K", K, ldk, a.cache.heads * hd, 4, 8);
  if (st == PQ_OK) st = check_rows("V", V, ldv, a.cache.heads * hd, 4, 8);
  if (st == PQ_OK) st = check_rows("Q_out", Q_out, heads_q * hd, heads_q * hd, 1, 16);
  if (st != PQ_OK) return st;
  if (T < 1 || T > kMaxRows) { set_error("T=%lld must be in 1..2^24", (long long)T); return PQ_ERR_INVALID_ARG; }
  if (T * (heads_q + 2 * (int64_t)a.cache.heads) >= ((int64_t)1 << 33)) {
    set_error("T times heads is too large for one call");
    return PQ_ERR_INVALID_ARG;
  }
  if (!slots || !aligned(slots, 8)) { set_error("slots must be non-NULL and 8-byte aligned"); return PQ_ERR_INVALID_ARG; }
  if (flags & ~PQ_KV4_INTERLEAVED) { set_error("unknown flags 0x%x", flags); return PQ_ERR_INVALID_ARG; }
  if ((q_norm && !aligned(q_norm, 8)) || (k_norm && !aligned(k_norm, 8))) {
    set_error("norm weights must be 8-byte aligned");
    return PQ_ERR_INVALID_ARG;
  }
  if ((q_norm || k_norm) && !(eps >= 0.0f && std::isfinite(eps))) {
    set_error("eps=%g must be finite and >= 0", (double)eps);
    return PQ_ERR_INVALID_ARG;
  }
  if (rope) {
    if (rope_dim < 8 || rope_dim > hd || rope_dim % 8 != 0) {
      set_error("rope_dim=%d must be a multiple of 8, at most head_dim=%d", rope_dim, (int)hd);
      return PQ_ERR_INVALID_ARG;
    }
    if (rope_rows < 1 || !positions || !aligned16(rope) || !aligned(positions, 4)) {
      set_error("a rope table needs rows, positions and 16-byte alignment");
      return PQ_ERR_INVALID_ARG;
    }
  }
  const cudaError_t e = gemm_status_address(&a.status);
  if (e != cudaSuccess) return cuda_fail(e, "status word");
  a.Q = static_cast<const uint16_t*>(Q), a.K = static_cast<const uint16_t*>(K), a.V = static_cast<const uint16_t*>(V);
  a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
  a.T = T;
  a.heads_q = heads_q;
  a.q_norm = static_cast<const uint16_t*>(q_norm), a.k_norm = static_cast<const uint16_t*>(k_norm);
  a.eps = eps;
  a.rope = rope;
  a.rope_rows = rope ? rope_rows : 0;
  a.rope_dim = rope ? rope_dim : 0;
  a.interleaved = (flags & PQ_KV4_INTERLEAVED) ? 1 : 0;
  a.positions = positions;
  a.slots = slots;
  a.Q_out = static_cast<uint16_t*>(Q_out);
  return cuda_fail(launch_kv4_append(a, reinterpret_cast<cudaStream_t>(stream)), "pq_kv4_append launch");
}

extern "C" pq_status pq_kv4_read(const pq_kv4_cache* cache, const int64_t* slots, int64_t T, void* K_out, void* V_out,
                                 void* stream) {
  clear_error();
  Kv4View c;
  const pq_status st = check_cache(cache, &c);
  if (st != PQ_OK) return st;
  if (!slots || !K_out || !V_out || !aligned(slots, 8) || !aligned16(K_out) || !aligned16(V_out)) {
    set_error("slots, K_out and V_out must be non-NULL and aligned (8 and 16 bytes)");
    return PQ_ERR_INVALID_ARG;
  }
  if (T < 1 || T > kMaxRows || T * c.heads >= ((int64_t)1 << 33)) { set_error("T=%lld is out of range", (long long)T); return PQ_ERR_INVALID_ARG; }
  unsigned int* status = nullptr;
  const cudaError_t e = gemm_status_address(&status);
  if (e != cudaSuccess) return cuda_fail(e, "status word");
  return cuda_fail(launch_kv4_read(c, slots, T, static_cast<uint16_t*>(K_out), static_cast<uint16_t*>(V_out), status,
                                   reinterpret_cast<cudaStream_t>(stream)),
                   "pq_kv4_read launch");
}

extern "C" pq_status pq_kv4_attention(const pq_kv4_cache* cache, const void* Q, int64_t ldq, int heads_q,
                                      const int32_t* q_start, const int32_t* seq_lens, const int32_t* block_table,
                                      int64_t table_width, int64_t B, int64_t T, int64_t max_q, int64_t max_len,
                                      float scale, int64_t window, void* O, int64_t ldo, void* stream) {
  clear_error();
  Kv4AttnArgs a = {};
  pq_status st = check_cache(cache, &a.cache);
  if (st == PQ_OK) st = check_heads(heads_q, a.cache.heads);
  if (st != PQ_OK) return st;
  const int64_t hd = a.cache.head_dim;
  st = check_rows("Q", Q, ldq, heads_q * hd, 8, 16);
  if (st == PQ_OK) st = check_rows("O", O, ldo, heads_q * hd, 8, 16);
  if (st != PQ_OK) return st;
  if (!q_start || !seq_lens || !block_table || !aligned(q_start, 4) || !aligned(seq_lens, 4) || !aligned(block_table, 4)) {
    set_error("q_start, seq_lens and block_table must be non-NULL and 4-byte aligned");
    return PQ_ERR_INVALID_ARG;
  }
  if (B < 1 || B > 65535) { set_error("B=%lld must be in 1..65535", (long long)B); return PQ_ERR_INVALID_ARG; }
  if (T < 1 || T > kMaxRows) { set_error("T=%lld must be in 1..2^24", (long long)T); return PQ_ERR_INVALID_ARG; }
  if (table_width < 1 || table_width > kMaxTokens || table_width * (int64_t)cache->page_size > kMaxTokens) {
    set_error("table_width=%lld pages must hold 1..2^30 tokens", (long long)table_width);
    return PQ_ERR_INVALID_ARG;
  }
  if (max_q < 1 || max_len < 1) {
    set_error("max_q=%lld and max_len=%lld must be >= 1", (long long)max_q, (long long)max_len);
    return PQ_ERR_INVALID_ARG;
  }
  if (window < 0 || window >= ((int64_t)1 << 31)) { set_error("window=%lld must be in 0..2^31-1", (long long)window); return PQ_ERR_INVALID_ARG; }
  if (!std::isfinite(scale)) { set_error("scale must be finite"); return PQ_ERR_INVALID_ARG; }
  const cudaError_t e = gemm_status_address(&a.status);
  if (e != cudaSuccess) return cuda_fail(e, "status word");
  a.Q = static_cast<const uint16_t*>(Q);
  a.ldq = ldq;
  a.heads_q = heads_q;
  a.q_start = q_start, a.seq_lens = seq_lens, a.table = block_table;
  a.table_stride = table_width;
  a.table_width = (int)table_width;
  a.B = (int)B;
  a.T = T;
  a.scale = scale;
  a.window = (int)std::min(window, kMaxTokens);          // a wider one hides nothing
  a.O = static_cast<uint16_t*>(O);
  a.ldo = ldo;
  // Bounds beyond what a call can hold say no more than that (and would wrap when multiplied with the heads).
  return kv4_attention_run(a, std::min(max_q, kMaxRows), std::min(max_len, kMaxTokens), reinterpret_cast<cudaStream_t>(stream));
}
