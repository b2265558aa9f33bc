// Internal declarations of the 4-bit key/value cache: launch arguments and shared constants.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/pq.h"

namespace pq {

// The cache as the kernels see it (validated; page_size = 1 << page_shift).
struct Kv4View {
  uint8_t* k_codes;
  float* k_scales;
  uint8_t* v_codes;
  float* v_scales;
  int64_t pages;
  int page_shift;
  int heads;
  int head_dim;
  int rotate_k, rotate_v;
};

struct Kv4AppendArgs {
  Kv4View cache;
  const uint16_t *Q, *K, *V;
  int64_t ldq, ldk, ldv;
  int64_t T;
  int heads_q;
  const uint16_t *q_norm, *k_norm;
  float eps;
  const float* rope;
  int64_t rope_rows;
  int rope_dim;
  int interleaved;
  const int32_t* positions;
  const int64_t* slots;
  uint16_t* Q_out;
  unsigned int* status;
};

struct Kv4AttnArgs {
  Kv4View cache;
  const uint16_t* Q;
  int64_t ldq;
  int heads_q;
  const int32_t* q_start;      // [B + 1]
  const int32_t* seq_lens;     // [B]
  const int32_t* table;        // [B][table_stride]
  int64_t table_stride;
  int table_width;             // pages a table row lists
  int B;
  int64_t T;
  float scale;
  int window;                  // 0: none
  uint16_t* O;
  int64_t ldo;
  unsigned int* status;
};

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4View& c, const int64_t* slots, int64_t T, uint16_t* K_out, uint16_t* V_out,
                            unsigned int* status, cudaStream_t stream);
// The kernel for many query rows (kv4_prompt.cu): tiles of 256 (token, head) rows at most, and its launch.
struct Partials;
int64_t kv4_prompt_tiles(const Kv4AttnArgs& a);
pq_status launch_kv4_prompt(const Kv4AttnArgs& a, const Partials& part, cudaStream_t stream);
pq_status kv4_attention_run(const Kv4AttnArgs& a, int64_t max_q, int64_t max_len, cudaStream_t stream);

}  // namespace pq
