// Internal launcher interface of the attention and eviction kernels (host
// side, C++ linkage).  The public C ABI in include/fp8blk.h validates
// arguments and calls these.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8blk {

struct KvAttnArgs {
  const void* q;              // [q_tokens, ld_q], dt q_dt (0 fp32, 1 bf16)
  const uint8_t* k;           // [num_slots, kv_heads, D] codes
  const uint8_t* v;
  const int64_t* table;       // [batch, max_blocks]
  const int64_t* q_starts;    // [batch + 1]
  const int64_t* kv_lens;     // [batch]
  const float* ks;
  const float* vs;
  void* out;                  // [q_tokens, heads, D]
  float* lse;                 // [q_tokens, heads] or null
  const float* w_in;          // [batch, kv_heads, ld_w] or null
  float* w_out;               // or null
  void* ws;
  int64_t q_tokens, ld_q, num_slots, max_blocks, block_size, batch, max_q, max_kv, ld_w;
  int heads, kv_heads, q_dt, out_dt, fmt, sk;
  float scale;
};

size_t kv_attention_workspace(int64_t q_tokens, int64_t heads, int64_t kv_heads, int head_dim, int64_t batch,
                              int64_t max_q, int64_t max_kv, bool with_weights);
// False where a launch would pass the grid limits.
bool kv_attention_fits(int64_t heads, int64_t kv_heads, int64_t batch, int64_t max_q, int64_t max_kv);
hipError_t launch_kv_attention(const KvAttnArgs& a, int head_dim, hipStream_t st);

struct PromptArgs {
  const uint16_t* q;          // bf16 [tokens, ld_q]
  const uint16_t* k;
  const uint16_t* v;
  const int64_t* starts;      // [batch + 1]
  uint16_t* out;              // [tokens, heads, D]
  float* lse;                 // or null
  void* ws;
  int64_t ld_q, ld_k, ld_v, tokens, batch, max_len;
  int heads, kv_heads;
  float scale;
};

size_t prompt_attention_workspace(int64_t tokens, int64_t heads, int64_t kv_heads, int head_dim, int64_t batch,
                                  int64_t max_len);
bool prompt_attention_fits(int64_t heads, int64_t kv_heads, int64_t batch, int64_t max_len);
hipError_t launch_prompt_attention(const PromptArgs& a, int head_dim, hipStream_t st);

size_t kv_evict_select_workspace(int64_t batch, int64_t max_kv);
hipError_t launch_kv_evict_select(const float* w, int64_t ld_w, int64_t batch, int64_t kv_heads,
                                  const int64_t* kv_lens, int64_t max_kv, int64_t keep, int64_t first, int64_t recent,
                                  int64_t* kept, int64_t* kept_lens, void* ws, hipStream_t st);

struct CompactArgs {
  uint8_t* cache[2];
  const int64_t* src;         // [batch, src_blocks]
  const int64_t* dst;         // [batch, dst_blocks]
  const int64_t* kept;        // [batch, keep]
  const int64_t* kept_lens;   // [batch]
  const float* w_in;
  float* w_out;
  int64_t num_slots, row, src_blocks, dst_blocks, block_size, batch, keep, ld_in, ld_out, kv_heads;
};

hipError_t launch_kv_compact(const CompactArgs& a, hipStream_t st);

}  // namespace fp8blk
