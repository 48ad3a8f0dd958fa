// Causal attention of packed prompts over bf16 states (the loop and its
// layout are in attention_tile.h).
//
// Bound: the matrix cores, 4 head_dim flops a (head, seen position), beside the
// exponentials and the other vector work of the softmax.
#include <math.h>

#include "attention.h"
#include "attention_tile.h"

namespace fp8blk {

namespace {

// Workgroups go over the rows from the sequences' ends, which see the most
// positions, so that the short ones fill the tail; neighbouring workgroups are
// different heads, so that with 8 kv heads those of one share an XCD's L2.
template <int D>
__global__ void __launch_bounds__(kTileThreads, D == 256 ? 1 : 2) k_prompt_attention(PromptArgs a, FastDiv group, int tiles) {
  __shared__ TileLds<D> lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int64_t heads = a.batch * a.kv_heads;
  const int kh = (int)(blockIdx.x % a.kv_heads);
  const int64_t b = blockIdx.x % heads / a.kv_heads;
  const int tile = tiles - 1 - (int)(blockIdx.x / heads);
  const int G = a.heads / a.kv_heads;
  const int t0 = clip(a.starts[b], 0, a.tokens), n = clip(a.starts[b + 1], t0, a.tokens) - t0;
  const int64_t rows = (int64_t)(n < a.max_len ? n : (int)a.max_len) * G;
  const int64_t first = (int64_t)tile * kTileRows;
  if (first >= rows) return;
  const int64_t end = first + kTileRows < rows ? first + kTileRows : rows;
  const int64_t w0 = first + 32 * wave;            // the wave's first row
  const int64_t q = w0 + (lane & 31);
  const bool in = q < rows;
  const int i = in ? (int)div_by((uint32_t)q, group) : 0, h = in ? kh * G + (int)(q - (int64_t)i * G) : kh * G;
  s8v qf[D / 16];
#pragma unroll
  for (int e = 0; e < D / 16; ++e)
    qf[e] = *(const s8v*)(a.q + (int64_t)(t0 + i) * a.ld_q + (int64_t)h * D + 16 * e + 8 * half);

  DenseTile<D> src;
  src.kp = a.k + (int64_t)t0 * a.ld_k + (int64_t)kh * D;
  src.vp = a.v + (int64_t)t0 * a.ld_v + (int64_t)kh * D;
  src.ld_k = a.ld_k;
  src.ld_v = a.ld_v;
  src.n = n;
  RowState<D> st;
  const int seen = w0 < rows ? (int)div_by((uint32_t)w0, group) + 1 : 0;
  const int j1 = (int)div_by((uint32_t)(end - 1), group) + 1;
  attend_tiles<DenseTile<D>, D, false, false>(src, lds, qf, qf, a.scale * kLog2e, i + 1, seen, 0, j1, st);
  if (!in) return;
  const float inv = 1.0f / st.l;
  const int64_t row = (int64_t)(t0 + i) * a.heads + h;
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      u32x2 w;
      w[0] = pack_bf16(st.o[d][r] * inv, st.o[d][r + 1] * inv);
      w[1] = pack_bf16(st.o[d][r + 2] * inv, st.o[d][r + 3] * inv);
      *(u32x2*)(a.out + row * D + 32 * d + 2 * r + 4 * half) = w;
    }
  if (a.lse && half == 0) a.lse[row] = (st.m + __log2f(st.l)) * kLn2;
}

int64_t tiles_of(int64_t heads, int64_t kv_heads, int64_t max_len) {
  return (max_len * (heads / kv_heads) + kTileRows - 1) / kTileRows;
}

}  // namespace

bool prompt_attention_fits(int64_t heads, int64_t kv_heads, int64_t batch, int64_t max_len) {
  if (kv_heads == 0) return true;
  if (max_len * (heads / kv_heads) >= INT64_C(0x7fffffff)) return false;   // a sequence's rows are indexed with 31 bits
  return tiles_of(heads, kv_heads, max_len) < INT64_C(0x7fffffff) / (batch * kv_heads + 1);
}

hipError_t launch_prompt_attention(const PromptArgs& a, int head_dim, hipStream_t st) {
  const int64_t tiles = tiles_of(a.heads, a.kv_heads, a.max_len);
  const unsigned grid = (unsigned)(tiles * a.batch * a.kv_heads);
  const FastDiv group = make_fastdiv(a.heads / a.kv_heads);
  if (head_dim == 64) k_prompt_attention<64><<<grid, kTileThreads, 0, st>>>(a, group, (int)tiles);
  else if (head_dim == 128) k_prompt_attention<128><<<grid, kTileThreads, 0, st>>>(a, group, (int)tiles);
  else k_prompt_attention<256><<<grid, kTileThreads, 0, st>>>(a, group, (int)tiles);
  return hipGetLastError();
}

}  // namespace fp8blk
