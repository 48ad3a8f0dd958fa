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
template <int D, int W>
__global__ void __launch_bounds__(64 * W, D == 256 ? 1 : 2) k_prompt_attention(PromptArgs a, FastDiv group, int tiles) {
  __shared__ TileLds<D> lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int64_t heads = a.batch * a.kv_heads;
  const int kh = (int)(blockIdx.x % a.kv_heads);
  const int64_t b = blockIdx.x % heads / a.kv_heads;
  const int tile = tiles - 1 - (int)(blockIdx.x / heads);
  const int G = a.heads / a.kv_heads;
  const int t0 = clip(a.starts[b], 0, a.tokens), n = clip(a.starts[b + 1], t0, a.tokens) - t0;
  const int64_t rows = (int64_t)(n < a.max_len ? n : (int)a.max_len) * G;
  const int64_t first = (int64_t)tile * 32 * W;
  if (first >= rows) return;
  const int64_t end = first + 32 * W < rows ? first + 32 * W : rows;
  const int64_t w0 = first + 32 * wave;            // the wave's first row
  const int64_t q = w0 + (lane & 31);
  const bool in = q < rows;
  const int i = in ? (int)div_by((uint32_t)q, group) : 0, h = in ? kh * G + (int)(q - (int64_t)i * G) : kh * G;
  s8v qf[D / 16];
#pragma unroll
  for (int e = 0; e < D / 16; ++e)
    qf[e] = *(const s8v*)(a.q + (int64_t)(t0 + i) * a.ld_q + (int64_t)h * D + 16 * e + 8 * half);

  DenseTile<D, W> src;
  src.kp = a.k + (int64_t)t0 * a.ld_k + (int64_t)kh * D;
  src.vp = a.v + (int64_t)t0 * a.ld_v + (int64_t)kh * D;
  src.ld_k = a.ld_k;
  src.ld_v = a.ld_v;
  src.n = n;
  RowState<D> st;
  const int seen = w0 < rows ? (int)div_by((uint32_t)w0, group) + 1 : 0;
  const int j1 = (int)div_by((uint32_t)(end - 1), group) + 1;
  attend_tiles<DenseTile<D, W>, D, false, false>(src, lds, qf, qf, a.scale * kLog2e, i + 1, seen,
                                                       (int)div_by((uint32_t)first, group) + 1, 0, j1, st);
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

int64_t tiles_of(int64_t heads, int64_t kv_heads, int64_t max_len, int waves) {
  return (max_len * (heads / kv_heads) + 32 * waves - 1) / (32 * waves);
}

template <int D, int W>
void launch(const PromptArgs& a, hipStream_t st) {
  const int64_t tiles = tiles_of(a.heads, a.kv_heads, a.max_len, W);
  k_prompt_attention<D, W><<<(unsigned)(tiles * a.batch * a.kv_heads), 64 * W, 0, st>>>(
      a, make_fastdiv(a.heads / a.kv_heads), (int)tiles);
}

}  // namespace

bool prompt_attention_fits(int64_t heads, int64_t kv_heads, int64_t batch, int64_t max_len) {
  if (kv_heads == 0) return true;
  if (max_len * (heads / kv_heads) >= INT64_C(0x7fffffff)) return false;   // a sequence's rows are indexed with 31 bits
  return tiles_of(heads, kv_heads, max_len, 4) < INT64_C(0x7fffffff) / (batch * kv_heads + 1);
}

namespace {

// Eight waves stage a tile for twice the rows, but only one such workgroup fits
// a CU: worth it from two workgroups a CU on (2 x 8192 tokens, 32 heads of 128:
// 1028 us against 1109; 1 x 4096: 140 against 154), and not below (1 x 2048: 58
// against 52; 1 x 8192 with 8 heads of 64 on one kv head: 137 against 113).
// Heads of 256 leave registers for one wave a SIMD.
template <int D>
void launch_by_rows(const PromptArgs& a, hipStream_t st) {
  if constexpr (D < 256) {
    if (tiles_of(a.heads, a.kv_heads, a.max_len, 8) * a.batch * a.kv_heads >= 512) return launch<D, 8>(a, st);
  }
  launch<D, 4>(a, st);
}

}  // namespace

hipError_t launch_prompt_attention(const PromptArgs& a, int head_dim, hipStream_t st) {
  if (head_dim == 64) launch_by_rows<64>(a, st);
  else if (head_dim == 128) launch_by_rows<128>(a, st);
  else launch_by_rows<256>(a, st);
  return hipGetLastError();
}

}  // namespace fp8blk
