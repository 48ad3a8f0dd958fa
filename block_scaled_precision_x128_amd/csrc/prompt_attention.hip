// Causal attention of packed prompts over bf16 states (the loop and its
// layout are in attention_tile.h).
//
// Bound: the matrix cores, 4 head_dim flops a (head, seen position), beside the
// exponentials and the LDS reads.  2 x 8192 tokens, 32 heads of 128 on 8: 1.10
// TFLOP in 1030 to 1090 us from card to card, 1010 to 1070 TFLOP/s, where a large matrix
// product of the library reaches 1230.  p is rounded to bf16 (half a step 2^-8,
// that of the output), since bf16 values do not fit fp16's range.
#include <math.h>

#include "attention.h"
#include "attention_tile.h"
#include "kv_attention.h"

namespace fp8blk {

namespace {

// Workgroups go over the rows from the sequences' ends, which see the most
// positions, so that the short ones fill the tail; neighbouring workgroups are
// different heads, so that with 8 kv heads those of one share an XCD's L2.
template <int D, int W>
__global__ void __launch_bounds__(64 * W, D == 256 ? 1 : 2) k_prompt_attention(PromptArgs a, KvPlan p, int tiles) {
  __shared__ TileLds<D> lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int64_t heads = a.batch * a.kv_heads;
  const int kh = (int)(blockIdx.x % a.kv_heads);
  const int64_t b = blockIdx.x % heads / a.kv_heads;
  const int split = (int)(blockIdx.x / heads % p.splits);
  const int tile = tiles - 1 - (int)(blockIdx.x / heads / p.splits);
  const int G = a.heads / a.kv_heads;
  const int t0 = clip(a.starts[b], 0, a.tokens), n = clip(a.starts[b + 1], t0, a.tokens) - t0;
  const int64_t rows = (int64_t)(n < a.max_len ? n : (int)a.max_len) * G;
  const int64_t first = (int64_t)tile * 32 * W;
  if (first >= rows) return;
  const int64_t end = first + 32 * W < rows ? first + 32 * W : rows;
  const int64_t w0 = first + 32 * wave;            // the wave's first row
  const int64_t q = w0 + (lane & 31);
  const bool in = q < rows;
  const int i = in ? (int)div_by((uint32_t)q, p.group) : 0, h = in ? kh * G + (int)(q - (int64_t)i * G) : kh * G;
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
  const int seen = w0 < rows ? (int)div_by((uint32_t)w0, p.group) + 1 : 0;
  const int stop = (int)div_by((uint32_t)(end - 1), p.group) + 1;       // no row of the workgroup sees more
  const int j0 = split * p.split_len, j1 = stop - j0 < p.split_len ? stop : j0 + p.split_len;
  const int64_t row = (int64_t)(t0 + i) * a.heads + h;
  if (j0 >= stop) {                                // then split > 0
    if (in && half == 0 && j0 < n) p.part_ml[split * p.part_rows + row] = v2f{kNoMax, 0.0f};
    return;
  }
  attend_tiles<DenseTile<D, W>, D, false, false>(src, lds, qf, qf, a.scale * kLog2e, i + 1, seen,
                                                 (int)div_by((uint32_t)first, p.group) + 1, j0, j1, st);
  if (!in) return;
  if (p.splits > 1) {
    store_part<D>(st, p, split, row);
    return;
  }
  const float inv = 1.0f / st.l;
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

struct Plan {
  KvPlan p;
  int waves;
  size_t ml, o, bytes;
};

// Eight waves stage a tile for twice the rows, but only one such workgroup fits
// a CU: worth it from two workgroups a CU on (2 x 8192 tokens, 32 heads of 128:
// 1028 us against 1109; 1 x 4096: 140 against 154), and not below (1 x 2048: 58
// against 52; 1 x 8192 with 8 heads of 64 on one kv head: 137 against 113).
// Heads of 256 leave registers for one wave a SIMD.  Where four waves leave half
// the CUs without a workgroup the positions are split (2 x 4655, one head: 46 us
// against 96; 4 x 1500, two heads: 26 against 36); with more workgroups than
// that the joining costs more than the split gains (1 x 700, 32 heads on 8: 31
// against 20; 1 x 6000, 8 heads: 142 against 126).
Plan plan(int64_t tokens, int64_t heads, int64_t kv_heads, int head_dim, int64_t batch, int64_t max_len) {
  Plan t{};
  const int64_t bk = batch * kv_heads;
  t.waves = head_dim < 256 && bk * tiles_of(heads, kv_heads, max_len, 8) >= 512 ? 8 : 4;
  const int64_t groups = bk * tiles_of(heads, kv_heads, max_len, 4);
  plan_splits(groups, groups <= 128 ? 512 : 0, 512, 64, max_len, t.p);
  t.p.part_rows = tokens * heads;
  if (t.p.splits > 1) {
    t.o = ((size_t)(t.p.splits * t.p.part_rows) * sizeof(v2f) + 255) / 256 * 256;
    t.bytes = t.o + (size_t)(t.p.splits * t.p.part_rows) * head_dim * sizeof(float);
  }
  return t;
}

template <int D, int W>
void launch(const PromptArgs& a, const Plan& t, hipStream_t st) {
  const int64_t tiles = tiles_of(a.heads, a.kv_heads, a.max_len, W);
  k_prompt_attention<D, W><<<(unsigned)(tiles * a.batch * a.kv_heads * t.p.splits), 64 * W, 0, st>>>(a, t.p, (int)tiles);
}

template <int D>
void launch_waves(const PromptArgs& a, const Plan& t, hipStream_t st) {
  if constexpr (D < 256) {
    if (t.waves == 8) return launch<D, 8>(a, t, st);
  }
  launch<D, 4>(a, t, st);
}

}  // namespace

size_t prompt_attention_workspace(int64_t tokens, int64_t heads, int64_t kv_heads, int head_dim, int64_t batch,
                                  int64_t max_len) {
  return heads > 0 && kv_heads > 0 ? plan(tokens, heads, kv_heads, head_dim, batch, max_len).bytes : 0;
}

bool prompt_attention_fits(int64_t heads, int64_t kv_heads, int64_t batch, int64_t max_len) {
  if (heads == 0 || kv_heads == 0 || batch == 0) return true;
  // A sequence's rows are indexed with 31 bits; workgroups stay below 2^31:
  // four waves' tiles, 512 more with splits, and those that join them.
  constexpr double kMost = 2147483647.0;
  const double rows = (double)max_len * (double)(heads / kv_heads);
  return rows < kMost && (double)batch * (double)kv_heads * (rows / 128 + 2) + 1024 < kMost &&
         (double)batch * (double)max_len * (double)heads < kMost;
}

hipError_t launch_prompt_attention(const PromptArgs& a, int head_dim, hipStream_t st) {
  Plan t = plan(a.tokens, a.heads, a.kv_heads, head_dim, a.batch, a.max_len);
  t.p.group = make_fastdiv(a.heads / a.kv_heads);
  t.p.part_ml = (v2f*)a.ws;
  t.p.part_o = (float*)((uint8_t*)a.ws + t.o);
  t.p.lse = a.lse;
  if (head_dim == 64) launch_waves<64>(a, t, st);
  else if (head_dim == 128) launch_waves<128>(a, t, st);
  else launch_waves<256>(a, t, st);
  if (t.p.splits > 1) {
    KvAttnArgs j{};
    j.q_starts = a.starts;
    j.out = a.out;
    j.q_tokens = a.tokens;
    j.num_slots = 1;
    j.batch = a.batch;
    j.max_q = j.max_kv = a.max_len;
    j.heads = a.heads;
    j.kv_heads = a.kv_heads;
    j.out_dt = DT_BF16;
    j.sk = kNoScale;
    launch_join(j, t.p, head_dim, st);
  }
  return hipGetLastError();
}

}  // namespace fp8blk
