// Attention over the paged FP8 cache for a chunk of new tokens (the loop and
// its layout are in attention_tile.h), and the weights that its positions
// received.
//
// Bound: the matrix cores beside the softmax's vector work and the LDS reads.
// Codes become fp16 on the way into LDS, once for a workgroup's 128 rows; a q
// that fp16 does not hold exactly goes through the first product as two halves
// (lse is fp32).  2 x 512 tokens on 8192 positions, 32 heads of 128 on 8: 133
// GFLOP in 171 us with per-head scales (780 TFLOP/s), 210 us with per-channel
// ones, whose half more products put the matrix cores at 950.  Few or short
// chunks leave workgroups too few for the chip: the positions are then split,
// and k_kv_finish joins the parts.
#include <math.h>

#include "attention.h"
#include "attention_tile.h"
#include "kv_attention.h"

namespace fp8blk {

namespace {

// Rows of one (sequence, kv head): row q is query token q / G, head q % G.
struct Rows {
  int64_t b;
  int kh, G;
  Span sp;
  int64_t rows;
  const KvPlan& p;
  const KvAttnArgs& a;
  __device__ Rows(const KvAttnArgs& args, const KvPlan& plan, int64_t bk) : p(plan), a(args) {
    b = bk / a.kv_heads;
    kh = (int)(bk % a.kv_heads);
    G = a.heads / a.kv_heads;
    sp = span_of(a.q_starts, a.kv_lens, b, a.q_tokens, a.max_kv);
    rows = (int64_t)(sp.n < a.max_q ? sp.n : (int)a.max_q) * G;
  }
  __device__ int token(int64_t q) const { return (int)div_by((uint32_t)q, p.group); }
  __device__ int limit(int64_t q) const { return sp.L - sp.n + token(q) + 1; }
  __device__ int64_t out_row(int64_t q) const {
    const int i = token(q);
    return (int64_t)(sp.t0 + i) * a.heads + kh * G + (int)(q - (int64_t)i * G);
  }
};

// The lane's query row as fp16 operands, times the key scales where they
// differ by channel and times a power of two; returns the factor from raw
// products to scores in powers of two.
template <int D, bool SPLITQ>
__device__ __forceinline__ float load_query(const Rows& w, int64_t q, bool in, s8v* hi, s8v* lo) {
  const KvAttnArgs& a = w.a;
  const int half = (threadIdx.x & 63) >> 5;
  const int i = in ? w.token(q) : 0, g = in ? (int)(q - (int64_t)i * w.G) : 0;
  const int64_t at = (int64_t)(w.sp.t0 + i) * a.ld_q + (int64_t)(w.kh * w.G + g) * D + 8 * half;
  const float* ks = a.ks + w.kh * D + 8 * half;
  float x[D / 16][8], top = 0.0f;
  load_pieces<D / 16, 8, 16>(a.q, a.q_dt, at, a.sk == 2 ? ks : nullptr, x);
#pragma unroll
  for (int e = 0; e < D / 16; ++e)
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[e][k] = in ? x[e][k] : 0.0f;
      top = fmaxf(top, fabsf(x[e][k]));
    }
  const int ex = row_exponent(max_halves(top));
#pragma unroll
  for (int e = 0; e < D / 16; ++e) {
    h8 y, z;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float v = ldexpf(x[e][k], 14 - ex);
      y[k] = (_Float16)v;
      z[k] = (_Float16)(v - (float)y[k]);
    }
    hi[e] = __builtin_bit_cast(s8v, y);
    if constexpr (SPLITQ) lo[e] = __builtin_bit_cast(s8v, z);
  }
  return ldexpf(a.scale * kLog2e * (a.sk == 2 ? 1.0f : a.ks[a.sk == 1 ? w.kh : 0]), ex - 14);
}

template <int FMT, int D, bool SPLITQ, bool SPLITP>
__global__ void __launch_bounds__(64 * kChunkWaves, D == 256 ? 1 : 2) k_kv_chunk(KvAttnArgs a, KvPlan p, int tiles) {
  constexpr int W = kChunkWaves;
  __shared__ TileLds<D> lds;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int64_t heads = a.batch * a.kv_heads, bk = blockIdx.x % heads;
  const int split = (int)(blockIdx.x / heads % p.splits);
  const int tile = tiles - 1 - (int)(blockIdx.x / heads / p.splits);
  const Rows w(a, p, bk);
  const int64_t first = (int64_t)tile * 32 * W;
  if (first >= w.rows) return;
  const int64_t end = first + 32 * W < w.rows ? first + 32 * W : w.rows;
  const int64_t w0 = first + 32 * wave;
  const int64_t q = w0 + (lane & 31);
  const bool in = q < w.rows;
  const int L = a.num_slots > 0 ? w.sp.L : 0;
  const int stop = min(L, w.limit(end - 1));        // no row of the tile sees more
  const int j0 = split * p.split_len;
  if (split > 0 && j0 >= L) return;
  const int j1 = stop - j0 < p.split_len ? stop : j0 + p.split_len;
  const int64_t row = in ? w.out_row(q) : 0;
  if (split > 0 && j0 >= j1) {
    if (in && half == 0) p.part_ml[split * p.part_rows + row] = v2f{kNoMax, 0.0f};
    return;
  }
  s8v qh[D / 16], ql[SPLITQ ? D / 16 : 1];
  const float c = load_query<D, SPLITQ>(w, q, in, qh, ql);
  if (p.queries && split == 0 && w0 < w.rows) {       // kept for the weights
    const int64_t at = bk * p.row_tiles + w0 / 32;
    s8v* to = (s8v*)p.queries + at * (2 * (D / 16) * 64) + lane;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {
      to[64 * e] = qh[e];
      if constexpr (SPLITQ) to[64 * (D / 16 + e)] = ql[e];
    }
    if (half == 0) p.factors[at * 32 + lane] = c;
  }
  PagedTile<FMT, D, W> src;
  src.kp = a.k + (int64_t)w.kh * D;
  src.vp = a.v + (int64_t)w.kh * D;
  src.table = a.table + w.b * a.max_blocks;
  src.slot_bytes = (int64_t)a.kv_heads * D;
  src.page = p.page;
  src.n = j1;
  src.num_slots = (int)a.num_slots;
  RowState<D> st;
  const int seen = w0 < w.rows ? min(L, w.limit(w0)) : 0;
  attend_tiles<PagedTile<FMT, D, W>, D, SPLITQ, SPLITP>(src, lds, qh, ql, c, in ? w.limit(q) : 0, seen,
                                                                min(L, w.limit(first)), j0, j1, st);
  if (!in) return;
  if (p.splits > 1) {
    store_part<D>(st, p, split, row);
    return;
  }
  const float inv = st.l != 0.0f ? 1.0f / st.l : 0.0f;
  const float one = a.sk == 2 ? 1.0f : a.vs[a.sk == 1 ? w.kh : 0];
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int ch = 32 * d + 2 * r + 4 * half;
      float y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = st.o[d][r + k] * inv * (a.sk == 2 ? a.vs[w.kh * D + ch + k] : one);
      if (a.out_dt == DT_BF16) *(u32x2*)((uint16_t*)a.out + row * D + ch) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
      else *(v4f*)((float*)a.out + row * D + ch) = v4f{y[0], y[1], y[2], y[3]};
    }
  if (p.lse && half == 0) p.lse[row] = st.l != 0.0f ? (st.m + __log2f(st.l)) * kLn2 : -INFINITY;
}

// ---- weights ------------------------------------------------------------------
// The sum over rows of p needs every row's final l, so a second pass forms the
// scores again, by positions: a wave keeps the keys of 64 positions in
// registers as first operands and walks tiles of 32 rows that see them, whose
// operands the chunk kernel has left as the instruction takes them (fp16 halves
// hi, lo [bk][row tile][D/16][64 lanes], and the factor of each row).  The four
// waves of a workgroup take every fourth tile for the same positions, so that a
// long chunk on a short cache still fills the chip (6 x 301 on 3001, ragged:
// 62 us, 104 with 64 positions of its own for each wave).  A lane sums over the
// rows of its column in order; lanes and waves are joined at the end, in order.

constexpr int kWeightKv = 64;       // positions of a workgroup

template <int FMT, int D, bool SPLITQ>
__global__ void __launch_bounds__(256, D == 256 ? 1 : 2) k_kv_weights_chunk(KvAttnArgs a, KvPlan p, int tiles) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = lane >> 5;
  const int64_t bk = blockIdx.x / tiles;
  const Rows w(a, p, bk);
  const int base = (int)(blockIdx.x % tiles) * kWeightKv;
  if (base >= w.sp.L) return;
  const int64_t* table = a.table + w.b * a.max_blocks;
  const int j = base + lane;
  const int slot = a.num_slots > 0 && j < w.sp.L ? slot_of(table, (uint32_t)j, p.page, (int)a.num_slots) : -1;
  const uint64_t live = __ballot(slot >= 0);
  float sum[2][16];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) sum[t][r] = 0.0f;
  // token i sees the first position from i = base - (L - n) on
  const int i0 = max(0, base - (w.sp.L - w.sp.n));
  const int64_t first = (int64_t)i0 * w.G / 32 + wave;
  if (live && 32 * first < w.rows) {
    s8v k[2][D / 16];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int s = __shfl(slot, 32 * t + (lane & 31));
      const uint8_t* at = a.k + ((int64_t)(s < 0 ? 0 : s) * a.kv_heads + w.kh) * D + 8 * half;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        u32x2 x = *(const u32x2*)(at + 16 * e);
        if (s < 0) x = u32x2{0, 0};                // a dead row's codes may be NaN
        k[t][e] = __builtin_bit_cast(s8v, codes_to_h8<FMT>(x[0], x[1]));
      }
    }
    for (int64_t t = first; 32 * t < w.rows; t += 4) {
      const int64_t q = 32 * t + (lane & 31), at = bk * p.row_tiles + t;
      const bool in = q < w.rows;
      const float c = p.factors[at * 32 + (lane & 31)];
      const float lse = in ? p.lse[w.out_row(q)] : -INFINITY;
      const float ref = lse == -INFINITY ? INFINITY : lse * kLog2e;   // exp2(s - Inf) = 0
      const int limit = in ? w.limit(q) : 0;
      const s8v* from = (const s8v*)p.queries + at * (2 * (D / 16) * 64) + lane;
      v16f s[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[u][r] = 0.0f;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const s8v hi = from[64 * e];
        s[0] = mfma32<false>(k[0][e], hi, s[0]);
        s[1] = mfma32<false>(k[1][e], hi, s[1]);
        if constexpr (SPLITQ) {
          const s8v lo = from[64 * (D / 16 + e)];
          s[0] = mfma32<false>(k[0][e], lo, s[0]);
          s[1] = mfma32<false>(k[1][e], lo, s[1]);
        }
      }
      const bool whole = base + kWeightKv <= w.limit(32 * t);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int pos = base + 32 * u + 8 * (r / 4) + 4 * half + r % 4;
          const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][r], c, -ref));
          sum[u][r] += whole || pos < limit ? x : 0.0f;
        }
    }
  }
  // Over the 32 lanes of a row: the swap adds the two rows of 16 lanes of both
  // halves of the positions at once, and leaves positions 32 u + .. in rows u.
  __shared__ float red[4][kWeightKv];
  const int u = lane >> 4 & 1;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(sum[0][r]), __float_as_uint(sum[1][r]), false, false);
    const float y = sum16(__uint_as_float(x[0]) + __uint_as_float(x[1]));
    if ((lane & 15) == 0) red[wave][32 * u + 8 * (r / 4) + 4 * half + r % 4] = y;
  }
  __syncthreads();
  if (wave == 0 && j < w.sp.L) {
    const float x = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
    const int64_t at = bk * a.ld_w + j;
    a.w_out[at] = (a.w_in ? a.w_in[at] : 0.0f) + (slot >= 0 ? x : 0.0f);
  }
}

}  // namespace

template <int FMT, int D>
static void launch(const KvAttnArgs& a, const KvPlan& p, hipStream_t st) {
  constexpr int T = 64 * kChunkWaves;
  const int tiles = (int)kv_chunk_tiles(a.heads, a.kv_heads, a.max_q);
  const unsigned grid = (unsigned)(a.batch * a.kv_heads * p.splits * tiles);
  // lse is fp32, so q has to be exact or carried in two halves.
  const bool so = a.out_dt == DT_F32, sq = a.q_dt == DT_F32 || a.sk == 2;
  if (sq && so) k_kv_chunk<FMT, D, true, true><<<grid, T, 0, st>>>(a, p, tiles);
  else if (sq) k_kv_chunk<FMT, D, true, false><<<grid, T, 0, st>>>(a, p, tiles);
  else if (so) k_kv_chunk<FMT, D, false, true><<<grid, T, 0, st>>>(a, p, tiles);
  else k_kv_chunk<FMT, D, false, false><<<grid, T, 0, st>>>(a, p, tiles);
}

template <int FMT, int D>
static void launch_weights(const KvAttnArgs& a, const KvPlan& p, hipStream_t st) {
  const int tiles = (int)((a.max_kv + kWeightKv - 1) / kWeightKv);
  const unsigned grid = (unsigned)(a.batch * a.kv_heads * tiles);
  if (a.q_dt == DT_F32 || a.sk == 2) k_kv_weights_chunk<FMT, D, true><<<grid, 256, 0, st>>>(a, p, tiles);
  else k_kv_weights_chunk<FMT, D, false><<<grid, 256, 0, st>>>(a, p, tiles);
}

#define FP8BLK_BY_SHAPE(fn)                                                                  \
  if (a.fmt == FMT_E4M3) {                                                                   \
    D == 64 ? fn<FMT_E4M3, 64>(a, p, st) : D == 128 ? fn<FMT_E4M3, 128>(a, p, st) : fn<FMT_E4M3, 256>(a, p, st); \
  } else {                                                                                   \
    D == 64 ? fn<FMT_E5M2, 64>(a, p, st) : D == 128 ? fn<FMT_E5M2, 128>(a, p, st) : fn<FMT_E5M2, 256>(a, p, st); \
  }

void launch_kv_chunk(const KvAttnArgs& a, const KvPlan& p, int D, hipStream_t st) { FP8BLK_BY_SHAPE(launch) }
void launch_kv_chunk_weights(const KvAttnArgs& a, const KvPlan& p, int D, hipStream_t st) { FP8BLK_BY_SHAPE(launch_weights) }

}  // namespace fp8blk
