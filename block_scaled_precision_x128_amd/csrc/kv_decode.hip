// Attention over the paged FP8 cache for few query rows: a decode step or a
// few drafted tokens (at most 32 rows = query tokens x heads of a kv head, 16
// for heads of 256).
//
// Mathematics: one pass over the positions with a running reference m (near the
// maximum), sum l and output o per row.  The positions are split over
// workgroups, and k_kv_finish joins the parts: with M the largest m_s,
// o = sum 2^(m_s - M) o_s / sum 2^(m_s - M) l_s.
//
// Bound: HBM.  A position costs 2 head_dim bytes a kv head and 4 head_dim
// flops a row, far below the matrix cores' rate at 32 rows, so everything is
// arranged for bytes in flight (32 sequences of 8192 positions, 8 heads of 128:
// 537 MB in 101 us, 5.3 TB/s): no LDS and no barrier in the loop; a wave takes
// 32 positions a step and has two steps in flight behind the one it computes
// (one step: 126 us against 120, before the heads stood side by side), and the
// codes go from the load to the matrix instruction's registers by conversion
// alone:
//   S^T = K Q^T   16x16x32, K as the first operand: its rows are positions and
//                 a lane's 8 k-values are 8 consecutive codes of one row
//   O^T = V^T P^T the k-values are positions.  S^T leaves position 4 g + i of
//                 tile T in register i of lane group g, so the k-order
//                 (T, g, i) is taken for P^T as it lies; V^T wants 8 positions
//                 of one channel in a lane, which a 4x4 byte transpose of the
//                 codes gives before the conversion (8 permutes for 16 codes).
// A lane's channels of V^T are (D/16) l + t for tile t, so that it loads D/16
// consecutive codes of each row and in the end owns D/4 consecutive outputs.
#include <math.h>

#include "attention.h"
#include "attention_common.h"
#include "kv_attention.h"

namespace fp8blk {

namespace {

constexpr int kWaves = 4;

template <int D>
struct VWord {
  typedef uint32_t type __attribute__((ext_vector_type(D / 64)));
};
template <>
struct VWord<64> {
  typedef uint32_t type;
};
template <int D>
__device__ __forceinline__ uint32_t vword(const typename VWord<D>::type& v, int i) {
  if constexpr (D == 64) return v;
  else return v[i];
}
template <int D>
__device__ __forceinline__ void clear_bits(typename VWord<D>::type& v, int i, uint32_t bits) {
  if constexpr (D == 64) v &= ~bits;
  else v[i] &= ~bits;
}

// The codes of 32 positions as one lane holds them.
template <int D>
struct Codes {
  u32x4 k[2][D / 64];                 // rows (lane & 15) and 16 + (lane & 15), 16 codes at 64 c + 16 g
  typename VWord<D>::type v[8];       // rows 4 g + i and 16 + 4 g + i, D/16 codes at (D/16) (lane & 15)
  uint32_t live;                      // bit j: position j is in the range and in the pool
};

template <int D>
__device__ __forceinline__ void load_codes(const KvAttnArgs& a, int slot, int kh, Codes<D>& x) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  x.live = (uint32_t)__ballot(slot >= 0);
  const int s = slot < 0 ? 0 : slot;  // a row of the pool, masked later
  const uint32_t row = (uint32_t)a.kv_heads * D;
  const uint8_t *k = a.k + kh * D + 16 * g, *v = a.v + kh * D + (D / 16) * r;
#pragma unroll
  for (int T = 0; T < 2; ++T) {
    const uint8_t* p = k + (uint64_t)(uint32_t)__shfl(s, 16 * T + r) * row;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) x.k[T][c] = *(const u32x4*)(p + 64 * c);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int pos = (i >> 2) * 16 + 4 * g + (i & 3);
    x.v[i] = *(const typename VWord<D>::type*)(v + (uint64_t)(uint32_t)__shfl(s, pos) * row);
  }
}

template <int FMT, int D, int NQ, bool SPLITQ, bool SPLITP>
__global__ void __launch_bounds__(64 * kWaves, D * NQ >= 256 ? 1 : 2) k_kv_decode(KvAttnArgs a, KvPlan p) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int HW = p.head_waves, KW = kWaves / HW, groups = a.kv_heads / HW;
  const int warp = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wave = warp / HW;
  const int kh = blockIdx.x % groups * HW + warp % HW;
  const int64_t b = blockIdx.x / groups % a.batch;
  const int split = (int)(blockIdx.x / groups / a.batch);
  const int G = a.heads / a.kv_heads;
  const Span sp = span_of(a.q_starts, a.kv_lens, b, a.q_tokens, a.max_kv);
  const int n = sp.n < a.max_q ? sp.n : (int)a.max_q, rows = n * G;
  const int L = a.num_slots > 0 ? sp.L : 0;
  const int j0 = split * p.split_len;
  if (rows == 0 || (j0 >= L && split > 0)) return;
  const int j1 = L - j0 < p.split_len ? L : j0 + p.split_len;
  const int64_t* table = a.table + b * a.max_blocks;

  // Row q of the tile: query token q / G, head q % G of the kv head.
  constexpr int KS = D / 32;
  h8 qh[NQ][KS], ql[SPLITQ ? NQ : 1][KS];
  float c[NQ];                        // raw product -> score in powers of two
  int limit[NQ];                      // positions the row sees
#pragma unroll
  for (int u = 0; u < NQ; ++u) {
    const int q = 16 * u + r, at = q < rows ? q : 0, i = (int)div_by(at, p.group), h = kh * G + at - i * G;
    limit[u] = q < rows ? sp.L - sp.n + i + 1 : 0;
    float y[D / 64][16], x[D / 4], top = 0.0f;
    load_pieces<D / 64, 16, 64>(a.q, a.q_dt, (int64_t)(sp.t0 + i) * a.ld_q + h * D + 16 * g,
                                a.sk == 2 ? a.ks + kh * D + 16 * g : nullptr, y);
#pragma unroll
    for (int k = 0; k < D / 4; ++k) {
      x[k] = q < rows ? y[k / 16][k % 16] : 0.0f;
      top = fmaxf(top, fabsf(x[k]));
    }
    const int e = row_exponent(max_rows(top));
    c[u] = ldexpf(a.scale * kLog2e * (a.sk == 2 ? 1.0f : a.ks[a.sk == 1 ? kh : 0]), e - 14);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = ldexpf(x[8 * s + j], 14 - e);
        const _Float16 hi = (_Float16)y;
        qh[u][s][j] = hi;
        if constexpr (SPLITQ) ql[u][s][j] = (_Float16)(y - (float)hi);
      }
  }

  v4f o[NQ][D / 16];
  float m[NQ], l[NQ];
#pragma unroll
  for (int u = 0; u < NQ; ++u) {
    m[u] = kNoMax;
    l[u] = 0.0f;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) o[u][t] = v4f{0, 0, 0, 0};
  }

  const int steps = (j1 - j0 + 31) / 32;
  // every row sees the positions below this one
  const int seen_by_all = sp.L - sp.n + 1;
  auto look_up = [&](int step) {
    const int j = j0 + 32 * step + (lane & 31);
    return step < steps && j < j1 ? slot_of(table, (uint32_t)j, p.page, (int)a.num_slots) : -1;
  };
  uint32_t odd = 0;
  // Two steps are in flight behind the one computed.  A step's page entries are
  // asked for before the codes of the step in front of it: loads return in
  // order, so that waiting for the entries leaves those codes in flight.
  auto compute = [&](Codes<D>& x_, int step) {
    const int base = j0 + 32 * step;

    v4f s[NQ][2];
#pragma unroll
    for (int T = 0; T < 2; ++T) {
#pragma unroll
      for (int u = 0; u < NQ; ++u) s[u][T] = v4f{0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const u32x4 w = x_.k[T][k / 2];
        const h8 kk = k & 1 ? codes_to_h8<FMT>(w[2], w[3]) : codes_to_h8<FMT>(w[0], w[1]);
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
          s[u][T] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kk, qh[u][k], s[u][T], 0, 0, 0);
          if constexpr (SPLITQ) s[u][T] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kk, ql[u][k], s[u][T], 0, 0, 0);
        }
      }
    }
    const bool whole = x_.live == 0xffffffffu && base + 32 <= seen_by_all;
    if (!whole) {
      // codes of dead positions may be NaN: no product with them is formed
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int pos = (i >> 2) * 16 + 4 * g + (i & 3);
        if (!(x_.live >> pos & 1)) x_.v[i] = typename VWord<D>::type{};
      }
      // nor with NaN or Inf values that some row does not see: p = 0 would
      // carry them into it; the rows that do see them get them at the end
      if (base + 32 > seen_by_all) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            const uint32_t m_ = odd_codes<FMT>(vword<D>(x_.v[i], w));
            odd |= m_;
            clear_bits<D>(x_.v[i], w, m_);
          }
      }
    }
    h8 ph[NQ], pl[SPLITP ? NQ : 1];
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
      float x[8], top = kNoMax;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = s[u][i >> 2][i & 3] * c[u];
        if (!whole) {
          const int pos = (i >> 2) * 16 + 4 * g + (i & 3);
          if (!(x_.live >> pos & 1) || base + pos >= limit[u]) x[i] = -INFINITY;
        }
        top = fmaxf(top, x[i]);
      }
      if (p.scores && 16 * u + r < rows) {
        float* to = p.scores + ((b * a.kv_heads + kh) * p.score_rows + 16 * u + r) * p.score_ld + base + 4 * g;
        *(v4f*)to = v4f{x[0], x[1], x[2], x[3]};
        *(v4f*)(to + 16) = v4f{x[4], x[5], x[6], x[7]};
      }
      if (__any(top > m[u] + kRefMove)) {
        const float mn = fmaxf(m[u], max_rows(top) - kRefBelow);
        const float f = __builtin_amdgcn_exp2f(m[u] - mn);
        m[u] = mn;
        l[u] *= f;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) o[u][t] *= f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = __builtin_amdgcn_exp2f(x[i] - m[u]);
        l[u] += x[i];
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const h2 y = pack_f16(x[i], x[i + 1]);
        ph[u][i] = y[0];
        ph[u][i + 1] = y[1];
        if constexpr (SPLITP) {
          const h2 z = pack_f16(x[i] - (float)y[0], x[i + 1] - (float)y[1]);
          pl[u][i] = z[0];
          pl[u][i + 1] = z[1];
        }
      }
    }
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
      uint32_t lo[4], hi[4];
      transpose4(vword<D>(x_.v[0], w), vword<D>(x_.v[1], w), vword<D>(x_.v[2], w), vword<D>(x_.v[3], w), lo);
      transpose4(vword<D>(x_.v[4], w), vword<D>(x_.v[5], w), vword<D>(x_.v[6], w), vword<D>(x_.v[7], w), hi);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const h8 vv = codes_to_h8<FMT>(lo[t], hi[t]);
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
          o[u][4 * w + t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, ph[u], o[u][4 * w + t], 0, 0, 0);
          if constexpr (SPLITP)
            o[u][4 * w + t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vv, pl[u], o[u][4 * w + t], 0, 0, 0);
        }
      }
    }
  };
  int slot = look_up(wave), ahead = look_up(wave + KW);
  Codes<D> buf[3];
  auto fetch = [&](Codes<D>& to, int step) {
    const int next = look_up(step + 2 * KW);
    if (step < steps) load_codes<D>(a, slot, kh, to);
    slot = ahead;
    ahead = next;
  };
  fetch(buf[0], wave);
  fetch(buf[1], wave + KW);
  for (int step = wave; step < steps; step += 3 * KW) {
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      const int at = step + u * KW;
      if (at >= steps) break;
      fetch(buf[(u + 2) % 3], at + 2 * KW);
      compute(buf[u], at);
    }
  }

  if (__any(odd != 0)) {
    for (int step = wave; step < steps; step += KW)
      for (int j = j0 + 32 * step; j < min(j0 + 32 * step + 32, j1); ++j) {
        const int slot = slot_of(table, (uint32_t)j, p.page, (int)a.num_slots);
        if (j0 + 32 * step + 32 <= seen_by_all || slot < 0) continue;
        const uint8_t* v = a.v + ((int64_t)slot * a.kv_heads + kh) * D + D / 4 * g;
#pragma unroll
        for (int e = 0; e < D / 4; e += 4) {
          const uint32_t w = *(const uint32_t*)(v + e);
          const v2f lo = decode2<FMT>(w, false), hi = decode2<FMT>(w, true);
          const float x[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int u = 0; u < NQ; ++u)
              if (j < limit[u] && !(fabsf(x[k]) < INFINITY)) o[u][(e + k) % (D / 16)][(e + k) / (D / 16)] += x[k];
        }
      }
  }

  // Join the waves of a head: a common reference, then the upper half of them
  // hand their sums to the lower, in that order always.
  __shared__ float red_m[kWaves][NQ][16], red_l[2][NQ][64];
  __shared__ v4f red_o[2][NQ][D / 16][64];
  if (KW > 1) {
#pragma unroll
    for (int u = 0; u < NQ; ++u)
      if (g == 0) red_m[warp][u][r] = m[u];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NQ; ++u) {
      float top = m[u];
      for (int w = warp % HW; w < kWaves; w += HW) top = fmaxf(top, red_m[w][u][r]);
      const float f = __builtin_amdgcn_exp2f(m[u] - top);
      m[u] = top;
      l[u] *= f;
#pragma unroll
      for (int t = 0; t < D / 16; ++t) o[u][t] *= f;
    }
    for (int half = KW / 2; half >= 1; half /= 2) {
      const int slot = (wave - half) * HW + warp % HW;
      if (wave >= half && wave < 2 * half) {
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
          red_l[slot][u][lane] = l[u];
#pragma unroll
          for (int t = 0; t < D / 16; ++t) red_o[slot][u][t][lane] = o[u][t];
        }
      }
      __syncthreads();
      if (wave < half) {
#pragma unroll
        for (int u = 0; u < NQ; ++u) {
          l[u] += red_l[slot + half * HW][u][lane];
#pragma unroll
          for (int t = 0; t < D / 16; ++t) o[u][t] += red_o[slot + half * HW][u][t][lane];
        }
      }
      __syncthreads();
    }
  }
  if (wave != 0) return;
#pragma unroll
  for (int u = 0; u < NQ; ++u) {
    const int q = 16 * u + r;
    const float sum = sum_rows(l[u]);
    if (q >= rows) continue;
    const int i = (int)div_by(q, p.group), h = kh * G + q - i * G;
    const int64_t row = (int64_t)(sp.t0 + i) * a.heads + h;
    const int d0 = D / 4 * g;
    if (p.splits > 1) {
      float* po = p.part_o + (split * p.part_rows + row) * D + d0;
#pragma unroll
      for (int e = 0; e < D / 4; e += 4) {
        v4f y;
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = o[u][(e + k) % (D / 16)][(e + k) / (D / 16)];
        *(v4f*)(po + e) = y;
      }
      if (g == 0) p.part_ml[split * p.part_rows + row] = v2f{m[u], sum};
      continue;
    }
    if (p.scores && g == 0) p.part_ml[row] = v2f{m[u], sum};
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    float y[D / 4];
#pragma unroll
    for (int e = 0; e < D / 4; ++e)
      y[e] = o[u][e % (D / 16)][e / (D / 16)] * inv * kv_scale(a.vs, a.sk, kh, D, d0 + e);
    if (a.out_dt == DT_BF16) {
      u32x4* to = (u32x4*)((uint16_t*)a.out + row * D + d0);
#pragma unroll
      for (int e = 0; e < D / 4; e += 8)
        to[e / 8] = u32x4{pack_bf16(y[e], y[e + 1]), pack_bf16(y[e + 2], y[e + 3]), pack_bf16(y[e + 4], y[e + 5]),
                          pack_bf16(y[e + 6], y[e + 7])};
    } else {
      v4f* to = (v4f*)((float*)a.out + row * D + d0);
#pragma unroll
      for (int e = 0; e < D / 4; e += 4) to[e / 4] = v4f{y[e], y[e + 1], y[e + 2], y[e + 3]};
    }
    if (g == 0 && p.lse) p.lse[row] = sum != 0.0f ? (m[u] + __log2f(sum)) * kLn2 : -INFINITY;
  }
}

}  // namespace

template <int FMT, int D, int NQ>
static void launch(const KvAttnArgs& a, const KvPlan& p, hipStream_t st) {
  const unsigned grid = (unsigned)(a.batch * (a.kv_heads / p.head_waves) * p.splits);
  const bool sq = a.q_dt == DT_F32 || a.sk == 2, so = a.out_dt == DT_F32;
  if (sq && so) k_kv_decode<FMT, D, NQ, true, true><<<grid, 64 * kWaves, 0, st>>>(a, p);
  else if (sq) k_kv_decode<FMT, D, NQ, true, false><<<grid, 64 * kWaves, 0, st>>>(a, p);
  else if (so) k_kv_decode<FMT, D, NQ, false, true><<<grid, 64 * kWaves, 0, st>>>(a, p);
  else k_kv_decode<FMT, D, NQ, false, false><<<grid, 64 * kWaves, 0, st>>>(a, p);
}

template <int FMT>
static void launch_fmt(const KvAttnArgs& a, const KvPlan& p, int D, hipStream_t st) {
  const bool two = a.max_q * (a.heads / a.kv_heads) > 16;
  if (D == 64) two ? launch<FMT, 64, 2>(a, p, st) : launch<FMT, 64, 1>(a, p, st);
  else if (D == 128) two ? launch<FMT, 128, 2>(a, p, st) : launch<FMT, 128, 1>(a, p, st);
  else launch<FMT, 256, 1>(a, p, st);
}

void launch_kv_decode(const KvAttnArgs& a, const KvPlan& p, int D, hipStream_t st) {
  a.fmt == FMT_E4M3 ? launch_fmt<FMT_E4M3>(a, p, D, st) : launch_fmt<FMT_E5M2>(a, p, D, st);
}

}  // namespace fp8blk
