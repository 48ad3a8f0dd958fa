// fp8_kv_attention: how a call is split and which kernels it takes, the kernel
// that joins the splits, and the collection of the attention weights.
#include <math.h>

#include "attention.h"
#include "attention_common.h"
#include "kv_attention.h"

namespace fp8blk {

namespace {

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Splits of the positions.  A launch should have about four workgroups a CU
// for its loads to fill the memory system; a split is at least 128 positions
// (one step of each of a workgroup's four waves), and there are at most 128 of
// them, which bounds the joining kernel's work.
void plan_splits(int64_t units, int64_t max_kv, KvPlan& p) {
  constexpr int64_t kGroups = 1024, kStep = 128, kMost = 128;
  int64_t n = units > 0 ? (kGroups + units - 1) / units : 1;
  const int64_t steps = (max_kv + kStep - 1) / kStep;
  n = n > kMost ? kMost : n;
  n = n > steps ? steps : n;
  n = n < 1 ? 1 : n;
  const int64_t len = round_up((max_kv + n - 1) / n, kStep);
  p.split_len = (int)(len > 0 ? len : kStep);
  p.splits = (int)((max_kv + p.split_len - 1) / p.split_len);
  if (p.splits < 1) p.splits = 1;
}

bool is_decode(int64_t heads, int64_t kv_heads, int head_dim, int64_t max_q) {
  return max_q * (heads / kv_heads) <= decode_rows(head_dim);
}

struct Parts {
  size_t lse, ml, o, scores, bytes;
};

// Lays the workspace out; what a call does not need takes no room.
Parts lay_out(KvPlan& p, int64_t q_tokens, int64_t heads, int64_t kv_heads, int head_dim, int64_t batch, int64_t max_q,
              int64_t max_kv, bool with_weights) {
  const bool decode = is_decode(heads, kv_heads, head_dim, max_q);
  if (decode) {
    plan_splits(batch * kv_heads, max_kv, p);
  } else {
    p.splits = 1;
    p.split_len = (int)max_kv;
  }
  p.part_rows = q_tokens * heads;
  p.score_rows = decode && with_weights ? max_q * (heads / kv_heads) : 0;
  p.score_ld = (int64_t)p.splits * p.split_len;
  Parts at{};
  size_t n = 0;
  auto take = [&](size_t bytes) {
    const size_t here = n;
    n += (bytes + 255) / 256 * 256;
    return here;
  };
  at.lse = take(with_weights ? p.part_rows * sizeof(float) : 0);
  at.ml = take(p.splits > 1 ? p.splits * p.part_rows * sizeof(v2f) : 0);
  at.o = take(p.splits > 1 ? p.splits * p.part_rows * head_dim * sizeof(float) : 0);
  at.scores = take(batch * kv_heads * p.score_rows * p.score_ld * sizeof(float));
  at.bytes = n;
  return at;
}

// Joins the splits of one (query token, head): wave w takes splits w, w + 4, ..
// and the four partial sums are added in one order.
template <int D>
__global__ void __launch_bounds__(256) k_kv_combine(KvAttnArgs a, KvPlan p) {
  const int64_t per = a.max_q * a.heads, b = blockIdx.x / per;
  const int at = (int)(blockIdx.x % per), i = at / a.heads, h = at - i * a.heads;
  const Span sp = span_of(a.q_starts, a.kv_lens, b, a.q_tokens, a.max_kv);
  if (i >= sp.n) return;
  const int L = a.num_slots > 0 ? sp.L : 0;
  const int n = L > 0 ? (L + p.split_len - 1) / p.split_len : 1;
  const int64_t row = (int64_t)(sp.t0 + i) * a.heads + h;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __shared__ float weight[128], red[4][D];
  __shared__ float s_sum, s_max;
  if (wave == 0) {                         // at most 128 splits
    const v2f x = lane < n ? p.part_ml[lane * p.part_rows + row] : v2f{kNoMax, 0.0f};
    const v2f y = lane + 64 < n ? p.part_ml[(lane + 64) * p.part_rows + row] : v2f{kNoMax, 0.0f};
    float m = fmaxf(x[0], y[0]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    const float wx = __builtin_amdgcn_exp2f(x[0] - m), wy = __builtin_amdgcn_exp2f(y[0] - m);
    float l = wx * x[1] + wy * y[1];
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) l += __shfl_xor(l, o);
    weight[lane] = wx;
    weight[lane + 64] = wy;
    if (lane == 0) {
      s_sum = l;
      s_max = m;
    }
  }
  __syncthreads();
  constexpr int P = D / 64;
  float o[P];
#pragma unroll
  for (int e = 0; e < P; ++e) o[e] = 0.0f;
#pragma unroll 8
  for (int s = wave; s < n; s += 4) {
    const float* po = p.part_o + ((int64_t)s * p.part_rows + row) * D + P * lane;
    const float w = weight[s];
#pragma unroll
    for (int e = 0; e < P; ++e) o[e] += w * po[e];
  }
#pragma unroll
  for (int e = 0; e < P; ++e) red[wave][P * lane + e] = o[e];
  __syncthreads();
  const float sum = s_sum, inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  const int kh = h / (a.heads / a.kv_heads);
  for (int d = threadIdx.x; d < D; d += 256) {
    const float y = (((red[0][d] + red[1][d]) + red[2][d]) + red[3][d]) * inv * kv_scale(a.vs, a.sk, kh, D, d);
    if (a.out_dt == DT_BF16) ((uint16_t*)a.out)[row * D + d] = (uint16_t)pack_bf16(y, 0.0f);
    else ((float*)a.out)[row * D + d] = y;
  }
  if (p.lse && threadIdx.x == 0) p.lse[row] = sum > 0.0f ? (s_max + __log2f(sum)) * kLn2 : -INFINITY;
}

// The weights of a decode call, from its scores: one thread a position.
__global__ void __launch_bounds__(256) k_kv_weights_decode(KvAttnArgs a, KvPlan p, int tiles) {
  const int j = (blockIdx.x % tiles) * 256 + threadIdx.x;
  const int64_t bk = blockIdx.x / tiles, b = bk / a.kv_heads;
  const int kh = (int)(bk % a.kv_heads), G = a.heads / a.kv_heads;
  const Span sp = span_of(a.q_starts, a.kv_lens, b, a.q_tokens, a.max_kv);
  if (j >= sp.L) return;
  const int n = sp.n < a.max_q ? sp.n : (int)a.max_q;
  float w = 0.0f;
  if (a.num_slots > 0)
    for (int q = 0; q < n * G; ++q) {
      const int i = (int)div_by(q, p.group);
      const float lse = p.lse[(int64_t)(sp.t0 + i) * a.heads + kh * G + q - i * G];
      const float s = p.scores[(bk * p.score_rows + q) * p.score_ld + j];
      w += lse == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(s - lse * kLog2e);
    }
  const int64_t at = bk * a.ld_w + j;
  a.w_out[at] = (a.w_in ? a.w_in[at] : 0.0f) + w;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// Slot of position j of sequence b, or -1 outside the pool.
__device__ __forceinline__ int64_t slot_of64(const KvAttnArgs& a, int64_t b, int64_t j) {
  const int64_t blk = a.table[b * a.max_blocks + j / a.block_size];
  if (blk < 0 || blk > a.num_slots / a.block_size) return -1;
  const int64_t s = blk * a.block_size + j % a.block_size;
  return s < a.num_slots ? s : -1;
}

__device__ __forceinline__ float scale_of(const float* s, int sk, int kh, int D, int d) {
  return sk == 0 ? s[0] : sk == 1 ? s[kh] : s[kh * D + d];
}

template <int FMT>
__device__ __forceinline__ float code_value(const uint8_t* p) { return decode2<FMT>((uint32_t)*p, false)[0]; }

__device__ __forceinline__ float load_q(const KvAttnArgs& a, int64_t i) {
  return a.q_dt == DT_BF16 ? bf16lo(((const uint16_t*)a.q)[i]) : ((const float*)a.q)[i];
}

__device__ __forceinline__ uint16_t to_bf16(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x7fffffffu) > 0x7f800000u ? (uint16_t)((u >> 16) | 0x40) : (uint16_t)((u + 0x7fffu + ((u >> 16) & 1)) >> 16);
}

// Sequence of token t, or -1.
__device__ __forceinline__ int64_t sequence_of(const int64_t* starts, int64_t batch, int64_t t) {
  for (int64_t b = 0; b < batch; ++b)
    if (t >= starts[b] && t < starts[b + 1]) return b;
  return -1;
}

__device__ __forceinline__ int64_t clamp_len(int64_t n, int64_t top) { return n < 0 ? 0 : n > top ? top : n; }

template <int FMT, int D>
__global__ void __launch_bounds__(64) k_kv_attention(KvAttnArgs a, float* lse) {
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, lane = threadIdx.x, kh = h / (a.heads / a.kv_heads);
  const int64_t b = sequence_of(a.q_starts, a.batch, t);
  if (b < 0) return;
  const int64_t i = t - a.q_starts[b], n = a.q_starts[b + 1] - a.q_starts[b];
  if (i >= a.max_q) return;
  const int64_t L = clamp_len(a.kv_lens[b], a.max_kv);
  const int64_t end = clamp_len(L - n + i + 1, L);
  constexpr int P = D / 64;
  float q[P], o[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int d = lane + 64 * p;
    q[p] = load_q(a, t * a.ld_q + h * D + d) * scale_of(a.ks, a.sk, kh, D, d);
    o[p] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = 0; j < end; ++j) {
    const int64_t s = slot_of64(a, b, j);
    if (s < 0) continue;
    const int64_t at = (s * a.kv_heads + kh) * D + lane;
    float x = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) x += q[p] * code_value<FMT>(a.k + at + 64 * p);
    x = wave_sum(x) * a.scale;
    const float mn = fmaxf(m, x), c = expf(m - mn), e = expf(x - mn);
    m = mn;
    l = l * c + e;
#pragma unroll
    for (int p = 0; p < P; ++p) o[p] = o[p] * c + e * code_value<FMT>(a.v + at + 64 * p);
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int d = lane + 64 * p;
    const float r = l > 0.0f ? o[p] / l * scale_of(a.vs, a.sk, kh, D, d) : 0.0f;
    const int64_t at = (t * a.heads + h) * D + d;
    if (a.out_dt == DT_BF16) ((uint16_t*)a.out)[at] = to_bf16(r);
    else ((float*)a.out)[at] = r;
  }
  if (lse && lane == 0) lse[t * a.heads + h] = m + logf(l);
}

// weights_out of one position: one wave per (position, kv head, sequence).
template <int FMT, int D>
__global__ void __launch_bounds__(64) k_kv_weights(KvAttnArgs a, const float* lse) {
  const int64_t j = blockIdx.x, b = blockIdx.z;
  const int kh = blockIdx.y, lane = threadIdx.x, G = a.heads / a.kv_heads;
  const int64_t L = clamp_len(a.kv_lens[b], a.max_kv);
  if (j >= L) return;
  const int64_t t0 = a.q_starts[b], n = a.q_starts[b + 1] - t0, s = slot_of64(a, b, j);
  constexpr int P = D / 64;
  float w = 0.0f;
  if (s >= 0) {
    float k[P];
#pragma unroll
    for (int p = 0; p < P; ++p)
      k[p] = code_value<FMT>(a.k + (s * a.kv_heads + kh) * D + lane + 64 * p) * scale_of(a.ks, a.sk, kh, D, lane + 64 * p);
    for (int64_t i = 0; i < n && i < a.max_q; ++i) {
      if (j >= L - n + i + 1) continue;
      for (int g = 0; g < G; ++g) {
        const int h = kh * G + g;
        float x = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) x += k[p] * load_q(a, (t0 + i) * a.ld_q + h * D + lane + 64 * p);
        w += expf(wave_sum(x) * a.scale - lse[(t0 + i) * a.heads + h]);
      }
    }
  }
  const int64_t at = (b * a.kv_heads + kh) * a.ld_w + j;
  if (lane == 0) a.w_out[at] = (a.w_in ? a.w_in[at] : 0.0f) + w;
}

template <int FMT, int D>
void launch_chunk(const KvAttnArgs& a, const KvPlan& p, hipStream_t st) {
  if (a.q_tokens > 0)
    k_kv_attention<FMT, D><<<dim3((unsigned)a.q_tokens, (unsigned)a.heads), 64, 0, st>>>(a, p.lse);
  if (a.w_out && a.max_kv > 0)
    k_kv_weights<FMT, D><<<dim3((unsigned)a.max_kv, (unsigned)a.kv_heads, (unsigned)a.batch), 64, 0, st>>>(a, p.lse);
}

template <int FMT>
void launch_chunk_fmt(const KvAttnArgs& a, const KvPlan& p, int D, hipStream_t st) {
  D == 64 ? launch_chunk<FMT, 64>(a, p, st) : D == 128 ? launch_chunk<FMT, 128>(a, p, st) : launch_chunk<FMT, 256>(a, p, st);
}

}  // namespace

size_t kv_attention_workspace(int64_t q_tokens, int64_t heads, int64_t kv_heads, int head_dim, int64_t batch,
                              int64_t max_q, int64_t max_kv, bool with_weights) {
  if (heads == 0 || kv_heads == 0) return 0;
  KvPlan p{};
  return lay_out(p, q_tokens, heads, kv_heads, head_dim, batch, max_q, max_kv, with_weights).bytes;
}

bool kv_attention_fits(int64_t heads, int64_t, int64_t batch, int64_t, int64_t) {
  return heads < 65536 && batch < 65536;
}

hipError_t launch_kv_attention(const KvAttnArgs& a, int head_dim, hipStream_t st) {
  KvPlan p{};
  const Parts at = lay_out(p, a.q_tokens, a.heads, a.kv_heads, head_dim, a.batch, a.max_q, a.max_kv, a.w_out != nullptr);
  uint8_t* ws = (uint8_t*)a.ws;
  p.page = make_fastdiv(a.block_size);
  p.group = make_fastdiv(a.heads / a.kv_heads);
  p.part_ml = (v2f*)(ws + at.ml);
  p.part_o = (float*)(ws + at.o);
  p.lse = a.lse || !a.w_out ? a.lse : (float*)(ws + at.lse);
  p.scores = p.score_rows > 0 ? (float*)(ws + at.scores) : nullptr;
  const bool any_q = a.q_tokens > 0 && a.max_q > 0;
  if (!is_decode(a.heads, a.kv_heads, head_dim, a.max_q)) {
    a.fmt == FMT_E4M3 ? launch_chunk_fmt<FMT_E4M3>(a, p, head_dim, st) : launch_chunk_fmt<FMT_E5M2>(a, p, head_dim, st);
    return hipGetLastError();
  }
  if (any_q) {
    launch_kv_decode(a, p, head_dim, st);
    if (p.splits > 1) {
      const unsigned grid = (unsigned)(a.batch * a.max_q * a.heads);
      if (head_dim == 64) k_kv_combine<64><<<grid, 256, 0, st>>>(a, p);
      else if (head_dim == 128) k_kv_combine<128><<<grid, 256, 0, st>>>(a, p);
      else k_kv_combine<256><<<grid, 256, 0, st>>>(a, p);
    }
  }
  if (a.w_out && a.max_kv > 0) {
    const int tiles = (int)((a.max_kv + 255) / 256);
    k_kv_weights_decode<<<(unsigned)(a.batch * a.kv_heads * tiles), 256, 0, st>>>(a, p, tiles);
  }
  return hipGetLastError();
}

}  // namespace fp8blk
