// Softmax attention of new tokens over the paged FP8 KV cache, plain form:
// one wave per (query token, head), fp32 throughout, two passes over the
// visible positions (max and sum, then the products with the values).
#include <math.h>

#include "attention.h"
#include "device_common.h"

namespace fp8blk {

namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// Slot of position j of sequence b, or -1 outside the pool.
__device__ __forceinline__ int64_t slot_of(const KvAttnArgs& a, int64_t b, int64_t j) {
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
    const int64_t s = slot_of(a, b, j);
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
  const int64_t t0 = a.q_starts[b], n = a.q_starts[b + 1] - t0, s = slot_of(a, b, j);
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
hipError_t launch(const KvAttnArgs& a, hipStream_t st) {
  float* lse = a.lse ? a.lse : (float*)a.ws;
  if (a.q_tokens > 0)
    k_kv_attention<FMT, D><<<dim3((unsigned)a.q_tokens, (unsigned)a.heads), 64, 0, st>>>(a, lse);
  if (a.w_out && a.max_kv > 0)
    k_kv_weights<FMT, D><<<dim3((unsigned)a.max_kv, (unsigned)a.kv_heads, (unsigned)a.batch), 64, 0, st>>>(a, lse);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_fmt(const KvAttnArgs& a, int D, hipStream_t st) {
  return D == 64 ? launch<FMT, 64>(a, st) : D == 128 ? launch<FMT, 128>(a, st) : launch<FMT, 256>(a, st);
}

}  // namespace

size_t kv_attention_workspace(int64_t q_tokens, int64_t heads, int64_t, int, int64_t, int64_t, int64_t,
                              bool with_weights) {
  return with_weights ? (size_t)(q_tokens * heads) * sizeof(float) : 0;
}

bool kv_attention_fits(int64_t heads, int64_t, int64_t batch, int64_t, int64_t) {
  return heads < 65536 && batch < 65536;
}

hipError_t launch_kv_attention(const KvAttnArgs& a, int head_dim, hipStream_t st) {
  return a.fmt == FMT_E4M3 ? launch_fmt<FMT_E4M3>(a, head_dim, st) : launch_fmt<FMT_E5M2>(a, head_dim, st);
}

}  // namespace fp8blk
