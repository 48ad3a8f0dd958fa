// Causal attention of packed prompts over bf16 states, plain form: one wave
// per (token, head), fp32 throughout.
#include <math.h>

#include "attention.h"
#include "device_common.h"

namespace fp8blk {

namespace {

template <int D>
__global__ void __launch_bounds__(64) k_prompt(PromptArgs a) {
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, lane = threadIdx.x, kh = h / (a.heads / a.kv_heads);
  int64_t b = 0;
  while (b < a.batch && !(t >= a.starts[b] && t < a.starts[b + 1])) ++b;
  if (b == a.batch || t - a.starts[b] >= a.max_len) return;
  constexpr int P = D / 64;
  float q[P], o[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    q[p] = bf16lo(a.q[t * a.ld_q + h * D + lane + 64 * p]);
    o[p] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = a.starts[b]; j <= t; ++j) {
    float x = 0.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) x += q[p] * bf16lo(a.k[j * a.ld_k + kh * D + lane + 64 * p]);
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) x += __shfl_xor(x, s);
    x *= a.scale;
    const float mn = fmaxf(m, x), c = expf(m - mn), e = expf(x - mn);
    m = mn;
    l = l * c + e;
#pragma unroll
    for (int p = 0; p < P; ++p) o[p] = o[p] * c + e * bf16lo(a.v[j * a.ld_v + kh * D + lane + 64 * p]);
  }
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t u = __float_as_uint(o[p] / l);
    a.out[(t * a.heads + h) * D + lane + 64 * p] =
        (u & 0x7fffffffu) > 0x7f800000u ? (uint16_t)((u >> 16) | 0x40) : (uint16_t)((u + 0x7fffu + ((u >> 16) & 1)) >> 16);
  }
  if (a.lse && lane == 0) a.lse[t * a.heads + h] = m + logf(l);
}

}  // namespace

bool prompt_attention_fits(int64_t heads, int64_t, int64_t, int64_t) { return heads < 65536; }

hipError_t launch_prompt_attention(const PromptArgs& a, int head_dim, hipStream_t st) {
  const dim3 g((unsigned)a.tokens, (unsigned)a.heads);
  if (head_dim == 64) k_prompt<64><<<g, 64, 0, st>>>(a);
  else if (head_dim == 128) k_prompt<128><<<g, 64, 0, st>>>(a);
  else k_prompt<256><<<g, 64, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace fp8blk
