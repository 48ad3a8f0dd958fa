// Device helpers shared by the attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "paging.h"

namespace fp8blk {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// Below every score: the running maximum before any position was seen.  It is
// finite, so that exp2(-Inf - m) of a masked score is 0 and not NaN.
constexpr float kNoMax = -1e38f;

// p = 2^(score - m) with a reference m that lies kRefBelow under the largest
// score when it is set and is only moved when a score passes it by kRefMove,
// so that the sums are rarely rescaled.  p then reaches 2^15 at most, inside
// fp16, and the largest p is at least 2^7: what fp16 cannot hold (below 2^-24)
// is 2^-31 of it.  The fp32 sums do not depend on the reference.
constexpr float kRefBelow = 7.0f;
constexpr float kRefMove = 15.0f;

// Codes to fp16, exactly: E4M3 spans 2^-9 to 448, E5M2 is fp16's exponent with
// two mantissa bits.
template <int FMT>
__device__ __forceinline__ h2 codes_to_h2(uint32_t w, bool hi) {
  if constexpr (FMT == FMT_E4M3)
    return hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true)
              : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
  else
    return hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(w, 1.0f, true)
              : __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(w, 1.0f, false);
}

template <int FMT>
__device__ __forceinline__ h8 codes_to_h8(uint32_t a, uint32_t b) {
  const h2 x = codes_to_h2<FMT>(a, false), y = codes_to_h2<FMT>(a, true);
  const h2 z = codes_to_h2<FMT>(b, false), w = codes_to_h2<FMT>(b, true);
  return h8{x[0], x[1], y[0], y[1], z[0], z[1], w[0], w[1]};
}

// 0xff in every byte of w that is a NaN or Inf code.
template <int FMT>
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) {
  const uint32_t t = (w & 0x7f7f7f7fu) + (FMT == FMT_E4M3 ? 0x01010101u : 0x04040404u);
  return (t >> 7 & 0x01010101u) * 0xffu;
}

// 0xffff in each half of w that is a NaN or Inf of bf16.
__device__ __forceinline__ uint32_t odd_bf16(uint32_t w) {
  const uint32_t t = (w & 0x7f807f80u) + 0x00800080u;
  return (t >> 15 & 0x00010001u) * 0xffffu;
}

// 4x4 byte transpose: byte c of in[r] becomes byte r of out[c].
__device__ __forceinline__ void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t* out) {
  const uint32_t t0 = __builtin_amdgcn_perm(b, a, 0x05010400u), t1 = __builtin_amdgcn_perm(b, a, 0x07030602u);
  const uint32_t u0 = __builtin_amdgcn_perm(d, c, 0x05010400u), u1 = __builtin_amdgcn_perm(d, c, 0x07030602u);
  out[0] = __builtin_amdgcn_perm(u0, t0, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(u0, t0, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(u1, t1, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(u1, t1, 0x07060302u);
}

// Max / sum over the two halves of a wave (lanes l and l ^ 32), and over the
// four rows of 16 lanes.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float max_rows(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_rows(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Sum over each row of 16 lanes, in all of them.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float sum16(float v) {
  return add_dpp<0x140>(add_dpp<0x141>(add_dpp<0x4E>(add_dpp<0xB1>(v))));
}

// Two floats to packed bf16, nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const v2f x = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, b2));
}

__device__ __forceinline__ h2 pack_f16(float a, float b) {
  const v2f x = {a, b};
  return __builtin_convertvector(x, h2);
}

// C pieces of N values of a row (bf16 or fp32), STEP apart from element `at` on,
// times the factors `by` (laid out as the row, null: none).  One branch around
// all loads: behind a branch of its own each would wait for the one before.
template <int C, int N, int STEP>
__device__ __forceinline__ void load_pieces(const void* q, int dt, int64_t at, const float* by, float (&x)[C][N]) {
  if (dt == DT_BF16) {
    u32x4 w[C][N / 8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < N / 8; ++i) w[c][i] = *(const u32x4*)((const uint16_t*)q + at + STEP * c + 8 * i);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        x[c][2 * i] = bf16lo(w[c][i / 4][i % 4]);
        x[c][2 * i + 1] = bf16hi(w[c][i / 4][i % 4]);
      }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < N / 4; ++i) *(v4f*)&x[c][4 * i] = *(const v4f*)((const float*)q + at + STEP * c + 4 * i);
  }
  if (by) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < N; ++i) x[c][i] *= by[STEP * c + i];
  }
}

// Binary exponent of a row's largest magnitude (0 for a row of zeros): the
// row times 2^(14 - e) lies below 2^15, inside fp16 with 2^-24 as the smallest
// step, and its products with codes below 2^31 (E4M3) or 2^39 (E5M2).
__device__ __forceinline__ int row_exponent(float amax) {
  return amax > 0.0f ? (int)((__float_as_uint(amax) >> 23) & 255) - 127 : 0;
}

// Queries and cache positions of one sequence.
struct Span {
  int t0, n, L;      // first query token, query tokens, positions
};

__device__ __forceinline__ int clip(int64_t x, int64_t lo, int64_t hi) { return (int)(x < lo ? lo : x > hi ? hi : x); }

__device__ __forceinline__ Span span_of(const int64_t* q_starts, const int64_t* kv_lens, int64_t b, int64_t q_tokens,
                                        int64_t max_kv) {
  Span s;
  s.t0 = clip(q_starts[b], 0, q_tokens);
  s.n = clip(q_starts[b + 1], s.t0, q_tokens) - s.t0;
  s.L = clip(kv_lens ? kv_lens[b] : s.n, 0, max_kv);       // without lengths a sequence's positions are its tokens
  return s;
}

constexpr int kNoScale = 3;           // beside the kinds of scales of the cache: values as they are

__device__ __forceinline__ float kv_scale(const float* s, int sk, int kh, int D, int d) {
  return sk == kNoScale ? 1.0f : sk == 0 ? s[0] : sk == 1 ? s[kh] : s[kh * D + d];
}

}  // namespace fp8blk
