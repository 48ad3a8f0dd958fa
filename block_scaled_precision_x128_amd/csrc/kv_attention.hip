// fp8_kv_attention: how a call is split and which kernels it takes, the kernel
// that joins the splits, and the collection of the attention weights.
#include <math.h>

#include "attention.h"
#include "attention_common.h"
#include "kv_attention.h"

namespace fp8blk {

namespace {

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

constexpr int64_t kMostSplits = 128;

}  // namespace

// At most `groups` workgroups in all, one round of them (a few more would run
// behind the others: 17 x 116 on 1024, 544 workgroups in splits of 256: 41 us,
// 34 with 408 in splits of 384), of at least `least` positions each in
// multiples of `grain`, and at most kMostSplits, which bounds the joining
// kernel's work.  More than half a round of workgroups take two long parts all
// the same: the sequences of a batch differ, and the longest one's workgroups
// are what is waited for (6 x 301 on 3001, ragged: 168 us against 183).
void plan_splits(int64_t units, int64_t groups, int64_t least, int64_t grain, int64_t max_kv, KvPlan& p) {
  int64_t n = units > 0 ? groups / units : 1;
  if (n == 1 && units < groups && max_kv >= 2048) n = 2;
  n = n > kMostSplits ? kMostSplits : n;
  n = n > max_kv / least ? max_kv / least : n;
  n = n < 1 ? 1 : n;
  const int64_t len = round_up((max_kv + n - 1) / n, grain);
  p.split_len = (int)(len > 0 ? len : grain);
  p.splits = (int)((max_kv + p.split_len - 1) / p.split_len);
  if (p.splits < 1) p.splits = 1;
}

namespace {

bool is_decode(int64_t heads, int64_t kv_heads, int head_dim, int64_t max_q) {
  return max_q * (heads / kv_heads) <= decode_rows(head_dim);
}

struct Parts {
  size_t lse, ml, o, scores, queries, factors, bytes;
};

// Lays the workspace out; what a call does not need takes no room.
Parts lay_out(KvPlan& p, int64_t q_tokens, int64_t heads, int64_t kv_heads, int head_dim, int64_t batch, int64_t max_q,
              int64_t max_kv, bool with_weights) {
  const bool decode = is_decode(heads, kv_heads, head_dim, max_q);
  const int64_t bk = batch * kv_heads;
  // Decode: two workgroups a CU keep the loads that fill the memory system in
  // flight.  A wave takes at least four steps of 32 positions: below that the
  // joining launch costs more than the split gains (32 sequences of 1000: 21.7
  // us, 26.5 with splits of 128).  The four waves are neighbouring kv heads
  // where that still leaves 512 workgroups, since the heads of a position lie
  // side by side in memory (32 sequences of 8k, 8 heads of 128: 106 us against
  // 120 with a head a workgroup; 8 of 32k, heads of 64: 67 against 90), and else
  // they share a head's positions, which needs no launch to join them.
  // Chunk: two workgroups fit a CU, and a split should be several tiles long
  // (1 x 512 on 8k: 99 us with 512 workgroups wanted, 117 with 1024, 162 with
  // 256; 17 x 116 on 768 in splits of 256: 32 us, in halves 38).
  p.head_waves = 1;
  if (decode) {
    constexpr int64_t kGroups = 512;
    for (int hw = 4; hw > 1 && p.head_waves == 1; hw /= 2) {
      const int64_t splits = max_kv / (512 / hw);
      if (kv_heads % hw == 0 && bk / hw * (splits < kMostSplits ? splits : kMostSplits) >= kGroups) p.head_waves = hw;
    }
    plan_splits(bk / p.head_waves, kGroups, 512 / p.head_waves, 128 / p.head_waves, max_kv, p);
  } else {
    plan_splits(bk * kv_chunk_tiles(heads, kv_heads, max_q), 512, 256, 64, max_kv, p);
  }
  p.part_rows = q_tokens * heads;
  p.score_rows = decode && with_weights ? max_q * (heads / kv_heads) : 0;
  p.score_ld = (int64_t)p.splits * p.split_len;
  p.row_tiles = !decode && with_weights ? (max_q * (heads / kv_heads) + 31) / 32 : 0;
  Parts at{};
  size_t n = 0;
  auto take = [&](size_t bytes) {
    const size_t here = n;
    n += (bytes + 255) / 256 * 256;
    return here;
  };
  at.lse = take(with_weights ? p.part_rows * sizeof(float) : 0);
  at.ml = take(p.splits > 1 || p.score_rows > 0 ? p.splits * p.part_rows * sizeof(v2f) : 0);
  at.o = take(p.splits > 1 ? p.splits * p.part_rows * head_dim * sizeof(float) : 0);
  at.scores = take(bk * p.score_rows * p.score_ld * sizeof(float));
  at.queries = take(bk * p.row_tiles * 32 * head_dim * 4);        // two fp16 halves
  at.factors = take(bk * p.row_tiles * 32 * sizeof(float));
  at.bytes = n;
  return at;
}

// Joins the splits of a (query token, head).
constexpr int kFewSplits = 8;

template <int D>
__device__ __forceinline__ void store_joined(const KvAttnArgs& a, int64_t row, int kh, int d, const v4f& o, float inv) {
  v4f y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = o[e] * inv * kv_scale(a.vs, a.sk, kh, D, d + e);
  if (a.out_dt == DT_F32) *(v4f*)((float*)a.out + row * D + d) = y;
  else *(u32x2*)((uint16_t*)a.out + row * D + d) = u32x2{pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
}

__device__ __forceinline__ float joined_lse(float m, float sum) {
  return sum != 0.0f ? (m + __log2f(sum)) * kLn2 : -INFINITY;
}

// Few splits: D/4 lanes a row, four channels each, every split's sums in flight.
template <int D>
__device__ __forceinline__ void combine_few(const KvAttnArgs& a, const KvPlan& p, int64_t block) {
  constexpr int kLanes = D / 4, kRows = 256 / kLanes;
  const int64_t per = (a.max_q * a.heads + kRows - 1) / kRows, b = block / per;
  const int at = (int)(block % per) * kRows + threadIdx.x / kLanes, i = at / a.heads, h = at - i * a.heads;
  const int d = threadIdx.x % kLanes * 4;
  const Span sp = span_of(a.q_starts, a.kv_lens, b, a.q_tokens, a.max_kv);
  if (i >= sp.n || i >= a.max_q) return;
  const int L = a.num_slots > 0 ? sp.L : 0;
  const int n = L > 0 ? (L + p.split_len - 1) / p.split_len : 1;
  const int64_t row = (int64_t)(sp.t0 + i) * a.heads + h;
  v2f ml[kFewSplits];
  v4f part[kFewSplits];
  float m = kNoMax;
#pragma unroll
  for (int s = 0; s < kFewSplits; ++s) {
    ml[s] = s < n ? p.part_ml[s * p.part_rows + row] : v2f{kNoMax, 0.0f};
    if (s < n) part[s] = *(const v4f*)(p.part_o + (s * p.part_rows + row) * D + d);
    m = fmaxf(m, ml[s][0]);
  }
  v4f o = {0, 0, 0, 0};
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < kFewSplits; ++s) {
    // a split in which the row sees nothing may not have written its sums
    const bool some = ml[s][1] != 0.0f;
    const float w = some ? __builtin_amdgcn_exp2f(ml[s][0] - m) : 0.0f;
    sum += w * ml[s][1];
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += some ? w * part[s][e] : 0.0f;
  }
  store_joined<D>(a, row, h / (a.heads / a.kv_heads), d, o, sum != 0.0f ? 1.0f / sum : 0.0f);
  if (p.lse && d == 0) p.lse[row] = joined_lse(m, sum);
}

// Many splits: a workgroup a row, its waves take every fourth split and their
// sums are added in one order.
template <int D>
__device__ __forceinline__ void combine_many(const KvAttnArgs& a, const KvPlan& p, int64_t block) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t per = a.max_q * a.heads, b = block / per;
  const int at = (int)(block % per), i = at / a.heads, h = at - i * a.heads;
  const Span sp = span_of(a.q_starts, a.kv_lens, b, a.q_tokens, a.max_kv);
  if (i >= sp.n) return;
  const int L = a.num_slots > 0 ? sp.L : 0;
  const int n = L > 0 ? (L + p.split_len - 1) / p.split_len : 1;       // at most 128
  const int64_t row = (int64_t)(sp.t0 + i) * a.heads + h;
  const v2f none = {kNoMax, 0.0f};
  const v2f x = lane < n ? p.part_ml[lane * p.part_rows + row] : none;
  const v2f y = lane + 64 < n ? p.part_ml[(lane + 64) * p.part_rows + row] : none;
  float m = fmaxf(x[0], y[0]);
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
  const float wx = x[1] != 0.0f ? __builtin_amdgcn_exp2f(x[0] - m) : 0.0f;
  const float wy = y[1] != 0.0f ? __builtin_amdgcn_exp2f(y[0] - m) : 0.0f;
  float sum = wx * x[1] + wy * y[1];
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o);
  constexpr int P = D / 64, U = 8;
  float o[P];
#pragma unroll
  for (int e = 0; e < P; ++e) o[e] = 0.0f;
  for (int s0 = wave; s0 < n; s0 += 4 * U) {
    float w[U], part[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u) {                    // eight splits' loads in flight
      const int s = s0 + u * 4;
      const int lo = __builtin_amdgcn_readlane(__float_as_int(wx), s & 63);
      const int hi = __builtin_amdgcn_readlane(__float_as_int(wy), s & 63);
      w[u] = s >= n ? 0.0f : __int_as_float(s < 64 ? lo : hi);
      if (w[u] != 0.0f) {
        const float* po = p.part_o + ((int64_t)s * p.part_rows + row) * D + P * lane;
#pragma unroll
        for (int e = 0; e < P; ++e) part[u][e] = po[e];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < P; ++e) o[e] += w[u] != 0.0f ? w[u] * part[u][e] : 0.0f;
  }
  __shared__ alignas(16) float red[4][D];
#pragma unroll
  for (int e = 0; e < P; ++e) red[wave][P * lane + e] = o[e];
  __syncthreads();
  const int d = 4 * threadIdx.x;
  if (d < D) {
    const v4f r = ((*(const v4f*)&red[0][d] + *(const v4f*)&red[1][d]) + *(const v4f*)&red[2][d]) + *(const v4f*)&red[3][d];
    store_joined<D>(a, row, h / (a.heads / a.kv_heads), d, r, sum != 0.0f ? 1.0f / sum : 0.0f);
  }
  if (p.lse && threadIdx.x == 0) p.lse[row] = joined_lse(m, sum);
}

// The weights of a decode call, from its scores: one thread a position.  The
// rows' log sums are joined here again, so that this does not wait for the
// joining of the outputs.
__device__ __forceinline__ void weights_decode(const KvAttnArgs& a, const KvPlan& p, int64_t block, int tiles) {
  const int j = (int)(block % tiles) * 256 + threadIdx.x;
  const int64_t bk = block / tiles, b = bk / a.kv_heads;
  const int kh = (int)(bk % a.kv_heads), G = a.heads / a.kv_heads;
  const Span sp = span_of(a.q_starts, a.kv_lens, b, a.q_tokens, a.max_kv);
  const int rows = (sp.n < a.max_q ? sp.n : (int)a.max_q) * G;
  __shared__ float ref[32];
  const int q = threadIdx.x / 8;            // eight lanes a row
  if (q < rows) {
    const int i = (int)div_by(q, p.group);
    const int64_t row = (int64_t)(sp.t0 + i) * a.heads + kh * G + q - i * G;
    float m = kNoMax, l = 0.0f;
    const int L = a.num_slots > 0 ? sp.L : 0, n = L > 0 ? (L + p.split_len - 1) / p.split_len : 1;
    for (int s = threadIdx.x % 8; s < n; s += 8) {
      const v2f x = p.part_ml[s * p.part_rows + row];
      const float top = fmaxf(m, x[0]);
      l = l * __builtin_amdgcn_exp2f(m - top) + x[1] * __builtin_amdgcn_exp2f(x[0] - top);
      m = top;
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const float m2 = __shfl_xor(m, o), l2 = __shfl_xor(l, o), top = fmaxf(m, m2);
      l = l * __builtin_amdgcn_exp2f(m - top) + l2 * __builtin_amdgcn_exp2f(m2 - top);
      m = top;
    }
    if (threadIdx.x % 8 == 0) ref[q] = l != 0.0f ? m + __log2f(l) : INFINITY;       // exp2(s - Inf) = 0
  }
  __syncthreads();
  if (j >= sp.L) return;
  float w = 0.0f;
  if (a.num_slots > 0)
    for (int r = 0; r < rows; ++r)
      w += __builtin_amdgcn_exp2f(p.scores[(bk * p.score_rows + r) * p.score_ld + j] - ref[r]);
  const int64_t at = bk * a.ld_w + j;
  a.w_out[at] = (a.w_in ? a.w_in[at] : 0.0f) + w;
}

// What is left of a call after its attention kernel: the first `joins`
// workgroups join the outputs, the others form a decode call's weights.
template <int D, bool FEW>
__global__ void __launch_bounds__(256) k_kv_finish(KvAttnArgs a, KvPlan p, int joins, int tiles) {
  if ((int)blockIdx.x >= joins) weights_decode(a, p, (int64_t)blockIdx.x - joins, tiles);
  else if constexpr (FEW) combine_few<D>(a, p, blockIdx.x);
  else combine_many<D>(a, p, blockIdx.x);
}

template <int D>
void launch_finish(const KvAttnArgs& a, const KvPlan& p, bool any_q, bool decode, hipStream_t st) {
  constexpr int kRows = 1024 / D;
  const bool few = p.splits <= kFewSplits;
  const int64_t rows = a.max_q * a.heads;
  const int joins = any_q && p.splits > 1 ? (int)(a.batch * (few ? (rows + kRows - 1) / kRows : rows)) : 0;
  const int tiles = (int)((a.max_kv + 255) / 256);
  const int64_t grid = joins + (decode && a.w_out ? a.batch * a.kv_heads * tiles : 0);
  if (grid == 0) return;
  if (few) k_kv_finish<D, true><<<(unsigned)grid, 256, 0, st>>>(a, p, joins, tiles);
  else k_kv_finish<D, false><<<(unsigned)grid, 256, 0, st>>>(a, p, joins, tiles);
}

}  // namespace

void launch_join(const KvAttnArgs& a, const KvPlan& p, int head_dim, hipStream_t st) {
  if (head_dim == 64) launch_finish<64>(a, p, true, false, st);
  else if (head_dim == 128) launch_finish<128>(a, p, true, false, st);
  else launch_finish<256>(a, p, true, false, st);
}

size_t kv_attention_workspace(int64_t q_tokens, int64_t heads, int64_t kv_heads, int head_dim, int64_t batch,
                              int64_t max_q, int64_t max_kv, bool with_weights) {
  if (heads == 0 || kv_heads == 0) return 0;
  KvPlan p{};
  return lay_out(p, q_tokens, heads, kv_heads, head_dim, batch, max_q, max_kv, with_weights).bytes;
}

bool kv_attention_fits(int64_t heads, int64_t kv_heads, int64_t batch, int64_t max_q, int64_t max_kv) {
  if (heads == 0 || kv_heads == 0 || batch == 0) return true;
  // Workgroups of every launch stay below 2^31, a sequence's rows and a kv
  // head's positions are indexed with 31 bits, and the workspace with 63.
  constexpr double kMost = 2147483647.0;
  const double rows = (double)max_q * (double)(heads / kv_heads), bk = (double)batch * (double)kv_heads;
  return rows < kMost && (double)batch * (double)max_q * (double)heads + bk * ((double)max_kv / 256 + 1) < kMost &&
         bk * 128 * (rows / 128 + 1) < kMost && bk * ((double)max_kv / 64 + 1) < kMost;
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
  p.queries = p.row_tiles > 0 ? ws + at.queries : nullptr;
  p.factors = (float*)(ws + at.factors);
  const bool decode = is_decode(a.heads, a.kv_heads, head_dim, a.max_q);
  const bool any_q = a.q_tokens > 0 && a.max_q > 0;
  if (any_q && decode) launch_kv_decode(a, p, head_dim, st);
  else if (any_q) launch_kv_chunk(a, p, head_dim, st);
  if (head_dim == 64) launch_finish<64>(a, p, any_q, decode, st);
  else if (head_dim == 128) launch_finish<128>(a, p, any_q, decode, st);
  else launch_finish<256>(a, p, any_q, decode, st);
  if (!decode && a.w_out && a.max_kv > 0) launch_kv_chunk_weights(a, p, head_dim, st);
  return hipGetLastError();
}

}  // namespace fp8blk
