// Eviction from the FP8 KV cache by received attention weight: the choice of
// the positions to keep, and the move of their cache rows and weights.
#include "attention.h"
#include "paging.h"

namespace fp8blk {

namespace {

// ---- choice -------------------------------------------------------------------
// Two launches.  k_evict_scores sums the heads' weights (64-bit sums, so the
// fp32 score does not depend on the order of the heads) and maps each score to
// a 32-bit key of the same order.  k_evict_select, one workgroup a sequence,
// finds the keep-th largest key T digit by digit (11 + 11 + 10 bits, a
// histogram of 2048 counters in LDS), then writes the positions with key > T
// and the lowest of those with key == T.  Each wave owns one contiguous range
// of positions, so the output order needs two counts a wave and no barrier
// inside the loops.

constexpr uint32_t kForced = 0xffffffffu;   // above the key of +Inf

__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0u;                    // below the key of -Inf
  const uint32_t u = __float_as_uint(x + 0.0f);   // -0 counts as +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int64_t clamp_len(int64_t n, int64_t top) { return n < 0 ? 0 : n > top ? top : n; }

__global__ void __launch_bounds__(256) k_evict_scores(const float* __restrict__ w, int64_t ld_w, int64_t kv_heads,
                                                      const int64_t* __restrict__ kv_lens, int64_t max_kv,
                                                      int64_t keep, int64_t first, int64_t recent, int64_t tiles,
                                                      uint32_t* __restrict__ keys) {
  const int64_t b = blockIdx.x / tiles, j = (blockIdx.x % tiles) * 256 + threadIdx.x;
  const int64_t n = clamp_len(kv_lens[b], max_kv);
  if (j >= n || n <= keep) return;
  double s = 0.0;
  for (int64_t h = 0; h < kv_heads; ++h) s += (double)w[(b * kv_heads + h) * ld_w + j];
  keys[b * max_kv + j] = j < first || j >= n - recent ? kForced : key_of((float)s);
}

constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64;

__global__ void __launch_bounds__(kSelThreads) k_evict_select(const uint32_t* __restrict__ keys_all,
                                                              const int64_t* __restrict__ kv_lens, int64_t max_kv,
                                                              int64_t keep, int64_t* __restrict__ kept_all,
                                                              int64_t* __restrict__ kept_lens) {
  const int64_t b = blockIdx.x, n = clamp_len(kv_lens[b], max_kv);
  int64_t* kept = kept_all + b * keep;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t count = n < keep ? n : keep;
  if (tid == 0) kept_lens[b] = count;
  if (keep == 0) return;                    // no key to find, and no row to write
  if (n <= keep) {
    for (int64_t i = tid; i < keep; i += kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const uint32_t* keys = keys_all + b * max_kv;
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t total[kSelWaves], s_digit, s_above;
  uint32_t prefix = 0, mask = 0;
  uint32_t want = (uint32_t)keep;           // how many of the keys under the prefix to take
  const int shift_of[3] = {21, 10, 0};
  const uint32_t bins_of[3] = {2048, 2048, 1024};
  for (int pass = 0; pass < 3; ++pass) {
    const int sh = shift_of[pass];
    const uint32_t bins = bins_of[pass];
    for (int i = tid; i < 2048; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int64_t j = tid; j < n; j += kSelThreads) {
      const uint32_t k = keys[j];
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> sh) & (bins - 1)], 1u);
    }
    __syncthreads();
    // From the top digit down: the digit at which the running count reaches
    // `want`.  Thread t holds digits bins-1-2t and bins-2-2t.
    const int d0 = (int)bins - 1 - 2 * tid;
    const uint32_t c0 = d0 >= 0 ? hist[d0] : 0u, c1 = d0 >= 1 ? hist[d0 - 1] : 0u;
    uint32_t run = c0 + c1;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t up = __shfl_up(run, o);
      if (lane >= o) run += up;
    }
    if (lane == 63) total[wave] = run;
    __syncthreads();
    uint32_t before = run - c0 - c1;
    for (int i = 0; i < wave; ++i) before += total[i];
    if (before < want && before + c0 >= want) {
      s_digit = (uint32_t)d0;
      s_above = before;
    } else if (before + c0 < want && before + c0 + c1 >= want) {
      s_digit = (uint32_t)d0 - 1;
      s_above = before + c0;
    }
    __syncthreads();
    prefix |= s_digit << sh;
    mask |= (bins - 1) << sh;
    want -= s_above;
    __syncthreads();
  }
  // prefix is the keep-th largest key; of the keys equal to it the `want`
  // lowest positions are kept.
  const int64_t seg = (n + kSelWaves * 64 - 1) / (kSelWaves * 64) * 64;
  const int64_t j0 = wave * seg, j1 = j0 + seg < n ? j0 + seg : n;
  __shared__ uint32_t n_gt[kSelWaves], n_eq[kSelWaves];
  uint32_t gt = 0, eq = 0;
  for (int64_t j = j0 + lane; j < j1; j += 64) {
    const uint32_t k = keys[j];
    gt += k > prefix;
    eq += k == prefix;
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    gt += __shfl_xor(gt, o);
    eq += __shfl_xor(eq, o);
  }
  if (lane == 0) {
    n_gt[wave] = gt;
    n_eq[wave] = eq;
  }
  __syncthreads();
  uint32_t at = 0, eq_before = 0;
  for (int i = 0; i < wave; ++i) {
    at += n_gt[i];
    eq_before += n_eq[i];
  }
  at += eq_before < want ? eq_before : want;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  for (int64_t j = j0; j < j1; j += 64) {
    const bool in = j + lane < j1;
    const uint32_t k = in ? keys[j + lane] : 0u;
    const bool e = in && k == prefix;
    const uint64_t be = __ballot(e);
    const bool take = (in && k > prefix) || (e && eq_before + __popcll(be & below) < want);
    const uint64_t bt = __ballot(take);
    const int64_t to = at + __popcll(bt & below);
    if (take && to < keep) kept[to] = j + lane;
    at += (uint32_t)__popcll(bt);
    eq_before += (uint32_t)__popcll(be);
  }
}

// ---- move ---------------------------------------------------------------------
// In place the move is safe in one order: kept[i] >= i, so output i can only
// overwrite sources of outputs up to i.  A workgroup owns a slice of bytes of
// every row of one sequence and walks the outputs upward in chunks: all loads
// of a chunk, a barrier, all its stores.  Slices are independent of each other.

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int kMoveThreads = 1024, kMoveUnroll = 4;

// One slice: V is the unit moved by a thread, C units a row.
template <typename V, typename Src, typename Dst>
__device__ __forceinline__ void move_rows(int64_t count, int c_units, Src src, Dst dst) {
  const int per = kMoveThreads / c_units, r = threadIdx.x / c_units;
  for (int64_t base = 0; base < count; base += (int64_t)per * kMoveUnroll) {
    V x[kMoveUnroll];
    V* to[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int64_t i = base + u * per + r;
      const V* from = i < count ? src(i) : nullptr;
      to[u] = from ? dst(i) : nullptr;
      if (to[u] == from) to[u] = nullptr;
      if (to[u]) x[u] = *from;
    }
    // every load has arrived before any thread of the workgroup stores
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) asm volatile("" : "+v"(x[u]));
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (to[u]) *to[u] = x[u];
  }
}

__global__ void __launch_bounds__(kMoveThreads) k_kv_compact(CompactArgs a, FastDiv f, int c_units, int slices) {
  const int per_seq = 2 * slices + (a.w_out ? (int)a.kv_heads : 0);
  const int64_t b = blockIdx.x / per_seq;
  const int part = blockIdx.x % per_seq;
  const int64_t* kept = a.kept + b * a.keep;
  const int64_t count = clamp_len(a.kept_lens[b], a.keep);
  if (part >= 2 * slices) {
    const int64_t h = part - 2 * slices;
    const float* in = a.w_in + (b * a.kv_heads + h) * a.ld_in;
    float* out = a.w_out + (b * a.kv_heads + h) * a.ld_out;
    move_rows<float>(
        count < a.ld_out ? count : a.ld_out, 1,
        [&](int64_t i) { return (uint64_t)kept[i] < (uint64_t)a.ld_in ? in + kept[i] : (const float*)nullptr; },
        [&](int64_t i) { return out + i; });
    return;
  }
  uint8_t* cache = a.cache[part >= slices];
  const int64_t units = a.row / 16, c = (int64_t)(part % slices) * c_units + threadIdx.x % c_units;
  const int64_t src_n = a.src_blocks * a.block_size, dst_n = a.dst_blocks * a.block_size;
  const int64_t* st = a.src + b * a.src_blocks;
  const int64_t* dt = a.dst + b * a.dst_blocks;
  auto row = [&](int slot) { return slot < 0 || c >= units ? (u32x4*)nullptr : (u32x4*)(cache + slot * a.row) + c; };
  move_rows<u32x4>(
      count < dst_n ? count : dst_n, c_units,
      [&](int64_t i) -> const u32x4* {
        const int64_t j = kept[i];
        return (uint64_t)j < (uint64_t)src_n ? row(slot_of(st, (uint32_t)j, f, (int)a.num_slots)) : nullptr;
      },
      [&](int64_t i) { return row(slot_of(dt, (uint32_t)i, f, (int)a.num_slots)); });
}

}  // namespace

size_t kv_evict_select_workspace(int64_t batch, int64_t max_kv) { return (size_t)(batch * max_kv) * sizeof(uint32_t); }

hipError_t launch_kv_evict_select(const float* w, int64_t ld_w, int64_t batch, int64_t kv_heads,
                                  const int64_t* kv_lens, int64_t max_kv, int64_t keep, int64_t first, int64_t recent,
                                  int64_t* kept, int64_t* kept_lens, void* ws, hipStream_t st) {
  uint32_t* keys = (uint32_t*)ws;
  const int64_t tiles = (max_kv + 255) / 256;
  if (max_kv > keep)
    k_evict_scores<<<(unsigned)(batch * tiles), 256, 0, st>>>(w, ld_w, kv_heads, kv_lens, max_kv, keep, first, recent,
                                                              tiles, keys);
  k_evict_select<<<(unsigned)batch, kSelThreads, 0, st>>>(keys, kv_lens, max_kv, keep, kept, kept_lens);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const CompactArgs& a, hipStream_t st) {
  const int c_units = 8;
  const int slices = (int)((a.row / 16 + c_units - 1) / c_units);
  const int64_t per_seq = 2 * slices + (a.w_out ? a.kv_heads : 0);
  k_kv_compact<<<(unsigned)(a.batch * per_seq), kMoveThreads, 0, st>>>(a, make_fastdiv(a.block_size), c_units, slices);
  return hipGetLastError();
}

}  // namespace fp8blk
