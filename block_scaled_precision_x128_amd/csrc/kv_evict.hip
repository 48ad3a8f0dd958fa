// Eviction from the FP8 KV cache by received attention weight: the choice of
// the positions to keep, and the move of their cache rows and weights.
#include "attention.h"
#include "paging.h"

namespace fp8blk {

namespace {

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// ---- choice -------------------------------------------------------------------
// A position's score is the sum of its heads' weights (in 64 bits, so that the
// fp32 score does not depend on the order of the heads), mapped to a 32-bit key
// of the same order.  One workgroup a sequence finds the keep-th largest key T
// digit by digit (11 + 11 + 10 bits, a histogram of 2048 bins in LDS), then
// writes the positions with key > T and the lowest of those with key == T.  Each
// wave owns one contiguous range of positions, so the output order needs two
// counts a wave and no barrier inside the loops.  Keys of short sequences are
// formed by that workgroup and stay in its LDS; those of long ones come from a
// launch of their own (k_evict_scores) through the workspace.

constexpr uint32_t kForced = 0xffffffffu;   // above the key of +Inf

__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0u;                    // below the key of -Inf
  const uint32_t u = __float_as_uint(x + 0.0f);   // -0 counts as +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Running sums over each row of 16 lanes, and over the wave.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t add_shifted(uint32_t v) {
  return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t row_scan(uint32_t v) {       // row_shr 1, 2, 4, 8; lanes shifted in add 0
  return add_shifted<0x118, 0xF>(add_shifted<0x114, 0xF>(add_shifted<0x112, 0xF>(add_shifted<0x111, 0xF>(v))));
}
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {      // row_bcast 15 into rows 1 and 3, 31 into 2 and 3
  return add_shifted<0x143, 0xC>(add_shifted<0x142, 0xA>(row_scan(v)));
}

__device__ __forceinline__ int64_t clamp_len(int64_t n, int64_t top) { return n < 0 ? 0 : n > top ? top : n; }

struct Choice {
  const float* w;
  const int64_t* kv_lens;
  int64_t *kept, *kept_lens;
  int64_t ld_w, kv_heads, max_kv, keep, first, recent, ld_keys;
};

// Keys of positions j, j + step, .. of sequence b, of n positions, with a head's
// loads of all of them in flight together.
template <int U>
__device__ __forceinline__ void score_keys(const Choice& c, int64_t b, int64_t j, int64_t step, int64_t n, uint32_t* keys) {
  double s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) s[u] = 0.0;
  uint32_t at[U];                           // behind the last position: that one's weight again, unused
#pragma unroll
  for (int u = 0; u < U; ++u) at[u] = (uint32_t)(j + u * step < n ? j + u * step : n - 1);
  const float* w = c.w + b * c.kv_heads * c.ld_w;
#pragma unroll 2
  for (int64_t h = 0; h < c.kv_heads; ++h, w += c.ld_w) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = w[at[u]];
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] += (double)x[u];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = j + u * step;
    if (i < n) keys[i] = i < c.first || i >= n - c.recent ? kForced : key_of((float)s[u]);
  }
}

__global__ void __launch_bounds__(256) k_evict_scores(Choice c, int64_t tiles, uint32_t* __restrict__ keys) {
  const int64_t b = blockIdx.x / tiles, j = (blockIdx.x % tiles) * 256 + threadIdx.x;
  const int64_t n = clamp_len(c.kv_lens[b], c.max_kv);
  if (j < n && n > c.keep) score_keys<1>(c, b, j, 0, n, keys + b * c.ld_keys);
}

constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64;

// Keys that a workgroup holds in LDS, and the weights it reads for them: at 64k
// weights a sequence (8 heads of 8192 positions) forming the keys here takes as
// long as the two kernels (32 sequences: 18.4 us, 11.8 + 5.1) and saves a
// launch; beyond, one workgroup's reads are the longer part.
constexpr int kLdsKeys = 8192;
constexpr int64_t kLdsWeights = 65536;

template <bool LDS_KEYS>
__global__ void __launch_bounds__(kSelThreads) k_evict_select(Choice c, const uint32_t* __restrict__ keys_all) {
  const int64_t b = blockIdx.x, n = clamp_len(c.kv_lens[b], c.max_kv), keep = c.keep;
  int64_t* kept = c.kept + b * keep;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t count = n < keep ? n : keep;
  if (tid == 0) c.kept_lens[b] = count;
  if (keep == 0) return;                    // no key to find, and no row to write
  if (n <= keep) {
    for (int64_t i = tid; i < keep; i += kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  __shared__ u32x4 held[LDS_KEYS ? kLdsKeys / 4 : 1];
  const uint32_t* keys = LDS_KEYS ? (const uint32_t*)held : keys_all + b * c.ld_keys;
  if constexpr (LDS_KEYS) {                 // n <= kLdsKeys
    for (int j = tid; j < (int)n; j += 8 * kSelThreads) score_keys<8>(c, b, j, kSelThreads, n, (uint32_t*)held);
    __syncthreads();
  }
  // Four counters a bin, side by side, for lanes l % 4: scores lie close
  // together, and lanes that count the same bin would wait for each other (64k
  // positions, one counter: 62 us).  A thread reads its two bins as two 16-byte
  // words, 32 bytes from the next thread's; eight counters put them 64 bytes
  // apart, four lanes on a bank (32 rows of 8192 positions: 16.8 us, 14.4
  // with four; one of 1500: 13.6, 11.2).
  __shared__ u32x4 hist[2048];
  __shared__ uint32_t total[kSelWaves], s_digit, s_above;
  uint32_t prefix = 0, mask = 0;
  uint32_t want = (uint32_t)keep;           // how many of the keys under the prefix to take
  for (int i = tid; i < 2048; i += kSelThreads) hist[i] = u32x4{0, 0, 0, 0};
  __syncthreads();
  for (int pass = 0; pass < 3; ++pass) {
    const int sh = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bins = pass < 2 ? 2048 : 1024;
    // sixteen keys a thread in flight (rows of keys are 16-byte aligned; behind
    // the last four keys those again, uncounted: a branch a load would wait)
    for (int64_t j0 = 4 * tid; j0 < n; j0 += 16 * kSelThreads) {
      u32x4 k[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t j = j0 + u * 4 * kSelThreads;
        k[u] = *(const u32x4*)(keys + (j < n ? j : (n - 1) / 4 * 4));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j0 + u * 4 * kSelThreads + e < n && (k[u][e] & mask) == prefix)
            atomicAdd((uint32_t*)hist + 4 * ((k[u][e] >> sh) & (bins - 1)) + (lane & 3), 1u);
    }
    __syncthreads();
    // From the top digit down: the digit at which the running count reaches
    // `want`.  Thread t holds digits bins-1-2t and bins-2-2t, and clears them for
    // the next pass.
    const int d0 = (int)bins - 1 - 2 * tid;
    auto counted = [&](int d) {
      const u32x4 x = hist[d];
      hist[d] = u32x4{0, 0, 0, 0};
      return x[0] + x[1] + x[2] + x[3];
    };
    const uint32_t c0 = d0 >= 0 ? counted(d0) : 0u, c1 = d0 >= 1 ? counted(d0 - 1) : 0u;
    const uint32_t run = wave_scan(c0 + c1);
    if (lane == 63) total[wave] = run;
    __syncthreads();
    const uint32_t waves = row_scan(total[lane & 15]);
    const uint32_t before = run - c0 - c1 + (wave > 0 ? __builtin_amdgcn_readlane(waves, wave - 1) : 0u);
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
  }
  // prefix is the keep-th largest key; of the keys equal to it the `want`
  // lowest positions are kept.
  const int64_t seg = (n + kSelWaves * 64 - 1) / (kSelWaves * 64) * 64;
  const int64_t j0 = wave * seg, j1 = j0 + seg < n ? j0 + seg : n;
  __shared__ uint32_t n_gt[kSelWaves], n_eq[kSelWaves];
  uint32_t gt = 0, eq = 0;
  constexpr int U = 8;
  for (int64_t j = j0 + lane; j < j1; j += 64 * U) {
    uint32_t k[U];
#pragma unroll
    for (int u = 0; u < U; ++u) k[u] = keys[j + 64 * u < j1 ? j + 64 * u : j1 - 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      gt += j + 64 * u < j1 && k[u] > prefix;
      eq += j + 64 * u < j1 && k[u] == prefix;
    }
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
  for (int64_t jb = j0; jb < j1; jb += 64 * U) {
    uint32_t k[U];
#pragma unroll
    for (int u = 0; u < U; ++u) k[u] = keys[jb + 64 * u + lane < j1 ? jb + 64 * u + lane : j1 - 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t j = jb + 64 * u + lane;
      const bool in = j < j1, e = in && k[u] == prefix;
      const uint64_t be = __ballot(e);
      const bool take = (in && k[u] > prefix) || (e && eq_before + __popcll(be & below) < want);
      const uint64_t bt = __ballot(take);
      const int64_t to = at + __popcll(bt & below);
      if (take && to < keep) kept[to] = j;
      at += (uint32_t)__popcll(bt);
      eq_before += (uint32_t)__popcll(be);
    }
  }
}

// ---- move ---------------------------------------------------------------------
// Bound: HBM, a kept position's bytes of both caches once in and once out.

// Slot under table row `t` of position j, -1 outside the table or the pool.
__device__ __forceinline__ int row_slot(const int64_t* t, int64_t blocks, int64_t j, FastDiv f, int64_t num_slots) {
  return (uint64_t)j < (uint64_t)blocks * f.d ? slot_of(t, (uint32_t)j, f, (int)num_slots) : -1;
}

// In place the move is safe in one order: kept[i] >= i, so output i can only
// overwrite sources of outputs up to i.  A workgroup owns a slice of bytes of
// every row of one sequence and walks the outputs upward in chunks: all loads
// of a chunk, a barrier, all its stores.  Sources of later chunks lie behind
// every destination of this one, so the next chunk's loads are issued before
// the barrier.  Slices are independent of each other.
constexpr int kMoveThreads = 1024, kMoveUnroll = 4;

template <typename V>
struct Chunk {
  V x[kMoveUnroll];
  V* to[kMoveUnroll];
};

// One slice: V is the unit moved by a thread, c_units of them a row.
template <int THREADS, typename V, typename Src, typename Dst>
__device__ __forceinline__ void move_rows(int64_t count, int c_units, Src src, Dst dst) {
  const int per = THREADS / c_units, r = threadIdx.x / c_units;
  auto fetch = [&](int64_t base, Chunk<V>& c) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int64_t i = base + u * per + r;
      const V* from = i < count ? src(i) : nullptr;
      c.to[u] = from ? dst(i) : nullptr;
      if (c.to[u] == from) c.to[u] = nullptr;
      c.x[u] = V{};
      if (c.to[u]) c.x[u] = *from;
    }
  };
  Chunk<V> cur, nxt;
  fetch(0, cur);
  for (int64_t base = 0; base < count; base += (int64_t)per * kMoveUnroll) {
    fetch(base + (int64_t)per * kMoveUnroll, nxt);
    // this chunk's loads have arrived in every wave before any of them stores;
    // a full fence would wait for the next chunk's too
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) asm volatile("" : "+v"(cur.x[u])::"memory");
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      asm volatile("" : "+v"(cur.x[u])::"memory");
      if (cur.to[u]) *cur.to[u] = cur.x[u];
    }
    cur = nxt;
  }
}

// Slice `part` of one sequence: the K rows' slices, then the V rows'.
template <int THREADS>
__device__ __forceinline__ void move_slice(const CompactArgs& a, FastDiv f, int64_t b, int part, int slices, int c_units,
                                           int64_t count) {
  const int64_t* kept = a.kept + b * a.keep;
  uint8_t* cache = a.cache[part >= slices];
  const int64_t units = a.row / 16, c = (int64_t)(part % slices) * c_units + threadIdx.x % c_units;
  const int64_t* st = a.src + b * a.src_blocks;
  const int64_t* dt = a.dst + b * a.dst_blocks;
  auto row = [&](int slot) { return slot < 0 || c >= units ? (u32x4*)nullptr : (u32x4*)(cache + slot * a.row) + c; };
  move_rows<THREADS, u32x4>(
      count, c_units,
      [&](int64_t i) -> const u32x4* { return row(row_slot(st, a.src_blocks, kept[i], f, a.num_slots)); },
      [&](int64_t i) { return row(row_slot(dt, a.dst_blocks, i, f, a.num_slots)); });
}

// Into pages of their own the rows move independently.  A workgroup takes
// kCopyRows positions of a sequence, looks their slots up once for both caches
// and the weights, and copies whole rows, so that its reads and writes are as
// long as the cache's rows (32 x 4000 positions of 8192, 8 heads of 128, and
// their weights: 118 us, 4.4 TB/s; slices of 128 bytes took over twice as long).
// A sequence whose tables name the same page in the same place is in place all
// the same, and its workgroups share its slices; to compare the pages costs 0.6
// us of 6 for a short sequence and 2 of 118 here.
constexpr int kCopyRows = 32, kCopyThreads = 256, kCopySlice = 4;

__global__ void __launch_bounds__(kCopyThreads) k_kv_copy(CompactArgs a, FastDiv f, FastDiv by_units, int tiles) {
  const int64_t b = blockIdx.x / tiles;
  const int i0 = (int)(blockIdx.x % tiles) * kCopyRows, tid = threadIdx.x;
  const int64_t count = clamp_len(a.kept_lens[b], a.keep);
  if (i0 >= count) return;
  int64_t pages = (count + f.d - 1) / f.d;
  pages = pages < a.src_blocks ? pages : a.src_blocks;
  pages = pages < a.dst_blocks ? pages : a.dst_blocks;
  const int64_t* st = a.src + b * a.src_blocks;
  const int64_t* dt = a.dst + b * a.dst_blocks;
  bool same = false;
  constexpr int P = 4;                      // pages a thread in flight; behind the last, the first again
  for (int64_t p = tid; p < pages; p += P * kCopyThreads) {
    int64_t x[P], y[P];
#pragma unroll
    for (int u = 0; u < P; ++u) {
      const int64_t at = p + u * kCopyThreads < pages ? p + u * kCopyThreads : p;
      x[u] = st[at];
      y[u] = dt[at];
    }
#pragma unroll
    for (int u = 0; u < P; ++u) same |= x[u] == y[u];
  }
  const int rows = count - i0 < kCopyRows ? (int)(count - i0) : kCopyRows;
  __shared__ int s_src[kCopyRows], s_dst[kCopyRows];
  __shared__ int64_t s_kept[kCopyRows];
  if (tid < kCopyRows) {
    int src = -1, dst = -1;
    int64_t j = -1;
    if (tid < rows) {
      j = a.kept[b * a.keep + i0 + tid];
      src = row_slot(st, a.src_blocks, j, f, a.num_slots);
      dst = row_slot(dt, a.dst_blocks, i0 + tid, f, a.num_slots);
    }
    s_src[tid] = src < 0 || dst < 0 ? -1 : src;
    s_dst[tid] = dst;
    s_kept[tid] = j;
  }
  const bool shared = __syncthreads_or(same);
  const uint32_t units = (uint32_t)(a.row / 16), pieces = rows * units;
  constexpr int U = 4;
  if (shared) {
    const int slices = (int)((units + kCopySlice - 1) / kCopySlice);
    const int stride = (int)((count + kCopyRows - 1) / kCopyRows);
    for (int part = blockIdx.x % tiles; part < 2 * slices; part += stride)
      move_slice<kCopyThreads>(a, f, b, part, slices, kCopySlice, count);
  }
  for (uint32_t p0 = tid; !shared && p0 < pieces; p0 += U * kCopyThreads) {
    u32x4 k[U], v[U];
    int64_t to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t p = p0 + u * kCopyThreads, r = p < pieces ? div_by(p, by_units) : 0;
      const int64_t c = (int64_t)(p - r * units) * 16;
      to[u] = -1;
      if (p < pieces && s_src[r] >= 0) {
        const int64_t from = s_src[r] * a.row + c;
        to[u] = s_dst[r] * a.row + c;
        k[u] = *(const u32x4*)(a.cache[0] + from);
        v[u] = *(const u32x4*)(a.cache[1] + from);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (to[u] >= 0) {
        *(u32x4*)(a.cache[0] + to[u]) = k[u];
        *(u32x4*)(a.cache[1] + to[u]) = v[u];
      }
  }
  if (a.w_out)
    for (int64_t p = tid; p < a.kv_heads * kCopyRows; p += kCopyThreads) {
      const int r = (int)(p % kCopyRows);
      const int64_t h = b * a.kv_heads + p / kCopyRows, j = s_kept[r];
      if (r < rows && (uint64_t)j < (uint64_t)a.ld_in && i0 + r < a.ld_out)
        a.w_out[h * a.ld_out + i0 + r] = a.w_in[h * a.ld_in + j];
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
    move_rows<kMoveThreads, float>(
        count < a.ld_out ? count : a.ld_out, 1,
        [&](int64_t i) { return (uint64_t)kept[i] < (uint64_t)a.ld_in ? in + kept[i] : (const float*)nullptr; },
        [&](int64_t i) { return out + i; });
    return;
  }
  move_slice<kMoveThreads>(a, f, b, part, slices, c_units, count);
}

}  // namespace

// A row of keys a sequence, 16-byte aligned.
static int64_t key_row(int64_t max_kv) { return (max_kv + 3) / 4 * 4; }

size_t kv_evict_select_workspace(int64_t batch, int64_t max_kv) {
  return (size_t)(batch * key_row(max_kv)) * sizeof(uint32_t);
}

hipError_t launch_kv_evict_select(const float* w, int64_t ld_w, int64_t batch, int64_t kv_heads,
                                  const int64_t* kv_lens, int64_t max_kv, int64_t keep, int64_t first, int64_t recent,
                                  int64_t* kept, int64_t* kept_lens, void* ws, hipStream_t st) {
  const Choice c{w, kv_lens, kept, kept_lens, ld_w, kv_heads, max_kv, keep, first, recent, key_row(max_kv)};
  if (max_kv <= kLdsKeys && max_kv * kv_heads <= kLdsWeights) {
    k_evict_select<true><<<(unsigned)batch, kSelThreads, 0, st>>>(c, nullptr);
    return hipGetLastError();
  }
  uint32_t* keys = (uint32_t*)ws;
  const int64_t tiles = (max_kv + 255) / 256;
  if (max_kv > keep) k_evict_scores<<<(unsigned)(batch * tiles), 256, 0, st>>>(c, tiles, keys);
  k_evict_select<false><<<(unsigned)batch, kSelThreads, 0, st>>>(c, keys);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const CompactArgs& a, hipStream_t st) {
  const FastDiv page = make_fastdiv(a.block_size);
  const int64_t units = a.row / 16;
  const bool in_place = a.src == a.dst || (a.w_out && a.w_in == a.w_out);
  if (!in_place) {
    const int tiles = (int)((a.keep + kCopyRows - 1) / kCopyRows);
    k_kv_copy<<<(unsigned)(a.batch * tiles), kCopyThreads, 0, st>>>(a, page, make_fastdiv(units), tiles);
    return hipGetLastError();
  }
  // 128 bytes of every row a workgroup, less for shorter rows and where that
  // would leave CUs without one
  int c_units = 8;
  while (c_units > 1 && (c_units > units || a.batch * 2 * (units / c_units) < 256)) c_units /= 2;
  const int slices = (int)((units + c_units - 1) / c_units);
  const int64_t per_seq = 2 * slices + (a.w_out ? a.kv_heads : 0);
  k_kv_compact<<<(unsigned)(a.batch * per_seq), kMoveThreads, 0, st>>>(a, page, c_units, slices);
  return hipGetLastError();
}

}  // namespace fp8blk
