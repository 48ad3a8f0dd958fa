// The tiled attention loop shared by the chunk kernel (paged FP8 cache) and
// the prompt kernel (dense bf16 states).
//
// A workgroup of four waves takes 128 query rows (query tokens x heads of one
// kv head, so that shared heads share the loads), 32 a wave, and walks the
// positions in tiles of 64.  Both products run on 32x32x16 matrix
// instructions in transposed form:
//   S^T = K Q^T    K rows from LDS as the first operand; a lane then holds 32
//                  scores of ONE row, so the maximum and the sum need one
//                  exchange between the halves of the wave and no LDS
//   O^T = V^T P^T  the k-values are positions.  The scores a lane holds are,
//                  in register order, the k-values of the second operand for
//                  the position order 16 t + 8 (j / 4) + 4 half + j % 4, so P
//                  stays in its registers; V^T in the same order comes from two
//                  transposing LDS reads (4 positions x 16 channels each).
// K rows in LDS are 16 bytes longer than their data, V rows 64 bytes: the
// 16-byte reads of 16 K rows and the transposing reads of 4 V rows then fall on
// all 64 banks once.  The tiles are double buffered with one barrier a tile:
// the global loads of the next tile are issued before the products of this
// one, and their data is stored (FP8 codes converted to fp16, once a
// workgroup) behind them.
#pragma once

#include "attention_common.h"
#include "kv_attention.h"

namespace fp8blk {

constexpr int kTileKv = 64;          // positions of a tile

// Instruction classes of __builtin_amdgcn_sched_group_barrier.
constexpr int kValu = 0x002, kMfma = 0x008, kDsRead = 0x100, kTrans = 0x400;

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));

// Matrix instruction of a 16-bit type, on raw 8 x 16-bit operands.
template <bool BF16>
__device__ __forceinline__ v16f mfma32(s8v a, s8v b, v16f c) {
  if constexpr (BF16) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
}

template <int D>
struct TileLds {
  static constexpr int kStrideK = 2 * D + 16, kStrideV = 2 * D + 64;   // bytes
  alignas(16) uint8_t k[2][kTileKv * kStrideK];
  alignas(16) uint8_t v[2][kTileKv * kStrideV];
  uint64_t live[2][8];                // a ballot of each wave: one bit of every thread's staged row
  uint32_t odd;                       // set where a NaN or Inf value was left out of a guarded tile
};

// With W waves thread t stages row t / W of a tile, 16-byte pieces t % W + W c
// of its bytes.

// Guarded tiles: where a tile holds positions that some rows of the workgroup do
// not see, p = 0 must not meet a NaN or Inf value, which a product would carry
// into those rows.  Such values are staged as zeros, and add_odd() gives them
// to the rows that do see them at the end; p being positive, a NaN or Inf is
// its own product.

// Dense bf16 rows; rows from `n` on read as zeros.
template <int D, int W>
struct DenseTile {
  static constexpr bool kBf16 = true, kHoles = false;
  static constexpr int kPieces = D / 8 / W;
  const uint16_t *kp, *vp;            // of the sequence's first token and the head
  int64_t ld_k, ld_v;
  int n, row;
  bool in;
  u32x4 kx[kPieces], vx[kPieces];

  __device__ __forceinline__ void look_up(int j0) {
    row = j0 + (int)threadIdx.x / W;
    in = row < n;
  }
  __device__ __forceinline__ void load() {
    const int at = in ? row : 0;
    const uint8_t* a = (const uint8_t*)(kp + at * ld_k) + 16 * (threadIdx.x % W);
    const uint8_t* b = (const uint8_t*)(vp + at * ld_v) + 16 * (threadIdx.x % W);
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      kx[c] = *(const u32x4*)(a + 16 * W * c);
      vx[c] = *(const u32x4*)(b + 16 * W * c);
    }
    loaded = in;
  }
  bool loaded;
  __device__ __forceinline__ void guard(TileLds<D>& s) {
    uint32_t any = 0;
#pragma unroll
    for (int c = 0; c < kPieces; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t m = odd_bf16(vx[c][i]);
        any |= m;
        vx[c][i] &= ~m;
      }
    if (loaded && any) s.odd = 1;
  }
  // Four values from channel d of position j.
  __device__ __forceinline__ v4f value(int j, int d) const {
    const u32x2 w = *(const u32x2*)(vp + j * ld_v + d);
    return v4f{bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1])};
  }
  __device__ __forceinline__ void store(TileLds<D>& s, int buf) const {
    const int r = threadIdx.x / W, p = threadIdx.x % W;
    uint8_t* a = s.k[buf] + r * TileLds<D>::kStrideK + 16 * p;
    uint8_t* b = s.v[buf] + r * TileLds<D>::kStrideV + 16 * p;
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      *(u32x4*)(a + 16 * W * c) = kx[c];
      *(u32x4*)(b + 16 * W * c) = loaded ? vx[c] : u32x4{0, 0, 0, 0};   // 0 * p, also where the memory holds NaN
    }
  }
};

// Rows of a paged cache of FP8 codes; rows outside [.., n) or the pool are dead.
template <int FMT, int D, int W>
struct PagedTile {
  static constexpr bool kBf16 = false, kHoles = true;
  static constexpr int kPieces = D / 16 / W;
  const uint8_t *kp, *vp;             // of slot 0 and the head
  const int64_t* table;
  int64_t slot_bytes;
  FastDiv page;
  int n, num_slots, slot, loaded;
  u32x4 kx[kPieces], vx[kPieces];

  __device__ __forceinline__ void look_up(int j0) {
    const int j = j0 + (int)threadIdx.x / W;
    slot = j < n ? slot_of(table, (uint32_t)j, page, num_slots) : -1;
  }
  __device__ __forceinline__ void load() {
    const int64_t at = (slot < 0 ? 0 : slot) * slot_bytes + 16 * (threadIdx.x % W);
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      kx[c] = *(const u32x4*)(kp + at + 16 * W * c);
      vx[c] = *(const u32x4*)(vp + at + 16 * W * c);
    }
    loaded = slot;
  }
  __device__ __forceinline__ void guard(TileLds<D>& s) {
    uint32_t any = 0;
#pragma unroll
    for (int c = 0; c < kPieces; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t m = odd_codes<FMT>(vx[c][i]);
        any |= m;
        vx[c][i] &= ~m;
      }
    if (loaded >= 0 && any) s.odd = 1;
  }
  // Four values from channel d of position j, zeros for a dead one.
  __device__ __forceinline__ v4f value(int j, int d) const {
    const int at = slot_of(table, (uint32_t)j, page, num_slots);
    if (at < 0) return v4f{0, 0, 0, 0};
    const uint32_t w = *(const uint32_t*)(vp + at * slot_bytes + d);
    const v2f a = decode2<FMT>(w, false), b = decode2<FMT>(w, true);
    return v4f{a[0], a[1], b[0], b[1]};
  }
  __device__ __forceinline__ void store(TileLds<D>& s, int buf) const {
    const int r = threadIdx.x / W, p = threadIdx.x % W;
    uint8_t* a = s.k[buf] + r * TileLds<D>::kStrideK + 32 * p;
    uint8_t* b = s.v[buf] + r * TileLds<D>::kStrideV + 32 * p;
    const uint64_t live = __ballot(loaded >= 0);
    if ((threadIdx.x & 63) == 0) s.live[buf][threadIdx.x / 64] = live;
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      *(h8*)(a + 32 * W * c) = codes_to_h8<FMT>(kx[c][0], kx[c][1]);
      *(h8*)(a + 32 * W * c + 16) = codes_to_h8<FMT>(kx[c][2], kx[c][3]);
      const u32x4 w = loaded >= 0 ? vx[c] : u32x4{0, 0, 0, 0};      // a dead row's codes may be NaN
      *(h8*)(b + 32 * W * c) = codes_to_h8<FMT>(w[0], w[1]);
      *(h8*)(b + 32 * W * c + 16) = codes_to_h8<FMT>(w[2], w[3]);
    }
  }
  __device__ __forceinline__ bool all_live(const TileLds<D>& s, int buf) const {
    uint64_t x = s.live[buf][0];
#pragma unroll
    for (int w = 1; w < W; ++w) x &= s.live[buf][w];
    return x == ~uint64_t(0);
  }
  __device__ __forceinline__ bool is_live(const TileLds<D>& s, int buf, int pos) const {
    return s.live[buf][pos / (64 / W)] >> (W * (pos % (64 / W))) & 1;
  }
};

// A wave's running result: row lane & 31, channels 32 t + 8 (r / 4) + 4 half + r % 4.
template <int D>
struct RowState {
  v16f o[D / 32];
  float m, l;                         // l: of the lane's own positions until finish()
};

template <bool SPLITP>
struct Probs {
  s8v hi, lo;
};

// p of 16 positions, registers 8 half_tile .. + 7 of the scores, as the second
// operand of a product; their sum is added to the row's.
template <bool BF16, bool SPLITP, int D>
__device__ __forceinline__ Probs<SPLITP> exponentials(const v16f& s, int half_tile, float c, RowState<D>& st) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * half_tile + i], c, -st.m));
  st.l += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
  asm volatile("" : "+v"(st.l));      // summed here, not with 32 values kept until the barrier
  u32x4 w, wl;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    } else {
      const h2 y = pack_f16(x[2 * i], x[2 * i + 1]);
      w[i] = __builtin_bit_cast(uint32_t, y);
      if constexpr (SPLITP)
        wl[i] = __builtin_bit_cast(uint32_t, pack_f16(x[2 * i] - (float)y[0], x[2 * i + 1] - (float)y[1]));
    }
  }
  Probs<SPLITP> p;
  p.hi = __builtin_bit_cast(s8v, w);
  if constexpr (SPLITP) p.lo = __builtin_bit_cast(s8v, wl);
  return p;
}

// V^T operands of positions 16 t .. + 15: lane i of a group of 16 reads row
// i / 4, channels 4 (i % 4) .. + 3 and gets channel i of the four rows.
template <int D>
__device__ __forceinline__ void read_values(const uint8_t* v, int t, s8v* out) {
  typedef __attribute__((address_space(3))) s4v* lds_p;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const uint8_t* at = v + (16 * t + 4 * half + (lane & 15) / 4) * TileLds<D>::kStrideV + 32 * (lane >> 4 & 1) + 8 * (lane & 3);
#pragma unroll
  for (int d = 0; d < D / 32; ++d) {
    const s4v a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(at + 64 * d));
    const s4v b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(at + 64 * d + 8 * TileLds<D>::kStrideV));
    out[d] = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
}

// The tiles of positions [j0, j1) for the wave's 32 rows.  q_hi (and q_lo):
// D/16 operands of the lane's row, channels 16 s + 8 half + i.  Position j is
// seen where j < limit; every row of the wave sees those below `seen`, every
// row of the workgroup those below `seen_by_all`.
template <typename Tile, int D, bool SPLITQ, bool SPLITP>
__device__ __forceinline__ void attend_tiles(Tile& src, TileLds<D>& lds, const s8v* q_hi, const s8v* q_lo, float factor,
                                             int limit, int seen, int seen_by_all, int j0, int j1,
                                             RowState<D>& st) {
  constexpr bool B = Tile::kBf16;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  // A factor that vanishes (a tiny row under a tiny scale) would turn the -Inf
  // of a masked score into NaN; every score is 0 beside the smallest one too.
  const float c = fmaxf(factor, 0x1p-126f);
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int r = 0; r < 16; ++r) st.o[t][r] = 0.0f;
  st.m = kNoMax;
  st.l = 0.0f;
  if (j0 >= j1) return;
  if (threadIdx.x == 0) lds.odd = 0;
  __syncthreads();
  src.look_up(j0);
  src.load();
  src.look_up(j0 + kTileKv);
  if (j0 + kTileKv > seen_by_all) src.guard(lds);
  src.store(lds, 0);
  __syncthreads();
  int buf = 0;
  for (int j = j0; j < j1; j += kTileKv, buf ^= 1) {
    // Past the last tile the look-up finds nothing and the loads take a row
    // that exists; branches here would cut the block that the loads, the
    // products and the stores are scheduled in.
    src.load();
    src.look_up(j + 2 * kTileKv);
    v16f s[2];
    const uint8_t* kb = lds.k[buf] + (lane & 31) * TileLds<D>::kStrideK + 16 * half;
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[t][r] = 0.0f;
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const s8v kk = *(const s8v*)(kb + t * 32 * TileLds<D>::kStrideK + 32 * e);
        s[t] = mfma32<B>(kk, q_hi[e], s[t]);
        if constexpr (SPLITQ) s[t] = mfma32<B>(kk, q_lo[e], s[t]);
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[t][r]);
    }
    // four reads ahead of the products
    __builtin_amdgcn_sched_group_barrier(kDsRead, 4, 0);
#pragma unroll
    for (int i = 0; i < D / 8 - 4; ++i) {
      __builtin_amdgcn_sched_group_barrier(kMfma, SPLITQ ? 2 : 1, 0);
      __builtin_amdgcn_sched_group_barrier(kDsRead, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(kMfma, SPLITQ ? 8 : 4, 0);
    bool whole = j + kTileKv <= seen;
    if constexpr (Tile::kHoles)
      whole = whole && src.all_live(lds, buf);
    if (!whole) {
      top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int pos = 32 * t + 8 * (r / 4) + 4 * half + r % 4;
          bool ok = j + pos < limit;
          if constexpr (Tile::kHoles) ok = ok && src.is_live(lds, buf, pos);
          s[t][r] = ok ? s[t][r] : -INFINITY;
          top = fmaxf(top, s[t][r]);
        }
    }
    top *= c;
    if (__any(top > st.m + kRefMove)) {
      const float mn = fmaxf(st.m, max_halves(top) - kRefBelow);
      const float f = __builtin_amdgcn_exp2f(st.m - mn);
      st.m = mn;
      st.l *= f;
#pragma unroll
      for (int t = 0; t < D / 32; ++t) st.o[t] *= f;
    }
    // Sixteen positions at a time: the reads and the exponentials of the next
    // run stand between the products of the last.
    Probs<SPLITP> p = exponentials<B, SPLITP, D>(s[0], 0, c, st);
    s8v vv[D / 32], vn[D / 32];
    read_values<D>(lds.v[buf], 0, vv);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      __builtin_amdgcn_sched_barrier(0);
      Probs<SPLITP> pn;
      if (t < 3) {
        read_values<D>(lds.v[buf], t + 1, vn);
        pn = exponentials<B, SPLITP, D>(s[(t + 1) / 2], (t + 1) % 2, c, st);
      }
#pragma unroll
      for (int d = 0; d < D / 32; ++d) {
        st.o[d] = mfma32<B>(vv[d], p.hi, st.o[d]);
        if constexpr (SPLITP) st.o[d] = mfma32<B>(vv[d], p.lo, st.o[d]);
      }
      if (t < 3) {
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
          __builtin_amdgcn_sched_group_barrier(kMfma, SPLITP ? 2 : 1, 0);
          __builtin_amdgcn_sched_group_barrier(kDsRead, 2, 0);
          __builtin_amdgcn_sched_group_barrier(kValu | kTrans, (SPLITP ? 44 : 28) * 32 / D, 0);
        }
        p = pn;
#pragma unroll
        for (int d = 0; d < D / 32; ++d) vv[d] = vn[d];
      }
    }
    if (j + 2 * kTileKv > seen_by_all) src.guard(lds);
    src.store(lds, buf ^ 1);
    __syncthreads();
  }
  st.l = sum_halves(st.l);
  if (lds.odd) {
    const int tiles = max(seen_by_all - j0, 0) / kTileKv;
    for (int j = j0 + tiles * kTileKv; j < min(j1, limit); ++j)
#pragma unroll
      for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const v4f x = src.value(j, 32 * t + 2 * r + 4 * half);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (!(fabsf(x[k]) < INFINITY)) st.o[t][r + k] += x[k];
        }
  }
}

// A lane's share of the sums of one split, for the kernel that joins them.
template <int D>
__device__ __forceinline__ void store_part(const RowState<D>& st, const KvPlan& p, int split, int64_t row) {
  const int half = (threadIdx.x & 63) >> 5;
  float* o = p.part_o + (split * p.part_rows + row) * D + 4 * half;
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *(v4f*)(o + 32 * d + 2 * r) = v4f{st.o[d][r], st.o[d][r + 1], st.o[d][r + 2], st.o[d][r + 3]};
  if (half == 0) p.part_ml[split * p.part_rows + row] = v2f{st.m, st.l};
}

}  // namespace fp8blk
