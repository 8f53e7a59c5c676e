// The tiled MFMA product of linear.hip, gated.hip and mx_linear.hip, instantiated once for each 16-bit type.
#pragma once

#include <type_traits>
#include <utility>

#include "linear.h"

namespace beam {

namespace {

constexpr int kBK = 64;  // K per stage

typedef __attribute__((address_space(3))) uint16_t lds_u16;
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Source of the chunks of an operand past its K, so that they add nothing.
__device__ const u32x4 zero_chunk = {0u, 0u, 0u, 0u};

// One operand's side of a tile: R rows of the output (M or N) by kBK of K per stage.
//
// K contiguous: LDS rows of 64 K (128 bytes), chunk c (8 elements) of row r at position
// c ^ ((r >> 1) & 7), so the 16 rows of a fragment read cover all banks once; a copy of
// 1 KB fills 8 rows from 128 contiguous bytes each.
// Transposed (TR): LDS rows of one k, R elements.  A fragment needs 8 consecutive k of a
// column; the transposing LDS read delivers 4 of them, taking 16 columns (32 bytes) of 4
// rows per 16 lanes.  The 32-byte granule g of row k sits at g ^ ((k & 3) | (k >> 1 & 4))
// (R = 64, where two rows make up all banks: g ^ (k >> 1 & 1 | k >> 2 & 2)): the 8 rows
// that 32 lanes read together fall on distinct banks.
template <bool TR, int R, int NW>
struct Side {
  static constexpr int kCopies = R / 8 / NW;     // per wave and stage
  static constexpr int kRowChunks = TR ? R / 8 : 8;
  static constexpr int kCopyRows = 64 / kRowChunks;  // LDS rows per copy
  const uint16_t* src[kCopies];
  int64_t step;

  static __device__ __forceinline__ int swz(int r) {
    if (!TR) return (r >> 1) & 7;
    return (R == 64 ? ((r >> 1) & 1) | ((r >> 2) & 2) : (r & 3) | ((r >> 1) & 4)) << 1;
  }
  // LDS row and source chunk of this lane in copy q
  static __device__ __forceinline__ int row(int q, int wave, int lane) {
    return (wave * kCopies + q) * kCopyRows + lane / kRowChunks;
  }
  static __device__ __forceinline__ int chunk(int r, int lane) { return (lane % kRowChunks) ^ swz(r); }

  // Rows i0 .. i0 + R - 1 of ni; K from k0.  Rows past the end repeat the last one (K
  // contiguous) or the last chunk of 8 (transposed): their results are never stored.
  __device__ __forceinline__ void init(const void* base, int64_t ld, int i0, int ni, int k0, int wave, int lane) {
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const int r = row(q, wave, lane), c = chunk(r, lane);
      if constexpr (TR)
        src[q] = static_cast<const uint16_t*>(base) + (int64_t)(k0 + r) * ld + min(i0 + 8 * c, (ni - 1) & ~7);
      else
        src[q] = static_cast<const uint16_t*>(base) + (int64_t)min(i0 + r, ni - 1) * ld + k0 + 8 * c;
    }
    step = TR ? kBK * ld : kBK;
  }

  // Rows of two matrices of ni rows each, 16 of the first and then 16 of the second in turn, R / 2 of
  // both from row i0 on.  A copy's 8 rows are of one of them.
  __device__ __forceinline__ void init_pair(const void* first, int64_t ld1, const void* second, int64_t ld2, int i0,
                                            int ni, int k0, int wave, int lane) {
    static_assert(!TR, "rows of K alone");
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const int r = row(q, wave, lane), c = chunk(r, lane), i = min(i0 + (r >> 5) * 16 + (r & 15), ni - 1);
      const bool other = r & 16;
      src[q] = static_cast<const uint16_t*>(other ? second : first) + (int64_t)i * (other ? ld2 : ld1) + k0 + 8 * c;
    }
    step = kBK;
  }

  // Copies a stage of which `left` K remain and moves on to the next.
  __device__ __forceinline__ void issue(lds_u16* slot, int left, int wave, int lane) {
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const void* p = src[q];
      if (left < kBK) {  // uniform; the last stage alone
        const int r = row(q, wave, lane);
        if ((TR ? r : 8 * chunk(r, lane)) >= left) p = &zero_chunk;
      }
      lds_copy16(p, __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(slot + (wave * kCopies + q) * 512)));
      src[q] += step;
    }
  }

  // The same through registers, for rows of K that start at any element and may end inside a
  // chunk (zeros follow).
  __device__ __forceinline__ void load(u32x4* regs, int left, int wave, int lane) {
    static_assert(!TR, "rows of K alone");
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const int n = left < kBK ? left - 8 * chunk(row(q, wave, lane), lane) : 8;
      if (n >= 8) {
        regs[q] = *reinterpret_cast<const u32x4_any*>(src[q]);
      } else {
        Raw8<F16> part;  // the bits alone matter
        part.load_part(src[q], n);
        regs[q] = part.w[0];
      }
      src[q] += step;
    }
  }
  static __device__ __forceinline__ void store(lds_u16* slot, const u32x4* regs, int wave, int lane) {
#pragma unroll
    for (int q = 0; q < kCopies; ++q)
      *(__attribute__((address_space(3))) u32x4*)(slot + (wave * kCopies + q) * 512 + lane * 8) = regs[q];
  }

  // The 16 rows from `r0` (a multiple of 16) of K 32 s .. 32 s + 31: lane l holds row
  // l % 16, K 8 (l / 16) .. + 7.
  static __device__ __forceinline__ u32x4 frag(const lds_u16* slot, int r0, int s, int lane) {
    const int l16 = lane & 15, g = lane >> 4;
    if constexpr (TR) {
      uint2 h[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k = 32 * s + 8 * g + 4 * half + (l16 >> 2);
        const int c = ((r0 >> 3) + ((lane & 3) >> 1)) ^ swz(k);
        const lds_u16* p = slot + k * R + 8 * c + 4 * (lane & 1);
        h[half] = __builtin_bit_cast(
            uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
      }
      return u32x4{h[0].x, h[0].y, h[1].x, h[1].y};
    } else {
      const lds_u16* p = slot + (r0 + l16) * 64 + (((4 * s + g) ^ swz(l16)) << 3);
      return *(const __attribute__((address_space(3))) u32x4*)p;
    }
  }
};

// The scales of a stage of 4-bit operands: 8 blocks (256 codes, 128 bytes as kBK 16-bit elements are) of R rows.
// The byte of block 4 s + g of row r lies at (r / 64, g, r % 16, s, r / 16 % 4), so that a lane (row l % 16, block
// l / 16 of each four) has those of 64 rows in 8 bytes, and the matrix instruction picks a byte of a word.
template <int R>
struct ScaleStage {
  static constexpr int kBytes = R * 8;
  typedef __attribute__((address_space(3))) uint8_t lds_u8;
  typedef uint64_t u64_byte __attribute__((aligned(1)));
  // Blocks b .. b + 7 of a row of `blocks`.  Past the row's end they are 0, where the codes are 0 too: there the row's
  // last eight are requested, and moved down when they are stored.
  static __device__ __forceinline__ uint64_t load(const uint8_t* row, int b, int blocks) {
    if (blocks >= 8) return *reinterpret_cast<const u64_byte*>(row + min(b, blocks - 8));
    uint64_t v = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < blocks) v |= (uint64_t)row[q] << (8 * q);
    return v;
  }
  static __device__ __forceinline__ void store(lds_u8* stage, int r, uint64_t v, int b, int blocks) {
    if (blocks >= 8) v >>= 8 * max(b + 8 - blocks, 0);
    lds_u8* p = stage + (r >> 6) * 512 + (r & 15) * 8 + ((r >> 4) & 3);
#pragma unroll
    for (int q = 0; q < 8; ++q) p[(q % 4) * 128 + (q / 4) * 4] = (uint8_t)(v >> (8 * q));
  }
  // The words (s = 0, 1) of rows r0 .. r0 + 63, or the upper half of them moved down where r0 is off 64 by 32.
  static __device__ __forceinline__ u32x2 words(const lds_u8* stage, int r0, int lane) {
    const lds_u8* p = stage + (r0 >> 6) * 512 + (lane >> 4) * 128 + (lane & 15) * 8;
    u32x2 v = *(const __attribute__((address_space(3))) u32x2*)p;
    const int down = r0 & 32 ? 16 : 0;
    v[0] >>= down;
    v[1] >>= down;
    return v;
  }
};

// f(integral_constant<int, 0>) .. f(integral_constant<int, N - 1>)
template <class F, int... I>
__device__ __forceinline__ void for_each_of(F& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F f) {
  for_each_of(f, std::make_integer_sequence<int, N>{});
}

// B's side of a tile from 4-bit codes: rows of K as Side's, eight codes and their scale to a lane and copy, converted
// on their way into LDS.
template <bool HALF, int R, int NW>
struct CodeSide {
  using Rows = Side<false, R, NW>;
  static constexpr int kCopies = Rows::kCopies;
  struct Eight {
    uint32_t codes, scale;
  };
  const uint8_t *codes[kCopies], *scales[kCopies];
  __device__ __forceinline__ void init(const CodeArgs& g, int i0, int k0, int wave, int lane) {
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const int r = Rows::row(q, wave, lane), k = k0 + 8 * Rows::chunk(r, lane);
      const int64_t row = min(i0 + r, g.N - 1);
      codes[q] = static_cast<const uint8_t*>(g.b) + row * g.ldb + k / 2;
      scales[q] = g.sb + row * g.ldsb + k / 32;
    }
  }
  __device__ __forceinline__ void load(Eight* regs, int left, int wave, int lane) {
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      regs[q] = {0u, 0u};
      if (8 * Rows::chunk(Rows::row(q, wave, lane), lane) < left)
        regs[q] = {*reinterpret_cast<const uint32_t*>(codes[q]), *scales[q]};
      codes[q] += kBK / 2;
      scales[q] += kBK / 32;
    }
  }
  static __device__ __forceinline__ void store(lds_u16* slot, const Eight* regs, int wave, int lane) {
    u32x4 v[kCopies];
#pragma unroll
    for (int q = 0; q < kCopies; ++q) v[q] = codes_to_16<HALF>(regs[q].codes, mx_scale(regs[q].scale));
    Rows::store(slot, v, wave, lane);
  }
};

struct Chunks {
  using Eight = u32x4;
};
__device__ __forceinline__ int codes_end(const CodeArgs& g) { return g.blocks * 32; }
__device__ __forceinline__ int codes_end(const GemmArgs& g) { return g.K; }

// XCD-aware order: workgroup b runs on XCD b % 8; each XCD takes a contiguous range.
__device__ __forceinline__ int xcd_lin(int b, int total) {
  const int full = total & ~7;
  return b >= full ? b : (b & 7) * (full >> 3) + (b >> 3);
}

}  // namespace

// Tiles of BM x BN outputs, one workgroup each, WM x WN waves; grid tiles * splits.
// Consecutive workgroups of an XCD take 8 row tiles of one column before the next, so
// the 32 that run at once share both operands in its L2.
// Two stages of both operands in LDS: the copies of stage t + 1 are requested at the
// start of step t and waited for at its end; they are issued and waited for by hand
// (the compiler's own tracking drains them at every loop head).
// The mfma's first operand is B's: a lane then holds four consecutive columns of a row.
// GatedArgs: the products of a gated layer.  Forward, a tile's B rows are those of both weights in turn, BN / 2
// columns of the result; in dx, K runs over the first half's columns and then the second's; in dw, the
// result's rows are the first half's and then the second's.
// lin is the tile's place in the order of all of them, split after split; ring holds
// kRing<BM, BN> elements of LDS.
template <int BM, int BN>
constexpr int kRing = 2 * (BM + BN) * kBK;
// and behind them, for 4-bit operands, two stages of scales
template <int BM, int BN, class G>
constexpr int kRingOf = kRing<BM, BN> + (std::is_same_v<G, MxArgs> ? ScaleStage<BM + BN>::kBytes : 0);

// Result and, in training, both arguments of a gated layer from a tile's sums, or the sums themselves where K is
// split.  A lane holds gate and up of the same elements, so the product is formed in registers, and one
// plane of BM x BN / 2 FP32 at a time goes through the ring to leave in whole lines.
template <bool HALF, int BM, int BN, int WM, int WN>
__device__ __forceinline__ void gated_epilogue(uint16_t* ring, const GatedArgs& g, f32x4 (&acc)[BM / WM / 16][BN / WN / 16],
                                               int m0, int n0, int split, float* __restrict__ part, int64_t ldpart) {
  constexpr int NW = WM * WN, FI = BM / WM / 16, FP = BN / WN / 32;  // pairs of fragments
  constexpr int kQuads = BN / 8, kRowsAtOnce = 64 * NW / kQuads, kMask = kQuads < 16 ? kQuads - 1 : 15;
  static_assert(BM * BN * 2 <= kRing<BM, BN> * 2, "a plane fits the ring");
  f32x4* plane = reinterpret_cast<f32x4*>(ring);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int c0 = wn * (BN / WN) / 8 + (lane >> 4), r0 = wm * (BM / WM) + (lane & 15);  // quad and row of this lane
  const int qn = tid % kQuads, qr = tid / kQuads, n = n0 + 4 * qn;
  const int rmax = n < g.N ? min(BM, g.M - m0) : 0;
  // value(i, j) to `to`, an array of `type` whose row m0 starts at `row0`
  auto put = [&](auto value, void* to, int type, int64_t row0, int64_t ld, int end) __attribute__((always_inline)) {
    __syncthreads();  // everyone is done with the stages, or with the last plane
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < FP; ++j) {
        const int r = r0 + 16 * i, c = c0 + 4 * j;
        plane[r * kQuads + (c ^ (r & kMask))] = value(i, j);
      }
    __syncthreads();
#pragma unroll 4
    for (int r = qr; r < rmax; r += kRowsAtOnce) {
      const f32x4 v = plane[r * kQuads + (qn ^ (r & kMask))];
      const int64_t at = row0 + r * ld + n;
      if (n + 4 <= end) {
        store_elem4(to, at, type, v);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (n + q < end) store_elem(to, at + q, type, v[q]);
      }
    }
  };
  if (part) {  // ldpart holds both halves, each a multiple of four columns
    const int64_t row0 = ((int64_t)split * g.M + m0) * ldpart;
    const int end = (int)(ldpart / 2);
    put([&](int i, int j) { return acc[i][2 * j]; }, part, kElemF32, row0, ldpart, end);
    put([&](int i, int j) { return acc[i][2 * j + 1]; }, part + ldpart / 2, kElemF32, row0, ldpart, end);
    return;
  }
  auto bias = [&](const float* b, int which) __attribute__((always_inline)) {
    if (!b) return;
#pragma unroll
    for (int j = 0; j < FP; ++j) {
      const int at = n0 + 4 * (c0 + 4 * j);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v = at + q < g.N ? b[at + q] : 0.f;
#pragma unroll
        for (int i = 0; i < FI; ++i) acc[i][2 * j + which][q] += v;
      }
    }
  };
  bias(g.bias, 0);
  bias(g.bias2, 1);
  by_act(g.act, [&](auto act) __attribute__((always_inline)) {
    put(
        [&](int i, int j) __attribute__((always_inline)) {
          f32x4 v;
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = act_f32<decltype(act)::value>(acc[i][2 * j][q]) * acc[i][2 * j + 1][q];
          return v;
        },
        g.out, g.out_type, m0 * g.ldo, g.ldo, g.N);
  });
  if (g.pre) put([&](int i, int j) { return acc[i][2 * j]; }, g.pre, g.type, m0 * g.ldp, g.ldp, g.N);
  if (g.pre2) put([&](int i, int j) { return acc[i][2 * j + 1]; }, g.pre2, g.type, m0 * g.ldp2, g.ldp2, g.N);
}

template <bool HALF, bool AT, bool BT, int BM, int BN, int WM, int WN, bool EPI, bool REGS = false, class G = GemmArgs>
__device__ __forceinline__ void gemm_tile(uint16_t* ring, G g, int mt, int nt, int lin, int k_per_split,
                                          float* __restrict__ part, int64_t ldpart) {
  constexpr bool kGated = std::is_same_v<G, GatedArgs>, kMx = std::is_same_v<G, MxArgs>;
  constexpr bool kCodes = std::is_same_v<G, CodeArgs>;
  constexpr int NW = WM * WN, FI = BM / WM / 16, FJ = BN / WN / 16;
  constexpr int kSlot = (BM + BN) * kBK;
  lds_u16* lds = (lds_u16*)ring;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int tiles = mt * nt;
  const int split = lin / tiles, t = lin % tiles;
  const int group = t / (8 * nt), in = t % (8 * nt), rows = min(8, mt - 8 * group);
  const int m0 = (8 * group + in % rows) * BM, n0 = in / rows * (kGated && EPI ? BN / 2 : BN);
  const int k0 = split * k_per_split, k1 = min(g.K, k0 + k_per_split);

  Side<AT, BM, NW> sa;
  std::conditional_t<kCodes, CodeSide<HALF, BN, NW>, Side<BT, BN, NW>> sb;
  sa.init(g.a, g.lda, m0, g.M, k0, wave, lane);
  if constexpr (kCodes)
    sb.init(g, n0, k0, wave, lane);
  else if constexpr (kGated && EPI)
    sb.init_pair(g.b, g.ldb, g.b2, g.ldb2, n0, g.N, k0, wave, lane);
  else if constexpr (kGated && !AT)
    sb.init(g.b, g.ldb, n0, g.N, min(k0, g.half - kBK), wave, lane);  // of the first half; the second's follows
  else
    sb.init(g.b, g.ldb, n0, g.N, k0, wave, lane);
  f32x4 acc[FI][FJ] = {};
  auto issue = [&](int slot, int t) {
    const int left = k1 - k0 - t * kBK;
    sa.issue(lds + slot * kSlot, left, wave, lane);
    if constexpr (kCodes) {
    } else if constexpr (kGated && !EPI && !AT) {
      const int k = k0 + t * kBK, in_half = k < g.half ? k : k - g.half;
      if (k == g.half || (t == 0 && k > g.half)) sb.init(g.b2, g.ldb2, n0, g.N, in_half, wave, lane);
      sb.issue(lds + slot * kSlot + BM * kBK, g.valid - in_half, wave, lane);
    } else {
      sb.issue(lds + slot * kSlot + BM * kBK, left, wave, lane);
    }
  };
  // 4-bit operands: a thread has a row's scales of a stage, requested a step before they go to LDS
  using Scales = ScaleStage<BM + BN>;
  using lds_u8 = typename Scales::lds_u8;
  [[maybe_unused]] lds_u8* scales = (lds_u8*)(lds + 2 * kSlot);
  [[maybe_unused]] const uint8_t* scale_row = nullptr;
  [[maybe_unused]] uint64_t next_scales = 0;
  [[maybe_unused]] auto load_scales = [&](int t) __attribute__((always_inline)) {
    if constexpr (kMx)
      if (tid < BM + BN && k0 + t * kBK < k1) next_scales = Scales::load(scale_row, (k0 + t * kBK) / 8, g.K / 8);
  };
  [[maybe_unused]] auto store_scales = [&](int t) __attribute__((always_inline)) {
    if constexpr (kMx)
      if (tid < BM + BN)
        Scales::store(scales + (t & 1) * Scales::kBytes, tid, next_scales, (k0 + t * kBK) / 8, g.K / 8);
  };
  if constexpr (kMx)
    scale_row = tid < BM ? g.sa + (int64_t)min(m0 + tid, g.M - 1) * g.ldsa
                         : g.sb + (int64_t)min(n0 + tid - BM, g.N - 1) * g.ldsb;
  auto compute = [&](int slot) __attribute__((always_inline)) {
    const lds_u16* A = lds + slot * kSlot;
    const lds_u16* B = A + BM * kBK;
    u32x4 fa[2][FI], fb[2][FJ];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int j = 0; j < FJ; ++j) fb[s][j] = Side<BT, BN, NW>::frag(B, wn * (BN / WN) + 16 * j, s, lane);
#pragma unroll
      for (int i = 0; i < FI; ++i) fa[s][i] = Side<AT, BM, NW>::frag(A, wm * (BM / WM) + 16 * i, s, lane);
    }
    if constexpr (kMx) {
      const lds_u8* stage = scales + slot * Scales::kBytes;
      u32x2 wa[(FI + 3) / 4], wb[(FJ + 3) / 4];
#pragma unroll
      for (int i = 0; i < (FI + 3) / 4; ++i) wa[i] = Scales::words(stage, wm * (BM / WM) + 64 * i, lane);
#pragma unroll
      for (int j = 0; j < (FJ + 3) / 4; ++j) wb[j] = Scales::words(stage, BM + wn * (BN / WN) + 64 * j, lane);
      static_for<2>([&](auto s) __attribute__((always_inline)) {
        static_for<FI>([&](auto i) __attribute__((always_inline)) {
          static_for<FJ>([&](auto j) __attribute__((always_inline)) {
            acc[i][j] = mfma_mx<j % 4, i % 4>(fb[s][j], fa[s][i], acc[i][j], wb[j / 4][decltype(s)::value],
                                                       wa[i / 4][decltype(s)::value]);
          });
        });
      });
      return;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) acc[i][j] = mfma<HALF>(fb[s][j], fa[s][i], acc[i][j]);
  };
  // the stage is there for every wave, and all are done with the other slot
  auto barrier = [] {
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  const int stages = (k1 - k0 + kBK - 1) / kBK;  // 0 when K is 0
  if constexpr (REGS) {
    using SA = Side<AT, BM, NW>;
    using SB = decltype(sb);
    using Eight = typename std::conditional_t<kCodes, CodeSide<HALF, BN, NW>, Chunks>::Eight;
    constexpr int kSets = BM == 64 ? 2 : 1;  // two of 128-row tiles spill
    u32x4 ra[kSets][SA::kCopies];
    Eight rb[kSets][SB::kCopies];
    // codes fill whole blocks of 32; x has zeros past its own end
    const int kb = kCodes ? min(codes_end(g) - k0, k_per_split) : k1 - k0;
    auto load = [&](auto set, int t) __attribute__((always_inline)) {
      if (t >= stages) return;
      sa.load(ra[set], k1 - k0 - t * kBK, wave, lane);
      sb.load(rb[set], kb - t * kBK, wave, lane);
    };
    auto store = [&](auto set, int t) __attribute__((always_inline)) {
      if (t >= stages) return;
      SA::store(lds + (t & 1) * kSlot, ra[set], wave, lane);
      SB::store(lds + (t & 1) * kSlot + BM * kBK, rb[set], wave, lane);
    };
    const std::integral_constant<int, 0> even;
    const std::integral_constant<int, kSets - 1> odd;
    load(even, 0);
    if constexpr (kSets == 2) {
      // stage t is requested in step t - 3 and goes to LDS in step t - 1: [1000, 1401] x [300,
      // 1401] 16.3 us, 19.8 with one set
      load(odd, 1);
      store(even, 0);
      load(even, 2);
      for (int st = 0; st < stages; st += 2) {
        barrier();
        store(odd, st + 1);
        load(odd, st + 3);
        compute(0);
        if (st + 1 == stages) break;
        barrier();
        store(even, st + 2);
        load(even, st + 4);
        compute(1);
      }
    } else {
      store(even, 0);
      for (int st = 0; st < stages; ++st) {
        barrier();
        load(even, st + 1);
        compute(st & 1);
        store(even, st + 1);
      }
    }
  } else {
    load_scales(0);
    if (stages > 0) issue(0, 0);
    store_scales(0);
    load_scales(1);
    for (int st = 0; st < stages; ++st) {
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
      barrier();
      if (st + 1 < stages) {
        store_scales(st + 1);
        load_scales(st + 2);
        issue((st + 1) & 1, st + 1);
      }
      compute(st & 1);
    }
  }

  if constexpr (kGated && EPI) {
    gated_epilogue<HALF, BM, BN, WM, WN>(ring, g, acc, m0, n0, split, part, ldpart);
    return;
  }

  // Epilogue through LDS: FP32 sums in the ring (WM / kPasses wave rows at a time), then
  // every wave takes whole rows of the tile, four columns to a lane, so memory sees full
  // lines.  16-byte chunk c of row r sits at c ^ (r & 15): the 16 rows that a wave writes
  // at once fall on distinct banks.
  constexpr int kPasses = (BM * BN * 4 + 2 * kSlot * 2 - 1) / (2 * kSlot * 2), kPassRows = BM / kPasses;
  static_assert(BM % kPasses == 0 && WM % kPasses == 0, "whole wave rows in a pass");
  f32x4* sums = reinterpret_cast<f32x4*>(ring);
  constexpr int kQuads = BN / 4, kRowsAtOnce = 64 * NW / kQuads;
  const int qn = tid % kQuads, qr = tid / kQuads;
  const int n = n0 + 4 * qn;
  auto fill = [&](int pass) __attribute__((always_inline)) {
    __syncthreads();  // everyone is done with the stages, or with the last pass
    if (wm / (WM / kPasses) == pass) {
#pragma unroll
      for (int i = 0; i < FI; ++i)
#pragma unroll
        for (int j = 0; j < FJ; ++j) {
          const int r = (wm % (WM / kPasses)) * (BM / WM) + 16 * i + (lane & 15);
          const int c = wn * (BN / WN) / 4 + 4 * j + (lane >> 4);
          sums[r * kQuads + (c ^ (r & 15))] = acc[i][j];
        }
    }
    __syncthreads();
  };
  auto sum_at = [&](int r) __attribute__((always_inline)) { return sums[r * kQuads + (qn ^ (r & 15))]; };

  // Tiles inside the result: batches of kBatch rows to a thread, the residual of the next
  // batch requested as this one's is used, so its latency shows once per tile.  A residual and
  // an FP32 result pass the caches by, which keep the operands: 500 -> 479 us at
  // [16384, 2560] x [5120, 2560] onto an FP32 stream.
  constexpr int kIters = kPassRows / kRowsAtOnce, kBatch = kIters < 8 ? kIters : 8, kBatches = kIters / kBatch;
  static_assert(kBatches * kBatch * kRowsAtOnce == kPassRows, "whole batches");
  if (EPI && !part && m0 + BM <= g.M && n0 + BN <= g.N) {
    auto inside = [&](auto out_type, auto act) __attribute__((always_inline)) {
      using OT = decltype(out_type);
      using Raw = std::conditional_t<sizeof(typename OT::S) == 4, f32x4, u32x2>;
      using RawAny = std::conditional_t<sizeof(typename OT::S) == 4, f32x4_any, u32x2_any>;
      const typename OT::S* res = static_cast<const typename OT::S*>(g.res) + (int64_t)(m0 + qr) * g.ldr + n;
      Raw rv[kBatch] = {};
      auto request = [&](int u, int row) __attribute__((always_inline)) {
        if (g.res) rv[u] = __builtin_nontemporal_load(reinterpret_cast<const RawAny*>(res + (int64_t)row * g.ldr));
      };
      f32x4 bias = {0.f, 0.f, 0.f, 0.f};
      if (g.bias) bias = *reinterpret_cast<const f32x4*>(g.bias + n);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) request(u, u * kRowsAtOnce);
#pragma unroll 1
      for (int b = 0; b < kPasses * kBatches; ++b) {
        if (b % kBatches == 0) fill(b / kBatches);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int row = (b * kBatch + u) * kRowsAtOnce;  // of the tile, before qr
          f32x4 z = sum_at(row % kPassRows + qr);
          const int m = m0 + qr + row;
          f32x4 r;
          if constexpr (sizeof(typename OT::S) == 4) {
            r = rv[u];
          } else {
            const uint32_t h[2] = {rv[u][0], rv[u][1]};
#pragma unroll
            for (int q = 0; q < 4; ++q) r[q] = OT::up((uint16_t)(h[q / 2] >> (16 * (q % 2))));
          }
          if (b + 1 < kPasses * kBatches) request(u, row + kBatch * kRowsAtOnce);
          f32x4 v;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            z[q] += bias[q];
            v[q] = g.add * act_f32<decltype(act)::value>(z[q]);
          }
          if (g.res) {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += g.keep * r[q];
          }
          if (g.pre) store_elem4(g.pre, (int64_t)m * g.ldp + n, g.type, z);
          if constexpr (sizeof(typename OT::S) == 4)
            __builtin_nontemporal_store(
                v, reinterpret_cast<f32x4_any*>(static_cast<float*>(g.out) + (int64_t)m * g.ldo + n));
          else
            store_elem4(g.out, (int64_t)m * g.ldo + n, g.type, v);
        }
      }
    };
    by_act(g.act, [&](auto act) {
      if (g.out_type == kElemF32)
        inside(F32{}, act);
      else
        inside(std::conditional_t<HALF, F16, BF16>{}, act);
    });
    return;
  }
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    fill(pass);
    const int mp = m0 + pass * kPassRows, rmax = n < g.N ? min(kPassRows, g.M - mp) : 0;
    auto rows_of = [&](auto f) __attribute__((always_inline)) {
#pragma unroll 4
      for (int r = qr; r < rmax; r += kRowsAtOnce) f(mp + r, sum_at(r));
    };
    if (part) {  // ldpart is a multiple of four and holds the columns past N
      float* p = part + (int64_t)split * g.M * ldpart + n;
      rows_of([&](int m, f32x4 v) { *reinterpret_cast<f32x4*>(p + (int64_t)m * ldpart) = v; });
    } else if constexpr (EPI) {
      by_act(g.act, [&](auto act) {
        for (int r = qr; r < rmax; r += kRowsAtOnce) epilogue4<decltype(act)::value>(g, g.add, mp + r, n, g.N, sum_at(r));
      });
    } else {
      const float add = add_of(g);
      rows_of([&](int m, f32x4 v) { gradient4(g, add, m, n, v); });
    }
  }
}

inline int sum_groups(const SumJob& j) { return j.out ? (j.cols + 15) / 16 : 0; }

template <bool HALF, bool AT, bool BT, int BM, int BN, int WM, int WN, bool EPI, bool REGS = false, class G = GemmArgs>
__global__ __launch_bounds__(64 * WM* WN) void gemm_kernel(G g, int mt, int nt, int total, int k_per_split,
                                                            float* __restrict__ part, int64_t ldpart) {
  __shared__ __align__(1024) uint16_t ring[kRingOf<BM, BN, G>];
  if constexpr (BT && !AT)
    if ((int)blockIdx.x >= total) return sum_columns(reinterpret_cast<float*>(ring), g.sums, blockIdx.x - total);
  gemm_tile<HALF, AT, BT, BM, BN, WM, WN, EPI, REGS>(ring, g, mt, nt, xcd_lin(blockIdx.x, total), k_per_split, part,
                                                     ldpart);
}

// dx = dz w and dw = dz^T x in one launch, where neither fills the card alone.  Those
// with the longer K come first.  (In 256-row tiles nothing is gained: 429 us either way at [8192,
// 5120] x [2560, 5120], 640 and 200 tiles, although fewer CUs idle; a gated layer's 640 and 400 do gain.)
template <bool HALF, int TILE, class G>
__global__ __launch_bounds__(TILE == 256 ? 512 : 256) void gemm_pair_kernel(G dx, GemmSplit sx, G dw, GemmSplit sw) {
  constexpr int WM = TILE == 256 ? 4 : 2;
  __shared__ __align__(1024) uint16_t ring[kRing<TILE, TILE>];
  const int mx = (dx.M + TILE - 1) / TILE, nx = (dx.N + TILE - 1) / TILE;
  const int mw = (dw.M + TILE - 1) / TILE, nw = (dw.N + TILE - 1) / TILE;
  const int first = mx * nx * sx.splits, second = mw * nw * sw.splits;
  int b = blockIdx.x;  // in the order dx, dw, sums
  if (b < first + second && sw.k_per_split > sx.k_per_split) b = b < second ? b + first : b - second;
  if (b < first)
    gemm_tile<HALF, false, true, TILE, TILE, WM, 2, false>(ring, dx, mx, nx, xcd_lin(b, first), sx.k_per_split,
                                                          sx.part, sx.ld);
  else if (b < first + second)
    gemm_tile<HALF, true, true, TILE, TILE, WM, 2, false>(ring, dw, mw, nw, xcd_lin(b - first, second),
                                                         sw.k_per_split, sw.part, sw.ld);
  else
    sum_columns(reinterpret_cast<float*>(ring), dx.sums, b - first - second);
}

template <bool HALF, int TILE, class G>
hipError_t launch_gemm_pair(const G& dx, const GemmSplit& sx, const G& dw, const GemmSplit& sw, hipStream_t st) {
  auto tiles = [](const GemmArgs& g) { return ((g.M + TILE - 1) / TILE) * ((g.N + TILE - 1) / TILE); };
  hipLaunchKernelGGL((gemm_pair_kernel<HALF, TILE, G>),
                     dim3(tiles(dx) * sx.splits + tiles(dw) * sw.splits + sum_groups(dx.sums)),
                     dim3(TILE == 256 ? 512 : 256), 0, st, dx, sx, dw, sw);
  return hipGetLastError();
}

// Launches the tiles of g's layout (A transposed implies B transposed).
template <bool HALF, class G>
hipError_t launch_gemm_tiles(const G& g, const GemmSplit& s, int tile, hipStream_t st) {
  const int wide = std::is_same_v<G, GatedArgs> && !g.bt ? tile / 2 : tile;  // columns
  const int mt = (g.M + tile - 1) / tile, nt = (g.N + wide - 1) / wide;
  const int total = mt * nt * s.splits;
  const dim3 grid(total + sum_groups(g.sums));
  auto go = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, st, g, mt, nt, total, s.k_per_split, s.part, s.ld);
    return hipGetLastError();
  };
  if (tile == 256) {
    if (!g.at && !g.bt) return go(gemm_kernel<HALF, false, false, 256, 256, 4, 2, true, false, G>, 512);
    if (!g.at) return go(gemm_kernel<HALF, false, true, 256, 256, 4, 2, false, false, G>, 512);
    return go(gemm_kernel<HALF, true, true, 256, 256, 4, 2, false, false, G>, 512);
  }
  if (g.regs)  // neither operand transposed
    return tile == 128 ? go(gemm_kernel<HALF, false, false, 128, 128, 2, 2, true, true, G>, 256)
                       : go(gemm_kernel<HALF, false, false, 64, 64, 2, 2, true, true, G>, 256);
  if (tile == 128) {
    if (!g.at && !g.bt) return go(gemm_kernel<HALF, false, false, 128, 128, 2, 2, true, false, G>, 256);
    if (!g.at) return go(gemm_kernel<HALF, false, true, 128, 128, 2, 2, false, false, G>, 256);
    return go(gemm_kernel<HALF, true, true, 128, 128, 2, 2, false, false, G>, 256);
  }
  if (!g.at && !g.bt) return go(gemm_kernel<HALF, false, false, 64, 64, 2, 2, true, false, G>, 256);
  if (!g.at) return go(gemm_kernel<HALF, false, true, 64, 64, 2, 2, false, false, G>, 256);
  return go(gemm_kernel<HALF, true, true, 64, 64, 2, 2, false, false, G>, 256);
}

}  // namespace beam
