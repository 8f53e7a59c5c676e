// The tiled MFMA product of linear.hip, instantiated once for each 16-bit type.
#pragma once

#include <type_traits>

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
// lin is the tile's place in the order of all of them, split after split; ring holds
// kRing<BM, BN> elements of LDS.
template <int BM, int BN>
constexpr int kRing = 2 * (BM + BN) * kBK;

template <bool HALF, bool AT, bool BT, int BM, int BN, int WM, int WN, bool EPI, bool REGS = false>
__device__ __forceinline__ void gemm_tile(uint16_t* ring, GemmArgs g, int mt, int nt, int lin, int k_per_split,
                                          float* __restrict__ part, int64_t ldpart) {
  constexpr int NW = WM * WN, FI = BM / WM / 16, FJ = BN / WN / 16;
  constexpr int kSlot = (BM + BN) * kBK;
  lds_u16* lds = (lds_u16*)ring;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int tiles = mt * nt;
  const int split = lin / tiles, t = lin % tiles;
  const int group = t / (8 * nt), in = t % (8 * nt), rows = min(8, mt - 8 * group);
  const int m0 = (8 * group + in % rows) * BM, n0 = in / rows * BN;
  const int k0 = split * k_per_split, k1 = min(g.K, k0 + k_per_split);

  Side<AT, BM, NW> sa;
  Side<BT, BN, NW> sb;
  sa.init(g.a, g.lda, m0, g.M, k0, wave, lane);
  sb.init(g.b, g.ldb, n0, g.N, k0, wave, lane);
  f32x4 acc[FI][FJ] = {};
  auto issue = [&](int slot, int left) {
    sa.issue(lds + slot * kSlot, left, wave, lane);
    sb.issue(lds + slot * kSlot + BM * kBK, left, wave, lane);
  };
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
    using SB = Side<BT, BN, NW>;
    constexpr int kSets = BM == 64 ? 2 : 1;  // two of 128-row tiles spill
    u32x4 ra[kSets][SA::kCopies], rb[kSets][SB::kCopies];
    auto load = [&](auto set, int t) __attribute__((always_inline)) {
      if (t >= stages) return;
      sa.load(ra[set], k1 - k0 - t * kBK, wave, lane);
      sb.load(rb[set], k1 - k0 - t * kBK, wave, lane);
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
    if (stages > 0) issue(0, k1 - k0);
    for (int st = 0; st < stages; ++st) {
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
      barrier();
      if (st + 1 < stages) issue((st + 1) & 1, k1 - k0 - (st + 1) * kBK);
      compute(st & 1);
    }
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

// The column sums that run beside dx's product, in workgroups behind its tiles: b's are those
// of 16 columns, thread (c, g) adds the rows g, g + 16, ... of column c, and a column's 16
// sums are added in order, in FP64.  As a launch of their own they take 3 to 5 us, mostly
// latency.
__device__ __forceinline__ void sum_columns(float* s, const SumJob& j, int b) {
  const int tid = threadIdx.x, c = tid & 15, h = b * 16 + c;
  float v = 0.f;
  if (tid < 256 && h < j.cols)
#pragma unroll 16
    for (int u = tid >> 4; u < j.units; u += 16) v += j.part[(int64_t)u * j.cols + h];
  s[tid] = v;
  __syncthreads();
  if (tid < 16 && h < j.cols) {
    double a = 0.0;
#pragma unroll
    for (int g = 0; g < 16; ++g) a += s[16 * g + c];
    j.out[h] = (float)a;
  }
}
inline int sum_groups(const SumJob& j) { return j.out ? (j.cols + 15) / 16 : 0; }

template <bool HALF, bool AT, bool BT, int BM, int BN, int WM, int WN, bool EPI, bool REGS = false>
__global__ __launch_bounds__(64 * WM* WN) void gemm_kernel(GemmArgs g, int mt, int nt, int total, int k_per_split,
                                                            float* __restrict__ part, int64_t ldpart) {
  __shared__ __align__(1024) uint16_t ring[kRing<BM, BN>];
  if constexpr (BT && !AT)
    if ((int)blockIdx.x >= total) return sum_columns(reinterpret_cast<float*>(ring), g.sums, blockIdx.x - total);
  gemm_tile<HALF, AT, BT, BM, BN, WM, WN, EPI, REGS>(ring, g, mt, nt, xcd_lin(blockIdx.x, total), k_per_split, part,
                                                     ldpart);
}

// dx = dz w and dw = dz^T x in one launch, where neither fills the card alone.  Those
// with the longer K come first.  (In 256-row tiles nothing is gained: 429 us either way at [8192,
// 5120] x [2560, 5120], 640 and 200 tiles, although fewer CUs idle.)
template <bool HALF, int TILE>
__global__ __launch_bounds__(256) void gemm_pair_kernel(GemmArgs dx, GemmSplit sx, GemmArgs dw, GemmSplit sw) {
  __shared__ __align__(1024) uint16_t ring[kRing<TILE, TILE>];
  const int mx = (dx.M + TILE - 1) / TILE, nx = (dx.N + TILE - 1) / TILE;
  const int mw = (dw.M + TILE - 1) / TILE, nw = (dw.N + TILE - 1) / TILE;
  const int first = mx * nx * sx.splits, second = mw * nw * sw.splits;
  int b = blockIdx.x;  // in the order dx, dw, sums
  if (b < first + second && sw.k_per_split > sx.k_per_split) b = b < second ? b + first : b - second;
  if (b < first)
    gemm_tile<HALF, false, true, TILE, TILE, 2, 2, false>(ring, dx, mx, nx, xcd_lin(b, first), sx.k_per_split,
                                                          sx.part, sx.ld);
  else if (b < first + second)
    gemm_tile<HALF, true, true, TILE, TILE, 2, 2, false>(ring, dw, mw, nw, xcd_lin(b - first, second),
                                                         sw.k_per_split, sw.part, sw.ld);
  else
    sum_columns(reinterpret_cast<float*>(ring), dx.sums, b - first - second);
}

template <bool HALF, int TILE>
hipError_t launch_gemm_pair(const GemmArgs& dx, const GemmSplit& sx, const GemmArgs& dw, const GemmSplit& sw,
                            hipStream_t st) {
  auto tiles = [](const GemmArgs& g) { return ((g.M + TILE - 1) / TILE) * ((g.N + TILE - 1) / TILE); };
  hipLaunchKernelGGL((gemm_pair_kernel<HALF, TILE>),
                     dim3(tiles(dx) * sx.splits + tiles(dw) * sw.splits + sum_groups(dx.sums)), dim3(256), 0, st, dx,
                     sx, dw, sw);
  return hipGetLastError();
}

// Launches the tiles of g's layout (A transposed implies B transposed).
template <bool HALF>
hipError_t launch_gemm_tiles(const GemmArgs& g, const GemmSplit& s, int tile, hipStream_t st) {
  const int mt = (g.M + tile - 1) / tile, nt = (g.N + tile - 1) / tile;
  const int total = mt * nt * s.splits;
  const dim3 grid(total + sum_groups(g.sums));
  auto go = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, st, g, mt, nt, total, s.k_per_split, s.part, s.ld);
    return hipGetLastError();
  };
  if (tile == 256) {
    if (!g.at && !g.bt) return go(gemm_kernel<HALF, false, false, 256, 256, 4, 2, true>, 512);
    if (!g.at) return go(gemm_kernel<HALF, false, true, 256, 256, 4, 2, false>, 512);
    return go(gemm_kernel<HALF, true, true, 256, 256, 4, 2, false>, 512);
  }
  if (g.regs)  // neither operand transposed
    return tile == 128 ? go(gemm_kernel<HALF, false, false, 128, 128, 2, 2, true, true>, 256)
                       : go(gemm_kernel<HALF, false, false, 64, 64, 2, 2, true, true>, 256);
  if (tile == 128) {
    if (!g.at && !g.bt) return go(gemm_kernel<HALF, false, false, 128, 128, 2, 2, true>, 256);
    if (!g.at) return go(gemm_kernel<HALF, false, true, 128, 128, 2, 2, false>, 256);
    return go(gemm_kernel<HALF, true, true, 128, 128, 2, 2, false>, 256);
  }
  if (!g.at && !g.bt) return go(gemm_kernel<HALF, false, false, 64, 64, 2, 2, true>, 256);
  if (!g.at) return go(gemm_kernel<HALF, false, true, 64, 64, 2, 2, false>, 256);
  return go(gemm_kernel<HALF, true, true, 64, 64, 2, 2, false>, 256);
}

}  // namespace beam
