// Large products in 256 x 256 tiles (gfx950): of two operands in microscaled 4 bits, and of 16-bit rows with both
// weights of a gated layer.
//
// Eight waves of 64 x 128 to a tile, and a workgroup to a CU that takes one tile after the other.  A stage of K is 128
// bytes of a row, 256 codes or 64 elements of 16 bits, 64 KB for both operands.  It costs a wave 64 matrix
// instructions of 16 cycles, 2048 cycles of each SIMD; 192 KB out of LDS, some 900 cycles; 64 KB from L2, at the 45
// to 55 bytes a nanosecond that a CU takes 1.2 to 1.4 us, as long as the products.  So all three have to run beside
// each other without a gap:
// - LDS is a ring of 19 units of 64 rows: two stages of eight, and three units more, so that memory has requests
//   while a stage is handed over.  A stage's units are free, and the next requested, once every wave has read them.
// - A wave reads a fragment two groups of four products after its last use, six groups before the next, and the
//   barrier of a stage lies between two groups, when the stage's last reads are under way for a while.
// - Copies are requested between the groups, one or two at a time, in as few instructions as that takes: a wave
//   issues one every four cycles, some seven between two of its products.
// - Scales come as tiles of their own: mx_scales_kernel lays them out by tile and stage in the order of the matrix
//   instructions' words, so that a stage's are 4 KB in a row (as they lie, a row's eight bytes to a cache line,
//   they took a third as long as the codes).
// - Results leave from registers, and the next tile's first stages are requested before.
// A stage of 4-bit operands takes 1.8 us, and 6 us lie between the last stage of one tile and the first of the next (calls
// with K of 512 to 10240 at [16384, K] x [5120, K]): twice the 0.94 us of its matrix instructions, so there it is bound by
// its feeding and, with a short K, by the epilogues.  [16384, 2560] x [5120, 2560] takes 123 to 131 us in calls (3.3 to 3.5
// PFLOP/s), of which the results' stores are 25 to 30; under the profiler, with inputs out of memory, 149, the matrix cores
// 31% busy at 2.17 GHz.  The largest products run into power, busy times clock near 1 GHz: 53% at 1.87 GHz at 8192^3 (260
// us, 4.2 PFLOP/s; 300 in the tiled product), 59% at 1.66 for [16384, 5120] x [2560, 5120] of a gated layer in bf16 (670 us
// in calls, 1280 TFLOP/s).
// A tile of a gated layer has 16 rows of one weight and 16 of the other in turn, 128 columns of the result.
#pragma once

#include <cstddef>

#include "gemm_tiles.h"

namespace beam {
namespace {

constexpr int kT = 256, kFI = 4, kFJ = 8;
constexpr int kUnit = 8192;       // bytes: 64 rows, 128 bytes of each
constexpr int kUnits = 19;
constexpr int kScales = 4096;     // bytes of a stage's scales, A's and then B's
static_assert(kUnits * kUnit + 2 * kScales <= 160 * 1024, "LDS");

// 16 bytes a lane to LDS, from base + off.
__device__ __forceinline__ void lds_copy16_at(const uint8_t* base, uint32_t off, uint32_t lds_base) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "global_load_lds_dwordx4 %1, %2\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(off), "s"(base), "s"(lds_base)
      : "memory");
}

// Fragments j and j + 1 of a 16-bit result, four columns to a lane in two words each, to eight columns to a lane, and
// back: a lane of 16-lane row r then holds columns 8 (r / 2) .. + 7 of fragment j + r % 2.
__device__ __forceinline__ u32x4 swap_fragments(u32x4 v) {  // (j low, j high, j + 1 low, j + 1 high)
  const auto a = __builtin_amdgcn_permlane16_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(v[1], v[3], false, false);
  return u32x4{a[0], b[0], a[1], b[1]};
}

// HALF: fp16 operands of a gated layer, not bf16; OT: the result's type.
template <class G, bool HALF, class OT>
__global__ __launch_bounds__(512) void stream_kernel(G g, int mt, int nt) {
  constexpr bool kMx = std::is_same_v<G, MxArgs>;
  constexpr int kOut = std::is_same_v<OT, F32> ? kElemF32 : std::is_same_v<OT, F16> ? kElemF16 : kElemBF16;
  constexpr bool kWide = kOut == kElemF32;
  constexpr int kCols = kMx ? kT : kT / 2;  // of the result, to a tile
  constexpr int kFrags = kMx ? kFJ : kFJ / 2;  // of 16 of them, to a wave
  constexpr int kStores = kWide ? kFI * kFrags : kFI * kFrags / 2;  // of a whole tile, to a wave
  __shared__ __align__(1024) uint8_t ring[kUnits * kUnit + (kMx ? 2 * kScales : 0)];
  typedef __attribute__((address_space(3))) uint8_t lds_u8;
  lds_u8* lds = (lds_u8*)ring;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, l16 = lane & 15, gr = lane >> 4;
  const int row_bytes = g.K * 2, stages = (row_bytes + 127) / 128;

  // this workgroup's tiles: an XCD's are consecutive, and 32 at a time share both operands in its L2
  const int total = mt * nt, xcd = blockIdx.x & 7, per = total >> 3, step = gridDim.x >> 3;
  const int mine = per + (xcd < (total & 7)), first = blockIdx.x >> 3;
  if (first >= mine) return;
  const int tiles = (mine - first + step - 1) / step, steps = tiles * stages;
  struct Place {
    int mi, ni;  // tiles
  };
  auto place = [&](int i) {
    const int l = first + i * step, t = l < per ? xcd * per + l : (total & ~7) + xcd;
    const int group = t / (8 * nt), in = t % (8 * nt), rows = min(8, mt - 8 * group);
    return Place{8 * group + in % rows, in / rows};
  };

  // What is copied next: stage `c_stage` of tile `c_tile`, c_steps stages with it to go, to LDS from c_to on.  A wave
  // copies an eighth of every unit, eight rows.
  int c_tile = 0, c_stage = 0, c_steps = steps;
  const uint32_t ring_from = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds + wave * 1024);
  const uint32_t ring_end = ring_from + kUnits * kUnit;
  uint32_t c_to = ring_from;
  const uint8_t *c_a = nullptr, *c_b = nullptr;
  uint32_t off_a[4], off_b[4], back = 0;
  const uint64_t lda = (uint64_t)g.lda * 2;
  const void* b = g.b;
  uint64_t ldb = (uint64_t)g.ldb * 2;
  if constexpr (!kMx)
    if (wave & 2) {  // this wave's rows are the second weight's
      b = g.b2;
      ldb = (uint64_t)g.ldb2 * 2;
    }
  const int copy_row = wave * 8 + (lane >> 3), copy_chunk = (lane & 7) ^ ((copy_row >> 1) & 7);
  auto copy = [&](auto kk) __attribute__((always_inline)) {
    constexpr int k = decltype(kk)::value;  // A's units 0 .. 3, then B's
    if (c_steps <= 0) return;
    if (k == 0) {
      // codes past K repeat the last chunk: their scales are 0, 2^-127 on either side, so they add nothing
      if (kMx) back = (uint32_t)max(16 * copy_chunk - (row_bytes - c_stage * 128 - 16), 0);
      if (c_stage == 0) {
        const Place p = place(c_tile);
        c_a = static_cast<const uint8_t*>(g.a) + p.mi * kT * lda;
        c_b = static_cast<const uint8_t*>(b) + p.ni * kCols * ldb;
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // rows past the end repeat the last; their results are not stored
          const int row = kMx ? q * 64 + copy_row : q * 32 + (copy_row >> 5) * 16 + (copy_row & 15);
          off_a[q] = (uint32_t)min(q * 64 + copy_row, g.M - 1 - p.mi * kT) * (uint32_t)lda + 16 * copy_chunk;
          off_b[q] = (uint32_t)min(row, g.N - 1 - p.ni * kCols) * (uint32_t)ldb + 16 * copy_chunk;
        }
      }
    }
    lds_copy16_at(k < 4 ? c_a : c_b, (k < 4 ? off_a[k & 3] : off_b[k & 3]) - back, c_to);
    c_to += kUnit;
    if (c_to == ring_end) c_to = ring_from;
    if (k == 7) {
      c_a += 128;
      c_b += 128;
      --c_steps;
      if (++c_stage == stages) c_stage = 0, ++c_tile;
    }
  };
  // The scales of a stage, of 4-bit operands: 1 KB to each of the first four waves, two of them A's.
  int s_tile = 0, s_stage = 0;
  const uint8_t* s_from = nullptr;
  auto copy_scales = [&](int slot) __attribute__((always_inline)) {
    if constexpr (kMx) {
      if (wave >= 4 || s_tile == tiles) return;
      if (s_stage == 0) {
        const Place p = place(s_tile);
        s_from = (wave < 2 ? g.sa + (int64_t)p.mi * stages * (kScales / 2)
                           : g.sb + (int64_t)p.ni * stages * (kScales / 2)) + (wave & 1) * 1024;
      }
      lds_copy16_at(s_from, lane * 16, ring_end + slot * kScales);
      s_from += kScales / 2;
      if (++s_stage == stages) s_stage = 0, ++s_tile;
    }
  };

  f32x4 acc[kFI][kFJ] = {};
  u32x4 fa[2][kFI], fb[kFJ];  // A's fragments of both halves, and B's as they are wanted next
  uint32_t sa[2], sb[2][2];
  const uint32_t at = l16 * 128 + ((gr ^ ((l16 >> 1) & 7)) << 4);  // in a unit; the second half's differs in one bit
  const uint32_t scale_at = gr * 128 + l16 * 8;
  // the units of this wave's rows in the stage that starts at unit u
  struct Units {
    uint32_t a, b0, b1;
  };
  auto units = [&](int u) __attribute__((always_inline)) {
    auto wrap = [](int v) { return (uint32_t)(v >= kUnits ? v - kUnits : v) * kUnit; };
    return Units{wrap(u + wm), wrap(u + 4 + 2 * wn), wrap(u + 5 + 2 * wn)};
  };
  auto read_b = [&](int j, const Units& u, int s) __attribute__((always_inline)) {
    fb[j] = *(const __attribute__((address_space(3))) u32x4*)(lds + (j < 4 ? u.b0 : u.b1) + (at ^ (64 * s)) + j % 4 * 2048);
  };
  auto read_a = [&](int i, const Units& u, int s) __attribute__((always_inline)) {
    fa[s][i] = *(const __attribute__((address_space(3))) u32x4*)(lds + u.a + (at ^ (64 * s)) + i * 2048);
  };
  auto read_scales = [&](int slot, int s) __attribute__((always_inline)) {
    if constexpr (!kMx) return;
    const lds_u8* q = lds + kUnits * kUnit + slot * kScales + 4 * s + scale_at;
    sa[s] = *(const __attribute__((address_space(3))) uint32_t*)(q + wm * 512);
    sb[s][0] = *(const __attribute__((address_space(3))) uint32_t*)(q + (4 + 2 * wn) * 512);
    sb[s][1] = *(const __attribute__((address_space(3))) uint32_t*)(q + (5 + 2 * wn) * 512);
  };
  auto group = [&](auto s, auto j) __attribute__((always_inline)) {
    constexpr int S = decltype(s)::value, J = decltype(j)::value;
    static_for<kFI>([&](auto i) __attribute__((always_inline)) {
      constexpr int I = decltype(i)::value;
      if constexpr (kMx)
        acc[I][J] = mfma_mx<J % 4, I>(fb[J], fa[S][I], acc[I][J], sb[S][J / 4], sa[S]);
      else
        acc[I][J] = mfma<HALF>(fb[J], fa[S][I], acc[I][J]);
    });
    // a product stays in its group: the compiler would move it behind the branches that follow
#pragma unroll
    for (int i = 0; i < kFI; ++i) {
      f32x4& v = acc[i][J];
      asm volatile("" : "+v"(v));
    }
  };
  auto barrier = [] {
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // the groups' order is the program's; nothing of one moves into another
  auto fence = [] { __builtin_amdgcn_sched_barrier(0); };

  copy_scales(0);
  static_for<8>(copy);
  copy_scales(1);
  static_for<8>(copy);
  static_for<3>(copy);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  barrier();
  int unit = 0, stage = 0, tile = 0;
  int pending = 0;  // of the last tile's stores: 0 none, 1 kStores, 2 some other number
  Units now = units(0);
  read_scales(0, 0);
#pragma unroll
  for (int i = 0; i < kFI; ++i) read_a(i, now, 0);
#pragma unroll
  for (int j = 0; j < kFJ - 2; ++j) read_b(j, now, 0);
  const std::integral_constant<int, 0> half0;
  const std::integral_constant<int, 1> half1;
#pragma unroll 1
  for (int f = 0; f < steps; ++f) {
    const int slot = f & 1;
    static_for<kFJ>([&](auto j) __attribute__((always_inline)) {
      constexpr int J = decltype(j)::value;
      group(half0, j);
      if constexpr (J < 2) read_b(J + 6, now, 0);
      if constexpr (J >= 2) read_b(J - 2, now, 1);
      if constexpr (J == 1) read_scales(slot, 1);
      if constexpr (J >= 2 && J < 6) read_a(J - 2, now, 1);
      fence();
    });
    group(half1, std::integral_constant<int, 0>{});
    read_b(6, now, 1);
    fence();
    group(half1, std::integral_constant<int, 1>{});
    read_b(7, now, 1);
    fence();
    group(half1, std::integral_constant<int, 2>{});
    fence();
    // The next stage has to be there; three units of the one after it, and stores behind them, may be under way.
    if (f + 2 >= steps || pending == 2)
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    else if (pending == 1)
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(3 + kStores));
    else
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(3));
    pending = 0;
    barrier();
    unit += 8;
    if (unit >= kUnits) unit -= kUnits;
    now = units(unit);
    static_for<kFJ>([&](auto j) __attribute__((always_inline)) {
      constexpr int J = decltype(j)::value;
      if constexpr (J > 2) group(half1, j);
      if constexpr (J >= 2) read_b(J - 2, now, 0);
      if constexpr (J == 2) read_scales(slot ^ 1, 0);
      if constexpr (J >= 3 && J < 7) read_a(J - 3, now, 0);
      if constexpr (J == 2) copy_scales(slot);
      if constexpr (J == 2 || J == 3) {
        copy(std::integral_constant<int, 2 * J - 1>{});
        copy(std::integral_constant<int, 2 * J>{});
      }
      if constexpr (J > 3) copy(std::integral_constant<int, (J + 3) % 8>{});
      fence();
    });
    if (++stage < stages) continue;
    stage = 0;
    const Place p = place(tile++);
    const int m = p.mi * kT + wm * 64 + l16, n = p.ni * kCols + wn * (kCols / 2);
    const bool inside = (p.mi + 1) * kT <= g.M && (p.ni + 1) * kCols <= g.N;
    if constexpr (kMx)
      pending = inside && !g.bias && !g.res ? 1 : 2;
    else
      pending = inside && !g.bias && !g.bias2 && !g.pre && !g.pre2 ? 1 : 2;
    // whole chunks of columns, eight to a lane: all but the last tiles of a row of results where N is no multiple
    const bool whole = (p.ni + 1) * kCols <= g.N || g.N % 8 == 0;
    // value(i, j), four columns of fragment j, and keep times a residual to `to`, rows of ld elements of T.
    auto put = [&](auto type, void* to, int64_t ld, auto value, auto residual) __attribute__((always_inline)) {
      using T = decltype(type);
      constexpr int kType = std::is_same_v<T, F32> ? kElemF32 : std::is_same_v<T, F16> ? kElemF16 : kElemBF16;
      constexpr bool kRes = !std::is_same_v<decltype(residual), std::nullptr_t>;
      typename T::S* out = static_cast<typename T::S*>(to);
      if (whole) {
#pragma unroll
        for (int i = 0; i < kFI; ++i) {
          const int end = m + 16 * i < g.M ? g.N : 0;  // of the columns that this row stores
          if constexpr (kType == kElemF32) {
            const int64_t o = (int64_t)(m + 16 * i) * ld + n + 4 * gr, r = (int64_t)(m + 16 * i) * g.ldr + n + 4 * gr;
#pragma unroll
            for (int j = 0; j < kFrags; ++j) {
              f32x4 v = value(i, j);
              const bool here = n + 4 * gr + 16 * j < end;
              if constexpr (kRes)
                if (residual && here) {
                  const f32x4 w = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(residual + r + 16 * j));
#pragma unroll
                  for (int q = 0; q < 4; ++q) v[q] += g.keep * w[q];
                }
              if (here) __builtin_nontemporal_store(v, reinterpret_cast<f32x4_any*>(out + o + 16 * j));
              fence();
            }
          } else {
            const int c = n + 16 * (gr & 1) + 8 * (gr >> 1);
            const int64_t o = (int64_t)(m + 16 * i) * ld + c, r = (int64_t)(m + 16 * i) * g.ldr + c;
#pragma unroll
            for (int j = 0; j < kFrags; j += 2) {
              f32x4 v = value(i, j), w = value(i, j + 1);
              const bool here = c + 16 * j < end;
              if constexpr (kRes)
                if (residual) {
                  u32x4 raw = {0u, 0u, 0u, 0u};
                  if (here) raw = *reinterpret_cast<const u32x4_any*>(residual + r + 16 * j);
                  raw = swap_fragments(raw);
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    v[q] += g.keep * T::up((uint16_t)(raw[q / 2] >> (16 * (q % 2))));
                    w[q] += g.keep * T::up((uint16_t)(raw[2 + q / 2] >> (16 * (q % 2))));
                  }
                }
              u32x4 h;
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                h[q] = T::down(v[2 * q]) | (uint32_t)T::down(v[2 * q + 1]) << 16;
                h[2 + q] = T::down(w[2 * q]) | (uint32_t)T::down(w[2 * q + 1]) << 16;
              }
              h = swap_fragments(h);
              if (here) *reinterpret_cast<u32x4_any*>(out + o + 16 * j) = h;
              fence();
            }
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kFI; ++i)
#pragma unroll
          for (int j = 0; j < kFrags; ++j) {
            const int mm = m + 16 * i, c = n + 16 * j + 4 * gr, left = g.N - c;
            if (mm < g.M && left > 0) {
              const int64_t o = (int64_t)mm * ld + c, r = (int64_t)mm * g.ldr + c;
              f32x4 v = value(i, j);
              if constexpr (kRes)
                if (residual) {
                  if (left >= 4) {
                    const f32x4 w = load_elem4(residual, r, kType);
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] += g.keep * w[q];
                  } else {
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                      if (q < left) v[q] += g.keep * load_elem(residual, r + q, kType);
                  }
                }
              if (left >= 4) {
                store_elem4(out, o, kType, v);
              } else {
#pragma unroll
                for (int q = 0; q < 3; ++q)
                  if (q < left) store_elem(out, o + q, kType, v[q]);
              }
            }
            fence();
          }
      }
    };
    // four columns of a bias from c on, 0 past N
    auto bias4 = [&](const float* bias, int c) __attribute__((always_inline)) {
      f32x4 b = {0.f, 0.f, 0.f, 0.f};
      if (bias && c + 4 <= g.N) {
        b = *reinterpret_cast<const f32x4_any*>(bias + c);
      } else if (bias) {
#pragma unroll
        for (int q = 0; q < 3; ++q)
          if (c + q < g.N) b[q] = bias[c + q];
      }
      return b;
    };
    if constexpr (kMx) {
      by_act(g.act, [&](auto act) __attribute__((always_inline)) {
        put(
            OT{}, g.out, g.ldo,
            [&](int i, int j) __attribute__((always_inline)) {
              f32x4 z = acc[i][j];
              const f32x4 b = bias4(g.bias, n + 16 * j + 4 * gr);
#pragma unroll
              for (int q = 0; q < 4; ++q) z[q] = g.add * act_f32<decltype(act)::value>(z[q] + b[q]);
              return z;
            },
            static_cast<const typename OT::S*>(g.res));
      });
    } else {
      if (g.bias || g.bias2) {
#pragma unroll
        for (int j = 0; j < kFrags; ++j) {
          const f32x4 b = bias4(g.bias, n + 16 * j + 4 * gr), c = bias4(g.bias2, n + 16 * j + 4 * gr);
#pragma unroll
          for (int i = 0; i < kFI; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              acc[i][2 * j][q] += b[q];
              acc[i][2 * j + 1][q] += c[q];
            }
        }
      }
      by_act(g.act, [&](auto act) __attribute__((always_inline)) {
        put(
            OT{}, g.out, g.ldo,
            [&](int i, int j) __attribute__((always_inline)) {
              f32x4 v;
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = act_f32<decltype(act)::value>(acc[i][2 * j][q]) * acc[i][2 * j + 1][q];
              return v;
            },
            nullptr);
      });
      using PT = std::conditional_t<HALF, F16, BF16>;
      if (g.pre) put(PT{}, g.pre, g.ldp, [&](int i, int j) { return acc[i][2 * j]; }, nullptr);
      if (g.pre2) put(PT{}, g.pre2, g.ldp2, [&](int i, int j) { return acc[i][2 * j + 1]; }, nullptr);
    }
#pragma unroll
    for (int i = 0; i < kFI; ++i)
#pragma unroll
      for (int j = 0; j < kFJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
}

}  // namespace
}  // namespace beam
