// The large product of two operands in microscaled 4 bits (gfx950), one instantiation to an output type.
//
// 256 x 256 outputs to a tile, eight waves of 64 x 128, and a workgroup to a CU that takes one tile after the other.
// What a stage of K (256 codes, 128 bytes a row, 64 KB for both operands) costs: 64 scaled matrix instructions of 16
// cycles to a wave, 2048 cycles of each SIMD; 192 KB out of LDS, some 900 cycles; 64 KB from L2, at the 45 to 55 bytes
// a nanosecond that a CU takes 1.2 to 1.4 us, as long as the products.  So all three have to run beside each other
// without a gap:
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
#pragma once

#include "gemm_tiles.h"

namespace beam {
namespace {

constexpr int kMxT = 256, kMxFI = 4, kMxFJ = 8;
constexpr int kMxUnit = 8192;       // bytes: 64 rows, 128 bytes of each
constexpr int kMxUnits = 19;
constexpr int kMxScales = 4096;     // bytes of a stage's scales, A's and then B's
static_assert(kMxUnits * kMxUnit + 2 * kMxScales <= 160 * 1024, "LDS");

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

template <class OT>
__global__ __launch_bounds__(512) void mx_stream_kernel(MxArgs g, int mt, int nt) {
  constexpr int kOut = std::is_same_v<OT, F32> ? kElemF32 : std::is_same_v<OT, F16> ? kElemF16 : kElemBF16;
  constexpr bool kWide = kOut == kElemF32;
  constexpr int kStores = kWide ? kMxFI * kMxFJ : kMxFI * kMxFJ / 2;  // of a whole tile, to a wave
  __shared__ __align__(1024) uint8_t ring[kMxUnits * kMxUnit + 2 * kMxScales];
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
  const uint32_t ring_end = ring_from + kMxUnits * kMxUnit;
  uint32_t c_to = ring_from;
  const uint8_t *c_a = nullptr, *c_b = nullptr;
  uint32_t off_a[4], off_b[4], back = 0;
  const uint64_t lda = (uint64_t)g.lda * 2, ldb = (uint64_t)g.ldb * 2;
  const int copy_row = wave * 8 + (lane >> 3), copy_chunk = (lane & 7) ^ ((copy_row >> 1) & 7);
  auto copy = [&](auto kk) __attribute__((always_inline)) {
    constexpr int k = decltype(kk)::value;  // A's units 0 .. 3, then B's
    if (c_steps <= 0) return;
    if (k == 0) {
      // chunks past K repeat the last one: their scales are 0, 2^-127 on either side, so they add nothing
      back = (uint32_t)max(16 * copy_chunk - (row_bytes - c_stage * 128 - 16), 0);
      if (c_stage == 0) {
        const Place p = place(c_tile);
        c_a = static_cast<const uint8_t*>(g.a) + p.mi * kMxT * lda;
        c_b = static_cast<const uint8_t*>(g.b) + p.ni * kMxT * ldb;
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // rows past the end repeat the last; their results are not stored
          off_a[q] = (uint32_t)min(q * 64 + copy_row, g.M - 1 - p.mi * kMxT) * (uint32_t)lda + 16 * copy_chunk;
          off_b[q] = (uint32_t)min(q * 64 + copy_row, g.N - 1 - p.ni * kMxT) * (uint32_t)ldb + 16 * copy_chunk;
        }
      }
    }
    lds_copy16_at(k < 4 ? c_a : c_b, (k < 4 ? off_a[k & 3] : off_b[k & 3]) - back, c_to);
    c_to += kMxUnit;
    if (c_to == ring_end) c_to = ring_from;
    if (k == 7) {
      c_a += 128;
      c_b += 128;
      --c_steps;
      if (++c_stage == stages) c_stage = 0, ++c_tile;
    }
  };
  // The scales of a stage: 1 KB to each of the first four waves, two of them A's.
  int s_tile = 0, s_stage = 0;
  const uint8_t* s_from = nullptr;
  auto copy_scales = [&](int slot) __attribute__((always_inline)) {
    if (wave >= 4 || s_tile == tiles) return;
    if (s_stage == 0) {
      const Place p = place(s_tile);
      s_from = (wave < 2 ? g.sa + (int64_t)p.mi * stages * (kMxScales / 2)
                         : g.sb + (int64_t)p.ni * stages * (kMxScales / 2)) + (wave & 1) * 1024;
    }
    lds_copy16_at(s_from, lane * 16, ring_end + slot * kMxScales);
    s_from += kMxScales / 2;
    if (++s_stage == stages) s_stage = 0, ++s_tile;
  };

  f32x4 acc[kMxFI][kMxFJ] = {};
  u32x4 fa[2][kMxFI], fb[kMxFJ];  // A's fragments of both halves, and B's as they are wanted next
  uint32_t sa[2], sb[2][2];
  const uint32_t at = l16 * 128 + ((gr ^ ((l16 >> 1) & 7)) << 4);  // in a unit; the second half's differs in one bit
  const uint32_t scale_at = gr * 128 + l16 * 8;
  // the units of this wave's rows in the stage that starts at unit u
  struct Units {
    uint32_t a, b0, b1;
  };
  auto units = [&](int u) __attribute__((always_inline)) {
    auto wrap = [](int v) { return (uint32_t)(v >= kMxUnits ? v - kMxUnits : v) * kMxUnit; };
    return Units{wrap(u + wm), wrap(u + 4 + 2 * wn), wrap(u + 5 + 2 * wn)};
  };
  auto read_b = [&](int j, const Units& u, int s) __attribute__((always_inline)) {
    fb[j] = *(const __attribute__((address_space(3))) u32x4*)(lds + (j < 4 ? u.b0 : u.b1) + (at ^ (64 * s)) + j % 4 * 2048);
  };
  auto read_a = [&](int i, const Units& u, int s) __attribute__((always_inline)) {
    fa[s][i] = *(const __attribute__((address_space(3))) u32x4*)(lds + u.a + (at ^ (64 * s)) + i * 2048);
  };
  auto read_scales = [&](int slot, int s) __attribute__((always_inline)) {
    const lds_u8* q = lds + kMxUnits * kMxUnit + slot * kMxScales + 4 * s + scale_at;
    sa[s] = *(const __attribute__((address_space(3))) uint32_t*)(q + wm * 512);
    sb[s][0] = *(const __attribute__((address_space(3))) uint32_t*)(q + (4 + 2 * wn) * 512);
    sb[s][1] = *(const __attribute__((address_space(3))) uint32_t*)(q + (5 + 2 * wn) * 512);
  };
  auto group = [&](auto s, auto j) __attribute__((always_inline)) {
    constexpr int S = decltype(s)::value, J = decltype(j)::value;
    static_for<kMxFI>([&](auto i) __attribute__((always_inline)) {
      constexpr int I = decltype(i)::value;
      acc[I][J] = mfma_mx<J % 4, I>(fb[J], fa[S][I], acc[I][J], sb[S][J / 4], sa[S]);
    });
    // a product stays in its group: the compiler would move it behind the branches that follow
#pragma unroll
    for (int i = 0; i < kMxFI; ++i) {
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
  for (int i = 0; i < kMxFI; ++i) read_a(i, now, 0);
#pragma unroll
  for (int j = 0; j < kMxFJ - 2; ++j) read_b(j, now, 0);
  const std::integral_constant<int, 0> half0;
  const std::integral_constant<int, 1> half1;
#pragma unroll 1
  for (int f = 0; f < steps; ++f) {
    const int slot = f & 1;
    static_for<kMxFJ>([&](auto j) __attribute__((always_inline)) {
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
    if (unit >= kMxUnits) unit -= kMxUnits;
    now = units(unit);
    static_for<kMxFJ>([&](auto j) __attribute__((always_inline)) {
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
    const int m = p.mi * kMxT + wm * 64 + l16, n = p.ni * kMxT + wn * 128;
    const bool inside = (p.mi + 1) * kMxT <= g.M && (p.ni + 1) * kMxT <= g.N;
    pending = inside && !g.bias && !g.res ? 1 : 2;
    typename OT::S* out = static_cast<typename OT::S*>(g.out);
    const typename OT::S* res = static_cast<const typename OT::S*>(g.res);
    auto results = [&](auto act) __attribute__((always_inline)) {
      constexpr int ACT = decltype(act)::value;
      auto value = [&](int i, int j) __attribute__((always_inline)) {
        f32x4 z = acc[i][j];
        if (g.bias && n + 16 * j + 4 * gr < g.N) {
          const f32x4 b = *reinterpret_cast<const f32x4_any*>(g.bias + n + 16 * j + 4 * gr);
#pragma unroll
          for (int q = 0; q < 4; ++q) z[q] += b[q];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) z[q] = g.add * act_f32<ACT>(z[q]);
        return z;
      };
#pragma unroll
      for (int i = 0; i < kMxFI; ++i) {
        const int end = m + 16 * i < g.M ? g.N : 0;  // of the columns that this row stores
        if constexpr (kWide) {
          const int64_t o = (int64_t)(m + 16 * i) * g.ldo + n + 4 * gr, r = (int64_t)(m + 16 * i) * g.ldr + n + 4 * gr;
#pragma unroll
          for (int j = 0; j < kMxFJ; ++j) {
            f32x4 v = value(i, j);
            const bool here = n + 4 * gr + 16 * j < end;
            if (g.res && here) {
              const f32x4 w = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(res + r + 16 * j));
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] += g.keep * w[q];
            }
            if (here) __builtin_nontemporal_store(v, reinterpret_cast<f32x4_any*>(out + o + 16 * j));
            fence();
          }
        } else {
          const int c = n + 16 * (gr & 1) + 8 * (gr >> 1);
          const int64_t o = (int64_t)(m + 16 * i) * g.ldo + c, r = (int64_t)(m + 16 * i) * g.ldr + c;
#pragma unroll
          for (int j = 0; j < kMxFJ; j += 2) {
            f32x4 v = value(i, j), w = value(i, j + 1);
            const bool here = c + 16 * j < end;
            if (g.res) {
              u32x4 raw = {0u, 0u, 0u, 0u};
              if (here) raw = *reinterpret_cast<const u32x4_any*>(res + r + 16 * j);
              raw = swap_fragments(raw);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[q] += g.keep * OT::up((uint16_t)(raw[q / 2] >> (16 * (q % 2))));
                w[q] += g.keep * OT::up((uint16_t)(raw[2 + q / 2] >> (16 * (q % 2))));
              }
            }
            u32x4 h;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              h[q] = OT::down(v[2 * q]) | (uint32_t)OT::down(v[2 * q + 1]) << 16;
              h[2 + q] = OT::down(w[2 * q]) | (uint32_t)OT::down(w[2 * q + 1]) << 16;
            }
            h = swap_fragments(h);
            if (here) *reinterpret_cast<u32x4_any*>(out + o + 16 * j) = h;
            fence();
          }
        }
      }
    };
    // whole chunks of columns, eight to a lane: all but the last tiles of a row of results where N is no multiple
    if ((p.ni + 1) * kMxT <= g.N || g.N % 8 == 0) {
      by_act(g.act, results);
    } else {
      auto edge = [&](auto act) __attribute__((always_inline)) {
        constexpr int ACT = decltype(act)::value;
#pragma unroll
        for (int i = 0; i < kMxFI; ++i)
#pragma unroll
          for (int j = 0; j < kMxFJ; ++j) {
            const int mm = m + 16 * i, c = n + 16 * j + 4 * gr;
            if (mm < g.M && c < g.N) {
              const int64_t o = (int64_t)mm * g.ldo + c, r = (int64_t)mm * g.ldr + c;
              const int left = g.N - c;
              f32x4 z = acc[i][j], b = {0.f, 0.f, 0.f, 0.f}, w = b;
              if (left >= 4) {
                if (g.bias) b = *reinterpret_cast<const f32x4_any*>(g.bias + c);
                if (g.res) w = load_elem4(res, r, kOut);
              } else {
#pragma unroll
                for (int q = 0; q < 3; ++q) {
                  if (g.bias && q < left) b[q] = g.bias[c + q];
                  if (g.res && q < left) w[q] = load_elem(res, r + q, kOut);
                }
              }
#pragma unroll
              for (int q = 0; q < 4; ++q) z[q] = g.add * act_f32<ACT>(z[q] + b[q]);
              if (g.res) {
#pragma unroll
                for (int q = 0; q < 4; ++q) z[q] += g.keep * w[q];
              }
              if (left >= 4) {
                store_elem4(out, o, kOut, z);
              } else {
#pragma unroll
                for (int q = 0; q < 3; ++q)
                  if (q < left) store_elem(out, o + q, kOut, z[q]);
              }
            }
            fence();
          }
      };
      by_act(g.act, edge);
    }
#pragma unroll
    for (int i = 0; i < kMxFI; ++i)
#pragma unroll
      for (int j = 0; j < kMxFJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
}

}  // namespace
}  // namespace beam
