// The tiled products of 4-bit operands, and of 16-bit rows with 4-bit weights (gfx950).
#include "gemm_tiles.h"

namespace beam {
namespace {

// A byte a lane to LDS, to four bytes of its own.
__device__ __forceinline__ void lds_copy1(const void* g, uint32_t lds_base) {
  uint32_t saved;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %2\n\t"
      "global_load_lds_ubyte %1, off\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(g), "s"(lds_base)
      : "memory");
}

// 16-bit rows in tiles of R = 32 FI rows and 128 columns, half of the rows and 32 columns to a wave.  A stage is 128 of
// K, and LDS a ring of six, so that a short part of K is requested at once.  x: 256 bytes of a row, chunk c (8 elements)
// of row r at c ^ (r & 15), so that 16 rows of a fragment cover all banks once.  Codes and scales lie by column and
// block, as a lane wants them: 16 bytes and one of each 32.  The products' K runs over four blocks' first 8 elements,
// then their second 8, and so on, which is the same sum.
// Bound by what a CU gets from L2, some 38 bytes a nanosecond of x and codes.  Four waves of all rows instead of eight
// took 2 to 15% longer, codes loaded to registers a stage of 256 ahead 3 to 25%.
template <bool HALF, int FI>
__global__ __launch_bounds__(512) void code_rows_kernel(CodeArgs g, int mt, int nt, int total, int k_per_split,
                                                        float* __restrict__ part, int64_t ldpart) {
  constexpr int R = 32 * FI, kSlots = 6;
  constexpr int kX = R * 256, kCodes = 8192, kSlot = kX + kCodes + 2048, kPer = FI + 2;  // copies of a wave and stage
  static_assert(kSlots * kSlot <= 160 * 1024 && (kSlots - 2) * kPer < 64, "LDS, and copies that can be counted");
  __shared__ __align__(1024) uint8_t ring[kSlots * kSlot];
  typedef __attribute__((address_space(3))) uint8_t lds_u8;
  lds_u8* lds = (lds_u8*)ring;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, gr = lane >> 4;
  const int lin = xcd_lin(blockIdx.x, total), split = lin / (mt * nt), in = lin % (mt * nt);
  const int k0 = split * k_per_split, stages = (min(g.K, k0 + k_per_split) - k0 + 127) / 128;
  const int m0 = in % mt * R, wm = wave >> 2, wn = wave & 3, n0 = in / mt * 128 + wn * 32;

  const uint16_t* x[FI];  // four rows a copy
  int kx[FI];
#pragma unroll
  for (int q = 0; q < FI; ++q) {
    const int r = 4 * (wave * FI + q) + (lane >> 4);
    kx[q] = k0 + 8 * ((lane & 15) ^ (r & 15));
    x[q] = static_cast<const uint16_t*>(g.a) + (int64_t)min(m0 + r, g.M - 1) * g.lda;
  }
  // the wave copies the codes and scales of one of its two fragments, the other is the other half's
  const int64_t column = min(n0 + 16 * wm + l16, g.N - 1);
  const uint8_t *codes = static_cast<const uint8_t*>(g.b) + column * g.ldb, *scales = g.sb + column * g.ldsb;
  const uint32_t base = lds_addr(ring);
  int c_stage = 0;
  uint32_t c_slot = 0;
  auto copy = [&]() __attribute__((always_inline)) {
    if (c_stage >= stages) return;
#pragma unroll
    for (int q = 0; q < FI; ++q) {
      const int k = kx[q] + c_stage * 128;
      lds_copy16(k < g.K ? (const void*)(x[q] + k) : (const void*)&zero_chunk, base + c_slot + (wave * FI + q) * 1024);
    }
    const int b = min(k0 / 32 + 4 * c_stage + gr, g.blocks - 1);  // past the end the last, its scale not taken
    lds_copy16(codes + 16 * b, base + c_slot + kX + (wn * 2 + wm) * 1024);
    lds_copy1(scales + b, base + c_slot + kX + kCodes + (wn * 2 + wm) * 256);
    ++c_stage;
    c_slot = c_slot == (kSlots - 1) * kSlot ? 0 : c_slot + kSlot;
  };
  f32x4 acc[FI][2] = {};
#pragma unroll
  for (int i = 0; i < kSlots - 1; ++i) copy();
  uint32_t slot = 0;
#pragma unroll 1
  for (int t = 0; t < stages; ++t) {
    // this stage has to be there; those requested after it may be under way
    const int after = min(stages - 1 - t, kSlots - 2);
    if (after == 4) __builtin_amdgcn_s_waitcnt(waitcnt_vm(4 * kPer));
    else if (after == 3) __builtin_amdgcn_s_waitcnt(waitcnt_vm(3 * kPer));
    else if (after == 2) __builtin_amdgcn_s_waitcnt(waitcnt_vm(2 * kPer));
    else if (after == 1) __builtin_amdgcn_s_waitcnt(waitcnt_vm(kPer));
    else __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    copy();  // over the stage before this one, which every wave has read
    const lds_u8* at = lds + slot;
    const bool here = k0 / 32 + 4 * t + gr < g.blocks;
    u32x4 w[2];
    float ws[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[j] = *(const __attribute__((address_space(3))) u32x4*)(at + kX + (wn * 2 + j) * 1024 + lane * 16);
      const uint32_t e =
          *(const __attribute__((address_space(3))) uint32_t*)(at + kX + kCodes + (wn * 2 + j) * 256 + lane * 4);
      ws[j] = mx_scale(here ? e & 255u : 0u);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4 f[FI];
#pragma unroll
      for (int i = 0; i < FI; ++i)
        f[i] = *(const __attribute__((address_space(3))) u32x4*)(at + (16 * (wm * FI + i) + l16) * 256 +
                                                                  (((4 * gr + s) ^ l16) << 4));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u32x4 v = codes_to_16<HALF>(w[j][s], ws[j]);
#pragma unroll
        for (int i = 0; i < FI; ++i) acc[i][j] = mfma<HALF>(v, f[i], acc[i][j]);
      }
    }
    slot = slot == (kSlots - 1) * kSlot ? 0 : slot + kSlot;
  }
  auto store = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int m = m0 + 16 * (wm * FI + i) + l16, n = n0 + 16 * j + 4 * gr;
        if (m < g.M && n < g.N) f(m, n, acc[i][j]);
      }
  };
  if (part)
    store([&](int m, int n, f32x4 z) { *reinterpret_cast<f32x4*>(part + ((int64_t)split * g.M + m) * ldpart + n) = z; });
  else
    by_act(g.act, [&](auto act) {
      store([&](int m, int n, f32x4 z) { epilogue4<decltype(act)::value>(g, g.add, m, n, g.N, z); });
    });
}

}  // namespace

hipError_t launch_code_rows(const CodeArgs& g, const GemmSplit& s, int rows, hipStream_t st) {
  const int mt = (g.M + rows - 1) / rows, nt = (g.N + 127) / 128, total = mt * nt * s.splits;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(total), dim3(512), 0, st, g, mt, nt, total, s.k_per_split, s.part, s.ld);
    return hipGetLastError();
  };
  if (g.type == kElemF16) return go(rows == 32 ? code_rows_kernel<true, 1> : code_rows_kernel<true, 2>);
  return go(rows == 32 ? code_rows_kernel<false, 1> : code_rows_kernel<false, 2>);
}

hipError_t launch_mx_tiles(const MxArgs& g, const GemmSplit& s, int tile, bool half, hipStream_t st) {
  const int mt = (g.M + tile - 1) / tile, nt = (g.N + tile - 1) / tile, total = mt * nt * s.splits;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(total), dim3(256), 0, st, g, mt, nt, total, s.k_per_split, s.part, s.ld);
    return hipGetLastError();
  };
  auto of = [&](auto h) {
    constexpr bool kHalf = decltype(h)::value;
    if (tile == 128) return go(gemm_kernel<kHalf, false, false, 128, 128, 2, 2, true, false, MxArgs>);
    return go(gemm_kernel<kHalf, false, false, 64, 64, 2, 2, true, false, MxArgs>);
  };
  return half ? of(std::true_type{}) : of(std::false_type{});
}

hipError_t launch_code_tiles(const CodeArgs& g, const GemmSplit& s, int tile, hipStream_t st) {
  const int mt = (g.M + tile - 1) / tile, nt = (g.N + tile - 1) / tile, total = mt * nt * s.splits;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(total), dim3(256), 0, st, g, mt, nt, total, s.k_per_split, s.part, s.ld);
    return hipGetLastError();
  };
  auto of = [&](auto h) {
    constexpr bool kHalf = decltype(h)::value;
    if (tile == 128) return go(gemm_kernel<kHalf, false, false, 128, 128, 2, 2, true, true, CodeArgs>);
    return go(gemm_kernel<kHalf, false, false, 64, 64, 2, 2, true, true, CodeArgs>);
  };
  return g.type == kElemF16 ? of(std::true_type{}) : of(std::false_type{});
}

}  // namespace beam
