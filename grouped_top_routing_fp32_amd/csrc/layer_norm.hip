// Layer norm and its backward pass (gfx950).
//
//   y  = (x - mean) rstd gamma + beta,  mean = sum x / H,  rstd = 1 / sqrt(sum (x - mean)^2 / H + eps)
//   with xh = (x - mean) rstd and g = dy gamma:
//   dx = rstd (g - sum g / H - xh sum(g xh) / H),  dgamma = sum_t dy xh,  dbeta = sum_t dy
//
// Both are bound by HBM: a row is read once and kept in registers between its
// sums and its result.  A row belongs to a team of `team` threads (whole waves;
// one wave per row up to 512 columns, several such rows in a workgroup); thread
// i of it holds chunks i, i + team, ... of 8 consecutive columns, moved 16 bytes at
// a time wherever the row starts.  TAIL: H is no multiple of 8, so a row's last chunk
// holds fewer columns.
#include <type_traits>

#include "elem.h"

namespace beam {

constexpr int kLnMaxThreads = 1024;
constexpr int kLnMaxWaves = kLnMaxThreads / 64;
// Up to here the backward pass is one launch: with 1021 rows of 2561 columns in bf16 10.6 us
// on the GPU, 12.8 in two launches, with 1024 rows of 512 5.8 and 9.2, with 256 rows of 5120
// 6.3 and 12.0, with 512 rows of 16384 in fp32 31.5 and 35.5, with 1500 rows of 5120 in fp32
// 22.8 and 20.9; the second launch takes the host 4 us besides.  With 1024 rows of 8192 columns
// and more, read twice, it is within 12% either way (16384 in fp32 68.6 and 61.1, in bf16 31.5
// and 33.0).
constexpr int kLnFewRows = 1024;
constexpr int kLnFewCols = 32;  // of a workgroup that adds columns
constexpr int kLnMaxJoin = 4096;  // columns of rows that share a workgroup with others
static_assert(kLnMaxWaves == 16, "16 lanes join the waves' sums");

// Columns in chunk ch of a row: a constant where every chunk is whole.
template <bool TAIL>
__device__ __forceinline__ int chunk_cols(int H, int ch) {
  return TAIL ? min(8, H - 8 * ch) : 8;
}

// Forward.  Statistics: each wave takes the mean m of its own columns, then the sum of
// squares about it (two passes over registers) and the rest c of its mean that m's
// rounding left.  The waves are joined about the first one's m, P: wave w's mean is
// P + d_w, d_w = (m_w - P) + c_w, the row's P + D, D = sum n_w d_w / H, and the squares
// add up to sum M2_w + n_w (d_w - D)^2.  One barrier; a mean far from zero cancels
// nothing, since only P holds its size, and y is taken from (x - P) - D.
template <class XT, class YT, int NCH, bool TAIL>
__global__ __launch_bounds__(kLnMaxThreads) void layer_norm_kernel(
    const typename XT::S* __restrict__ x, int64_t ldx, const float* __restrict__ gamma,
    const float* __restrict__ beta, typename YT::S* __restrict__ y, int64_t ldy, float* __restrict__ mean_out,
    float* __restrict__ rstd_out, int T, int H, float eps) {
  __shared__ f32x4 parts[kLnMaxWaves];
  const int tid = threadIdx.x, team = blockDim.x, wave = tid >> 6, nw = team >> 6;
  const int t = blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= T) return;  // blockDim.y > 1 only for one-wave teams, which meet no barrier
  const int nch = (H + 7) / 8;
  const typename XT::S* xr = x + (int64_t)t * ldx;
  float v[NCH][8];
  float s = 0.f;
  int cols = 0;  // the wave's
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = tid + c * team, w0 = 8 * (c * team + 64 * wave);
    cols += min(H, w0 + 512) - min(H, w0);
    if (ch < nch) {
      load8<XT>(xr + 8 * ch, chunk_cols<TAIL>(H, ch), v[c]);
#pragma unroll
      for (int q = 0; q < 8; ++q) s += v[c][q];
    }
  }
  float P = cols ? wave_sum(s) / cols : 0.f;
  float r = 0.f, m2 = 0.f;
#pragma unroll
  for (int c = 0; c < NCH; ++c)
    if (tid + c * team < nch) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float d = !TAIL || q < chunk_cols<TAIL>(H, tid + c * team) ? v[c][q] - P : 0.f;
        r += d;
        m2 += d * d;
      }
    }
  r = wave_sum(r);
  float D = cols ? r / cols : 0.f;
  m2 = wave_sum(m2) - r * D;
  if (nw > 1) {
    if ((tid & 63) == 0) parts[wave] = f32x4{P, D, m2, (float)cols};
    __syncthreads();
    // every 16 lanes join the waves' parts among themselves
    const int w = tid & 15;
    const f32x4 mine = w < nw ? parts[w] : f32x4{0.f, 0.f, 0.f, 0.f};
    P = parts[0][0];
    const float d = mine[3] > 0.f ? (mine[0] - P) + mine[1] : 0.f;
    D = row16_sum(mine[3] * d) / H;
    m2 = row16_sum(mine[2] + mine[3] * (d - D) * (d - D));
  }
  const float rs = 1.f / sqrtf(m2 / H + eps);
  if (tid == 0) {
    if (mean_out) mean_out[t] = P + D;
    if (rstd_out) rstd_out[t] = rs;
  }
  typename YT::S* yr = y + (int64_t)t * ldy;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = tid + c * team;
    if (ch < nch) {
      const int n = chunk_cols<TAIL>(H, ch);
      float g[8], b[8], o[8];
      if (gamma) load8<F32>(gamma + 8 * ch, n, g);
      if (beta) load8<F32>(beta + 8 * ch, n, b);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        o[q] = ((v[c][q] - P) - D) * rs;
        if (gamma) o[q] *= g[q];
        if (beta) o[q] += b[q];
      }
      store8<YT>(yr + 8 * ch, n, o);
    }
  }
}

// Backward.  A workgroup of blockDim.y teams takes rows block * blockDim.y + team,
// then those blocks * blockDim.y further on; a thread's columns stay the same from
// row to row, so it sums their dgamma and dbeta in registers.  At the end the teams add
// up in LDS, in order, and the workgroup writes one row of part [2][blocks][H], which
// column_sums_kernel adds up: no atomics, so the sums' order is fixed.  Above 8192 columns, two
// chunks a thread, FP32 dy spills up to 7 registers.
template <class DT, class XT, int NCH, bool TAIL, bool SUMS>
__device__ __forceinline__ void backward_rows(
    const typename DT::S* __restrict__ dy, int64_t lddy, const typename XT::S* __restrict__ x, int64_t ldx,
    const float* __restrict__ mean, const float* __restrict__ rstd, const float* __restrict__ gamma,
    typename XT::S* __restrict__ dx, int64_t lddx, float* __restrict__ part, int T, int H, int block, int blocks) {
  __shared__ float red[2][kLnMaxWaves][2];
  __shared__ __align__(16) float joined[2][kLnMaxJoin];
  const int tid = threadIdx.x, team = blockDim.x, nw = team >> 6;
  const int wave0 = threadIdx.y * nw, wave = wave0 + (tid >> 6);
  const int teams = blockDim.y, stride = blocks * teams;
  const int nch = (H + 7) / 8;
  // few columns to a thread: gamma stays in registers, and rows are requested one ahead
  constexpr bool kAhead = NCH == 1;
  float g[NCH][8], dg[NCH][8] = {}, db[NCH][8] = {};
  auto load_gamma = [&](int c) __attribute__((always_inline)) {
    const int ch = tid + c * team;
#pragma unroll
    for (int q = 0; q < 8; ++q) g[c][q] = 1.f;
    if (gamma && ch < nch) load8<F32>(gamma + 8 * ch, chunk_cols<TAIL>(H, ch), g[c]);
  };
  if (kAhead) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) load_gamma(c);
  }
  Raw8<XT> xr[NCH];
  Raw8<DT> yr[NCH];
  float mu = 0.f, rs = 0.f;
  auto request = [&](int t) __attribute__((always_inline)) {
    if (t >= T) return;
    mu = mean[t];
    rs = rstd[t];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int ch = tid + c * team;
      if (ch < nch) {
        const typename XT::S* xp = x + (int64_t)t * ldx + 8 * ch;
        const typename DT::S* yp = dy + (int64_t)t * lddy + 8 * ch;
        const int n = chunk_cols<TAIL>(H, ch);
        if (!TAIL || n == 8) {
          xr[c].load(xp);
          yr[c].load(yp);
        } else {  // dy is 0 past the row's end, which leaves the sums alone
          xr[c].load_part(xp, n);
          yr[c].load_part(yp, n);
        }
      }
    }
  };
  if (kAhead) request(block * teams + threadIdx.y);
  int buf = 0;
  // every team makes the same number of rounds; one past the end has no row in the last
  for (int t0 = block * teams; t0 < T; t0 += stride, buf ^= 1) {
    const int t = t0 + threadIdx.y;
    const bool live = t < T;
    float xh[NCH][8], gy[NCH][8];
    float s1 = 0.f, s2 = 0.f;
    if (!kAhead) request(t);
    const float r = rs;
    if (live) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        if (!kAhead) load_gamma(c);
        if (tid + c * team < nch) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            xh[c][q] = (xr[c][q] - mu) * r;
            gy[c][q] = yr[c][q];
            if constexpr (SUMS) {
              dg[c][q] += gy[c][q] * xh[c][q];
              db[c][q] += gy[c][q];
            }
            gy[c][q] *= g[c][q];
            s1 += gy[c][q];
            s2 += gy[c][q] * xh[c][q];
          }
        }
      }
    }
    if (kAhead) request(t + stride);  // the next row comes in while this one is reduced and written
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if (nw > 1) {  // two buffers: the next row's sums do not wait for this row's readers
      if ((tid & 63) == 0) {
        red[buf][wave][0] = s1;
        red[buf][wave][1] = s2;
      }
      __syncthreads();
      const int w = tid & 15;  // every 16 lanes add the waves' sums among themselves
      s1 = row16_sum(w < nw ? red[buf][wave0 + w][0] : 0.f);
      s2 = row16_sum(w < nw ? red[buf][wave0 + w][1] : 0.f);
    }
    if (dx && live) {
      const float c1 = s1 / H, c2 = s2 / H;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int ch = tid + c * team;
        if (ch < nch) {
          float o[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) o[q] = r * (gy[c][q] - c1 - xh[c][q] * c2);
          store8<XT>(dx + (int64_t)t * lddx + 8 * ch, chunk_cols<TAIL>(H, ch), o);
        }
      }
    }
  }
  if constexpr (!SUMS) return;
  float* pg = part + (int64_t)block * H;
  float* pb = part + ((int64_t)blocks + block) * H;
  for (int y = 0; y < teams; ++y) {
    if ((int)threadIdx.y == y) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int ch = tid + c * team;
        if (ch < nch) {
          if (y > 0) {  // teams > 1: H <= kLnMaxJoin, a multiple of 8
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              dg[c][q] += joined[0][8 * ch + q];
              db[c][q] += joined[1][8 * ch + q];
            }
          }
          if (y + 1 < teams) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              joined[0][8 * ch + q] = dg[c][q];
              joined[1][8 * ch + q] = db[c][q];
            }
          } else {
            store8<F32>(pg + 8 * ch, chunk_cols<TAIL>(H, ch), dg[c]);
            store8<F32>(pb + 8 * ch, chunk_cols<TAIL>(H, ch), db[c]);
          }
        }
      }
    }
    if (y + 1 < teams) __syncthreads();
  }
}

template <class DT, class XT, int NCH, bool TAIL>
__global__ __launch_bounds__(kLnMaxThreads) void layer_norm_backward_kernel(
    const typename DT::S* __restrict__ dy, int64_t lddy, const typename XT::S* __restrict__ x, int64_t ldx,
    const float* __restrict__ mean, const float* __restrict__ rstd, const float* __restrict__ gamma,
    typename XT::S* __restrict__ dx, int64_t lddx, float* __restrict__ part, int T, int H) {
  backward_rows<DT, XT, NCH, TAIL, true>(dy, lddy, x, ldx, mean, rstd, gamma, dx, lddx, part, T, H, blockIdx.x,
                                         gridDim.x);
}

// Few rows: one launch without partial sums.  Workgroups [0, cgroups) own 32 columns each and
// add all rows of them (xh needs the row's mean and rstd alone, so nothing waits for dx): thread
// (c, g) takes chunk c of four in rows g, g + threads / 4, ...; a wave's 16 rows are joined by
// shuffles, the waves in order, in FP64.  The others take dx's rows, of which x and dy come a
// second time, from the caches.  Bound by what one CU takes from beyond its L2: 1021 rows of
// 2561 fp32 12.5 us, with 64 columns a workgroup 15.0, with 16, which share lines, 13.9.
template <class DT, class XT, int NCH, bool TAIL>
__global__ __launch_bounds__(kLnMaxThreads) void layer_norm_backward_few_kernel(
    const typename DT::S* __restrict__ dy, int64_t lddy, const typename XT::S* __restrict__ x, int64_t ldx,
    const float* __restrict__ mean, const float* __restrict__ rstd, const float* __restrict__ gamma,
    typename XT::S* __restrict__ dx, int64_t lddx, float* __restrict__ dgamma, float* __restrict__ dbeta, int T, int H,
    int cgroups) {
  if ((int)blockIdx.x >= cgroups)
    return backward_rows<DT, XT, NCH, TAIL, false>(dy, lddy, x, ldx, mean, rstd, gamma, dx, lddx, nullptr, T, H,
                                                   blockIdx.x - cgroups, gridDim.x - cgroups);
  constexpr int kChunks = kLnFewCols / 8;
  __shared__ float sums[kLnMaxWaves][2][kLnFewCols];
  const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
  const int full = cgroups & ~7, b = blockIdx.x;  // neighbours share lines: on one XCD
  const int h0 = kLnFewCols * (b >= full ? b : (b & 7) * (full >> 3) + (b >> 3));
  const int h = h0 + 8 * (tid % kChunks), n = min(8, H - h);  // n <= 0: none
  float dg[8] = {}, db[8] = {};
  if (n > 0) {
#pragma unroll 4
    for (int t = tid / kChunks; t < T; t += threads / kChunks) {
      float xv[8], yv[8];
      load8<XT>(x + (int64_t)t * ldx + h, chunk_cols<TAIL>(H, h / 8), xv);
      load8<DT>(dy + (int64_t)t * lddy + h, chunk_cols<TAIL>(H, h / 8), yv);
      const float mu = mean[t], r = rstd[t];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        dg[q] += yv[q] * ((xv[q] - mu) * r);
        db[q] += yv[q];
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 8; ++q)
#pragma unroll
    for (int off = kChunks; off < 64; off *= 2) {
      dg[q] += __shfl_xor(dg[q], off);
      db[q] += __shfl_xor(db[q], off);
    }
  if ((tid & 63) < kChunks) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      sums[tid >> 6][0][8 * (tid % kChunks) + q] = dg[q];
      sums[tid >> 6][1][8 * (tid % kChunks) + q] = db[q];
    }
  }
  __syncthreads();
  const int c = tid % kLnFewCols;
  float* out = tid / kLnFewCols ? dbeta : dgamma;
  if (tid < 2 * kLnFewCols && h0 + c < H && out) {
    double a = 0.0;
    for (int w = 0; w < threads >> 6; ++w) a += sums[w][tid / kLnFewCols][c];
    out[h0 + c] = (float)a;
  }
}

// out0[h] = sum_u part[0][u][h], out1[h] = sum_u part[1][u][h] (either may be null).
// grid (ceil(H / 64), 2), block (64, 16): thread (c, g) adds rows g, g + 16, ...;
// the 16 sums of a column are added in order, in FP64.
__global__ __launch_bounds__(1024) void column_sums_kernel(const float* __restrict__ part, float* __restrict__ out0,
                                                           float* __restrict__ out1, int units, int H) {
  __shared__ float s[16][64];
  float* out = blockIdx.y ? out1 : out0;
  if (!out) return;
  const float* p = part + (int64_t)blockIdx.y * units * H;
  const int h = blockIdx.x * 64 + threadIdx.x;
  float v = 0.f;
  if (h < H)
#pragma unroll 8
    for (int u = threadIdx.y; u < units; u += 16) v += p[(int64_t)u * H + h];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && h < H) {
    double a = 0.0;
#pragma unroll
    for (int g = 0; g < 16; ++g) a += s[g][threadIdx.x];
    out[h] = (float)a;
  }
}

hipError_t launch_column_sums(const float* part, float* out0, float* out1, int units, int H, hipStream_t st) {
  hipLaunchKernelGGL(column_sums_kernel, dim3((H + 63) / 64, out1 ? 2 : 1), dim3(64, 16), 0, st, part, out0, out1,
                     units, H);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// launch shapes
// ---------------------------------------------------------------------------
int layer_norm_max_cols() { return 16384; }

namespace {

struct Shape {
  int nch;   // chunks per thread
  int team;  // threads per row
  int rows;  // rows per workgroup of the forward kernel (one-wave teams only)
};

Shape shape(int H) {
  const int chunks = (H + 7) / 8;
  Shape s;
  s.nch = chunks <= 1024 ? 1 : 2;
  s.team = ((chunks + s.nch - 1) / s.nch + 63) / 64 * 64;
  s.rows = s.team == 64 ? 4 : 1;
  return s;
}

template <class F>
hipError_t by_type(int type, F f) {
  return type == kElemBF16 ? f(BF16{}) : type == kElemF16 ? f(F16{}) : f(F32{});
}

template <class F>
hipError_t by_chunks(int H, int nch, F f) {
  using std::integral_constant;
  using std::bool_constant;
  if (H % 8 == 0)
    return nch == 1 ? f(integral_constant<int, 1>{}, bool_constant<false>{})
                    : f(integral_constant<int, 2>{}, bool_constant<false>{});
  return nch == 1 ? f(integral_constant<int, 1>{}, bool_constant<true>{})
                  : f(integral_constant<int, 2>{}, bool_constant<true>{});
}

}  // namespace

hipError_t launch_layer_norm(const void* x, int x_type, int64_t ldx, const float* gamma, const float* beta, void* y,
                             int y_type, int64_t ldy, float* mean, float* rstd, int T, int H, float eps,
                             hipStream_t st) {
  const Shape s = shape(H);
  return by_type(x_type, [&](auto xt) {
    return by_type(y_type, [&](auto yt) {
      return by_chunks(H, s.nch, [&](auto n, auto tail) {
        using XT = decltype(xt);
        using YT = decltype(yt);
        hipLaunchKernelGGL((layer_norm_kernel<XT, YT, decltype(n)::value, decltype(tail)::value>),
                           dim3((T + s.rows - 1) / s.rows), dim3(s.team, s.rows), 0, st,
                           static_cast<const typename XT::S*>(x), ldx, gamma, beta, static_cast<typename YT::S*>(y),
                           ldy, mean, rstd, T, H, eps);
        return hipGetLastError();
      });
    });
  });
}

// Teams of a backward workgroup, and workgroups (rows of partial column sums): as many
// teams as 1024 threads hold, one workgroup to a CU.  More of either costs more in
// partial sums than it gains: [8192, 5120] fp32 / bf16 80 us with 256 workgroups, 84
// with 192, 86 with 512.
static int backward_teams(int H) { return H <= kLnMaxJoin ? kLnMaxThreads / shape(H).team : 1; }
static int backward_groups(int T, int teams) {
  const int n = (T + teams - 1) / teams;
  return n < 256 ? n : 256;
}

// The most rows of partial sums of a call.
int layer_norm_backward_units(int T) { return T <= kLnFewRows ? 0 : 256; }

hipError_t launch_layer_norm_backward(const void* dy, int dy_type, int64_t lddy, const void* x, int x_type,
                                      int64_t ldx, const float* mean, const float* rstd, const float* gamma, void* dx,
                                      int64_t lddx, float* dgamma, float* dbeta, float* part, int T, int H,
                                      hipStream_t st) {
  const Shape s = shape(H);
  const int teams = backward_teams(H), units = backward_groups(T, teams);
  const bool sums = dgamma || dbeta;
  if (!sums || T <= kLnFewRows) {
    const int cgroups = sums ? (H + kLnFewCols - 1) / kLnFewCols : 0, rgroups = dx ? (T + teams - 1) / teams : 0;
    return by_type(dy_type, [&](auto dt) {
      return by_type(x_type, [&](auto xt) {
        return by_chunks(H, s.nch, [&](auto n, auto tail) {
          using DT = decltype(dt);
          using XT = decltype(xt);
          hipLaunchKernelGGL((layer_norm_backward_few_kernel<DT, XT, decltype(n)::value, decltype(tail)::value>),
                             dim3(cgroups + rgroups), dim3(s.team, teams), 0, st,
                             static_cast<const typename DT::S*>(dy), lddy, static_cast<const typename XT::S*>(x), ldx,
                             mean, rstd, gamma, static_cast<typename XT::S*>(dx), lddx, dgamma, dbeta, T, H, cgroups);
          return hipGetLastError();
        });
      });
    });
  }
  hipError_t e = by_type(dy_type, [&](auto dt) {
    return by_type(x_type, [&](auto xt) {
      return by_chunks(H, s.nch, [&](auto n, auto tail) {
        using DT = decltype(dt);
        using XT = decltype(xt);
        hipLaunchKernelGGL((layer_norm_backward_kernel<DT, XT, decltype(n)::value, decltype(tail)::value>),
                           dim3(units), dim3(s.team, teams), 0, st, static_cast<const typename DT::S*>(dy), lddy,
                           static_cast<const typename XT::S*>(x), ldx, mean, rstd, gamma,
                           static_cast<typename XT::S*>(dx), lddx, part, T, H);
        return hipGetLastError();
      });
    });
  });
  if (e != hipSuccess) return e;
  return launch_column_sums(part, dgamma, dbeta, units, H, st);
}

}  // namespace beam
