// Training side of the router (gfx950): the load-balance loss with the per-expert
// counts, and the gradient of the routing weights and of that loss with respect
// to the router's logits.
//
// Tokens are packed: sequence b holds rows [off[b], off[b+1]); rows outside every
// sequence are padding.  With n tokens in sequence b, s the sigmoid scores and
// p[t,e] = s[t,e] / sum_j s[t,j]:
//   count[b,e] = chosen slots of e,  P[b,e] = sum_t p[t,e] / n,
//   loss[b] = alpha sum_e E count[b,e] / (K n) P[b,e]
// (the per-sequence form of the balance loss; one sequence holding the whole
// batch gives the per-batch form).
//
// One wave per row of scores: lane i holds experts 4 i .. 4 i + 3 (V4) or i, i + 64, ...
#include "elem.h"

namespace beam {

constexpr int kBalMaxE = 256;
// Up to here one workgroup per sequence does everything, in one launch: on the GPU 4.0 us
// for 64 tokens against 7.1 in two launches, 7.7 against 7.8 for 250, 12.4 against 8.2 for
// 512, where the second launch still takes 4 us longer to issue.  (In a captured graph, which
// issues for nothing, two launches would be the faster from some 260 tokens on.)
constexpr int kBalSmallT = 512;
constexpr int kBalSmallThreads = 1024;
constexpr int kBalUnitThreads = 512;
constexpr int kBalFinishThreads = 1024;

// Offset i of the packed sequences; without offsets, one sequence of T rows.  Values
// outside [0, T] (the caller's error) are clamped, so no row outside the batch is touched.
struct Sequences {
  const int32_t* off;
  int B, T;
  __device__ __forceinline__ int at(int i) const { return off ? min(max(off[i], 0), T) : (i ? T : 0); }
};

// Number of i in [0, n) with pred(i), pred true on a prefix: 64 probes a round, so
// log64(n) dependent loads.  Every lane gets the result.
template <class P>
__device__ __forceinline__ int wave_prefix_count(int n, P pred) {
  const int lane = threadIdx.x & 63;
  int lo = 0;
  while (n > 0) {
    const int step = (n + 63) / 64;
    const int i = lane * step + step - 1;  // lane's probe: the last of its step
    const uint64_t hit = __ballot(i < n && pred(lo + i));
    const int c = __popcll(hit);
    lo += c * step;
    n = min(n - c * step, step - 1);
  }
  return lo;
}

template <bool V4>
__device__ __forceinline__ int expert_of(int lane, int i) {
  return V4 ? 4 * lane + i : lane + 64 * i;
}

// Four values of a row of E at this lane's experts, 0 past E.
template <bool V4>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int lane, float* v) {
  if constexpr (V4) {
    f32x4 r = {0.f, 0.f, 0.f, 0.f};
    if (4 * lane < E) r = *reinterpret_cast<const f32x4*>(row + 4 * lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = r[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lane + 64 * i < E ? row[lane + 64 * i] : 0.f;
  }
}

// Scores that sum to less than kTiny are taken kUp times as large (exactly, so their shares
// of the sum stay the same): the reciprocal of a sum near 2^-128 or below is infinite.
constexpr float kTiny = 0x1p-100f, kUp = 0x1p64f;

// Adds rows [r0, r1) of p and their slots' experts: sp[e] (this workgroup's sums,
// one plane per wave, added in wave order at the end) and the integer counts sc[e].
// Both are complete for every thread on return.
template <bool V4>
__device__ void sum_rows(const float* __restrict__ scores, const int32_t* __restrict__ ids, int r0, int r1, int E,
                         int K, float (*sp)[kBalMaxE], int* sc) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nw = blockDim.x >> 6;
  for (int e = tid; e < E; e += blockDim.x) sc[e] = 0;
  __syncthreads();
  for (int64_t i = (int64_t)r0 * K + tid; i < (int64_t)r1 * K; i += blockDim.x) {
    const int id = ids[i];
    if (id >= 0 && id < E) atomicAdd(&sc[id], 1);
  }
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  constexpr int U = 4;  // rows in flight per wave
  for (int r = r0 + wave; r < r1; r += nw * U) {
    float v[U][4], s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = r + u * nw;
      if (row < r1) {
        load_row<V4>(scores + (int64_t)row * E, E, lane, v[u]);
      } else {
        v[u][0] = v[u][1] = v[u][2] = v[u][3] = 0.f;
      }
      s[u] = (v[u][0] + v[u][1]) + (v[u][2] + v[u][3]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] = wave_sum(s[u]);
      if (s[u] < kTiny) {  // uniform, as the sum is
        s[u] *= kUp;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] *= kUp;
      }
      const float inv = s[u] == 0.f ? 0.f : 1.f / s[u];  // a row of zeros (or past the end) adds nothing
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += v[u][i] * inv;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (expert_of<V4>(lane, i) < E) sp[wave][expert_of<V4>(lane, i)] = acc[i];
  __syncthreads();
}

// loss, counts and P of one sequence from its sums (thread e < E holds expert e's).
__device__ void finish_sequence(int b, int n, int E, int K, float alpha, int count, double psum, double* buf,
                                float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ prob) {
  const int tid = threadIdx.x, nw = blockDim.x >> 6;
  double term = 0.0;
  if (tid < E) {
    const double P = n ? psum / n : 0.0;
    counts[(int64_t)b * E + tid] = count;
    prob[(int64_t)b * E + tid] = (float)P;
    term = n ? count * P : 0.0;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) term += __shfl_xor(term, off);
  if ((tid & 63) == 0) buf[tid >> 6] = term;
  __syncthreads();
  if (tid == 0) {
    double s = 0.0;
    for (int w = 0; w < min(nw, kBalMaxE / 64); ++w) s += buf[w];
    loss[b] = n ? (float)((double)alpha * E / ((double)K * n) * s) : 0.f;
  }
}

// Few tokens: grid B, one workgroup per sequence, one launch.
template <bool V4>
__global__ __launch_bounds__(kBalSmallThreads) void balance_small_kernel(
    const float* __restrict__ scores, const int32_t* __restrict__ ids, Sequences q, int E, int K, float alpha,
    float* __restrict__ loss, int32_t* __restrict__ counts, float* __restrict__ prob) {
  __shared__ float sp[kBalSmallThreads / 64][kBalMaxE];
  __shared__ int sc[kBalMaxE];
  __shared__ double buf[kBalSmallThreads / 64];
  const int b = blockIdx.x, tid = threadIdx.x, nw = blockDim.x >> 6;
  const int r0 = q.at(b), r1 = max(r0, q.at(b + 1));
  sum_rows<V4>(scores, ids, r0, r1, E, K, sp, sc);
  double psum = 0.0;
  if (tid < E)
    for (int w = 0; w < nw; ++w) psum += sp[w][tid];
  finish_sequence(b, r1 - r0, E, K, alpha, tid < E ? sc[tid] : 0, psum, buf, loss, counts, prob);
}

// Many tokens: units of at most R rows of one sequence.  Sequence b's units are
// first(b) .. first(b) + off[b+1] / R - off[b] / R with first(b) = off[b] / R + b:
// one for each stretch [c R, (c+1) R) that its rows meet, and never more than
// T / R + B in all, so a unit finds its rows from the offsets alone.
struct Units {
  Sequences q;
  int R;
  __device__ __forceinline__ int first(int b) const { return q.at(b) / R + b; }
};

template <bool V4>
__global__ __launch_bounds__(kBalUnitThreads) void balance_unit_kernel(const float* __restrict__ scores,
                                                                       const int32_t* __restrict__ ids, Units un,
                                                                       int E, int K, int32_t* __restrict__ part_count,
                                                                       float* __restrict__ part_sum) {
  __shared__ float sp[kBalUnitThreads / 64][kBalMaxE];
  __shared__ int sc[kBalMaxE];
  const int u = blockIdx.x;
  const int b = wave_prefix_count(un.q.B, [&](int i) { return un.first(i) <= u; }) - 1;
  if (b < 0) return;  // uniform over the workgroup: every wave finds the same b
  const int lo = un.q.at(b), hi = un.q.at(b + 1);
  const int c = u - un.first(b) + lo / un.R;
  if (c > hi / un.R) return;  // past the last sequence's units
  const int r0 = max(lo, c * un.R), r1 = max(r0, min(hi, (c + 1) * un.R));
  sum_rows<V4>(scores, ids, r0, r1, E, K, sp, sc);
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kBalUnitThreads / 64; ++w) s += sp[w][e];
    part_count[(int64_t)u * E + e] = sc[e];
    part_sum[(int64_t)u * E + e] = s;
  }
}

// grid B: adds a sequence's units, four threads to an expert, each in unit order.
__global__ __launch_bounds__(kBalFinishThreads) void balance_finish_kernel(Units un, int max_units, int E, int K,
                                                                           float alpha,
                                                                           const int32_t* __restrict__ part_count,
                                                                           const float* __restrict__ part_sum,
                                                                           float* __restrict__ loss,
                                                                           int32_t* __restrict__ counts,
                                                                           float* __restrict__ prob) {
  __shared__ double sp[4][kBalMaxE];
  __shared__ int sc[4][kBalMaxE];
  __shared__ double buf[kBalFinishThreads / 64];
  const int b = blockIdx.x, tid = threadIdx.x, e = tid & (kBalMaxE - 1), g = tid / kBalMaxE;
  const int lo = un.q.at(b), hi = un.q.at(b + 1);
  const int first = un.first(b), last = min(first + hi / un.R - lo / un.R, max_units - 1);
  double s = 0.0;
  int c = 0;
  if (e < E) {
#pragma unroll 4
    for (int u = first + g; u <= last; u += 4) {
      s += part_sum[(int64_t)u * E + e];
      c += part_count[(int64_t)u * E + e];
    }
    sp[g][e] = s;
    sc[g][e] = c;
  }
  __syncthreads();
  if (tid < E) {
    s = ((sp[0][tid] + sp[1][tid]) + sp[2][tid]) + sp[3][tid];
    c = sc[0][tid] + sc[1][tid] + sc[2][tid] + sc[3][tid];
  }
  finish_sequence(b, max(0, hi - lo), E, K, alpha, c, s, buf, loss, counts, prob);
}

// ---------------------------------------------------------------------------
// gradient with respect to the logits
// ---------------------------------------------------------------------------
// dlogit = ds s (1 - s); ds s is the sum of two parts, in shares p = s / S of a sum:
//   routing weights w_k = scale p_k over the K chosen experts, S = sum_k s_k:
//     scale p_k (dw_k - sum_j dw_j p_j)
//   balance loss, g_e = dloss[b] alpha E count[b,e] / (K n^2), S = sum_e s_e:
//     p_e (g_e - sum_j g_j p_j)
// A constant added to every g_e changes nothing, so g is taken from the exact integers
// E count - K n: with near-even counts the difference would lose most of its digits.
// One wave per token; a slot whose id lies outside [0, E) is skipped.  Bound by vector
// instructions next to the memory (16 waves to a SIMD at 16384 tokens): what the slots
// need of the row goes through the wave's own LDS row instead of compares over all
// experts (13.0 -> 11.4 us), and up to 64 sequences a token's is found in one load
// (11.7 -> 11.3 us with 37).  Everything that
// does not hang on another load is requested at the start.
constexpr int kGradWaves = 4;

template <bool V4>
__global__ __launch_bounds__(64 * kGradWaves) void route_backward_kernel(
    const float* __restrict__ scores, const int32_t* __restrict__ ids, const float* __restrict__ dw, float scale,
    Sequences q, float alpha, const float* __restrict__ dloss, const int32_t* __restrict__ counts,
    float* __restrict__ dlogits, int E, int K) {
  // experts of lane l at 4 l .. 4 l + 3 with V4, else at place(e) = 4 (e % 64) + e / 64
  __shared__ f32x4 rows[kGradWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = __builtin_amdgcn_readfirstlane(blockIdx.x * kGradWaves + wave);
  if (t >= q.T) return;  // no barrier follows
  float s[4], ds[4] = {0.f, 0.f, 0.f, 0.f};
  load_row<V4>(scores + (int64_t)t * E, E, lane, s);
  int id = -1;
  float d = 0.f;
  if (dw && lane < K) {
    id = ids[(int64_t)t * K + lane];
    d = dw[(int64_t)t * K + lane];
  }
  if (dloss) {
    int b, lo, hi;
    if (!q.off) {
      b = lo = 0;
      hi = q.T;
    } else if (q.B <= 64) {
      const int first = q.at(0);
      const int end = q.at(lane < q.B ? lane + 1 : q.B);
      b = __popcll(__ballot(lane < q.B && end <= t));
      lo = b ? __builtin_amdgcn_readlane(end, b - 1) : first;
      hi = __builtin_amdgcn_readlane(end, min(b, 63));
    } else {
      b = wave_prefix_count(q.B, [&](int i) { return q.at(i + 1) <= t; });
      lo = q.at(min(b, q.B - 1));
      hi = q.at(min(b, q.B - 1) + 1);
    }
    const int n = hi - lo;
    if (b < q.B && n > 0 && t >= lo) {  // else padding
      const int32_t* cb = counts + (int64_t)b * E;
      int cnt[4];
      if constexpr (V4) {
        int4 c4 = {0, 0, 0, 0};
        if (4 * lane < E) c4 = *reinterpret_cast<const int4*>(cb + 4 * lane);
        cnt[0] = c4.x;
        cnt[1] = c4.y;
        cnt[2] = c4.z;
        cnt[3] = c4.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) cnt[i] = lane + 64 * i < E ? cb[lane + 64 * i] : 0;
      }
      const float c = dloss[b] * alpha / ((float)K * n * n);
      float g[4];
      // E count - K n, exact: in 24-bit products while K n (>= count) fits one, else in FP64.
      // Past E the score is 0 and the result is not stored.
      if ((int64_t)K * n < (1 << 23)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = (float)(__mul24(cnt[i], E) - K * n);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = (float)((double)cnt[i] * E - (double)K * n);
      }
      float tot = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tot += s[i];
        dot += g[i] * s[i];
      }
      tot = wave_sum(tot);
      dot = wave_sum(dot);
      if (tot < kTiny) {  // uniform; 1 - s is 1 for these either way
        tot *= kUp;
        dot = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[i] *= kUp;
          dot += g[i] * s[i];
        }
        dot = wave_sum(dot);
      }
      const float inv = tot == 0.f ? 0.f : 1.f / tot;
      const float m = dot * inv, ci = c * inv;
#pragma unroll
      for (int i = 0; i < 4; ++i) ds[i] = ci * s[i] * (g[i] - m);
    }
  }
  if (dw) {
    float* row = reinterpret_cast<float*>(rows[wave]);
    auto in_order = [] {  // LDS operations of one wave execute in order; this keeps the compiler to it
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };
    const bool ok = id >= 0 && id < E;
    const int place = V4 ? id : 4 * (id & 63) + (id >> 6);
    rows[wave][lane] = f32x4{s[0], s[1], s[2], s[3]};
    in_order();
    float sk = ok ? row[place] : 0.f;
    in_order();
    rows[wave][lane] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (!ok) d = 0.f;
    // K <= 16: the slots all lie in the first 16 lanes
    auto slot_sum = [](float v) {
      return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(row16_sum(v)), 0));
    };
    float tot = slot_sum(sk), dot = slot_sum(d * sk);
    if (tot < kTiny) {  // uniform
      tot *= kUp;
      sk *= kUp;
      dot = slot_sum(d * sk);
    }
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
    const float a = scale * inv * sk * (d - dot * inv);
    // slots of one expert: each holds the sum over all of them, in slot order
    float all = 0.f;
    for (int k = 0; k < K; ++k) {
      const int ik = __builtin_amdgcn_readlane(id, k);
      const float ak = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(a), k));
      all += id == ik ? ak : 0.f;
    }
    in_order();
    if (ok) row[place] = all;
    in_order();
    const f32x4 add = rows[wave][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) ds[i] += add[i];
  }
  float* out = dlogits + (int64_t)t * E;
  float o[4];
  // an expert without any gradient has 0 whatever its score holds (padding may hold anything)
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = ds[i] == 0.f ? 0.f : ds[i] * (1.f - s[i]);
  if constexpr (V4) {
    if (4 * lane < E) *reinterpret_cast<f32x4*>(out + 4 * lane) = f32x4{o[0], o[1], o[2], o[3]};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (lane + 64 * i < E) out[lane + 64 * i] = o[i];
  }
}

// Rows of four experts to a lane (16-byte loads) where every row starts on 16 bytes: at
// 16384 tokens of 256 experts 11.4 us for the loss and 11.3 for the gradient, 11.8 and 11.8
// with four 4-byte loads; the same within 0.3 us at 64 and 128 experts.
static bool balance_v4(int E) { return E % 4 == 0; }

// Rows per unit, and the units' number; 0 units: the one-launch path.
static int balance_rows(int T) {
  int R = 64;
  while (T / R > 512) R *= 2;
  return R;
}
int balance_units(int T, int B) { return T <= kBalSmallT ? 0 : T / balance_rows(T) + B; }

hipError_t launch_balance(const float* scores, const int32_t* ids, int B, const int32_t* off, int T, int E, int K,
                          float alpha, float* loss, int32_t* counts, float* prob, int32_t* part_count, float* part_sum,
                          hipStream_t st) {
  const Sequences q{off, B, T};
  const int units = balance_units(T, B);
  const bool v4 = balance_v4(E);
  if (units == 0) {
    // one wave per row for the smallest batches, down to the waves that finish_sequence needs
    const int waves = T >= 16 ? 16 : T > 4 ? T : 4;
    hipLaunchKernelGGL(v4 ? balance_small_kernel<true> : balance_small_kernel<false>, dim3(B), dim3(64 * waves), 0,
                       st, scores, ids, q, E, K, alpha, loss, counts, prob);
    return hipGetLastError();
  }
  const Units un{q, balance_rows(T)};
  hipLaunchKernelGGL(v4 ? balance_unit_kernel<true> : balance_unit_kernel<false>, dim3(units), dim3(kBalUnitThreads),
                     0, st, scores, ids, un, E, K, part_count, part_sum);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(balance_finish_kernel, dim3(B), dim3(kBalFinishThreads), 0, st, un, units, E, K, alpha,
                     part_count, part_sum, loss, counts, prob);
  return hipGetLastError();
}

hipError_t launch_route_backward(const float* scores, const int32_t* ids, const float* dw, float scale, int B,
                                 const int32_t* off, float alpha, const float* dloss, const int32_t* counts,
                                 float* dlogits, int T, int E, int K, hipStream_t st) {
  const Sequences q{off, B, T};
  hipLaunchKernelGGL(balance_v4(E) ? route_backward_kernel<true> : route_backward_kernel<false>,
                     dim3((T + kGradWaves - 1) / kGradWaves), dim3(64 * kGradWaves), 0, st, scores, ids, dw, scale, q,
                     alpha, dloss, counts, dlogits, E, K);
  return hipGetLastError();
}

}  // namespace beam
