// The norm of all gradients of a step and their clipping (gfx950).
//
//   norm = |scale| sqrt(sum over all tensors of g^2),  out = g scale min(1, max_norm / (norm + eps))
//
// Bound by HBM: every gradient is read for the norm and again for its scaling (600 M elements of 16 bits into
// FP32, 4.8 GB, 258 us for the squares and 755 for the scaling, 4.7 TB/s).  Squares are summed in FP64, where
// neither they nor their sum leave the range whatever the gradients' size, at two more instructions an element that
// the memory hides.  The list is cut into chunks, and each workgroup takes an equal stretch of them; the order of
// every sum depends on the sizes alone.  The table of tensors comes with a launch's arguments where it fits them,
// else small launches lay it down in the workspace first, so that a captured launch keeps its own.
#include <algorithm>

#include "grads.h"

namespace beam {
namespace {

constexpr int kPerLaunch = 112;  // tensors that fit a launch's 4 KB of arguments
constexpr int kChunk = 2048;     // elements: eight to a thread
constexpr int kUnits = 1024;     // workgroups, and partial sums, at most: sixteen waves a CU
struct GradTable {
  GradTensor t[kPerLaunch];
  int count;
};
static_assert(sizeof(GradTable) <= 3600, "room for the other arguments");

__global__ __launch_bounds__(128) void grad_table_kernel(GradTable part, GradTensor* __restrict__ to) {
  if ((int)threadIdx.x < part.count) to[threadIdx.x] = part.t[threadIdx.x];
}

// Sum over the workgroup's threads, for all of them; s holds a value of each wave.
template <class V>
__device__ __forceinline__ V block_sum(V v, V* s) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  const int waves = blockDim.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  V a = 0;
  for (int w = 0; w < waves; ++w) a += s[w];
  return a;
}

__device__ __forceinline__ double sum_partials(const double* part, int n, double* s) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) v += part[i];
  return block_sum(v, s);
}

// f(tensor, first element, end) for the stretches of the list's chunks from c0 to c1, or from c1 back to c0.  The first
// tensor is found by all threads together, each looking at its share of the table: one latency whatever its length.
template <bool BACK, class F>
__device__ __forceinline__ void stretch(const GradTensor* t, int count, uint32_t c0, uint32_t c1, int* s, F f) {
  if (c0 >= c1) return;
  const uint32_t from = BACK ? c1 - 1 : c0;
  int before = 0;
  for (int i = threadIdx.x; i < count; i += blockDim.x) before += t[i].end <= from;
  int k = __builtin_amdgcn_readfirstlane(block_sum(before, s));
  for (uint32_t c = BACK ? c1 : c0; BACK ? c > c0 : c < c1; BACK ? --k : ++k) {
    const uint32_t start = k ? t[k - 1].end : 0u;
    const uint32_t a = BACK ? max(c0, start) : c, b = BACK ? c : min(c1, t[k].end);
    f(t[k], (int64_t)(a - start) * kChunk, min(t[k].n, (int64_t)(b - start) * kChunk));
    c = BACK ? a : b;
  }
}

template <class F>
__device__ __forceinline__ void by_type(int type, F f) {
  if (type == kElemF32) f(F32{});
  else if (type == kElemF16) f(F16{});
  else f(BF16{});
}

// g(first of eight elements, how many, the eight) for a thread's share of i0 .. i1, four loads in flight, from the
// first on or from the last back.
template <class T, bool BACK, class G>
__device__ __forceinline__ void eights(const typename T::S* p, int64_t i0, int64_t i1, G g) {
  const int64_t across = (int64_t)blockDim.x * 8;
  const int64_t whole = (i1 - i0) / (4 * across), mid = i0 + whole * 4 * across;  // four full rounds at a time, and the rest
  auto rest = [&]() __attribute__((always_inline)) {
    for (int64_t i = mid + (int64_t)threadIdx.x * 8; i < i1; i += across) {
      const int n = (int)min((int64_t)8, i1 - i);
      Raw8<T> r;
      if (n == 8)
        r.load(p + i);
      else
        r.load_part(p + i, n);
      g(i, n, r);
    }
  };
  if (BACK) rest();
  for (int64_t w = 0; w < whole; ++w) {
    const int64_t i = i0 + (BACK ? whole - 1 - w : w) * 4 * across + (int64_t)threadIdx.x * 8;
    Raw8<T> r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) r[u].load(p + i + u * across);
#pragma unroll
    for (int u = 0; u < 4; ++u) g(i + u * across, 8, r[u]);
  }
  if (!BACK) rest();
}

__device__ __forceinline__ double squares(const GradTensor* t, int count, uint32_t c0, uint32_t c1, int* s) {
  double sum = 0.0;
  stretch<false>(t, count, c0, c1, s, [&](const GradTensor& k, int64_t i0, int64_t i1) {
    by_type(k.type, [&](auto type) {
      using T = decltype(type);
      eights<T, false>(static_cast<const typename T::S*>(k.p), i0, i1, [&](int64_t, int, const Raw8<T>& r) {
#pragma unroll
        for (int q = 0; q < 8; ++q) sum = fma((double)r[q], (double)r[q], sum);
      });
    });
  });
  return sum;
}

__device__ __forceinline__ void scaled(const GradTensor* t, int count, uint32_t c0, uint32_t c1, int* s, float f) {
  stretch<true>(t, count, c0, c1, s, [&](const GradTensor& k, int64_t i0, int64_t i1) {
    if (f == 1.f && k.p == k.out) return;  // as they are
    by_type(k.type, [&](auto type) {
      by_type(k.out_type, [&](auto out_type) {
        using T = decltype(type);
        using O = decltype(out_type);
        typename O::S* o = static_cast<typename O::S*>(k.out);
        eights<T, true>(static_cast<const typename T::S*>(k.p), i0, i1, [&](int64_t i, int n, const Raw8<T>& r) {
          float v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = r[q] * f;
          store8<O>(o + i, n, v);
        });
      });
    });
  });
}

__device__ __forceinline__ float factor(const ClipArgs& a, double norm) {
  const double c = a.max_norm / (norm + a.eps);
  return (float)(a.scale * (c > 1.0 ? 1.0 : c));  // NaN stays NaN
}

// This workgroup's stretch of the chunks.
__device__ __forceinline__ uint32_t cut(uint32_t chunks, uint32_t b) {
  return (uint32_t)((uint64_t)chunks * b / gridDim.x);
}

// The table, from the launch's arguments or the workspace.
struct Inline {
  GradTable t;
  __device__ const GradTensor* table() const { return t.t; }
};
struct Laid {
  const GradTensor* t;
  __device__ const GradTensor* table() const { return t; }
};

template <class L>
__global__ __launch_bounds__(256) void grad_squares_kernel(L list, int count, uint32_t chunks,
                                                           double* __restrict__ part) {
  __shared__ double s[4];
  __shared__ int si[4];
  const double sum = block_sum(
      squares(list.table(), count, cut(chunks, blockIdx.x), cut(chunks, blockIdx.x + 1), si), s);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ __launch_bounds__(256) void grad_norm_kernel(const double* __restrict__ part, int n, double scale,
                                                        float* __restrict__ norm) {
  __shared__ double s[4];
  const double sum = sum_partials(part, n, s);
  if (threadIdx.x == 0) *norm = (float)(fabs(scale) * sqrt(sum));
}

// Every workgroup adds the partial sums by itself, so that no launch stands between the norm and the scaling.
template <class L>
__global__ __launch_bounds__(256) void clip_grads_kernel(L list, int count, uint32_t chunks, ClipArgs a,
                                                         const double* __restrict__ part, int parts) {
  __shared__ double s[4];
  __shared__ int si[4];
  const double norm = a.norm_in ? (double)*a.norm_in : fabs(a.scale) * sqrt(sum_partials(part, parts, s));
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  scaled(list.table(), count, cut(chunks, blockIdx.x), cut(chunks, blockIdx.x + 1), si, factor(a, norm));
}

// All of it in one launch of few chunks, one to a wave at a time, so that their latencies run beside each other (30011
// elements 7.4 us; a chunk to a workgroup at a time took 11): every workgroup adds up all squares by itself, or, where
// results replace gradients that others still read, there is one alone.  write: whether there are results besides the norm.
constexpr int kAloneWaves = 16;
// Up to so many chunks, in place or not, and for the norm by itself, so that the norm is one and the same.  On the GPU, in
// place, 5.5 us at 16 chunks and 6.6 above against 6.9 in two launches, but 8.9 at 31 (apart 8.3 and 8.2).
constexpr uint32_t kAlone = 24;
__global__ __launch_bounds__(64 * kAloneWaves) void clip_alone_kernel(Inline list, int count, uint32_t chunks, ClipArgs a,
                                                                      bool write) {
  __shared__ double s[kAloneWaves];
  const GradTensor* t = list.table();
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // f(tensor, first element, eight of them and how many), a quarter of chunk c at a time
  auto chunk = [&](uint32_t c, auto f) __attribute__((always_inline)) {
    static_assert(kPerLaunch <= 128, "two entries to a lane");
    const int k = __popcll(__ballot(lane < count && t[lane].end <= c)) +
                  __popcll(__ballot(lane + 64 < count && t[lane + 64 < count ? lane + 64 : 0].end <= c));
    const GradTensor& e = t[k];
    const int64_t i0 = (int64_t)(c - (k ? t[k - 1].end : 0u)) * kChunk;
    by_type(e.type, [&](auto type) {
      using T = decltype(type);
      const typename T::S* p = static_cast<const typename T::S*>(e.p);
      Raw8<T> r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u * 512 + lane * 8, n = e.n - i;
        if (n >= 8)
          r[u].load(p + i);
        else
          r[u].load_part(p + i, (int)max(n, (int64_t)0));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) f(e, i0 + u * 512 + lane * 8, r[u]);
    });
  };
  double sum = 0.0;
  for (uint32_t c = wave; c < chunks; c += kAloneWaves)
    chunk(c, [&](const GradTensor&, int64_t, const auto& r) {
#pragma unroll
      for (int q = 0; q < 8; ++q) sum = fma((double)r[q], (double)r[q], sum);
    });
  const double norm = fabs(a.scale) * sqrt(block_sum(sum, s));  // all reads lie before its barriers
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  const float f = factor(a, norm);
  if (!write) return;
  for (uint32_t c = blockIdx.x * kAloneWaves + wave; c < chunks; c += gridDim.x * kAloneWaves)
    chunk(c, [&](const GradTensor& e, int64_t i, const auto& r) {
      if (i >= e.n || (f == 1.f && e.p == e.out)) return;
      by_type(e.out_type, [&](auto out_type) {
        using O = decltype(out_type);
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = r[q] * f;
        store8<O>(static_cast<typename O::S*>(e.out) + i, (int)min((int64_t)8, e.n - i), v);
      });
    });
}

struct List {
  const GradTensor* laid;  // in the workspace; null: `all` goes with the launch
  Inline all;
  int count;
  uint32_t chunks;
  int units;
  double* part;
};

size_t table_bytes(int count) { return count > kPerLaunch ? (size_t)count * sizeof(GradTensor) : 0; }

hipError_t prepare(List& l, GradTensor* t, int count, void* ws, hipStream_t st) {
  l.count = count;
  l.chunks = 0;
  for (int i = 0; i < count; ++i) t[i].end = l.chunks += (uint32_t)((t[i].n + kChunk - 1) / kChunk);
  l.units = (int)std::min<uint32_t>(l.chunks, kUnits);
  l.laid = nullptr;
  l.part = reinterpret_cast<double*>(static_cast<char*>(ws) + table_bytes(count));
  if (count <= kPerLaunch) {
    std::copy(t, t + count, l.all.t.t);
    return hipSuccess;
  }
  l.laid = static_cast<GradTensor*>(ws);
  for (int i = 0; i < count; i += kPerLaunch) {
    GradTable& g = l.all.t;
    g.count = std::min(count - i, kPerLaunch);
    std::copy(t + i, t + i + g.count, g.t);
    hipLaunchKernelGGL(grad_table_kernel, dim3(1), dim3(128), 0, st, g, static_cast<GradTensor*>(ws) + i);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_squares(const List& l, hipStream_t st) {
  if (l.laid)
    hipLaunchKernelGGL(grad_squares_kernel<Laid>, dim3(l.units), dim3(256), 0, st, Laid{l.laid}, l.count, l.chunks,
                       l.part);
  else
    hipLaunchKernelGGL(grad_squares_kernel<Inline>, dim3(l.units), dim3(256), 0, st, l.all, l.count, l.chunks, l.part);
  return hipGetLastError();
}

hipError_t launch_alone(const List& l, const ClipArgs& a, bool write, int groups, hipStream_t st) {
  hipLaunchKernelGGL(clip_alone_kernel, dim3(groups), dim3(64 * kAloneWaves), 0, st, l.all, l.count, l.chunks, a, write);
  return hipGetLastError();
}

}  // namespace

size_t grad_workspace(int count) { return table_bytes(count) + kUnits * sizeof(double); }

hipError_t launch_grad_norm(GradTensor* t, int count, double scale, void* ws, float* norm, hipStream_t st) {
  List l;
  hipError_t e = prepare(l, t, count, ws, st);
  if (e != hipSuccess) return e;
  if (!l.laid && l.chunks <= kAlone)
    return launch_alone(l, {scale, 0.0, 1.0, nullptr, norm}, false, 1, st);
  if ((e = launch_squares(l, st)) != hipSuccess) return e;
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(256), 0, st, l.part, l.units, scale, norm);
  return hipGetLastError();
}

hipError_t launch_clip_grads(GradTensor* t, int count, const ClipArgs& a, void* ws, hipStream_t st) {
  List l;
  hipError_t e = prepare(l, t, count, ws, st);
  if (e != hipSuccess) return e;
  if (!l.laid && !a.norm_in && l.chunks <= kAlone) {
    const bool in_place = std::any_of(t, t + count, [](const GradTensor& k) { return k.p == k.out; });
    return launch_alone(l, a, true, in_place ? 1 : std::max(1, (int)(l.chunks + kAloneWaves - 1) / kAloneWaves), st);
  }
  if (!a.norm_in && (e = launch_squares(l, st)) != hipSuccess) return e;
  if (l.chunks == 0 && !a.norm) return hipSuccess;  // nothing to scale by a given norm, nor to write
  const dim3 grid(std::max(l.units, 1));
  if (l.laid)
    hipLaunchKernelGGL(clip_grads_kernel<Laid>, grid, dim3(256), 0, st, Laid{l.laid}, l.count, l.chunks, a, l.part,
                       l.units);
  else
    hipLaunchKernelGGL(clip_grads_kernel<Inline>, grid, dim3(256), 0, st, l.all, l.count, l.chunks, a, l.part, l.units);
  return hipGetLastError();
}

}  // namespace beam
