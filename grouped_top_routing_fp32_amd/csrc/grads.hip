// The norm of all gradients of a step and their clipping (gfx950).
//
//   norm = |scale| sqrt(sum over all tensors of g^2),  out = g scale min(1, max_norm / (norm + eps))
//
// Bound by HBM: every gradient is read for the norm and again for its scaling.  Squares are summed in FP64, where
// neither they nor their sum leave the range whatever the gradients' size, at two more instructions an element that
// the memory hides.  A launch takes as many tensors as its arguments hold, so no table is copied to the device
// and a captured launch keeps its own.  A workgroup takes chunks of the list in turn; the order of every
// sum depends on the sizes alone.
#include "grads.h"

namespace beam {
namespace {

constexpr int kPerLaunch = 120;   // tensors whose table fits a launch's 4 KB of arguments
constexpr int kChunk = 8192;      // elements
constexpr int kUnits = 1024;      // workgroups that share the chunks, about: four to a CU

struct GradTable {
  const void* p[kPerLaunch];
  void* out[kPerLaunch];
  int64_t n[kPerLaunch];
  uint32_t end[kPerLaunch];  // chunks up to this tensor's last
  uint8_t type[kPerLaunch], out_type[kPerLaunch];
  int count;
  uint32_t chunks;
};
static_assert(sizeof(GradTable) <= 3800, "room for the other arguments");

// Sum over the workgroup's threads, for all of them.
__device__ __forceinline__ double block_sum(double v, double* s) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  const int waves = blockDim.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  double a = 0.0;
  for (int w = 0; w < waves; ++w) a += s[w];
  return a;
}

__device__ __forceinline__ double sum_partials(const double* part, int n, double* s) {
  double v = 0.0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) v += part[i];
  return block_sum(v, s);
}

// f(tensor, first element, elements) for each chunk of this workgroup.
template <class F>
__device__ __forceinline__ void chunks_of(const GradTable& t, F f) {
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {  // the first tensor that ends behind c
      const int mid = (lo + hi) / 2;
      if (t.end[mid] > c) hi = mid;
      else lo = mid + 1;
    }
    const int64_t i0 = (int64_t)(c - (lo ? t.end[lo - 1] : 0u)) * kChunk;
    f(lo, i0, (int)min((int64_t)kChunk, t.n[lo] - i0));
  }
}

template <class F>
__device__ __forceinline__ void by_type(int type, F f) {
  if (type == kElemF32) f(F32{});
  else if (type == kElemF16) f(F16{});
  else f(BF16{});
}

__global__ __launch_bounds__(256) void grad_squares_kernel(GradTable t, double* __restrict__ part) {
  __shared__ double s[4];
  double sum = 0.0;
  chunks_of(t, [&](int k, int64_t i0, int n) {
    by_type(t.type[k], [&](auto type) {
      using T = decltype(type);
      const typename T::S* p = static_cast<const typename T::S*>(t.p[k]) + i0;
#pragma unroll 4
      for (int i = threadIdx.x * 8; i < n; i += 256 * 8) {
        float v[8];
        load8<T>(p + i, n - i, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum = fma((double)v[q], (double)v[q], sum);
      }
    });
  });
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ __launch_bounds__(256) void grad_norm_kernel(const double* __restrict__ part, int n, double scale,
                                                        float* __restrict__ norm) {
  __shared__ double s[4];
  const double sum = sum_partials(part, n, s);
  if (threadIdx.x == 0) *norm = (float)(fabs(scale) * sqrt(sum));
}

// Every workgroup adds the partial sums by itself, so that no launch stands between the norm and the scaling.
__global__ __launch_bounds__(256) void clip_grads_kernel(GradTable t, ClipArgs a, const double* __restrict__ part,
                                                         int parts) {
  __shared__ double s[4];
  const double norm = a.norm_in ? (double)*a.norm_in : fabs(a.scale) * sqrt(sum_partials(part, parts, s));
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  const double c = a.max_norm / (norm + a.eps);
  const float f = (float)(a.scale * (c > 1.0 ? 1.0 : c));  // NaN stays NaN
  chunks_of(t, [&](int k, int64_t i0, int n) {
    if (f == 1.f && t.p[k] == t.out[k]) return;  // as they are
    by_type(t.type[k], [&](auto type) {
      by_type(t.out_type[k], [&](auto out_type) {
        using T = decltype(type);
        using O = decltype(out_type);
        const typename T::S* p = static_cast<const typename T::S*>(t.p[k]) + i0;
        typename O::S* o = static_cast<typename O::S*>(t.out[k]) + i0;
#pragma unroll 4
        for (int i = threadIdx.x * 8; i < n; i += 256 * 8) {
          float v[8];
          load8<T>(p + i, n - i, v);
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] *= f;
          store8<O>(o + i, n - i, v);
        }
      });
    });
  });
}

uint32_t chunks(int64_t n) { return (uint32_t)((n + kChunk - 1) / kChunk); }

// f(table, workgroups) for each launch's share of the list; stops at the first error.
template <class F>
hipError_t each_launch(const GradTensor* t, int count, F f) {
  uint64_t total = 0;
  for (int i = 0; i < count; ++i) total += chunks(t[i].n);
  for (int i = 0; i < count;) {
    GradTable g{};
    for (; i < count && g.count < kPerLaunch; ++i) {
      if (t[i].n == 0) continue;
      const int k = g.count++;
      g.p[k] = t[i].p;
      g.out[k] = t[i].out;
      g.n[k] = t[i].n;
      g.type[k] = (uint8_t)t[i].type;
      g.out_type[k] = (uint8_t)t[i].out_type;
      g.end[k] = g.chunks += chunks(t[i].n);
    }
    if (g.count == 0) break;
    const uint32_t units = (uint32_t)(total <= kUnits ? g.chunks : (g.chunks * (uint64_t)kUnits + total - 1) / total);
    const hipError_t e = f(g, (int)units);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_squares(const GradTensor* t, int count, double* part, int* parts, hipStream_t st) {
  *parts = 0;
  return each_launch(t, count, [&](const GradTable& g, int units) {
    hipLaunchKernelGGL(grad_squares_kernel, dim3(units), dim3(256), 0, st, g, part + *parts);
    *parts += units;
    return hipGetLastError();
  });
}

}  // namespace

// The shares of kUnits are rounded up, one more to a launch at most.
int grad_partials(int count) { return kUnits + (count + kPerLaunch - 1) / kPerLaunch; }

hipError_t launch_grad_norm(const GradTensor* t, int count, double scale, double* part, float* norm, hipStream_t st) {
  int parts = 0;
  const hipError_t e = launch_squares(t, count, part, &parts, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(256), 0, st, part, parts, scale, norm);
  return hipGetLastError();
}

hipError_t launch_clip_grads(const GradTensor* t, int count, const ClipArgs& args, double* part, hipStream_t st) {
  int parts = 0;
  if (!args.norm_in) {
    const hipError_t e = launch_squares(t, count, part, &parts, st);
    if (e != hipSuccess) return e;
  }
  ClipArgs a = args;
  bool any = false;
  const hipError_t e = each_launch(t, count, [&](const GradTable& g, int units) {
    hipLaunchKernelGGL(clip_grads_kernel, dim3(units), dim3(256), 0, st, g, a, part, parts);
    a.norm = nullptr;
    any = true;
    return hipGetLastError();
  });
  if (e != hipSuccess || any || !a.norm) return e;
  // no element at all
  hipLaunchKernelGGL(clip_grads_kernel, dim3(1), dim3(256), 0, st, GradTable{}, a, part, 0);
  return hipGetLastError();
}

}  // namespace beam
