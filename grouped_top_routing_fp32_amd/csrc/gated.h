// What the kernels of gated.hip share with the ABI: the two projections of a gated layer and their gradients.
#pragma once

#include "linear.h"

namespace beam {

// Columns of dz_gate and of dz_up in their common buffer: whole stages of the products that read it.
__host__ __device__ inline int gated_half(int N) { return (N + 63) / 64 * 64; }

struct GatedPlan {
  GemmPlan gemm;
  bool stream;                      // the persistent kernel's 256-row tiles
  bool copy_x, copy_gate, copy_up;  // laid out anew in the workspace, in this order
  size_t off_gate, off_up, off_gemm, total;
};
GatedPlan plan_gated(int M, int N, int K, int64_t ldx, int64_t ldg, int64_t ldu);
hipError_t launch_gated(const GatedArgs& g, const GatedPlan& p, void* ws, hipStream_t st);

// dx and dw of a gated layer of N columns, planned together.
void plan_gated_gradients(int rows, int N, int inner, GemmPlan* dx, GemmPlan* dw);
int gated_dz_units(int M);
size_t gated_peak_bytes();
struct GatedDz {
  const void* dh;
  int dh_type;
  int64_t lddh;
  const void *zg, *zu;
  int64_t ldzg, ldzu;
  int act, type;
  uint32_t* peaks;  // both with an fp16 dz alone
  float* unscale;
  uint16_t* dz;  // [M][2 half]; null: not wanted
  float* part;   // [units][2 N]; null: not wanted
  int M, N;
};
// With them the operands that have to be laid out anew.
hipError_t launch_gated_dz(const GatedDz& d, PadJobs pad, hipStream_t st);
// The bias gradients by themselves (beside dx's product they need no launch).
hipError_t launch_gated_sums(const SumJob& j, hipStream_t st);
// Both products of the backward pass, or one (the other's out null), as planned together.
hipError_t launch_gated_gradients(const GatedArgs& dx, const GemmPlan& px, const GatedArgs& dw, const GemmPlan& pw,
                                  void* ws, hipStream_t st);

}  // namespace beam
