// C ABI of the operators around the block (layer norm, balance loss, the
// router's gradient, linear): argument validation, workspace carving and kernel
// launches on the caller's stream.  The operations and conventions are stated in
// include/beam_moe.h.
#include <cmath>

#include "abi_util.h"
#include "linear.h"

namespace beam {
int layer_norm_max_cols();
int layer_norm_backward_units(int T);
hipError_t launch_layer_norm(const void* x, int x_type, int64_t ldx, const float* gamma, const float* beta, void* y,
                             int y_type, int64_t ldy, float* mean, float* rstd, int T, int H, float eps,
                             hipStream_t st);
hipError_t launch_layer_norm_backward(const void* dy, int dy_type, int64_t lddy, const void* x, int x_type,
                                      int64_t ldx, const float* mean, const float* rstd, const float* gamma, void* dx,
                                      int64_t lddx, float* dgamma, float* dbeta, float* part, int T, int H,
                                      hipStream_t st);
int balance_units(int T, int B);
hipError_t launch_balance(const float* scores, const int32_t* ids, int B, const int32_t* off, int T, int E, int K,
                          float alpha, float* loss, int32_t* counts, float* prob, int32_t* part_count, float* part_sum,
                          hipStream_t st);
hipError_t launch_route_backward(const float* scores, const int32_t* ids, const float* dw, float scale, int B,
                                 const int32_t* off, float alpha, const float* dloss, const int32_t* counts,
                                 float* dlogits, int T, int E, int K, hipStream_t st);
int linear_dz_units(int M);
size_t linear_peak_bytes();
hipError_t launch_linear_dz(const void* dy, int dy_type, int64_t lddy, const void* z, int64_t ldz, int act, float keep,
                            float add, uint32_t* peaks, float* unscale, uint16_t* dz, int64_t lddz, int type,
                            float* part, void* dres, int64_t lddres, int M, int N, const PadJob& first,
                            const PadJob& second, hipStream_t st);
}  // namespace beam

namespace {

using beam::act_ok;
using beam::align_up;
using beam::aligned16;
using beam::at;
using beam::check_optional;
using beam::check_ptrs;
using beam::half_type;
using beam::hip_status;
using beam::ld_ok;
using beam::type_ok;

constexpr int32_t kMaxNormRows = 1 << 21;   // the grid's threads fit 32 bits
constexpr int32_t kMaxGradTokens = 1 << 25;
constexpr int32_t kMaxSeqs = 1 << 20;
constexpr int32_t kMaxLinearRows = 1 << 20;
constexpr int32_t kMaxLinearCols = 1 << 18;

int check_norm(int32_t rows, int32_t cols) {
  if (rows < 0) return BEAM_MOE_ERR_INVALID_ARG;
  if (cols < 1 || cols > beam::layer_norm_max_cols() || rows > kMaxNormRows) return BEAM_MOE_ERR_UNSUPPORTED;
  return BEAM_MOE_OK;
}

int check_seqs(int32_t num_seqs, const int32_t* seq_offsets) {
  if (num_seqs < 1 || (!seq_offsets && num_seqs != 1) || !aligned16(seq_offsets)) return BEAM_MOE_ERR_INVALID_ARG;
  return num_seqs > kMaxSeqs ? BEAM_MOE_ERR_UNSUPPORTED : BEAM_MOE_OK;
}

int check_linear(int32_t rows, int32_t cols, int32_t inner) {
  if (rows < 0) return BEAM_MOE_ERR_INVALID_ARG;
  if (rows > kMaxLinearRows || cols < 1 || cols > kMaxLinearCols || inner < 1 || inner > kMaxLinearCols)
    return BEAM_MOE_ERR_UNSUPPORTED;
  return BEAM_MOE_OK;
}

// Workspace of the backward pass: dz, the partial sums of dbias, the inverse of an fp16 dz's
// scale with the maxima that give it, w and x where they are laid out anew, then the partial sums of the two products, in the same place unless they
// run in one launch.  Where dz is dy itself its place stays unused; the size does not depend on it.
struct BackwardPlan {
  size_t off_dz, off_part, off_scale, off_w, off_x, off_gemm, total;
  int64_t lddz;
  bool copy_w, copy_x;
  beam::GemmPlan dx, dw;
};

constexpr size_t kScaleBytes = 256;  // before the maxima

BackwardPlan backward_plan(int32_t rows, int32_t cols, int32_t inner, int64_t ldx, int64_t ldw) {
  BackwardPlan p;
  p.lddz = beam::up8(cols);
  p.copy_w = !beam::regular_rows(ldw, inner);
  p.copy_x = !beam::regular_rows(ldx, inner);
  beam::plan_gradients(rows, cols, inner, &p.dx, &p.dw);
  p.off_dz = 0;
  p.off_part = align_up(beam::padded_bytes(rows, cols));
  p.off_scale = p.off_part + align_up((size_t)beam::linear_dz_units(rows) * cols * sizeof(float));
  p.off_w = p.off_scale + kScaleBytes + align_up(beam::linear_peak_bytes());
  p.off_x = p.off_w + align_up(p.copy_w ? beam::padded_bytes(cols, inner) : 0);
  p.off_gemm = p.off_x + align_up(p.copy_x ? beam::padded_bytes(rows, inner) : 0);
  p.total = p.off_gemm + (p.dx.paired                   ? p.dx.total + p.dw.total
                          : p.dx.total > p.dw.total ? p.dx.total
                                                    : p.dw.total);
  return p;
}

}  // namespace

extern "C" {

int beam_moe_layer_norm(int32_t rows, int32_t cols, const void* x, int x_type, int64_t ldx, const float* gamma,
                        const float* beta, float eps, void* y, int y_type, int64_t ldy, float* mean, float* rstd,
                        void* stream) {
  int rc = check_norm(rows, cols);
  if (rc != BEAM_MOE_OK) return rc;
  if (!type_ok(x_type) || !type_ok(y_type) || !std::isfinite(eps) || eps < 0.f) return BEAM_MOE_ERR_INVALID_ARG;
  if (rows == 0) return BEAM_MOE_OK;
  if (!ld_ok(ldx, cols) || !ld_ok(ldy, cols)) return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_ptrs({x, y})) != BEAM_MOE_OK) return rc;
  if ((rc = check_optional({gamma, beta, mean, rstd})) != BEAM_MOE_OK) return rc;
  return hip_status(beam::launch_layer_norm(x, x_type, ldx, gamma, beta, y, y_type, ldy, mean, rstd, rows, cols, eps,
                                            static_cast<hipStream_t>(stream)));
}

size_t beam_moe_layer_norm_backward_workspace_bytes(int32_t rows, int32_t cols) {
  if (check_norm(rows, cols) != BEAM_MOE_OK) return SIZE_MAX;
  return (size_t)beam::layer_norm_backward_units(rows) * cols * 2 * sizeof(float);
}

int beam_moe_layer_norm_backward(int32_t rows, int32_t cols, const void* dy, int dy_type, int64_t lddy, const void* x,
                                 int x_type, int64_t ldx, const float* mean, const float* rstd, const float* gamma,
                                 void* dx, int64_t lddx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                                 void* stream) {
  int rc = check_norm(rows, cols);
  if (rc != BEAM_MOE_OK) return rc;
  if (!type_ok(dy_type) || !type_ok(x_type)) return BEAM_MOE_ERR_INVALID_ARG;
  const bool sums = dgamma || dbeta;
  if (!dx && !sums) return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_optional({gamma, dx, dgamma, dbeta})) != BEAM_MOE_OK) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (rows == 0) return sums ? hip_status(beam::launch_column_sums(nullptr, dgamma, dbeta, 0, cols, st)) : BEAM_MOE_OK;
  if (!ld_ok(lddy, cols) || !ld_ok(ldx, cols) || (dx && !ld_ok(lddx, cols))) return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_ptrs({dy, x, mean, rstd})) != BEAM_MOE_OK) return rc;
  const size_t need = sums ? beam_moe_layer_norm_backward_workspace_bytes(rows, cols) : 0;
  if (need && (!ws || !aligned16(ws) || ws_bytes < need)) return BEAM_MOE_ERR_WORKSPACE;
  return hip_status(beam::launch_layer_norm_backward(dy, dy_type, lddy, x, x_type, ldx, mean, rstd, gamma, dx, lddx,
                                                     dgamma, dbeta, static_cast<float*>(ws), rows, cols, st));
}

size_t beam_moe_balance_loss_workspace_bytes(const beam_moe_dims* dims, int32_t T, int32_t num_seqs) {
  if (beam::check_block(dims, T) != BEAM_MOE_OK || num_seqs < 1 || num_seqs > kMaxSeqs) return SIZE_MAX;
  return 2 * align_up((size_t)beam::balance_units(T, num_seqs) * dims->num_experts * 4);
}

int beam_moe_balance_loss(const beam_moe_dims* d, int32_t T, const float* scores, const int32_t* topk_ids,
                          int32_t num_seqs, const int32_t* seq_offsets, float alpha, float* loss, int32_t* counts,
                          float* prob, void* ws, size_t ws_bytes, void* stream) {
  int rc = beam::check_block(d, T);
  if (rc != BEAM_MOE_OK) return rc;
  if ((rc = check_seqs(num_seqs, seq_offsets)) != BEAM_MOE_OK) return rc;
  if (!std::isfinite(alpha)) return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_ptrs({loss, counts, prob})) != BEAM_MOE_OK) return rc;
  if (T > 0 && (rc = check_ptrs({scores, topk_ids})) != BEAM_MOE_OK) return rc;
  const size_t need = beam_moe_balance_loss_workspace_bytes(d, T, num_seqs);
  if (need && (!ws || !aligned16(ws) || ws_bytes < need)) return BEAM_MOE_ERR_WORKSPACE;
  return hip_status(beam::launch_balance(scores, topk_ids, num_seqs, seq_offsets, T, d->num_experts, d->topk, alpha,
                                         loss, counts, prob, at<int32_t>(ws, 0), at<float>(ws, need / 2),
                                         static_cast<hipStream_t>(stream)));
}

int beam_moe_route_backward(const beam_moe_dims* d, int32_t T, const float* scores, const int32_t* topk_ids,
                            const float* dw, int32_t num_seqs, const int32_t* seq_offsets, float alpha,
                            const float* dloss, const int32_t* counts, float* dlogits, void* stream) {
  int rc = beam::check_block(d, T);
  if (rc != BEAM_MOE_OK) return rc;
  if (T > kMaxGradTokens) return BEAM_MOE_ERR_UNSUPPORTED;
  if ((rc = check_seqs(num_seqs, seq_offsets)) != BEAM_MOE_OK) return rc;
  if (!std::isfinite(alpha) || (!dw && !dloss) || (dloss && !counts)) return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_optional({dw, dloss, counts})) != BEAM_MOE_OK || T == 0) return rc;
  if ((rc = check_ptrs({scores, topk_ids, dlogits})) != BEAM_MOE_OK) return rc;
  return hip_status(beam::launch_route_backward(scores, topk_ids, dw, d->routed_scaling, num_seqs, seq_offsets, alpha,
                                                dloss, counts, dlogits, T, d->num_experts, d->topk,
                                                static_cast<hipStream_t>(stream)));
}

size_t beam_moe_linear_workspace_bytes(int32_t rows, int32_t cols, int32_t inner, int64_t ldx, int64_t ldw) {
  if (check_linear(rows, cols, inner) != BEAM_MOE_OK || !ld_ok(ldx, inner) || !ld_ok(ldw, inner)) return SIZE_MAX;
  return beam::plan_linear(rows, cols, inner, ldx, ldw).total;
}

int beam_moe_linear(int32_t rows, int32_t cols, int32_t inner, int type, const void* x, int64_t ldx, const void* w,
                    int64_t ldw, const float* bias, int act, const void* res, int64_t ldr, float keep, float add,
                    void* y, int y_type, int64_t ldy, void* pre, int64_t ldpre, void* ws, size_t ws_bytes,
                    void* stream) {
  int rc = check_linear(rows, cols, inner);
  if (rc != BEAM_MOE_OK) return rc;
  if (!half_type(type) || (y_type != type && y_type != BEAM_MOE_F32) || !act_ok(act) || !std::isfinite(keep) ||
      !std::isfinite(add))
    return BEAM_MOE_ERR_INVALID_ARG;
  if (rows == 0) return BEAM_MOE_OK;
  if (!ld_ok(ldx, inner) || !ld_ok(ldw, inner) || !ld_ok(ldy, cols) || (res && !ld_ok(ldr, cols)) ||
      (pre && !ld_ok(ldpre, cols)) || (res == y && ldr != ldy))
    return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_ptrs({x, w, y})) != BEAM_MOE_OK) return rc;
  if ((rc = check_optional({bias, res, pre})) != BEAM_MOE_OK) return rc;
  const beam::GemmPlan plan = beam::plan_linear(rows, cols, inner, ldx, ldw);
  if (plan.total && (!ws || !aligned16(ws) || ws_bytes < plan.total)) return BEAM_MOE_ERR_WORKSPACE;
  beam::GemmArgs g{};
  g.a = x;
  g.lda = ldx;
  g.b = w;
  g.ldb = ldw;
  g.M = rows;
  g.N = cols;
  g.K = inner;
  g.type = type;
  g.bias = bias;
  g.act = act;
  g.res = res;
  g.ldr = ldr;
  g.keep = keep;
  g.add = add;
  g.out = y;
  g.out_type = y_type;
  g.ldo = ldy;
  g.pre = pre;
  g.ldp = ldpre;
  return hip_status(beam::launch_gemm(g, plan, ws, static_cast<hipStream_t>(stream)));
}

size_t beam_moe_linear_backward_workspace_bytes(int32_t rows, int32_t cols, int32_t inner, int64_t ldx, int64_t ldw) {
  if (check_linear(rows, cols, inner) != BEAM_MOE_OK || !ld_ok(ldx, inner) || !ld_ok(ldw, inner)) return SIZE_MAX;
  return backward_plan(rows, cols, inner, ldx, ldw).total;
}

int beam_moe_linear_backward(int32_t rows, int32_t cols, int32_t inner, int type, const void* dy, int dy_type,
                             int64_t lddy, const void* x, int64_t ldx, const void* w, int64_t ldw, const void* pre,
                             int64_t ldpre, int act, float keep, float add, void* dx, int64_t lddx, void* dw,
                             int64_t lddw, float* dbias, void* dres, int64_t lddres, void* ws, size_t ws_bytes,
                             void* stream) {
  int rc = check_linear(rows, cols, inner);
  if (rc != BEAM_MOE_OK) return rc;
  if (!half_type(type) || (dy_type != type && dy_type != BEAM_MOE_F32) || !act_ok(act) || !std::isfinite(keep) ||
      !std::isfinite(add) || (!dx && !dw && !dbias && !dres))
    return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_optional({x, w, pre, dx, dw, dbias, dres})) != BEAM_MOE_OK) return rc;
  if ((dx && !ld_ok(lddx, inner)) || (dw && !ld_ok(lddw, inner)) || (dres && !ld_ok(lddres, cols)))
    return BEAM_MOE_ERR_INVALID_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (rows > 0) {
    if ((rc = check_ptrs({dy})) != BEAM_MOE_OK) return rc;
    if ((dx && !w) || (dw && !x) || (act != BEAM_MOE_ACT_NONE && !pre) || !ld_ok(lddy, cols) ||
        (pre && !ld_ok(ldpre, cols)) || (x && !ld_ok(ldx, inner)) || (w && !ld_ok(ldw, inner)))
      return BEAM_MOE_ERR_INVALID_ARG;
  }
  const BackwardPlan p = backward_plan(rows, cols, inner, x ? ldx : inner, w ? ldw : inner);
  if (rows > 0 && (!ws || !aligned16(ws) || ws_bytes < p.total)) return BEAM_MOE_ERR_WORKSPACE;
  float* part = dbias ? at<float>(ws, p.off_part) : nullptr;
  void* gemm_ws = at<void*>(ws, p.off_gemm);
  // dz is dy itself where nothing changes it and its rows are whole chunks
  const bool same = act == BEAM_MOE_ACT_NONE && add == 1.f && dy_type == type && lddy % 8 == 0 && cols % 8 == 0;
  uint16_t* dz = same || !(dx || dw) ? nullptr : at<uint16_t>(ws, p.off_dz);
  beam::PadJob jw{}, jx{};
  if (dx && p.copy_w && rows > 0) {
    jw = {w, ldw, cols, inner, at<void*>(ws, p.off_w)};
    w = jw.dst;
    ldw = beam::up8(inner);
  }
  if (dw && p.copy_x && rows > 0) {
    jx = {x, ldx, rows, inner, at<void*>(ws, p.off_x)};
    x = jx.dst;
    ldx = beam::up8(inner);
  }
  float* unscale = dz && type == BEAM_MOE_F16 && rows > 0 ? at<float>(ws, p.off_scale) : nullptr;
  rc = hip_status(rows > 0 && (dz || part || dres)
                      ? beam::launch_linear_dz(dy, dy_type, lddy, pre, ldpre, act, keep, add,
                                               at<uint32_t>(ws, p.off_scale + kScaleBytes), unscale, dz, p.lddz, type,
                                               part, dres, lddres, rows, cols, jw, jx, st)
                      : beam::launch_pad(jw, jx, {}, st));
  if (rc != BEAM_MOE_OK) return rc;
  beam::GemmArgs gx{}, gw{};
  gx.type = gx.out_type = gw.type = gw.out_type = type;
  gx.add = gw.add = 1.f;
  gx.add_at = gw.add_at = unscale;
  gx.a = gw.a = same ? dy : dz;
  gx.lda = gw.lda = same ? lddy : p.lddz;
  gx.b = w;
  gx.ldb = ldw;
  gx.bt = true;
  gx.M = rows;
  gx.N = inner;
  gx.K = cols;
  gx.out = dx;
  gx.ldo = lddx;
  gw.b = x;
  gw.ldb = ldx;
  gw.at = gw.bt = true;
  gw.M = cols;
  gw.N = inner;
  gw.K = rows;
  gw.out = dw;
  gw.ldo = lddw;
  const int units = rows > 0 ? beam::linear_dz_units(rows) : 0;
  if (dx && rows > 0) {
    gx.sums = {part, dbias, units, cols};
    return hip_status(dw ? beam::launch_gemm_pair(gx, p.dx, gw, p.dw, gemm_ws, st)
                         : beam::launch_gemm(gx, p.dx, gemm_ws, st));
  }
  if (dbias) {
    rc = hip_status(beam::launch_column_sums(part, dbias, nullptr, units, cols, st));
    if (rc != BEAM_MOE_OK) return rc;
  }
  if (dw) return hip_status(beam::launch_gemm(gw, p.dw, gemm_ws, st));
  return BEAM_MOE_OK;
}

}  // extern "C"
