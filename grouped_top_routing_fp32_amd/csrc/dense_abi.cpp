// C ABI of the operators of a dense gated sublayer, trained and served (the gated projections and their
// gradients, the norm of all gradients and their clipping, microscaled 4-bit floating point): argument validation,
// workspace carving and kernel launches on the caller's stream.  The operations and conventions are stated in include/beam_moe.h.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "abi_util.h"
#include "gated.h"
#include "grads.h"
#include "mxfp4.h"

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

constexpr int32_t kMaxGrads = 1 << 16;
constexpr int64_t kMaxGradSize = int64_t(1) << 40;
constexpr int64_t kMaxGradTotal = int64_t(1) << 42;  // chunks fit 32 bits
constexpr int32_t kMaxMxRows = 1 << 20;
constexpr int32_t kMaxMxCols = 1 << 18;

int64_t elem_bytes(int type) { return type == BEAM_MOE_F32 ? 4 : 2; }

int check_grads(int32_t count, const void* const* grads, const int32_t* types, const int64_t* sizes) {
  if (count < 0 || (count > 0 && (!grads || !types || !sizes))) return BEAM_MOE_ERR_INVALID_ARG;
  if (count > kMaxGrads) return BEAM_MOE_ERR_UNSUPPORTED;
  int64_t total = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (!type_ok(types[i]) || sizes[i] < 0) return BEAM_MOE_ERR_INVALID_ARG;
    if (sizes[i] > kMaxGradSize) return BEAM_MOE_ERR_UNSUPPORTED;
    if (sizes[i] > 0 && (!grads[i] || reinterpret_cast<uintptr_t>(grads[i]) % elem_bytes(types[i]) != 0))
      return BEAM_MOE_ERR_INVALID_ARG;
    total += sizes[i];
  }
  return total > kMaxGradTotal ? BEAM_MOE_ERR_UNSUPPORTED : BEAM_MOE_OK;
}

// Whether every output lies apart from the other outputs and from the other gradients, the norm that is read apart from
// the outputs, and the one that is written apart from all.
bool apart(const std::vector<beam::GradTensor>& t, const float* norm_in, const float* norm) {
  struct Span {
    uintptr_t a, b;
    bool out;
  };
  auto grad = [](const beam::GradTensor& k) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(k.p);
    return Span{p, p + k.n * elem_bytes(k.type), false};
  };
  auto out = [](const beam::GradTensor& k) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(k.out);
    return Span{p, p + k.n * elem_bytes(k.out_type), true};
  };
  auto replaced = [](const beam::GradTensor& k) { return k.p == k.out && k.type == k.out_type; };
  auto clear = [&](const float* one, bool written) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(one);
    auto off = [p](const Span& s) { return p + sizeof(float) <= s.a || p >= s.b; };
    return !one || std::all_of(t.begin(), t.end(), [&](const beam::GradTensor& k) {
      return off(out(k)) && (!written || off(grad(k)));
    });
  };
  if (!clear(norm_in, false) || !clear(norm, true)) return false;
  // outputs in order, and no gradient among them, as with a flat buffer: no sorting
  uintptr_t first = UINTPTR_MAX, last = 0;
  bool ordered = true;
  for (const auto& k : t) {
    const Span o = out(k);
    ordered = ordered && o.a >= last;
    first = std::min(first, o.a);
    last = std::max(last, o.b);
  }
  if (ordered && std::none_of(t.begin(), t.end(), [&](const beam::GradTensor& k) {
        const Span g = grad(k);
        return !replaced(k) && g.a < last && g.b > first;
      }))
    return true;
  std::vector<Span> spans;
  spans.reserve(2 * t.size());
  for (const auto& k : t) {
    spans.push_back(out(k));
    if (!replaced(k)) spans.push_back(grad(k));
  }
  std::sort(spans.begin(), spans.end(), [](const Span& x, const Span& y) { return x.a < y.a; });
  uintptr_t out_end = 0, grad_end = 0;  // of what lies before
  for (const Span& s : spans) {
    if (s.a < out_end || (s.out && s.a < grad_end)) return false;
    uintptr_t& end = s.out ? out_end : grad_end;
    end = std::max(end, s.b);
  }
  return true;
}

int check_mx(int32_t rows, int32_t cols) {
  if (rows < 0) return BEAM_MOE_ERR_INVALID_ARG;
  return rows > kMaxMxRows || cols < 1 || cols > kMaxMxCols ? BEAM_MOE_ERR_UNSUPPORTED : BEAM_MOE_OK;
}

bool mx_rows_ok(int64_t cols, int64_t ldc, int64_t lds) {
  const int64_t blocks = beam::mx_blocks(cols);
  return ldc % 16 == 0 && ld_ok(ldc, 16 * blocks) && ld_ok(lds, blocks);
}

int check_mx_linear(int32_t rows, int32_t cols, int32_t inner) {
  if (rows < 0) return BEAM_MOE_ERR_INVALID_ARG;
  return cols < 1 || cols > kMaxMxCols ? BEAM_MOE_ERR_UNSUPPORTED : check_mx(rows, inner);
}

constexpr int32_t kMaxGatedRows = 1 << 20;
constexpr int32_t kMaxGatedCols = 1 << 17;  // both projections' are those of one product
constexpr int32_t kMaxGatedInner = 1 << 18;

int check_gated(int32_t rows, int32_t cols, int32_t inner) {
  if (rows < 0) return BEAM_MOE_ERR_INVALID_ARG;
  return rows > kMaxGatedRows || cols < 1 || cols > kMaxGatedCols || inner < 1 || inner > kMaxGatedInner
             ? BEAM_MOE_ERR_UNSUPPORTED
             : BEAM_MOE_OK;
}

// Workspace of the gated backward pass: both dz, the partial sums of the bias gradients, the inverse of an fp16
// dz's scale with the maxima that give it, the operands that are laid out anew, then the partial sums of the two
// products, in the same place unless they run in one launch.
struct GatedBackwardPlan {
  size_t off_part, off_scale, off_gate, off_up, off_x, off_gemm, total;
  bool copy_gate, copy_up, copy_x;
  beam::GemmPlan dx, dw;
};

constexpr size_t kScaleBytes = 256;  // before the maxima

GatedBackwardPlan gated_backward_plan(int32_t rows, int32_t cols, int32_t inner, int64_t ldx, int64_t ldg, int64_t ldu) {
  GatedBackwardPlan p;
  const int wide = 2 * beam::gated_half(cols);
  p.copy_gate = !beam::regular_rows(ldg, inner);
  p.copy_up = !beam::regular_rows(ldu, inner);
  p.copy_x = !beam::regular_rows(ldx, inner);
  beam::plan_gated_gradients(rows, cols, inner, &p.dx, &p.dw);
  p.off_part = align_up((size_t)rows * wide * 2);
  p.off_scale = p.off_part + align_up((size_t)beam::gated_dz_units(rows) * 2 * cols * sizeof(float));
  p.off_gate = p.off_scale + kScaleBytes + align_up(beam::gated_peak_bytes());
  p.off_up = p.off_gate + align_up(p.copy_gate ? beam::padded_bytes(cols, inner) : 0);
  p.off_x = p.off_up + align_up(p.copy_up ? beam::padded_bytes(cols, inner) : 0);
  p.off_gemm = p.off_x + align_up(p.copy_x ? beam::padded_bytes(rows, inner) : 0);
  p.total = p.off_gemm + (p.dx.paired ? p.dx.total + p.dw.total : std::max(p.dx.total, p.dw.total));
  return p;
}

}  // namespace

extern "C" {

size_t beam_moe_gated_linear_workspace_bytes(int32_t rows, int32_t cols, int32_t inner, int64_t ldx, int64_t ldg,
                                             int64_t ldu) {
  if (check_gated(rows, cols, inner) != BEAM_MOE_OK || !ld_ok(ldx, inner) || !ld_ok(ldg, inner) || !ld_ok(ldu, inner))
    return SIZE_MAX;
  return beam::plan_gated(rows, cols, inner, ldx, ldg, ldu).total;
}

int beam_moe_gated_linear(int32_t rows, int32_t cols, int32_t inner, int type, const void* x, int64_t ldx,
                          const void* w_gate, int64_t ldg, const void* w_up, int64_t ldu, const float* bias_gate,
                          const float* bias_up, int act, void* h, int h_type, int64_t ldh, void* pre_gate,
                          int64_t ldpg, void* pre_up, int64_t ldpu, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_gated(rows, cols, inner);
  if (rc != BEAM_MOE_OK) return rc;
  if (!half_type(type) || (h_type != type && h_type != BEAM_MOE_F32) || !act_ok(act)) return BEAM_MOE_ERR_INVALID_ARG;
  if (rows == 0) return BEAM_MOE_OK;
  if (!ld_ok(ldx, inner) || !ld_ok(ldg, inner) || !ld_ok(ldu, inner) || !ld_ok(ldh, cols) ||
      (pre_gate && !ld_ok(ldpg, cols)) || (pre_up && !ld_ok(ldpu, cols)))
    return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_ptrs({x, w_gate, w_up, h})) != BEAM_MOE_OK) return rc;
  if ((rc = check_optional({bias_gate, bias_up, pre_gate, pre_up})) != BEAM_MOE_OK) return rc;
  const beam::GatedPlan plan = beam::plan_gated(rows, cols, inner, ldx, ldg, ldu);
  if (plan.total && (!ws || !aligned16(ws) || ws_bytes < plan.total)) return BEAM_MOE_ERR_WORKSPACE;
  beam::GatedArgs g{};
  g.a = x;
  g.lda = ldx;
  g.b = w_gate;
  g.ldb = ldg;
  g.b2 = w_up;
  g.ldb2 = ldu;
  g.M = rows;
  g.N = cols;
  g.K = inner;
  g.type = type;
  g.bias = bias_gate;
  g.bias2 = bias_up;
  g.act = act;
  g.out = h;
  g.out_type = h_type;
  g.ldo = ldh;
  g.pre = pre_gate;
  g.ldp = ldpg;
  g.pre2 = pre_up;
  g.ldp2 = ldpu;
  return hip_status(beam::launch_gated(g, plan, ws, static_cast<hipStream_t>(stream)));
}

size_t beam_moe_gated_linear_backward_workspace_bytes(int32_t rows, int32_t cols, int32_t inner, int64_t ldx,
                                                      int64_t ldg, int64_t ldu) {
  if (check_gated(rows, cols, inner) != BEAM_MOE_OK || !ld_ok(ldx, inner) || !ld_ok(ldg, inner) || !ld_ok(ldu, inner))
    return SIZE_MAX;
  return gated_backward_plan(rows, cols, inner, ldx, ldg, ldu).total;
}

int beam_moe_gated_linear_backward(int32_t rows, int32_t cols, int32_t inner, int type, const void* dh, int dh_type,
                                   int64_t lddh, const void* x, int64_t ldx, const void* w_gate, int64_t ldg,
                                   const void* w_up, int64_t ldu, const void* pre_gate, int64_t ldpg,
                                   const void* pre_up, int64_t ldpu, int act, void* dx, int64_t lddx, void* dw_gate,
                                   int64_t lddwg, void* dw_up, int64_t lddwu, float* dbias_gate, float* dbias_up,
                                   void* ws, size_t ws_bytes, void* stream) {
  int rc = check_gated(rows, cols, inner);
  if (rc != BEAM_MOE_OK) return rc;
  if (!half_type(type) || (dh_type != type && dh_type != BEAM_MOE_F32) || !act_ok(act) || !dw_gate != !dw_up ||
      !dbias_gate != !dbias_up || (!dx && !dw_gate && !dbias_gate))
    return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_optional({x, w_gate, w_up, dx, dw_gate, dw_up, dbias_gate, dbias_up})) != BEAM_MOE_OK) return rc;
  if ((dx && !ld_ok(lddx, inner)) || (dw_gate && (!ld_ok(lddwg, inner) || !ld_ok(lddwu, inner))))
    return BEAM_MOE_ERR_INVALID_ARG;
  if (rows > 0) {
    if ((rc = check_ptrs({dh, pre_gate, pre_up})) != BEAM_MOE_OK) return rc;
    if ((dx && (!w_gate || !w_up)) || (dw_gate && !x) || !ld_ok(lddh, cols) || !ld_ok(ldpg, cols) ||
        !ld_ok(ldpu, cols) || (x && !ld_ok(ldx, inner)) || (w_gate && !ld_ok(ldg, inner)) || (w_up && !ld_ok(ldu, inner)))
      return BEAM_MOE_ERR_INVALID_ARG;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  const GatedBackwardPlan p =
      gated_backward_plan(rows, cols, inner, x ? ldx : inner, w_gate ? ldg : inner, w_up ? ldu : inner);
  if (rows > 0 && (!ws || !aligned16(ws) || ws_bytes < p.total)) return BEAM_MOE_ERR_WORKSPACE;
  const int half = beam::gated_half(cols), units = rows > 0 ? beam::gated_dz_units(rows) : 0;
  float* part = dbias_gate ? at<float>(ws, p.off_part) : nullptr;
  const bool products = dx || dw_gate, scaled = products && type == BEAM_MOE_F16 && rows > 0;
  float* unscale = scaled ? at<float>(ws, p.off_scale) : nullptr;
  uint16_t* dz = products ? at<uint16_t>(ws, 0) : nullptr;
  beam::PadJob jg{}, ju{}, jx{};
  auto copy = [&](beam::PadJob& j, const void*& m, int64_t& ld, int n, size_t off) {
    j = {m, ld, n, inner, at<void*>(ws, off)};
    m = j.dst;
    ld = beam::up8(inner);
  };
  if (rows > 0) {
    if (dx && p.copy_gate) copy(jg, w_gate, ldg, cols, p.off_gate);
    if (dx && p.copy_up) copy(ju, w_up, ldu, cols, p.off_up);
    if (dw_gate && p.copy_x) copy(jx, x, ldx, rows, p.off_x);
    const beam::GatedDz d{dh,   dh_type, lddh, pre_gate, pre_up, ldpg, ldpu, act, type,
                          at<uint32_t>(ws, p.off_scale + kScaleBytes), unscale, dz, part, rows, cols};
    if ((rc = hip_status(beam::launch_gated_dz(d, beam::pad_jobs(jg, ju, jx), st))) != BEAM_MOE_OK) return rc;
  }
  beam::GatedArgs gx{}, gw{};
  gx.type = gx.out_type = gw.type = gw.out_type = type;
  gx.add = gw.add = 1.f;
  gx.add_at = gw.add_at = unscale;
  gx.a = gw.a = dz;
  gx.lda = gw.lda = 2 * half;
  gx.half = gw.half = half;
  gx.valid = gw.valid = cols;
  gx.b = w_gate;
  gx.ldb = ldg;
  gx.b2 = w_up;
  gx.ldb2 = ldu;
  gx.bt = true;
  gx.M = rows;
  gx.N = inner;
  gx.K = 2 * half;
  gx.out = rows > 0 ? dx : nullptr;
  gx.ldo = lddx;
  gw.b = x;
  gw.ldb = ldx;
  gw.at = gw.bt = true;
  gw.M = 2 * half;
  gw.N = inner;
  gw.K = rows;
  gw.out = dw_gate;
  gw.ldo = lddwg;
  gw.out2 = dw_up;
  gw.ldo2 = lddwu;
  const beam::SumJob sums{part, dbias_gate, units, 2 * cols, dbias_up};
  if (gx.out)
    gx.sums = sums;
  else if (dbias_gate && (rc = hip_status(beam::launch_gated_sums(sums, st))) != BEAM_MOE_OK)
    return rc;
  return hip_status(beam::launch_gated_gradients(gx, p.dx, gw, p.dw, at<void>(ws, p.off_gemm), st));
}

size_t beam_moe_grad_norm_workspace_bytes(int32_t count) {
  if (count < 0 || count > kMaxGrads) return SIZE_MAX;
  return beam::grad_workspace(count);
}

int beam_moe_grad_norm(int32_t count, const void* const* grads, const int32_t* types, const int64_t* sizes, float scale,
                       float* norm, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_grads(count, grads, types, sizes);
  if (rc != BEAM_MOE_OK) return rc;
  if (!std::isfinite(scale)) return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_ptrs({norm})) != BEAM_MOE_OK) return rc;
  if (!ws || !aligned16(ws) || ws_bytes < beam_moe_grad_norm_workspace_bytes(count)) return BEAM_MOE_ERR_WORKSPACE;
  try {
    std::vector<beam::GradTensor> t;
    t.reserve(count);
    for (int32_t i = 0; i < count; ++i)
      if (sizes[i] > 0) t.push_back({grads[i], nullptr, sizes[i], 0u, (uint8_t)types[i], (uint8_t)types[i]});
    return hip_status(beam::launch_grad_norm(t.data(), (int)t.size(), scale, ws, norm, static_cast<hipStream_t>(stream)));
  } catch (const std::bad_alloc&) {
    return BEAM_MOE_ERR_UNSUPPORTED;
  }
}

int beam_moe_clip_grads(int32_t count, const void* const* grads, const int32_t* types, const int64_t* sizes, float scale,
                        float max_norm, float eps, const float* norm_in, void* const* outs, const int32_t* out_types,
                        float* norm, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_grads(count, grads, types, sizes);
  if (rc != BEAM_MOE_OK) return rc;
  if (!std::isfinite(scale) || !std::isfinite(max_norm) || max_norm < 0.f || !std::isfinite(eps) || !(eps > 0.f))
    return BEAM_MOE_ERR_INVALID_ARG;
  if (out_types && !outs) return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_optional({norm})) != BEAM_MOE_OK) return rc;
  if (reinterpret_cast<uintptr_t>(norm_in) % sizeof(float) != 0) return BEAM_MOE_ERR_INVALID_ARG;
  if (!ws || !aligned16(ws) || ws_bytes < beam_moe_grad_norm_workspace_bytes(count)) return BEAM_MOE_ERR_WORKSPACE;
  try {
    std::vector<beam::GradTensor> t;
    t.reserve(count);
    for (int32_t i = 0; i < count; ++i) {
      void* out = outs ? outs[i] : const_cast<void*>(grads[i]);
      const int type = out_types ? out_types[i] : types[i];
      if (!type_ok(type)) return BEAM_MOE_ERR_INVALID_ARG;
      if (sizes[i] == 0) continue;
      if (!out || reinterpret_cast<uintptr_t>(out) % elem_bytes(type) != 0) return BEAM_MOE_ERR_INVALID_ARG;
      t.push_back({grads[i], out, sizes[i], 0u, (uint8_t)types[i], (uint8_t)type});
    }
    if (!apart(t, norm_in, norm)) return BEAM_MOE_ERR_INVALID_ARG;
    const beam::ClipArgs a{scale, max_norm, eps, norm_in, norm};
    return hip_status(beam::launch_clip_grads(t.data(), (int)t.size(), a, ws, static_cast<hipStream_t>(stream)));
  } catch (const std::bad_alloc&) {
    return BEAM_MOE_ERR_UNSUPPORTED;
  }
}

int beam_moe_quantize_mxfp4(int32_t rows, int32_t cols, const void* x, int x_type, int64_t ldx, uint8_t* codes,
                            int64_t ldc, uint8_t* scales, int64_t lds, void* stream) {
  int rc = check_mx(rows, cols);
  if (rc != BEAM_MOE_OK) return rc;
  if (!type_ok(x_type)) return BEAM_MOE_ERR_INVALID_ARG;
  if (rows == 0) return BEAM_MOE_OK;
  if (!ld_ok(ldx, cols) || !mx_rows_ok(cols, ldc, lds)) return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_ptrs({x, codes, scales})) != BEAM_MOE_OK) return rc;
  return hip_status(beam::launch_quantize_mx(x, x_type, ldx, codes, ldc, scales, lds, rows, cols,
                                             static_cast<hipStream_t>(stream)));
}

int beam_moe_dequantize_mxfp4(int32_t rows, int32_t cols, const uint8_t* codes, int64_t ldc, const uint8_t* scales,
                              int64_t lds, void* y, int y_type, int64_t ldy, void* stream) {
  int rc = check_mx(rows, cols);
  if (rc != BEAM_MOE_OK) return rc;
  if (!type_ok(y_type)) return BEAM_MOE_ERR_INVALID_ARG;
  if (rows == 0) return BEAM_MOE_OK;
  if (!ld_ok(ldy, cols) || !mx_rows_ok(cols, ldc, lds)) return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_ptrs({codes, scales, y})) != BEAM_MOE_OK) return rc;
  return hip_status(beam::launch_dequantize_mx(codes, ldc, scales, lds, y, y_type, ldy, rows, cols,
                                               static_cast<hipStream_t>(stream)));
}

size_t beam_moe_linear_mxfp4_workspace_bytes(int32_t rows, int32_t cols, int32_t inner, int x_type, int64_t ldx,
                                             int64_t ldw) {
  const bool four = x_type == BEAM_MOE_MXFP4;
  if (check_mx_linear(rows, cols, inner) != BEAM_MOE_OK || !(four || half_type(x_type)) ||
      !ld_ok(ldx, four ? 16 * beam::mx_blocks(inner) : inner) || !ld_ok(ldw, 16 * beam::mx_blocks(inner)))
    return SIZE_MAX;
  return beam::plan_mx(rows, cols, inner, four, ldx, ldw).total;
}

int beam_moe_linear_mxfp4(int32_t rows, int32_t cols, int32_t inner, int x_type, const void* x, int64_t ldx,
                          const uint8_t* x_scales, int64_t ldxs, const uint8_t* w, int64_t ldw, const uint8_t* w_scales,
                          int64_t ldws, const float* bias, int act, const void* res, int64_t ldr, float keep, float add,
                          void* y, int y_type, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_mx_linear(rows, cols, inner);
  if (rc != BEAM_MOE_OK) return rc;
  const bool four = x_type == BEAM_MOE_MXFP4;
  if (!(four || half_type(x_type)) || !(four ? type_ok(y_type) : y_type == x_type || y_type == BEAM_MOE_F32) ||
      !act_ok(act) || !std::isfinite(keep) || !std::isfinite(add))
    return BEAM_MOE_ERR_INVALID_ARG;
  if (rows == 0) return BEAM_MOE_OK;
  if (!(four ? mx_rows_ok(inner, ldx, ldxs) : ld_ok(ldx, inner)) || !mx_rows_ok(inner, ldw, ldws) ||
      !ld_ok(ldy, cols) || (res && !ld_ok(ldr, cols)) || (res == y && ldr != ldy))
    return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_ptrs({x, w, w_scales, y})) != BEAM_MOE_OK) return rc;
  if (four && (rc = check_ptrs({x_scales})) != BEAM_MOE_OK) return rc;
  if ((rc = check_optional({bias, res})) != BEAM_MOE_OK) return rc;
  const beam::MxPlan plan = beam::plan_mx(rows, cols, inner, four, ldx, ldw);
  if (plan.total && (!ws || !aligned16(ws) || ws_bytes < plan.total)) return BEAM_MOE_ERR_WORKSPACE;
  beam::MxLinear a{};
  a.four = four;
  a.x = x;
  a.ldx = ldx;
  a.x_scales = x_scales;
  a.ldxs = ldxs;
  a.w = w;
  a.ldw = ldw;
  a.w_scales = w_scales;
  a.ldws = ldws;
  beam::GemmArgs& g = a.g;
  g.M = rows;
  g.N = cols;
  g.K = inner;
  g.type = !four ? x_type : y_type == BEAM_MOE_F16 ? BEAM_MOE_F16 : BEAM_MOE_BF16;
  g.bias = bias;
  g.act = act;
  g.res = res;
  g.ldr = ldr;
  g.keep = keep;
  g.add = add;
  g.out = y;
  g.out_type = y_type;
  g.ldo = ldy;
  return hip_status(beam::launch_linear_mx(a, plan, ws, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
