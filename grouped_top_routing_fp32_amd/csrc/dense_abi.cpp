// C ABI of the operators of a dense gated sublayer, trained and served (the norm of all gradients and their
// clipping, microscaled 4-bit floating point): argument validation, workspace carving and
// kernel launches on the caller's stream.  The operations and conventions are stated in include/beam_moe.h.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "abi_util.h"
#include "grads.h"
#include "mxfp4.h"

namespace {

using beam::aligned16;
using beam::check_optional;
using beam::check_ptrs;
using beam::hip_status;
using beam::ld_ok;
using beam::type_ok;

constexpr int32_t kMaxGrads = 1 << 16;
constexpr int64_t kMaxGradSize = int64_t(1) << 40;
constexpr int64_t kMaxGradTotal = int64_t(1) << 44;  // chunks fit 32 bits
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

// Whether every output lies apart from the other outputs and from the other gradients.
bool apart(const std::vector<beam::GradTensor>& t) {
  struct Span {
    uintptr_t a, b;
    int64_t of;  // a gradient's index, or ~ an output's
  };
  std::vector<Span> spans;
  spans.reserve(2 * t.size());
  for (size_t i = 0; i < t.size(); ++i) {
    if (t[i].n == 0) continue;
    const uintptr_t p = reinterpret_cast<uintptr_t>(t[i].p), o = reinterpret_cast<uintptr_t>(t[i].out);
    spans.push_back({o, o + t[i].n * elem_bytes(t[i].out_type), ~(int64_t)i});
    if (p != o || t[i].type != t[i].out_type) spans.push_back({p, p + t[i].n * elem_bytes(t[i].type), (int64_t)i});
  }
  std::sort(spans.begin(), spans.end(), [](const Span& x, const Span& y) { return x.a < y.a; });
  uintptr_t out_end = 0, grad_end = 0;  // of what lies before
  for (const Span& s : spans) {
    if (s.a < out_end || (s.of < 0 && s.a < grad_end)) return false;
    uintptr_t& end = s.of < 0 ? out_end : grad_end;
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

}  // namespace

extern "C" {

size_t beam_moe_grad_norm_workspace_bytes(int32_t count) {
  if (count < 0 || count > kMaxGrads) return SIZE_MAX;
  return beam::grad_partials(count) * sizeof(double);
}

int beam_moe_grad_norm(int32_t count, const void* const* grads, const int32_t* types, const int64_t* sizes, float scale,
                       float* norm, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_grads(count, grads, types, sizes);
  if (rc != BEAM_MOE_OK) return rc;
  if (!std::isfinite(scale)) return BEAM_MOE_ERR_INVALID_ARG;
  if ((rc = check_ptrs({norm})) != BEAM_MOE_OK) return rc;
  if (!ws || !aligned16(ws) || ws_bytes < beam_moe_grad_norm_workspace_bytes(count)) return BEAM_MOE_ERR_WORKSPACE;
  try {
    std::vector<beam::GradTensor> t(count);
    for (int32_t i = 0; i < count; ++i) t[i] = {grads[i], nullptr, sizes[i], types[i], types[i]};
    return hip_status(beam::launch_grad_norm(t.data(), count, scale, static_cast<double*>(ws), norm,
                                             static_cast<hipStream_t>(stream)));
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
  if ((rc = check_optional({norm_in, norm})) != BEAM_MOE_OK) return rc;
  if (!norm_in && (!ws || !aligned16(ws) || ws_bytes < beam_moe_grad_norm_workspace_bytes(count)))
    return BEAM_MOE_ERR_WORKSPACE;
  try {
    std::vector<beam::GradTensor> t(count);
    for (int32_t i = 0; i < count; ++i) {
      t[i] = {grads[i], outs ? outs[i] : const_cast<void*>(grads[i]), sizes[i], types[i],
              out_types ? out_types[i] : types[i]};
      if (!type_ok(t[i].out_type)) return BEAM_MOE_ERR_INVALID_ARG;
      if (t[i].n > 0 && (!t[i].out || reinterpret_cast<uintptr_t>(t[i].out) % elem_bytes(t[i].out_type) != 0))
        return BEAM_MOE_ERR_INVALID_ARG;
    }
    if (!apart(t)) return BEAM_MOE_ERR_INVALID_ARG;
    const beam::ClipArgs a{scale, max_norm, eps, norm_in, norm};
    return hip_status(beam::launch_clip_grads(t.data(), count, a, static_cast<double*>(ws),
                                              static_cast<hipStream_t>(stream)));
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

}  // extern "C"
