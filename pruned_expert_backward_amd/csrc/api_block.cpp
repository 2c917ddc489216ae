// C-ABI entry points around the expert products: 8-bit blocks and their product,
// the norms around a block, the optimizer's step.  Argument checks, then one launcher
// each.
#include "checks.h"
#include "forward.h"

using namespace lrmoe;

namespace {

constexpr int64_t kMaxElements = int64_t(1) << 36;   // of a tensor of the optimizer's step

lrmoe_status check_rows(int64_t T) { return T < 0 || T >= kMaxRows ? LRMOE_ERR_SHAPE : LRMOE_OK; }

// A row length in 8 bits: whole 16-byte pieces.
lrmoe_status check_fp8_width(int64_t d) {
  if (d < 1 || d > (1 << 20)) return LRMOE_ERR_SHAPE;
  return d % 16 == 0 ? LRMOE_OK : LRMOE_ERR_ALIGN;
}

lrmoe_status check_norm(const lrmoe_norm* nm) {
  if (nm == nullptr) return LRMOE_ERR_NULL;
  LRMOE_TRY(check_dtype(nm->dtype));
  LRMOE_TRY(check_rows(nm->T));
  if (nm->D > LRMOE_MAX_NORM_WIDTH) return LRMOE_ERR_SHAPE;
  LRMOE_TRY(check_width(nm->dtype, nm->D));
  if (nm->gate < LRMOE_BRANCH_GATE_NONE || nm->gate > LRMOE_BRANCH_GATE_TOKEN)
    return LRMOE_ERR_INVALID;
  return nm->eps >= 0.f ? LRMOE_OK : LRMOE_ERR_INVALID;
}

// What goes with a branch.  Without rows a NULL y says nothing.
lrmoe_status check_branch(const lrmoe_norm* nm, const void* y, const void* branch_weight,
                          const void* gate) {
  LRMOE_TRY(optional(y));
  LRMOE_TRY(optional(branch_weight));
  LRMOE_TRY(optional(gate));
  if (nm->gate == LRMOE_BRANCH_GATE_NONE ? gate != nullptr
                                         : gate == nullptr && (nm->T > 0 || nm->gate == LRMOE_BRANCH_GATE_CHANNEL))
    return nm->gate == LRMOE_BRANCH_GATE_NONE ? LRMOE_ERR_INVALID : LRMOE_ERR_NULL;
  if (nm->T > 0 && y == nullptr &&
      (branch_weight != nullptr || gate != nullptr || nm->scale != 1.f))
    return LRMOE_ERR_INVALID;
  return LRMOE_OK;
}

NormArgs norm_args(const lrmoe_norm* nm, const void* x, const void* y, const void* branch_weight,
                   const void* gate, const void* weight) {
  return NormArgs{x,     y,        branch_weight, gate,    weight,
                  nm->T, nm->D, nm->gate,      nm->scale, nm->eps};
}

bool misaligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0;
}

}  // namespace

extern "C" {

lrmoe_status lrmoe_quantize_rows(int32_t dtype, int64_t T, int32_t D, const void* x, uint8_t* q,
                                uint8_t* scale, void* stream) {
  LRMOE_TRY(check_dtype(dtype));
  LRMOE_TRY(check_rows(T));
  LRMOE_TRY(check_fp8_width(D));
  LRMOE_TRY(need(x, T));
  LRMOE_TRY(need(q, T));
  LRMOE_TRY(need(scale, T));
  return hip_status(launch_fp8_quantize(dtype, x, T, D, q, scale, stream_of(stream)));
}

lrmoe_status lrmoe_quantize_weights(int32_t dtype, int32_t E, int32_t d_out, int32_t d_in,
                                        const void* W, uint8_t* q, uint8_t* scale, uint8_t* qt,
                                        uint8_t* scale_t, void* stream) {
  LRMOE_TRY(check_dtype(dtype));
  LRMOE_TRY(check_experts(E));
  LRMOE_TRY(check_fp8_width(d_in));
  LRMOE_TRY(check_width(LRMOE_BF16, d_out));
  if (qt != nullptr) LRMOE_TRY(check_fp8_width(d_out));
  LRMOE_TRY(need(W, 1));
  LRMOE_TRY(need(q, 1));
  LRMOE_TRY(need(scale, 1));
  LRMOE_TRY(optional(qt));
  LRMOE_TRY(optional(scale_t));
  if ((qt == nullptr) != (scale_t == nullptr)) return LRMOE_ERR_NULL;
  return hip_status(launch_fp8_quantize_weights(dtype, W, E, d_out, d_in, q, scale, qt, scale_t,
                                                stream_of(stream)));
}

lrmoe_status lrmoe_grouped_forward_quantized(const lrmoe_forward* fw, const int32_t* seg_offsets,
                                       const int32_t* row_index, const uint8_t* xq,
                                       const uint8_t* x_scale, const uint8_t* Wq,
                                       const uint8_t* W_scale, const void* bias,
                                       const void* residual, void* y, void* pre_a, void* pre_b,
                                       void* stream) {
  LRMOE_TRY(check_forward(fw));
  if (fw->dtype != LRMOE_BF16) return LRMOE_ERR_DTYPE;
  LRMOE_TRY(check_fp8_width(fw->d_in));
  const bool glu = fw->act == LRMOE_ACT_SWIGLU;
  if (row_index == nullptr && fw->T != fw->P) return LRMOE_ERR_SHAPE;
  if (fw->P > 0 && fw->T == 0) return LRMOE_ERR_SHAPE;
  LRMOE_TRY(need(seg_offsets, fw->E + 1));
  LRMOE_TRY(optional(row_index));
  LRMOE_TRY(need(xq, fw->P));
  LRMOE_TRY(need(x_scale, fw->P));
  LRMOE_TRY(need(Wq, fw->P));
  LRMOE_TRY(need(W_scale, fw->P));
  LRMOE_TRY(optional(bias));
  LRMOE_TRY(optional(residual));
  LRMOE_TRY(need(y, fw->P));
  LRMOE_TRY(optional(pre_a));
  LRMOE_TRY(optional(pre_b));
  if (fw->P > 0 && (glu ? (pre_a == nullptr) != (pre_b == nullptr) : pre_b != nullptr))
    return glu ? LRMOE_ERR_NULL : LRMOE_ERR_INVALID;
  const ForwardArgs a{seg_offsets, row_index, xq,    Wq,    bias,      residual, y,      pre_a,
                      pre_b,       fw->P,     fw->T, fw->E, fw->d_out, fw->d_in, fw->act};
  return hip_status(launch_grouped_forward_fp8(a, x_scale, W_scale, stream_of(stream)));
}

lrmoe_status lrmoe_residual_norm(const lrmoe_norm* nm, const void* x, const void* y,
                                 const void* branch_weight, const void* gate, const void* weight,
                                 void* s, void* h, void* stream) {
  LRMOE_TRY(check_norm(nm));
  LRMOE_TRY(need(x, nm->T));
  LRMOE_TRY(check_branch(nm, y, branch_weight, gate));
  LRMOE_TRY(optional(weight));
  LRMOE_TRY(optional(s));
  LRMOE_TRY(optional(h));
  if (nm->T == 0) return LRMOE_OK;
  if (y == nullptr && s != nullptr) return LRMOE_ERR_INVALID;
  if (y != nullptr && s == nullptr) return LRMOE_ERR_NULL;
  if ((weight == nullptr) != (h == nullptr)) return LRMOE_ERR_NULL;
  if (y == nullptr && weight == nullptr) return LRMOE_ERR_NULL;   // nothing to do
  return hip_status(launch_residual_norm(nm->dtype,
                                         norm_args(nm, x, y, branch_weight, gate, weight), s, h,
                                         stream_of(stream)));
}

lrmoe_status lrmoe_residual_norm_backward_workspace(const lrmoe_norm* nm, size_t* bytes_out) {
  if (bytes_out == nullptr) return LRMOE_ERR_NULL;
  LRMOE_TRY(check_norm(nm));
  *bytes_out = residual_norm_workspace(nm->T, nm->D);
  return LRMOE_OK;
}

lrmoe_status lrmoe_residual_norm_backward(const lrmoe_norm* nm, const void* ds, const void* dh,
                                          const void* s, const void* y, const void* branch_weight,
                                          const void* gate, const void* weight, void* dx, void* dy,
                                          float* dweight, float* dbranch_weight, float* dgate,
                                          void* workspace, size_t ws_bytes, void* stream) {
  LRMOE_TRY(check_norm(nm));
  LRMOE_TRY(check_branch(nm, y, branch_weight, gate));
  LRMOE_TRY(optional(ds));
  LRMOE_TRY(optional(dh));
  LRMOE_TRY(optional(weight));
  if (weight != nullptr) LRMOE_TRY(need(s, nm->T));
  LRMOE_TRY(need(dx, nm->T));
  LRMOE_TRY(optional(dy));
  LRMOE_TRY(optional(dweight));
  LRMOE_TRY(optional(dbranch_weight));
  LRMOE_TRY(optional(dgate));
  if (nm->T > 0) {
    if ((weight == nullptr) != (dh == nullptr)) return LRMOE_ERR_NULL;
    if (weight == nullptr && ds == nullptr) return LRMOE_ERR_NULL;
    if ((y == nullptr) != (dy == nullptr)) return LRMOE_ERR_NULL;
  }
  if ((dweight != nullptr && weight == nullptr) ||
      (dbranch_weight != nullptr && branch_weight == nullptr) ||
      (dgate != nullptr && nm->gate == LRMOE_BRANCH_GATE_NONE))
    return LRMOE_ERR_INVALID;
  if (dweight != nullptr || dbranch_weight != nullptr ||
      (dgate != nullptr && nm->gate == LRMOE_BRANCH_GATE_CHANNEL)) {
    const size_t ws = residual_norm_workspace(nm->T, nm->D);
    LRMOE_TRY(need(workspace, (int64_t)ws));
    if (ws_bytes < ws) return LRMOE_ERR_WORKSPACE;
  }
  return hip_status(launch_residual_norm_backward(
      nm->dtype, norm_args(nm, s, y, branch_weight, gate, weight), ds, dh, dx, dy, dweight,
      dbranch_weight, dgate, static_cast<float*>(workspace), stream_of(stream)));
}

lrmoe_status lrmoe_adamw_step(const lrmoe_adamw* cfg, const lrmoe_adamw_tensor* tensors,
                              int32_t count, void* stream) {
  if (cfg == nullptr || (count > 0 && tensors == nullptr)) return LRMOE_ERR_NULL;
  if (count < 0) return LRMOE_ERR_INVALID;
  const bool unit = cfg->beta1 >= 0 && cfg->beta1 < 1 && cfg->beta2 >= 0 && cfg->beta2 < 1;
  if (!unit || !(cfg->lr >= 0) || !(cfg->eps >= 0) || !(cfg->weight_decay >= 0))
    return LRMOE_ERR_INVALID;
  if (cfg->step_at == nullptr && cfg->step < 1) return LRMOE_ERR_INVALID;
  if (misaligned(cfg->lr_at, 4) || misaligned(cfg->step_at, 8) || misaligned(cfg->grad_scale, 4) ||
      misaligned(cfg->skip, 4))
    return LRMOE_ERR_ALIGN;
  for (int32_t k = 0; k < count; ++k) {
    const lrmoe_adamw_tensor& t = tensors[k];
    if (t.n < 0 || t.n >= kMaxElements) return LRMOE_ERR_SHAPE;
    LRMOE_TRY(check_dtype(t.p_dtype));
    LRMOE_TRY(check_dtype(t.g_dtype));
    LRMOE_TRY(need(t.p, t.n));
    LRMOE_TRY(need(t.g, t.n));
    LRMOE_TRY(need(t.m, t.n));
    LRMOE_TRY(need(t.v, t.n));
    LRMOE_TRY(optional(t.m_scale));
    LRMOE_TRY(optional(t.v_scale));
    LRMOE_TRY(optional(t.copy));
    if ((t.m_scale == nullptr) != (t.v_scale == nullptr)) return LRMOE_ERR_NULL;
    if (t.copy != nullptr && t.p_dtype != LRMOE_F32) return LRMOE_ERR_DTYPE;
  }
  return hip_status(launch_adamw(cfg, tensors, count, stream_of(stream)));
}

}  // extern "C"
