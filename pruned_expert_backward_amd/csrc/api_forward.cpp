// C-ABI entry points of the forward side: argument checks, then one launcher
// each.
#include "checks.h"
#include "forward.h"

using namespace lrmoe;

namespace {

// T tokens with K slots each: the pairs fit in 31 bits.
lrmoe_status check_slots(int64_t T, int32_t K) {
  if (K < 1 || K > LRMOE_MAX_TOPK) return LRMOE_ERR_INVALID;
  if (T < 0 || T >= kMaxRows || T * K >= kMaxRows) return LRMOE_ERR_SHAPE;
  return LRMOE_OK;
}

lrmoe_status check_gate(const lrmoe_gate* gt) {
  if (gt == nullptr) return LRMOE_ERR_NULL;
  if (gt->E < 1 || gt->E > LRMOE_MAX_GATE_EXPERTS) return LRMOE_ERR_INVALID;
  if (gt->score != LRMOE_GATE_SOFTMAX && gt->score != LRMOE_GATE_SIGMOID) return LRMOE_ERR_INVALID;
  LRMOE_TRY(check_dtype(gt->dtype));
  LRMOE_TRY(check_slots(gt->T, gt->K));
  return gt->K <= gt->E ? LRMOE_OK : LRMOE_ERR_INVALID;
}

}  // namespace

extern "C" {

lrmoe_status lrmoe_gate_topk(const lrmoe_gate* gt, const void* logits, const float* select_bias,
                             int32_t* ids, float* weights, void* stream) {
  LRMOE_TRY(check_gate(gt));
  LRMOE_TRY(need(logits, gt->T));
  LRMOE_TRY(optional(select_bias));
  LRMOE_TRY(need(ids, gt->T));
  LRMOE_TRY(need(weights, gt->T));
  if (select_bias != nullptr && gt->score != LRMOE_GATE_SIGMOID) return LRMOE_ERR_INVALID;
  return hip_status(launch_gate_topk(gt->dtype, gt->score, gt->renorm != 0, gt->scale, logits,
                                     select_bias, gt->T, gt->E, gt->K, ids, weights,
                                     stream_of(stream)));
}

lrmoe_status lrmoe_gate_topk_backward(const lrmoe_gate* gt, const void* logits, const int32_t* ids,
                                      const float* dweights, void* dlogits, void* stream) {
  LRMOE_TRY(check_gate(gt));
  LRMOE_TRY(need(logits, gt->T));
  LRMOE_TRY(need(ids, gt->T));
  LRMOE_TRY(need(dweights, gt->T));
  LRMOE_TRY(need(dlogits, gt->T));
  return hip_status(launch_gate_topk_backward(gt->dtype, gt->score, gt->renorm != 0, gt->scale,
                                              logits, ids, dweights, gt->T, gt->E, gt->K, dlogits,
                                              stream_of(stream)));
}

lrmoe_status lrmoe_route_sort_workspace(int64_t T, int32_t K, int32_t E, size_t* bytes_out) {
  if (bytes_out == nullptr) return LRMOE_ERR_NULL;
  LRMOE_TRY(check_experts(E));
  LRMOE_TRY(check_slots(T, K));
  *bytes_out = route_sort_workspace(T * K, E);
  return LRMOE_OK;
}

lrmoe_status lrmoe_route_sort(int64_t T, int32_t K, int32_t E, const int32_t* ids,
                              const float* weights, int64_t* counts, int32_t* seg_offsets,
                              int32_t* row_index, int32_t* pos, float* alpha, void* workspace,
                              size_t ws_bytes, void* stream) {
  LRMOE_TRY(check_experts(E));
  LRMOE_TRY(check_slots(T, K));
  LRMOE_TRY(need(ids, T));
  LRMOE_TRY(optional(weights));
  LRMOE_TRY(need(counts, E));
  LRMOE_TRY(need(seg_offsets, E + 1));
  LRMOE_TRY(need(row_index, T));
  LRMOE_TRY(need(pos, T));
  LRMOE_TRY(optional(alpha));
  if (alpha != nullptr && weights == nullptr && T > 0) return LRMOE_ERR_NULL;
  const size_t ws = route_sort_workspace(T * K, E);
  LRMOE_TRY(need(workspace, (int64_t)ws));
  if (ws_bytes < ws) return LRMOE_ERR_WORKSPACE;
  return hip_status(launch_route_sort(ids, weights, T, K, E, counts, seg_offsets, row_index, pos,
                                      alpha, static_cast<uint32_t*>(workspace),
                                      stream_of(stream)));
}

lrmoe_status lrmoe_dispatch(int32_t dtype, int64_t T, int32_t K, int32_t D, int64_t P,
                            const void* x, const int32_t* pos, void* xp, void* stream) {
  LRMOE_TRY(check_dtype(dtype));
  LRMOE_TRY(check_slots(T, K));
  LRMOE_TRY(check_width(dtype, D));
  if (P < 0 || P >= kMaxRows) return LRMOE_ERR_SHAPE;
  LRMOE_TRY(need(x, T));
  LRMOE_TRY(need(pos, T));
  LRMOE_TRY(need(xp, P));
  if (P == 0) return LRMOE_OK;
  return hip_status(launch_dispatch(dtype, x, pos, T, K, D, P, xp, stream_of(stream)));
}

lrmoe_status lrmoe_dispatch_backward(int32_t dtype, int32_t out_dtype, int64_t T, int32_t K,
                                     int32_t D, int64_t P, const void* dxp, const int32_t* pos,
                                     void* dx, void* stream) {
  LRMOE_TRY(check_dtype(dtype));
  LRMOE_TRY(check_dtype(out_dtype));
  LRMOE_TRY(check_slots(T, K));
  LRMOE_TRY(check_width(dtype, D));
  LRMOE_TRY(check_width(out_dtype, D));
  if (P < 0 || P >= kMaxRows) return LRMOE_ERR_SHAPE;
  LRMOE_TRY(need(dxp, P));
  LRMOE_TRY(need(pos, T));
  LRMOE_TRY(need(dx, T));
  return hip_status(launch_combine(dtype, out_dtype, dxp, pos, nullptr, nullptr, T, K, D, P, dx,
                                   stream_of(stream)));
}

lrmoe_status lrmoe_combine(int32_t dtype, int64_t T, int32_t K, int32_t D, int64_t P,
                           const void* yp, const int32_t* pos, const float* weights,
                           const void* residual, void* y, void* stream) {
  LRMOE_TRY(check_dtype(dtype));
  LRMOE_TRY(check_slots(T, K));
  LRMOE_TRY(check_width(dtype, D));
  if (P < 0 || P >= kMaxRows) return LRMOE_ERR_SHAPE;
  LRMOE_TRY(need(yp, P));
  LRMOE_TRY(need(pos, T));
  LRMOE_TRY(need(weights, T));
  LRMOE_TRY(optional(residual));
  LRMOE_TRY(need(y, T));
  return hip_status(launch_combine(dtype, dtype, yp, pos, weights, residual, T, K, D, P, y,
                                   stream_of(stream)));
}

lrmoe_status lrmoe_combine_backward(int32_t dtype, int64_t T, int32_t K, int32_t D, int64_t P,
                                    const void* dy, const void* yp, const int32_t* pos,
                                    const float* weights, void* dyp, float* dweights,
                                    void* stream) {
  LRMOE_TRY(check_dtype(dtype));
  LRMOE_TRY(check_slots(T, K));
  LRMOE_TRY(check_width(dtype, D));
  if (P < 0 || P >= kMaxRows) return LRMOE_ERR_SHAPE;
  LRMOE_TRY(need(dy, T));
  LRMOE_TRY(need(yp, P));
  LRMOE_TRY(need(pos, T));
  LRMOE_TRY(need(weights, T));
  LRMOE_TRY(need(dyp, P));
  LRMOE_TRY(need(dweights, T));
  return hip_status(launch_combine_backward(dtype, dy, yp, pos, weights, T, K, D, P, dyp, dweights,
                                            stream_of(stream)));
}

lrmoe_status lrmoe_grouped_forward(const lrmoe_forward* fw, const int32_t* seg_offsets,
                                   const int32_t* row_index, const void* x, const void* W,
                                   const void* bias, const void* residual, void* y, void* pre_a,
                                   void* pre_b, void* stream) {
  LRMOE_TRY(check_forward(fw));
  const bool glu = fw->act == LRMOE_ACT_SWIGLU;
  if (row_index == nullptr && fw->T != fw->P) return LRMOE_ERR_SHAPE;
  if (fw->P > 0 && fw->T == 0) return LRMOE_ERR_SHAPE;
  LRMOE_TRY(need(seg_offsets, fw->E + 1));
  LRMOE_TRY(optional(row_index));
  LRMOE_TRY(need(x, fw->P));
  LRMOE_TRY(need(W, fw->P));
  LRMOE_TRY(optional(bias));
  LRMOE_TRY(optional(residual));
  LRMOE_TRY(need(y, fw->P));
  LRMOE_TRY(optional(pre_a));
  LRMOE_TRY(optional(pre_b));
  if (fw->P > 0 && (glu ? (pre_a == nullptr) != (pre_b == nullptr) : pre_b != nullptr))
    return glu ? LRMOE_ERR_NULL : LRMOE_ERR_INVALID;
  const ForwardArgs a{seg_offsets, row_index, x,     W,     bias,      residual, y,      pre_a,
                      pre_b,       fw->P,     fw->T, fw->E, fw->d_out, fw->d_in, fw->act};
  return hip_status(launch_grouped_forward(fw->dtype, a, stream_of(stream)));
}

lrmoe_status lrmoe_act_backward_workspace(const lrmoe_forward* fw, size_t* bytes_out) {
  if (bytes_out == nullptr) return LRMOE_ERR_NULL;
  LRMOE_TRY(check_forward(fw));
  *bytes_out = act_backward_workspace(fw->P, fw->E, fw->d_out);
  return LRMOE_OK;
}

lrmoe_status lrmoe_act_backward(const lrmoe_forward* fw, int32_t dz_dtype,
                                const int32_t* seg_offsets, const void* dy, const void* pre_a,
                                const void* pre_b, void* dz, float* dbias, void* workspace,
                                size_t ws_bytes, void* stream) {
  LRMOE_TRY(check_forward(fw));
  LRMOE_TRY(check_dtype(dz_dtype));
  if (fw->dtype == LRMOE_F32 && dz_dtype != LRMOE_F32) return LRMOE_ERR_DTYPE;
  const bool glu = fw->act == LRMOE_ACT_SWIGLU;
  LRMOE_TRY(need(seg_offsets, fw->E + 1));
  LRMOE_TRY(need(dy, fw->P));
  if (fw->act != LRMOE_ACT_NONE) LRMOE_TRY(need(pre_a, fw->P));
  if (glu) LRMOE_TRY(need(pre_b, fw->P));
  LRMOE_TRY(need(dz, fw->P));
  LRMOE_TRY(optional(dbias));
  if (dbias != nullptr) {
    const size_t ws = act_backward_workspace(fw->P, fw->E, fw->d_out);
    LRMOE_TRY(need(workspace, (int64_t)ws));
    if (ws_bytes < ws) return LRMOE_ERR_WORKSPACE;
  }
  return hip_status(launch_act_backward(fw->dtype, dz_dtype, fw->act, seg_offsets, dy, pre_a, pre_b,
                                        fw->P, fw->E, glu ? fw->d_out / 2 : fw->d_out, dz, dbias,
                                        static_cast<float*>(workspace), stream_of(stream)));
}

}  // extern "C"
