// Host side of the training-step calls of include/mok.h around the layer: expert routing and the
// optimizer step. Checks arguments, then enqueues kernels on the caller's stream.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "mok_internal.h"

using namespace mok;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool is_elem(int e) { return e == MOK_ELEM_F32 || e == MOK_ELEM_BF16; }

mok_status check_route(const mok_route_desc* d) {
  if (!d) return MOK_ERR_NULL;
  if (!is_elem(d->elem)) return MOK_ERR_DTYPE;
  if (d->score != MOK_SCORE_SOFTMAX && d->score != MOK_SCORE_SIGMOID) return MOK_ERR_SHAPE;
  if (d->group_score != MOK_GROUP_MAX && d->group_score != MOK_GROUP_TOP2) return MOK_ERR_SHAPE;
  if (d->renorm != 0 && d->renorm != 1) return MOK_ERR_SHAPE;
  if (!std::isfinite(d->scale) || !(d->scale > 0.f)) return MOK_ERR_SHAPE;
  if (d->num_experts < 1 || d->num_experts > kMaxExperts) return MOK_ERR_SHAPE;
  if (d->num_groups < 1 || d->num_groups > 64 || d->num_experts % d->num_groups) return MOK_ERR_SHAPE;
  if (d->top_groups < 1 || d->top_groups > d->num_groups) return MOK_ERR_SHAPE;
  if (d->top_k < 1 || d->top_k > kMaxTopK ||
      d->top_k > d->top_groups * (d->num_experts / d->num_groups))
    return MOK_ERR_SHAPE;
  if (d->num_tokens < 0 || d->num_tokens > INT32_MAX) return MOK_ERR_SHAPE;
  if (d->logits_stride < d->num_experts || d->logits_stride > (int64_t(1) << 31)) return MOK_ERR_SHAPE;
  return MOK_OK;
}

mok_status hip_status(hipError_t e) { return e == hipSuccess ? MOK_OK : MOK_ERR_HIP; }

}  // namespace

extern "C" {

mok_status mok_route_fwd(const mok_route_desc* desc, const void* logits_dev, const float* bias_dev,
                         const uint8_t* token_mask_dev, int32_t* topk_idx_dev, float* topk_w_dev,
                         int32_t* load_dev, void* stream) {
  const mok_status st = check_route(desc);
  if (st != MOK_OK) return st;
  if (desc->num_tokens > 0 && (!logits_dev || !topk_idx_dev || !topk_w_dev)) return MOK_ERR_NULL;
  if (!aligned(logits_dev, desc->elem == MOK_ELEM_BF16 ? 2 : 4) || !aligned(bias_dev, 4) ||
      !aligned(topk_idx_dev, 4) || !aligned(topk_w_dev, 4) || !aligned(load_dev, 4))
    return MOK_ERR_ALIGN;
  return hip_status(launch_route_fwd(*desc, logits_dev, bias_dev, token_mask_dev, topk_idx_dev,
                                     topk_w_dev, load_dev, static_cast<hipStream_t>(stream)));
}

mok_status mok_route_bwd(const mok_route_desc* desc, const void* logits_dev,
                         const int32_t* topk_idx_dev, const float* dw_dev, void* dlogits_dev,
                         void* stream) {
  const mok_status st = check_route(desc);
  if (st != MOK_OK) return st;
  if (desc->num_tokens == 0) return MOK_OK;
  if (!logits_dev || !topk_idx_dev || !dw_dev || !dlogits_dev) return MOK_ERR_NULL;
  if (!aligned(logits_dev, desc->elem == MOK_ELEM_BF16 ? 2 : 4) || !aligned(topk_idx_dev, 4) ||
      !aligned(dw_dev, 4) || !aligned(dlogits_dev, 16))
    return MOK_ERR_ALIGN;
  return hip_status(launch_route_bwd(*desc, logits_dev, topk_idx_dev, dw_dev, dlogits_dev,
                                     static_cast<hipStream_t>(stream)));
}

mok_status mok_sumsq_ws_size(int32_t num_tensors, size_t* ws_bytes) {
  if (!ws_bytes) return MOK_ERR_NULL;
  if (num_tensors < 0) return MOK_ERR_SHAPE;
  *ws_bytes = size_t(sumsq_ws_bytes(num_tensors));
  return MOK_OK;
}

mok_status mok_grad_sumsq(int32_t num_tensors, const mok_sumsq_tensor* tensors, int32_t elem,
                          double* out_dev, void* ws_dev, void* stream) {
  if (num_tensors < 0) return MOK_ERR_SHAPE;
  if (!is_elem(elem)) return MOK_ERR_DTYPE;
  if ((num_tensors > 0 && !tensors) || !out_dev || !ws_dev) return MOK_ERR_NULL;
  if (!aligned(out_dev, 8) || !aligned(ws_dev, 8)) return MOK_ERR_ALIGN;
  for (int32_t t = 0; t < num_tensors; ++t) {
    if (tensors[t].n < 0 || tensors[t].n > kMaxOptElements) return MOK_ERR_SHAPE;
    if (tensors[t].n > 0 && !tensors[t].g) return MOK_ERR_NULL;
    if (!aligned(tensors[t].g, 16)) return MOK_ERR_ALIGN;
  }
  return hip_status(launch_sumsq(num_tensors, tensors, elem == MOK_ELEM_BF16, out_dev,
                                 static_cast<uint8_t*>(ws_dev), static_cast<hipStream_t>(stream)));
}

mok_status mok_adamw(int32_t num_tensors, const mok_adamw_tensor* tensors,
                     const mok_adamw_config* config, void* stream) {
  if (!config) return MOK_ERR_NULL;
  if (num_tensors < 0) return MOK_ERR_SHAPE;
  if (num_tensors > 0 && !tensors) return MOK_ERR_NULL;
  const mok_adamw_config& c = *config;
  if (!is_elem(c.grad_elem) || !is_elem(c.param_elem) ||
      (c.state != MOK_STATE_F32 && c.state != MOK_STATE_MX8))
    return MOK_ERR_DTYPE;
  // (written so that NaN fails)
  if (!(c.lr >= 0 && std::isfinite(c.lr)) || !(c.weight_decay >= 0 && std::isfinite(c.weight_decay)) ||
      !(c.beta1 >= 0 && c.beta1 < 1) || !(c.beta2 >= 0 && c.beta2 < 1) ||
      !(float(c.eps) > 0.f && std::isfinite(float(c.eps))) || c.step < 1)
    return MOK_ERR_SHAPE;
  if (c.sumsq_dev && !(c.max_norm > 0)) return MOK_ERR_SHAPE;
  if (!aligned(c.sumsq_dev, 8) || !aligned(c.lr_dev, 8) || !aligned(c.step_dev, 8)) return MOK_ERR_ALIGN;
  const bool mx = c.state == MOK_STATE_MX8;
  for (int32_t k = 0; k < num_tensors; ++k) {
    const mok_adamw_tensor& t = tensors[k];
    if (t.n < 0 || t.n > kMaxOptElements) return MOK_ERR_SHAPE;
    if (t.copy && c.param_elem != MOK_ELEM_F32) return MOK_ERR_DTYPE;
    if (t.n == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v || (mx && (!t.m_scale || !t.v_scale))) return MOK_ERR_NULL;
    if (!aligned(t.p, 16) || !aligned(t.copy, 16) || !aligned(t.g, 16) || !aligned(t.m, 16) ||
        !aligned(t.v, 16))
      return MOK_ERR_ALIGN;
  }
  return hip_status(launch_adamw(num_tensors, tensors, c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
