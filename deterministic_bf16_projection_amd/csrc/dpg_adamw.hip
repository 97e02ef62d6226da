// C ABI of the AdamW step: validation and launches.  Conventions are in
// include/dpg.h, the kernel in adamw_kernel.h.
#include <hip/hip_runtime.h>
#include <math.h>

#include "adamw_kernel.h"
#include "api_common.h"

namespace dpg {
namespace {

// workgroups of one launch: below 2^32 threads
constexpr int64_t kMaxChunks = 1 << 23;
// Calls of up to so many elements give a wave one block of 256 instead of four:
// 1.8 million elements with 8-bit moments 12.8 -> 9.4 us, 4 million 20.3 -> 18.0;
// with 32-bit moments 1.5 million 10.9 -> 9.8, but 4 million 19.7 -> 20.5.
constexpr int64_t kFewElements[2] = {2 << 20, 4 << 20};  // 32-bit, 8-bit moments

bool aligned_to(const void* p, unsigned bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

dpg_status check_adamw(const dpg_adamw_tensor& t, int grad_dtype, bool e4m3) {
  if (t.numel < 0) return DPG_ERR_INVALID_ARG;
  if (t.numel == 0) return DPG_OK;
  if (t.numel > kMaxChunks * adamw_chunk(kAdamwSteps)) return DPG_ERR_UNSUPPORTED;
  if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return DPG_ERR_INVALID_ARG;
  if (e4m3 && (!t.avg_scale || !t.sq_scale)) return DPG_ERR_INVALID_ARG;
  if (!aligned_to(t.param, 4) || !aligned_to(t.grad, grad_dtype == DPG_F32 ? 4 : 2) || !aligned_to(t.copy, 2))
    return DPG_ERR_ALIGNMENT;
  if (e4m3 ? !aligned_to(t.avg_scale, 4) || !aligned_to(t.sq_scale, 4)
           : !aligned_to(t.exp_avg, 4) || !aligned_to(t.exp_avg_sq, 4))
    return DPG_ERR_ALIGNMENT;
  return DPG_OK;
}

template <int STEPS>
const void* adamw_fn(bool bf16, bool e4m3) {
  if (bf16) return e4m3 ? (const void*)&adamw_kernel<2, true, STEPS> : (const void*)&adamw_kernel<2, false, STEPS>;
  return e4m3 ? (const void*)&adamw_kernel<4, true, STEPS> : (const void*)&adamw_kernel<4, false, STEPS>;
}

}  // namespace
}  // namespace dpg

using namespace dpg;

extern "C" dpg_status dpg_adamw(const dpg_adamw_tensor* tensors, int64_t count, const dpg_adamw_options* o,
                                hipStream_t stream) {
  if (count < 0 || !o || (count > 0 && !tensors)) return DPG_ERR_INVALID_ARG;
  if (o->grad_dtype != DPG_BF16 && o->grad_dtype != DPG_F32) return DPG_ERR_INVALID_ARG;
  if (o->state_dtype != DPG_F32 && o->state_dtype != DPG_E4M3) return DPG_ERR_INVALID_ARG;
  if (!(o->lr >= 0) || !(o->eps >= 0) || !(o->weight_decay >= 0) || !isfinite(o->lr) || !isfinite(o->eps) ||
      !isfinite(o->weight_decay) || !(o->beta1 >= 0 && o->beta1 < 1) || !(o->beta2 >= 0 && o->beta2 < 1) ||
      o->step < 1)
    return DPG_ERR_INVALID_ARG;
  if (!aligned_to(o->grad_scale, 4)) return DPG_ERR_ALIGNMENT;
  const bool e4m3 = o->state_dtype == DPG_E4M3;
  for (int64_t i = 0; i < count; ++i) {
    const dpg_status st = check_adamw(tensors[i], o->grad_dtype, e4m3);
    if (st != DPG_OK) return st;
  }
  AdamwParams p{};
  p.beta1 = (float)o->beta1;
  p.rest1 = (float)(1 - o->beta1);
  p.beta2 = (float)o->beta2;
  p.rest2 = (float)(1 - o->beta2);
  p.decay = (float)(1 - o->lr * o->weight_decay);
  p.rate = (float)(o->lr / (1 - pow(o->beta1, (double)o->step)));
  p.root_scale = (float)(1 / sqrt(1 - pow(o->beta2, (double)o->step)));
  p.eps = (float)o->eps;
  p.grad_scale = o->grad_scale;
  int64_t elements = 0;
  for (int64_t i = 0; i < count; ++i) elements += tensors[i].numel;
  const bool few = elements <= kFewElements[e4m3];
  const int chunk = adamw_chunk(few ? 1 : kAdamwSteps);
  const bool bf16 = o->grad_dtype == DPG_BF16;
  const void* fn = few ? adamw_fn<1>(bf16, e4m3) : adamw_fn<kAdamwSteps>(bf16, e4m3);
  void* args[] = {&p};
  int64_t chunks = 0;
  for (int64_t i = 0; i <= count; ++i) {
    const int64_t more = i < count ? (tensors[i].numel + chunk - 1) / chunk : 0;
    if (p.count > 0 && (i == count || p.count == kAdamwTensors || chunks + more > kMaxChunks)) {
      const dpg_status st = launch(fn, chunks, 256, 0, args, stream);
      if (st != DPG_OK) return st;
      p.count = 0;
      chunks = 0;
    }
    if (more == 0) continue;
    const dpg_adamw_tensor& t = tensors[i];
    p.t[p.count] = AdamwTensor{t.param,     t.grad,     t.exp_avg,               t.exp_avg_sq,
                               t.avg_scale, t.sq_scale, (unsigned short*)t.copy, t.numel};
    p.chunk0[p.count] = (int)chunks;
    p.key[p.count] = adamw_mix(o->seed + (unsigned)(i + 1) * kAdamwStride);
    ++p.count;
    chunks += more;
  }
  return DPG_OK;
}
