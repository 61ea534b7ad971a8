// capi_train.cu - C-ABI of the training operators (include/moe.h): argument
// validation, then the launch. No device memory is allocated, and only constants of
// a device (its kernels' attributes) are kept.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"

using namespace sgl;

namespace {

// The calls launch with programmatic stream serialization: their kernels wait
// for the kernel before them at once and never release the next one early, so
// only the launch latency overlaps (2 us of a 30 us SwiGLU).
constexpr int kMaxRows = 1 << 25;
constexpr int kMaxFeatures = 16384;

bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
moe_status cu(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
bool features_ok(int v) { return v >= 8 && v <= kMaxFeatures && v % 8 == 0; }
bool stride_ok(int ld, int width) { return ld >= width && ld % 8 == 0; }

bool linear_ok(const moe_linear_desc* d) {
  if (d == nullptr) return false;
  if (d->E < 1 || d->E > kMaxExpertsCfg || d->R < 0 || d->R > kMaxRows) return false;
  if (!features_ok(d->N) || !features_ok(d->K)) return false;
  if (!stride_ok(d->ld_x, d->K) || !stride_ok(d->ld_y, d->N)) return false;
  if (d->out_type != MOE_T_BF16 && d->out_type != MOE_T_F32) return false;
  if (d->accumulate && d->out_type != MOE_T_F32) return false;
  return true;
}

bool swiglu_ok(const moe_swiglu_desc* d, bool backward) {
  if (d == nullptr || d->R < 0 || d->R > kMaxRows || !features_ok(d->I)) return false;
  if (!stride_ok(d->ld_g, d->I) || !stride_ok(d->ld_h, d->I)) return false;
  if (backward && !stride_ok(d->ld_dg, d->I)) return false;
  return !isnan(d->limit);
}

moe_status grouped(const moe_linear_desc* d, LinearDir dir, const void* a, const void* b,
                   const int32_t* offsets, void* out, void* ws, size_t ws_bytes, void* stream) {
  PdlScope pdl_scope(0);  // programmatic dependent launch
  if (!linear_ok(d)) return MOE_ERR_CFG;
  // row-wise tensors without rows may have no address: a, and out or (wgrad) b
  const bool rows = d->R > 0, wg = dir == kWgrad;
  if (!offsets || (rows && !a) || ((rows || !wg) && !b) || ((rows || wg) && !out))
    return MOE_ERR_NULL;
  if (!al16(a) || !al16(b) || !al16(offsets) || !al16(out)) return MOE_ERR_ALIGN;
  if (ws == nullptr || ws_bytes < moe_linear_workspace_size(d) || !al16(ws))
    return MOE_ERR_WORKSPACE;
  const moe_status st = device_ok();
  if (st != MOE_OK) return st;
  if (d->R == 0 && dir != kWgrad) return MOE_OK;
  return cu(launch_grouped_linear(*d, dir, a, b, offsets, out, static_cast<int32_t*>(ws),
                                  static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_size(const moe_linear_desc* desc) {
  return linear_ok(desc) ? kCtrlBytes : 0;
}

moe_status moe_grouped_linear(const moe_linear_desc* desc, const void* x, const int32_t* offsets,
                              const void* W, void* y, void* ws, size_t ws_bytes, void* stream) {
  return grouped(desc, kFwd, x, W, offsets, y, ws, ws_bytes, stream);
}

moe_status moe_grouped_linear_dgrad(const moe_linear_desc* desc, const void* dy,
                                    const int32_t* offsets, const void* W, void* dx, void* ws,
                                    size_t ws_bytes, void* stream) {
  return grouped(desc, kDgrad, dy, W, offsets, dx, ws, ws_bytes, stream);
}

moe_status moe_grouped_linear_wgrad(const moe_linear_desc* desc, const void* dy, const void* x,
                                    const int32_t* offsets, void* dW, void* ws, size_t ws_bytes,
                                    void* stream) {
  return grouped(desc, kWgrad, dy, x, offsets, dW, ws, ws_bytes, stream);
}

moe_status moe_linear_read_error(void* ws, size_t ws_bytes, void* stream, int32_t* code) {
  if (!code) return MOE_ERR_NULL;
  if (ws == nullptr || ws_bytes < kCtrlBytes) return MOE_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, ws, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return MOE_ERR_CUDA;
  if (cudaMemsetAsync(ws, 0, 4, s) != cudaSuccess) return MOE_ERR_CUDA;
  *code = v;
  return MOE_OK;
}

moe_status moe_swiglu(const moe_swiglu_desc* desc, const void* g, const void* u, const float* w,
                      const int32_t* perm, int32_t n_w, const int32_t* rows, void* h,
                      void* stream) {
  PdlScope pdl_scope(0);
  if (!swiglu_ok(desc, false)) return MOE_ERR_CFG;
  if (w != nullptr && perm != nullptr && n_w < 0) return MOE_ERR_CFG;
  if (desc->R > 0 && (!g || !u || !h)) return MOE_ERR_NULL;
  if (!al16(g) || !al16(u) || !al16(h) || !al16(w) || !al16(perm) || !al4(rows))
    return MOE_ERR_ALIGN;
  const moe_status st = device_ok();
  if (st != MOE_OK) return st;
  if (desc->R == 0) return MOE_OK;
  return cu(launch_swiglu(*desc, g, u, w, perm, n_w, rows, h, static_cast<cudaStream_t>(stream)));
}

moe_status moe_swiglu_backward(const moe_swiglu_desc* desc, const void* dh, const void* g,
                               const void* u, const float* w, const int32_t* perm, int32_t n_w,
                               const int32_t* rows, void* dg, void* du, float* dw, void* stream) {
  PdlScope pdl_scope(0);
  if (!swiglu_ok(desc, true)) return MOE_ERR_CFG;
  if (w != nullptr && perm != nullptr && n_w < 0) return MOE_ERR_CFG;
  if (dw && !w) return MOE_ERR_NULL;
  if (desc->R > 0 && (!dh || !g || !u || !dg || !du)) return MOE_ERR_NULL;
  if (!al16(dh) || !al16(g) || !al16(u) || !al16(dg) || !al16(du) || !al16(w) || !al16(perm) ||
      !al4(rows) || !al16(dw))
    return MOE_ERR_ALIGN;
  const moe_status st = device_ok();
  if (st != MOE_OK) return st;
  if (desc->R == 0) return MOE_OK;
  return cu(launch_swiglu_backward(*desc, dh, g, u, w, perm, n_w, rows, dg, du, dw,
                                   static_cast<cudaStream_t>(stream)));
}

moe_status moe_adamw_step(const moe_adamw_cfg* cfg, const moe_adamw_tensor* tensors,
                          int32_t n_tensors, void* stream) {
  PdlScope pdl_scope(0);
  if (cfg == nullptr || n_tensors < 0) return MOE_ERR_CFG;
  if (n_tensors > 0 && tensors == nullptr) return MOE_ERR_NULL;
  // written so that a NaN fails its test
  if (!(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0 && cfg->beta2 >= 0.0 && cfg->beta2 < 1.0))
    return MOE_ERR_CFG;
  if (!(cfg->eps >= 0.0) || !isfinite(cfg->eps) || !isfinite(cfg->weight_decay)) return MOE_ERR_CFG;
  if (cfg->eps > 0.0 && cfg->eps < 0x1p-126) return MOE_ERR_CFG;  // its fp32 reciprocal may be infinite
  if (cfg->dyn == nullptr &&
      (cfg->step < 1 || !isfinite(cfg->lr) || !isfinite(cfg->grad_scale)))
    return MOE_ERR_CFG;
  if (!al16(cfg->dyn)) return MOE_ERR_ALIGN;
  for (int i = 0; i < n_tensors; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    const bool p_ok = t.p_type == MOE_T_BF16 || (t.p_type == MOE_T_F32 && t.master == nullptr);
    const bool q8 = t.state_type == MOE_STATE_8BIT;
    if (!p_ok || (t.g_type != MOE_T_BF16 && t.g_type != MOE_T_F32)) return MOE_ERR_CFG;
    if (!q8 && t.state_type != MOE_STATE_F32) return MOE_ERR_CFG;
    if (t.n < 0 || t.n > (1LL << 40) || !isfinite(t.wd_scale)) return MOE_ERR_CFG;
    if (t.n == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v || (q8 && (!t.m_scale || !t.v_scale))) return MOE_ERR_NULL;
    if (!al16(t.p) || !al16(t.master) || !al16(t.g) || !al16(t.m) || !al16(t.v)) return MOE_ERR_ALIGN;
    // one scale is read or written at a time: a view that starts at any block will do
    if (!al4(t.m_scale) || !al4(t.v_scale)) return MOE_ERR_ALIGN;
  }
  const moe_status st = device_ok();
  if (st != MOE_OK) return st;
  return cu(launch_adamw(*cfg, tensors, n_tensors, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
