// C ABI of the training-step operators (include/himuon.h): argument checks and launches of
// the policy loss, the gradient norm and AdamW.  Nothing here allocates or waits, and no
// state is kept between calls.
#include <hip/hip_runtime.h>

#include <cmath>

#include "himuon.h"
#include "himuon_internal.h"

namespace {

himuon_status bad(const char *msg) { return himuon::set_error(HIMUON_EINVAL, msg); }

himuon_status launched(hipError_t e, const char *what) {
  if (e == hipSuccess) return HIMUON_OK;
  return himuon::set_error(HIMUON_EDEVICE, std::string(what) + ": " + hipGetErrorString(e));
}

bool is_dtype(himuon_dtype d) { return d == HIMUON_F32 || d == HIMUON_BF16; }

// A tensor's bytes have to be addressable; its size is otherwise free.
constexpr int64_t kMostElements = (int64_t)1 << 40;
constexpr int32_t kMostTensors = 1 << 24;

himuon_status check_workspace(const void *ws, size_t have, size_t need) {
  if (need == 0) return HIMUON_OK;
  if (!ws || have < need) return bad("workspace smaller than the workspace query says");
  if (reinterpret_cast<uintptr_t>(ws) % 16) return bad("workspace must be 16-byte aligned");
  return HIMUON_OK;
}

himuon_status check_policy(const himuon_policy *p) {
  if (!p) return bad("NULL argument");
  if (p->rows < 0 || p->rows > kMostElements) return bad("rows must be in [0, 2^40]");
  if (p->vocab < 1 || p->vocab > INT32_MAX / 2) return bad("vocab must be in [1, 2^30)");
  if (!is_dtype(p->dtype)) return bad("dtype");
  if (p->ld_logits < p->vocab) return bad("ld_logits must be >= vocab");
  if (p->dlogits && p->ld_dlogits < p->vocab) return bad("ld_dlogits must be >= vocab");
  if (p->ld_logits > kMostElements || (p->dlogits && p->ld_dlogits > kMostElements)) return bad("leading dimension too large");
  if (p->dlogits && p->dlogits == p->logits && p->ld_dlogits != p->ld_logits)
    return bad("dlogits in the place of logits needs the same leading dimension");
  if (!(p->clip_low >= 0 && p->clip_low <= 1) || !(p->clip_high >= 0 && std::isfinite(p->clip_high)))
    return bad("clip_low must be in [0, 1] and clip_high finite and >= 0");
  if (!std::isfinite(p->kl_coef) || !std::isfinite(p->grad_scale)) return bad("kl_coef and grad_scale must be finite");
  if (!(p->temperature >= 0x1p-20 && p->temperature <= 0x1p20)) return bad("temperature must be in [2^-20, 2^20]");
  return HIMUON_OK;
}

himuon_status check_adamw(const himuon_adamw_tensor *tensors, int32_t n_tensors, const himuon_adamw_config *cfg) {
  if (n_tensors < 0 || (n_tensors > 0 && !tensors) || !cfg) return bad("bad argument");
  if (n_tensors > kMostTensors) return bad("more than 2^24 tensors");
  if (!is_dtype(cfg->weight_dtype) || !is_dtype(cfg->grad_dtype)) return bad("dtype");
  if (cfg->state_bits != 32 && cfg->state_bits != 8) return bad("state_bits must be 32 or 8");
  if (!(cfg->beta1 >= 0 && cfg->beta1 < 1 && cfg->beta2 >= 0 && cfg->beta2 < 1)) return bad("betas must be in [0, 1)");
  if (!(cfg->eps >= 1e-30 && std::isfinite((float)cfg->eps))) return bad("eps must be finite and >= 1e-30");
  int64_t total = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    const himuon_adamw_tensor &x = tensors[i];
    if (x.n < 0 || x.n > kMostElements - total) return bad("n must be >= 0, 2^40 in all at most");
    total += x.n;
    if (!std::isfinite((float)x.weight_decay)) return bad("weight_decay must be finite");
    if (x.n == 0) continue;
    if (!x.weight || !x.grad || !x.m || !x.v) return bad("NULL pointer");
    if (cfg->state_bits == 8 && (!x.m_scale || !x.v_scale)) return bad("8-bit states need their scales");
  }
  return HIMUON_OK;
}

}  // namespace

extern "C" {

HIMUON_API himuon_status himuon_policy_workspace(const himuon_policy *p, size_t *bytes) try {
  if (!bytes) return bad("NULL argument");
  himuon_status s = check_policy(p);
  if (s != HIMUON_OK) return s;
  *bytes = himuon::policy_workspace(*p);
  return HIMUON_OK;
} catch (...) {
  return HIMUON_ENOMEM;
}

HIMUON_API himuon_status himuon_policy_loss(const himuon_policy *p, void *workspace, size_t ws_bytes,
                                            void *hip_stream) try {
  himuon_status s = check_policy(p);
  if (s != HIMUON_OK) return s;
  if (!p->stats) return bad("NULL pointer");
  if (p->rows > 0 && (!p->logits || !p->label || !p->weight || !p->advantage || !p->logp)) return bad("NULL pointer");
  if ((s = check_workspace(workspace, ws_bytes, himuon::policy_workspace(*p))) != HIMUON_OK) return s;
  return launched(himuon::launch_policy(*p, workspace, reinterpret_cast<hipStream_t>(hip_stream)),
                  "policy loss launch");
} catch (...) {
  return HIMUON_ENOMEM;
}

HIMUON_API himuon_status himuon_grad_norm_workspace(int32_t n_tensors, size_t *bytes) try {
  if (!bytes || n_tensors < 0 || n_tensors > kMostTensors) return bad("bad argument");
  *bytes = himuon::grad_norm_workspace(n_tensors);
  return HIMUON_OK;
} catch (...) {
  return HIMUON_ENOMEM;
}

HIMUON_API himuon_status himuon_grad_norm(const himuon_grad *tensors, int32_t n_tensors, himuon_dtype dtype,
                                          double max_norm, float *out, void *workspace, size_t ws_bytes,
                                          void *hip_stream) try {
  if (n_tensors < 0 || (n_tensors > 0 && !tensors) || !out) return bad("bad argument");
  if (n_tensors > kMostTensors) return bad("more than 2^24 tensors");
  if (!is_dtype(dtype)) return bad("dtype");
  if (!std::isfinite(max_norm) || max_norm < 0) return bad("max_norm must be finite and >= 0");
  int64_t total = 0;
  for (int32_t i = 0; i < n_tensors; ++i) {
    if (tensors[i].n < 0 || tensors[i].n > kMostElements - total) return bad("n must be >= 0, 2^40 in all at most");
    total += tensors[i].n;
    if (tensors[i].n > 0 && !tensors[i].grad) return bad("NULL pointer");
  }
  himuon_status s = check_workspace(workspace, ws_bytes, himuon::grad_norm_workspace(n_tensors));
  if (s != HIMUON_OK) return s;
  return launched(himuon::launch_grad_norm(tensors, n_tensors, dtype == HIMUON_BF16, max_norm, out, workspace,
                                           reinterpret_cast<hipStream_t>(hip_stream)),
                  "gradient norm launch");
} catch (...) {
  return HIMUON_ENOMEM;
}

HIMUON_API himuon_status himuon_adamw_table_size(const himuon_adamw_tensor *tensors, int32_t n_tensors,
                                                 const himuon_adamw_config *cfg, size_t *bytes) try {
  if (!bytes) return bad("NULL argument");
  himuon_status s = check_adamw(tensors, n_tensors, cfg);
  if (s != HIMUON_OK) return s;
  *bytes = n_tensors > himuon::adamw_few_tensors() ? himuon::adamw_table_size(n_tensors, cfg->state_bits) : 0;
  return HIMUON_OK;
} catch (...) {
  return HIMUON_ENOMEM;
}

HIMUON_API himuon_status himuon_adamw_table(const himuon_adamw_tensor *tensors, int32_t n_tensors,
                                            const himuon_adamw_config *cfg, void *host, size_t bytes) try {
  himuon_status s = check_adamw(tensors, n_tensors, cfg);
  if (s != HIMUON_OK) return s;
  if (!host || bytes < himuon::adamw_table_size(n_tensors, cfg->state_bits)) return bad("table too small");
  if (reinterpret_cast<uintptr_t>(host) % 8) return bad("table must be 8-byte aligned");
  himuon::adamw_table(tensors, n_tensors, cfg->state_bits, host);
  return HIMUON_OK;
} catch (...) {
  return HIMUON_ENOMEM;
}

HIMUON_API himuon_status himuon_adamw_step(const himuon_adamw_tensor *tensors, int32_t n_tensors,
                                           const himuon_adamw_config *cfg, int64_t t, double lr,
                                           const float *grad_scale, const uint32_t *dither, const void *table,
                                           void *hip_stream) try {
  himuon_status s = check_adamw(tensors, n_tensors, cfg);
  if (s != HIMUON_OK) return s;
  if (t < 1) return bad("t must be >= 1");
  if (!std::isfinite((float)lr)) return bad("lr must be finite");
  if (reinterpret_cast<uintptr_t>(table) % 16) return bad("table must be 16-byte aligned");
  himuon::AdamWParams p{};
  p.beta1 = (float)cfg->beta1;
  p.omb1 = (float)(1.0 - cfg->beta1);
  p.beta2 = (float)cfg->beta2;
  p.omb2 = (float)(1.0 - cfg->beta2);
  const double bias1 = 1.0 - std::pow(cfg->beta1, (double)t), bias2 = 1.0 - std::pow(cfg->beta2, (double)t);
  p.root_scale = (float)(1.0 / std::sqrt(bias2));
  p.eps = (float)cfg->eps;
  p.step = (float)(lr / bias1);
  p.lr = (float)lr;
  p.dither[0] = dither ? dither[0] : 0;
  p.dither[1] = dither ? dither[1] : 0;
  p.grad_scale = grad_scale;
  return launched(himuon::launch_adamw(tensors, n_tensors, cfg->weight_dtype == HIMUON_BF16,
                                       cfg->grad_dtype == HIMUON_BF16, cfg->state_bits, p, table,
                                       reinterpret_cast<hipStream_t>(hip_stream)),
                  "AdamW step launch");
} catch (...) {
  return HIMUON_ENOMEM;
}

}  // extern "C"
