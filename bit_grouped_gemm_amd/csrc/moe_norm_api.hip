// moe_norm_api.hip -- the C ABI of the RMS norm declared in include/moe.h:
// argument checks and launches.  Host code only; the kernels live in
// moe_norm.hip.
#include "moe_check.h"
#include "moe_norm.h"

using namespace moe;

namespace {

constexpr int kMaxK = 1 << 14;  // what a workgroup's registers hold of a row

int check_norm(const moe_norm_cfg* c) {
  if (c->R < 0 || c->R > kMaxRows || c->K < 8 || c->K % 8 || c->K > kMaxK) return MOE_ERR_BAD_SHAPE;
  if (c->dtype != MOE_DT_BF16 && c->dtype != MOE_DT_FP16) return MOE_ERR_UNSUPPORTED;
  if (c->weight_dtype != c->dtype && c->weight_dtype != MOE_DT_FP32) return MOE_ERR_UNSUPPORTED;
  if (!(c->eps >= 1e-30f && c->eps <= 1.0f)) return MOE_ERR_UNSUPPORTED;  // (NaN too)
  return MOE_OK;
}

NormArgs args_of(const moe_norm_cfg* c, const void* x, const void* residual, const void* weight, void* y, void* sum) {
  NormArgs a{};
  a.x = x; a.res = residual; a.weight = weight; a.y = y; a.sum = residual ? sum : nullptr;
  a.R = c->R; a.K = c->K; a.ty = c->dtype; a.weight_fp32 = c->weight_dtype == MOE_DT_FP32; a.eps = c->eps;
  a.fmt = kQNone;
  return a;
}

}  // namespace

extern "C" int moe_rms_norm(const moe_norm_cfg* cfg, const void* x, const void* residual, const void* weight, void* y,
                            void* sum, float* rstd, void* stream) {
  if (!cfg) return MOE_ERR_NULL_ARG;
  const bool some = cfg->R != 0;
  int rc;
  if ((rc = null_ptrs({{x, some}, {weight, true}, {y, some}}))) return rc;
  if ((rc = check_norm(cfg))) return rc;
  if ((rc = misaligned_ptrs({x, residual, weight, y, sum, rstd}))) return rc;
  NormArgs a = args_of(cfg, x, residual, weight, y, sum);
  a.rstd = rstd;
  return hip_status(launch_norm(a, static_cast<hipStream_t>(stream)));
}

extern "C" int moe_rms_norm_quant(const moe_norm_cfg* cfg, const void* x, const void* residual, const void* weight,
                                  void* y, void* sum, void* codes, void* scales, void* stream) {
  if (!cfg) return MOE_ERR_NULL_ARG;
  const bool some = cfg->R != 0;
  int rc;
  if ((rc = null_ptrs({{x, some}, {weight, true}, {codes, some}, {scales, some}}))) return rc;
  if ((rc = check_norm(cfg))) return rc;
  switch (cfg->fmt) {
    case MOE_QFMT_E4M3:
      if (cfg->group != 32 && cfg->group != 128) return MOE_ERR_UNSUPPORTED;
      if (cfg->K % cfg->group) return MOE_ERR_BAD_SHAPE;
      break;
    case MOE_QFMT_I8:
      if (cfg->K % 16) return MOE_ERR_BAD_SHAPE;  // as moe_quant_i8
      break;
    case MOE_QFMT_MXFP4:
      if (cfg->K % 32) return MOE_ERR_BAD_SHAPE;
      break;
    default: return MOE_ERR_UNSUPPORTED;
  }
  if ((rc = misaligned_ptrs({x, residual, weight, y, sum, codes, scales}))) return rc;
  NormArgs a = args_of(cfg, x, residual, weight, y, sum);
  a.codes = codes;
  a.scales = scales;
  a.fmt = cfg->fmt;
  a.group = cfg->group;
  return hip_status(launch_norm(a, static_cast<hipStream_t>(stream)));
}

extern "C" int moe_rms_norm_backward_workspace_size(const moe_norm_cfg* cfg, size_t* bytes) {
  if (!cfg || !bytes) return MOE_ERR_NULL_ARG;
  const int rc = check_norm(cfg);
  if (rc) return rc;
  *bytes = norm_grad_bytes(cfg->R, cfg->K);
  return MOE_OK;
}

extern "C" int moe_rms_norm_backward(const moe_norm_cfg* cfg, const void* dy, const void* dsum, const void* sum,
                                     const float* rstd, const void* weight, void* dx, void* dweight, void* work,
                                     size_t work_bytes, void* stream) {
  if (!cfg) return MOE_ERR_NULL_ARG;
  const bool some = cfg->R != 0;
  int rc;
  if ((rc = null_ptrs({{dy, some}, {sum, some}, {rstd, some}, {weight, true}, {work, some && dweight}}))) return rc;
  if ((rc = check_norm(cfg))) return rc;
  if ((rc = misaligned_ptrs({dy, dsum, sum, rstd, weight, dx, dweight, work}))) return rc;
  if (dweight && work_bytes < norm_grad_bytes(cfg->R, cfg->K)) return MOE_ERR_WORKSPACE;
  NormGradArgs a{};
  a.dy = dy; a.dsum = dsum; a.sum = sum; a.rstd = rstd; a.weight = weight; a.dx = dx; a.dw = dweight;
  a.partial = static_cast<float*>(work);
  a.R = cfg->R; a.K = cfg->K; a.ty = cfg->dtype; a.weight_fp32 = cfg->weight_dtype == MOE_DT_FP32;
  return hip_status(launch_norm_grad(a, static_cast<hipStream_t>(stream)));
}
