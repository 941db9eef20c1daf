// moe_few_api.hip -- the C ABI of the few-token layer on 16-bit row-major
// weights declared in include/moe.h: argument checks and launches.  Host code
// only; the kernels live in moe_few.hip.
#include "moe_check.h"
#include "moe_few.h"

using namespace moe;

namespace {

constexpr int kMaxWidth = 1 << 16;

int check_few(const moe_few_cfg* c) {
  if (c->T < 0 || c->H < 1 || c->I < 1 || c->E < 1 || c->topk < 1) return MOE_ERR_BAD_SHAPE;
  if (c->H % 8 || c->I % 8 || c->H > kMaxWidth || c->I > kMaxWidth || c->E > 1024 || c->topk > 32)
    return MOE_ERR_BAD_SHAPE;
  if (c->T > kFewTokens) return MOE_ERR_UNSUPPORTED;
  if (c->dtype != MOE_DT_BF16 && c->dtype != MOE_DT_FP16) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" int moe_layer_mm_workspace_size(const moe_few_cfg* cfg, size_t* bytes) {
  if (!cfg || !bytes) return MOE_ERR_NULL_ARG;
  const int rc = check_few(cfg);
  if (rc) return rc;
  *bytes = cfg->T ? few_bytes(cfg->T, cfg->H, cfg->I, cfg->E, cfg->topk) : 0;
  return MOE_OK;
}

extern "C" int moe_layer_mm(const moe_few_cfg* cfg, const void* x, const int32_t* topk_ids, const float* topk_weights,
                            const void* w1, const void* w2, void* out, void* ws, size_t ws_bytes, void* stream) {
  if (!cfg) return MOE_ERR_NULL_ARG;
  const bool some = cfg->T != 0;
  int rc;
  if ((rc = null_ptrs({{x, some}, {topk_ids, some}, {topk_weights, some}, {w1, true}, {w2, true}, {out, some},
                       {ws, some}})))
    return rc;
  if ((rc = check_few(cfg))) return rc;
  if ((rc = misaligned_ptrs({x, w1, w2, out, ws}, {topk_ids, reinterpret_cast<const int32_t*>(topk_weights)}))) return rc;
  if (!some) return MOE_OK;
  if (ws_bytes < few_bytes(cfg->T, cfg->H, cfg->I, cfg->E, cfg->topk)) return MOE_ERR_WORKSPACE;
  FewArgs a{};
  a.x = x; a.ids = topk_ids; a.weights = topk_weights; a.w1 = w1; a.w2 = w2; a.out = out;
  a.T = cfg->T; a.H = cfg->H; a.I = cfg->I; a.E = cfg->E; a.k = cfg->topk; a.ty = cfg->dtype;
  few_carve(a, ws);
  return hip_status(launch_few(a, static_cast<hipStream_t>(stream)));
}
