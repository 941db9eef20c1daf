// moe_mx4_api.hip -- the C ABI of the row-major MXFP4 operators declared in
// include/moe.h: argument checks and launches.  Host code only; the kernels live
// in moe_mx4.hip.
#include "moe_check.h"
#include "moe_mx4.h"

using namespace moe;

namespace {

constexpr int kMaxDim = 1 << 20;  // N, K: a tile's rows stay inside a 32-bit byte range

int check_mm(const moe_mm_cfg* c, const int32_t* offsets, const int32_t* row_token, int x_rows) {
  if (c->R < 0 || c->R > kMaxRows || c->N < 1 || c->K < 1 || c->E < 1 || c->E > 1024) return MOE_ERR_BAD_SHAPE;
  if (c->N % 8 || c->K % 32 || c->N > kMaxDim || c->K > kMaxDim) return MOE_ERR_BAD_SHAPE;
  if (c->clear_rest != 0 && c->clear_rest != 1) return MOE_ERR_BAD_SHAPE;
  if (!offsets && c->E != 1) return MOE_ERR_BAD_SHAPE;
  if (x_rows < 0 || (row_token && int64_t(x_rows) * (c->K / 2) >= (int64_t(1) << 31))) return MOE_ERR_BAD_SHAPE;
  if (c->out_dtype != MOE_DT_BF16 && c->out_dtype != MOE_DT_FP16 && c->out_dtype != MOE_DT_FP32)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_x(int dtype, int swiglu) {
  return (dtype != MOE_DT_BF16 && dtype != MOE_DT_FP16) || (swiglu != 0 && swiglu != 1) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

Mx4Args args_of(const moe_mm_cfg* c, const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws,
                const int32_t* offsets, const int32_t* row_token, void* y) {
  Mx4Args a{};
  a.p = xq; a.q = wq; a.pe = xs; a.qe = ws; a.out = y; a.offsets = offsets; a.row_token = row_token;
  a.R = c->R; a.N = c->N; a.K = c->K; a.E = c->E; a.T = c->T;
  a.out_ty = c->out_dtype; a.clear_rest = c->clear_rest;
  return a;
}

int enqueue(const Mx4Args& a, void* stream) {
  bool too_large = false;
  const hipError_t e = launch_mx4(a, static_cast<hipStream_t>(stream), &too_large);
  return too_large ? MOE_ERR_BAD_SHAPE : hip_status(e);
}

// codes and scales of the rows of x: the tokens where rows are gathered, else the output's rows
size_t codes_bytes(size_t rows, int K) { return align256(rows * (K / 2)); }
size_t linear_bytes(const moe_mm_cfg* c, int gathered) {
  const size_t rows = size_t(gathered ? c->T : c->R);
  if (linear_mx4_is_one_launch(c->R, c->K)) return 0;
  return rows ? codes_bytes(rows, c->K) + align256(rows * (c->K / 32)) : 0;
}

}  // namespace

extern "C" int moe_quant_mx4(int R, int K, int dtype, int swiglu, const void* x, uint8_t* codes, uint8_t* scales,
                             void* stream) {
  int rc;
  if ((rc = null_ptrs({{x, R != 0}, {codes, R != 0}, {scales, R != 0}}))) return rc;
  if (R < 0 || K < 1 || K % 32 || K > kMaxDim) return MOE_ERR_BAD_SHAPE;
  if ((rc = check_x(dtype, swiglu))) return rc;
  if ((rc = misaligned_ptrs({x, codes, scales}))) return rc;
  return hip_status(launch_quant_mx4(x, dtype, swiglu, R, K, codes, scales, static_cast<hipStream_t>(stream)));
}

extern "C" int moe_mm_mx4(const moe_mm_cfg* cfg, const uint8_t* xq, const uint8_t* xs, const uint8_t* wq,
                          const uint8_t* ws, const int32_t* offsets, const int32_t* row_token, void* y,
                          void* stream) {
  if (!cfg) return MOE_ERR_NULL_ARG;
  const bool some = cfg->R != 0, tokens = some && (!row_token || cfg->T != 0);
  int rc;
  if ((rc = null_ptrs({{xq, tokens}, {xs, tokens}, {wq, true}, {ws, true}, {y, some}}))) return rc;
  if ((rc = check_mm(cfg, offsets, row_token, row_token ? cfg->T : cfg->R))) return rc;
  if ((rc = misaligned_ptrs({xq, xs, wq, ws, y}, {offsets, row_token}))) return rc;
  return enqueue(args_of(cfg, xq, xs, wq, ws, offsets, row_token, y), stream);
}

extern "C" int moe_linear_mx4_workspace_size(const moe_mm_cfg* cfg, int gathered, size_t* bytes) {
  if (!cfg || !bytes) return MOE_ERR_NULL_ARG;
  moe_mm_cfg c = *cfg;
  c.out_dtype = MOE_DT_BF16;  // the size does not depend on it, nor on whether there are offsets
  static const int32_t some = 0;
  const int rc = check_mm(&c, &some, nullptr, 0);
  if (rc) return rc;
  if (c.T < 0 || (gathered != 0 && gathered != 1)) return MOE_ERR_BAD_SHAPE;
  *bytes = linear_bytes(cfg, gathered);
  return MOE_OK;
}

extern "C" int moe_linear_mx4(const moe_mm_cfg* cfg, const void* x, int swiglu, const uint8_t* wq, const uint8_t* ws,
                              const int32_t* offsets, const int32_t* row_token, void* y, void* work,
                              size_t work_bytes, void* stream) {
  if (!cfg) return MOE_ERR_NULL_ARG;
  const int rows = row_token ? cfg->T : cfg->R;
  const bool some = cfg->R != 0, tokens = some && rows != 0;
  int rc;
  if ((rc = null_ptrs({{x, tokens}, {wq, true}, {ws, true}, {y, some}}))) return rc;
  const bool two = tokens && !linear_mx4_is_one_launch(cfg->R, cfg->K);  // launches, with scratch between them
  if (two && !work) return MOE_ERR_NULL_ARG;
  if ((rc = check_mm(cfg, offsets, row_token, rows))) return rc;
  if ((rc = check_x(cfg->dtype, swiglu))) return rc;
  if ((rc = misaligned_ptrs({x, wq, ws, y, work}, {offsets, row_token}))) return rc;
  if (two && work_bytes < linear_bytes(cfg, row_token != nullptr)) return MOE_ERR_WORKSPACE;
  if (some && linear_mx4_is_one_launch(cfg->R, cfg->K)) {
    Mx4Args a = args_of(cfg, nullptr, nullptr, wq, ws, offsets, row_token, y);
    a.p = x;
    return hip_status(launch_linear_mx4_one(a, cfg->dtype, swiglu, static_cast<hipStream_t>(stream)));
  }
  uint8_t* codes = static_cast<uint8_t*>(work);
  uint8_t* scales = two ? codes + codes_bytes(size_t(rows), cfg->K) : nullptr;
  const Mx4Args a = args_of(cfg, codes, scales, wq, ws, offsets, row_token, y);
  if (mx4_too_large(a)) return MOE_ERR_BAD_SHAPE;  // before the quantiser goes out
  if (two && (rc = hip_status(launch_quant_mx4(x, cfg->dtype, swiglu, rows, cfg->K, codes, scales,
                                                  static_cast<hipStream_t>(stream)))))
    return rc;
  return enqueue(a, stream);
}
