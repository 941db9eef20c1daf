// moe_mm_api.hip -- the C ABI of the row-major products and the int8
// quantiser declared in include/moe.h: argument checks and launches.  Host
// code only; the kernels live in moe_mm.hip and moe_quant_i8.hip.
#include <cstdint>
#include <initializer_list>
#include <utility>

#include "../../include/moe.h"
#include "moe_mm.h"

using namespace moe;

namespace {

constexpr int kMaxDim = 1 << 20;   // N, K: a tile's rows stay inside a 32-bit byte range
constexpr int kMaxRows = 0x7FFFFFFF - 1023;  // a row count rounded up to a tile stays an int32
constexpr int kMaxKInt8 = 1 << 16;  // 128 * 128 * K stays inside an int32 sum

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }
int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// (pointer, required)
using PtrList = std::initializer_list<std::pair<const void*, bool>>;
int null_ptrs(PtrList ps) {
  for (auto& p : ps)
    if (p.second && !p.first) return MOE_ERR_NULL_ARG;
  return MOE_OK;
}
// tensors on 16 bytes, index arrays (a slice of a longer one, say) on 4
int misaligned_ptrs(std::initializer_list<const void*> tensors, std::initializer_list<const int32_t*> indices = {}) {
  for (auto p : tensors)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return MOE_ERR_MISALIGNED;
  for (auto p : indices)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

int check_dims(const moe_mm_cfg* c) {
  if (c->R < 0 || c->R > kMaxRows || c->N < 1 || c->K < 1 || c->E < 1 || c->E > 1024) return MOE_ERR_BAD_SHAPE;
  if (c->N % 8 || c->K % 8 || c->N > kMaxDim || c->K > kMaxDim) return MOE_ERR_BAD_SHAPE;
  if (c->clear_rest != 0 && c->clear_rest != 1) return MOE_ERR_BAD_SHAPE;
  return MOE_OK;
}

// 16-bit operands; the output in their type or in fp32
int check_types(const moe_mm_cfg* c) {
  if (c->dtype != MOE_DT_BF16 && c->dtype != MOE_DT_FP16) return MOE_ERR_UNSUPPORTED;
  if (c->out_dtype != c->dtype && c->out_dtype != MOE_DT_FP32) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_i8(const moe_mm_cfg* c, const int32_t* offsets, const int32_t* row_token, int x_rows) {
  int rc = check_dims(c);
  if (rc) return rc;
  if (c->K % 16 || c->K > kMaxKInt8) return MOE_ERR_BAD_SHAPE;
  if (!offsets && c->E != 1) return MOE_ERR_BAD_SHAPE;
  if (x_rows < 0 || (row_token && int64_t(x_rows) * c->K >= (int64_t(1) << 31))) return MOE_ERR_BAD_SHAPE;
  if (c->out_dtype != MOE_DT_BF16 && c->out_dtype != MOE_DT_FP16 && c->out_dtype != MOE_DT_FP32)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

MmArgs args_of(const moe_mm_cfg* c, const void* p, const void* q, const int32_t* offsets, void* out) {
  MmArgs a{};
  a.p = p; a.q = q; a.out = out; a.offsets = offsets;
  a.R = c->R; a.N = c->N; a.K = c->K; a.E = c->E; a.T = c->T;
  a.ty = c->dtype; a.out_ty = c->out_dtype; a.clear_rest = c->clear_rest;
  return a;
}

int enqueue(int op, const MmArgs& a, void* stream) {
  bool too_large = false;
  const hipError_t e = launch_mm(op, a, static_cast<hipStream_t>(stream), &too_large);
  return too_large ? MOE_ERR_BAD_SHAPE : hip_status(e);
}

int grouped(int op, const moe_mm_cfg* c, const void* p, const void* q, const int32_t* offsets, void* out,
            bool p_rows, bool q_rows, bool out_rows, void* stream, void* work = nullptr, size_t work_bytes = 0) {
  if (!c) return MOE_ERR_NULL_ARG;
  const bool some = c->R != 0;  // operands with one row per R may be null where there is none
  int rc;
  if ((rc = null_ptrs({{p, some || !p_rows}, {q, some || !q_rows}, {offsets, true}, {out, some || !out_rows}}))) return rc;
  if ((rc = check_dims(c)) || (rc = check_types(c))) return rc;
  if ((rc = misaligned_ptrs({p, q, out, work}, {offsets}))) return rc;
  MmArgs a = args_of(c, p, q, offsets, out);
  const size_t need = op == kWgrad ? wgrad_bytes(a) : 0;
  if (need && !work) return MOE_ERR_NULL_ARG;
  if (need > work_bytes) return MOE_ERR_WORKSPACE;
  a.partial = static_cast<float*>(work);
  return enqueue(op, a, stream);
}

}  // namespace

extern "C" int moe_grouped_mm(const moe_mm_cfg* cfg, const void* x, const void* w, const int32_t* offsets, void* y,
                              void* stream) {
  return grouped(kFwd, cfg, x, w, offsets, y, true, false, true, stream);
}

extern "C" int moe_grouped_mm_dgrad(const moe_mm_cfg* cfg, const void* dy, const void* w, const int32_t* offsets,
                                    void* dx, void* stream) {
  return grouped(kDgrad, cfg, dy, w, offsets, dx, true, false, true, stream);
}

extern "C" int moe_grouped_mm_wgrad_workspace_size(const moe_mm_cfg* cfg, size_t* bytes) {
  if (!cfg || !bytes) return MOE_ERR_NULL_ARG;
  int rc;
  if ((rc = check_dims(cfg)) || (rc = check_types(cfg))) return rc;
  *bytes = wgrad_bytes(args_of(cfg, nullptr, nullptr, nullptr, nullptr));
  return MOE_OK;
}

extern "C" int moe_grouped_mm_wgrad(const moe_mm_cfg* cfg, const void* dy, const void* x, const int32_t* offsets,
                                    void* dw, void* work, size_t work_bytes, void* stream) {
  return grouped(kWgrad, cfg, dy, x, offsets, dw, true, true, false, stream, work, work_bytes);
}

extern "C" int moe_quant_i8(int R, int K, int dtype, int swiglu, const void* x, int8_t* codes, float* scales,
                            void* stream) {
  int rc;
  if ((rc = null_ptrs({{x, R != 0}, {codes, R != 0}, {scales, R != 0}}))) return rc;
  if (R < 0 || K < 1 || K % 16 || K > kMaxDim) return MOE_ERR_BAD_SHAPE;
  if ((dtype != MOE_DT_BF16 && dtype != MOE_DT_FP16) || (swiglu != 0 && swiglu != 1)) return MOE_ERR_UNSUPPORTED;
  if ((rc = misaligned_ptrs({x, codes, scales}))) return rc;
  return hip_status(launch_quant_i8(x, dtype, swiglu, R, K, codes, scales, static_cast<hipStream_t>(stream)));
}

static MmArgs args_i8(const moe_mm_cfg* c, const int8_t* xq, const float* xs, const int8_t* wq, const float* ws,
                      const int32_t* offsets, const int32_t* row_token, void* y) {
  MmArgs a = args_of(c, xq, wq, offsets, y);
  a.ty = kInt8;
  a.row_token = row_token;
  a.ps = xs;
  a.qs = ws;
  return a;
}

extern "C" int moe_mm_i8(const moe_mm_cfg* cfg, const int8_t* xq, const float* xs, const int8_t* wq, const float* ws,
                         const int32_t* offsets, const int32_t* row_token, void* y, void* stream) {
  if (!cfg) return MOE_ERR_NULL_ARG;
  const bool some = cfg->R != 0, tokens = some && (!row_token || cfg->T != 0);
  int rc;
  if ((rc = null_ptrs({{xq, tokens}, {xs, tokens}, {wq, true}, {ws, true}, {y, some}}))) return rc;
  if ((rc = check_i8(cfg, offsets, row_token, row_token ? cfg->T : cfg->R))) return rc;
  if ((rc = misaligned_ptrs({xq, xs, wq, ws, y}, {offsets, row_token})))
    return rc;
  return enqueue(kFwd, args_i8(cfg, xq, xs, wq, ws, offsets, row_token, y), stream);
}

// codes and scales of the rows of x: the tokens where rows are gathered, else the output's rows
static size_t linear_bytes(const moe_mm_cfg* c, int gathered) {
  if (linear_is_one_launch(c->R, c->K)) return 0;
  const size_t rows = size_t(gathered ? c->T : c->R);
  return rows ? align256(rows * c->K) + align256(4 * rows) : 0;
}

extern "C" int moe_linear_i8_workspace_size(const moe_mm_cfg* cfg, int gathered, size_t* bytes) {
  if (!cfg || !bytes) return MOE_ERR_NULL_ARG;
  int rc = check_dims(cfg);
  if (rc) return rc;
  if (cfg->K % 16 || cfg->K > kMaxKInt8 || cfg->T < 0 || (gathered != 0 && gathered != 1)) return MOE_ERR_BAD_SHAPE;
  *bytes = linear_bytes(cfg, gathered);
  return MOE_OK;
}

extern "C" int moe_linear_i8(const moe_mm_cfg* cfg, const void* x, int swiglu, const int8_t* wq, const float* ws,
                             const int32_t* offsets, const int32_t* row_token, void* y, void* work,
                             size_t work_bytes, void* stream) {
  if (!cfg) return MOE_ERR_NULL_ARG;
  const int rows = row_token ? cfg->T : cfg->R;
  const bool some = cfg->R != 0, tokens = some && rows != 0;
  int rc;
  if ((rc = null_ptrs({{x, tokens}, {wq, true}, {ws, true}, {y, some}}))) return rc;
  const bool two = tokens && !linear_is_one_launch(cfg->R, cfg->K);  // launches, with scratch between them
  if (two && !work) return MOE_ERR_NULL_ARG;
  if ((rc = check_i8(cfg, offsets, row_token, rows))) return rc;
  if ((cfg->dtype != MOE_DT_BF16 && cfg->dtype != MOE_DT_FP16) || (swiglu != 0 && swiglu != 1))
    return MOE_ERR_UNSUPPORTED;
  if ((rc = misaligned_ptrs({x, wq, ws, y, work}, {offsets, row_token})))
    return rc;
  if (two && work_bytes < linear_bytes(cfg, row_token != nullptr)) return MOE_ERR_WORKSPACE;
  if (some && linear_is_one_launch(cfg->R, cfg->K)) {
    MmArgs a = args_of(cfg, x, wq, offsets, y);
    a.row_token = row_token;
    a.qs = ws;
    return hip_status(launch_linear_one(a, cfg->dtype, swiglu, static_cast<hipStream_t>(stream)));
  }
  int8_t* codes = static_cast<int8_t*>(work);
  float* scales = two ? reinterpret_cast<float*>(codes + align256(size_t(rows) * cfg->K)) : nullptr;
  const MmArgs a = args_i8(cfg, codes, scales, wq, ws, offsets, row_token, y);
  if (mm_too_large(kFwd, a)) return MOE_ERR_BAD_SHAPE;  // before the quantiser goes out
  if (two && (rc = hip_status(launch_quant_i8(x, cfg->dtype, swiglu, rows, cfg->K, codes, scales,
                                              static_cast<hipStream_t>(stream)))))
    return rc;
  return enqueue(kFwd, a, stream);
}
