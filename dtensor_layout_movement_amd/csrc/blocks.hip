// C ABI of the block-scaled 8-bit matrices: argument checks and launches.
#include "blocks.h"
#include "checks.h"

#include <cstdint>

namespace {

using namespace rs;

reshard_status_t check_matmul(const reshard_matrix_t* a, const reshard_matrix_t* b, const reshard_matrix_t* out) {
  if (const reshard_status_t s = check_shape(a, "a", kAny)) return s;
  if (const reshard_status_t s = check_shape(b, "b", kHeld)) return s;
  if (const reshard_status_t s = check_shape(out, "out", kPlain)) return s;
  if (a->cols != b->cols) return report(RESHARD_ERR_INVALID_ARGUMENT, "a and b differ in columns (the contraction)");
  if (out->rows != a->rows || out->cols != b->rows)
    return report(RESHARD_ERR_INVALID_ARGUMENT, "out is not (rows of a) x (rows of b)");
  const MatmulPlan p = plan_matmul(*a, *b, *out);
  if (p.too_wide) return report(RESHARD_ERR_INVALID_ARGUMENT, "rows more than 2^23 bytes apart with more than 4 rows of a");
  if (p.groups > kMaxGroups) return too_many();
  return RESHARD_OK;
}

reshard_status_t check_grad(const reshard_matrix_t* dy, const reshard_matrix_t* x, const reshard_matrix_t* dw) {
  if (const reshard_status_t s = check_shape(dy, "dy", kPlain)) return s;
  if (const reshard_status_t s = check_shape(x, "x", kHeld)) return s;
  if (const reshard_status_t s = check_shape(dw, "dw", kPlain)) return s;
  if (dy->rows != x->rows) return report(RESHARD_ERR_INVALID_ARGUMENT, "dy and x differ in rows (the contraction)");
  if (dw->rows != dy->cols || dw->cols != x->cols)
    return report(RESHARD_ERR_INVALID_ARGUMENT, "dw is not (columns of dy) x (columns of x)");
  if (dy->cols > kMaxGradCols || dy->rows * grad_planes(dy->dtype) > kMaxGradRows)
    return bad("dy", "too many rows or columns for a weight gradient");
  if (plan_grad(*dy, *x, *dw).groups > kMaxGroups) return too_many();
  return RESHARD_OK;
}

reshard_status_t block_quantize(const reshard_matrix_t* src, const reshard_matrix_t* dst,
                                const reshard_matrix_t* dst_t, void* stream) {
  if (const reshard_status_t s = check_shape(src, "src", kPlain)) return s;
  if (const reshard_status_t s = check_shape(dst, "dst", kHeld)) return s;
  if (dst->rows != src->rows || dst->cols != src->cols)
    return report(RESHARD_ERR_INVALID_ARGUMENT, "src and dst differ in shape");
  if (dst_t) {
    if (const reshard_status_t s = check_shape(dst_t, "dst_t", kHeld)) return s;
    if (dst_t->rows != src->cols || dst_t->cols != src->rows)
      return report(RESHARD_ERR_INVALID_ARGUMENT, "dst_t is not of src's transposed shape");
    if (dst->block_rows != RESHARD_BLOCK || dst_t->block_rows != RESHARD_BLOCK)
      return report(RESHARD_ERR_INVALID_ARGUMENT, "a transposed copy needs blocks of 128 rows on both sides");
    if (dst_t->dtype != dst->dtype) return report(RESHARD_ERR_INVALID_ARGUMENT, "dst and dst_t differ in dtype");
  }
  if (dst->block_rows != 1 && ceil_div(src->rows, kBlock) * blocks_of(src->cols) > kMaxGroups)
    return too_many();
  const reshard_status_t s = dst_t ? check_call({{src, "src", false}, {dst, "dst", true}, {dst_t, "dst_t", true}},
                                                {}, nullptr, 0, 0, stream)
                                   : check_call({{src, "src", false}, {dst, "dst", true}}, {}, nullptr, 0, 0, stream);
  if (s) return s;
  if (empty(*src)) return RESHARD_OK;
  return launched(launch_quantize(*src, *dst, dst_t, static_cast<hipStream_t>(stream)), "block quantize launch");
}

reshard_status_t block_dequantize(const reshard_matrix_t* src, const reshard_matrix_t* dst, void* stream) {
  if (const reshard_status_t s = check_shape(src, "src", kHeld)) return s;
  if (const reshard_status_t s = check_shape(dst, "dst", kPlain)) return s;
  if (dst->rows != src->rows || dst->cols != src->cols)
    return report(RESHARD_ERR_INVALID_ARGUMENT, "src and dst differ in shape");
  if (const reshard_status_t s = check_call({{src, "src", false}, {dst, "dst", true}}, {}, nullptr, 0, 0, stream)) return s;
  if (empty(*src)) return RESHARD_OK;
  return launched(launch_dequantize(*src, *dst, static_cast<hipStream_t>(stream)), "block dequantize launch");
}

reshard_status_t block_matmul(const reshard_matrix_t* a, const reshard_matrix_t* b, const reshard_matrix_t* out,
                              void* workspace, int64_t workspace_bytes, void* stream) {
  if (const reshard_status_t s = check_matmul(a, b, out)) return s;
  const MatmulPlan plan = plan_matmul(*a, *b, *out);
  if (const reshard_status_t s = check_call({{a, "a", false}, {b, "b", false}, {out, "out", true}}, {}, workspace,
                                            plan.bytes(), workspace_bytes, stream))
    return s;
  if (empty(*out)) return RESHARD_OK;
  return launched(launch_matmul(plan, *a, *b, *out, workspace, static_cast<hipStream_t>(stream)),
                  "block matmul launch");
}

reshard_status_t block_grad(const reshard_matrix_t* dy, const reshard_matrix_t* x, const reshard_matrix_t* dw,
                            int accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
  if (const reshard_status_t s = check_grad(dy, x, dw)) return s;
  const GradPlan plan = plan_grad(*dy, *x, *dw);
  if (const reshard_status_t s = check_call({{dy, "dy", false}, {x, "x", false}, {dw, "dw", true}}, {}, workspace,
                                            plan.bytes(), workspace_bytes, stream))
    return s;
  if (empty(*dw)) return RESHARD_OK;
  return launched(launch_grad(plan, *dy, *x, *dw, accumulate != 0, workspace, static_cast<hipStream_t>(stream)),
                  "block grad launch");
}

}  // namespace

extern "C" {

reshard_status_t reshard_block_quantize(const reshard_matrix_t* src, const reshard_matrix_t* dst,
                                        const reshard_matrix_t* dst_t, void* stream) {
  return guarded([&] { return block_quantize(src, dst, dst_t, stream); });
}

reshard_status_t reshard_block_dequantize(const reshard_matrix_t* src, const reshard_matrix_t* dst, void* stream) {
  return guarded([&] { return block_dequantize(src, dst, stream); });
}

reshard_status_t reshard_block_matmul_workspace(const reshard_matrix_t* a, const reshard_matrix_t* b,
                                                const reshard_matrix_t* out, int64_t* bytes) {
  return guarded([&]() -> reshard_status_t {
    if (!bytes) return report(RESHARD_ERR_INVALID_ARGUMENT, "bytes is NULL");
    *bytes = 0;
    if (const reshard_status_t s = check_matmul(a, b, out)) return s;
    *bytes = plan_matmul(*a, *b, *out).bytes();
    return RESHARD_OK;
  });
}

reshard_status_t reshard_block_matmul(const reshard_matrix_t* a, const reshard_matrix_t* b,
                                      const reshard_matrix_t* out, void* workspace, int64_t workspace_bytes,
                                      void* stream) {
  return guarded([&] { return block_matmul(a, b, out, workspace, workspace_bytes, stream); });
}

reshard_status_t reshard_block_grad_workspace(const reshard_matrix_t* dy, const reshard_matrix_t* x,
                                              const reshard_matrix_t* dw, int64_t* bytes) {
  return guarded([&]() -> reshard_status_t {
    if (!bytes) return report(RESHARD_ERR_INVALID_ARGUMENT, "bytes is NULL");
    *bytes = 0;
    if (const reshard_status_t s = check_grad(dy, x, dw)) return s;
    *bytes = plan_grad(*dy, *x, *dw).bytes();
    return RESHARD_OK;
  });
}

reshard_status_t reshard_block_grad(const reshard_matrix_t* dy, const reshard_matrix_t* x, const reshard_matrix_t* dw,
                                    int accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&] { return block_grad(dy, x, dw, accumulate, workspace, workspace_bytes, stream); });
}

}  // extern "C"
