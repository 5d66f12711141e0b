// C ABI of the group-scaled 4-bit matrices and of tokens sorted by expert: argument
// checks and launches.
#include "groups.h"
#include "checks.h"

#include <cstdint>

namespace {

using namespace rs;

reshard_status_t invalid(const char* what) { return report(RESHARD_ERR_INVALID_ARGUMENT, what); }

reshard_status_t check_product(const reshard_matrix_t* a, const reshard_matrix_t* b, int64_t experts,
                               const reshard_matrix_t* out) {
  if (const reshard_status_t s = check_shape(a, "a", kPlain)) return s;
  if (const reshard_status_t s = check_shape(b, "b", kGrouped)) return s;
  if (const reshard_status_t s = check_shape(out, "out", kPlain)) return s;
  if (a->cols != b->cols) return invalid("a and b differ in columns (the contraction)");
  if (experts) {
    if (experts < 1 || experts > kMaxExperts) return invalid("experts is not 1 to 1024");
    if (b->rows % experts) return invalid("b is not one matrix of equal rows for each expert");
    if (out->rows != a->rows || out->cols != b->rows / experts)
      return invalid("out is not (rows of a) x (rows of an expert's part of b)");
  } else if (out->rows != a->rows || out->cols != b->rows) {
    return invalid("out is not (rows of a) x (rows of b)");
  }
  if (plan_group_matmul(*a, *b, experts, *out).groups > kMaxGroups) return too_many();
  return RESHARD_OK;
}

reshard_status_t product(const reshard_matrix_t* a, const reshard_matrix_t* b, const int32_t* offsets, int64_t experts,
                         const reshard_matrix_t* out, void* workspace, int64_t workspace_bytes, void* stream) {
  if (const reshard_status_t s = check_product(a, b, experts, out)) return s;
  const GroupPlan plan = plan_group_matmul(*a, *b, experts, *out);
  const int64_t list = experts && !empty(*out) ? (experts + 1) * int64_t(sizeof(int32_t)) : 0;
  if (const reshard_status_t s =
          check_call({{a, "a", false}, {b, "b", false}, {out, "out", true}}, {{offsets, list, "offsets", false, 4}},
                     workspace, plan.bytes(), workspace_bytes, stream))
    return s;
  if (empty(*out)) return RESHARD_OK;
  return launched(launch_group_matmul(plan, *a, *b, offsets, experts, *out, workspace, static_cast<hipStream_t>(stream)),
                  "group matmul launch");
}

reshard_status_t product_workspace(const reshard_matrix_t* a, const reshard_matrix_t* b, int64_t experts,
                                   const reshard_matrix_t* out, int64_t* bytes) {
  if (!bytes) return invalid("bytes is NULL");
  *bytes = 0;
  if (const reshard_status_t s = check_product(a, b, experts, out)) return s;
  *bytes = plan_group_matmul(*a, *b, experts, *out).bytes();
  return RESHARD_OK;
}

reshard_status_t group_quantize(const reshard_matrix_t* src, const reshard_matrix_t* dst, void* stream) {
  if (const reshard_status_t s = check_shape(src, "src", kPlain)) return s;
  if (const reshard_status_t s = check_shape(dst, "dst", kGrouped)) return s;
  if (dst->rows != src->rows || dst->cols != src->cols) return invalid("src and dst differ in shape");
  if (const reshard_status_t s = check_call({{src, "src", false}, {dst, "dst", true}}, {}, nullptr, 0, 0, stream)) return s;
  if (empty(*src)) return RESHARD_OK;
  return launched(launch_group_quantize(*src, *dst, static_cast<hipStream_t>(stream)), "group quantize launch");
}

reshard_status_t group_dequantize(const reshard_matrix_t* src, const reshard_matrix_t* dst, void* stream) {
  if (const reshard_status_t s = check_shape(src, "src", kGrouped)) return s;
  if (const reshard_status_t s = check_shape(dst, "dst", kPlain)) return s;
  if (dst->rows != src->rows || dst->cols != src->cols) return invalid("src and dst differ in shape");
  if (const reshard_status_t s = check_call({{src, "src", false}, {dst, "dst", true}}, {}, nullptr, 0, 0, stream)) return s;
  if (empty(*src)) return RESHARD_OK;
  return launched(launch_group_dequantize(*src, *dst, static_cast<hipStream_t>(stream)), "group dequantize launch");
}

// ------------------------------------------------------- tokens and experts

reshard_status_t check_choices(int64_t tokens, int choices) {
  if (choices < 1 || choices > RESHARD_MAX_CHOICES) return invalid("choices is not 1 to 64");
  if (tokens < 0 || tokens > kMaxChosen || tokens * choices > kMaxChosen) return invalid("too many tokens");
  return RESHARD_OK;
}

// The bytes of positions that a call looks at.
Array positions(const int32_t* position, int64_t tokens, int choices) {
  return Array{position, tokens * choices * int64_t(sizeof(int32_t)), "position", false, 4};
}

reshard_status_t check_sort(int64_t tokens, int choices, int64_t experts) {
  if (const reshard_status_t s = check_choices(tokens, choices)) return s;
  if (experts < 1 || experts > kMaxExperts) return invalid("experts is not 1 to 1024");
  return RESHARD_OK;
}

reshard_status_t expert_sort(const void* ids, int ids_dtype, int64_t tokens, int choices, int64_t first,
                             int64_t experts, int32_t* offsets, int32_t* position, void* workspace,
                             int64_t workspace_bytes, void* stream) {
  if (ids_dtype != RESHARD_DTYPE_I32 && ids_dtype != RESHARD_DTYPE_I64) return bad("ids", "dtype is not I32 or I64");
  if (const reshard_status_t s = check_sort(tokens, choices, experts)) return s;
  if (first < 0 || first > (int64_t(1) << 40)) return invalid("first is out of range");
  const bool wide = ids_dtype == RESHARD_DTYPE_I64;
  const int64_t chosen = tokens * choices;
  const SortPlan plan = plan_sort(chosen, experts);
  if (const reshard_status_t s =
          check_call({}, {{ids, chosen * (wide ? 8 : 4), "ids", false, wide ? 8u : 4u},
                          {offsets, (experts + 1) * int64_t(sizeof(int32_t)), "offsets", true, 4},
                          {position, chosen * int64_t(sizeof(int32_t)), "position", true, 4}},
                     workspace, plan.bytes, workspace_bytes, stream))
    return s;
  return launched(launch_sort(plan, ids, wide, chosen, first, int(experts), offsets, position, workspace,
                              static_cast<hipStream_t>(stream)),
                  "expert sort launch");
}

reshard_status_t expert_gather(const reshard_matrix_t* x, const int32_t* position, int choices,
                               const reshard_matrix_t* rows, void* stream) {
  if (const reshard_status_t s = check_shape(x, "x", kPlain)) return s;
  if (const reshard_status_t s = check_shape(rows, "rows", kPlain)) return s;
  if (const reshard_status_t s = check_choices(x->rows, choices)) return s;
  if (rows->cols != x->cols) return invalid("x and rows differ in columns");
  if (rows->dtype != x->dtype) return invalid("x and rows differ in dtype");
  if (const reshard_status_t s = check_call({{x, "x", false}, {rows, "rows", true}},
                                            {positions(position, empty(*x) ? 0 : x->rows, choices)}, nullptr, 0, 0, stream))
    return s;
  if (empty(*x) || empty(*rows)) return RESHARD_OK;
  return launched(launch_gather(*x, position, choices, *rows, static_cast<hipStream_t>(stream)), "expert gather launch");
}

reshard_status_t check_weights(const reshard_matrix_t* weights, const char* name, int64_t tokens, int choices) {
  if (const reshard_status_t s = check_shape(weights, name, kPlain)) return s;
  if (weights->rows != tokens || weights->cols != choices) return bad(name, "is not tokens x choices");
  return RESHARD_OK;
}

constexpr reshard_matrix_t kNone{};  // stands for a matrix that was not given: no elements

reshard_status_t expert_combine(const reshard_matrix_t* rows, const int32_t* position, int choices,
                                const reshard_matrix_t* weights, const reshard_matrix_t* out, void* stream) {
  if (const reshard_status_t s = check_shape(rows, "rows", kPlain)) return s;
  if (const reshard_status_t s = check_shape(out, "out", kPlain)) return s;
  if (const reshard_status_t s = check_choices(out->rows, choices)) return s;
  if (rows->cols != out->cols) return invalid("rows and out differ in columns");
  if (rows->dtype != out->dtype) return invalid("rows and out differ in dtype");
  if (weights)
    if (const reshard_status_t s = check_weights(weights, "weights", out->rows, choices)) return s;
  const bool none = empty(*out);
  if (const reshard_status_t s =
          check_call({{rows, "rows", false}, {weights && !none ? weights : &kNone, "weights", false}, {out, "out", true}},
                     {positions(position, none ? 0 : out->rows, choices)}, nullptr, 0, 0, stream))
    return s;
  if (none) return RESHARD_OK;
  return launched(launch_combine(*rows, position, choices, weights, *out, static_cast<hipStream_t>(stream)),
                  "expert combine launch");
}

reshard_status_t expert_combine_grad(const reshard_matrix_t* dout, const reshard_matrix_t* rows, const int32_t* position,
                                     int choices, const reshard_matrix_t* weights, const reshard_matrix_t* drows,
                                     const reshard_matrix_t* dweights, void* stream) {
  if (const reshard_status_t s = check_shape(dout, "dout", kPlain)) return s;
  const int64_t tokens = dout->rows;
  if (const reshard_status_t s = check_choices(tokens, choices)) return s;
  if (!drows && !dweights) return invalid("neither drows nor dweights is given");
  if (weights)
    if (const reshard_status_t s = check_weights(weights, "weights", tokens, choices)) return s;
  if (dweights) {
    if (const reshard_status_t s = check_shape(rows, "rows", kPlain)) return s;
    if (const reshard_status_t s = check_weights(dweights, "dweights", tokens, choices)) return s;
    if (rows->cols != dout->cols) return invalid("rows and dout differ in columns");
    if (rows->dtype != dout->dtype) return invalid("rows and dout differ in dtype");
  }
  if (drows) {
    if (const reshard_status_t s = check_shape(drows, "drows", kPlain)) return s;
    if (drows->cols != dout->cols) return invalid("drows and dout differ in columns");
    if (drows->dtype != dout->dtype) return invalid("drows and dout differ in dtype");
    if (dweights && drows->rows != rows->rows) return invalid("drows and rows differ in rows");
  }
  const bool none = tokens == 0 || (!dweights && (empty(*dout) || empty(*drows)));
  if (const reshard_status_t s = check_call({{dout, "dout", false},
                                             {dweights ? rows : &kNone, "rows", false},
                                             {weights && drows ? weights : &kNone, "weights", false},
                                             {drows ? drows : &kNone, "drows", true},
                                             {dweights ? dweights : &kNone, "dweights", true}},
                                            {positions(position, none ? 0 : tokens, choices)}, nullptr, 0, 0, stream))
    return s;
  if (none) return RESHARD_OK;
  return launched(launch_combine_grad(*dout, rows, position, choices, weights, drows, dweights,
                                      static_cast<hipStream_t>(stream)),
                  "expert combine grad launch");
}

}  // namespace

extern "C" {

reshard_status_t reshard_group_quantize(const reshard_matrix_t* src, const reshard_matrix_t* dst, void* stream) {
  return guarded([&] { return group_quantize(src, dst, stream); });
}

reshard_status_t reshard_group_dequantize(const reshard_matrix_t* src, const reshard_matrix_t* dst, void* stream) {
  return guarded([&] { return group_dequantize(src, dst, stream); });
}

reshard_status_t reshard_group_matmul(const reshard_matrix_t* a, const reshard_matrix_t* b, const reshard_matrix_t* out,
                                      void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&] { return product(a, b, nullptr, 0, out, workspace, workspace_bytes, stream); });
}

reshard_status_t reshard_group_matmul_workspace(const reshard_matrix_t* a, const reshard_matrix_t* b,
                                                const reshard_matrix_t* out, int64_t* bytes) {
  return guarded([&] { return product_workspace(a, b, 0, out, bytes); });
}

reshard_status_t reshard_expert_matmul(const reshard_matrix_t* a, const reshard_matrix_t* b, const int32_t* offsets,
                                       int64_t experts, const reshard_matrix_t* out, void* workspace,
                                       int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> reshard_status_t {
    if (experts < 1) return invalid("experts is not 1 to 1024");
    return product(a, b, offsets, experts, out, workspace, workspace_bytes, stream);
  });
}

reshard_status_t reshard_expert_matmul_workspace(const reshard_matrix_t* a, const reshard_matrix_t* b, int64_t experts,
                                                 const reshard_matrix_t* out, int64_t* bytes) {
  return guarded([&]() -> reshard_status_t {
    if (bytes) *bytes = 0;
    if (experts < 1) return invalid("experts is not 1 to 1024");
    return product_workspace(a, b, experts, out, bytes);
  });
}

reshard_status_t reshard_expert_sort(const void* ids, int ids_dtype, int64_t tokens, int choices, int64_t first,
                                     int64_t experts, int32_t* offsets, int32_t* position, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
  return guarded([&] {
    return expert_sort(ids, ids_dtype, tokens, choices, first, experts, offsets, position, workspace, workspace_bytes,
                       stream);
  });
}

reshard_status_t reshard_expert_sort_workspace(int64_t tokens, int choices, int64_t experts, int64_t* bytes) {
  return guarded([&]() -> reshard_status_t {
    if (!bytes) return invalid("bytes is NULL");
    *bytes = 0;
    if (const reshard_status_t s = check_sort(tokens, choices, experts)) return s;
    *bytes = plan_sort(tokens * choices, experts).bytes;
    return RESHARD_OK;
  });
}

reshard_status_t reshard_expert_gather(const reshard_matrix_t* x, const int32_t* position, int choices,
                                       const reshard_matrix_t* rows, void* stream) {
  return guarded([&] { return expert_gather(x, position, choices, rows, stream); });
}

reshard_status_t reshard_expert_combine(const reshard_matrix_t* rows, const int32_t* position, int choices,
                                        const reshard_matrix_t* weights, const reshard_matrix_t* out, void* stream) {
  return guarded([&] { return expert_combine(rows, position, choices, weights, out, stream); });
}

reshard_status_t reshard_expert_combine_grad(const reshard_matrix_t* dout, const reshard_matrix_t* rows,
                                             const int32_t* position, int choices, const reshard_matrix_t* weights,
                                             const reshard_matrix_t* drows, const reshard_matrix_t* dweights,
                                             void* stream) {
  return guarded([&] { return expert_combine_grad(dout, rows, position, choices, weights, drows, dweights, stream); });
}

}  // extern "C"
