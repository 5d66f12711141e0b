// C ABI of the block-scaled 8-bit matrices: argument checks and launches.
#include "blocks.h"

#include <cstdint>
#include <initializer_list>
#include <string>

namespace {

using rs::report;

constexpr int64_t kMaxSide = int64_t(1) << 30;
constexpr int64_t kMaxElems = int64_t(1) << 56;  // rows * row_stride, far beyond any memory

bool is_plain(int dtype) {
  return dtype == RESHARD_DTYPE_F32 || dtype == RESHARD_DTYPE_BF16 || dtype == RESHARD_DTYPE_F16;
}
bool is_held(int dtype) { return dtype == RESHARD_DTYPE_FP8_E4M3 || dtype == RESHARD_DTYPE_FP8_E5M2; }
int64_t elem_size(int dtype) { return dtype == RESHARD_DTYPE_F32 ? 4 : is_plain(dtype) ? 2 : 1; }

enum Kind { kPlain = 1, kHeld = 2, kAny = 3 };

reshard_status_t bad(const char* name, const char* what) {
  return report(RESHARD_ERR_INVALID_ARGUMENT, std::string(name) + ": " + what);
}

bool empty(const reshard_matrix_t& m) { return m.rows == 0 || m.cols == 0; }

// Shape, type and strides of one matrix.
reshard_status_t check_shape(const reshard_matrix_t* m, const char* name, Kind kind) {
  if (!m) return bad(name, "matrix is NULL");
  if (m->rows < 0 || m->cols < 0 || m->rows > kMaxSide || m->cols > kMaxSide) return bad(name, "rows or cols out of range");
  // the strides of a matrix without elements mean nothing
  if (!empty(*m) && (m->row_stride < 0 || m->row_stride > kMaxSide * 2 || m->rows * m->row_stride > kMaxElems))
    return bad(name, "row_stride out of range");
  if (is_plain(m->dtype) && (kind & kPlain)) {
    if (m->block_rows != 0) return bad(name, "a plain matrix has block_rows 0");
    if (!empty(*m) && m->row_stride < m->cols) return bad(name, "row_stride is below cols");
    return RESHARD_OK;
  }
  if (is_held(m->dtype) && (kind & kHeld)) {
    if (m->block_rows != 1 && m->block_rows != RESHARD_BLOCK) return bad(name, "block_rows is neither 1 nor 128");
    if (empty(*m)) return RESHARD_OK;
    if (m->row_stride < rs::blocks_of(m->cols) * rs::kBlock || m->row_stride % 16)
      return bad(name, "row_stride is not a multiple of 16 that holds whole blocks of 128 columns");
    if (m->scale_stride < rs::blocks_of(m->cols) || m->scale_stride > kMaxSide)
      return bad(name, "scale_stride is below the blocks of a row");
    return RESHARD_OK;
  }
  return bad(name, kind == kPlain  ? "dtype is not F32, BF16 or F16"
                   : kind == kHeld ? "dtype is not FP8_E4M3 or FP8_E5M2"
                                   : "dtype is not F32, BF16, F16, FP8_E4M3 or FP8_E5M2");
}

// The bytes a matrix spans: rows of `width` bytes, `stride` apart.
struct Span {
  uintptr_t lo, hi;
  uintptr_t width, stride;
};
Span data_span(const reshard_matrix_t& m) {
  const int64_t cols = m.block_rows ? rs::blocks_of(m.cols) * rs::kBlock : m.cols, size = elem_size(m.dtype);
  const uintptr_t lo = reinterpret_cast<uintptr_t>(m.data);
  return Span{lo, lo + uintptr_t(((m.rows - 1) * m.row_stride + cols) * size), uintptr_t(cols * size),
              uintptr_t(m.row_stride * size)};
}
Span scale_span(const reshard_matrix_t& m) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(m.scales), width = uintptr_t(rs::blocks_of(m.cols));
  return Span{lo, lo + uintptr_t((rs::ceil_div(m.rows, m.block_rows) - 1) * m.scale_stride) + width, width,
              uintptr_t(m.scale_stride)};
}
// Whether two matrices share bytes.  Rows of one stride may lie between each
// other's (columns of one larger matrix); with different strides whole spans count.
bool overlap(const Span& a, const Span& b) {
  if (a.lo >= b.hi || b.lo >= a.hi) return false;
  if (a.stride != b.stride || !a.stride) return true;
  if (b.lo < a.lo) return overlap(b, a);
  const uintptr_t d = (b.lo - a.lo) % a.stride;
  return d < a.width || d + b.width > a.stride;
}

// Pointers and alignment of one matrix with elements (host only).
reshard_status_t check_pointers(const reshard_matrix_t& m, const char* name) {
  if (!m.data) return report(RESHARD_ERR_NULL_SHARD, std::string(name) + ": data is NULL");
  const uintptr_t align = m.block_rows ? 16 : uintptr_t(elem_size(m.dtype));
  if (reinterpret_cast<uintptr_t>(m.data) % align) return bad(name, "data is misaligned");
  if (m.block_rows && !m.scales) return report(RESHARD_ERR_NULL_SHARD, std::string(name) + ": scales is NULL");
  return RESHARD_OK;
}

struct Use {
  const reshard_matrix_t* m;
  const char* name;
  bool written;
};

reshard_status_t hip_fail(hipError_t e, const char* what) {
  return report(e == hipErrorOutOfMemory ? RESHARD_ERR_OUT_OF_MEMORY : RESHARD_ERR_HIP,
                std::string(what) + ": " + hipGetErrorString(e));
}

// Device memory that kernels on `dev` may use.
reshard_status_t check_memory(const void* p, const char* name, int dev) {
  hipPointerAttribute_t at;
  const hipError_t e = hipPointerGetAttributes(&at, p);
  if (e != hipSuccess) {
    (void)hipGetLastError();  // not an error of any launch
    return e == hipErrorInvalidValue ? bad(name, "not device memory") : hip_fail(e, "hipPointerGetAttributes");
  }
  if (at.type == hipMemoryTypeUnregistered || at.type == hipMemoryTypeHost) return bad(name, "not device memory");
  if (at.type == hipMemoryTypeDevice && at.device != dev)
    return report(RESHARD_ERR_DEVICE_MISMATCH, std::string(name) + " is on device " + std::to_string(at.device) +
                                                   ", current device is " + std::to_string(dev));
  return RESHARD_OK;
}

// Everything about the matrices of a call that have elements, and the stream.
reshard_status_t check_call(std::initializer_list<Use> uses, const void* workspace, int64_t need, int64_t given,
                            void* stream_arg) {
  for (const Use& u : uses)
    if (!empty(*u.m))
      if (const reshard_status_t s = check_pointers(*u.m, u.name)) return s;
  Span work{};
  if (given < need)
    return report(RESHARD_ERR_INVALID_ARGUMENT, "workspace of " + std::to_string(given) + " bytes, " +
                                                    std::to_string(need) + " needed");
  if (need) {
    if (!workspace) return report(RESHARD_ERR_INVALID_ARGUMENT, "workspace is NULL");
    work.lo = reinterpret_cast<uintptr_t>(workspace);
    work.hi = work.lo + uintptr_t(need);
    if (work.lo % 16) return report(RESHARD_ERR_INVALID_ARGUMENT, "workspace is misaligned");
  }
  for (const Use& w : uses) {
    if (empty(*w.m)) continue;
    const Span wd = data_span(*w.m), ws = w.m->block_rows ? scale_span(*w.m) : Span{};
    if (need && (overlap(wd, work) || overlap(ws, work))) return bad(w.name, "overlaps the workspace");
    if (!w.written) continue;
    if (w.m->block_rows && overlap(wd, ws)) return bad(w.name, "scales overlap the data");
    for (const Use& r : uses) {
      if (&r == &w || empty(*r.m)) continue;
      const Span rd = data_span(*r.m), rsc = r.m->block_rows ? scale_span(*r.m) : Span{};
      if (overlap(wd, rd) || overlap(wd, rsc) || overlap(ws, rd) || overlap(ws, rsc))
        return report(RESHARD_ERR_INVALID_ARGUMENT, std::string(w.name) + " overlaps " + r.name);
    }
  }
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (stream_arg) {
    hipDevice_t on = 0;
    e = hipStreamGetDevice(static_cast<hipStream_t>(stream_arg), &on);
    if (e != hipSuccess) return hip_fail(e, "hipStreamGetDevice");
    if (int(on) != dev)
      return report(RESHARD_ERR_DEVICE_MISMATCH, "stream is on device " + std::to_string(int(on)) +
                                                     ", current device is " + std::to_string(dev));
  }
  for (const Use& u : uses) {
    if (empty(*u.m)) continue;
    if (const reshard_status_t s = check_memory(u.m->data, u.name, dev)) return s;
    if (u.m->block_rows)
      if (const reshard_status_t s = check_memory(u.m->scales, u.name, dev)) return s;
  }
  if (need)
    if (const reshard_status_t s = check_memory(workspace, "workspace", dev)) return s;
  return RESHARD_OK;
}

reshard_status_t launched(hipError_t e, const char* what) {
  return e == hipSuccess ? RESHARD_OK : hip_fail(e, what);
}

reshard_status_t too_many() { return report(RESHARD_ERR_INVALID_ARGUMENT, "too many tiles for one launch"); }

reshard_status_t check_matmul(const reshard_matrix_t* a, const reshard_matrix_t* b, const reshard_matrix_t* out) {
  if (const reshard_status_t s = check_shape(a, "a", kAny)) return s;
  if (const reshard_status_t s = check_shape(b, "b", kHeld)) return s;
  if (const reshard_status_t s = check_shape(out, "out", kPlain)) return s;
  if (a->cols != b->cols) return report(RESHARD_ERR_INVALID_ARGUMENT, "a and b differ in columns (the contraction)");
  if (out->rows != a->rows || out->cols != b->rows)
    return report(RESHARD_ERR_INVALID_ARGUMENT, "out is not (rows of a) x (rows of b)");
  const rs::MatmulPlan p = rs::plan_matmul(*a, *b, *out);
  if (p.too_wide) return report(RESHARD_ERR_INVALID_ARGUMENT, "rows more than 2^23 bytes apart with more than 4 rows of a");
  if (p.groups > rs::kMaxGroups) return too_many();
  return RESHARD_OK;
}

reshard_status_t check_grad(const reshard_matrix_t* dy, const reshard_matrix_t* x, const reshard_matrix_t* dw) {
  if (const reshard_status_t s = check_shape(dy, "dy", kPlain)) return s;
  if (const reshard_status_t s = check_shape(x, "x", kHeld)) return s;
  if (const reshard_status_t s = check_shape(dw, "dw", kPlain)) return s;
  if (dy->rows != x->rows) return report(RESHARD_ERR_INVALID_ARGUMENT, "dy and x differ in rows (the contraction)");
  if (dw->rows != dy->cols || dw->cols != x->cols)
    return report(RESHARD_ERR_INVALID_ARGUMENT, "dw is not (columns of dy) x (columns of x)");
  if (dy->cols > rs::kMaxGradCols || dy->rows * rs::grad_planes(dy->dtype) > rs::kMaxGradRows)
    return bad("dy", "too many rows or columns for a weight gradient");
  if (rs::plan_grad(*dy, *x, *dw).groups > rs::kMaxGroups) return too_many();
  return RESHARD_OK;
}

// No exception may cross the C ABI (messages allocate).
template <typename F> reshard_status_t guarded(F call) {
  try {
    return call();
  } catch (...) {
    return RESHARD_ERR_OUT_OF_MEMORY;
  }
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
  if (dst->block_rows != 1 && rs::ceil_div(src->rows, rs::kBlock) * rs::blocks_of(src->cols) > rs::kMaxGroups)
    return too_many();
  const reshard_status_t s = dst_t ? check_call({{src, "src", false}, {dst, "dst", true}, {dst_t, "dst_t", true}},
                                                nullptr, 0, 0, stream)
                                   : check_call({{src, "src", false}, {dst, "dst", true}}, nullptr, 0, 0, stream);
  if (s) return s;
  if (empty(*src)) return RESHARD_OK;
  return launched(rs::launch_quantize(*src, *dst, dst_t, static_cast<hipStream_t>(stream)), "block quantize launch");
}

reshard_status_t block_dequantize(const reshard_matrix_t* src, const reshard_matrix_t* dst, void* stream) {
  if (const reshard_status_t s = check_shape(src, "src", kHeld)) return s;
  if (const reshard_status_t s = check_shape(dst, "dst", kPlain)) return s;
  if (dst->rows != src->rows || dst->cols != src->cols)
    return report(RESHARD_ERR_INVALID_ARGUMENT, "src and dst differ in shape");
  if (const reshard_status_t s = check_call({{src, "src", false}, {dst, "dst", true}}, nullptr, 0, 0, stream)) return s;
  if (empty(*src)) return RESHARD_OK;
  return launched(rs::launch_dequantize(*src, *dst, static_cast<hipStream_t>(stream)), "block dequantize launch");
}

reshard_status_t block_matmul(const reshard_matrix_t* a, const reshard_matrix_t* b, const reshard_matrix_t* out,
                              void* workspace, int64_t workspace_bytes, void* stream) {
  if (const reshard_status_t s = check_matmul(a, b, out)) return s;
  const rs::MatmulPlan plan = rs::plan_matmul(*a, *b, *out);
  if (const reshard_status_t s = check_call({{a, "a", false}, {b, "b", false}, {out, "out", true}}, workspace,
                                            plan.bytes(), workspace_bytes, stream))
    return s;
  if (empty(*out)) return RESHARD_OK;
  return launched(rs::launch_matmul(plan, *a, *b, *out, workspace, static_cast<hipStream_t>(stream)),
                  "block matmul launch");
}

reshard_status_t block_grad(const reshard_matrix_t* dy, const reshard_matrix_t* x, const reshard_matrix_t* dw,
                            int accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
  if (const reshard_status_t s = check_grad(dy, x, dw)) return s;
  const rs::GradPlan plan = rs::plan_grad(*dy, *x, *dw);
  if (const reshard_status_t s = check_call({{dy, "dy", false}, {x, "x", false}, {dw, "dw", true}}, workspace,
                                            plan.bytes(), workspace_bytes, stream))
    return s;
  if (empty(*dw)) return RESHARD_OK;
  return launched(rs::launch_grad(plan, *dy, *x, *dw, accumulate != 0, workspace, static_cast<hipStream_t>(stream)),
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
    *bytes = rs::plan_matmul(*a, *b, *out).bytes();
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
    *bytes = rs::plan_grad(*dy, *x, *dw).bytes();
    return RESHARD_OK;
  });
}

reshard_status_t reshard_block_grad(const reshard_matrix_t* dy, const reshard_matrix_t* x, const reshard_matrix_t* dw,
                                    int accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&] { return block_grad(dy, x, dw, accumulate, workspace, workspace_bytes, stream); });
}

}  // extern "C"
