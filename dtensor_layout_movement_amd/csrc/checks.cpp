// Argument checks shared by the calls over matrices in device memory.
#include "checks.h"

#include "blocks.h"
#include "groups.h"

namespace rs {
namespace {

constexpr int64_t kMaxSide = int64_t(1) << 30;
constexpr int64_t kMaxElems = int64_t(1) << 56;  // rows * row_stride, far beyond any memory

int64_t elem_size(int dtype) { return dtype == RESHARD_DTYPE_F32 ? 4 : is_plain(dtype) ? 2 : 1; }

// Bytes of a row and between rows of a matrix's data.
int64_t row_bytes(const reshard_matrix_t& m) {
  if (is_grouped(m.dtype)) return groups_of(m.cols) * (kGroup / 2);
  return (m.block_rows ? blocks_of(m.cols) * kBlock : m.cols) * elem_size(m.dtype);
}
int64_t stride_bytes(const reshard_matrix_t& m) {
  return is_grouped(m.dtype) ? m.row_stride / 2 : m.row_stride * elem_size(m.dtype);
}

// The bytes something spans: rows of `width` bytes, `stride` apart.
struct Span {
  uintptr_t lo, hi;
  uintptr_t width, stride;
};
Span data_span(const reshard_matrix_t& m) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(m.data), width = uintptr_t(row_bytes(m));
  return Span{lo, lo + uintptr_t((m.rows - 1) * stride_bytes(m)) + width, width, uintptr_t(stride_bytes(m))};
}
Span scale_span(const reshard_matrix_t& m) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(m.scales),
                  width = uintptr_t(is_grouped(m.dtype) ? groups_of(m.cols) : blocks_of(m.cols));
  return Span{lo, lo + uintptr_t((ceil_div(m.rows, m.block_rows) - 1) * m.scale_stride) + width, width,
              uintptr_t(m.scale_stride)};
}
Span array_span(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{lo, lo + uintptr_t(bytes), uintptr_t(bytes), 0};
}
// Whether two of them share bytes.  Rows of one stride may lie between each
// other's (columns of one larger matrix); with different strides whole spans count.
bool overlap(const Span& a, const Span& b) {
  if (a.lo >= b.hi || b.lo >= a.hi) return false;
  if (a.stride != b.stride || !a.stride) return true;
  if (b.lo < a.lo) return overlap(b, a);
  const uintptr_t d = (b.lo - a.lo) % a.stride;
  return d < a.width || d + b.width > a.stride;
}

// A matrix or an array with elements, as the overlap checks see it.
struct Region {
  const char* name;
  bool written;
  Span data, scales;  // scales empty (lo = hi = 0) where there are none
};

// Pointers and alignment of one matrix with elements (host only).
reshard_status_t check_pointers(const reshard_matrix_t& m, const char* name) {
  if (!m.data) return report(RESHARD_ERR_NULL_SHARD, std::string(name) + ": data is NULL");
  const uintptr_t align = m.block_rows ? 16 : uintptr_t(elem_size(m.dtype));
  if (reinterpret_cast<uintptr_t>(m.data) % align) return bad(name, "data is misaligned");
  if (m.block_rows && !m.scales) return report(RESHARD_ERR_NULL_SHARD, std::string(name) + ": scales is NULL");
  return RESHARD_OK;
}

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

}  // namespace

reshard_status_t bad(const char* name, const char* what) {
  return report(RESHARD_ERR_INVALID_ARGUMENT, std::string(name) + ": " + what);
}
reshard_status_t too_many() { return report(RESHARD_ERR_INVALID_ARGUMENT, "too many tiles for one launch"); }

bool is_plain(int dtype) {
  return dtype == RESHARD_DTYPE_F32 || dtype == RESHARD_DTYPE_BF16 || dtype == RESHARD_DTYPE_F16;
}
bool is_held(int dtype) { return dtype == RESHARD_DTYPE_FP8_E4M3 || dtype == RESHARD_DTYPE_FP8_E5M2; }
bool is_grouped(int dtype) { return dtype == RESHARD_DTYPE_FP4_E2M1; }

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
    if (m->row_stride < blocks_of(m->cols) * kBlock || m->row_stride % 16)
      return bad(name, "row_stride is not a multiple of 16 that holds whole blocks of 128 columns");
    if (m->scale_stride < blocks_of(m->cols) || m->scale_stride > kMaxSide)
      return bad(name, "scale_stride is below the blocks of a row");
    return RESHARD_OK;
  }
  if (is_grouped(m->dtype) && (kind & kGrouped)) {
    if (m->block_rows != 1) return bad(name, "a group-scaled matrix has block_rows 1");
    if (empty(*m)) return RESHARD_OK;
    if (m->row_stride < groups_of(m->cols) * kGroup || m->row_stride % kGroup)
      return bad(name, "row_stride is not a multiple of 32 that holds whole groups of 32 columns");
    if (m->scale_stride < groups_of(m->cols) || m->scale_stride > kMaxSide)
      return bad(name, "scale_stride is below the groups of a row");
    return RESHARD_OK;
  }
  return bad(name, kind == kPlain     ? "dtype is not F32, BF16 or F16"
                   : kind == kHeld    ? "dtype is not FP8_E4M3 or FP8_E5M2"
                   : kind == kGrouped ? "dtype is not FP4_E2M1"
                                      : "dtype is not F32, BF16, F16, FP8_E4M3 or FP8_E5M2");
}

reshard_status_t check_call(std::initializer_list<Use> uses, std::initializer_list<Array> arrays, const void* workspace,
                            int64_t need, int64_t given, void* stream_arg) {
  Region regions[2 * kMaxUses];
  int n = 0;
  for (const Use& u : uses) {
    if (empty(*u.m)) continue;
    if (const reshard_status_t s = check_pointers(*u.m, u.name)) return s;
    regions[n++] = Region{u.name, u.written, data_span(*u.m), u.m->block_rows ? scale_span(*u.m) : Span{}};
  }
  for (const Array& a : arrays) {
    if (a.bytes == 0) continue;
    if (!a.data) return report(RESHARD_ERR_NULL_SHARD, std::string(a.name) + " is NULL");
    if (reinterpret_cast<uintptr_t>(a.data) % a.align) return bad(a.name, "misaligned");
    regions[n++] = Region{a.name, a.written, array_span(a.data, a.bytes), Span{}};
  }
  Span work{};
  if (given < need)
    return report(RESHARD_ERR_INVALID_ARGUMENT, "workspace of " + std::to_string(given) + " bytes, " +
                                                    std::to_string(need) + " needed");
  if (need) {
    if (!workspace) return report(RESHARD_ERR_INVALID_ARGUMENT, "workspace is NULL");
    work = array_span(workspace, need);
    if (work.lo % 16) return report(RESHARD_ERR_INVALID_ARGUMENT, "workspace is misaligned");
  }
  for (int i = 0; i < n; ++i) {
    const Region& w = regions[i];
    if (need && (overlap(w.data, work) || overlap(w.scales, work))) return bad(w.name, "overlaps the workspace");
    if (!w.written) continue;
    if (overlap(w.data, w.scales)) return bad(w.name, "scales overlap the data");
    for (int j = 0; j < n; ++j) {
      const Region& r = regions[j];
      if (i == j) continue;
      if (overlap(w.data, r.data) || overlap(w.data, r.scales) || overlap(w.scales, r.data) || overlap(w.scales, r.scales))
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
  for (int i = 0; i < n; ++i) {
    const Region& r = regions[i];
    if (const reshard_status_t s = check_memory(reinterpret_cast<const void*>(r.data.lo), r.name, dev)) return s;
    if (r.scales.hi)
      if (const reshard_status_t s = check_memory(reinterpret_cast<const void*>(r.scales.lo), r.name, dev)) return s;
  }
  if (need)
    if (const reshard_status_t s = check_memory(workspace, "workspace", dev)) return s;
  return RESHARD_OK;
}

reshard_status_t launched(hipError_t e, const char* what) { return e == hipSuccess ? RESHARD_OK : hip_fail(e, what); }

}  // namespace rs
