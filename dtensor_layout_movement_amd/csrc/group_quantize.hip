// Quantizing to and reading back from group-scaled 4-bit matrices (the format is in
// reshard.h).  Both are bound by HBM: each element is read and written once.
#include "block_device.h"
#include "groups.h"

#include <algorithm>

namespace rs {
namespace {

constexpr int kThreads = 256;
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Where a group-scaled matrix lies (strides in bytes).
struct Packed {
  uint8_t* data;
  int64_t stride;
  uint8_t* scales;
  int64_t scale_stride;
};
Packed packed(const reshard_matrix_t& m, int64_t row) {
  return Packed{static_cast<uint8_t*>(m.data) + row * (m.row_stride / 2), m.row_stride / 2,
                static_cast<uint8_t*>(m.scales) + row * m.scale_stride, m.scale_stride};
}

// The scale byte of a group whose largest magnitude has bits `amax`: with amax = m *
// 2^x, 1 <= m < 2, the largest value being 1.5 * 2^2, the exponent is x - 2, one more
// where m > 1.5, and at least -127.  Infinities and NaN give 255.
__device__ __forceinline__ uint32_t group_scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255;
  if (amax == 0) return 127;
  return uint32_t(max(int(amax >> 23) - 2 + ((amax & 0x7fffffu) > 0x400000u ? 1 : 0), 0));
}

// Eight elements times `inv` (exact, or too small to matter) in 4 bits, the first lowest.
__device__ __forceinline__ uint32_t quantize8_fp4(const float* x, float inv) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[0] * inv, x[1] * inv, 1.f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[2] * inv, x[3] * inv, 1.f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[4] * inv, x[5] * inv, 1.f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[6] * inv, x[7] * inv, 1.f, 3);
}

// Four lanes a group, eight elements a lane; workgroups dealt to the XCDs in contiguous
// runs, whose neighbouring scale bytes meet in one L2.  14336 x 4096 fp32 takes 50 us, 5.3 TB/s
// of reads and writes, 5000 x 3001 bf16, whose rows start off the 16-byte grid, 8.7 (4.4).
template <int DT>
__global__ __launch_bounds__(kThreads) void quantize_groups(const typename Elem<DT>::type* src, int64_t stride, int cols,
                                                            Divisor groups, uint32_t items, Packed dst) {
  const int part = threadIdx.x & 3;
  const uint32_t i = run_of(blockIdx.x, gridDim.x) * (kThreads / 4) + (threadIdx.x >> 2);
  if (i >= items) return;  // whole groups of four lanes
  const uint32_t row = quotient(i, groups), group = i - row * groups.d;
  float x[8];
  load_up<DT, 8>(src + int64_t(row) * stride, int(group) * kGroup + part * 8, cols, x);
  uint32_t amax = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) amax = max(amax, __builtin_bit_cast(uint32_t, x[k]) & 0x7fffffffu);
  amax = max_with<0xb1>(amax);
  amax = max_with<0x4e>(amax);
  const uint32_t s = group_scale_byte(amax);
  const uint32_t q = s == 255 ? 0 : quantize8_fp4(x, inverse_scale(s));
  *reinterpret_cast<uint32_t*>(dst.data + int64_t(row) * dst.stride + group * (kGroup / 2) + part * 4) = q;
  if (part == 0) dst.scales[int64_t(row) * dst.scale_stride + group] = uint8_t(s);
}

// As many elements a lane as make 16 bytes of output, so that a wave's stores are
// contiguous, kBack pieces a lane whose loads are under way together, stores past the
// caches.  14336 x 4096 to bf16 takes 22 us (6.7 TB/s with the payload still in the last-level
// cache), 5000 x 3001 8.0.
constexpr int kBack = 2;

template <int DT>
__global__ __launch_bounds__(kThreads) void dequantize_groups(Packed src, Divisor chunks, uint32_t items,
                                                              typename Elem<DT>::type* dst, int64_t stride, int cols) {
  typedef typename Elem<DT>::type T;
  constexpr int N = 16 / sizeof(T);
  const uint32_t first = blockIdx.x * (kThreads * kBack) + threadIdx.x;
  uint32_t q[kBack], s[kBack], row[kBack];
  int c[kBack];
#pragma unroll
  for (int u = 0; u < kBack; ++u) {
    const uint32_t i = min(first + u * kThreads, items - 1);
    row[u] = quotient(i, chunks);
    c[u] = int(i - row[u] * chunks.d) * N;
    const uint8_t* p = src.data + int64_t(row[u]) * src.stride + c[u] / 2;
    q[u] = N == 8 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
    s[u] = src.scales[int64_t(row[u]) * src.scale_stride + c[u] / kGroup];
  }
#pragma unroll
  for (int u = 0; u < kBack; ++u) {
    if (first + u * kThreads >= items) break;
    const float f = scale_value(s[u]);
    f32x2 w[4];
    w[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 0);
    w[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 1);
    w[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 2);
    w[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 3);
    Pack<T, N> v;
#pragma unroll
    for (int k = 0; k < N; ++k) v.v[k] = Elem<DT>::down(w[k / 2][k % 2] * f);
    T* p = dst + int64_t(row[u]) * stride + c[u];
    if (c[u] + N <= cols) {
      store_stream<T, N>(p, v);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (c[u] + k < cols) p[k] = v.v[k];
    }
  }
}

template <int DT>
hipError_t quantize_as(const reshard_matrix_t& src, const reshard_matrix_t& dst, hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const uint32_t groups = uint32_t(groups_of(src.cols));
  const int64_t rows = rows_per_launch(groups, kThreads / 4);
  for (int64_t r = 0; r < src.rows; r += rows) {
    const uint32_t items = uint32_t(std::min(rows, src.rows - r) * groups);
    quantize_groups<DT><<<dim3(uint32_t(ceil_div(items, kThreads / 4))), kThreads, 0, stream>>>(
        static_cast<const T*>(src.data) + r * src.row_stride, src.row_stride, int(src.cols), divisor(groups), items,
        packed(dst, r));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT>
hipError_t dequantize_as(const reshard_matrix_t& src, const reshard_matrix_t& dst, hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const uint32_t chunks = uint32_t(ceil_div(src.cols, 16 / sizeof(T)));
  const int64_t rows = rows_per_launch(chunks, kThreads * kBack);
  for (int64_t r = 0; r < src.rows; r += rows) {
    const uint32_t items = uint32_t(std::min(rows, src.rows - r) * chunks);
    dequantize_groups<DT><<<dim3(uint32_t(ceil_div(items, kThreads * kBack))), kThreads, 0, stream>>>(
        packed(src, r), divisor(chunks), items, static_cast<T*>(dst.data) + r * dst.row_stride, dst.row_stride,
        int(dst.cols));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_group_quantize(const reshard_matrix_t& src, const reshard_matrix_t& dst, hipStream_t stream) {
  switch (src.dtype) {
    case RESHARD_DTYPE_F32: return quantize_as<RESHARD_DTYPE_F32>(src, dst, stream);
    case RESHARD_DTYPE_BF16: return quantize_as<RESHARD_DTYPE_BF16>(src, dst, stream);
    default: return quantize_as<RESHARD_DTYPE_F16>(src, dst, stream);
  }
}

hipError_t launch_group_dequantize(const reshard_matrix_t& src, const reshard_matrix_t& dst, hipStream_t stream) {
  switch (dst.dtype) {
    case RESHARD_DTYPE_F32: return dequantize_as<RESHARD_DTYPE_F32>(src, dst, stream);
    case RESHARD_DTYPE_BF16: return dequantize_as<RESHARD_DTYPE_BF16>(src, dst, stream);
    default: return dequantize_as<RESHARD_DTYPE_F16>(src, dst, stream);
  }
}

}  // namespace rs
