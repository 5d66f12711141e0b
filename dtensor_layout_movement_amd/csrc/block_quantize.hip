// Quantizing to and reading back from block-scaled 8-bit matrices (the format is
// in reshard.h).  Both directions are bound by HBM: each element is read and
// written once.
#include "block_device.h"
#include "blocks.h"

namespace rs {
namespace {

constexpr int kThreads = 256;

// Where a block-scaled matrix lies.
struct Held {
  uint8_t* data;
  int64_t stride;
  uint8_t* scales;
  int64_t scale_stride;
};

Held held(const reshard_matrix_t& m) {
  return Held{static_cast<uint8_t*>(m.data), m.row_stride, static_cast<uint8_t*>(m.scales), m.scale_stride};
}

// 16 elements of row p from column c on as binary32, zero past `cols`.
template <int DT> __device__ __forceinline__ void load16(const typename Elem<DT>::type* p, int c, int cols, float* x) {
  typedef typename Elem<DT>::type T;
  if (c + 16 <= cols) {
    const Pack<T, 16> v = load_pack<T, 16>(p + c);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = Elem<DT>::up(v.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = c + i < cols ? Elem<DT>::up(p[c + i]) : 0.f;
  }
}

template <bool E5M2> __device__ __forceinline__ i32x4 quantize16(const float* x, float inv) {
  i32x4 q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = int(quantize4<E5M2>(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], inv));
  return q;
}

// Blocks of 1 x 128: eight lanes a block, 16 elements a lane, so that a lane
// stores 16 payload bytes; the block's largest magnitude goes round by three
// exchanges.
template <int DT, bool E5M2>
__global__ __launch_bounds__(kThreads) void quantize_rows(const typename Elem<DT>::type* src, int64_t stride, int cols,
                                                          uint32_t blocks, int64_t items, Held dst) {
  const int part = threadIdx.x & 7;
  const int64_t step = int64_t(gridDim.x) * (kThreads / 8);
  for (int64_t i = int64_t(blockIdx.x) * (kThreads / 8) + (threadIdx.x >> 3); i < items; i += step) {
    const int64_t r = i / blocks;
    const uint32_t b = uint32_t(i - r * blocks);
    const int c = int(b) * kBlock + part * 16;
    float x[16];
    load16<DT>(src + r * stride, c, cols, x);
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) amax = max(amax, finite_magnitude(x[k]));
#pragma unroll
    for (int m = 1; m < 8; m *= 2) amax = max(amax, uint32_t(__shfl_xor(int(amax), m)));
    const uint32_t s = scale_byte<E5M2>(amax);
    *reinterpret_cast<i32x4*>(dst.data + r * dst.stride + c) = quantize16<E5M2>(x, inverse_scale(s));
    if (part == 0) dst.scales[r * dst.scale_stride + b] = uint8_t(s);
  }
}

// Blocks of 128 x 128: a workgroup a block, eight lanes a row, four passes of 32
// rows held in registers until the block's scale is known.  The transpose goes
// through LDS a byte at a time.
constexpr int kTPitch = 132;

template <int DT, bool E5M2, bool TRANSPOSE>
__global__ __launch_bounds__(kThreads) void quantize_squares(const typename Elem<DT>::type* src, int64_t stride,
                                                             int rows, int cols, uint32_t blocks, Held dst,
                                                             Held dst_t) {
  __shared__ uint32_t wave_max[kThreads / 64];
  __shared__ uint32_t tile[TRANSPOSE ? kBlock * kTPitch / 4 : 1];
  const int R = int(blockIdx.x / blocks), C = int(blockIdx.x % blocks);
  const int part = threadIdx.x & 7, lane_row = threadIdx.x >> 3;
  const int c = C * kBlock + part * 16;
  float x[4][16];
  uint32_t amax = 0;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int r = R * kBlock + p * 32 + lane_row;
    if (r < rows) {
      load16<DT>(src + int64_t(r) * stride, c, cols, x[p]);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) x[p][k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) amax = max(amax, finite_magnitude(x[p][k]));
  }
#pragma unroll
  for (int m = 1; m < 64; m *= 2) amax = max(amax, uint32_t(__shfl_xor(int(amax), m)));
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) amax = max(amax, wave_max[w]);
  const uint32_t s = scale_byte<E5M2>(amax);
  const float inv = inverse_scale(s);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int row = p * 32 + lane_row, r = R * kBlock + row;
    const i32x4 q = quantize16<E5M2>(x[p], inv);
    if (r < rows) *reinterpret_cast<i32x4*>(dst.data + int64_t(r) * dst.stride + c) = q;
    if (TRANSPOSE) {
#pragma unroll
      for (int k = 0; k < 4; ++k) tile[(row * kTPitch + part * 16) / 4 + k] = uint32_t(q[k]);
    }
  }
  if (threadIdx.x == 0) {
    dst.scales[int64_t(R) * dst.scale_stride + C] = uint8_t(s);
    if (TRANSPOSE) dst_t.scales[int64_t(C) * dst_t.scale_stride + R] = uint8_t(s);
  }
  if (TRANSPOSE) {
    __syncthreads();
    const uint8_t* bytes = reinterpret_cast<const uint8_t*>(tile);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int col = p * 32 + lane_row;
      if (C * kBlock + col >= cols) continue;
      i32x4 q;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) w |= uint32_t(bytes[(part * 16 + 4 * k + j) * kTPitch + col]) << (8 * j);
        q[k] = int(w);
      }
      *reinterpret_cast<i32x4*>(dst_t.data + int64_t(C * kBlock + col) * dst_t.stride + R * kBlock + part * 16) = q;
    }
  }
}

// Reading back: 16 elements a lane.
template <int DT, bool E5M2>
__global__ __launch_bounds__(kThreads) void dequantize_rows(Held src, int row_shift, uint32_t chunks, int64_t items,
                                                            typename Elem<DT>::type* dst, int64_t stride, int cols) {
  typedef typename Elem<DT>::type T;
  const int64_t step = int64_t(gridDim.x) * kThreads;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < items; i += step) {
    const int64_t r = i / chunks;
    const int c = int(uint32_t(i - r * chunks)) * 16;
    const i32x4 q = *reinterpret_cast<const i32x4*>(src.data + r * src.stride + c);
    const float s = scale_value(src.scales[(r >> row_shift) * src.scale_stride + c / kBlock]);
    Pack<T, 16> v;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const f32x4 f = widen4<E5M2>(uint32_t(q[k]));
#pragma unroll
      for (int j = 0; j < 4; ++j) v.v[4 * k + j] = Elem<DT>::down(f[j] * s);
    }
    T* p = dst + r * stride + c;
    if (c + 16 <= cols) {
      store_pack<T, 16>(p, v);
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (c + k < cols) p[k] = v.v[k];
    }
  }
}

template <int DT, bool E5M2>
hipError_t quantize_as(const reshard_matrix_t& src, const reshard_matrix_t& dst, const reshard_matrix_t* dst_t,
                       hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const T* p = static_cast<const T*>(src.data);
  const uint32_t blocks = uint32_t(blocks_of(src.cols));
  if (dst.block_rows == 1) {
    const int64_t items = src.rows * blocks;
    const int64_t groups = std::min<int64_t>(ceil_div(items, kThreads / 8), kMaxGroups);
    quantize_rows<DT, E5M2><<<dim3(uint32_t(groups)), kThreads, 0, stream>>>(p, src.row_stride, int(src.cols), blocks,
                                                                              items, held(dst));
    return hipGetLastError();
  }
  const dim3 grid(uint32_t(ceil_div(src.rows, kBlock) * blocks));
  if (dst_t)
    quantize_squares<DT, E5M2, true><<<grid, kThreads, 0, stream>>>(p, src.row_stride, int(src.rows), int(src.cols),
                                                                    blocks, held(dst), held(*dst_t));
  else
    quantize_squares<DT, E5M2, false><<<grid, kThreads, 0, stream>>>(p, src.row_stride, int(src.rows), int(src.cols),
                                                                     blocks, held(dst), Held{});
  return hipGetLastError();
}

template <int DT, bool E5M2>
hipError_t dequantize_as(const reshard_matrix_t& src, const reshard_matrix_t& dst, hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const uint32_t chunks = uint32_t(ceil_div(src.cols, 16));
  const int64_t items = src.rows * chunks;
  const int64_t groups = std::min<int64_t>(ceil_div(items, kThreads), kMaxGroups);
  dequantize_rows<DT, E5M2><<<dim3(uint32_t(groups)), kThreads, 0, stream>>>(
      held(src), src.block_rows == 1 ? 0 : 7, chunks, items, static_cast<T*>(dst.data), dst.row_stride, int(dst.cols));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(const reshard_matrix_t& src, const reshard_matrix_t& dst, const reshard_matrix_t* dst_t,
                           hipStream_t stream) {
  const bool e5m2 = dst.dtype == RESHARD_DTYPE_FP8_E5M2;
  switch (src.dtype) {
    case RESHARD_DTYPE_F32:
      return e5m2 ? quantize_as<RESHARD_DTYPE_F32, true>(src, dst, dst_t, stream)
                  : quantize_as<RESHARD_DTYPE_F32, false>(src, dst, dst_t, stream);
    case RESHARD_DTYPE_BF16:
      return e5m2 ? quantize_as<RESHARD_DTYPE_BF16, true>(src, dst, dst_t, stream)
                  : quantize_as<RESHARD_DTYPE_BF16, false>(src, dst, dst_t, stream);
    default:
      return e5m2 ? quantize_as<RESHARD_DTYPE_F16, true>(src, dst, dst_t, stream)
                  : quantize_as<RESHARD_DTYPE_F16, false>(src, dst, dst_t, stream);
  }
}

hipError_t launch_dequantize(const reshard_matrix_t& src, const reshard_matrix_t& dst, hipStream_t stream) {
  const bool e5m2 = src.dtype == RESHARD_DTYPE_FP8_E5M2;
  switch (dst.dtype) {
    case RESHARD_DTYPE_F32:
      return e5m2 ? dequantize_as<RESHARD_DTYPE_F32, true>(src, dst, stream)
                  : dequantize_as<RESHARD_DTYPE_F32, false>(src, dst, stream);
    case RESHARD_DTYPE_BF16:
      return e5m2 ? dequantize_as<RESHARD_DTYPE_BF16, true>(src, dst, stream)
                  : dequantize_as<RESHARD_DTYPE_BF16, false>(src, dst, stream);
    default:
      return e5m2 ? dequantize_as<RESHARD_DTYPE_F16, true>(src, dst, stream)
                  : dequantize_as<RESHARD_DTYPE_F16, false>(src, dst, stream);
  }
}

}  // namespace rs
