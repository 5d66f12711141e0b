// dw = dy^T x^ from an 8-bit checkpoint x (the format is in reshard.h).
#include "block_device.h"
#include "blocks.h"

namespace rs {
namespace {

constexpr int kTile = 64;     // rows and columns of dw a workgroup makes
constexpr int kDepth = 32;    // rows of dy and x a step takes
constexpr int kPitch = kDepth + 8;
constexpr int kThreads = 256;

struct Checkpoint {
  const uint8_t* data;
  int64_t stride;
  const uint8_t* scales;
  int64_t scale_stride;
  int row_shift;
};

// Part p of a value as bfloat16 bits: the leading 8 significant bits, the next 8,
// the last 8, each cut off exactly, so that the parts add up to the value.
template <int PARTS> __device__ __forceinline__ uint16_t part_of(float v, int p) {
  uint32_t bits = __builtin_bit_cast(uint32_t, v);
  if (PARTS == 1) return uint16_t(bits >> 16);
  if ((bits & 0x7fffffffu) > 0x7f800000u) bits |= 0x00400000u;  // a NaN whose payload lies in the low bits
  const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const uint32_t hi = bits & 0xffff0000u;
    if (i == p) return uint16_t(hi >> 16);
    bits = finite ? __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, bits) - __builtin_bit_cast(float, hi)) : 0u;
  }
  return 0;
}

// The simple form: 64 x 64 tiles of dw, both operands staged through LDS with the
// contraction (the rows of dy and x) turned inwards, four waves of 16 x 64.
template <int DT_Y, int DT_W, bool E5M2>
__global__ __launch_bounds__(kThreads) void grad_tiles(const typename Elem<DT_Y>::type* dy, int64_t dy_stride,
                                                       Checkpoint x, int rows, int n_cols, int k_cols,
                                                       uint32_t k_tiles, typename Elem<DT_W>::type* dw,
                                                       int64_t dw_stride, int accumulate) {
  constexpr int kParts = DT_Y == RESHARD_DTYPE_BF16 ? 1 : DT_Y == RESHARD_DTYPE_F16 ? 2 : 3;
  __shared__ __align__(16) uint16_t ys[kTile * kPitch];
  __shared__ __align__(16) uint16_t xs[kTile * kPitch];
  const int n0 = int(blockIdx.x / k_tiles) * kTile, k0 = int(blockIdx.x % k_tiles) * kTile;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  f32x4 acc[4] = {};
  for (int m0 = 0; m0 < rows; m0 += kDepth) {
    for (int part = 0; part < kParts; ++part) {
      __syncthreads();
      for (int i = threadIdx.x; i < kTile * kDepth; i += kThreads) {
        const int c = i % kTile, r = i / kTile, m = m0 + r;
        uint16_t v = 0;
        if (m < rows && n0 + c < n_cols) v = part_of<kParts>(Elem<DT_Y>::up(dy[m * dy_stride + n0 + c]), part);
        ys[c * kPitch + r] = v;
        if (part == 0) {
          float f = 0.f;
          if (m < rows && k0 + c < k_cols) {
            const uint32_t q = x.data[m * x.stride + k0 + c];
            f = widen4<E5M2>(q)[0] *
                scale_value(x.scales[int64_t(m >> x.row_shift) * x.scale_stride + (k0 + c) / kBlock]);
          }
          xs[c * kPitch + r] = __builtin_bit_cast(uint16_t, __bf16(f));
        }
      }
      __syncthreads();
      const int at = (lane & 15) * kPitch + (lane >> 4) * 8;
      const bf16x8 u = *reinterpret_cast<const bf16x8*>(ys + wave * 16 * kPitch + at);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
            *reinterpret_cast<const bf16x8*>(xs + t * 16 * kPitch + at), u, acc[t], 0, 0, 0);
    }
  }
  const int n = n0 + wave * 16 + (lane & 15);
  if (n >= n_cols) return;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + t * 16 + (lane >> 4) * 4 + i;
      if (k >= k_cols) continue;
      typename Elem<DT_W>::type* p = dw + n * dw_stride + k;
      const float f = acc[t][i];
      *p = Elem<DT_W>::down(accumulate ? Elem<DT_W>::up(*p) + f : f);
    }
  }
}

template <int DT_Y, int DT_W, bool E5M2>
hipError_t grad_as(const GradPlan& plan, const reshard_matrix_t& dy, const reshard_matrix_t& x,
                   const reshard_matrix_t& dw, bool accumulate, hipStream_t stream) {
  const Checkpoint c{static_cast<const uint8_t*>(x.data), x.row_stride, static_cast<const uint8_t*>(x.scales),
                     x.scale_stride, x.block_rows == 1 ? 0 : 7};
  grad_tiles<DT_Y, DT_W, E5M2><<<dim3(uint32_t(plan.groups)), kThreads, 0, stream>>>(
      static_cast<const typename Elem<DT_Y>::type*>(dy.data), dy.row_stride, c, int(dy.rows), int(dy.cols),
      int(x.cols), uint32_t(ceil_div(x.cols, kTile)), static_cast<typename Elem<DT_W>::type*>(dw.data), dw.row_stride,
      accumulate ? 1 : 0);
  return hipGetLastError();
}

template <int DT_Y, int DT_W>
hipError_t grad_format(const GradPlan& plan, const reshard_matrix_t& dy, const reshard_matrix_t& x,
                       const reshard_matrix_t& dw, bool accumulate, hipStream_t stream) {
  return x.dtype == RESHARD_DTYPE_FP8_E5M2 ? grad_as<DT_Y, DT_W, true>(plan, dy, x, dw, accumulate, stream)
                                           : grad_as<DT_Y, DT_W, false>(plan, dy, x, dw, accumulate, stream);
}

template <int DT_Y>
hipError_t grad_out(const GradPlan& plan, const reshard_matrix_t& dy, const reshard_matrix_t& x,
                    const reshard_matrix_t& dw, bool accumulate, hipStream_t stream) {
  switch (dw.dtype) {
    case RESHARD_DTYPE_F32: return grad_format<DT_Y, RESHARD_DTYPE_F32>(plan, dy, x, dw, accumulate, stream);
    case RESHARD_DTYPE_BF16: return grad_format<DT_Y, RESHARD_DTYPE_BF16>(plan, dy, x, dw, accumulate, stream);
    default: return grad_format<DT_Y, RESHARD_DTYPE_F16>(plan, dy, x, dw, accumulate, stream);
  }
}

}  // namespace

GradPlan plan_grad(const reshard_matrix_t& dy, const reshard_matrix_t& x, const reshard_matrix_t& dw) {
  GradPlan p;
  p.groups = ceil_div(dy.cols, kTile) * ceil_div(x.cols, kTile);
  return p;
}

hipError_t launch_grad(const GradPlan& plan, const reshard_matrix_t& dy, const reshard_matrix_t& x,
                       const reshard_matrix_t& dw, bool accumulate, void* workspace, hipStream_t stream) {
  switch (dy.dtype) {
    case RESHARD_DTYPE_F32: return grad_out<RESHARD_DTYPE_F32>(plan, dy, x, dw, accumulate, stream);
    case RESHARD_DTYPE_BF16: return grad_out<RESHARD_DTYPE_BF16>(plan, dy, x, dw, accumulate, stream);
    default: return grad_out<RESHARD_DTYPE_F16>(plan, dy, x, dw, accumulate, stream);
  }
}

}  // namespace rs
