// out = a^ b^T over block-scaled 8-bit matrices (the format is in reshard.h).
#include "block_device.h"
#include "blocks.h"

namespace rs {
namespace {

// An operand as the kernels read it: rows of 8-bit elements contiguous along the
// contraction, scales by block.
struct Operand {
  const uint8_t* data;
  int64_t stride;
  const uint8_t* scales;
  int64_t scale_stride;
  int rows;
  int row_shift;  // log2 of the rows of a scale block: 0 or 7
};

Operand operand(const reshard_matrix_t& m) {
  return Operand{static_cast<const uint8_t*>(m.data),   m.row_stride,   static_cast<const uint8_t*>(m.scales),
                 m.scale_stride, int(m.rows), m.block_rows == 1 ? 0 : 7};
}

// One 16 x 16 tile's step over 128 columns.  With 16-bit results the scaled
// matrix instruction takes the payload and the scale bytes as they are.  It
// aligns the products of one instruction to the largest of them and drops what
// is shifted out: relative to the result's norm 1.6e-5 was measured on normal
// values (contraction 4096) and 7.5e-5 with large channels, against 2^-9 and
// 2^-12 of rounding the result.  For F32 results the elements are widened to
// bfloat16, which holds them exactly, and go through four bfloat16
// instructions, whose products and sums lose nothing above binary32's
// rounding (8e-8 in the same test).  Each lane holds 32 consecutive elements of
// its row, on both sides, so the order within the step is the same for both.
template <bool EXACT, bool E5_1, bool E5_2>
__device__ __forceinline__ f32x4 step128(const i32x8& x, uint32_t sx, const i32x8& y, uint32_t sy, f32x4 acc) {
  if (!EXACT)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, E5_1 ? 1 : 0, E5_2 ? 1 : 0, 0, int(sx), 0,
                                                            int(sy));
  const float fx = scale_value(sx), fy = scale_value(sy);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8_bf16<E5_1>(uint32_t(x[2 * k]), uint32_t(x[2 * k + 1]), fx),
                                                  widen8_bf16<E5_2>(uint32_t(y[2 * k]), uint32_t(y[2 * k + 1]), fy),
                                                  acc, 0, 0, 0);
  return acc;
}

__device__ __forceinline__ i32x8 load32(const uint8_t* p) {
  const i32x4 a = reinterpret_cast<const i32x4*>(p)[0], b = reinterpret_cast<const i32x4*>(p)[1];
  return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// The simple form, for any shape: a workgroup makes a 16 (columns of out) x
// 16 * MT (rows) tile; its four waves share the contraction and join their sums
// through LDS in wave order.  The weight's rows are the instruction's first
// operand, so that a lane ends with four neighbouring columns of one row of out.
constexpr int kWaves = 4;

template <int DT, bool E5_A, bool E5_B, int MT>
__global__ __launch_bounds__(64 * kWaves) void matmul_rows(Operand a, Operand b, uint32_t blocks, uint32_t n_tiles,
                                                           typename Elem<DT>::type* out, int64_t out_stride) {
  constexpr bool kExact = DT == RESHARD_DTYPE_F32;
  __shared__ f32x4 sums[kWaves - 1][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = int(blockIdx.x % n_tiles) * 16, m0 = int(blockIdx.x / n_tiles) * (16 * MT);
  const int part = lane >> 4;
  const int rb = min(n0 + (lane & 15), b.rows - 1);
  const uint8_t* pb = b.data + rb * b.stride + part * 32;
  const uint8_t* sb = b.scales + int64_t(rb >> b.row_shift) * b.scale_stride;
  const uint8_t* pa[MT];
  const uint8_t* sa[MT];
  f32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int ra = min(m0 + 16 * t + (lane & 15), a.rows - 1);
    pa[t] = a.data + ra * a.stride + part * 32;
    sa[t] = a.scales + int64_t(ra >> a.row_shift) * a.scale_stride;
    acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  for (uint32_t k = wave; k < blocks; k += kWaves) {
    const i32x8 x = load32(pb + int64_t(k) * kBlock);
    const uint32_t sx = sb[k];
#pragma unroll
    for (int t = 0; t < MT; ++t)
      acc[t] = step128<kExact, E5_B, E5_A>(x, sx, load32(pa[t] + int64_t(k) * kBlock), sa[t][k], acc[t]);
  }
  if (wave) {
#pragma unroll
    for (int t = 0; t < MT; ++t) sums[wave - 1][t][lane] = acc[t];
  }
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
#pragma unroll
    for (int w = 0; w < kWaves - 1; ++w) acc[t] += sums[w][t][lane];
    const int m = m0 + 16 * t + (lane & 15), n = n0 + part * 4;
    if (m >= a.rows) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < b.rows) out[m * out_stride + n + i] = Elem<DT>::down(acc[t][i]);
  }
}

constexpr int kMT = 4;

template <int DT, bool E5_A, bool E5_B>
hipError_t matmul_as(const MatmulPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b,
                     const reshard_matrix_t& out, hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const uint32_t blocks = uint32_t(blocks_of(a.cols)), n_tiles = uint32_t(ceil_div(b.rows, 16));
  if (a.rows <= 16)
    matmul_rows<DT, E5_A, E5_B, 1><<<dim3(uint32_t(plan.groups)), 64 * kWaves, 0, stream>>>(
        operand(a), operand(b), blocks, n_tiles, static_cast<T*>(out.data), out.row_stride);
  else
    matmul_rows<DT, E5_A, E5_B, kMT><<<dim3(uint32_t(plan.groups)), 64 * kWaves, 0, stream>>>(
        operand(a), operand(b), blocks, n_tiles, static_cast<T*>(out.data), out.row_stride);
  return hipGetLastError();
}

template <int DT>
hipError_t matmul_formats(const MatmulPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b,
                          const reshard_matrix_t& out, hipStream_t stream) {
  const bool ea = a.dtype == RESHARD_DTYPE_FP8_E5M2, eb = b.dtype == RESHARD_DTYPE_FP8_E5M2;
  if (ea) return eb ? matmul_as<DT, true, true>(plan, a, b, out, stream) : matmul_as<DT, true, false>(plan, a, b, out, stream);
  return eb ? matmul_as<DT, false, true>(plan, a, b, out, stream) : matmul_as<DT, false, false>(plan, a, b, out, stream);
}

}  // namespace

MatmulPlan plan_matmul(const reshard_matrix_t& a, const reshard_matrix_t& b, const reshard_matrix_t& out) {
  MatmulPlan p;
  p.groups = ceil_div(b.rows, 16) * ceil_div(a.rows, a.rows <= 16 ? 16 : 16 * kMT);
  if (!a.block_rows && a.rows && a.cols) {
    p.quantized = round_up(a.rows * blocks_of(a.cols) * kBlock, 256);
    p.quantized_scales = a.rows * blocks_of(a.cols);
  }
  return p;
}

hipError_t launch_matmul(const MatmulPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b,
                         const reshard_matrix_t& out, void* workspace, hipStream_t stream) {
  reshard_matrix_t q = a;
  if (!a.block_rows) {
    q.dtype = RESHARD_DTYPE_FP8_E4M3;
    q.block_rows = 1;
    q.data = workspace;
    q.row_stride = blocks_of(a.cols) * kBlock;
    q.scales = static_cast<uint8_t*>(workspace) + plan.quantized;
    q.scale_stride = blocks_of(a.cols);
    if (plan.quantized) {
      const hipError_t e = launch_quantize(a, q, nullptr, stream);
      if (e != hipSuccess) return e;
    }
  }
  switch (out.dtype) {
    case RESHARD_DTYPE_F32: return matmul_formats<RESHARD_DTYPE_F32>(plan, q, b, out, stream);
    case RESHARD_DTYPE_BF16: return matmul_formats<RESHARD_DTYPE_BF16>(plan, q, b, out, stream);
    default: return matmul_formats<RESHARD_DTYPE_F16>(plan, q, b, out, stream);
  }
}

}  // namespace rs
