// Quantizing to and reading back from block-scaled 8-bit matrices (the format is
// in reshard.h).  Both directions are bound by HBM: each element is read and
// written once.
#include "block_device.h"
#include "blocks.h"

#include <algorithm>

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

// Blocks of 1 x 128: sixteen lanes a block, eight elements a lane.  Workgroups are
// dealt to the XCDs in contiguous runs: neighbours write parts of one line of
// scale bytes, which then meet in one L2 (4096 x 4096 bf16 10.4 -> 9.3 us).  4096 x
// 14336 bf16 takes 33 us, 5.3 TB/s of reads and writes; two or four blocks a lane
// were 10 to 25% slower, and so were loads past the caches on small matrices.
template <int DT, bool E5M2>
__global__ __launch_bounds__(kThreads) void quantize_rows(const typename Elem<DT>::type* src, int64_t stride, int cols,
                                                          Divisor blocks, uint32_t items, Held dst) {
  const int part = threadIdx.x & 15;
  const uint32_t i = run_of(blockIdx.x, gridDim.x) * (kThreads / 16) + (threadIdx.x >> 4);
  if (i >= items) return;  // whole groups of sixteen lanes
  const uint32_t row = quotient(i, blocks), block = i - row * blocks.d;
  float x[8];
  load_up<DT, 8>(src + int64_t(row) * stride, int(block) * kBlock + part * 8, cols, x);
  uint32_t amax = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) amax = max(amax, finite_magnitude(x[k]));
  const uint32_t s = scale_byte<E5M2>(max_of_16(amax));
  *reinterpret_cast<i32x2*>(dst.data + int64_t(row) * dst.stride + block * kBlock + part * 8) =
      quantize8<E5M2>(x, inverse_scale(s));
  if (part == 0) dst.scales[int64_t(row) * dst.scale_stride + block] = uint8_t(s);
}

// Blocks of 128 x 128: a workgroup a block, sixteen lanes a row, eight passes of
// 16 rows held in registers until the block's scale is known.  For the transpose
// the payload goes through LDS: a lane reads one dword (4 columns) of each of 16
// rows, turns them four by four with byte permutes and stores 16 bytes of four
// rows of the transpose; eight lanes make a whole 128-byte row of it.  Rows lie 33
// dwords apart and the lower half 8 dwords further, which puts the 64 dwords of a
// read into distinct banks.  14336 x 4096 fp32 takes 53 us, 65 with the transpose
// (5.6 and 5.4 TB/s), bf16 40 (4.4); 5000 x 3001 bf16 13 and 16.7 us (3.4 and 3.6 TB/s).
// Gathering the transpose byte by byte took 75 for 66.
__device__ __forceinline__ int lds_row(int r) { return r * 33 + (r >> 6) * 8; }

template <int DT, bool E5M2, bool TRANSPOSE>
__global__ __launch_bounds__(kThreads) void quantize_squares(const typename Elem<DT>::type* src, int64_t stride,
                                                             int rows, int cols, uint32_t blocks, Held dst,
                                                             Held dst_t) {
  __shared__ uint32_t wave_max[kThreads / 64];
  __shared__ uint32_t tile[TRANSPOSE ? kBlock * 33 + 8 : 1];
  const int R = int(blockIdx.x / blocks), C = int(blockIdx.x % blocks);
  const int part = threadIdx.x & 15, lane_row = threadIdx.x >> 4;
  const int c = C * kBlock + part * 8;
  float x[8][8];
  uint32_t amax = 0;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int r = R * kBlock + p * 16 + lane_row;
    if (r < rows) {
      load_up<DT, 8>(src + int64_t(r) * stride, c, cols, x[p]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) x[p][k] = 0.f;
    }
  }
#pragma unroll
  for (int p = 0; p < 8; ++p)
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = max(amax, finite_magnitude(x[p][k]));
  amax = max_of_16(amax);
  amax = max(amax, uint32_t(__shfl_xor(int(amax), 16)));
  amax = max(amax, uint32_t(__shfl_xor(int(amax), 32)));
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) amax = max(amax, wave_max[w]);
  const uint32_t s = scale_byte<E5M2>(amax);
  const float inv = inverse_scale(s);
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int row = p * 16 + lane_row, r = R * kBlock + row;
    const i32x2 q = quantize8<E5M2>(x[p], inv);
    if (r < rows) *reinterpret_cast<i32x2*>(dst.data + int64_t(r) * dst.stride + c) = q;
    if (TRANSPOSE) {
      tile[lds_row(row) + part * 2] = uint32_t(q[0]);
      tile[lds_row(row) + part * 2 + 1] = uint32_t(q[1]);
    }
  }
  if (threadIdx.x == 0) {
    dst.scales[int64_t(R) * dst.scale_stride + C] = uint8_t(s);
    if (TRANSPOSE) dst_t.scales[int64_t(C) * dst_t.scale_stride + R] = uint8_t(s);
  }
  if (TRANSPOSE) {
    __syncthreads();
    const int chunk = threadIdx.x & 7, quad = threadIdx.x >> 3;  // 16 rows, 4 columns
    uint32_t out[4][4];  // [column][dword of 4 rows]
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = tile[lds_row(chunk * 16 + g * 4 + k) + quad];
      // bytes (b0 of w0, b0 of w1), (b1 of w0, b1 of w1), then pairs of pairs
      const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), b = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
      const uint32_t d = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u), e = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
      out[0][g] = __builtin_amdgcn_perm(b, a, 0x05040100u);
      out[1][g] = __builtin_amdgcn_perm(b, a, 0x07060302u);
      out[2][g] = __builtin_amdgcn_perm(e, d, 0x05040100u);
      out[3][g] = __builtin_amdgcn_perm(e, d, 0x07060302u);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int col = C * kBlock + quad * 4 + k;
      if (col < cols)
        *reinterpret_cast<i32x4*>(dst_t.data + int64_t(col) * dst_t.stride + R * kBlock + chunk * 16) =
            i32x4{int(out[k][0]), int(out[k][1]), int(out[k][2]), int(out[k][3])};
    }
  }
}

// Reading back: as many elements a lane as make 16 bytes of output, so that a
// wave's stores are contiguous, kBack pieces a lane whose loads are under way
// together, stores past the caches (kept in them, 4096 x 14336 bf16 took 32 us
// instead of 26, 6.8 TB/s with the payload still in the last-level cache; 16
// elements a lane whatever the type took 50).
constexpr int kBack = 2;

template <int DT, bool E5M2>
__global__ __launch_bounds__(kThreads) void dequantize_rows(Held src, int64_t first_row, int row_shift, Divisor chunks,
                                                            uint32_t items, typename Elem<DT>::type* dst,
                                                            int64_t stride, int cols) {
  typedef typename Elem<DT>::type T;
  constexpr int N = 16 / sizeof(T);
  const uint32_t first = blockIdx.x * (kThreads * kBack) + threadIdx.x;
  uint32_t q[kBack][N / 4], s[kBack], row[kBack];
  int c[kBack];
#pragma unroll
  for (int u = 0; u < kBack; ++u) {
    const uint32_t i = min(first + u * kThreads, items - 1);
    row[u] = quotient(i, chunks);
    c[u] = int(i - row[u] * chunks.d) * N;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(src.data + int64_t(row[u]) * src.stride + c[u]);
    const Pack<uint32_t, N / 4> v = load_pack<uint32_t, N / 4>(p);
#pragma unroll
    for (int k = 0; k < N / 4; ++k) q[u][k] = v.v[k];
    s[u] = src.scales[((first_row + row[u]) >> row_shift) * src.scale_stride + c[u] / kBlock];
  }
#pragma unroll
  for (int u = 0; u < kBack; ++u) {
    if (first + u * kThreads >= items) break;
    const float f = scale_value(s[u]);
    Pack<T, N> v;
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      const f32x4 w = widen4<E5M2>(q[u][k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v.v[4 * k + j] = Elem<DT>::down(w[j] * f);
    }
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

template <int DT, bool E5M2>
hipError_t quantize_as(const reshard_matrix_t& src, const reshard_matrix_t& dst, const reshard_matrix_t* dst_t,
                       hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const T* p = static_cast<const T*>(src.data);
  const uint32_t blocks = uint32_t(blocks_of(src.cols));
  if (dst.block_rows == 1) {
    const Held to = held(dst);
    const int64_t rows = rows_per_launch(blocks, kThreads / 16);
    for (int64_t r = 0; r < src.rows; r += rows) {
      const uint32_t items = uint32_t(std::min(rows, src.rows - r) * blocks);
      quantize_rows<DT, E5M2><<<dim3(uint32_t(ceil_div(items, kThreads / 16))), kThreads, 0, stream>>>(
          p + r * src.row_stride, src.row_stride, int(src.cols), divisor(blocks), items,
          Held{to.data + r * to.stride, to.stride, to.scales + r * to.scale_stride, to.scale_stride});
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
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
  constexpr int N = 16 / sizeof(T);
  const uint32_t chunks = uint32_t(ceil_div(src.cols, N));
  const Held from = held(src);
  const int64_t rows = rows_per_launch(chunks, kThreads * kBack);
  for (int64_t r = 0; r < src.rows; r += rows) {
    const uint32_t items = uint32_t(std::min(rows, src.rows - r) * chunks);
    dequantize_rows<DT, E5M2><<<dim3(uint32_t(ceil_div(items, kThreads * kBack))), kThreads, 0, stream>>>(
        Held{from.data + r * from.stride, from.stride, from.scales, from.scale_stride}, r, src.block_rows == 1 ? 0 : 7,
        divisor(chunks), items, static_cast<T*>(dst.data) + r * dst.row_stride,
        dst.row_stride, int(dst.cols));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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
