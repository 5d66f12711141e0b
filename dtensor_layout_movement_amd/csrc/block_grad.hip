// dw = dy^T x^ from an 8-bit checkpoint x (the format is in reshard.h).
//
// The contraction runs over the rows of both operands, so both are turned on
// their way from LDS to the matrix instruction (ds_read_b64_tr_b16).  x is widened
// to bfloat16 under its scale when it is put into LDS, which is exact, and dy
// goes in as bfloat16 as it is.
#include "block_device.h"
#include "blocks.h"

#include <algorithm>

namespace rs {
namespace {

constexpr int kDepth = 64;  // rows of dy and x a step takes

struct Checkpoint {
  const uint8_t* data;
  int64_t stride;
  const uint8_t* scales;
  int64_t scale_stride;
  int row_shift;
  int rows, cols;
};

// Part p of a value as bfloat16 bits: the leading 8 significant bits, the next 8,
// the last 8, each cut off exactly, so that the parts add up to the value.
template <int PARTS> __device__ __forceinline__ uint16_t part_of(float v, int p) {
  uint32_t bits = __builtin_bit_cast(uint32_t, v);
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

// An fp16 or fp32 dy, or a bf16 one off the 16-byte grid, is first written to the
// workspace as 2, 3 or 1 bfloat16 planes whose sum it is, rows of `width` elements
// (a multiple of 8) on the grid.  The product then runs over the rows of all planes,
// each against the same rows of x.  Bound by HBM.
template <int DT, int PARTS>
__global__ __launch_bounds__(256) void split_parts(const typename Elem<DT>::type* src, int64_t stride, int cols,
                                                   uint32_t width8, int64_t items, uint16_t* planes) {
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < items; i += step) {
    const int64_t r = i / width8;
    const int c = int(uint32_t(i - r * width8)) * 8;
    const typename Elem<DT>::type* p = src + r * stride + c;
    float v[8];
    if (c + 8 <= cols) {
      const Pack<typename Elem<DT>::type, 8> x = load_pack<typename Elem<DT>::type, 8>(p);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = Elem<DT>::up(x.v[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = c + k < cols ? Elem<DT>::up(p[k]) : 0.f;
    }
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = uint32_t(part_of<PARTS>(v[2 * k], q)) | uint32_t(part_of<PARTS>(v[2 * k + 1], q)) << 16;
      *reinterpret_cast<i32x4*>(planes + (int64_t(q) * items + i) * 8) =
          i32x4{int(w[0]), int(w[1]), int(w[2]), int(w[3])};
    }
  }
}

// dy as the product reads it: bfloat16 rows on the 16-byte grid, `planes` times
// the rows of x.
struct Output {
  const uint16_t* data;
  int64_t stride;
  int cols;
};

typedef short s16x4 __attribute__((ext_vector_type(4)));

// LDS holds a step's rows one after another; the 32-byte pieces (16 columns) of a
// row are permuted by the row, so that the eight rows that half a wave turns at
// a time lie in distinct banks.  (The stores of the widened x, 32 bytes a lane in two
// halves, meet two to a bank: a fifth of the LDS cycles of a large gradient.)
__device__ __forceinline__ int piece_of(int row, int piece) { return piece ^ ((row & 3) | ((row >> 1) & 4)); }

// A lane's four values down the rows of one column: lanes 4 e .. 4 e + 3 of each 16
// address row e's 16 columns, lane i receives column i of the four rows.
__device__ __forceinline__ s16x4 turned(const uint8_t* p) {
  typedef __attribute__((address_space(3))) s16x4* Ptr;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((Ptr)p);
}

// One operand fragment: 16 columns, 32 rows; `half` is four rows on.
__device__ __forceinline__ bf16x8 fragment(const uint8_t* p, int half) {
  const s16x4 a = turned(p), b = turned(p + half);
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}

// One BN (columns of dy, from n0) x BK (columns of x, from k0) tile of dw with
// WN x WK waves over the steps [first, last) of the contraction, within the
// caller's LDS, two buffers of kDepth * (BN + BK) * 2 bytes.  The next step's dy goes
// straight to LDS and its x to registers while this step is multiplied; x is then
// widened and put into the other buffer.  dw of 14336 x 4096 over 4096 rows of bf16
// takes 499 us (960 TFLOP/s, the matrix pipe busy 43% of the time; a bfloat16 library
// product 505): the waits at a step's barrier, with two waves a SIMD.  Short ones pay
// each step's latency, one being under way: 1024 x 4096 over 257 rows (128 x 128 tiles, 5
// steps) 10.8 us.  An fp32 dy goes over x three times: 5000 x 3001 over 301 rows 44 us
// and 6.8 for the planes, an fp16 one twice: 4096 x 4096 over 1024 rows 79 and 7.
template <int DT_W, bool E5M2, int BN, int BK, int WN, int WK>
__device__ __forceinline__ void make_tile(const Output& dy, const Checkpoint& x, int rows, int n0, int k0,
                                          uint32_t first, uint32_t last, typename Elem<DT_W>::type* base,
                                          int64_t dw_stride, int accumulate, uint8_t* tile0, uint8_t* tile1) {
  constexpr int kThreads = 64 * WN * WK, kN = BN / WN / 16, kK = BK / WK / 16;
  constexpr int kRowY = BN * 2, kRowX = BK * 2;  // bytes of a row in LDS
  constexpr int kLoadsY = kDepth * kRowY / 16 / kThreads, kLoadsX = kDepth * BK / 16 / kThreads;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / WK, wk = wave % WK;

  // Where a lane's loads come from, within the step's rows.  Its loads of dy lie
  // kRowsY rows apart, a multiple of 16, so that their columns are the same.
  constexpr int kRowsY = kThreads * 16 / kRowY;
  static_assert(kRowsY % 16 == 0, "");
  const int row_y = int(threadIdx.x) / (kRowY / 16), chunk = int(threadIdx.x) % (kRowY / 16);
  const int col_y = min(n0 + (piece_of(row_y, chunk >> 1) * 2 + (chunk & 1)) * 8, (dy.cols - 1) & ~7);
  const uint32_t stride_y = uint32_t(dy.stride) * 2, off_y = uint32_t(row_y) * stride_y + uint32_t(col_y) * 2;
  int row_x[kLoadsX];
  const int col_x = min(k0 + int(threadIdx.x) % (BK / 16) * 16, int(uint32_t(x.cols - 1) & ~15u));
#pragma unroll
  for (int i = 0; i < kLoadsX; ++i) row_x[i] = (i * kThreads + int(threadIdx.x)) / (BK / 16);

  // (whole 16-byte pieces: the last one of a row may hold bytes past its columns,
  // within the same 16 aligned bytes)
  const auto load_y = [&](uint8_t* to, uint32_t s) {
    const int m0 = int(s) * kDepth, left = min(rows - 1 - m0, kDepth - 1);
    const Buffer from = buffer_of(dy.data + m0 * dy.stride, uint32_t(left) * stride_y + uint32_t(dy.cols + 7) / 8 * 16);
    if (left == kDepth - 1) {
#pragma unroll
      for (int i = 0; i < kLoadsY; ++i)
        load_to_lds(from, to + (i * kThreads + wave * 64) * 16, off_y, uint32_t(i * kRowsY) * stride_y);
    } else {  // a row past the last reads the last again; x is zero there
#pragma unroll
      for (int i = 0; i < kLoadsY; ++i)
        load_to_lds(from, to + (i * kThreads + wave * 64) * 16,
                    uint32_t(min(row_y + i * kRowsY, left)) * stride_y + uint32_t(col_y) * 2, 0);
    }
  };
  i32x4 qx[kLoadsX];
  uint32_t sx[kLoadsX];
  const auto load_x = [&](uint32_t s) {
#pragma unroll
    for (int i = 0; i < kLoadsX; ++i) {
      int m = min(int(s) * kDepth + row_x[i], rows - 1);
      while (m >= x.rows) m -= x.rows;  // the plane's row
      qx[i] = *reinterpret_cast<const i32x4*>(x.data + m * x.stride + col_x);
      sx[i] = x.scales[int64_t(m >> x.row_shift) * x.scale_stride + col_x / kBlock];
    }
  };
  const auto put_x = [&](uint8_t* to, uint32_t s) {
#pragma unroll
    for (int i = 0; i < kLoadsX; ++i) pin(qx[i]), pin(sx[i]);  // no use of the loads, and no wait, before this
#pragma unroll
    for (int i = 0; i < kLoadsX; ++i) {
      const bool in = int(s) * kDepth + row_x[i] < rows;
      const float f = scale_value(sx[i]);
      const int piece = int(threadIdx.x) % (BK / 16);
      uint8_t* p = to + kDepth * kRowY + row_x[i] * kRowX + piece_of(row_x[i], piece) * 32;
      const i32x4 q = in ? qx[i] : i32x4{0, 0, 0, 0};
      const float g = in ? f : 1.f;
      reinterpret_cast<bf16x8*>(p)[0] = widen8_bf16<E5M2>(uint32_t(q[0]), uint32_t(q[1]), g);
      reinterpret_cast<bf16x8*>(p)[1] = widen8_bf16<E5M2>(uint32_t(q[2]), uint32_t(q[3]), g);
    }
  };

  f32x4 acc[kK][kN];
#pragma unroll
  for (int i = 0; i < kK; ++i)
#pragma unroll
    for (int j = 0; j < kN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // this lane's addresses within a tile: its row of the first four of every
  // eight, its 8 bytes of each fragment's columns
  const int group = lane >> 4, row = group * 8 + ((lane >> 2) & 3), bytes = (lane & 3) * 8;
  int at_y[kN], at_x[kK];
#pragma unroll
  for (int j = 0; j < kN; ++j) at_y[j] = row * kRowY + piece_of(row, wn * kN + j) * 32 + bytes;
#pragma unroll
  for (int i = 0; i < kK; ++i) at_x[i] = kDepth * kRowY + row * kRowX + piece_of(row, wk * kK + i) * 32 + bytes;
  const auto step = [&](const uint8_t* tile) {
#pragma unroll 1  // unrolled, the compiler keeps the sums twice and spills
    for (int sub = 0; sub < kDepth / 32; ++sub) {
      bf16x8 u[kK];
#pragma unroll
      for (int i = 0; i < kK; ++i) u[i] = fragment(tile + at_x[i] + sub * 32 * kRowX, 4 * kRowX);
      bf16x8 v = fragment(tile + at_y[0] + sub * 32 * kRowY, 4 * kRowY);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        bf16x8 next = v;
        if (j + 1 < kN) next = fragment(tile + at_y[j + 1] + sub * 32 * kRowY, 4 * kRowY);
#pragma unroll
        for (int i = 0; i < kK; ++i) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u[i], v, acc[i][j], 0, 0, 0);
          pin(acc[i][j]);
        }
        __builtin_amdgcn_sched_barrier(0);
        v = next;
      }
    }
  };

  if (first < last) {
    load_x(first);
    load_y(tile0, first);
    put_x(tile0, first);
  }
  for (uint32_t s = first; s + 1 < last; s += 2) {
    loads_barrier<0>();  // tile0 is whole, tile1 is free
    load_x(s + 1);
    load_y(tile1, s + 1);
    step(tile0);
    put_x(tile1, s + 1);
    loads_barrier<0>();
    const bool more = s + 2 < last;
    if (more) {
      load_x(s + 2);
      load_y(tile0, s + 2);
    }
    step(tile1);
    if (more) put_x(tile0, s + 2);
  }
  if (first < last && ((last - first) & 1)) {
    loads_barrier<0>();
    step(tile0);
  }

#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const int n = n0 + (wn * kN + j) * 16 + (lane & 15);
    if (n >= dy.cols) continue;
    typename Elem<DT_W>::type* out = base + n * dw_stride;
#pragma unroll
    for (int i = 0; i < kK; ++i) {
      const int k = k0 + (wk * kK + i) * 16 + group * 4;
      if (k + 4 <= x.cols) {
        Pack<typename Elem<DT_W>::type, 4> p;
        if (accumulate) p = load_pack<typename Elem<DT_W>::type, 4>(out + k);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          p.v[e] = Elem<DT_W>::down(accumulate ? Elem<DT_W>::up(p.v[e]) + acc[i][j][e] : acc[i][j][e]);
        store_pack<typename Elem<DT_W>::type, 4>(out + k, p);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (k + e < x.cols)
            out[k + e] = Elem<DT_W>::down(accumulate ? Elem<DT_W>::up(out[k + e]) + acc[i][j][e] : acc[i][j][e]);
      }
    }
  }
}

// A tile a workgroup, or a tile's split.  Workgroups from `whole` on, which would
// leave half of the card idle in the last round, share a tile between two.
template <int DT_W, bool E5M2, int B, int WN, int WK>
__global__ __launch_bounds__(64 * WN * WK, 2) void grad_tiles(Output dy, Checkpoint x, int rows, uint32_t k_tiles,
                                                              uint32_t tiles, uint32_t whole, uint32_t steps_per_split,
                                                              typename Elem<DT_W>::type* dw, int64_t dw_stride,
                                                              int64_t split_stride, int accumulate) {
  __shared__ __align__(128) uint8_t tile0[kDepth * 4 * B];
  __shared__ __align__(128) uint8_t tile1[kDepth * 4 * B];
  const uint32_t all = uint32_t((rows + kDepth - 1) / kDepth);
  if (blockIdx.x < whole) {
    // tiles to XCDs in contiguous runs, whose tiles share operands in its L2
    const uint32_t split = blockIdx.x / tiles, t = run_of(blockIdx.x % tiles, min(whole, tiles));
    const uint32_t first = split * steps_per_split, last = min(first + steps_per_split, all);
    make_tile<DT_W, E5M2, B, B, WN, WK>(dy, x, rows, int(t / k_tiles) * B, int(t % k_tiles) * B, first, last,
                                        dw + split * split_stride, dw_stride, accumulate, tile0, tile1);
  } else if constexpr (B == 256) {  // (one split)
    const uint32_t half = run_of(blockIdx.x - whole, gridDim.x - whole), t = whole + half / 2;
    const int k0 = int(t % k_tiles) * B + int(half % 2) * (B / 2);
    if (k0 < x.cols)
      make_tile<DT_W, E5M2, B, B / 2, 4, 2>(dy, x, rows, int(t / k_tiles) * B, k0, 0, all, dw, dw_stride, accumulate,
                                            tile0, tile1);
  }
}

template <int DT_W, bool E5M2>
hipError_t grad_as(const GradPlan& plan, const Output& dy, const Checkpoint& c, int rows, void* dw, int64_t dw_stride,
                   int64_t split_stride, int accumulate, hipStream_t stream) {
  typedef typename Elem<DT_W>::type T;
  const uint32_t k_tiles = uint32_t(ceil_div(c.cols, plan.tile));
  const uint32_t tiles = k_tiles * uint32_t(ceil_div(dy.cols, plan.tile));
  if (plan.tile == 256)
    grad_tiles<DT_W, E5M2, 256, 2, 4><<<dim3(uint32_t(plan.groups)), 512, 0, stream>>>(
        dy, c, rows, k_tiles, tiles, uint32_t(plan.whole), plan.steps_per_split, static_cast<T*>(dw), dw_stride, split_stride, accumulate);
  else
    grad_tiles<DT_W, E5M2, 128, 2, 2><<<dim3(uint32_t(plan.groups)), 256, 0, stream>>>(
        dy, c, rows, k_tiles, tiles, uint32_t(plan.whole), plan.steps_per_split, static_cast<T*>(dw), dw_stride, split_stride, accumulate);
  return hipGetLastError();
}

template <int DT_W>
hipError_t grad_format(bool e5m2, const GradPlan& plan, const Output& dy, const Checkpoint& c, int rows, void* dw,
                       int64_t dw_stride, int64_t split_stride, int accumulate, hipStream_t stream) {
  return e5m2 ? grad_as<DT_W, true>(plan, dy, c, rows, dw, dw_stride, split_stride, accumulate, stream)
              : grad_as<DT_W, false>(plan, dy, c, rows, dw, dw_stride, split_stride, accumulate, stream);
}

template <int DT, int PARTS> hipError_t split_as(const reshard_matrix_t& dy, uint16_t* planes, hipStream_t stream) {
  const int64_t width8 = ceil_div(dy.cols, 8), items = dy.rows * width8;
  const int64_t groups = std::min<int64_t>(ceil_div(items, 256), kMaxGroups);
  split_parts<DT, PARTS><<<dim3(uint32_t(groups)), 256, 0, stream>>>(
      static_cast<const typename Elem<DT>::type*>(dy.data), dy.row_stride, int(dy.cols), uint32_t(width8), items, planes);
  return hipGetLastError();
}

// Adds the parts of a split contraction in order.
constexpr int kTogether = 7;

template <int DT>
__global__ __launch_bounds__(256) void join_parts(const float* parts, int n_parts, int64_t part_stride, int cols,
                                                  uint32_t width4, int64_t items, typename Elem<DT>::type* out,
                                                  int64_t out_stride, int accumulate) {
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < items; i += step) {
    const int64_t r = i / width4;
    const int c = int(uint32_t(i - r * width4)) * 4;
    f32x4 sum = *reinterpret_cast<const f32x4*>(parts + i * 4);
    for (int p = 1; p < n_parts; p += kTogether) {  // loads of several parts under way together
      f32x4 v[kTogether];
#pragma unroll
      for (int q = 0; q < kTogether; ++q)
        v[q] = *reinterpret_cast<const f32x4*>(parts + min(p + q, n_parts - 1) * part_stride + i * 4);
#pragma unroll
      for (int q = 0; q < kTogether; ++q)
        if (p + q < n_parts) sum += v[q];
    }
    typename Elem<DT>::type* o = out + r * out_stride + c;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < cols) o[e] = Elem<DT>::down(accumulate ? Elem<DT>::up(o[e]) + sum[e] : sum[e]);
  }
}

}  // namespace

int64_t grad_planes(int dtype) { return dtype == RESHARD_DTYPE_F32 ? 3 : dtype == RESHARD_DTYPE_F16 ? 2 : 1; }

hipError_t launch_join(const float* parts, int n_parts, int64_t part_stride, const reshard_matrix_t& out,
                       bool accumulate, hipStream_t stream) {
  const int64_t width4 = ceil_div(out.cols, 4), items = out.rows * width4;
  const dim3 grid(uint32_t(std::min<int64_t>(ceil_div(items, 256), kMaxGroups)));
  const int add = accumulate ? 1 : 0;
  switch (out.dtype) {
    case RESHARD_DTYPE_F32:
      join_parts<RESHARD_DTYPE_F32><<<grid, 256, 0, stream>>>(parts, n_parts, part_stride, int(out.cols), uint32_t(width4),
                                                              items, static_cast<float*>(out.data), out.row_stride, add);
      break;
    case RESHARD_DTYPE_BF16:
      join_parts<RESHARD_DTYPE_BF16><<<grid, 256, 0, stream>>>(parts, n_parts, part_stride, int(out.cols),
                                                               uint32_t(width4), items, static_cast<__bf16*>(out.data),
                                                               out.row_stride, add);
      break;
    default:
      join_parts<RESHARD_DTYPE_F16><<<grid, 256, 0, stream>>>(parts, n_parts, part_stride, int(out.cols),
                                                              uint32_t(width4), items, static_cast<_Float16*>(out.data),
                                                              out.row_stride, add);
  }
  return hipGetLastError();
}

GradPlan plan_grad(const reshard_matrix_t& dy, const reshard_matrix_t& x, const reshard_matrix_t& dw) {
  GradPlan p;
  const int64_t rows = dy.rows * grad_planes(dy.dtype), steps = ceil_div(rows, kDepth);
  // Large tiles where they nearly fill the card, us against 128 x 128: dw of 4096 x 4096
  // (256 of them) over 4096 rows 132 to 141 and 169, 14336 x 4096 over 257 69 and 85, 5000 x
  // 3001 (240) over 301 of fp32 48 and 56; 4096 x 2048 (128) over 4096 128 and 85 to 91.
  p.tile = ceil_div(dy.cols, 256) * ceil_div(x.cols, 256) >= 192 ? 256 : 128;
  const int64_t tiles = ceil_div(dy.cols, p.tile) * ceil_div(x.cols, p.tile);
  // Few tiles and a long contraction: several workgroups share it.
  int64_t splits = 1;
  if (tiles && tiles < 256 && p.tile == 128) splits = std::max<int64_t>(1, std::min(512 / tiles, steps / 4));
  p.steps_per_split = uint32_t(std::max<int64_t>(1, ceil_div(steps, splits)));
  splits = std::max<int64_t>(1, ceil_div(steps, p.steps_per_split));
  p.splits = int(splits);
  p.whole = p.groups = tiles * splits;
  if (p.tile == 256) {
    p.whole = whole_tiles(tiles);
    p.groups = 2 * tiles - p.whole;
  }
  // bf16 rows on the 16-byte grid are read where they lie
  p.direct = dy.dtype == RESHARD_DTYPE_BF16 && dy.row_stride % 8 == 0 && dy.row_stride <= kMaxGradCols &&
             reinterpret_cast<uintptr_t>(dy.data) % 16 == 0;
  if (!p.direct) p.planes = round_up(rows * round_up(dy.cols, 8) * 2, 256);
  if (splits > 1) p.parts = splits * dw.rows * round_up(dw.cols, 4) * 4;
  return p;
}

hipError_t launch_grad(const GradPlan& plan, const reshard_matrix_t& dy, const reshard_matrix_t& x,
                       const reshard_matrix_t& dw, bool accumulate, void* workspace, hipStream_t stream) {
  const Checkpoint c{static_cast<const uint8_t*>(x.data), x.row_stride, static_cast<const uint8_t*>(x.scales),
                     x.scale_stride, x.block_rows == 1 ? 0 : 7, int(x.rows), int(x.cols)};
  Output y{static_cast<const uint16_t*>(dy.data), dy.row_stride, int(dy.cols)};
  if (!plan.direct) {
    uint16_t* planes = static_cast<uint16_t*>(workspace);
    if (dy.rows) {
      const hipError_t e = dy.dtype == RESHARD_DTYPE_F32    ? split_as<RESHARD_DTYPE_F32, 3>(dy, planes, stream)
                           : dy.dtype == RESHARD_DTYPE_F16 ? split_as<RESHARD_DTYPE_F16, 2>(dy, planes, stream)
                                                           : split_as<RESHARD_DTYPE_BF16, 1>(dy, planes, stream);
      if (e != hipSuccess) return e;
    }
    y.data = planes;
    y.stride = round_up(dy.cols, 8);
  }
  const int rows = int(dy.rows * grad_planes(dy.dtype));
  const bool e5m2 = x.dtype == RESHARD_DTYPE_FP8_E5M2;
  if (plan.splits > 1) {
    float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.planes);
    const int64_t stride = round_up(dw.cols, 4), size = dw.rows * stride;
    const hipError_t e = grad_format<RESHARD_DTYPE_F32>(e5m2, plan, y, c, rows, parts, stride, size, 0, stream);
    if (e != hipSuccess) return e;
    return launch_join(parts, plan.splits, size, dw, accumulate, stream);
  }
  const int add = accumulate ? 1 : 0;
  switch (dw.dtype) {
    case RESHARD_DTYPE_F32: return grad_format<RESHARD_DTYPE_F32>(e5m2, plan, y, c, rows, dw.data, dw.row_stride, 0, add, stream);
    case RESHARD_DTYPE_BF16: return grad_format<RESHARD_DTYPE_BF16>(e5m2, plan, y, c, rows, dw.data, dw.row_stride, 0, add, stream);
    default: return grad_format<RESHARD_DTYPE_F16>(e5m2, plan, y, c, rows, dw.data, dw.row_stride, 0, add, stream);
  }
}

}  // namespace rs
