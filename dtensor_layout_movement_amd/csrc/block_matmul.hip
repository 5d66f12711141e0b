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

// The tiled form.  A workgroup makes a BM (rows of a) x BN (rows of b) tile with
// WM x WN waves; a step takes 128 columns of both operands through LDS, loaded
// straight there (16 bytes a lane) one step ahead into the other of two
// buffers.  Rows lie 128 bytes apart in LDS, and 16-byte chunk c of row r sits in
// slot c ^ (r / 2 % 8), so that the 16 rows a matrix instruction's operand
// takes its chunk from lie in distinct banks.  A load to LDS writes lane
// order, so the permutation is made on the address that each lane loads.
__device__ __forceinline__ int slot_of(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// Moves a tile's rows, 128 bytes from column byte `col` of each, into `to`.
template <int ROWS, int THREADS>
__device__ __forceinline__ void stage(Buffer base, const uint32_t (&off)[ROWS * 8 / THREADS],
                                      uint32_t col, uint8_t* to, int wave) {
#pragma unroll
  for (int i = 0; i < ROWS * 8 / THREADS; ++i) load_to_lds(base, to + (i * THREADS + wave * 64) * 16, off[i], col);
}

// The operand's rows from r0 on as a buffer: 32-bit offsets for its loads, and
// none past its end.
__device__ __forceinline__ Buffer rows_of(const Operand& o, int r0, int rows, uint32_t blocks) {
  const int last = min(r0 + rows, o.rows) - 1 - r0;
  return buffer_of(o.data + r0 * o.stride, uint32_t(last) * uint32_t(o.stride) + blocks * kBlock);
}

// A lane's offsets (row and chunk) in the staging of the rows from r0 on; rows
// past the operand's last are read from the last (their results are not stored).
template <int ROWS, int THREADS>
__device__ __forceinline__ void stage_offsets(const Operand& o, int r0, uint32_t (&off)[ROWS * 8 / THREADS]) {
#pragma unroll
  for (int i = 0; i < ROWS * 8 / THREADS; ++i) {
    const int at = i * THREADS + int(threadIdx.x), row = at >> 3;
    off[i] = uint32_t(min(row, o.rows - 1 - r0)) * uint32_t(o.stride) + uint32_t(slot_of(row, at & 7) * 16);
  }
}

// A lane's 32 bytes of a fragment's row, in two slots of it.
__device__ __forceinline__ i32x8 fragment(const uint8_t* lo, const uint8_t* hi, int at) {
  const i32x4 a = *reinterpret_cast<const i32x4*>(lo + at), b = *reinterpret_cast<const i32x4*>(hi + at);
  return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Scale bytes of four steps of one row.
__device__ __forceinline__ uint32_t load_scales(const uint8_t* row, uint32_t k, uint32_t blocks) {
  if (k + 4 <= blocks) return load_pack<uint32_t, 1>(reinterpret_cast<const uint32_t*>(row + k)).v[0];
  uint32_t v = 0;
  for (uint32_t i = 0; k + i < blocks; ++i) v |= uint32_t(row[k + i]) << (8 * i);
  return v;
}

template <int DT, bool E5_A, bool E5_B, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void matmul_tiles(Operand a, Operand b, uint32_t blocks, uint32_t m_tiles,
                                                                uint32_t n_tiles, typename Elem<DT>::type* out,
                                                                int64_t out_stride) {
  constexpr bool kExact = DT == RESHARD_DTYPE_F32;
  constexpr int kThreads = 64 * WM * WN, kM = BM / WM / 16, kN = BN / WN / 16;
  __shared__ __align__(128) uint8_t tile0[(BM + BN) * kBlock];
  __shared__ __align__(128) uint8_t tile1[(BM + BN) * kBlock];
  __shared__ uint32_t scales[2][BM + BN];  // four steps of every row, two groups of steps
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  // tiles to XCDs: each takes a contiguous run of tiles, rows of tiles fastest,
  // so that the tiles in flight on one share their operands in its L2
  const uint32_t t = run_of(blockIdx.x, m_tiles * n_tiles);
  const int m0 = int(t % m_tiles) * BM, n0 = int(t / m_tiles) * BN;

  uint32_t off_a[BM * 8 / kThreads], off_b[BN * 8 / kThreads];
  stage_offsets<BM, kThreads>(a, m0, off_a);
  stage_offsets<BN, kThreads>(b, n0, off_b);
  const Buffer base_a = rows_of(a, m0, BM, blocks), base_b = rows_of(b, n0, BN, blocks);
  const auto load = [&](uint8_t* to, uint32_t k) {
    stage<BM, kThreads>(base_a, off_a, k * kBlock, to, wave);
    stage<BN, kThreads>(base_b, off_b, k * kBlock, to + BM * kBlock, wave);
  };
  // one row's scales a thread
  constexpr int kScaleRows = (BM + BN + kThreads - 1) / kThreads;
  const uint8_t* srow[kScaleRows];
#pragma unroll
  for (int i = 0; i < kScaleRows; ++i) {
    const int r = int(threadIdx.x) + i * kThreads;
    if (r < BM)  // (a thread without a row of its own loads the last one's)
      srow[i] = a.scales + int64_t(min(m0 + r, a.rows - 1) >> a.row_shift) * a.scale_stride;
    else
      srow[i] = b.scales + int64_t(min(n0 + r - BM, b.rows - 1) >> b.row_shift) * b.scale_stride;
  }
  uint32_t held_scales[kScaleRows];
  const auto load_scale_group = [&](uint32_t k) {
#pragma unroll
    for (int i = 0; i < kScaleRows; ++i) held_scales[i] = load_scales(srow[i], k, blocks);
  };
  const auto store_scale_group = [&](uint32_t k) {
#pragma unroll
    for (int i = 0; i < kScaleRows; ++i) {
      const int r = int(threadIdx.x) + i * kThreads;
      if (r < BM + BN) scales[(k >> 2) & 1][r] = held_scales[i];
    }
  };

  f32x4 acc[kN][kM];
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int j = 0; j < kM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int frow = lane & 15, part = lane >> 4;
  // where this lane's fragments lie in a tile: rows 16 apart keep their slots
  const int slot0 = slot_of(frow, 2 * part) * 16, slot1 = slot_of(frow, 2 * part + 1) * 16;
  const int row_a = (wm * (BM / WM) + frow), row_b = BM + wn * (BN / WN) + frow;
  const uint8_t* scale_bytes = reinterpret_cast<const uint8_t*>(scales);
  const auto step = [&](const uint8_t* tile, uint32_t k) {
    const uint8_t* sk = scale_bytes + ((k >> 2) & 1) * ((BM + BN) * 4) + (k & 3);
    const uint8_t *a0 = tile + row_a * kBlock + slot0, *a1 = tile + row_a * kBlock + slot1;
    const uint8_t *b0 = tile + row_b * kBlock + slot0, *b1 = tile + row_b * kBlock + slot1;
    i32x8 y[kN];
    uint32_t sb[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      y[i] = fragment(b0, b1, i * 16 * kBlock);
      sb[i] = sk[row_b * 4 + i * 64];
    }
    // one fragment of a ahead of its products; the pins keep the compiler from
    // reading all of them first, which does not fit the registers
    i32x8 x = fragment(a0, a1, 0);
    uint32_t sa = sk[row_a * 4];
#pragma unroll
    for (int j = 0; j < kM; ++j) {
      i32x8 next = x;
      uint32_t snext = sa;
      if (j + 1 < kM) {
        next = fragment(a0, a1, (j + 1) * 16 * kBlock);
        snext = sk[row_a * 4 + (j + 1) * 64];
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        acc[i][j] = step128<kExact, E5_B, E5_A>(y[i], sb[i], x, sa, acc[i][j]);
        pin(acc[i][j]);
      }
      __builtin_amdgcn_sched_barrier(0);
      x = next;
      sa = snext;
    }
  };

  if (blocks) {
    load(tile0, 0);
    load_scale_group(0);
    store_scale_group(0);
  }
  for (uint32_t k = 0; k + 1 < blocks; k += 2) {
    __syncthreads();  // tile0 has arrived, tile1 is free
    load(tile1, k + 1);
    // the next four steps' scales: loaded in one step, put down in the next,
    // into the group that was last read four steps ago
    const bool scale_turn = (k & 2) == 0 && k + 4 < blocks;
    if (scale_turn) load_scale_group(k + 4);
    step(tile0, k);
    __syncthreads();
    if (k + 2 < blocks) load(tile0, k + 2);
    if (scale_turn) store_scale_group(k + 4);
    step(tile1, k + 1);
  }
  if (blocks & 1) {
    __syncthreads();
    step(tile0, blocks - 1);
  }
#pragma unroll
  for (int j = 0; j < kM; ++j) {
    const int m = m0 + wm * (BM / WM) + j * 16 + frow;
    if (m >= a.rows) continue;
    typename Elem<DT>::type* row = out + m * out_stride;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int n = n0 + wn * (BN / WN) + i * 16 + part * 4;
      Pack<typename Elem<DT>::type, 4> v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v.v[e] = Elem<DT>::down(acc[i][j][e]);
      if (n + 4 <= b.rows) {
        store_pack<typename Elem<DT>::type, 4>(row + n, v);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < b.rows) row[n + e] = v.v[e];
      }
    }
  }
}

constexpr int kMT = 4;

template <int DT, bool E5_A, bool E5_B>
hipError_t matmul_as(const MatmulPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b,
                     const reshard_matrix_t& out, hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const uint32_t blocks = uint32_t(blocks_of(a.cols)), n_tiles = uint32_t(ceil_div(b.rows, 16));
  if (plan.tile == 256) {
    if constexpr (DT != RESHARD_DTYPE_F32)
      matmul_tiles<DT, E5_A, E5_B, 256, 256, 2, 4><<<dim3(uint32_t(plan.groups)), 512, 0, stream>>>(
          operand(a), operand(b), blocks, uint32_t(ceil_div(a.rows, 256)), uint32_t(ceil_div(b.rows, 256)),
          static_cast<T*>(out.data), out.row_stride);
  } else if (plan.tile == 128) {
    matmul_tiles<DT, E5_A, E5_B, 128, 128, 2, 2><<<dim3(uint32_t(plan.groups)), 256, 0, stream>>>(
        operand(a), operand(b), blocks, uint32_t(ceil_div(a.rows, 128)), uint32_t(ceil_div(b.rows, 128)),
        static_cast<T*>(out.data), out.row_stride);
  } else if (a.rows <= 16)
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
  const int64_t stride = std::max(a.block_rows ? a.row_stride : 0, b.row_stride);
  if (a.rows > 64 && stride <= (1 << 23)) {
    p.tile = out.dtype != RESHARD_DTYPE_F32 && ceil_div(a.rows, 256) * ceil_div(b.rows, 256) >= 192 ? 256 : 128;
    p.groups = ceil_div(a.rows, p.tile) * ceil_div(b.rows, p.tile);
  }
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
