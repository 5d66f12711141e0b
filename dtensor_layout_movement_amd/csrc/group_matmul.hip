// out = a b^T with group-scaled 4-bit weights b (the format is in reshard.h), one
// weight for all rows or one for each expert's rows.
#include "group_device.h"
#include "groups.h"

#include <algorithm>

namespace rs {
namespace {

// A workgroup makes 16 columns of out for a chunk of up to 16 rows; its waves take the
// contraction in blocks of 128 columns in turn and their sums are joined through LDS in
// wave order.  Lane (row r, quarter q) of the 16 x 16 x 32 instruction's operands
// holds all 32 columns of group 4 k + q of its row: 16 bytes of the weight with one
// scale, used by four instructions of 8 columns each (the order within a block only has
// to be the same on both sides).
constexpr int kRowsHeight = 16, kMaxWaves = 16;

template <int SRC, int DT>
__global__ __launch_bounds__(64 * kMaxWaves) void group_rows(const typename Elem<SRC>::type* a, int64_t a_stride, int rows,
                                                             int cols, Weight b, const int32_t* offsets, int experts,
                                                             uint32_t n_tiles, typename Elem<DT>::type* out,
                                                             int64_t out_stride) {
  __shared__ f32x4 sums[kMaxWaves * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  Chunk c;
  uint32_t n_tile;
  if (offsets) {
    if (!find_tile(offsets, experts, rows, kRowsHeight, blockIdx.x, n_tiles, &c, &n_tile)) return;
  } else {
    const uint32_t id = run_of(blockIdx.x, gridDim.x);
    const int first = int(id / n_tiles) * kRowsHeight;
    c = Chunk{0, first, min(first + kRowsHeight, rows)};
    n_tile = id % n_tiles;
  }
  const int n0 = int(n_tile) * 16, part = lane >> 4;
  const int64_t rb = int64_t(c.expert) * b.rows + min(n0 + (lane & 15), b.rows - 1);
  const uint8_t* pb = b.data + rb * b.stride;
  const uint8_t* sb = b.scales + rb * b.scale_stride;
  const typename Elem<SRC>::type* pa = a + int64_t(min(c.first + (lane & 15), c.last - 1)) * a_stride;
  const int groups = (cols + kGroup - 1) / kGroup;
  f32x4 acc{0.f, 0.f, 0.f, 0.f};
  for (int k = wave * 4; k < groups; k += waves * 4) {
    const int g = k + part, at = min(g, groups - 1);
    const i32x4 q = *reinterpret_cast<const i32x4*>(pb + at * (kGroup / 2));
    const float scale = scale_value(sb[at]);
    bf16x8 y[4][Parts<SRC>::count];
    if ((k + 4) * kGroup <= cols) {
#pragma unroll
      for (int j = 0; j < 4; ++j) load_parts<SRC, false>(pa, g * kGroup + j * 8, cols, y[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) load_parts<SRC, true>(pa, g * kGroup + j * 8, cols, y[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 w = widen8_fp4(uint32_t(q[j]), scale);
#pragma unroll
      for (int n = 0; n < Parts<SRC>::count; ++n)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, y[j][n], acc, 0, 0, 0);
    }
  }
  sums[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave) return;
  for (int w = 1; w < waves; ++w) acc += sums[w * 64 + lane];
  const int m = c.first + (lane & 15), n = n0 + part * 4;
  if (m < c.last) store4<DT>(out + m * out_stride + n, acc, b.rows - n);
}

template <int SRC, int DT>
hipError_t product_as(const GroupPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b, const int32_t* offsets,
                      int64_t experts, const reshard_matrix_t& out, hipStream_t stream) {
  const Weight w{static_cast<const uint8_t*>(b.data), b.row_stride / 2, static_cast<const uint8_t*>(b.scales),
                 b.scale_stride, int(out.cols)};
  group_rows<SRC, DT><<<dim3(uint32_t(plan.groups)), 64 * plan.waves, 0, stream>>>(
      static_cast<const typename Elem<SRC>::type*>(a.data), a.row_stride, int(a.rows), int(a.cols), w, offsets,
      int(experts), uint32_t(ceil_div(out.cols, 16)), static_cast<typename Elem<DT>::type*>(out.data), out.row_stride);
  return hipGetLastError();
}

template <int SRC>
hipError_t product_from(const GroupPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b,
                        const int32_t* offsets, int64_t experts, const reshard_matrix_t& out, hipStream_t stream) {
  switch (out.dtype) {
    case RESHARD_DTYPE_F32: return product_as<SRC, RESHARD_DTYPE_F32>(plan, a, b, offsets, experts, out, stream);
    case RESHARD_DTYPE_BF16: return product_as<SRC, RESHARD_DTYPE_BF16>(plan, a, b, offsets, experts, out, stream);
    default: return product_as<SRC, RESHARD_DTYPE_F16>(plan, a, b, offsets, experts, out, stream);
  }
}

}  // namespace

GroupPlan plan_group_matmul(const reshard_matrix_t& a, const reshard_matrix_t& b, int64_t experts,
                            const reshard_matrix_t& out) {
  GroupPlan p;
  // Chunks of at most `height` rows, at most: every expert with a row may end in one
  // that is not full.
  const auto chunks = [&](int64_t height) {
    if (!experts) return ceil_div(a.rows, height);
    const int64_t ends = std::min(experts, a.rows);
    return ends + (a.rows - ends) / height;
  };
  const auto tiles = [&](int64_t bm, int64_t bn) { return chunks(bm) * ceil_div(out.cols, bn); };
  const int64_t parts = a.dtype == RESHARD_DTYPE_F32 ? 3 : a.dtype == RESHARD_DTYPE_F16 ? 2 : 1;
  const bool direct = parts == 1 && a.cols % 8 == 0 && a.row_stride % 8 == 0 && reinterpret_cast<uintptr_t>(a.data) % 16 == 0;
  // steps of the tiles: of a weight's contraction, in threes where its parts follow each other
  const int64_t part_steps = parts == 1 ? ceil_div(a.cols, 64) : ceil_div(a.cols, 192) * 3;
  const int64_t stride = std::max(direct ? a.row_stride * 2 : parts * part_steps * 128, std::max(b.row_stride / 2, b.scale_stride));
  // (their rows are at most 2^22 bytes apart, a tile's within 32-bit offsets, and they load
  // eight scales of a row together)
  const int64_t mean = experts ? a.rows / experts : a.rows;
  if (mean > kRowsHeight && groups_of(a.cols) >= 8 && out.cols && stride <= (int64_t(1) << 22)) {
    if (tiles(256, 256) >= 192 && (!experts || mean >= 192)) {
      p.form = GroupPlan::kTiles256;
      p.groups = tiles(256, 256);
    } else if (tiles(128, 128) >= 256 && mean > 64) {
      p.form = GroupPlan::kTiles128;
      p.groups = tiles(128, 128);
    } else {
      p.form = GroupPlan::kTiles64;
      p.groups = tiles(64, 128);
    }
    p.part_steps = uint32_t(part_steps);
    p.steps = uint32_t(parts * part_steps);
    p.steps_per_split = p.steps;
    if (!direct) p.planes = round_up(a.rows * parts * part_steps * 128, 256);
    if (p.form == GroupPlan::kTiles64 && !experts) {
      const int64_t t = p.groups;
      int64_t splits = std::max<int64_t>(1, std::min(2 * kCus / t, ceil_div(p.steps, 6)));
      p.steps_per_split = uint32_t(ceil_div(ceil_div(p.steps, splits), 3) * 3);
      p.splits = int(ceil_div(p.steps, p.steps_per_split));
      p.groups = t * p.splits;
      if (p.splits > 1) p.parts = p.splits * out.rows * round_up(out.cols, 4) * 4;
    }
    return p;
  }
  p.groups = tiles(kRowsHeight, 16);
  const int64_t blocks = ceil_div(a.cols, 4 * kGroup);
  p.waves = 4;
  while (p.waves < kMaxWaves && p.groups * p.waves < 4096 && p.waves < blocks) p.waves *= 2;
  return p;
}

hipError_t launch_group_matmul(const GroupPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b,
                               const int32_t* offsets, int64_t experts, const reshard_matrix_t& out, void* workspace,
                               hipStream_t stream) {
  if (plan.form != GroupPlan::kRows)
    return launch_group_tiles(plan, a, b, offsets, experts, out, workspace, stream);
  switch (a.dtype) {
    case RESHARD_DTYPE_F32: return product_from<RESHARD_DTYPE_F32>(plan, a, b, offsets, experts, out, stream);
    case RESHARD_DTYPE_BF16: return product_from<RESHARD_DTYPE_BF16>(plan, a, b, offsets, experts, out, stream);
    default: return product_from<RESHARD_DTYPE_F16>(plan, a, b, offsets, experts, out, stream);
  }
}

}  // namespace rs
