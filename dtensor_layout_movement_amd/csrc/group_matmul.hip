// out = a b^T with group-scaled 4-bit weights b (the format is in reshard.h), one
// weight for all rows or one for each expert's rows.
#include "group_device.h"
#include "groups.h"

#include <algorithm>

namespace rs {
namespace {

// Four words of four neighbouring lane groups of 16, exchanged: word j of group q was word q
// of group j.
__device__ __forceinline__ i32x4 exchange(const i32x4& v) {
  const auto a = __builtin_amdgcn_permlane32_swap(uint32_t(v[0]), uint32_t(v[2]), false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(uint32_t(v[1]), uint32_t(v[3]), false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return i32x4{int(c[0]), int(c[1]), int(d[0]), int(d[1])};
}

// A workgroup makes 16 NT columns of out for a chunk of up to 16 rows; its waves take the
// contraction in runs of kRun blocks of 128 columns in turn, the next run's loads under way
// as one is used up, and their sums are joined through LDS in wave order.  An instruction
// multiplies one group of 32 columns: lane (row r, quarter q) of its operands holds columns
// 8 q to 8 q + 7 of the group.  The weight is read by quads of lanes, the block's 64 bytes
// of a row each, and comes to its lanes through two exchanges; a, of which few rows are
// often all the same one, is read where it is used.
//
// Bound by the weight's bytes where they are many: 128 rows at 64 experts of 2048 x 7168,
// 437 MB of weights, take 79 us (5.5 TB/s); by a launch and one trip to HBM where they are
// few: one token through 14336 x 4096, 31 MB, 9.7 us, through 4096 x 14336 7.8.  Read without
// quads those took 92, 9.3 and 9.0, 16 rows through 4096 x 14336 18.2 for 15.7; with a read by
// quads too the tokens took 11.0 and 13.5.  Eight waves: 77 tokens' experts 171 for 151.
constexpr int kRowsHeight = 16, kMaxWaves = 4, kRun = 4, kBlockCols = 4 * kGroup;

template <int SRC, int DT, int NT>
__global__ __launch_bounds__(64 * kMaxWaves) void group_rows(const typename Elem<SRC>::type* a, int64_t a_stride, int rows,
                                                             int cols, Weight b, const int32_t* offsets, int experts,
                                                             uint32_t n_tiles, typename Elem<DT>::type* out,
                                                             int64_t out_stride) {
  typedef typename Elem<SRC>::type S;
  constexpr int kParts = Parts<SRC>::count;
  extern __shared__ __align__(16) f32x4 sums[];
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
  const int n0 = int(n_tile) * (16 * NT), part = lane >> 4, quad = lane >> 2, in_quad = lane & 3, from = from_quads();
  const uint8_t *pb[NT], *sb[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t rb = int64_t(c.expert) * b.rows + min(n0 + i * 16 + quad, b.rows - 1);
    pb[i] = b.data + rb * b.stride;
    sb[i] = b.scales + rb * b.scale_stride;
  }
  const S* pa = a + int64_t(min(c.first + (lane & 15), c.last - 1)) * a_stride;
  const int groups = (cols + kGroup - 1) / kGroup;
  const int full = cols / kBlockCols >= kRun ? cols / kBlockCols : 0;  // blocks taken in runs

  f32x4 acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const auto multiply = [&](int i, const i32x4& q, uint32_t scales, const bf16x8 (&y)[4][kParts]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 w = widen8_fp4(uint32_t(q[j]), scale_of(scales, j));
#pragma unroll
      for (int n = 0; n < kParts; ++n) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, y[j][n], acc[i], 0, 0, 0);
    }
  };

  // A wave's run: blocks k to k + kRun - 1, the last run moved back to end with the last block.
  i32x4 q[kRun][NT];
  uint32_t s[NT];  // a quad's lanes hold a run's four words
  const auto load_scales = [&](int k) {
#pragma unroll
    for (int i = 0; i < NT; ++i) s[i] = load_pack<uint32_t, 1>(reinterpret_cast<const uint32_t*>(sb[i] + (k + in_quad) * 4)).v[0];
  };
  const auto load_block = [&](int u, int k) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
      q[u][i] = *reinterpret_cast<const i32x4*>(pb[i] + (int64_t(k + u) * (kBlockCols / 2) + in_quad * 16));
  };
  struct Raw {
    Pack<S, 8> v[4];
  };
  const auto load_a = [&](Raw& r, int k) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[j] = load_pack<S, 8>(pa + (k * kBlockCols + j * kGroup + part * 8));
  };
  // With NEXT the wave's next run, from block `to` on, is asked for as this one is used up.
  Raw x[kRun];
  const auto run = [&](int at, int to, auto next) {
    const int k = min(at, full - kRun);
    uint32_t s_now[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) s_now[i] = s[i];
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      if (k + u >= at) {  // not the run's before
        bf16x8 y[4][kParts];
#pragma unroll
        for (int j = 0; j < 4; ++j) split8<SRC>(x[u].v[j], y[j]);
#pragma unroll
        for (int i = 0; i < NT; ++i) multiply(i, exchange(permuted(q[u][i], from)), permuted(s_now[i], ((lane & 15) * 4 + u) * 4), y);
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (decltype(next)::value) {
        if (u == 0) load_scales(to);
        load_block(u, to);
        load_a(x[u], to + u);
      }
    }
  };
  int at = wave * kRun;
  if (at < full) {
    const int k = min(at, full - kRun);
    load_scales(k);
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      load_block(u, k);
      load_a(x[u], k + u);
    }
    __builtin_amdgcn_sched_barrier(0);
    for (; at + waves * kRun < full; at += waves * kRun) run(at, min(at + waves * kRun, full - kRun), Index<1>{});
    run(at, 0, Index<0>{});
  }
  // what no run takes: the columns past the last whole block, or few blocks
  for (int k = full + wave; k * 4 < groups; k += waves) {
    const int g = min(k * 4 + in_quad, groups - 1);
    bf16x8 y[4][kParts];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      load_parts<SRC>(pa, k * kBlockCols + j * kGroup + part * 8, cols, y[j]);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      uint32_t scales = 0;  // of groups that there are not, one that is finite
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (k * 4 + j < groups) scales |= uint32_t(sb[i][k * 4 + j]) << (8 * j);
      multiply(i, exchange(permuted(*reinterpret_cast<const i32x4*>(pb[i] + int64_t(g) * 16), from)),
               permuted(scales, (lane & 15) * 16), y);
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) sums[(wave * NT + i) * 64 + lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < NT; i += waves) {
    f32x4 sum = sums[i * 64 + lane];
    for (int w = 1; w < waves; ++w) sum += sums[(w * NT + i) * 64 + lane];
    const int m = c.first + (lane & 15), n = n0 + i * 16 + part * 4;
    if (m < c.last) store4<DT>(out + m * out_stride + n, sum, b.rows - n);
  }
}

template <int SRC, int DT, int NT>
hipError_t rows_as(const GroupPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b, const int32_t* offsets,
                   int64_t experts, const reshard_matrix_t& out, hipStream_t stream) {
  const Weight w{static_cast<const uint8_t*>(b.data), b.row_stride / 2, static_cast<const uint8_t*>(b.scales),
                 b.scale_stride, int(out.cols)};
  group_rows<SRC, DT, NT><<<dim3(uint32_t(plan.groups)), 64 * plan.waves, plan.waves * NT * 64 * sizeof(f32x4), stream>>>(
      static_cast<const typename Elem<SRC>::type*>(a.data), a.row_stride, int(a.rows), int(a.cols), w, offsets,
      int(experts), uint32_t(ceil_div(out.cols, 16 * NT)), static_cast<typename Elem<DT>::type*>(out.data), out.row_stride);
  return hipGetLastError();
}

template <int SRC, int DT>
hipError_t product_as(const GroupPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b, const int32_t* offsets,
                      int64_t experts, const reshard_matrix_t& out, hipStream_t stream) {
  switch (plan.n_tiles) {
    case 1: return rows_as<SRC, DT, 1>(plan, a, b, offsets, experts, out, stream);
    case 2: return rows_as<SRC, DT, 2>(plan, a, b, offsets, experts, out, stream);
    default:
      if constexpr (Parts<SRC>::count == 1) return rows_as<SRC, DT, 4>(plan, a, b, offsets, experts, out, stream);
  }
  return hipErrorInvalidValue;
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
  // Which form, by the rows of a weight (us): a's rows over the experts, which is all that the
  // host knows, and too many where some are no held expert's.  Up to 16, 16 x 14336 x 4096 11.4
  // with the form for few rows and 13.9 with tiles of 64; up to 64, 33 x 14336 x 4096 18.3 with
  // those.  Larger tiles where they fill the card: 512 x 14336 x 4096 63 with 128 x 128, 73 with
  // 64 x 128; 64 experts' 9600 rows 417 and 450, their 4800 294 and 290; 4096 x 14336 x 4096 445
  // with 256 x 256, 64 experts' 16384 rows 603 and 645 with 128 x 128, their 4800 393 and 294.
  const int64_t mean = experts ? a.rows / experts : a.rows;
  if (mean > kRowsHeight && groups_of(a.cols) >= 8 && out.cols && stride <= (int64_t(1) << 22)) {
    if (tiles(256, 256) >= 192 && out.cols > 128 && (!experts || mean >= 192)) {
      p.form = GroupPlan::kTiles256;
      p.whole = experts ? 0 : whole_tiles(tiles(256, 256));
      p.groups = experts ? tiles(256, 256) : 2 * tiles(256, 256) - p.whole;
    } else if (tiles(128, 128) >= 256 && mean > 64) {
      p.form = GroupPlan::kTiles128;
      p.whole = p.groups = tiles(128, 128);
    } else {
      p.form = GroupPlan::kTiles64;
      p.groups = tiles(64, 128);
    }
    p.part_steps = uint32_t(part_steps);
    p.steps = uint32_t(parts * part_steps);
    p.steps_per_split = p.steps;
    if (!direct) p.planes = round_up(a.rows * parts * part_steps * 128, 256);
    if (p.form == GroupPlan::kTiles64 && !experts) {
      // a workgroup a CU shares the contractions, six steps at least each (128 x 14336 x 4096
      // 25 us, with two a CU 28)
      const int64_t t = p.groups;
      const int64_t splits = std::max<int64_t>(1, std::min(kCus / t, ceil_div(p.steps, 6)));
      p.steps_per_split = uint32_t(ceil_div(ceil_div(p.steps, splits), 3) * 3);
      p.splits = int(ceil_div(p.steps, p.steps_per_split));
      p.whole = p.groups = t * p.splits;
      if (p.splits > 1) p.parts = p.splits * out.rows * round_up(out.cols, 4) * 4;
    }
    return p;
  }
  // As many columns a workgroup as leave 200 of them: what a costs is a workgroup's reading
  // of all of it (16 x 14336 x 4096 11.4 us with 64 columns, 14.4 with 32).  Elements in
  // parts have registers for 32.
  const int most = parts == 1 ? 4 : 2;
  p.n_tiles = 1;
  while (p.n_tiles < most && tiles(kRowsHeight, 32 * p.n_tiles) >= 200) p.n_tiles *= 2;
  p.groups = tiles(kRowsHeight, 16 * p.n_tiles);
  const int64_t runs = std::max<int64_t>(1, ceil_div(a.cols / kBlockCols, kRun));
  p.waves = int(ceil_div(runs, ceil_div(runs, kMaxWaves)));
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
