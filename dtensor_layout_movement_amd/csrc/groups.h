// Group-scaled 4-bit matrices and tokens sorted by expert: the launch interface of
// their kernels (group_quantize.hip, group_matmul.hip, expert_route.hip), used by
// the host code of the C ABI (groups.hip).  The callers have checked every argument.
#pragma once

#include "blocks.h"

namespace rs {

constexpr int kGroup = RESHARD_GROUP;

inline int64_t groups_of(int64_t cols) { return ceil_div(cols, kGroup); }

hipError_t launch_group_quantize(const reshard_matrix_t& src, const reshard_matrix_t& dst, hipStream_t stream);
hipError_t launch_group_dequantize(const reshard_matrix_t& src, const reshard_matrix_t& dst, hipStream_t stream);

// How a product by 4-bit weights runs: workspace bytes and launches.
struct GroupPlan {
  enum Form { kRows, kTiles64, kTiles128, kTiles256 };
  Form form = kRows;
  int waves = 0;                  // of a workgroup, and its tiles of 16 columns (kRows)
  int n_tiles = 1;
  int64_t groups = 0;             // workgroups of the product
  int64_t whole = 0;              // of them those that make a whole tile, or a split of one (tiles)
  uint32_t steps = 0;             // of a tile's contraction, and of one part of a's
  uint32_t part_steps = 0;
  int splits = 1;                 // workgroups that share a tile's contraction (kTiles64)
  uint32_t steps_per_split = 0;
  int64_t planes = 0;             // bytes of a's bfloat16 parts in the workspace (0: read as it lies)
  int64_t parts = 0;              // bytes of the splits' sums
  int64_t bytes() const { return planes + parts; }
};
// `experts` matrices of b.rows / experts rows each; 0: b is one matrix for all rows of a.
GroupPlan plan_group_matmul(const reshard_matrix_t& a, const reshard_matrix_t& b, int64_t experts,
                            const reshard_matrix_t& out);
hipError_t launch_group_matmul(const GroupPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b,
                               const int32_t* offsets, int64_t experts, const reshard_matrix_t& out, void* workspace,
                               hipStream_t stream);

// The tiled forms of it.
hipError_t launch_group_tiles(const GroupPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b,
                              const int32_t* offsets, int64_t experts, const reshard_matrix_t& out, void* workspace,
                              hipStream_t stream);

constexpr int kMaxExperts = RESHARD_MAX_EXPERTS;
constexpr int64_t kMaxChosen = int64_t(1) << 30;  // tokens times choices

struct SortPlan {
  int64_t blocks = 0;  // workgroups that count and place; 1: one launch
  int64_t rounds = 0;  // of kSortThreads choices each takes
  int64_t bytes = 0;   // workspace: the blocks' counts
};
SortPlan plan_sort(int64_t chosen, int64_t experts);
hipError_t launch_sort(const SortPlan& plan, const void* ids, bool wide, int64_t chosen, int64_t first, int experts,
                       int32_t* offsets, int32_t* position, void* workspace, hipStream_t stream);

hipError_t launch_gather(const reshard_matrix_t& x, const int32_t* position, int choices, const reshard_matrix_t& rows,
                         hipStream_t stream);
hipError_t launch_combine(const reshard_matrix_t& rows, const int32_t* position, int choices,
                          const reshard_matrix_t* weights, const reshard_matrix_t& out, hipStream_t stream);
hipError_t launch_combine_grad(const reshard_matrix_t& dout, const reshard_matrix_t* rows, const int32_t* position,
                               int choices, const reshard_matrix_t* weights, const reshard_matrix_t* drows,
                               const reshard_matrix_t* dweights, hipStream_t stream);

}  // namespace rs
