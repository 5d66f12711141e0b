// Block-scaled 8-bit matrices: the launch interface of their kernels
// (block_quantize.hip, block_matmul.hip, block_grad.hip), used by the host code
// of the C ABI (blocks.hip).  The callers have checked every matrix.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "reshard.h"

namespace rs {

// Keeps `msg` as the calling thread's last error and returns `s` (reshard.hip).
reshard_status_t report(reshard_status_t s, const std::string& msg);

constexpr int kBlock = RESHARD_BLOCK;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }
inline int64_t blocks_of(int64_t cols) { return ceil_div(cols, kBlock); }

// Of n tiles that take a CU each, those whose rounds over the card are full; where
// the rest are at most half a round, two workgroups share each of them (4096 x 14336
// in tiles of 256 x 256 is 3.5 rounds: a product over 4096 columns takes 261 us for 302
// with it, a weight gradient over 4096 rows 459 for 486).  Otherwise all n.
constexpr int64_t kCus = 256;
inline int64_t whole_tiles(int64_t n) { return n % kCus <= kCus / 2 && n > kCus ? n / kCus * kCus : n; }

// Workgroups of one launch at most: a dispatch counts its work-items in 32 bits
// (512 of them in the largest workgroup used here).
constexpr int64_t kMaxGroups = (int64_t(1) << 23) - 1;

hipError_t launch_quantize(const reshard_matrix_t& src, const reshard_matrix_t& dst, const reshard_matrix_t* dst_t,
                           hipStream_t stream);
hipError_t launch_dequantize(const reshard_matrix_t& src, const reshard_matrix_t& dst, hipStream_t stream);

// How a product runs: workspace bytes and launches.
struct MatmulPlan {
  enum Form { kRows, kRing16, kRing32, kRing64, kTiles128, kTiles256 };
  Form form = kRows;
  int waves = 0;             // of a workgroup (kRows)
  bool fused = false;        // a plain a is quantized by the product's own workgroups (kRows)
  bool too_wide = false;     // a stride that the form does not take
  int splits = 1;            // workgroups that share a tile's contraction (kRing)
  uint32_t steps_per_split = 0;
  int64_t whole = 0;         // tiles of which each is one workgroup's (kTiles)
  int64_t groups = 0;        // workgroups of the product
  int64_t quantized = 0;     // bytes of a's quantized payload in the workspace (0: not needed)
  int64_t quantized_scales = 0;
  int64_t parts = 0;         // bytes of the splits' sums
  int64_t bytes() const { return quantized + quantized_scales + parts; }
};
MatmulPlan plan_matmul(const reshard_matrix_t& a, const reshard_matrix_t& b, const reshard_matrix_t& out);
hipError_t launch_matmul(const MatmulPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b,
                         const reshard_matrix_t& out, void* workspace, hipStream_t stream);

// Sums n_parts binary32 matrices (rows of out.cols rounded up to 4 elements,
// `part_stride` elements apart) in order into `out`, or adds the sum to it.
hipError_t launch_join(const float* parts, int n_parts, int64_t part_stride, const reshard_matrix_t& out,
                       bool accumulate, hipStream_t stream);

// Columns of dy and rows of dy times its bfloat16 planes, at most: a step's rows
// within 32-bit offsets, and rows in 32 bits.
constexpr int64_t kMaxGradCols = int64_t(1) << 24, kMaxGradRows = int64_t(3) << 29;
int64_t grad_planes(int dtype);

struct GradPlan {
  int tile = 0;                  // rows and columns of a tile of dw
  int splits = 1;                // workgroups that share a tile's contraction
  uint32_t steps_per_split = 1;
  int64_t whole = 0;             // workgroups of a whole tile, or a split of one
  int64_t groups = 0;
  bool direct = false;           // dy is read where it lies
  int64_t planes = 0;            // bytes of dy as bfloat16 planes in the workspace
  int64_t parts = 0;             // bytes of the splits' sums
  int64_t bytes() const { return planes + parts; }
};
GradPlan plan_grad(const reshard_matrix_t& dy, const reshard_matrix_t& x, const reshard_matrix_t& dw);
hipError_t launch_grad(const GradPlan& plan, const reshard_matrix_t& dy, const reshard_matrix_t& x,
                       const reshard_matrix_t& dw, bool accumulate, void* workspace, hipStream_t stream);

}  // namespace rs
