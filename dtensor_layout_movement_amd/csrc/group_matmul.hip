// out = a b^T with group-scaled 4-bit weights b (the format is in reshard.h), one
// weight for all rows or one for each expert's rows.
#include "block_device.h"
#include "groups.h"

#include <algorithm>

namespace rs {
namespace {

// b as the kernels read it; expert e's rows start at e * rows.
struct Weight {
  const uint8_t* data;
  int64_t stride;  // bytes
  const uint8_t* scales;
  int64_t scale_stride;
  int rows;  // of one expert
};

// The rows of a that a workgroup multiplies, and by which weight.
struct Chunk {
  int expert, first, last;
};

// The slot-th chunk of at most `height` rows, counting every expert's own, each of
// them cut to the `rows` there are.  Every wave finds it for itself, 64 experts at a
// time.  False: there are fewer.
__device__ __forceinline__ bool find_chunk(const int32_t* offsets, int experts, int rows, int slot, int height, Chunk* c) {
  if (!offsets) {
    *c = Chunk{0, slot * height, min(slot * height + height, rows)};
    return c->first < rows;
  }
  const int lane = threadIdx.x & 63;
  for (int base = 0; base < experts; base += 64) {
    const int e = min(base + lane, experts - 1);
    const int lo = min(max(offsets[e], 0), rows), hi = min(max(offsets[e + 1], lo), rows);
    const int n = base + lane < experts ? (hi - lo + height - 1) / height : 0;
    int upto = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int other = __shfl_up(upto, d);
      if (lane >= d) upto += other;
    }
    const uint64_t past = __ballot(upto > slot);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int first = __builtin_amdgcn_readlane(lo, l) + (slot - __builtin_amdgcn_readlane(upto - n, l)) * height;
      *c = Chunk{base + l, first, min(first + height, __builtin_amdgcn_readlane(hi, l))};
      return true;
    }
    slot -= __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// Eight 4-bit elements times a power of two as bfloat16: exact in bfloat16's normal
// range (two significant bits).
__device__ __forceinline__ bf16x8 widen8_fp4(uint32_t q, float scale) {
  bf16x2 p[4];
  p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
  p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
  p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
  p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
  bf16x8 r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}

// bfloat16 parts that add up to an element of a: its leading bits, those that follow,
// and so on, each cut off (so that a part of a finite element is finite).
template <int DT> struct Parts;
template <> struct Parts<RESHARD_DTYPE_BF16> { static constexpr int count = 1; };
template <> struct Parts<RESHARD_DTYPE_F16> { static constexpr int count = 2; };
template <> struct Parts<RESHARD_DTYPE_F32> { static constexpr int count = 3; };

// The bits of a part, and what is left of x (nothing of infinities and NaN).
__device__ __forceinline__ uint32_t take_part(float* x) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, *x);
  const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
  // a NaN keeps its quiet bit: cut off, its payload might be an infinity's
  const uint32_t part = ((bits & 0x7fffffffu) > 0x7f800000u ? bits | 0x00400000u : bits) & 0xffff0000u;
  *x = finite ? *x - __builtin_bit_cast(float, part) : 0.f;
  return part >> 16;
}

// Eight elements of a row from column c on, zero past `cols`, as parts.
template <int DT, bool GUARD>
__device__ __forceinline__ void load_parts(const typename Elem<DT>::type* p, int c, int cols, bf16x8 (&y)[Parts<DT>::count]) {
  typedef typename Elem<DT>::type T;
  Pack<T, 8> v;
  if (!GUARD || c + 8 <= cols) {
    v = load_pack<T, 8>(p + c);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.v[i] = c + i < cols ? p[c + i] : T(0.f);
  }
  if constexpr (DT == RESHARD_DTYPE_BF16) {
    __builtin_memcpy(&y[0], &v, sizeof(v));
  } else {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = Elem<DT>::up(v.v[i]);
#pragma unroll
    for (int n = 0; n < Parts<DT>::count; ++n) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = take_part(&x[2 * i]), hi = take_part(&x[2 * i + 1]);
        w[i] = lo | hi << 16;
      }
      __builtin_memcpy(&y[n], w, sizeof(w));
    }
  }
}

// Four neighbouring results, of which `left` are inside the row.
template <int DT>
__device__ __forceinline__ void store4(typename Elem<DT>::type* p, const f32x4& v, int left) {
  Pack<typename Elem<DT>::type, 4> r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r.v[e] = Elem<DT>::down(v[e]);
  if (left >= 4) {
    store_pack<typename Elem<DT>::type, 4>(p, r);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) p[e] = r.v[e];
  }
}

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
  const uint32_t id = run_of(blockIdx.x, gridDim.x);
  Chunk c;
  if (!find_chunk(offsets, experts, rows, int(id / n_tiles), kRowsHeight, &c)) return;
  const int n0 = int(id % n_tiles) * 16, part = lane >> 4;
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

GroupPlan plan_group_matmul(const reshard_matrix_t& a, const reshard_matrix_t&, int64_t experts,
                            const reshard_matrix_t& out) {
  GroupPlan p;
  // every expert with a row may end in a chunk that is not full
  const int64_t ends = std::max<int64_t>(1, std::min(experts, a.rows));
  p.slots = a.rows ? ends + (a.rows - ends) / kRowsHeight + (experts ? 0 : 1) : 0;
  if (!experts) p.slots = ceil_div(a.rows, kRowsHeight);
  p.groups = p.slots * ceil_div(out.cols, 16);
  const int64_t blocks = ceil_div(a.cols, 4 * kGroup);
  p.waves = 4;
  while (p.waves < kMaxWaves && p.groups * p.waves < 4096 && p.waves < blocks) p.waves *= 2;
  return p;
}

hipError_t launch_group_matmul(const GroupPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b,
                               const int32_t* offsets, int64_t experts, const reshard_matrix_t& out, void*,
                               hipStream_t stream) {
  switch (a.dtype) {
    case RESHARD_DTYPE_F32: return product_from<RESHARD_DTYPE_F32>(plan, a, b, offsets, experts, out, stream);
    case RESHARD_DTYPE_BF16: return product_from<RESHARD_DTYPE_BF16>(plan, a, b, offsets, experts, out, stream);
    default: return product_from<RESHARD_DTYPE_F16>(plan, a, b, offsets, experts, out, stream);
  }
}

}  // namespace rs
