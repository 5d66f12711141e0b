// Device helpers of the products by group-scaled 4-bit weights.
#pragma once

#include "block_device.h"

namespace rs {

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

// Chunks of at most `height` rows, counting every expert's own, of the experts base to
// base + 63: lane l has expert base + l's first and last row, cut to the `rows` there
// are, its chunks and the sum of those up to it.
struct Counted {
  int lo, hi, n, upto;
};
__device__ __forceinline__ Counted count_chunks(const int32_t* offsets, int experts, int rows, int height, int base) {
  const int lane = threadIdx.x & 63, e = min(base + lane, experts - 1);
  Counted c;
  c.lo = min(max(offsets[e], 0), rows);
  c.hi = min(max(offsets[e + 1], c.lo), rows);
  c.n = base + lane < experts ? (c.hi - c.lo + height - 1) / height : 0;
  c.upto = c.n;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int other = __shfl_up(c.upto, d);
    if (lane >= d) c.upto += other;
  }
  return c;
}

// The tile of a workgroup: a chunk of rows and, of `n_tiles`, the columns.  The tiles that
// there are go to the XCDs in contiguous runs, chunk by chunk; workgroups past them
// have none (false).  Every wave finds it for itself.
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int experts, int rows, int height, uint32_t id,
                                          uint32_t n_tiles, Chunk* c, uint32_t* n_tile) {
  Counted of = count_chunks(offsets, experts, rows, height, 0);
  int total = __builtin_amdgcn_readlane(of.upto, 63);
  for (int base = 64; base < experts; base += 64)
    total += __builtin_amdgcn_readlane(count_chunks(offsets, experts, rows, height, base).upto, 63);
  if (id >= uint32_t(total) * n_tiles) return false;
  const uint32_t t = run_of(id, uint32_t(total) * n_tiles);
  int slot = int(t / n_tiles);
  *n_tile = t % n_tiles;
  // (bounded, and cut to the expert's rows: offsets that overlap may count more chunks
  // than an integer holds)
  for (int base = 0; base < experts; base += 64) {
    if (base) of = count_chunks(offsets, experts, rows, height, base);
    const uint64_t past = __ballot(of.upto > slot);
    if (past) {
      const int l = __builtin_ctzll(past), lo = __builtin_amdgcn_readlane(of.lo, l), hi = __builtin_amdgcn_readlane(of.hi, l);
      const int first = lo + (slot - __builtin_amdgcn_readlane(of.upto - of.n, l)) * height;
      *c = Chunk{base + l, first, min(first + height, hi)};
      return first >= lo && first < hi;
    }
    slot -= __builtin_amdgcn_readlane(of.upto, 63);
  }
  return false;
}

// The scale of scale byte `at` of a word, as the conversions take it: they read its exponent
// only, of which 0 is 2^-127 and 255 NaN.
__device__ __forceinline__ float scale_of(uint32_t word, int at) {
  const uint32_t exponent = at < 3 ? word << (23 - 8 * at) : word >> 1;
  return __builtin_bit_cast(float, exponent & 0x7f800000u);
}

// Eight 4-bit elements times a power of two as bfloat16: exact (two significant bits, from
// 2^-128 on, a subnormal, which the matrix instructions take as it is), infinite where 4 or 6
// is scaled by 2^126, or 2 and more by 2^127.
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

// What a load of 16 bytes a lane costs the first cache are the lines that neighbouring
// lanes touch: 16 where a quad of lanes reads 64 bytes of one of 16 rows, 64 where
// neighbouring lanes read different rows.  So rows are read by quads, and what lane 4 r + q
// read goes to lane r + 16 q, where the matrix instructions take it.
__device__ __forceinline__ int from_quads() { return int(((threadIdx.x & 15) * 4 + (threadIdx.x >> 4 & 3)) * 4); }
template <typename T> __device__ __forceinline__ T permuted(const T& v, int from) {
  static_assert(sizeof(T) % 4 == 0, "");
  int w[sizeof(T) / 4];
  __builtin_memcpy(w, &v, sizeof(T));
#pragma unroll
  for (int i = 0; i < int(sizeof(T) / 4); ++i) w[i] = __builtin_amdgcn_ds_bpermute(from, w[i]);
  T r;
  __builtin_memcpy(&r, w, sizeof(T));
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

// Eight elements as parts.
template <int DT>
__device__ __forceinline__ void split8(const Pack<typename Elem<DT>::type, 8>& v, bf16x8 (&y)[Parts<DT>::count]) {
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

// Eight elements of a row from column c on, zero past `cols`, as parts.
template <int DT>
__device__ __forceinline__ void load_parts(const typename Elem<DT>::type* p, int c, int cols, bf16x8 (&y)[Parts<DT>::count]) {
  typedef typename Elem<DT>::type T;
  Pack<T, 8> v;
  if (c + 8 <= cols) {
    v = load_pack<T, 8>(p + c);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v.v[i] = c + i < cols ? p[c + i] : T(0.f);
  }
  split8<DT>(v, y);
}

}  // namespace rs
