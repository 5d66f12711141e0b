// Device helpers of the block-scaled kernels: float formats, scale bytes and
// vector types.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "plan.h"
#include "reshard.h"

namespace rs {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Workgroup `id` of `n` by the order in which workgroups go to the 8 XCDs in turn,
// so that each XCD takes a contiguous run.
__device__ __forceinline__ uint32_t run_of(uint32_t id, uint32_t n) {
  const uint32_t xcd = id % 8;
  return xcd * (n / 8) + min(xcd, n % 8) + id / 8;
}

// n / d for n < 2^31 by a multiplier (magic_u31 of plan.h).
struct Divisor {
  uint32_t d, m, s;
};
__device__ __forceinline__ uint32_t quotient(uint32_t n, const Divisor& v) { return (__umulhi(n, v.m) + n) >> v.s; }
inline Divisor divisor(uint32_t d) {
  Divisor v{d, 0, 0};
  magic_u31(d, &v.m, &v.s);
  return v;
}

// Keeps a value in registers at this point of the program: no use of it moves
// above, no computation of it below.
template <typename T> __device__ __forceinline__ void pin(T& x) {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("" : "+v"(x));
#endif
}

// Memory read by 32-bit offsets (no load reaches past its `bytes`).
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, int(bytes), 0x00020000);
}

// 16 bytes a lane from `lane_off + off` straight to LDS: lane l's to byte 16 l from
// `to` on, the same `to` and `off` for the whole wave.
__device__ __forceinline__ void load_to_lds(Buffer from, uint8_t* to, uint32_t lane_off, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) uint32_t*)to, 16, int(lane_off),
                                           int(off), 0, 0);
}

// Waits for all but `left` of this wave's loads (to LDS too) and for its LDS accesses,
// then for the other waves: what they loaded is there, what they read may be written.
// __syncthreads does not say this of loads to LDS: the compiler adds the wait where it
// follows them to the barrier, but not, for one, around a loop that loads under a
// condition.
template <int LEFT> __device__ __forceinline__ void loads_barrier() {
#ifdef __HIP_DEVICE_COMPILE__
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((LEFT & 15) | ((LEFT >> 4) << 14) | (7 << 4));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#endif
}

// Element types by their dtype code.
template <int DT> struct Elem;
template <> struct Elem<RESHARD_DTYPE_F32> {
  typedef float type;
  static __device__ float up(float x) { return x; }
  static __device__ float down(float x) { return x; }
};
template <> struct Elem<RESHARD_DTYPE_BF16> {
  typedef __bf16 type;
  static __device__ float up(__bf16 x) { return float(x); }
  static __device__ __bf16 down(float x) { return __bf16(x); }  // to nearest, ties to even
};
template <> struct Elem<RESHARD_DTYPE_F16> {
  typedef _Float16 type;
  static __device__ float up(_Float16 x) { return float(x); }
  static __device__ _Float16 down(float x) { return _Float16(x); }
};

// N elements from or to any address aligned to one element (gfx950 global
// accesses need no alignment: one wide access each).
template <typename T, int N> struct Pack {
  T v[N];
};
template <typename T, int N> __device__ __forceinline__ Pack<T, N> load_pack(const T* p) {
  Pack<T, N> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}
template <typename T, int N> __device__ __forceinline__ void store_pack(T* p, const Pack<T, N>& r) {
  __builtin_memcpy(p, &r, sizeof(r));
}

// A store past the caches, for what is not read again soon.
template <int B> struct Words;
template <> struct Words<4> { typedef uint32_t type __attribute__((aligned(1))); };
template <> struct Words<8> { typedef uint32_t type __attribute__((ext_vector_type(2), aligned(1))); };
template <> struct Words<16> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(1))); };
template <typename T, int N> __device__ __forceinline__ void store_stream(T* p, const Pack<T, N>& r) {
  constexpr int B = sizeof(T) * N > 16 ? 16 : sizeof(T) * N;
  typedef typename Words<B>::type W;
#pragma unroll
  for (int i = 0; i < int(sizeof(T)) * N / B; ++i) {
    W w;
    __builtin_memcpy(&w, reinterpret_cast<const char*>(&r) + i * B, B);
    __builtin_nontemporal_store(w, reinterpret_cast<W*>(p) + i);
  }
}

template <int N> struct Index {
  static constexpr int value = N;
};
template <int N, typename F> __device__ __forceinline__ void for_each_index(F f) {
  if constexpr (N > 0) {
    for_each_index<N - 1>(f);
    f(Index<N - 1>{});
  }
}

// Where 16-byte chunk `chunk` of row `row` of a tile lies, rows 128 bytes apart in LDS: 16
// rows' reads of one chunk fall into distinct banks.
__device__ __forceinline__ int slot_of(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

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

// 2^(b - 127) of a scale byte (255: NaN, 0: the subnormal 2^-127).
__device__ __forceinline__ float scale_value(uint32_t b) {
  const uint32_t bits = b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23;
  return __builtin_bit_cast(float, bits);
}

// The bits of |x| where x is finite, else 0: as unsigned integers they order as
// the magnitudes do.
__device__ __forceinline__ uint32_t finite_magnitude(float x) {
  const uint32_t m = __builtin_bit_cast(uint32_t, x) & 0x7fffffffu;
  return m < 0x7f800000u ? m : 0u;
}

// The scale byte of a block whose largest finite magnitude has bits `amax`.  The
// format's largest value is 1.75 * 2^t (t = 8 for E4M3, 15 for E5M2), so with
// amax = m * 2^x, 1 <= m < 2, the exponent is x - t, one more where m > 1.75,
// and at least -127.
template <bool E5M2> __device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax == 0) return 127;
  const int e = int(amax >> 23) - (E5M2 ? 15 : 8) + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return uint32_t(max(e, 0));
}

// 2^(127 - b), the inverse of a scale that scale_byte gave (b <= 247: a normal
// number), by which an element is multiplied exactly before it is rounded.
__device__ __forceinline__ float inverse_scale(uint32_t b) {
  return __builtin_bit_cast(float, (254u - b) << 23);
}

// Four elements times `inv`, rounded to 8 bits; what is not finite becomes NaN
// (E5M2 has infinities, which the conversion would give).
template <bool E5M2> __device__ __forceinline__ uint32_t quantize4(float a, float b, float c, float d, float inv) {
  if (E5M2) {
    const auto nan = [](float x) {
      return (__builtin_bit_cast(uint32_t, x) & 0x7fffffffu) < 0x7f800000u ? x : __builtin_nanf("");
    };
    a = nan(a), b = nan(b), c = nan(c), d = nan(d);
    int r = __builtin_amdgcn_cvt_pk_bf8_f32(a * inv, b * inv, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_bf8_f32(c * inv, d * inv, r, true));
  }
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, r, true));
}

// N elements of a row from column c on as binary32, zero past `cols`.
template <int DT, int N>
__device__ __forceinline__ void load_up(const typename Elem<DT>::type* p, int c, int cols, float* x) {
  typedef typename Elem<DT>::type T;
  if (c + N <= cols) {
    const Pack<T, N> v = load_pack<T, N>(p + c);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = Elem<DT>::up(v.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = c + i < cols ? Elem<DT>::up(p[c + i]) : 0.f;
  }
}

// The largest of 16 neighbouring lanes, in all of them.
template <int CTRL> __device__ __forceinline__ uint32_t max_with(uint32_t v) {
  return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xf, 0xf, true)));
}
__device__ __forceinline__ uint32_t max_of_16(uint32_t v) {
  v = max_with<0xb1>(v);      // lane ^ 1
  v = max_with<0x4e>(v);      // lane ^ 2
  v = max_with<0x141>(v);     // 7 - lane of 8
  return max_with<0x140>(v);  // 15 - lane of 16
}

// Eight elements as payload bytes.
template <bool E5M2> __device__ __forceinline__ i32x2 quantize8(const float* x, float inv) {
  return i32x2{int(quantize4<E5M2>(x[0], x[1], x[2], x[3], inv)), int(quantize4<E5M2>(x[4], x[5], x[6], x[7], inv))};
}

// Four 8-bit elements as binary32 (exact).
template <bool E5M2> __device__ __forceinline__ f32x4 widen4(uint32_t q) {
  f32x4 r;
  if (E5M2) {
    r[0] = __builtin_amdgcn_cvt_f32_bf8(int(q), 0);
    r[1] = __builtin_amdgcn_cvt_f32_bf8(int(q), 1);
    r[2] = __builtin_amdgcn_cvt_f32_bf8(int(q), 2);
    r[3] = __builtin_amdgcn_cvt_f32_bf8(int(q), 3);
  } else {
    r[0] = __builtin_amdgcn_cvt_f32_fp8(int(q), 0);
    r[1] = __builtin_amdgcn_cvt_f32_fp8(int(q), 1);
    r[2] = __builtin_amdgcn_cvt_f32_fp8(int(q), 2);
    r[3] = __builtin_amdgcn_cvt_f32_fp8(int(q), 3);
  }
  return r;
}

// Eight 8-bit elements times a power of two as bfloat16: exact while the value
// stays in bfloat16's normal range (three significant bits and the hidden one).
template <bool E5M2> __device__ __forceinline__ bf16x8 widen8_bf16(uint32_t lo, uint32_t hi, float scale) {
  bf16x2 p[4];
  if (E5M2) {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, scale, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, scale, true);
  } else {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  }
  bf16x8 r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}

}  // namespace rs
