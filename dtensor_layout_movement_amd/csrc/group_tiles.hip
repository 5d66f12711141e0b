// out = a b^T with group-scaled 4-bit weights b: the tiled form, for products of many
// rows (the form for few is in group_matmul.hip).
#include "group_device.h"
#include "groups.h"

#include <algorithm>

namespace rs {
namespace {

// a as bfloat16 rows: as it lies, or its parts one behind the other (split_rows).
struct Rows {
  const uint8_t* data;
  int64_t stride;   // bytes
  int rows;
  uint32_t chunks;  // of 8 columns that a row has, parts together
};

constexpr int kStep = 64;                        // columns of a step
constexpr int kThree = 3;                         // steps that share a load of the weight
constexpr int kRowA = kStep * 2, kRowB = kThree * kStep / 2;  // bytes of a row of a step, and of three

// A workgroup makes a BM (rows of a) x BN (rows of b) tile with WM x WN waves.  A step
// takes 64 columns of a through LDS, loaded straight there (16 bytes a lane) two steps
// ahead into the third of three buffers; rows lie 128 bytes apart, their 16-byte chunks
// permuted (slot_of).  The weight goes there three steps at a time, 96 bytes a row, into
// the other of two buffers: with 32 bytes a row each step, three of four loads found their
// line still on its way, which holds up the first cache (a third of all cycles of 4096 x
// 14336 x 4096).  A lane (row, quarter q) reads 16 consecutive columns of its row on both
// sides, 8 for each of two instructions, and widens the weight's to bfloat16, scaled, in
// registers: one scale of the row's two.  The scales of three steps (6 bytes a row) are
// loaded into registers, as they lie: a shift there would wait for them.  SHARED: by one
// thread a row and through LDS (512 x 14336 x 4096 72 -> 63 us; neighbouring lanes that each
// read another row cost the first cache a line each).  In tiles of 256 rows, whose registers
// are full, by every lane that uses them.
//
// 256 x 256 tiles: 4096 x 14336 x 4096 takes 445 us (1080 TFLOP/s; the library's product of
// bfloat16 matrices 406), with an MFMA pipe that is busy for 45% of the time; of 440, 382 were
// left without the loads and 435 without the conversions.  128 x 128, two workgroups a CU:
// 512 x 14336 x 4096 63 us.  64 x 128: 33 x 4096 x 14336 14 us and 4 for the join.
template <int DT, int BM, int BN, int WM, int WN, bool SHARED>
__device__ __forceinline__ void make_tile(const Rows& a, const Weight& b, int groups, const Chunk& c, int n0,
                                          uint32_t first, uint32_t last, uint32_t part_steps,
                                          typename Elem<DT>::type* out, int64_t out_stride, uint8_t* a0, uint8_t* a1,
                                          uint8_t* a2, uint8_t* b0, uint8_t* b1, uint64_t* row_scales) {
  constexpr int kThreads = 64 * WM * WN, kM = BM / WM / 16, kN = BN / WN / 16;
  constexpr int kLoadsA = BM * 8 / kThreads, kLoadsB = BN * 6 / kThreads;
  static_assert(kM > 2 && kThreads % 128 == 0 && BN * 6 % kThreads == 0 && BM * 8 % kThreads == 0, "");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN, frow = lane & 15, part = lane >> 4;
  const int m_rows = c.last - c.first, n_rows = min(BN, b.rows - n0);
  const int64_t row_b0 = int64_t(c.expert) * b.rows + n0;
  // rows past a tile's last lie past the buffer's end, where a load fetches nothing and gives zeros
  const Buffer base_a = buffer_of(a.data + c.first * a.stride, uint32_t(m_rows - 1) * uint32_t(a.stride) + a.chunks * 16);
  const Buffer base_b = buffer_of(b.data + row_b0 * b.stride,
                                  uint32_t(n_rows - 1) * uint32_t(b.stride) + uint32_t(groups) * (kGroup / 2));
  // rows of one thread's loads are a multiple of 16 apart: they have one chunk in common
  const uint32_t chunk = uint32_t(slot_of(int(threadIdx.x) >> 3, int(threadIdx.x) & 7));
  const uint32_t off_a = (threadIdx.x >> 3) * uint32_t(a.stride) + chunk * 16;
  const auto load_a = [&](uint8_t* to, uint32_t k) {
    const bool inside = k * 8 + chunk < a.chunks;
#pragma unroll
    for (int i = 0; i < kLoadsA; ++i)
      load_to_lds(base_a, to + (i * kThreads + wave * 64) * 16,
                  inside ? off_a + uint32_t(i * (kThreads / 8)) * uint32_t(a.stride) : 0x7ffffff0u, k * kRowA);
  };
  uint32_t off_b[kLoadsB];
#pragma unroll
  for (int i = 0; i < kLoadsB; ++i) {
    const uint32_t at = threadIdx.x + i * kThreads;
    off_b[i] = at / 6 * uint32_t(b.stride) + at % 6 * 16;
  }
  // Three steps of the weight from step kb on.  (What lies past a row's groups meets zeros of
  // a; loads past the contraction's last step are made to no use.)
  const uint32_t last_b = uint32_t(groups - 1) / 6 * 3;
  const auto load_b = [&](uint8_t* to, uint32_t kb) {
#pragma unroll
    for (int i = 0; i < kLoadsB; ++i)
      load_to_lds(base_b, to + (i * kThreads + wave * 64) * 16, off_b[i], min(kb, last_b) * (kStep / 2));
  };

  // Eight scale bytes of a row of the weight for its steps kb to kb + 2, whose first is at bit
  // scales_at(kb): the row's last eight at most.  Past the last group the byte is 0 or 1 (the
  // last one's top bit): what lies there, whatever it is, has to be finite, since a is zero.
  const uint8_t* scales = b.scales + row_b0 * b.scale_stride;
  const auto scales_at = [&](uint32_t kb) { return 8 * (int(kb) * 2 - min(int(kb) * 2, groups - 8)); };
  constexpr int kScaleRows = SHARED ? 1 : kN;
  uint32_t off_s[kScaleRows];
#pragma unroll
  for (int i = 0; i < kScaleRows; ++i)
    off_s[i] = uint32_t(min(SHARED ? int(threadIdx.x) : wn * (BN / WN) + i * 16 + frow, n_rows - 1)) * uint32_t(b.scale_stride);
  uint64_t loaded[kScaleRows];
  const auto load_scales = [&](uint32_t kb) {
    if (!SHARED || threadIdx.x < BN) {
#pragma unroll
      for (int i = 0; i < kScaleRows; ++i)
        __builtin_memcpy(&loaded[i], scales + (off_s[i] + uint32_t(min(int(kb) * 2, groups - 8))), 8);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto share_scales = [&] {
    if (SHARED && threadIdx.x < BN) row_scales[threadIdx.x] = loaded[0];
  };
  uint64_t s[kN];
  const auto take_scales = [&] {
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i] = SHARED ? row_scales[wn * (BN / WN) + i * 16 + frow] : loaded[i % kScaleRows];
  };

  f32x4 acc[kN][kM];
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int j = 0; j < kM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // where this lane's chunks lie in a tile: rows 16 apart keep their slots
  const int slot0 = slot_of(frow, 2 * part) * 16, slot1 = slot_of(frow, 2 * part + 1) * 16;
  const int row_a = (wm * (BM / WM) + frow) * kRowA, row_b = (wn * (BN / WN) + frow) * kRowB + part * 8;
  struct Fragment {
    bf16x8 half[2];
  };
  const auto fragment_a = [&](const uint8_t* tile, int j) {
    Fragment f;
    f.half[0] = *reinterpret_cast<const bf16x8*>(tile + row_a + slot0 + j * (16 * kRowA));
    f.half[1] = *reinterpret_cast<const bf16x8*>(tile + row_a + slot1 + j * (16 * kRowA));
    return f;
  };
  // the weight's columns of a step and the first rows of a, read before the step begins
  i32x2 raw[kN];
  Fragment x;
  const auto begin = [&](const uint8_t* tile, const uint8_t* weight, int third) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      raw[i] = *reinterpret_cast<const i32x2*>(weight + row_b + i * (16 * kRowB) + third * (kStep / 2));
    x = fragment_a(tile, 0);
  };
  Fragment w[kN];
  const auto products = [&](auto J, const Fragment& xj) {
    constexpr int j = decltype(J)::value;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kN; ++i)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i].half[h], xj.half[h], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // `fill` asks for what comes later, behind the step's first reads; `turn`, between the
  // step's last read and its last products, waits for the next step's and reads its first.
  const auto step = [&](const uint8_t* tile, const uint64_t (&s)[kN], int bit, auto fill, auto turn) {
    const int by = min(bit + 8 * (part >> 1), 63);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const float f = scale_of(uint32_t(s[i] >> by), 0);
      w[i].half[0] = widen8_fp4(uint32_t(raw[i][0]), f);
      w[i].half[1] = widen8_fp4(uint32_t(raw[i][1]), f);
    }
    Fragment next = fragment_a(tile, 1);
    __builtin_amdgcn_s_setprio(1);
    for_each_index<kM - 2>([&](auto J) {
      const Fragment second = fragment_a(tile, decltype(J)::value + 2);
      if constexpr (decltype(J)::value == 0) fill();
      products(J, x);
      x = next;
      next = second;
    });
    __builtin_amdgcn_s_setprio(0);
    const Fragment xl = x;
    turn();
    products(Index<kM - 2>{}, xl);
    products(Index<kM - 1>{}, next);
  };

  // Every load is made at every turn, past the last step to no use: then the loads under
  // way behind those that a barrier waits for are known, a's next but one step at least
  // and, while they are young, the weight's next three.  (Scales come on top of them: a
  // barrier that waits for more than it has to is no fault.)
  uint32_t kb = first % part_steps, k = first;
  load_scales(kb);
  load_b(b0, kb);
  load_a(a0, first);
  load_a(a1, min(first + 1, last - 1));
  share_scales();
  loads_barrier<kLoadsA>();
  take_scales();
  begin(a0, b0, 0);
  uint32_t kn;  // the weight's next three: it starts over for a's next part
  int bit;
  const auto first_of = [&](const uint8_t* now, uint8_t* later) {
    kn = kb + 3 < part_steps ? kb + 3 : 0;
    bit = scales_at(kb);
    if constexpr (SHARED) load_scales(kn);
    step(a0, s, bit, [&] { load_a(a2, min(k + 2, last - 1)); load_b(later, kn); }, [&] {
      loads_barrier<kLoadsA + kLoadsB>();  // a1 has arrived, a0 has been read
      begin(a1, now, 1);
    });
  };
  const auto second_of = [&](const uint8_t* now) {
    step(a1, s, bit + 16, [&] { load_a(a0, min(k + 3, last - 1)); }, [&] {
      share_scales();  // those before were taken before the last barrier
      loads_barrier<kLoadsA + kLoadsB>();
      begin(a2, now, 2);
    });
  };
  const auto third_of = [&](const uint8_t* later) {
    step(a2, s, bit + 32, [&] {
      if constexpr (!SHARED) load_scales(kn);
      load_a(a1, min(k + 4, last - 1));
    }, [&] {
      loads_barrier<kLoadsA>();  // the next three steps' weight too
      take_scales();             // this step's are in use already
      begin(a0, later, 0);
    });
    kb = kn;
    k += 3;
  };
  while (k + 6 <= last) {
    first_of(b0, b1);
    second_of(b0);
    third_of(b1);
    first_of(b1, b0);
    second_of(b1);
    third_of(b0);
  }
  // (the rest in one line of steps: with branches that join the sums do not stay in place)
  const uint32_t left = last - k;
  if (left > 0) first_of(b0, b1);
  if (left > 1) second_of(b0);
  if (left > 2) third_of(b1);
  if (left > 3) first_of(b1, b0);
  if (left > 4) second_of(b1);
  loads_barrier<0>();  // no load may outlive its use of LDS
#pragma unroll
  for (int j = 0; j < kM; ++j) {
    const int m = wm * (BM / WM) + j * 16 + frow;
    if (m >= m_rows) continue;
    typename Elem<DT>::type* row = out + int64_t(c.first + m) * out_stride + n0;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int n = wn * (BN / WN) + i * 16 + part * 4;
      store4<DT>(row + n, acc[i][j], n_rows - n);
    }
  }
}

// Bands of kBand rows of tiles: what is in flight on an XCD is nearly square and shares
// the most in its L2.
constexpr uint32_t kBand = 8;

// Tiles of 256 rows with at most 128 of them are made as tiles of 128; workgroups from
// `whole` on, which would leave half of the card idle in the last round, make half a tile
// each.
template <int DT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void group_tiles(Rows a, Weight b, int groups, const int32_t* offsets,
                                                               int experts, uint32_t m_tiles, uint32_t n_tiles,
                                                               uint32_t whole, uint32_t steps, uint32_t part_steps,
                                                               uint32_t steps_per_split,
                                                               typename Elem<DT>::type* out, int64_t out_stride,
                                                               int64_t split_stride) {
  __shared__ __align__(128) uint8_t a0[BM * kRowA];
  __shared__ __align__(128) uint8_t a1[BM * kRowA];
  __shared__ __align__(128) uint8_t a2[BM * kRowA];
  __shared__ __align__(128) uint8_t b0[BN * kRowB];
  __shared__ __align__(128) uint8_t b1[BN * kRowB];
  constexpr bool kShared = BM < 256;
  __shared__ uint64_t row_scales[kShared ? BN : 1];
  Chunk c;
  uint32_t n_tile, split = 0;
  if (offsets) {
    if (!find_tile(offsets, experts, a.rows, BM, blockIdx.x, n_tiles, &c, &n_tile)) return;
  } else {
    const uint32_t tiles = m_tiles * n_tiles;
    uint32_t t, half = 2;
    if (blockIdx.x < whole) {
      split = blockIdx.x / tiles;
      t = run_of(blockIdx.x % tiles, min(tiles, whole));
    } else {
      const uint32_t i = run_of(blockIdx.x - whole, gridDim.x - whole);
      t = whole + i / 2;
      half = i % 2;
    }
    const uint32_t band = t / (kBand * n_tiles), rows = min(kBand, m_tiles - band * kBand), in = t - band * kBand * n_tiles;
    const int first = int(band * kBand + in % rows) * BM;
    c = Chunk{0, first, min(first + BM, a.rows)};
    n_tile = in / rows;
    if (half < 2) {
      c = Chunk{0, first + int(half) * (BM / 2), min(first + int(half + 1) * (BM / 2), a.rows)};
      if (c.first >= c.last) return;
    }
  }
  const uint32_t first = split * steps_per_split, last = min(first + steps_per_split, steps);
  if (BM == 256 && c.last - c.first <= BM / 2)
    make_tile<DT, BM == 256 ? 128 : BM, BN, WM, WN, kShared>(a, b, groups, c, int(n_tile) * BN, first, last, part_steps,
                                                    out + split * split_stride, out_stride, a0, a1, a2, b0, b1, row_scales);
  else
    make_tile<DT, BM, BN, WM, WN, kShared>(a, b, groups, c, int(n_tile) * BN, first, last, part_steps, out + split * split_stride,
                                  out_stride, a0, a1, a2, b0, b1, row_scales);
}

// The bfloat16 parts of a's rows, one behind the other, each of `width` columns, zero past
// the matrix's.  Eight columns a lane.
template <int SRC>
__global__ __launch_bounds__(256) void split_rows(const typename Elem<SRC>::type* a, int64_t stride, int cols,
                                                  Divisor chunks, uint32_t items, uint8_t* to, int64_t to_stride) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= items) return;
  const uint32_t row = quotient(i, chunks), chunk = i - row * chunks.d;
  bf16x8 y[Parts<SRC>::count];
  load_parts<SRC>(a + int64_t(row) * stride, int(chunk) * 8, cols, y);
#pragma unroll
  for (int n = 0; n < Parts<SRC>::count; ++n)
    *reinterpret_cast<bf16x8*>(to + int64_t(row) * to_stride + (uint32_t(n) * chunks.d + chunk) * 16) = y[n];
}

template <int SRC>
hipError_t split_as(const reshard_matrix_t& a, int64_t width, void* to, hipStream_t stream) {
  typedef typename Elem<SRC>::type T;
  const int64_t chunks = width / 8, stride = width * 2 * Parts<SRC>::count, rows = rows_per_launch(chunks, 256);
  for (int64_t r = 0; r < a.rows; r += rows) {
    const uint32_t items = uint32_t(std::min(rows, a.rows - r) * chunks);
    split_rows<SRC><<<dim3(uint32_t(ceil_div(items, 256))), 256, 0, stream>>>(
        static_cast<const T*>(a.data) + r * a.row_stride, a.row_stride, int(a.cols), divisor(uint32_t(chunks)), items,
        static_cast<uint8_t*>(to) + r * stride, stride);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int DT, int BM, int BN, int WM, int WN>
hipError_t tiles_as(const GroupPlan& plan, const Rows& a, const Weight& b, int groups, const int32_t* offsets,
                    int64_t experts, void* out, int64_t out_stride, int64_t split_stride, hipStream_t stream) {
  group_tiles<DT, BM, BN, WM, WN><<<dim3(uint32_t(plan.groups)), 64 * WM * WN, 0, stream>>>(
      a, b, groups, offsets, int(experts), uint32_t(ceil_div(a.rows, BM)), uint32_t(ceil_div(b.rows, BN)),
      uint32_t(plan.whole), plan.steps,
      plan.part_steps, plan.steps_per_split, static_cast<typename Elem<DT>::type*>(out), out_stride, split_stride);
  return hipGetLastError();
}

template <int DT>
hipError_t tiles_to(const GroupPlan& plan, const Rows& a, const Weight& b, int groups, const int32_t* offsets,
                    int64_t experts, void* out, int64_t out_stride, int64_t split_stride, hipStream_t stream) {
  switch (plan.form) {
    case GroupPlan::kTiles64:
      return tiles_as<DT, 64, 128, 1, 4>(plan, a, b, groups, offsets, experts, out, out_stride, split_stride, stream);
    case GroupPlan::kTiles128:
      return tiles_as<DT, 128, 128, 2, 2>(plan, a, b, groups, offsets, experts, out, out_stride, split_stride, stream);
    default:
      return tiles_as<DT, 256, 256, 2, 4>(plan, a, b, groups, offsets, experts, out, out_stride, split_stride, stream);
  }
}

}  // namespace

hipError_t launch_group_tiles(const GroupPlan& plan, const reshard_matrix_t& a, const reshard_matrix_t& b,
                              const int32_t* offsets, int64_t experts, const reshard_matrix_t& out, void* workspace,
                              hipStream_t stream) {
  Rows rows{static_cast<const uint8_t*>(a.data), a.row_stride * 2, int(a.rows), uint32_t(a.cols / 8)};
  if (plan.planes) {
    const int64_t width = int64_t(plan.part_steps) * kStep;
    hipError_t e;
    switch (a.dtype) {
      case RESHARD_DTYPE_F32: e = split_as<RESHARD_DTYPE_F32>(a, width, workspace, stream); break;
      case RESHARD_DTYPE_BF16: e = split_as<RESHARD_DTYPE_BF16>(a, width, workspace, stream); break;
      default: e = split_as<RESHARD_DTYPE_F16>(a, width, workspace, stream);
    }
    if (e != hipSuccess) return e;
    const int64_t bytes = int64_t(plan.steps) * kStep * 2;
    rows = Rows{static_cast<const uint8_t*>(workspace), bytes, int(a.rows), uint32_t(bytes / 16)};
  }
  const Weight w{static_cast<const uint8_t*>(b.data), b.row_stride / 2, static_cast<const uint8_t*>(b.scales),
                 b.scale_stride, int(out.cols)};
  const int groups = int(groups_of(b.cols));
  if (plan.splits > 1) {
    float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.planes);
    const int64_t stride = round_up(out.cols, 4), size = out.rows * stride;
    const hipError_t e = tiles_to<RESHARD_DTYPE_F32>(plan, rows, w, groups, nullptr, 0, parts, stride, size, stream);
    if (e != hipSuccess) return e;
    return launch_join(parts, plan.splits, size, out, false, stream);
  }
  switch (out.dtype) {
    case RESHARD_DTYPE_F32:
      return tiles_to<RESHARD_DTYPE_F32>(plan, rows, w, groups, offsets, experts, out.data, out.row_stride, 0, stream);
    case RESHARD_DTYPE_BF16:
      return tiles_to<RESHARD_DTYPE_BF16>(plan, rows, w, groups, offsets, experts, out.data, out.row_stride, 0, stream);
    default:
      return tiles_to<RESHARD_DTYPE_F16>(plan, rows, w, groups, offsets, experts, out.data, out.row_stride, 0, stream);
  }
}

}  // namespace rs
