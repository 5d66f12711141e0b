// Tokens sorted by expert, their rows moved there and back, and the gradients of the
// way back (the definitions are in reshard.h).
#include "block_device.h"
#include "groups.h"

#include <algorithm>

namespace rs {
namespace {

// ------------------------------------------------------------------- sorting
//
// A stable counting sort.  A choice's row is its expert's offset plus the choices of
// that expert before it.  Workgroup b takes a run of consecutive choices, kSortThreads
// a round: a first launch counts its experts, a second adds the counts of the
// workgroups before it to the offsets and places its choices round by round.  Within
// a round a choice's rank is its wave's (lanes below with the same expert, found
// with a ballot for each bit of the expert's number) plus what the waves before
// counted.  Bound by latency: the data are a few bytes a choice.

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kOneLaunchRounds = 4;  // choices that one workgroup takes alone, in rounds
constexpr int kMaxSortBlocks = 128;

// The held expert of choice i, or -1.
template <typename I>
__device__ __forceinline__ int expert_of(const I* ids, uint32_t i, uint32_t chosen, int64_t first, int experts) {
  if (i >= chosen) return -1;
  const uint64_t e = uint64_t(int64_t(ids[i]) - first);
  return e < uint64_t(experts) ? int(e) : -1;
}

// Exclusive sums over a workgroup's threads, and the sum of all.
__device__ __forceinline__ int sums_before(int v, int* wave_sums, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int upto = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int other = __shfl_up(upto, d);
    if (lane >= d) upto += other;
  }
  __syncthreads();  // the last use of wave_sums is over
  if (lane == 63) wave_sums[wave] = upto;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    const int s = wave_sums[w];
    if (w < wave) before += s;
    all += s;
  }
  *total = all;
  return before + upto - v;
}

template <typename I>
__global__ __launch_bounds__(kSortThreads) void count_choices(const I* ids, uint32_t chosen, int64_t first, int experts,
                                                              uint32_t rounds, int* counts) {
  __shared__ int mine[kMaxExperts];
  for (int e = threadIdx.x; e < experts; e += kSortThreads) mine[e] = 0;
  __syncthreads();
  for (uint32_t r = 0; r < rounds; ++r) {
    const int e = expert_of(ids, (blockIdx.x * rounds + r) * kSortThreads + threadIdx.x, chosen, first, experts);
    if (e >= 0) atomicAdd(&mine[e], 1);  // whole numbers: their order does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += kSortThreads) counts[blockIdx.x * experts + e] = mine[e];
}

// ALONE: one workgroup, which counts for itself.
template <typename I, bool ALONE>
__global__ __launch_bounds__(kSortThreads) void place_choices(const I* ids, uint32_t chosen, int64_t first, int experts,
                                                              int bits, uint32_t rounds, const int* counts,
                                                              int32_t* offsets, int32_t* position) {
  __shared__ int next[kMaxExperts];                      // the row that the expert's next choice gets
  __shared__ uint16_t of_wave[kSortWaves][kMaxExperts];  // a round's choices by wave
  __shared__ int wave_sums[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e0 = threadIdx.x;
  int own[kOneLaunchRounds];
  int before = 0, all = 0;  // of expert e0: in the workgroups before this one, and in all
  for (int e = threadIdx.x; e < experts; e += kSortThreads) {
    next[e] = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) of_wave[w][e] = 0;
  }
  if constexpr (ALONE) {
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kOneLaunchRounds; ++r) {
      own[r] = expert_of(ids, r * kSortThreads + threadIdx.x, chosen, first, experts);
      if (own[r] >= 0) atomicAdd(&next[own[r]], 1);
    }
    __syncthreads();
    if (e0 < experts) all = next[e0];
  } else if (e0 < experts) {
    for (uint32_t b = 0; b < gridDim.x; ++b) {
      const int n = counts[b * experts + e0];
      all += n;
      if (b < blockIdx.x) before += n;
    }
  }
  int total;
  const int offset = sums_before(all, wave_sums, &total);
  if (e0 < experts) {
    next[e0] = offset + before;
    if (blockIdx.x == 0) offsets[e0] = offset;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[experts] = total;

  const auto place = [&](uint32_t i, int e) {
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(e >> b & 1);
      same &= e >> b & 1 ? set : ~set;
    }
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    const bool leads = e >= 0 && rank == 0;
    if (leads) of_wave[wave][e] = uint16_t(__popcll(same));
    __syncthreads();
    int row = -1;
    if (e >= 0) {
      row = next[e] + rank;
      for (int w = 0; w < wave; ++w) row += of_wave[w][e];
    }
    __syncthreads();
    if (leads) {
      atomicAdd(&next[e], __popcll(same));
      of_wave[wave][e] = 0;
    }
    if (i < chosen) position[i] = row;
  };
  __syncthreads();
  if constexpr (ALONE) {
#pragma unroll
    for (int r = 0; r < kOneLaunchRounds; ++r)
      if (uint32_t(r) < rounds) {  // the same for all threads
        place(r * kSortThreads + threadIdx.x, own[r]);
        __syncthreads();
      }
  } else {
    for (uint32_t r = 0; r < rounds; ++r) {
      const uint32_t i = (blockIdx.x * rounds + r) * kSortThreads + threadIdx.x;
      place(i, expert_of(ids, i, chosen, first, experts));
      __syncthreads();
    }
  }
}

// --------------------------------------------------------------------- moving
//
// Bound by HBM: a token's row is read (written) once and the rows of its choices are
// written (read) once.  A lane takes 16 bytes of a token's row, consecutive lanes
// consecutive pieces, and all the choices of that token.

constexpr int kThreads = 256;

template <typename T> constexpr int piece_of() { return 16 / int(sizeof(T)); }

// N elements from column c on, of which those past `cols` are zero.
template <typename T, int N> __device__ __forceinline__ Pack<T, N> load_piece(const T* p, int c, int cols) {
  if (c + N <= cols) return load_pack<T, N>(p + c);
  Pack<T, N> v;
#pragma unroll
  for (int i = 0; i < N; ++i) v.v[i] = c + i < cols ? p[c + i] : T(0);
  return v;
}
template <typename T, int N> __device__ __forceinline__ void store_piece(T* p, int c, int cols, const Pack<T, N>& v) {
  if (c + N <= cols) {
    store_pack<T, N>(p + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < cols) p[c + i] = v.v[i];
  }
}

// T: an unsigned integer of the elements' size (the copy is by bits).
template <typename T>
__global__ __launch_bounds__(kThreads) void gather_rows(const T* x, int64_t x_stride, int cols, Divisor pieces,
                                                        uint32_t items, const int32_t* position, int choices, T* rows,
                                                        int64_t rows_stride, uint32_t n_rows) {
  constexpr int N = piece_of<T>();
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= items) return;
  const uint32_t token = quotient(i, pieces);
  const int c = int(i - token * pieces.d) * N;
  const Pack<T, N> v = load_piece<T, N>(x + int64_t(token) * x_stride, c, cols);
  const int32_t* p = position + int64_t(token) * choices;
  for (int j = 0; j < choices; ++j) {
    const uint32_t row = uint32_t(p[j]);
    if (row < n_rows) store_piece<T, N>(rows + int64_t(row) * rows_stride, c, cols, v);
  }
}

// Weights of any type, or none.
struct Scalars {
  const void* data;
  int64_t stride;
  int dtype;
};
__device__ __forceinline__ float scalar_at(const Scalars& s, int64_t row, int col) {
  if (!s.data) return 1.f;
  const int64_t at = row * s.stride + col;
  if (s.dtype == RESHARD_DTYPE_F32) return static_cast<const float*>(s.data)[at];
  if (s.dtype == RESHARD_DTYPE_BF16) return float(static_cast<const __bf16*>(s.data)[at]);
  return float(static_cast<const _Float16*>(s.data)[at]);
}

// Four choices' pieces are on their way together.
constexpr int kTogether = 4;

template <int DT>
__global__ __launch_bounds__(kThreads) void combine_rows(const typename Elem<DT>::type* rows, int64_t rows_stride,
                                                         uint32_t n_rows, const int32_t* position, int choices,
                                                         Scalars weights, Divisor pieces, uint32_t items,
                                                         typename Elem<DT>::type* out, int64_t out_stride, int cols) {
  typedef typename Elem<DT>::type T;
  constexpr int N = piece_of<T>();
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= items) return;
  const uint32_t token = quotient(i, pieces);
  const int c = int(i - token * pieces.d) * N;
  const int32_t* p = position + int64_t(token) * choices;
  float sum[N];
#pragma unroll
  for (int k = 0; k < N; ++k) sum[k] = 0.f;
  for (int j = 0; j < choices; j += kTogether) {
    Pack<T, N> v[kTogether];
    float w[kTogether];
    bool has[kTogether];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      has[u] = false;
      if (j + u >= choices) continue;
      const uint32_t row = uint32_t(p[j + u]);
      has[u] = row < n_rows;
      if (!has[u]) continue;
      v[u] = load_piece<T, N>(rows + int64_t(row) * rows_stride, c, cols);
      w[u] = scalar_at(weights, token, j + u);
    }
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
      if (has[u]) {
#pragma unroll
        for (int k = 0; k < N; ++k) sum[k] = fmaf(w[u], Elem<DT>::up(v[u].v[k]), sum[k]);
      }
  }
  Pack<T, N> v;
#pragma unroll
  for (int k = 0; k < N; ++k) v.v[k] = Elem<DT>::down(sum[k]);
  store_piece<T, N>(out + int64_t(token) * out_stride, c, cols, v);
}

// A workgroup of WAVES waves a token, up to kBatch of its choices at a time: dout's row is
// read once for each batch, each choice's row of the forward pass once, and the
// choice's gradient row written once.  The products' sums go over a lane's pieces, then
// over a wave's lanes, then over the waves, always in this order.
constexpr int kBatch = 8;

template <int DT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void combine_grad(const typename Elem<DT>::type* dout, int64_t dout_stride,
                                                           const typename Elem<DT>::type* rows, int64_t rows_stride,
                                                           const int32_t* position, int choices, Scalars weights,
                                                           typename Elem<DT>::type* drows, int64_t drows_stride,
                                                           uint32_t n_rows, void* dweights, int64_t dweights_stride,
                                                           int dweights_dtype, int cols) {
  typedef typename Elem<DT>::type T;
  constexpr int N = piece_of<T>();
  __shared__ float wave_sums[WAVES][kBatch];
  const int64_t token = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const T* d = dout + token * dout_stride;
  for (int j0 = 0; j0 < choices; j0 += kBatch) {
    uint32_t row[kBatch];
    float w[kBatch], sum[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      row[u] = j0 + u < choices ? uint32_t(position[token * choices + j0 + u]) : ~0u;
      w[u] = row[u] < n_rows && drows ? scalar_at(weights, token, j0 + u) : 0.f;
      sum[u] = 0.f;
    }
    for (int c = int(threadIdx.x) * N; c < cols; c += 64 * WAVES * N) {
      const Pack<T, N> g = load_piece<T, N>(d, c, cols);
      float x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = Elem<DT>::up(g.v[k]);
      if (dweights) {
        Pack<T, N> v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (row[u] < n_rows) v[u] = load_piece<T, N>(rows + int64_t(row[u]) * rows_stride, c, cols);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (row[u] < n_rows) {
#pragma unroll
            for (int k = 0; k < N; ++k) sum[u] = fmaf(x[k], Elem<DT>::up(v[u].v[k]), sum[u]);
          }
      }
      if (drows) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (row[u] < n_rows) {
            Pack<T, N> v;
#pragma unroll
            for (int k = 0; k < N; ++k) v.v[k] = Elem<DT>::down(w[u] * x[k]);
            store_piece<T, N>(drows + int64_t(row[u]) * drows_stride, c, cols, v);
          }
      }
    }
    if (!dweights) continue;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
#pragma unroll
      for (int m = 32; m >= 1; m /= 2) sum[u] += __shfl_xor(sum[u], m);
      if (lane == 0) wave_sums[wave][u] = sum[u];
    }
    __syncthreads();
    if (threadIdx.x < kBatch && j0 + int(threadIdx.x) < choices) {
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < WAVES; ++v) s += wave_sums[v][threadIdx.x];
      const int64_t at = token * dweights_stride + j0 + threadIdx.x;
      if (dweights_dtype == RESHARD_DTYPE_F32) static_cast<float*>(dweights)[at] = s;
      else if (dweights_dtype == RESHARD_DTYPE_BF16) static_cast<__bf16*>(dweights)[at] = __bf16(s);
      else static_cast<_Float16*>(dweights)[at] = _Float16(s);
    }
    __syncthreads();
  }
}

// Tokens that one launch takes: their pieces within 31 bits.
template <typename F> hipError_t in_launches(int64_t tokens, int64_t pieces, F launch) {
  const int64_t most = rows_per_launch(pieces, kThreads);
  for (int64_t t = 0; t < tokens; t += most) {
    const int64_t n = std::min(most, tokens - t);
    launch(t, uint32_t(n * pieces), dim3(uint32_t(ceil_div(n * pieces, kThreads))));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

Scalars scalars(const reshard_matrix_t* m, int64_t row) {
  if (!m) return Scalars{nullptr, 0, 0};
  const int64_t size = m->dtype == RESHARD_DTYPE_F32 ? 4 : 2;
  return Scalars{static_cast<const uint8_t*>(m->data) + row * m->row_stride * size, m->row_stride, m->dtype};
}

template <typename T>
hipError_t gather_as(const reshard_matrix_t& x, const int32_t* position, int choices, const reshard_matrix_t& rows,
                     hipStream_t stream) {
  const int64_t pieces = ceil_div(x.cols, piece_of<T>());
  return in_launches(x.rows, pieces, [&](int64_t t, uint32_t items, dim3 grid) {
    gather_rows<T><<<grid, kThreads, 0, stream>>>(static_cast<const T*>(x.data) + t * x.row_stride, x.row_stride,
                                                  int(x.cols), divisor(uint32_t(pieces)), items, position + t * choices,
                                                  choices, static_cast<T*>(rows.data), rows.row_stride,
                                                  uint32_t(rows.rows));
  });
}

template <int DT>
hipError_t combine_as(const reshard_matrix_t& rows, const int32_t* position, int choices, const reshard_matrix_t* weights,
                      const reshard_matrix_t& out, hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const int64_t pieces = ceil_div(out.cols, piece_of<T>());
  return in_launches(out.rows, pieces, [&](int64_t t, uint32_t items, dim3 grid) {
    combine_rows<DT><<<grid, kThreads, 0, stream>>>(
        static_cast<const T*>(rows.data), rows.row_stride, uint32_t(rows.rows), position + t * choices, choices,
        scalars(weights, t), divisor(uint32_t(pieces)), items, static_cast<T*>(out.data) + t * out.row_stride,
        out.row_stride, int(out.cols));
  });
}

template <int DT, int WAVES>
hipError_t grad_as(const reshard_matrix_t& dout, const reshard_matrix_t* rows, const int32_t* position, int choices,
                   const reshard_matrix_t* weights, const reshard_matrix_t* drows, const reshard_matrix_t* dweights,
                   hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const uint32_t n_rows = uint32_t(rows ? rows->rows : drows->rows);
  for (int64_t t = 0; t < dout.rows; t += kMaxGroups) {
    uint8_t* dw = nullptr;
    if (dweights)
      dw = static_cast<uint8_t*>(dweights->data) + t * dweights->row_stride * (dweights->dtype == RESHARD_DTYPE_F32 ? 4 : 2);
    combine_grad<DT, WAVES><<<dim3(uint32_t(std::min(kMaxGroups, dout.rows - t))), 64 * WAVES, 0, stream>>>(
        static_cast<const T*>(dout.data) + t * dout.row_stride, dout.row_stride,
        rows ? static_cast<const T*>(rows->data) : nullptr, rows ? rows->row_stride : 0, position + t * choices, choices,
        scalars(weights, t), drows ? static_cast<T*>(drows->data) : nullptr, drows ? drows->row_stride : 0, n_rows, dw,
        dweights ? dweights->row_stride : 0, dweights ? dweights->dtype : 0, int(dout.cols));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

SortPlan plan_sort(int64_t chosen, int64_t experts) {
  SortPlan p;
  const int64_t rounds = ceil_div(chosen, kSortThreads);
  if (rounds <= kOneLaunchRounds) {
    p.blocks = 1;
    p.rounds = rounds;
    return p;
  }
  p.rounds = ceil_div(rounds, kMaxSortBlocks);
  p.blocks = ceil_div(rounds, p.rounds);
  p.bytes = p.blocks * experts * int64_t(sizeof(int));
  return p;
}

template <typename I>
static hipError_t sort_as(const SortPlan& plan, const I* ids, int64_t chosen, int64_t first, int experts, int32_t* offsets,
                          int32_t* position, void* workspace, hipStream_t stream) {
  int bits = 0;
  while ((1 << bits) < experts) ++bits;
  if (plan.blocks == 1) {
    place_choices<I, true><<<dim3(1), kSortThreads, 0, stream>>>(ids, uint32_t(chosen), first, experts, bits,
                                                                 uint32_t(plan.rounds), nullptr, offsets, position);
    return hipGetLastError();
  }
  int* counts = static_cast<int*>(workspace);
  count_choices<I><<<dim3(uint32_t(plan.blocks)), kSortThreads, 0, stream>>>(ids, uint32_t(chosen), first, experts,
                                                                             uint32_t(plan.rounds), counts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  place_choices<I, false><<<dim3(uint32_t(plan.blocks)), kSortThreads, 0, stream>>>(
      ids, uint32_t(chosen), first, experts, bits, uint32_t(plan.rounds), counts, offsets, position);
  return hipGetLastError();
}

hipError_t launch_sort(const SortPlan& plan, const void* ids, bool wide, int64_t chosen, int64_t first, int experts,
                       int32_t* offsets, int32_t* position, void* workspace, hipStream_t stream) {
  if (wide)
    return sort_as(plan, static_cast<const int64_t*>(ids), chosen, first, experts, offsets, position, workspace, stream);
  return sort_as(plan, static_cast<const int32_t*>(ids), chosen, first, experts, offsets, position, workspace, stream);
}

hipError_t launch_gather(const reshard_matrix_t& x, const int32_t* position, int choices, const reshard_matrix_t& rows,
                         hipStream_t stream) {
  if (x.dtype == RESHARD_DTYPE_F32) return gather_as<uint32_t>(x, position, choices, rows, stream);
  return gather_as<uint16_t>(x, position, choices, rows, stream);
}

hipError_t launch_combine(const reshard_matrix_t& rows, const int32_t* position, int choices,
                          const reshard_matrix_t* weights, const reshard_matrix_t& out, hipStream_t stream) {
  switch (out.dtype) {
    case RESHARD_DTYPE_F32: return combine_as<RESHARD_DTYPE_F32>(rows, position, choices, weights, out, stream);
    case RESHARD_DTYPE_BF16: return combine_as<RESHARD_DTYPE_BF16>(rows, position, choices, weights, out, stream);
    default: return combine_as<RESHARD_DTYPE_F16>(rows, position, choices, weights, out, stream);
  }
}

hipError_t launch_combine_grad(const reshard_matrix_t& dout, const reshard_matrix_t* rows, const int32_t* position,
                               int choices, const reshard_matrix_t* weights, const reshard_matrix_t* drows,
                               const reshard_matrix_t* dweights, hipStream_t stream) {
  if (!dweights) rows = nullptr;
  const auto as = [&](auto narrow, auto wide) {
    // a wave a token where its row is at most a piece a lane of four waves
    return dout.cols * (dout.dtype == RESHARD_DTYPE_F32 ? 4 : 2) <= 64 * 16 ? narrow() : wide();
  };
  switch (dout.dtype) {
    case RESHARD_DTYPE_F32:
      return as([&] { return grad_as<RESHARD_DTYPE_F32, 1>(dout, rows, position, choices, weights, drows, dweights, stream); },
                [&] { return grad_as<RESHARD_DTYPE_F32, 4>(dout, rows, position, choices, weights, drows, dweights, stream); });
    case RESHARD_DTYPE_BF16:
      return as([&] { return grad_as<RESHARD_DTYPE_BF16, 1>(dout, rows, position, choices, weights, drows, dweights, stream); },
                [&] { return grad_as<RESHARD_DTYPE_BF16, 4>(dout, rows, position, choices, weights, drows, dweights, stream); });
    default:
      return as([&] { return grad_as<RESHARD_DTYPE_F16, 1>(dout, rows, position, choices, weights, drows, dweights, stream); },
                [&] { return grad_as<RESHARD_DTYPE_F16, 4>(dout, rows, position, choices, weights, drows, dweights, stream); });
  }
}

}  // namespace rs
