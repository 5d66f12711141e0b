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
// that expert before it.  A workgroup takes a run of consecutive choices, kSortThreads
// a round, and gives each its rank among its expert's in the run: within a wave from
// the lanes below that have the same expert (a ballot for each bit of the expert's
// number), plus what the waves and the rounds before counted.  One workgroup then adds
// the offsets itself; several leave their counts to a second launch, which adds what
// the runs before hold too.  Bound by latency: the data are a few bytes a choice.  8
// choices take 2.9 us, 32768 of 64 experts 8.5 (13.9 with the counts in the first launch and
// the ranks in the second).

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kAloneRounds = 4;  // choices that one workgroup takes alone, in rounds
constexpr int kMaxSortBlocks = 128;

// The held expert of choice i, or -1.
template <typename I>
__device__ __forceinline__ int expert_of(const I* ids, uint32_t i, uint32_t chosen, int64_t first, int experts) {
  if (i >= chosen) return -1;
  const uint64_t e = uint64_t(int64_t(ids[i]) - first);
  return e < uint64_t(experts) ? int(e) : -1;
}

// Sums over the threads before one of a workgroup, and over all.
__device__ __forceinline__ int sums_before(int v, int* wave_sums, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int upto = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int other = __shfl_up(upto, d);
    if (lane >= d) upto += other;
  }
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

// ALONE: one workgroup for all choices.
template <typename I, bool ALONE>
__global__ __launch_bounds__(kSortThreads) void rank_choices(const I* ids, uint32_t chosen, int64_t first, int experts,
                                                             int bits, uint32_t rounds, int* counts, int32_t* offsets,
                                                             int32_t* position) {
  __shared__ int counted[kMaxExperts];                   // in the rounds before
  __shared__ uint16_t of_wave[kSortWaves][kMaxExperts];  // a round's choices by wave
  __shared__ int wave_sums[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, e0 = threadIdx.x;
  const auto choice = [&](uint32_t r) { return (blockIdx.x * rounds + r) * kSortThreads + threadIdx.x; };
  int own[kAloneRounds], rank_of[kAloneRounds];
  if constexpr (ALONE) {
#pragma unroll
    for (int r = 0; r < kAloneRounds; ++r) own[r] = expert_of(ids, choice(r), chosen, first, experts);
  }
  for (int e = lane; e < experts; e += 64) of_wave[wave][e] = 0;
  if (e0 < experts) counted[e0] = 0;
  __syncthreads();

  // the rank of this round's choice; a barrier has to follow before the next
  const auto rank = [&](int e) {
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot(e >> b & 1);
      same &= e >> b & 1 ? set : ~set;
    }
    const int below = __popcll(same & ((uint64_t(1) << lane) - 1));
    const bool leads = e >= 0 && below == 0;
    if (leads) of_wave[wave][e] = uint16_t(__popcll(same));
    __syncthreads();
    int n = -1;
    if (e >= 0) {
      n = counted[e] + below;
#pragma unroll
      for (int w = 0; w < kSortWaves - 1; ++w) n += w < wave ? of_wave[w][e] : 0;
    }
    __syncthreads();
    if (leads) {
      atomicAdd(&counted[e], __popcll(same));  // whole numbers: their order does not matter
      of_wave[wave][e] = 0;
    }
    return n;
  };
  if constexpr (ALONE) {
#pragma unroll
    for (int r = 0; r < kAloneRounds; ++r)
      if (uint32_t(r) < rounds) {  // the same for all threads
        rank_of[r] = rank(own[r]);
        __syncthreads();
      }
    int total;
    const int offset = sums_before(e0 < experts ? counted[e0] : 0, wave_sums, &total);
    __syncthreads();
    if (e0 < experts) offsets[e0] = counted[e0] = offset;
    if (e0 == 0) offsets[experts] = total;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kAloneRounds; ++r)
      if (choice(r) < chosen) position[choice(r)] = own[r] >= 0 ? counted[own[r]] + rank_of[r] : -1;
  } else {
    for (uint32_t r = 0; r < rounds; ++r) {
      const int n = rank(expert_of(ids, choice(r), chosen, first, experts));
      if (choice(r) < chosen) position[choice(r)] = n;
      __syncthreads();
    }
    if (e0 < experts) counts[blockIdx.x * experts + e0] = counted[e0];
  }
}

// The second launch of several runs: adds the offsets and the counts of the runs before.
// A run's counts are read by 2^bits threads, at least one an expert.
template <typename I>
__global__ __launch_bounds__(kSortThreads) void place_choices(const I* ids, uint32_t chosen, int64_t first, int experts,
                                                              int bits, uint32_t rounds, const int* counts,
                                                              int32_t* offsets, int32_t* position) {
  __shared__ int all[kMaxExperts], before[kMaxExperts];
  __shared__ int wave_sums[kSortWaves];
  const int e0 = threadIdx.x, e = e0 & ((1 << bits) - 1);
  all[e0] = before[e0] = 0;
  __syncthreads();
  if (e < experts) {
    int n = 0, earlier = 0;
#pragma unroll 8
    for (uint32_t b = uint32_t(e0) >> bits; b < gridDim.x; b += kSortThreads >> bits) {
      const int c = counts[b * experts + e];
      n += c;
      earlier += b < blockIdx.x ? c : 0;
    }
    atomicAdd(&all[e], n);
    atomicAdd(&before[e], earlier);
  }
  __syncthreads();
  int total;
  const int offset = sums_before(e0 < experts ? all[e0] : 0, wave_sums, &total);
  if (e0 < experts) {
    before[e0] += offset;
    if (blockIdx.x == 0) offsets[e0] = offset;
  }
  if (blockIdx.x == 0 && e0 == 0) offsets[experts] = total;
  __syncthreads();
  for (uint32_t r = 0; r < rounds; ++r) {
    const uint32_t i = (blockIdx.x * rounds + r) * kSortThreads + threadIdx.x;
    const int mine = expert_of(ids, i, chosen, first, experts);
    if (mine >= 0) position[i] += before[mine];
  }
}

// --------------------------------------------------------------------- moving
//
// Bound by HBM: a token's row is read (written) once and the rows of its choices are
// written (read) once.  A lane takes 16 bytes of a token's row, consecutive lanes
// consecutive pieces, and all the choices of that token.  4096 tokens of 7168 bf16
// columns with 8 choices each, 529 MB one way: gather 91 us (5.8 TB/s), combine 94 (5.6),
// its gradient, twice the bytes, 205 (5.1).

constexpr int kThreads = 256, kMaxThreads = 512;

template <typename T> constexpr int piece_of() { return 16 / int(sizeof(T)); }

// Where a lane works.  A token with at least a wave's worth of pieces has workgroups of
// its own, `groups` of them, so that its positions are read once for a wave; smaller
// ones follow each other.
struct Place {
  Divisor by;        // pieces of a token, or its workgroups
  uint32_t pieces;   // of a token
  uint32_t items;    // pieces of all tokens of a launch
  bool own;          // a token has workgroups of its own
};
__device__ __forceinline__ bool place_of(const Place& at, uint32_t* token, uint32_t* piece) {
  if (at.own) {
    *token = quotient(blockIdx.x, at.by);
    *piece = (blockIdx.x - *token * at.by.d) * blockDim.x + threadIdx.x;
    return *piece < at.pieces;
  }
  const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
  *token = quotient(i, at.by);
  *piece = i - *token * at.by.d;
  return i < at.items;
}

// N elements from column c on, of which those past `cols` are zero.  STREAM: past the
// caches, for what is not used again soon.
template <bool STREAM, typename T, int N> __device__ __forceinline__ Pack<T, N> load_piece(const T* p, int c, int cols) {
  Pack<T, N> v;
  if (c + N <= cols) {
    if (!STREAM) return load_pack<T, N>(p + c);
    const typename Words<16>::type w = __builtin_nontemporal_load(reinterpret_cast<const typename Words<16>::type*>(p + c));
    __builtin_memcpy(&v, &w, 16);
    return v;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v.v[i] = c + i < cols ? p[c + i] : T(0);
  return v;
}
template <bool STREAM, typename T, int N>
__device__ __forceinline__ void store_piece(T* p, int c, int cols, const Pack<T, N>& v) {
  if (c + N <= cols) {
    if (STREAM) store_stream<T, N>(p + c, v);
    else store_pack<T, N>(p + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (c + i < cols) p[c + i] = v.v[i];
  }
}

// T: an unsigned integer of the elements' size (the copy is by bits).
template <typename T, int STREAM>
__global__ __launch_bounds__(kMaxThreads) void gather_rows(const T* x, int64_t x_stride, int cols, Place at,
                                                           const int32_t* __restrict__ position, int choices, T* rows,
                                                           int64_t rows_stride, uint32_t n_rows) {
  constexpr int N = piece_of<T>();
  uint32_t token, piece;
  if (!place_of(at, &token, &piece)) return;
  const int c = int(piece) * N;
  const Pack<T, N> v = load_piece<false, T, N>(x + int64_t(token) * x_stride, c, cols);
  const int32_t* p = position + int64_t(token) * choices;
  for (int j = 0; j < choices; ++j) {
    const uint32_t row = uint32_t(p[j]);
    if (row < n_rows) store_piece<STREAM != 0, T, N>(rows + int64_t(row) * rows_stride, c, cols, v);
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

// kTogether choices' pieces are on their way together (eight took 122 us for 95 where the
// rows are 470 MB: more rows open at once than HBM likes).
constexpr int kTogether = 4;

template <int DT, int STREAM>
__global__ __launch_bounds__(kMaxThreads) void combine_rows(const typename Elem<DT>::type* rows, int64_t rows_stride,
                                                            uint32_t n_rows, const int32_t* __restrict__ position,
                                                            int choices, Scalars weights, Place at,
                                                            typename Elem<DT>::type* out, int64_t out_stride, int cols) {
  typedef typename Elem<DT>::type T;
  constexpr int N = piece_of<T>();
  uint32_t token, piece;
  if (!place_of(at, &token, &piece)) return;
  const int c = int(piece) * N;
  const int32_t* p = position + int64_t(token) * choices;
  float sum[N];
#pragma unroll
  for (int k = 0; k < N; ++k) sum[k] = 0.f;
  for (int j = 0; j < choices; j += kTogether) {
    Pack<T, N> v[kTogether];
    uint32_t row[kTogether];
    float w[kTogether];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      row[u] = j + u < choices ? uint32_t(p[j + u]) : ~0u;
      w[u] = j + u < choices ? scalar_at(weights, token, j + u) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
      if (row[u] < n_rows) v[u] = load_piece<STREAM == 2, T, N>(rows + int64_t(row[u]) * rows_stride, c, cols);
#pragma unroll
    for (int u = 0; u < kTogether; ++u)
      if (row[u] < n_rows) {
#pragma unroll
        for (int k = 0; k < N; ++k) sum[k] = fmaf(w[u], Elem<DT>::up(v[u].v[k]), sum[k]);
      }
  }
  Pack<T, N> v;
#pragma unroll
  for (int k = 0; k < N; ++k) v.v[k] = Elem<DT>::down(sum[k]);
  store_piece<STREAM != 0, T, N>(out + int64_t(token) * out_stride, c, cols, v);
}

// A workgroup a token, up to kBatch of its choices at a time: dout's row is read once for
// each batch, each choice's row of the forward pass once, and the choice's gradient row
// written once.  The products' sums go over a lane's pieces, then over a wave's lanes, then
// over the waves, always in this order.
constexpr int kBatch = 8;

template <int DT, int STREAM>
__global__ __launch_bounds__(kMaxThreads) void combine_grad(const typename Elem<DT>::type* dout, int64_t dout_stride,
                                                            const typename Elem<DT>::type* rows, int64_t rows_stride,
                                                            const int32_t* __restrict__ position, int choices,
                                                            Scalars weights, typename Elem<DT>::type* drows,
                                                            int64_t drows_stride, uint32_t n_rows, void* dweights,
                                                            int64_t dweights_stride, int dweights_dtype, int cols) {
  typedef typename Elem<DT>::type T;
  constexpr int N = piece_of<T>();
  __shared__ float wave_sums[kMaxThreads / 64][kBatch];
  const int64_t token = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
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
    for (int c = int(threadIdx.x) * N; c < cols; c += int(blockDim.x) * N) {
      const Pack<T, N> g = load_piece<STREAM == 2, T, N>(d, c, cols);
      Pack<T, N> v[kBatch];
      if (dweights) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (row[u] < n_rows) v[u] = load_piece<STREAM == 2, T, N>(rows + int64_t(row[u]) * rows_stride, c, cols);
      }
      float x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = Elem<DT>::up(g.v[k]);
      if (drows) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (row[u] < n_rows) {
            Pack<T, N> r;
#pragma unroll
            for (int k = 0; k < N; ++k) r.v[k] = Elem<DT>::down(w[u] * x[k]);
            store_piece<STREAM != 0, T, N>(drows + int64_t(row[u]) * drows_stride, c, cols, r);
          }
      }
      if (dweights) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (row[u] < n_rows) {
#pragma unroll
            for (int k = 0; k < N; ++k) sum[u] = fmaf(x[k], Elem<DT>::up(v[u].v[k]), sum[u]);
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
      for (int v = 0; v < waves; ++v) s += wave_sums[v][threadIdx.x];
      const int64_t at = token * dweights_stride + j0 + threadIdx.x;
      if (dweights_dtype == RESHARD_DTYPE_F32) static_cast<float*>(dweights)[at] = s;
      else if (dweights_dtype == RESHARD_DTYPE_BF16) static_cast<__bf16*>(dweights)[at] = __bf16(s);
      else static_cast<_Float16*>(dweights)[at] = _Float16(s);
    }
    __syncthreads();
  }
}

// Waves of a token's workgroups: as many as make its pieces in the fewest rounds.
int waves_for(int64_t pieces) {
  const int64_t waves = std::max<int64_t>(1, ceil_div(pieces, 64));
  return int(ceil_div(waves, ceil_div(waves, kMaxThreads / 64)));
}
// Waves of the workgroup that makes a token's gradient: 2 to 4, the number with the fewest
// idle in its last round, of equals the largest (3001 fp32 columns, 12 waves' worth of
// pieces: 17 us with 4, 18 with 2 and 22 with 6; 7168 bf16, 14: 205 with 2, 211 with 4).
int grad_waves(int64_t pieces) {
  const int64_t waves = std::max<int64_t>(1, ceil_div(pieces, 64));
  if (waves <= 4) return int(waves);
  int best = 4;
  for (int w = 3; w >= 2; --w)
    if (round_up(waves, w) < round_up(waves, best)) best = w;
  return best;
}

// Launches over the pieces of tokens, each within 31 bits.
template <typename F> hipError_t in_launches(int64_t tokens, int64_t pieces, F launch) {
  const bool own = pieces >= 64;
  const int threads = own ? 64 * waves_for(pieces) : kThreads;
  const int64_t groups = ceil_div(pieces, threads);  // of a token's own
  const int64_t most = own ? std::max<int64_t>(1, kMaxGroups / groups) : rows_per_launch(pieces, kThreads);
  for (int64_t t = 0; t < tokens; t += most) {
    const int64_t n = std::min(most, tokens - t);
    Place at{divisor(uint32_t(own ? groups : pieces)), uint32_t(pieces), uint32_t(own ? 0 : n * pieces), own};
    launch(t, at, dim3(uint32_t(own ? n * groups : ceil_div(n * pieces, kThreads))), threads);
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

// What goes past the caches: 0 nothing, 1 stores, 2 loads too, by the bytes of the
// rows.  Where the rows fill the last-level cache, loads that pass it leave it to what is
// used again: the calls of a training step over 470 MB of rows took 492 us for 634 with
// stores alone and 673 with neither.  Over 36 MB, of which it holds much, stores alone are
// best: 50 us, 57 with the loads, 70 with neither.
int streams(const reshard_matrix_t& m) {
  const int64_t bytes = m.rows * m.cols * (m.dtype == RESHARD_DTYPE_F32 ? 4 : 2);
  return bytes > (int64_t(128) << 20) ? 2 : bytes > (int64_t(16) << 20) ? 1 : 0;
}

template <typename T, int STREAM>
hipError_t gather_as(const reshard_matrix_t& x, const int32_t* position, int choices, const reshard_matrix_t& rows,
                     hipStream_t stream) {
  const int64_t pieces = ceil_div(x.cols, piece_of<T>());
  return in_launches(x.rows, pieces, [&](int64_t t, const Place& at, dim3 grid, int threads) {
    gather_rows<T, STREAM><<<grid, threads, 0, stream>>>(static_cast<const T*>(x.data) + t * x.row_stride, x.row_stride,
                                                 int(x.cols), at, position + t * choices, choices,
                                                 static_cast<T*>(rows.data), rows.row_stride, uint32_t(rows.rows));
  });
}

template <int DT, int STREAM>
hipError_t combine_as(const reshard_matrix_t& rows, const int32_t* position, int choices, const reshard_matrix_t* weights,
                      const reshard_matrix_t& out, hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const int64_t pieces = ceil_div(out.cols, piece_of<T>());
  return in_launches(out.rows, pieces, [&](int64_t t, const Place& at, dim3 grid, int threads) {
    combine_rows<DT, STREAM><<<grid, threads, 0, stream>>>(
        static_cast<const T*>(rows.data), rows.row_stride, uint32_t(rows.rows), position + t * choices, choices,
        scalars(weights, t), at, static_cast<T*>(out.data) + t * out.row_stride,
        out.row_stride, int(out.cols));
  });
}

template <int DT, int STREAM>
hipError_t grad_as(const reshard_matrix_t& dout, const reshard_matrix_t* rows, const int32_t* position, int choices,
                   const reshard_matrix_t* weights, const reshard_matrix_t* drows, const reshard_matrix_t* dweights,
                   hipStream_t stream) {
  typedef typename Elem<DT>::type T;
  const uint32_t n_rows = uint32_t(rows ? rows->rows : drows->rows);
  const int threads = 64 * grad_waves(ceil_div(dout.cols, piece_of<T>()));
  for (int64_t t = 0; t < dout.rows; t += kMaxGroups) {
    uint8_t* dw = nullptr;
    if (dweights)
      dw = static_cast<uint8_t*>(dweights->data) + t * dweights->row_stride * (dweights->dtype == RESHARD_DTYPE_F32 ? 4 : 2);
    combine_grad<DT, STREAM><<<dim3(uint32_t(std::min(kMaxGroups, dout.rows - t))), threads, 0, stream>>>(
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
  if (rounds <= kAloneRounds) {
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
    rank_choices<I, true><<<dim3(1), kSortThreads, 0, stream>>>(ids, uint32_t(chosen), first, experts, bits,
                                                                uint32_t(plan.rounds), nullptr, offsets, position);
    return hipGetLastError();
  }
  int* counts = static_cast<int*>(workspace);
  const dim3 grid(uint32_t(plan.blocks));
  rank_choices<I, false><<<grid, kSortThreads, 0, stream>>>(ids, uint32_t(chosen), first, experts, bits,
                                                            uint32_t(plan.rounds), counts, offsets, position);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  place_choices<I><<<grid, kSortThreads, 0, stream>>>(ids, uint32_t(chosen), first, experts, bits, uint32_t(plan.rounds),
                                                      counts, offsets, position);
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
  const bool past = streams(rows) != 0;
  if (x.dtype == RESHARD_DTYPE_F32)
    return past ? gather_as<uint32_t, 1>(x, position, choices, rows, stream)
                : gather_as<uint32_t, 0>(x, position, choices, rows, stream);
  return past ? gather_as<uint16_t, 1>(x, position, choices, rows, stream)
              : gather_as<uint16_t, 0>(x, position, choices, rows, stream);
}

template <int STREAM>
static hipError_t combine_dtypes(const reshard_matrix_t& rows, const int32_t* position, int choices,
                                 const reshard_matrix_t* weights, const reshard_matrix_t& out, hipStream_t stream) {
  switch (out.dtype) {
    case RESHARD_DTYPE_F32: return combine_as<RESHARD_DTYPE_F32, STREAM>(rows, position, choices, weights, out, stream);
    case RESHARD_DTYPE_BF16: return combine_as<RESHARD_DTYPE_BF16, STREAM>(rows, position, choices, weights, out, stream);
    default: return combine_as<RESHARD_DTYPE_F16, STREAM>(rows, position, choices, weights, out, stream);
  }
}

hipError_t launch_combine(const reshard_matrix_t& rows, const int32_t* position, int choices,
                          const reshard_matrix_t* weights, const reshard_matrix_t& out, hipStream_t stream) {
  switch (streams(rows)) {
    case 0: return combine_dtypes<0>(rows, position, choices, weights, out, stream);
    case 1: return combine_dtypes<1>(rows, position, choices, weights, out, stream);
    default: return combine_dtypes<2>(rows, position, choices, weights, out, stream);
  }
}

template <int STREAM>
static hipError_t grad_dtypes(const reshard_matrix_t& dout, const reshard_matrix_t* rows, const int32_t* position,
                              int choices, const reshard_matrix_t* weights, const reshard_matrix_t* drows,
                              const reshard_matrix_t* dweights, hipStream_t stream) {
  switch (dout.dtype) {
    case RESHARD_DTYPE_F32:
      return grad_as<RESHARD_DTYPE_F32, STREAM>(dout, rows, position, choices, weights, drows, dweights, stream);
    case RESHARD_DTYPE_BF16:
      return grad_as<RESHARD_DTYPE_BF16, STREAM>(dout, rows, position, choices, weights, drows, dweights, stream);
    default:
      return grad_as<RESHARD_DTYPE_F16, STREAM>(dout, rows, position, choices, weights, drows, dweights, stream);
  }
}

hipError_t launch_combine_grad(const reshard_matrix_t& dout, const reshard_matrix_t* rows, const int32_t* position,
                               int choices, const reshard_matrix_t* weights, const reshard_matrix_t* drows,
                               const reshard_matrix_t* dweights, hipStream_t stream) {
  if (!dweights) rows = nullptr;
  switch (streams(rows ? *rows : *drows)) {
    case 0: return grad_dtypes<0>(dout, rows, position, choices, weights, drows, dweights, stream);
    case 1: return grad_dtypes<1>(dout, rows, position, choices, weights, drows, dweights, stream);
    default: return grad_dtypes<2>(dout, rows, position, choices, weights, drows, dweights, stream);
  }
}

}  // namespace rs
