// lh_moe.hip - tokens sorted by expert, their rows sent to the experts and
// back with the routing weights, and the gradients of both ways.
//
// Every token t chooses top_k experts; assignment a = t * top_k + k carries
// token t's row to expert expert_ids[a].  A stable counting sort by expert
// gives each assignment a row p, so that expert g owns rows offsets[g] ..
// offsets[g+1]-1 (the layout lh_accumulate_hessian_ragged and
// lh_linear_nvfp4_ragged read).  Assignments without a valid expert sort to
// the rows past offsets[n_groups]; they are marked by negative entries
// (-1 - row in position, -1 - a in order) and contribute nothing.
//   dispatch      xs[p] = x[t]             gradient: combine with weights 1
//   combine       y[t] = sum_k w[t,k] ys[p]
//   its gradient  dys[p] = w[t,k] dy[t],  dw[t,k] = <dy[t], ys[p]>
// All sums run in a fixed order (k, then columns by lane, wave and workgroup):
// no atomics on data, so results do not change from run to run.
#include "lh_internal.h"
#include "lh_rows.h"

namespace lh {
namespace {

// ---------------------------------------------------------------------------
// Sort.  A workgroup of 8 waves takes `chunk` consecutive assignments, each
// wave a consecutive eighth.  A wave counts its assignments per expert in its
// own row of LDS counters, the workgroup turns the counters into first rows
// (rows of smaller experts, of earlier chunks, of earlier waves), and the
// wave walks its assignments again, 64 at a time: the lanes with the same
// expert find each other by one ballot per bit of the expert number, so the
// rank within the wave is a population count and the order is stable.
// Bound by latency (a few dependent passes over 16 workgroups): 4096 x 8
// assignments to 64 experts 8.7 us with both launches, 16 x 8 4.0 in one.
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;

template <typename TI>
__device__ __forceinline__ int expert_of(const TI* __restrict__ ids, int64_t a, int n_groups) {
  const TI v = ids[a];
  return (v >= 0 && v < (TI)n_groups) ? (int)v : n_groups;  // n_groups: no expert
}

// The first kHold * 64 assignments of a wave's share, looked up once: all of
// them in a chunk of the usual size.
constexpr int kHold = 4;
template <typename TI>
__device__ __forceinline__ void hold_share(const TI* __restrict__ ids, int64_t a0, int64_t a1, int n_groups,
                                           int (&held)[kHold]) {
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int64_t a = a0 + 64 * i + (threadIdx.x & 63);
    held[i] = a < a1 ? expert_of(ids, a, n_groups) : -1;
  }
}

// counts[wave][bin] += this wave's share of the chunk; bins 0..n_groups.
template <typename TI>
__device__ __forceinline__ void count_share(const TI* __restrict__ ids, int64_t a0, int64_t a1, int n_groups,
                                            const int (&held)[kHold], unsigned int* mine) {
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (held[i] >= 0) atomicAdd(&mine[held[i]], 1u);
  for (int64_t a = a0 + 64 * kHold + (threadIdx.x & 63); a < a1; a += 64)
    atomicAdd(&mine[expert_of(ids, a, n_groups)], 1u);
}

// The wave's share [a0, a1) of chunk `c`.
__device__ __forceinline__ void wave_share(int64_t n, int64_t chunk, int64_t c, int wave, int64_t& a0, int64_t& a1) {
  const int64_t share = chunk / kSortWaves;
  a0 = min(c * chunk + wave * share, n);
  a1 = min(a0 + share, n);
}

// hist[chunk][bin]: the assignments of each chunk per expert.
template <typename TI>
__global__ __launch_bounds__(kSortThreads) void moe_count_kernel(const TI* __restrict__ ids, int64_t n, int64_t chunk,
                                                                 int n_groups, int* __restrict__ hist) {
  extern __shared__ unsigned int counts[];  // [kSortWaves][n_groups + 1]
  const int bins = n_groups + 1;
  int64_t a0, a1;
  const int wave = threadIdx.x >> 6;
  wave_share(n, chunk, blockIdx.x, wave, a0, a1);
  int held[kHold];
  hold_share(ids, a0, a1, n_groups, held);
  for (int i = threadIdx.x; i < kSortWaves * bins; i += kSortThreads) counts[i] = 0u;
  __syncthreads();
  count_share(ids, a0, a1, n_groups, held, counts + wave * bins);
  __syncthreads();
  for (int e = threadIdx.x; e < bins; e += kSortThreads) {
    unsigned int s = 0;
    for (int w = 0; w < kSortWaves; ++w) s += counts[w * bins + e];
    hist[(int64_t)blockIdx.x * bins + e] = (int)s;
  }
}

template <typename TI>
__global__ __launch_bounds__(kSortThreads) void moe_sort_kernel(const TI* __restrict__ ids, int64_t n, int64_t chunk,
                                                                int64_t n_chunks, int n_groups,
                                                                const int* __restrict__ hist,
                                                                int64_t* __restrict__ offsets,
                                                                int* __restrict__ order, int* __restrict__ position) {
  extern __shared__ unsigned int counts[];  // [kSortWaves][bins], then total[bins]
  const int bins = n_groups + 1;
  unsigned int* const total = counts + kSortWaves * bins;
  __shared__ unsigned int wave_sum[kSortWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  int64_t a0, a1;
  wave_share(n, chunk, blockIdx.x, wave, a0, a1);
  int held[kHold];
  hold_share(ids, a0, a1, n_groups, held);
  for (int i = tid; i < kSortWaves * bins; i += kSortThreads) counts[i] = 0u;
  __syncthreads();
  count_share(ids, a0, a1, n_groups, held, counts + wave * bins);
  __syncthreads();
  // per expert: its rows in all chunks (total) and in earlier ones, and its
  // waves' first rows within them
  for (int e = tid; e < bins; e += kSortThreads) {
    unsigned int before = 0, all = 0;
    if (n_chunks > 1) {
#pragma unroll 16
      for (int64_t c = 0; c < n_chunks; ++c) {
        const unsigned int h = (unsigned int)hist[c * bins + e];
        before += c < (int64_t)blockIdx.x ? h : 0u;
        all += h;
      }
    }
    unsigned int run = before;
    for (int w = 0; w < kSortWaves; ++w) {
      const unsigned int v = counts[w * bins + e];
      counts[w * bins + e] = run;
      run += v;
    }
    total[e] = n_chunks > 1 ? all : run;
  }
  __syncthreads();
  // exclusive scan of total over the experts, kSortThreads at a time
  unsigned int carry = 0;
  for (int e0 = 0; e0 < bins; e0 += kSortThreads) {
    const int e = e0 + tid;
    const unsigned int v = e < bins ? total[e] : 0u;
    unsigned int incl = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const unsigned int u = (unsigned int)__shfl_up((int)incl, off);
      if (lane >= off) incl += u;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    unsigned int base = carry;
    for (int w = 0; w < wave; ++w) base += wave_sum[w];
    const unsigned int first = base + incl - v;
    if (e < bins) {
      for (int w = 0; w < kSortWaves; ++w) counts[w * bins + e] += first;
      if (blockIdx.x == 0) offsets[e] = (int64_t)first;  // offsets[n_groups]: the rows that have an expert
    }
    for (int w = 0; w < kSortWaves; ++w) carry += wave_sum[w];
    __syncthreads();
  }
  int bits = 0;
  while ((1 << bits) < bins) ++bits;
  unsigned int* const mine = counts + wave * bins;
  // 64 assignments from `a` on, e the expert of this lane's (-1: past the share)
  auto place = [&](int64_t a, int e) {
    const bool have = e >= 0;
    unsigned long long same = __ballot(have);
    for (int b = 0; b < bits; ++b) {
      const unsigned long long set = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? set : ~set;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1ull));
    unsigned int row = 0;
    if (have) row = mine[e] + (unsigned int)rank;
    // every lane of the expert reads the counter before its first lane moves
    // it on; LDS serves one wave's accesses in order, the fences keep the
    // compiler from moving or reusing them
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (have && rank == 0) mine[e] += (unsigned int)__popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (have) {
      const int64_t at = a + lane;
      const bool live = e < n_groups;
      position[at] = live ? (int)row : -1 - (int)row;
      if (order) order[row] = live ? (int)at : -1 - (int)at;
    }
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (a0 + 64 * i < a1) place(a0 + 64 * i, held[i]);  // a wave-uniform branch
  for (int64_t a = a0 + 64 * kHold; a < a1; a += 64)  // the same trip count for every lane of the wave
    place(a, a + lane < a1 ? expert_of(ids, a + lane, n_groups) : -1);
}

// ---------------------------------------------------------------------------
// Rows.  A thread moves 16 bytes of a row at a time; rows of any length and
// alignment (the loads and stores are written for unaligned addresses, and
// the last elements of a row go one by one).  Memory-bound: 4096 tokens x 8
// experts of 2048 bf16, dispatch 151 MB in 24 us (6.4 TB/s), combine 151 MB in
// 29 us (5.2; 38 us where the rows were written just before), its gradient
// 285 MB in 46 to 50 us (5.7).
// ---------------------------------------------------------------------------
template <typename T>
struct Vec {
  static constexpr int kN = 16 / sizeof(T);
};

template <typename T>
__device__ __forceinline__ uint4 load_raw16(const T* p, int n) {
  if (n >= Vec<T>::kN) return load_u128(p);
  T raw[Vec<T>::kN];
#pragma unroll
  for (int i = 0; i < Vec<T>::kN; ++i) raw[i] = i < n ? p[i] : T(0);
  return __builtin_bit_cast(uint4, raw);
}
template <typename T>
__device__ __forceinline__ void values_of(const uint4 u, float (&v)[Vec<T>::kN]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
      v[i] = __uint_as_float(w[i]);
    }
  }
}
// The first n values of 16 bytes.
template <typename T>
__device__ __forceinline__ void store_raw16(T* p, int n, const uint4 u) {
  if (n >= Vec<T>::kN) {
    __builtin_memcpy(p, &u, 16);
  } else {
    T raw[Vec<T>::kN];
    __builtin_memcpy(raw, &u, 16);
#pragma unroll
    for (int i = 0; i < Vec<T>::kN; ++i)
      if (i < n) p[i] = raw[i];
  }
}

template <typename T>
__device__ __forceinline__ uint4 raw_of(const float (&v)[Vec<T>::kN]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    else w[i] = __float_as_uint(v[i]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The row an entry of `position` names, or -1 - row for an assignment without
// an expert; INT64_MIN for an entry outside the buffer (ignored).
__device__ __forceinline__ int64_t row_of(int entry, int64_t n_rows) {
  const int64_t r = entry >= 0 ? (int64_t)entry : -1 - (int64_t)entry;
  if (r >= n_rows) return INT64_MIN;
  return entry;
}

// The wave's unit of work, as scalars: what depends on it (positions,
// weights, row addresses) then comes through the scalar cache.
__device__ __forceinline__ int64_t wave_unit() {
  const uint32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  return block_id() * (kThreads / 64) + w;
}

// Assignments of a token that are looked up and moved together: their loads
// are all in flight before the first is used.
constexpr int kAtOnce = 8;

// One wave per (token, 64-lane span of columns): the token's span is read
// once and written top_k times.
template <typename T>
__global__ __launch_bounds__(kThreads) void moe_dispatch_kernel(const T* __restrict__ x, int64_t ld_x, int64_t n_tok,
                                                                int64_t cols, int top_k, int64_t spans,
                                                                const int* __restrict__ position, T* __restrict__ xs,
                                                                int64_t ld_xs, int64_t n_rows) {
  constexpr int kN = Vec<T>::kN;
  const int64_t unit = wave_unit();
  const int64_t t = unit / spans;
  if (t >= n_tok) return;
  const int64_t c = (unit - t * spans) * (64 * kN) + (threadIdx.x & 63) * kN;
  if (c >= cols) return;
  const int n = (int)min((int64_t)kN, cols - c);
  const uint4 v = load_raw16<T>(x + t * ld_x + c, n), zero = make_uint4(0u, 0u, 0u, 0u);
  for (int k0 = 0; k0 < top_k; k0 += kAtOnce) {
    int at[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) at[k] = position[t * top_k + min(k0 + k, top_k - 1)];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int64_t r = row_of(at[k], n_rows);
      if (k0 + k >= top_k || r == INT64_MIN) continue;
      if (r >= 0) store_raw16<T>(xs + r * ld_xs + c, n, v);
      else store_raw16<T>(xs + (-1 - r) * ld_xs + c, n, zero);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void moe_combine_kernel(const T* __restrict__ ys, int64_t ld_ys, int64_t n_rows,
                                                               int64_t n_tok, int64_t cols, int top_k, int64_t spans,
                                                               const int* __restrict__ position,
                                                               const float* __restrict__ weights, T* __restrict__ y,
                                                               int64_t ld_y) {
  constexpr int kN = Vec<T>::kN;
  const int64_t unit = wave_unit();
  const int64_t t = unit / spans;
  if (t >= n_tok) return;
  const int64_t c = (unit - t * spans) * (64 * kN) + (threadIdx.x & 63) * kN;
  if (c >= cols) return;
  const int n = (int)min((int64_t)kN, cols - c);
  float sum[kN] = {};
  for (int k0 = 0; k0 < top_k; k0 += kAtOnce) {
    uint4 raw[kAtOnce];
    float w[kAtOnce];
    bool live[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int64_t a = t * top_k + min(k0 + k, top_k - 1);
      const int64_t r = row_of(position[a], n_rows);
      live[k] = k0 + k < top_k && r >= 0;
      w[k] = weights ? weights[a] : 1.0f;
      if (live[k]) raw[k] = load_raw16<T>(ys + r * ld_ys + c, n);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (live[k]) {
        float v[kN];
        values_of<T>(raw[k], v);
#pragma unroll
        for (int i = 0; i < kN; ++i) sum[i] = __builtin_fmaf(w[k], v[i], sum[i]);
      }
  }
  store_raw16<T>(y + t * ld_y + c, n, raw_of<T>(sum));
}

// One workgroup per token, kAtOnce assignments at a time: dy's columns are
// read once for all of them, each thread's dots are reduced over the wave
// (the lanes exchange halves of the values), then over the waves in order.
template <typename T>
__global__ __launch_bounds__(kThreads) void moe_combine_grad_kernel(
    const T* __restrict__ dy, int64_t ld_dy, int64_t n_tok, const T* __restrict__ ys, int64_t ld_ys, int64_t n_rows,
    int64_t cols, int top_k, const int* __restrict__ position, const float* __restrict__ weights, T* __restrict__ dys,
    int64_t ld_dys, float* __restrict__ dw) {
  constexpr int kN = Vec<T>::kN;
  __shared__ float part[kThreads / 64][kAtOnce];
  const int64_t t = block_id();
  if (t >= n_tok) return;  // the whole workgroup
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (int k0 = 0; k0 < top_k; k0 += kAtOnce) {
    int64_t row[kAtOnce];  // the same for the whole workgroup
    float w[kAtOnce], dot[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int64_t a = t * top_k + min(k0 + k, top_k - 1);
      row[k] = k0 + k < top_k ? row_of(position[a], n_rows) : INT64_MIN;
      w[k] = weights ? weights[a] : 1.0f;
      dot[k] = 0.0f;
    }
    for (int64_t c = (int64_t)tid * kN; c < cols; c += (int64_t)kThreads * kN) {
      const int n = (int)min((int64_t)kN, cols - c);
      uint4 raw[kAtOnce];
      const uint4 rawd = load_raw16<T>(dy + t * ld_dy + c, n);
      if (dw) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
          if (row[k] >= 0) raw[k] = load_raw16<T>(ys + row[k] * ld_ys + c, n);
      }
      float d[kN];
      values_of<T>(rawd, d);
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (row[k] == INT64_MIN) continue;
        if (row[k] < 0) {
          if (dys) store_raw16<T>(dys + (-1 - row[k]) * ld_dys + c, n, make_uint4(0u, 0u, 0u, 0u));
          continue;
        }
        if (dw) {
          float v[kN];
          values_of<T>(raw[k], v);
#pragma unroll
          for (int i = 0; i < kN; ++i) dot[k] = __builtin_fmaf(d[i], v[i], dot[k]);
        }
        if (dys) {
          float g[kN];
#pragma unroll
          for (int i = 0; i < kN; ++i) g[i] = d[i] * w[k];
          store_raw16<T>(dys + row[k] * ld_dys + c, n, raw_of<T>(g));
        }
      }
    }
    if (dw) {
      const float s = wave_sums(dot);  // lane l: assignment l / (64 / kAtOnce)
      if (lane % (64 / kAtOnce) == 0) part[wave][lane / (64 / kAtOnce)] = s;
      __syncthreads();
      if (tid < kAtOnce && k0 + tid < top_k) {
        float sum = part[0][tid];
        for (int i = 1; i < kThreads / 64; ++i) sum += part[i][tid];
        dw[t * top_k + k0 + tid] = sum;
      }
      __syncthreads();
    }
  }
}

// Chunks of the sort: 2048 assignments each, or more where that made over 512
// (every chunk reads the counts of all chunks).
int64_t sort_chunk(int64_t n) {
  const int64_t most = 512;
  int64_t c = (n + most - 1) / most;
  c = (c + 2047) / 2048 * 2048;
  return c < 2048 ? 2048 : c;
}

template <typename TI>
hipError_t launch_sort_typed(const MoeSortArgs& a, hipStream_t stream) {
  const int64_t chunk = sort_chunk(a.n);
  const int64_t chunks = a.n == 0 ? 1 : (a.n + chunk - 1) / chunk;
  const int bins = (int)a.n_groups + 1;
  const TI* ids = static_cast<const TI*>(a.ids);
  int* hist = static_cast<int*>(a.ws);
  if (chunks > 1) {
    moe_count_kernel<TI><<<dim3((unsigned)chunks), dim3(kSortThreads), kSortWaves * bins * 4, stream>>>(
        ids, a.n, chunk, (int)a.n_groups, hist);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  moe_sort_kernel<TI><<<dim3((unsigned)chunks), dim3(kSortThreads), (kSortWaves + 1) * bins * 4, stream>>>(
      ids, a.n, chunk, chunks, (int)a.n_groups, hist, a.offsets, a.order, a.position);
  return hipGetLastError();
}

template <typename T>
dim3 row_grid(int64_t n_tok, int64_t cols, int64_t& spans) {
  const int64_t per = 64 * (16 / (int64_t)sizeof(T));
  spans = (cols + per - 1) / per;
  return grid_of((n_tok * spans + kThreads / 64 - 1) / (kThreads / 64));
}

template <typename T>
hipError_t launch_dispatch_typed(const MoeRowsArgs& a, hipStream_t stream) {
  int64_t spans;
  const dim3 grid = row_grid<T>(a.n_tok, a.cols, spans);
  moe_dispatch_kernel<T><<<grid, dim3(kThreads), 0, stream>>>(
      static_cast<const T*>(a.tok), a.ld_tok, a.n_tok, a.cols, (int)a.top_k, spans, a.position,
      static_cast<T*>(a.rows_out), a.ld_out, a.n_rows);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_combine_typed(const MoeRowsArgs& a, hipStream_t stream) {
  int64_t spans;
  const dim3 grid = row_grid<T>(a.n_tok, a.cols, spans);
  moe_combine_kernel<T><<<grid, dim3(kThreads), 0, stream>>>(
      static_cast<const T*>(a.rows), a.ld_rows, a.n_rows, a.n_tok, a.cols, (int)a.top_k, spans, a.position, a.weights,
      static_cast<T*>(a.rows_out), a.ld_out);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_combine_grad_typed(const MoeRowsArgs& a, hipStream_t stream) {
  moe_combine_grad_kernel<T><<<grid_of(a.n_tok), dim3(kThreads), 0, stream>>>(
      static_cast<const T*>(a.tok), a.ld_tok, a.n_tok, static_cast<const T*>(a.rows), a.ld_rows, a.n_rows, a.cols,
      (int)a.top_k, a.position, a.weights, static_cast<T*>(a.rows_out), a.ld_out, a.dweights);
  return hipGetLastError();
}

}  // namespace

size_t moe_sort_ws_bytes(int64_t n, int64_t n_groups) {
  const int64_t chunk = sort_chunk(n);
  const int64_t chunks = (n + chunk - 1) / chunk;
  return chunks > 1 ? (size_t)chunks * (size_t)(n_groups + 1) * sizeof(int) : 0;
}

hipError_t launch_moe_sort(const MoeSortArgs& a, hipStream_t stream) {
  return a.ids_i64 ? launch_sort_typed<int64_t>(a, stream) : launch_sort_typed<int32_t>(a, stream);
}
hipError_t launch_moe_dispatch(const MoeRowsArgs& a, hipStream_t stream) {
  return a.dtype == 1 ? launch_dispatch_typed<uint16_t>(a, stream) : launch_dispatch_typed<float>(a, stream);
}
hipError_t launch_moe_combine(const MoeRowsArgs& a, hipStream_t stream) {
  return a.dtype == 1 ? launch_combine_typed<uint16_t>(a, stream) : launch_combine_typed<float>(a, stream);
}
hipError_t launch_moe_combine_grad(const MoeRowsArgs& a, hipStream_t stream) {
  return a.dtype == 1 ? launch_combine_grad_typed<uint16_t>(a, stream) : launch_combine_grad_typed<float>(a, stream);
}

}  // namespace lh
