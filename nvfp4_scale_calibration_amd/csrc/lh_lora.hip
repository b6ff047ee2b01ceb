// lh_lora.hip - low-rank adapters beside a frozen projection, for many
// requests at once, and their gradients.
//
//   s[t][r] = sum_c x[t][c] in[g][r][c]            (the row into the rank)
//   y[t][o] = base[t][o] + scale[g] sum_r s[t][r] out[g][r][o]
// with g the adapter of t's segment.  Both factors are stored with the rank
// first, so the gradient to the input (dy for x, b for in, a for out) is the
// same two kernels.  The gradients to the factors are sums over an adapter's
// rows, out[g][r][c] = scale[g] sum_t p[t][r] x[t][c].
//
// All of it is bound by memory at the ranks in use (a rank of 16 is 32 operations
// for every element of x or y), or by latency where there are few rows.
#include <type_traits>

#include "lh_internal.h"
#include "lh_rows.h"

namespace lh {
namespace {

// Segment `i`'s adapter, -1 for none.
__device__ __forceinline__ int64_t adapter_of(const SegmentArgs& g, int64_t i) {
  int64_t id = i;
  if (g.ids) id = g.ids_i64 ? static_cast<const int64_t*>(g.ids)[i] : (int64_t) static_cast<const int32_t*>(g.ids)[i];
  return id >= 0 && id < g.n_adapters ? id : -1;
}

// Row t's adapter, -1 for none, -2 where t is in no segment (the first one, where
// segments overlap).  All lanes of the wave ask for the same row.
__device__ __forceinline__ int64_t adapter_of_row(const SegmentArgs& g, int64_t t) {
  if (!g.offsets) return adapter_of(g, g.n == 1 ? 0 : t);
  const int lane = threadIdx.x & 63;
  for (int64_t i0 = 0; i0 < g.n; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool mine = i < g.n && g.offsets[i] <= t && t < g.offsets[i + 1];
    const unsigned long long hit = __ballot(mine);
    if (hit) return uniform(adapter_of(g, i0 + __ffsll(hit) - 1));
  }
  return -2;
}

// The same for the rows t0 .. t0 + kRows - 1 of a tile, into LDS, by the whole
// workgroup; rows past n_rows are in no segment.  Every thread looks at its
// share of the segments; the smallest segment wins a row that several claim.
template <int kRows>
__device__ __forceinline__ void tile_adapters(const SegmentArgs& g, int64_t t0, int64_t n_rows, int (&of)[kRows]) {
  __shared__ unsigned long long claim[kRows];
  const int tid = threadIdx.x;
  const int64_t t1 = min(t0 + kRows, n_rows);
  if (!g.offsets) {  // all rows are one segment (a row each takes the row kernels)
    if (tid < kRows) of[tid] = t0 + tid < t1 ? (int)adapter_of(g, 0) : -2;
    __syncthreads();
    return;
  }
  if (tid < kRows) claim[tid] = ~0ull;
  __syncthreads();
  for (int64_t i = tid; i < g.n; i += blockDim.x) {
    const int64_t lo = max(g.offsets[i], t0), hi = min(g.offsets[i + 1], t1);
    const unsigned long long mine = ((unsigned long long)i << 32) | (uint32_t)(int)adapter_of(g, i);
    for (int64_t t = lo; t < hi; ++t) atomicMin(&claim[t - t0], mine);
  }
  __syncthreads();
  if (tid < kRows) of[tid] = claim[tid] == ~0ull ? -2 : (int)(uint32_t)claim[tid];
  __syncthreads();
}

// Eight values of a row from p on as fp32, the first n of them inside it
// (the others are zero).
__device__ __forceinline__ void load8(const uint16_t* p, int64_t n, float (&v)[8]) {
  uint32_t w[4] = {};
  if (n >= 8) {
    __builtin_memcpy(w, p, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, int64_t n, float (&v)[8]) {
  if (n >= 8) {
    __builtin_memcpy(v, p, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
}

// ---------------------------------------------------------------------------
// The row kernels, for few rows and for segments of a row or so: no matrix cores,
// every row with its own adapter.  Latency is what counts, so all loads that do not
// wait for an adapter's number are issued before it, and a workgroup's four waves
// share the sum that its outputs need.  1 row, 17408 -> 5120, rank 16: 4.1 us each,
// of which a launch is 3.5; 48 rows, 4096 -> 12288: 4.6 and 4.8.
// ---------------------------------------------------------------------------
constexpr int kRowRanks = 4;

// Into the rank: a workgroup takes a row, four ranks and a span of the contraction
// (a multiple of 512), its waves 512 elements in turn.
template <typename TX, typename TW>
__global__ __launch_bounds__(kThreads) void lora_row_in_kernel(LoraArgs a, int64_t groups, int splits, int64_t span,
                                                               float* __restrict__ part) {
  __shared__ float red[kThreads / 64][kRowRanks];
  const int64_t unit = block_id(), t = unit / (groups * splits);
  if (t >= a.rows) return;
  const int64_t rest = unit - t * (groups * splits), split = rest / groups, r0 = (rest - split * groups) * kRowRanks;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int64_t c0 = split * span + 512 * wave, end = min(split * span + span, a.c_x);
  const TX* const x = static_cast<const TX*>(a.x) + t * a.ld_x + lane * 8;
  float first[8] = {};
  if (c0 + 512 <= end) load8(x + c0, 8, first);
  const int64_t g = adapter_of_row(a.seg, t);
  if (g == -2) return;  // the whole workgroup
  float acc[kRowRanks] = {};
  if (g >= 0) {
    const TW* w[kRowRanks];
#pragma unroll
    for (int r = 0; r < kRowRanks; ++r)
      w[r] = static_cast<const TW*>(a.in) + (g * a.rank + min(r0 + r, a.rank - 1)) * a.c_x + lane * 8;
    int64_t c = c0;
    if (c + 512 <= end) {
      float wv[kRowRanks][8];
#pragma unroll
      for (int r = 0; r < kRowRanks; ++r) load8(w[r] + c, 8, wv[r]);
#pragma unroll
      for (int r = 0; r < kRowRanks; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[r] = __builtin_fmaf(first[i], wv[r][i], acc[r]);
      c += 512 * (kThreads / 64);
    }
#pragma unroll 2
    for (; c + 512 <= end; c += 512 * (kThreads / 64)) {
      float xv[8], wv[kRowRanks][8];
      load8(x + c, 8, xv);
#pragma unroll
      for (int r = 0; r < kRowRanks; ++r) load8(w[r] + c, 8, wv[r]);
#pragma unroll
      for (int r = 0; r < kRowRanks; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[r] = __builtin_fmaf(xv[i], wv[r][i], acc[r]);
    }
    if (c + lane * 8 < end) {  // the row's last elements
      const int64_t n = end - c - lane * 8;
      float xv[8], wv[8];
      load8(x + c, n, xv);
#pragma unroll
      for (int r = 0; r < kRowRanks; ++r) {
        load8(w[r] + c, n, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[r] = __builtin_fmaf(xv[i], wv[i], acc[r]);
      }
    }
  }
  const float v = wave_sums(acc);
  if (lane % (64 / kRowRanks) == 0) red[wave][lane / (64 / kRowRanks)] = v;
  __syncthreads();
  if (tid < kRowRanks && r0 + tid < a.rank) {
    float sum = red[0][tid];
#pragma unroll
    for (int u = 1; u < kThreads / 64; ++u) sum += red[u][tid];
    part[(split * a.rows + t) * a.rank + r0 + tid] = sum;
  }
}

// Out of the rank: a workgroup takes a row and 512 outputs, its waves every fourth
// rank, a lane eight outputs.
template <typename TW, typename TY>
__global__ __launch_bounds__(kThreads) void lora_row_out_kernel(LoraArgs a, int64_t spans, const float* __restrict__ part,
                                                                int splits) {
  constexpr int kWaves = kThreads / 64, kAhead = 4;
  __shared__ float s[kLoraMaxRank];
  __shared__ __attribute__((aligned(16))) float red[kWaves][512];
  const int64_t unit = block_id(), t = unit / spans, c_tile = (unit - t * spans) * 512;
  if (t >= a.rows) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, rank = (int)a.rank;
  const int64_t c = c_tile + lane * 8, n = a.c_y - c, o = c_tile + 2 * tid, left = a.c_y - o;  // o: the two outputs it stores
  TY* const y = static_cast<TY*>(a.y) + t * a.ld_y + o;
  float b[2] = {};
  if (a.base) {
    const TY* p = static_cast<const TY*>(a.base) + t * a.ld_base + o;
    if (left > 0) b[0] = load_as_f32<TY>(p, 0);
    if (left > 1) b[1] = load_as_f32<TY>(p, 1);
  }
  const int64_t g = adapter_of_row(a.seg, t);
  if (g == -2) return;  // the whole workgroup
  if (g >= 0 && rank > 0) {
    const TW* const w = static_cast<const TW*>(a.out) + g * a.rank * a.c_y + c;
    float first[kAhead][8];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load8(w + min(wave + kWaves * u, rank - 1) * a.c_y, n, first[u]);
    if (tid < rank) {
      const int64_t at = t * a.rank + tid;
      const float v = sum_slices(part + at, a.rows * a.rank, splits);
      s[tid] = v;
      if (a.s && a.s != part && c_tile == 0) a.s[at] = v;
    }
    __syncthreads();
    float acc[8] = {};
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (wave + kWaves * u < rank) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(s[wave + kWaves * u], first[u][i], acc[i]);
      }
#pragma unroll 4
    for (int r = wave + kWaves * kAhead; r < rank; r += kWaves) {
      float wv[8];
      load8(w + r * a.c_y, n, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(s[r], wv[i], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) red[wave][8 * lane + i] = acc[i];
    __syncthreads();
    const float scale = a.scale ? a.scale[g] : 1.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v = red[0][2 * tid + h];
#pragma unroll
      for (int u = 1; u < kWaves; ++u) v += red[u][2 * tid + h];
      b[h] = __builtin_fmaf(scale, v, b[h]);
    }
  } else if (a.s && a.s != part && c_tile == 0 && tid < rank) {
    a.s[t * a.rank + tid] = 0.0f;
  }
  if (left > 1) {
    if constexpr (sizeof(TY) == 2) {
      const uint32_t v = pack_bf16(b[0], b[1]);
      __builtin_memcpy(y, &v, 4);
    } else {
      __builtin_memcpy(y, b, 8);
    }
  } else if (left > 0) {
    if constexpr (sizeof(TY) == 2) y[0] = f32_to_bf16_bits(b[0]);
    else y[0] = b[0];
  }
}

// ---------------------------------------------------------------------------
// The tile kernels: rows in tiles on the matrix cores, the rank in groups of 16.
// bf16 inputs meet bf16 factors on v_mfma_f32_16x16x32_bf16 (exact products,
// fp32 sums); where either is fp32 both are, on v_mfma_f32_16x16x4_f32.  The
// adapters that a tile's rows take are gone through one after the other, each
// over all of the tile; a row keeps its own adapter's result (rows and ranks of
// a matrix product do not mix, so what belongs to others never has to be masked).
// ---------------------------------------------------------------------------
typedef short s16x4_t __attribute__((ext_vector_type(4)));

template <typename T>
__device__ __forceinline__ const T* at_byte(const T* p, uint32_t offset) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) + offset);
}
template <typename T>
__device__ __forceinline__ T* at_byte(T* p, uint32_t offset) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(p) + offset);
}

// One lane's eight consecutive contraction elements of an operand.
struct Frag {
  float v[8];
};
template <typename T>
__device__ __forceinline__ void load_frag(const T* p, Frag& f) {
  load8(p, 8, f.v);
}
template <typename T>
__device__ __forceinline__ void load_frag(const T* p, int64_t n, Frag& f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f.v[i] = i < n ? load_as_f32<T>(p, i) : 0.0f;
}
__device__ __forceinline__ f32x4_t multiply(const Frag& a, const Frag& b, f32x4_t c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

// Into the rank where the input or the factor is fp32: a workgroup takes 32 rows
// and a share of the contraction, its four waves a quarter of that each.  Operands
// come straight from global memory, a lane eight consecutive elements of its row,
// the next steps' while the matrix cores work on these; the waves' sums are joined
// through LDS, those of the shares by the kernel that reads them.
constexpr int kInSub = 2, kInRows = 16 * kInSub, kInWaves = 4;

template <typename TX, typename TW, int kR16>
__global__ __launch_bounds__(64 * kInWaves) void lora_tile_in_kernel(LoraArgs a, int splits, int64_t k_wave,
                                                                     float* __restrict__ part) {
  constexpr int kSub = kInSub, kWaves = kInWaves;
  constexpr int kSteps = kR16 <= 2 ? 2 : 1;  // contraction steps of 32 that are loaded together (twice as many are in flight)
  __shared__ int of[kInRows];
  __shared__ __attribute__((aligned(16))) float red[kWaves][kInRows][16];
  const int64_t tile = block_id() / splits, split = block_id() - tile * splits, t0 = tile * kInRows;
  if (t0 >= a.rows) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, r16 = lane & 15, q = lane >> 4;
  const int64_t k0 = min((split * kWaves + wave) * k_wave, a.c_x), k1 = min(k0 + k_wave, a.c_x);
  const int64_t stages = (k1 - k0) / (32 * kSteps);
  // a uniform address and 32 bits of a lane's own: bytes of its rows
  const TX* const xt = static_cast<const TX*>(a.x) + t0 * a.ld_x;
  uint32_t x[kSub];
#pragma unroll
  for (int h = 0; h < kSub; ++h) x[h] = ((uint32_t)(min((int64_t)(16 * h + r16), a.rows - 1 - t0) * a.ld_x) + 8 * q) * sizeof(TX);
  struct Stage {
    Frag x[kSteps][kSub], w[kSteps][kR16];
  };
  const auto load_x = [&](Stage& f, int64_t k) {
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
#pragma unroll
      for (int h = 0; h < kSub; ++h) load_frag(at_byte(xt + k + 32 * u, x[h]), f.x[u][h]);
  };
  Stage f0, f1;
  if (stages > 0) load_x(f0, k0);  // before it is known whose rows they are
  tile_adapters<kInRows>(a.seg, t0, a.rows, of);
  const int mine = of[lane % kInRows];
  unsigned long long left = __ballot(mine >= 0);
  float* const dst = part + split * a.rows * a.rank;
  bool again = false;
  while (left) {  // the same for the whole workgroup
    const int g = __builtin_amdgcn_readlane(mine, __ffsll(left) - 1);
    left &= ~__ballot(mine == g);
    const TW* const wt = static_cast<const TW*>(a.in) + (int64_t)g * a.rank * a.c_x;
    uint32_t w[kR16];
#pragma unroll
    for (int i = 0; i < kR16; ++i) w[i] = ((uint32_t)(min((int64_t)(16 * i + r16), a.rank - 1) * a.c_x) + 8 * q) * sizeof(TW);
    f32x4_t acc[kR16][kSub];
#pragma unroll
    for (int i = 0; i < kR16; ++i)
#pragma unroll
      for (int h = 0; h < kSub; ++h) acc[i][h] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const auto load_w = [&](Stage& f, int64_t k) {
#pragma unroll
      for (int u = 0; u < kSteps; ++u)
#pragma unroll
        for (int i = 0; i < kR16; ++i) load_frag(at_byte(wt + k + 32 * u, w[i]), f.w[u][i]);
    };
    const auto add = [&](const Stage& f) {
#pragma unroll
      for (int u = 0; u < kSteps; ++u)
#pragma unroll
        for (int i = 0; i < kR16; ++i)
#pragma unroll
          for (int h = 0; h < kSub; ++h) acc[i][h] = multiply(f.w[u][i], f.x[u][h], acc[i][h]);
    };
    int64_t k = k0, n = stages;
    if (n > 0) {
      if (again) load_x(f0, k);
      load_w(f0, k);
    }
    while (n >= 2) {
      load_x(f1, k + 32 * kSteps);
      load_w(f1, k + 32 * kSteps);
      add(f0);
      if (n > 2) {
        load_x(f0, k + 64 * kSteps);
        load_w(f0, k + 64 * kSteps);
      }
      add(f1);
      k += 64 * kSteps;
      n -= 2;
    }
    if (n > 0) {
      add(f0);
      k += 32 * kSteps;
    }
    again = true;
    for (; k < k1; k += 32) {
      Frag fx[kSub];
      const int64_t in = k1 - k - 8 * q;  // elements of this lane inside the row
#pragma unroll
      for (int h = 0; h < kSub; ++h) {
        if (in >= 8) load_frag(at_byte(xt + k, x[h]), fx[h]);
        else load_frag(at_byte(xt + k, x[h]), in, fx[h]);
      }
#pragma unroll
      for (int i = 0; i < kR16; ++i) {
        Frag fw;
        if (in >= 8) load_frag(at_byte(wt + k, w[i]), fw);
        else load_frag(at_byte(wt + k, w[i]), in, fw);
#pragma unroll
        for (int h = 0; h < kSub; ++h) acc[i][h] = multiply(fw, fx[h], acc[i][h]);
      }
    }
    // lane: ranks 16 i + 4 q .. + 3 of the row 16 h + r16
#pragma unroll
    for (int i = 0; i < kR16; ++i) {
#pragma unroll
      for (int h = 0; h < kSub; ++h) *reinterpret_cast<f32x4_t*>(&red[wave][16 * h + r16][4 * q]) = acc[i][h];
      __syncthreads();
#pragma unroll
      for (int e = tid; e < kInRows * 16; e += 64 * kWaves) {
        const int t = e >> 4, r = e & 15;
        if (of[t] == g && 16 * i + r < a.rank) {
          float v = red[0][t][r];
#pragma unroll
          for (int u = 1; u < kWaves; ++u) v += red[u][t][r];
          dst[(t0 + t) * a.rank + 16 * i + r] = v;
        }
      }
      __syncthreads();
    }
  }
  for (int64_t e = tid; e < kInRows * a.rank; e += 64 * kWaves) {
    const int64_t t = e / a.rank;
    if (of[t] == -1) dst[t0 * a.rank + e] = 0.0f;
  }
}

// kN consecutive values of a row as they are, the first n of them inside it (the
// others are zero), in whole words.
template <int kN, typename T>
struct Run {
  static constexpr int kWords = kN * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    else return __uint_as_float(w[i]);
  }
};
template <int kN, typename T>
__device__ __forceinline__ Run<kN, T> load_raw(const T* p, int64_t n) {
  Run<kN, T> r;
  if (n >= kN) {
    __builtin_memcpy(r.w, p, sizeof r.w);
    return r;
  }
#pragma unroll
  for (int i = 0; i < Run<kN, T>::kWords; ++i) {
    if constexpr (sizeof(T) == 2)
      r.w[i] = (2 * i < n ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    else
      r.w[i] = i < n ? __float_as_uint(p[i]) : 0u;
  }
  return r;
}
// The same as fp32.
template <int kN, typename T>
__device__ __forceinline__ void load_run(const T* p, int64_t n, float (&v)[kN]) {
  const Run<kN, T> r = load_raw<kN>(p, n);
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = r.at(i);
}
template <int kN>
__device__ __forceinline__ void store_run(float* p, int64_t n, const float (&v)[kN]) {
  if (n >= kN) {
    __builtin_memcpy(p, v, sizeof v);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i < n) p[i] = v[i];
  }
}
template <int kN>
__device__ __forceinline__ void store_run(uint16_t* p, int64_t n, const float (&v)[kN]) {
  uint32_t w[kN / 2];
#pragma unroll
  for (int i = 0; i < kN / 2; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  if (n >= kN) {
    __builtin_memcpy(p, w, sizeof w);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}

// kN consecutive values but for the first `skip`.
template <int kN, typename T>
__device__ __forceinline__ void store_own(T* p, int skip, const float (&v)[kN]) {
  if (skip == 0) {
    store_run<kN>(p, kN, v);
  } else if (skip < kN) {
#pragma unroll
    for (int i = 1; i < kN; ++i)
      if (i >= skip) {
        if constexpr (sizeof(T) == 2) p[i] = f32_to_bf16_bits(v[i]);
        else p[i] = v[i];
      }
  }
}

// Out of the rank: a workgroup takes up to 64 rows and 64 kOut outputs, each
// wave 16 kOut of them, a lane kOut consecutive ones (those of one MFMA tile
// are kOut apart, so that a row's outputs are read and written 16 bytes at a
// lane).  A wave's part of the factor stays in its registers, as operands, while
// it goes through the rows 16 at a time, what base holds of the next ones being
// loaded meanwhile.  Factors are stored with the rank first, and an operand wants
// four ranks of one output: bf16 ones are paired across two ranks' rows by byte
// permutation.  s comes through LDS; bf16 factors meet it in three bf16 values that
// add up to it exactly.  8192 rows, 4096
// -> 12288, rank 16: 80 us, 5.0 TB/s, as a copy; rank 64 (4096 x 4096) 26 us, 2.6, at
// two waves a SIMD.  128 or 256 rows a workgroup: 99 -> 105 to 111 us with both kernels.
constexpr int kOutRows = 64;

// kOut outputs of four ranks to the four ranks of each output.
template <int kOut>
__device__ __forceinline__ void pair_ranks(const Run<kOut, uint16_t> (&d)[4], s16x4_t (&to)[kOut]) {
#pragma unroll
  for (int o = 0; o < kOut / 2; ++o) {
    const uint32_t lo[2] = {__builtin_amdgcn_perm(d[1].w[o], d[0].w[o], 0x05040100u),
                            __builtin_amdgcn_perm(d[3].w[o], d[2].w[o], 0x05040100u)};
    const uint32_t hi[2] = {__builtin_amdgcn_perm(d[1].w[o], d[0].w[o], 0x07060302u),
                            __builtin_amdgcn_perm(d[3].w[o], d[2].w[o], 0x07060302u)};
    __builtin_memcpy(&to[2 * o], lo, 8);
    __builtin_memcpy(&to[2 * o + 1], hi, 8);
  }
}

// The bf16 parts of s that bf16 factors meet (0: fp32 factors meet s itself).
template <typename TW>
constexpr int out_planes = sizeof(TW) == 4 ? 0 : 3;

// Four bf16 values, zeros in the place of infinities and NaN.
__device__ __forceinline__ s16x4_t finite_or_zero(s16x4_t v) {
  asm volatile("" : "+v"(v));  // computed where it is used: all of a wave's factors at once would spill
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (v[i] & 0x7f80) == 0x7f80 ? (short)0 : v[i];
  return v;
}

// acc[o] = the sums over all ranks of s, whose parts are part(p, i) for the ranks 16 i on,
// and bf16 factors.  A factor that is infinite or NaN is met by the first part of s alone,
// which has the sign of s and is zero, infinite or NaN where s is (but for s below 2^-133):
// a lower part that is zero would make NaN of the infinity.  As they are rare, all parts
// meet all factors first, and a sum that is NaN has the wave add once more (which costs
// the others 1 us of 79: 8192 rows, 4096 -> 12288, rank 16).
template <int kPlanes, int kR16, int kOut, typename F>
__device__ __forceinline__ void out_of_rank(const s16x4_t (&w)[kR16][kOut], F&& part, f32x4_t (&acc)[kOut]) {
#pragma unroll
  for (int o = 0; o < kOut; ++o) acc[o] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kR16; ++i)
#pragma unroll
    for (int p = kPlanes - 1; p >= 0; --p) {  // the smallest part first
      const s16x4_t sv = part(p, i);
#pragma unroll
      for (int o = 0; o < kOut; ++o) acc[o] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(sv, w[i][o], acc[o], 0, 0, 0);
    }
  bool nan = false;
#pragma unroll
  for (int o = 0; o < kOut; ++o)
    nan |= __builtin_isunordered(acc[o][0], acc[o][1]) | __builtin_isunordered(acc[o][2], acc[o][3]);
  if (__ballot(nan) == 0) return;
#pragma unroll
  for (int o = 0; o < kOut; ++o) {
    acc[o] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kR16; ++i) {
      const s16x4_t finite = finite_or_zero(w[i][o]);
#pragma unroll
      for (int p = kPlanes - 1; p >= 0; --p)
        acc[o] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(part(p, i), p > 0 ? finite : w[i][o], acc[o], 0, 0, 0);
    }
  }
}

// Outputs a lane, so that a wave's part of the factor takes 128 registers at most.
template <typename TW, int kR16>
constexpr int out_run = sizeof(TW) == 2 ? (kR16 <= 4 ? 8 : kR16 <= 8 ? 4 : 2) : (kR16 <= 8 ? 4 : 2);

// Waves per SIMD that the registers are held to: as many as go without spilling.
template <typename TW, typename TY, int kR16>
constexpr int out_waves = sizeof(TW) == 2 ? (kR16 == 1 && sizeof(TY) == 2 ? 3 : kR16 <= 2 || (kR16 <= 8 && sizeof(TY) == 2) ? 2 : 1)
                                          : (kR16 <= 2 ? 3 : kR16 <= 4 ? 2 : 1);

template <typename TW, typename TY, int kR16>
__global__ __launch_bounds__(kThreads, (out_waves<TW, TY, kR16>)) void lora_tile_out_kernel(LoraArgs a, const float* __restrict__ part, int splits,
                                                                 int row_tile, int64_t col_tiles) {
  constexpr int kPlanes = out_planes<TW>, kOut = out_run<TW, kR16>;
  constexpr int kPitch = 16 * kR16 + (kPlanes ? 8 : 4);  // elements of a row in LDS
  extern __shared__ __attribute__((aligned(16))) char lds[];  // kPlanes x [row_tile][kPitch] bf16, or [row_tile][kPitch] fp32
  __shared__ int of[kOutRows];
  const int64_t tile = block_id() / col_tiles, ct = block_id() - tile * col_tiles, t0 = tile * row_tile;
  if (t0 >= a.rows) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, j16 = lane & 15, q = lane >> 4;
  const int64_t rank = a.rank, t1 = min(t0 + row_tile, a.rows);
  // The lane's outputs.  At the end of a row they are moved back, so that all of
  // them can be loaded, and the `skip` first belong to another lane.
  const int64_t c_own = (ct * 64 + 16 * wave) * kOut + kOut * j16, c0 = min(c_own, a.c_y - kOut);
  const int skip = (int)min(c_own - c0, (int64_t)kOut);
  const TY* const base = static_cast<const TY*>(a.base);
  Run<kOut, TY> b[4], next[4];
  const auto load_base = [&](int t, Run<kOut, TY> (&to)[4]) {  // the lane's rows t + 4 q + v
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (base) __builtin_memcpy(to[v].w, base + min(t0 + t + 4 * q + v, t1 - 1) * a.ld_base + c0, sizeof to[v].w);
      else to[v] = Run<kOut, TY>{};
    }
  };
  load_base(0, next);  // before it is known whose rows they are
  tile_adapters<kOutRows>(a.seg, t0, t1, of);
  // s of the tile's rows: the sum of the contraction's shares, in their order
#pragma unroll 2
  for (int e = tid; e < row_tile * 4 * kR16; e += kThreads) {
    const int t = e / (4 * kR16), r = 4 * (e % (4 * kR16));
    float v[4] = {};
    if (of[t] >= -1 && r < rank) {
      const int64_t at = (t0 + t) * rank + r, in = rank - r;
      load_run<4>(part + at, in, v);
      for (int u = 1; u < splits; ++u) {
        float w[4];
        load_run<4>(part + u * a.rows * rank + at, in, w);
#pragma unroll
        for (int h = 0; h < 4; ++h) v[h] += w[h];
      }
      if (a.s && ct == 0 && a.s != part) store_run<4>(a.s + at, in, v);
    }
    if constexpr (kPlanes == 0) {
      *reinterpret_cast<float4*>(lds + (t * kPitch + r) * 4) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint32_t p[2][3];
      split3(v[0], v[1], p[0]);
      split3(v[2], v[3], p[1]);
#pragma unroll
      for (int i = 0; i < kPlanes; ++i)
        *reinterpret_cast<uint2*>(lds + ((i * row_tile + t) * kPitch + r) * 2) = make_uint2(p[0][i], p[1][i]);
    }
  }
  __syncthreads();
  TY* const y = static_cast<TY*>(a.y);
  const int mine = of[lane];
  unsigned long long left = __ballot(mine >= 0);
  while (left) {
    const int g = __builtin_amdgcn_readlane(mine, __ffsll(left) - 1);
    const unsigned long long rows = __ballot(mine == g);
    left &= ~rows;
    const float scale = a.scale ? a.scale[g] : 1.0f;
    // ranks 16 i + 4 q + 0..3 of this lane's outputs
    s16x4_t wb[kPlanes ? kR16 : 1][kOut];
    float wf[kPlanes ? 1 : kR16][4][kOut];
#pragma unroll
    for (int i = 0; i < kR16; ++i) {
      const TW* w = static_cast<const TW*>(a.out) + (int64_t)g * rank * a.c_y + c0;
      Run<kOut, TW> d[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int64_t r = 16 * i + 4 * q + c;
        __builtin_memcpy(d[c].w, w + min(r, rank - 1) * a.c_y, sizeof d[c].w);
#pragma unroll
        for (int o = 0; o < Run<kOut, TW>::kWords; ++o) d[c].w[o] = r < rank ? d[c].w[o] : 0u;
      }
      if constexpr (kPlanes == 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int o = 0; o < kOut; ++o) wf[i][c][o] = d[c].at(o);
      } else {
        pair_ranks<kOut>(d, wb[i]);
      }
    }
#pragma unroll 1
    for (int t = 0; t < row_tile; t += 16) {
#pragma unroll
      for (int v = 0; v < 4; ++v) b[v] = next[v];
      if (t + 16 < row_tile) load_base(t + 16, next);
      if ((rows >> t) & 0xffffull) {
        f32x4_t acc[kOut];
        if constexpr (kPlanes == 0) {
#pragma unroll
          for (int o = 0; o < kOut; ++o) acc[o] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < kR16; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(lds + ((t + j16) * kPitch + 16 * i + 4 * q) * 4);
            const float sv[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int o = 0; o < kOut; ++o) acc[o] = __builtin_amdgcn_mfma_f32_16x16x4f32(sv[c], wf[i][c][o], acc[o], 0, 0, 0);
          }
        } else {
          out_of_rank<kPlanes>(wb, [&](int p, int i) {
            return *reinterpret_cast<const s16x4_t*>(lds + ((p * row_tile + t + j16) * kPitch + 16 * i + 4 * q) * 2);
          }, acc);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t at = t + 4 * q + v;
          if (((rows >> at) & 1) == 0) continue;
          float out[kOut];
#pragma unroll
          for (int o = 0; o < kOut; ++o) out[o] = __builtin_fmaf(scale, acc[o][v], b[v].at(o));
          store_own<kOut>(y + (t0 + at) * a.ld_y + c0, skip, out);
        }
      }
    }
    if (left) load_base(0, next);
  }
  // rows without an adapter
  const unsigned long long bare = __ballot(mine == -1);
  if (bare == 0 || a.base == a.y) return;
#pragma unroll 1
  for (int t = 0; t < row_tile; t += 16) {
    load_base(t, b);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t at = t + 4 * q + v;
      if (((bare >> at) & 1) == 0) continue;
      float out[kOut];
#pragma unroll
      for (int o = 0; o < kOut; ++o) out[o] = b[v].at(o);
      store_own<kOut>(y + (t0 + at) * a.ld_y + c0, skip, out);
    }
  }
}

// ---------------------------------------------------------------------------
// Into the rank for bf16 inputs and factors: the contraction goes in pieces of 64
// elements, a piece of a row being one line of 128 bytes that eight lanes load.
// (Operands straight from global memory take 64 bytes of 16 rows a load, at a
// third of the rate: 201 MB of factors read by 128 workgroups 21 us, in lines
// 6.5.)  The wave's own part of LDS turns lines into operands, without a barrier:
// piece p of row r lies at p ^ (r / 2 % 8), where the 16 rows that are read
// together meet all banks once.  kDeep pieces are in flight.
// ---------------------------------------------------------------------------
// Eight bf16 of a row from p on, the first n of them inside it.
__device__ __forceinline__ uint4 load_piece(const uint16_t* p, int64_t n) {
  if (n >= 8) return load_u128(p);
  uint32_t w[4] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int line_lds(int r16, int sub) { return (r16 + sub) * 16 * 128; }  // bytes a wave

// The sums of a wave over the pieces at k_first, k_first + k_step, .. for the
// rows t0 .. + 16 kSub - 1, adapter by adapter: done(g, acc), in which lanes hold
// the ranks 16 i + 4 q .. + 3 of the row 16 h + j16 (rows of other adapters hold
// what this adapter would give them).  Fills `of`; the whole workgroup calls it.
template <int kR16, int kSub, int kDeep, typename F>
__device__ __forceinline__ void into_rank(const LoraArgs& a, int64_t t0, int64_t k_first, int64_t k_step, char* wave_lds,
                                          int (&of)[16 * kSub], F&& done) {
  const int lane = threadIdx.x & 63, j16 = lane & 15, q = lane >> 4;
  const int l8 = lane >> 3, p8 = lane & 7;  // loading: the row of eight and its piece of 16 bytes
  const uint16_t* const xt = static_cast<const uint16_t*>(a.x) + t0 * a.ld_x;
  uint32_t x_at[2 * kSub], w_at[2 * kR16];  // bytes
#pragma unroll
  for (int i = 0; i < 2 * kSub; ++i) x_at[i] = ((uint32_t)(min((int64_t)(8 * i + l8), a.rows - 1 - t0) * a.ld_x) + 8 * p8) * 2;
#pragma unroll
  for (int i = 0; i < 2 * kR16; ++i) w_at[i] = ((uint32_t)(min((int64_t)(8 * i + l8), a.rank - 1) * a.c_x) + 8 * p8) * 2;
  struct Piece {
    uint4 x[2 * kSub], w[2 * kR16];
  } f[kDeep];
  const auto load_x = [&](Piece& to, int64_t k) {
    if (k + 64 <= a.c_x) {
#pragma unroll
      for (int i = 0; i < 2 * kSub; ++i) to.x[i] = load_u128(at_byte(xt + k, x_at[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 2 * kSub; ++i) to.x[i] = load_piece(at_byte(xt + k, x_at[i]), a.c_x - k - 8 * p8);
    }
  };
  // rows 8 i + l8 go in, operands (row j16 of 16, pieces q and 4 + q) come out
  const uint32_t to_even = l8 * 128 + ((p8 ^ (l8 >> 1)) << 4), to_odd = l8 * 128 + ((p8 ^ ((l8 >> 1) + 4)) << 4);
  const uint32_t from0 = j16 * 128 + ((q ^ (j16 >> 1)) << 4), from1 = j16 * 128 + (((q + 4) ^ (j16 >> 1)) << 4);
  static_for<kDeep>([&](auto d) {  // before it is known whose rows they are
    if (k_first + d * k_step < a.c_x) load_x(f[d], k_first + d * k_step);
  });
  tile_adapters<16 * kSub>(a.seg, t0, a.rows, of);
  const int mine = of[lane % (16 * kSub)];
  unsigned long long left = __ballot(mine >= 0);
  bool again = false;
  while (left) {  // the same for the whole workgroup
    const int g = __builtin_amdgcn_readlane(mine, __ffsll(left) - 1);
    left &= ~__ballot(mine == g);
    const uint16_t* const wt = static_cast<const uint16_t*>(a.in) + (int64_t)g * a.rank * a.c_x;
    const auto load_w = [&](Piece& to, int64_t k) {
      if (k + 64 <= a.c_x) {
#pragma unroll
        for (int i = 0; i < 2 * kR16; ++i) to.w[i] = load_u128(at_byte(wt + k, w_at[i]));
      } else {
#pragma unroll
        for (int i = 0; i < 2 * kR16; ++i) to.w[i] = load_piece(at_byte(wt + k, w_at[i]), a.c_x - k - 8 * p8);
      }
    };
    f32x4_t acc[kR16][kSub];
#pragma unroll
    for (int i = 0; i < kR16; ++i)
#pragma unroll
      for (int h = 0; h < kSub; ++h) acc[i][h] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    static_for<kDeep>([&](auto d) {
      const int64_t k = k_first + d * k_step;
      if (k >= a.c_x) return;
      if (again) load_x(f[d], k);
      load_w(f[d], k);
    });
    again = true;
#pragma unroll 1
    for (int64_t k0 = k_first; k0 < a.c_x; k0 += kDeep * k_step) {
      static_for<kDeep>([&](auto d) {
        const int64_t k = k0 + d * k_step;
        if (k >= a.c_x) return;
#pragma unroll
        for (int i = 0; i < 2 * kSub; ++i)
          *reinterpret_cast<uint4*>(wave_lds + i * 1024 + (i & 1 ? to_odd : to_even)) = f[d].x[i];
#pragma unroll
        for (int i = 0; i < 2 * kR16; ++i)
          *reinterpret_cast<uint4*>(wave_lds + (2 * kSub + i) * 1024 + (i & 1 ? to_odd : to_even)) = f[d].w[i];
        if (k + kDeep * k_step < a.c_x) {
          load_x(f[d], k + kDeep * k_step);
          load_w(f[d], k + kDeep * k_step);
        }
        // a wave's own accesses to LDS are served in order; the fences keep the compiler to it
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          bf16x8_t x[kSub];
#pragma unroll
          for (int h = 0; h < kSub; ++h)
            x[h] = __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const uint4*>(wave_lds + h * 2048 + (u ? from1 : from0)));
#pragma unroll
          for (int i = 0; i < kR16; ++i) {
            const bf16x8_t w =
                __builtin_bit_cast(bf16x8_t, *reinterpret_cast<const uint4*>(wave_lds + (kSub + i) * 2048 + (u ? from1 : from0)));
#pragma unroll
            for (int h = 0; h < kSub; ++h) acc[i][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[h], acc[i][h], 0, 0, 0);
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      });
    }
    done(g, acc);
  }
}

// A workgroup takes 32 rows and a share of the pieces, its waves taking them in
// turn.  (Ranks of 17 to 32 are held to 128 registers, at which two are spilled: 32768
// rows, 2048 -> 1024, 79 us with the way out, and 86 with the registers they ask for.)
template <int kR16>
struct LineShape {
  static constexpr int kSub = 2, kRows = 16 * kSub, kWaves = kR16 <= 4 ? 8 : 4;
  static constexpr int kDeep = kR16 == 1 || kR16 == 4 ? 2 : 1;
};
template <int kR16>
__global__ __launch_bounds__((LineShape<kR16>::kWaves * 64), (kR16 <= 2 ? 4 : kR16 <= 4 ? 2 : 1)) void lora_line_in_kernel(LoraArgs a, int splits,
                                                                                       float* __restrict__ part) {
  using Shape = LineShape<kR16>;
  constexpr int kSub = Shape::kSub, kRows = Shape::kRows, kWaves = Shape::kWaves;
  constexpr int kLds = line_lds(kR16, kSub) * kWaves, kRed = kWaves * kRows * 16 * 4;
  __shared__ __attribute__((aligned(16))) char lds[kLds > kRed ? kLds : kRed];
  __shared__ int of[kRows];
  const int64_t tile = block_id() / splits, split = block_id() - tile * splits, t0 = tile * kRows;
  if (t0 >= a.rows) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, j16 = lane & 15, q = lane >> 4;
  float* const dst = part + split * a.rows * a.rank;
  into_rank<kR16, kSub, Shape::kDeep>(
      a, t0, 64 * (split * kWaves + wave), (int64_t)64 * kWaves * splits, lds + wave * line_lds(kR16, kSub), of,
      [&](int g, const f32x4_t (&acc)[kR16][kSub]) {
        float* const red = reinterpret_cast<float*>(lds);  // [kWaves][kRows][16]
#pragma unroll
        for (int i = 0; i < kR16; ++i) {
          __syncthreads();
#pragma unroll
          for (int h = 0; h < kSub; ++h)
            *reinterpret_cast<f32x4_t*>(red + (wave * kRows + 16 * h + j16) * 16 + 4 * q) = acc[i][h];
          __syncthreads();
          for (int e = tid; e < kRows * 16; e += 64 * kWaves) {
            const int t = e >> 4, r = e & 15;
            if (of[t] == g && 16 * i + r < a.rank) {
              float v = red[e];
#pragma unroll
              for (int u = 1; u < kWaves; ++u) v += red[u * kRows * 16 + e];
              dst[(t0 + t) * a.rank + 16 * i + r] = v;
            }
          }
        }
        __syncthreads();
      });
  for (int e = tid; e < kRows * (int)a.rank; e += 64 * kWaves)
    if (of[e / (int)a.rank] == -1) dst[t0 * a.rank + e] = 0.0f;
}

// ---------------------------------------------------------------------------
// Both ways in one launch, for bf16 inputs and factors, a rank up to 16 and many
// rows: a workgroup of eight waves takes 16 rows through the whole contraction and
// out to all outputs, so that s stays in LDS.  It saves a launch and what the first
// kernel leaves in memory, but has fewer bytes in flight on the way out: see both_ways.
// ---------------------------------------------------------------------------
constexpr int kBothWaves = 8;

template <typename TY>
__global__ __launch_bounds__(64 * kBothWaves, (sizeof(TY) == 2 ? 4 : 2)) void lora_both_kernel(LoraArgs a) {
  constexpr int kRows = 16, kOut = 4, kPlanes = out_planes<uint16_t>;
  constexpr int kPitch = 16 + 8;  // elements of a row of a plane
  __shared__ __attribute__((aligned(16))) char lds[kBothWaves * line_lds(1, 1)];  // (the sums take a quarter of it)
  __shared__ __attribute__((aligned(16))) uint16_t planes[kPlanes][kRows][kPitch];
  __shared__ int of[kRows];
  const int64_t t0 = block_id() * kRows;
  if (t0 >= a.rows) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, j16 = lane & 15, q = lane >> 4;
  const int64_t rank = a.rank, t1 = min(t0 + kRows, a.rows);
  into_rank<1, 1, 2>(a, t0, 64 * wave, 64 * kBothWaves, lds + wave * line_lds(1, 1), of,
                           [&](int g, const f32x4_t (&acc)[1][1]) {
                             float* const red = reinterpret_cast<float*>(lds);  // [kBothWaves][kRows][16]
                             __syncthreads();
                             *reinterpret_cast<f32x4_t*>(red + (wave * kRows + j16) * 16 + 4 * q) = acc[0][0];
                             __syncthreads();
                             const int t = tid >> 2, r = 4 * (tid & 3);
                             if (tid < 4 * kRows && of[t] == g) {
                               float v[4] = {};
#pragma unroll
                               for (int u = 0; u < kBothWaves; ++u) {
                                 const f32x4_t p = *reinterpret_cast<const f32x4_t*>(red + (u * kRows + t) * 16 + r);
#pragma unroll
                                 for (int i = 0; i < 4; ++i) v[i] += p[i];
                               }
#pragma unroll
                               for (int i = 0; i < 4; ++i) v[i] = r + i < rank ? v[i] : 0.0f;
                               if (a.s && r < rank) store_run<4>(a.s + (t0 + t) * rank + r, rank - r, v);
                               uint32_t p[2][3];
                               split3(v[0], v[1], p[0]);
                               split3(v[2], v[3], p[1]);
#pragma unroll
                               for (int i = 0; i < kPlanes; ++i)
                                 *reinterpret_cast<uint2*>(&planes[i][t][r]) = make_uint2(p[0][i], p[1][i]);
                             }
                             __syncthreads();
                           });
  const int mine = of[j16];
  const unsigned long long all = __ballot(mine >= 0) & 0xffffull, bare = __ballot(mine == -1) & 0xffffull;
  unsigned long long left = all;
  for (int e = tid; a.s && bare && e < kRows * (int)rank; e += 64 * kBothWaves)
    if (of[e / (int)rank] == -1) a.s[t0 * rank + e] = 0.0f;

  // out of the rank: a wave takes 16 kOut outputs in turn, a lane kOut
  const TY* const base = static_cast<const TY*>(a.base);
  TY* const y = static_cast<TY*>(a.y);
  Run<kOut, TY> b[4], b_next[4];
  Run<kOut, uint16_t> w_next[4];
  // uniform addresses and bytes of the lane's own: its outputs of the rows 4 q + v and of the ranks 4 q + v
  uint32_t b_at[4], y_at[4], f_at[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const uint32_t t = (uint32_t)min((int64_t)(4 * q + v), t1 - t0 - 1);
    b_at[v] = (t * (uint32_t)a.ld_base + kOut * j16) * sizeof(TY);
    y_at[v] = (t * (uint32_t)a.ld_y + kOut * j16) * sizeof(TY);
    f_at[v] = (min((uint32_t)(4 * q + v), (uint32_t)rank - 1) * (uint32_t)a.c_y + kOut * j16) * 2;
  }
  // At the end of a row a lane's outputs are moved back, so that all of them can
  // be loaded, and the first ones belong to another lane.
  const auto past = [&](int c_wave) { return max(c_wave + kOut * j16 + kOut - (int)a.c_y, 0); };
  const TY* const base_t = base ? base + t0 * a.ld_base : nullptr;
  const auto load_base = [&](int c_wave, Run<kOut, TY> (&to)[4]) {
    const uint32_t c = (c_wave - past(c_wave)) * (int)sizeof(TY);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (base) __builtin_memcpy(to[v].w, at_byte(base_t, b_at[v] + c), sizeof to[v].w);
      else to[v] = Run<kOut, TY>{};
    }
  };
  const int c_first = wave * 16 * kOut, c_step = 16 * kOut * kBothWaves, c_end = (int)a.c_y;
  left = all;
  while (left) {
    const int g = __builtin_amdgcn_readlane(mine, __ffsll(left) - 1);
    const unsigned long long rows = __ballot(mine == g);
    left &= ~rows;
    const float scale = a.scale ? a.scale[g] : 1.0f;
    const uint16_t* const wt = static_cast<const uint16_t*>(a.out) + (int64_t)g * rank * a.c_y;
    const auto load_w = [&](int c_wave) {
      const uint32_t at = (c_wave - past(c_wave)) * 2;
#pragma unroll
      for (int c = 0; c < 4; ++c) __builtin_memcpy(w_next[c].w, at_byte(wt, f_at[c] + at), sizeof w_next[c].w);
    };
    if (c_first < c_end) {
      load_w(c_first);
      load_base(c_first, b_next);
    }
#pragma unroll 1
    for (int c_wave = c_first; c_wave < c_end; c_wave += c_step) {
      s16x4_t wb[1][kOut];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int o = 0; o < kOut / 2; ++o) w_next[c].w[o] = 4 * q + c < rank ? w_next[c].w[o] : 0u;
      pair_ranks<kOut>(w_next, wb[0]);
#pragma unroll
      for (int v = 0; v < 4; ++v) b[v] = b_next[v];
      if (c_wave + c_step < c_end) {
        load_w(c_wave + c_step);
        load_base(c_wave + c_step, b_next);
      }
      const int skip = min(past(c_wave), kOut);
      TY* const y_t = y + t0 * a.ld_y;
      const uint32_t y_c = (c_wave - past(c_wave)) * (int)sizeof(TY);
      f32x4_t acc[kOut];
      out_of_rank<kPlanes>(wb, [&](int p, int) { return *reinterpret_cast<const s16x4_t*>(&planes[p][j16][4 * q]); }, acc);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if (((rows >> (4 * q + v)) & 1) == 0) continue;
        float out[kOut];
#pragma unroll
        for (int o = 0; o < kOut; ++o) out[o] = __builtin_fmaf(scale, acc[o][v], b[v].at(o));
        store_own<kOut>(at_byte(y_t, y_at[v] + y_c), skip, out);
      }
    }
  }
  // rows without an adapter
  if (bare == 0 || a.base == a.y) return;
#pragma unroll 1
  for (int c_wave = c_first; c_wave < c_end; c_wave += c_step) {
    const int skip = min(past(c_wave), kOut);
    const uint32_t y_c = (c_wave - past(c_wave)) * (int)sizeof(TY);
    load_base(c_wave, b);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (((bare >> (4 * q + v)) & 1) == 0) continue;
      float out[kOut];
#pragma unroll
      for (int o = 0; o < kOut; ++o) out[o] = b[v].at(o);
      store_own<kOut>(at_byte(y + t0 * a.ld_y, y_at[v] + y_c), skip, out);
    }
  }
}

// ---------------------------------------------------------------------------
// Gradients to the factors, out[g][r][c] = scale[g] sum_t p[t][r] x[t][c]: a
// product whose contraction runs over an adapter's rows.  The rows of adapter g
// are those of all its segments, one after the other; a workgroup takes `chunk`
// of them (a slot) and 16 kOut columns, its waves every fourth step of 32 rows.
// A lane loads kOut consecutive columns of the eight rows 8 q .. 8 q + 7 of a
// step and pairs rows by byte permutation, so that tile i of the product has the
// columns kOut j + i; p meets them in three bf16 values that add up to it
// exactly.  (fp32 rows: both as they are, v_mfma_f32_16x16x4_f32.)  Checkpoints
// in 8 bits are decoded straight into that pairing, in bf16, which holds them.
// Adapters of one slot are finished here; the sums of the others' slots are
// added by lora_weight_sum_kernel in order: no atomics on data.  4096 rows of rank 64,
// 4096 and 12288 columns: 49 us and 6 for the sums, 2.9 TB/s; 32768 rows on 64 adapters
// of rank 16, 2048 columns in 8 bits and 1024: 48 and 8.  Bound by vector issue (p is
// cut by every wave) and the latency of a step's loads, one step ahead, at two or three
// waves a SIMD.
// ---------------------------------------------------------------------------
// Where slot `s` works: adapter g, its rows k chunk .. in their order, and how
// many there are; `parts` counts the slots of adapters with several before it.
struct Slot {
  int g;
  int64_t row0, row1;  // of the adapter's rows
  int slots;           // the adapter's
  int part;            // the adapter's first place among the parts
};

// The rows of segment i, clamped into the buffer; whether its end lies before its beginning.
__device__ __forceinline__ bool segment_rows(const SegmentArgs& g, int64_t n_rows, int64_t i, int64_t& lo, int64_t& hi) {
  if (g.offsets) {
    lo = min(max(g.offsets[i], (int64_t)0), n_rows);
    hi = min(max(g.offsets[i + 1], (int64_t)0), n_rows);
  } else {
    lo = g.n == 1 ? 0 : i;
    hi = g.n == 1 ? n_rows : i + 1;
  }
  const bool falls = hi < lo;
  hi = max(lo, hi);
  return falls;
}

// Segments overlap only where offsets decrease.  A row is then the first segment's
// that has it: the runs of rows that are a segment's own, f(i, lo, hi), for the
// segments that are wanted, in order, by a whole wave.  (Not a path for speed: a run
// looks at all earlier segments, unless they are known to have the whole segment.)
template <typename W, typename F>
__device__ __forceinline__ void own_runs(const SegmentArgs& g, int64_t n_rows, W&& wanted, F&& f) {
  const int lane = threadIdx.x & 63;
  int64_t c0 = 0, c1 = 0;  // rows that earlier segments have without a gap
  for (int64_t i0 = 0; i0 < g.n; i0 += 64) {
    int64_t lo = 0, hi = 0;
    if (i0 + lane < g.n) segment_rows(g, n_rows, i0 + lane, lo, hi);
    unsigned long long left = __ballot(lo < hi);
    while (left) {
      const int l = __ffsll(left) - 1;
      left &= left - 1;
      const int64_t i = i0 + l, from = __shfl(lo, l), to = __shfl(hi, l);
      if (c0 <= from && to <= c1) continue;
      if (wanted(i))
        for (int64_t at = from; at < to;) {
          int64_t past = at, next = to;  // where those that have row `at` end, and where another begins
          for (int64_t j = lane; j < i; j += 64) {
            int64_t a, b;
            segment_rows(g, n_rows, j, a, b);
            if (a <= at) past = max(past, b);
            else if (a < b) next = min(next, a);
          }
#pragma unroll
          for (int off = 1; off < 64; off <<= 1) {
            past = max(past, (int64_t)__shfl_xor(past, off));
            next = min(next, (int64_t)__shfl_xor(next, off));
          }
          if (past == at) f(i, at, next);
          at = past == at ? next : past;
        }
      if (from <= c1 && c0 <= to) {
        c0 = min(c0, from);
        c1 = max(c1, to);
      } else if (to - from > c1 - c0) {
        c0 = from;
        c1 = to;
      }
    }
  }
}

// The first segments as the workgroup has read them, for list_rows.
constexpr int kKnown = 256;
struct Segments {
  unsigned long long cnt[kLoraMaxAdapters];
  int lo[kKnown], len[kKnown], id[kKnown];
  int falls;  // whether offsets decrease anywhere
};
// cnt[g] = rows of adapter g, by the whole workgroup; n_rows at most over all adapters.
__device__ __forceinline__ void count_rows(const SegmentArgs& g, int64_t n_rows, Segments& s) {
  const int tid = threadIdx.x;
  int64_t lo = 0, hi = 0, id = -1;
  bool falls = false;
  if (tid < g.n) {  // loaded while the counters are cleared
    falls = segment_rows(g, n_rows, tid, lo, hi);
    id = adapter_of(g, tid);
  }
  for (int i = tid; i < (int)g.n_adapters; i += kThreads) s.cnt[i] = 0;
  if (tid == 0) s.falls = 0;
  __syncthreads();
  s.lo[tid] = (int)lo;
  s.len[tid] = (int)(hi - lo);
  s.id[tid] = (int)id;
  if (id >= 0 && hi > lo) atomicAdd(&s.cnt[id], (unsigned long long)(hi - lo));
  for (int64_t i = tid + kThreads; i < g.n; i += kThreads) {
    id = adapter_of(g, i);
    falls |= segment_rows(g, n_rows, i, lo, hi);
    if (id >= 0 && hi > lo) atomicAdd(&s.cnt[id], (unsigned long long)(hi - lo));
  }
  if (falls) s.falls = 1;
  __syncthreads();
  if (s.falls == 0) return;
  for (int i = tid; i < (int)g.n_adapters; i += kThreads) s.cnt[i] = 0;
  __syncthreads();
  if (tid < 64)
    own_runs(g, n_rows, [&](int64_t i) { return adapter_of(g, i) >= 0; }, [&](int64_t i, int64_t a, int64_t b) {
      if (tid == 0) s.cnt[adapter_of(g, i)] += (unsigned long long)(b - a);
    });
  __syncthreads();
}
static_assert(kKnown == kThreads);
// The slot `want` (kByAdapter: the first slot of adapter `want`), every wave for itself.
template <bool kByAdapter>
__device__ __forceinline__ bool find_slot(const unsigned long long* cnt, int n_adapters, int chunk, int64_t want, Slot& s) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0, parts = 0;
  for (int g0 = 0; g0 < n_adapters; g0 += 64) {
    const bool in = g0 + lane < n_adapters;
    const unsigned long long rows = in ? cnt[g0 + lane] : 0;
    const int slots = in ? max(1, (int)((rows + chunk - 1) / (unsigned)chunk)) : 0;
    int incl = slots, pin = slots > 1 ? slots : 0;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int u = __shfl_up(incl, off), v = __shfl_up(pin, off);
      if (lane >= off) incl += u, pin += v;
    }
    const unsigned long long hit = kByAdapter ? __ballot(g0 + lane == want) : __ballot(before + incl > want);
    if (hit) {
      const int l = __ffsll(hit) - 1;
      s.g = g0 + l;
      s.slots = __builtin_amdgcn_readlane(slots, l);
      s.part = (int)parts + __builtin_amdgcn_readlane(pin, l) - (s.slots > 1 ? s.slots : 0);
      const int64_t k = kByAdapter ? 0 : want - before - (__builtin_amdgcn_readlane(incl, l) - s.slots);
      s.row0 = k * chunk;
      s.row1 = min(s.row0 + chunk, uniform((int64_t)cnt[s.g]));
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
    parts += __builtin_amdgcn_readlane(pin, 63);
  }
  return false;
}

constexpr int kMostChunk = 2048;  // rows of a slot, which are listed in LDS

// list[0 .. row1 - row0): the buffer's rows, by the whole workgroup; the caller
// waits before it reads them.
__device__ __forceinline__ void list_rows(const SegmentArgs& g, int64_t n_rows, const Segments& known, const Slot& s,
                                          int* list) {
  const int tid = threadIdx.x, lane = tid & 63;
  int64_t at = 0;  // the adapter's rows before this group of segments
  if (known.falls) {  // every wave goes through the runs and lists its threads' share
    own_runs(g, n_rows, [&](int64_t i) { return at < s.row1 && adapter_of(g, i) == s.g; }, [&](int64_t, int64_t a, int64_t b) {
      const int64_t f1 = min(at + b - a, s.row1);
      for (int64_t f = max(at, s.row0) + tid; f < f1; f += kThreads) list[f - s.row0] = (int)(a + f - at);
      at += b - a;
    });
    return;
  }
  for (int64_t i0 = 0; i0 < g.n && at < s.row1; i0 += 64) {
    int64_t lo = 0, hi = 0;
    const int64_t i = i0 + lane;
    if (i0 < kKnown) {
      lo = known.lo[i];
      hi = known.id[i] == s.g ? lo + known.len[i] : lo;
    } else if (i < g.n && adapter_of(g, i) == s.g) {
      segment_rows(g, n_rows, i, lo, hi);
    }
    const int64_t len = hi - lo;
    uint32_t incl = (uint32_t)len;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t u = (uint32_t)__shfl_up((int)incl, off);
      if (lane >= off) incl += u;
    }
    const int64_t first = at + incl - len;
    const int64_t f0 = max(first, s.row0), f1 = min(first + len, s.row1);  // the part of the segment that is wanted
    if (f1 > f0 && len <= 4 && tid < 64)
      for (int64_t f = f0; f < f1; ++f) list[f - s.row0] = (int)(lo + f - first);
    unsigned long long more = __ballot(f1 > f0 && len > 4);
    while (more) {
      const int l = __ffsll(more) - 1;
      more &= more - 1;
      const int64_t a0 = __shfl(f0, l), a1 = __shfl(f1, l), from = __shfl(lo - first, l);
      for (int64_t f = a0 + tid; f < a1; f += kThreads) list[f - s.row0] = (int)(from + f);
    }
    at += (uint32_t)__builtin_amdgcn_readlane((int)incl, 63);
  }
}

// kOut consecutive columns of one row, the first n of them inside it (kWhole: all
// are): bf16 pairs (dtypes 1, 2) or fp32.  Checkpoints come as their bytes, and
// their scale beside them.
template <int kDtype, int kOut>
struct Cols {
  uint32_t w[kDtype == 0 ? kOut : kDtype == 1 ? kOut / 2 : (kOut + 3) / 4];
  uint32_t scale;
};
template <int kDtype, int kOut, bool kWhole>
__device__ __forceinline__ void load_cols(const LoraFactor& f, int row, int64_t c, int64_t n, Cols<kDtype, kOut>& r) {
  using T = std::conditional_t<kDtype == 0, float, std::conditional_t<kDtype == 1, uint16_t, uint8_t>>;
  // (one 32 x 32 bit product each: no row is 2^31 elements long)
  const uint32_t ld = (uint32_t)(kDtype == 2 ? f.cols : f.ld);
  const T* p = static_cast<const T*>(f.x) + ((uint64_t)(uint32_t)row * ld + (uint64_t)c);
  if constexpr (kDtype == 2) {
    const uint32_t blocks = (ld + 31) / 32;
    r.scale = kWhole || n > 0 ? f.x_scale[(uint64_t)(uint32_t)row * blocks + (uint64_t)(c >> 5)] : 127u;
  }
  if (kWhole || n >= kOut) {
    __builtin_memcpy(r.w, p, kOut * sizeof(T));
  } else {
    constexpr int kPer = 4 / sizeof(T);
#pragma unroll
    for (int i = 0; i < (int)(sizeof r.w / 4); ++i) {
      r.w[i] = 0;
#pragma unroll
      for (int o = 0; o < kPer; ++o) {
        T v = T(0);
        if (kPer * i + o < n) v = p[kPer * i + o];
        if constexpr (sizeof(T) == 4) r.w[i] = __float_as_uint(v);
        else r.w[i] |= (uint32_t)v << (8 * (int)sizeof(T) * o);
      }
    }
  }
}
// Pair o of them as bf16 (exact: E4M3 has 4 significant bits).
template <int o, int kDtype, int kOut>
__device__ __forceinline__ uint32_t pair_of(const Cols<kDtype, kOut>& r) {
  if constexpr (kDtype == 1) {
    return r.w[o];
  } else {
    const bf16x2_t v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.w[o / 2], e8m0_to_f32(r.scale), o % 2 != 0);
    return __builtin_bit_cast(uint32_t, v);
  }
}

// split3 without its care for infinities: they leave NaN in the second part.
__device__ __forceinline__ void split3_finite(float a, float b, uint32_t (&p)[3]) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  const uint32_t ra = __float_as_uint(a - __uint_as_float(ua & 0xffff0000u)), rb = __float_as_uint(b - __uint_as_float(ub & 0xffff0000u));
  const float la = __uint_as_float(ra) - __uint_as_float(ra & 0xffff0000u), lb = __uint_as_float(rb) - __uint_as_float(rb & 0xffff0000u);
  p[0] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
  p[1] = __builtin_amdgcn_perm(rb, ra, 0x07060302u);
  p[2] = __builtin_amdgcn_perm(__float_as_uint(lb), __float_as_uint(la), 0x07060302u);
}

// A lane's share of a step of 32 rows of the list: the rows 8 q + j.  kWhole: rows
// and columns are all inside; else those past `count` are zeros.
template <int kDtype, int kR16, int kOut>
struct Step {
  Cols<kDtype, kOut> x[8];
  float p[kR16][8];
};
template <int kDtype, int kR16, int kOut, bool kWhole>
__device__ __forceinline__ void load_step(const LoraFactor& f, int64_t rank, const int* list, int at, int count, int64_t c,
                                          int64_t n, Step<kDtype, kR16, kOut>& s) {
  const int r16 = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
  int row[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = at + 8 * q + j;
    row[j] = kWhole || i < count ? list[i] : -1;
    if (kWhole || i < count) load_cols<kDtype, kOut, kWhole>(f, row[j], c, n, s.x[j]);
    else s.x[j] = Cols<kDtype, kOut>{};
  }
  int r[kR16];
#pragma unroll
  for (int i = 0; i < kR16; ++i) r[i] = min(16 * i + r16, (int)rank - 1);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float* p = f.p + (uint64_t)(uint32_t)row[j] * (uint32_t)rank;
#pragma unroll
    for (int i = 0; i < kR16; ++i) s.p[i][j] = kWhole || row[j] >= 0 ? p[r[i]] : 0.0f;
  }
}
template <int kDtype, int kR16, int kOut>
__device__ __forceinline__ void add_step(const Step<kDtype, kR16, kOut>& s, f32x4_t (&acc)[kR16][kOut]) {
  const auto& p = s.p;
  if constexpr (kDtype == 0) {
#pragma unroll
    for (int i = 0; i < kR16; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int o = 0; o < kOut; ++o)
          acc[i][o] = __builtin_amdgcn_mfma_f32_16x16x4f32(p[i][j], __uint_as_float(s.x[j].w[o]), acc[i][o], 0, 0, 0);
  } else {
    uint32_t b[kOut][4];  // operands: rows 8 q + 2 j, + 1 of one column
    static_for<kOut / 2>([&](auto o) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = pair_of<o>(s.x[2 * j]), hi = pair_of<o>(s.x[2 * j + 1]);
        b[2 * o][j] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
        b[2 * o + 1][j] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
      }
    });
#pragma unroll
    for (int i = 0; i < kR16; ++i) {
      uint32_t a[4][3];
#pragma unroll
      for (int j = 0; j < 4; ++j) split3_finite(p[i][2 * j], p[i][2 * j + 1], a[j]);
#pragma unroll
      for (int u = 2; u >= 0; --u) {  // the smallest part first
        const bf16x8_t fa = __builtin_bit_cast(bf16x8_t, make_uint4(a[0][u], a[1][u], a[2][u], a[3][u]));
#pragma unroll
        for (int o = 0; o < kOut; ++o)
          acc[i][o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              fa, __builtin_bit_cast(bf16x8_t, make_uint4(b[o][0], b[o][1], b[o][2], b[o][3])), acc[i][o], 0, 0, 0);
      }
    }
  }
}

// scale v + beta out, kN consecutive elements, the first n of them inside the row.
template <int kN>
__device__ __forceinline__ void finish(const LoraWeightArgs& a, const LoraFactor& f, float scale, int64_t at, int64_t n,
                                       const float (&v)[kN]) {
  float w[kN], old[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) w[i] = scale * v[i];
  if (a.out_dtype == 1) {
    uint16_t* p = static_cast<uint16_t*>(f.out) + at;
    if (a.beta != 0.0f) {
      load_run<kN>(p, n, old);
#pragma unroll
      for (int i = 0; i < kN; ++i) w[i] = __builtin_fmaf(a.beta, old[i], w[i]);
    }
    store_run<kN>(p, n, w);
  } else {
    float* p = static_cast<float*>(f.out) + at;
    if (a.beta != 0.0f) {
      load_run<kN>(p, n, old);
#pragma unroll
      for (int i = 0; i < kN; ++i) w[i] = __builtin_fmaf(a.beta, old[i], w[i]);
    }
    store_run<kN>(p, n, w);
  }
}

// Columns a lane takes, so that the sums of a wave take 128 registers at most.
constexpr int weight_run(int r16, int dtype) { return r16 <= 2 ? (dtype == 0 ? 4 : 8) : r16 <= 8 ? 4 : 2; }

template <int kOut>
union WeightLds {  // the sums come last
  struct {
    Segments segments;
    int list[kMostChunk];
  };
  float red[kThreads / 64 * 16 * 16 * kOut];
};

template <int kDtype, int kR16>
__device__ __forceinline__ void weight_tile(const LoraWeightArgs& a, const LoraFactor& f, int64_t chunk, int64_t want,
                                            int64_t ct, float* __restrict__ part,
                                            WeightLds<weight_run(kR16, kDtype)>& lds) {
  constexpr int kOut = weight_run(kR16, kDtype);
  float* const red = lds.red;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, j16 = lane & 15, q = lane >> 4;
  count_rows(a.seg, a.rows, lds.segments);
  Slot s;
  if (!find_slot<false>(lds.segments.cnt, (int)a.seg.n_adapters, (int)chunk, want, s)) return;  // the whole workgroup
  list_rows(a.seg, a.rows, lds.segments, s, lds.list);
  __syncthreads();
  const int count = (int)(s.row1 - s.row0);
  const int64_t c_tile = ct * 16 * kOut, c = c_tile + kOut * j16, n = f.cols - c;
  f32x4_t acc[kR16][kOut];
#pragma unroll
  for (int i = 0; i < kR16; ++i)
#pragma unroll
    for (int o = 0; o < kOut; ++o) acc[i][o] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  int at = 32 * wave;
  if (c_tile + 16 * kOut <= f.cols && at + 32 <= count) {  // the next step's loads are in flight while this one is added
    Step<kDtype, kR16, kOut> next;
    load_step<kDtype, kR16, kOut, true>(f, a.rank, lds.list, at, count, c, n, next);
#pragma unroll 1
    for (; at + 32 <= count; at += 128) {
      const Step<kDtype, kR16, kOut> s0 = next;
      if (at + 160 <= count) load_step<kDtype, kR16, kOut, true>(f, a.rank, lds.list, at + 128, count, c, n, next);
      add_step(s0, acc);
    }
  }
#pragma unroll 1
  for (; at < count; at += 128) {
    Step<kDtype, kR16, kOut> s0;
    load_step<kDtype, kR16, kOut, false>(f, a.rank, lds.list, at, count, c, n, s0);
    add_step(s0, acc);
  }
  // the waves' sums, 16 ranks at a time; a thread has kOut columns of one rank
  const float scale = a.scale ? a.scale[s.g] : 1.0f;
  const int r = tid >> 4;
#pragma unroll
  for (int i = 0; i < kR16; ++i) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int o = 0; o < kOut; ++o) red[(wave * 16 + 4 * q + v) * 16 * kOut + kOut * j16 + o] = acc[i][o][v];
    __syncthreads();
    float sum[kOut];
#pragma unroll
    for (int o = 0; o < kOut; ++o) {
      sum[o] = red[r * 16 * kOut + kOut * j16 + o];
#pragma unroll
      for (int w = 1; w < kThreads / 64; ++w) sum[o] += red[(w * 16 + r) * 16 * kOut + kOut * j16 + o];
    }
    if (16 * i + r < a.rank && n > 0) {
      const int64_t k = s.slots > 1 ? s.part + s.row0 / chunk : s.g;
      const int64_t to = (k * a.rank + 16 * i + r) * f.cols + c;
      if (s.slots == 1) finish<kOut>(a, f, scale, to, n, sum);
      else store_run<kOut>(part + to, n, sum);
    }
  }
}

// Both factors' tiles, those of the first before those of the second; a factor
// that is not asked for has none.
struct WeightWork {
  int64_t chunk, slots;
  int64_t tiles[2];  // of columns
  float* part[2];
};
template <int kDx, int kDy, int kR16>
__global__ __launch_bounds__(kThreads, (kR16 <= 1 ? 3 : kR16 <= 4 ? 2 : 1)) void lora_weight_kernel(LoraWeightArgs a, WeightWork w) {
  __shared__ __attribute__((aligned(16))) union Lds {
    WeightLds<weight_run(kR16, kDx)> x;
    WeightLds<weight_run(kR16, kDy)> y;
  } lds;
  int64_t b = block_id();
  if (b < w.slots * w.tiles[0]) {
    weight_tile<kDx, kR16>(a, a.f[0], w.chunk, b / w.tiles[0], b % w.tiles[0], w.part[0], lds.x);
    return;
  }
  b -= w.slots * w.tiles[0];
  if (w.tiles[1] == 0) return;
  weight_tile<kDy, kR16>(a, a.f[1], w.chunk, b / w.tiles[1], b % w.tiles[1], w.part[1], lds.y);
}

// The sums of an adapter's slots, if it has several.
constexpr int kSumRun = 4;
__global__ __launch_bounds__(kThreads) void lora_weight_sum_kernel(LoraWeightArgs a, WeightWork w, int64_t spans0,
                                                                   int64_t spans) {
  __shared__ Segments segments;
  const int64_t g = block_id() / spans;
  int64_t span = block_id() - g * spans;
  if (g >= a.seg.n_adapters) return;
  const int which = span < spans0 ? 0 : 1;
  if (which) span -= spans0;
  const LoraFactor f = a.f[which];
  count_rows(a.seg, a.rows, segments);
  Slot s;
  if (!find_slot<true>(segments.cnt, (int)a.seg.n_adapters, (int)w.chunk, g, s) || s.slots < 2) return;
  const int64_t all = a.rank * f.cols, e = (span * kThreads + threadIdx.x) * kSumRun, n = all - e;
  if (n <= 0) return;
  const float* p = w.part[which] + s.part * all + e;
  float v[kSumRun] = {}, t[kSumRun];
#pragma unroll 4
  for (int k = 0; k < s.slots; ++k) {
    load_run<kSumRun>(p + k * all, n, t);
#pragma unroll
    for (int i = 0; i < kSumRun; ++i) v[i] += t[i];
  }
  finish<kSumRun>(a, f, a.scale ? a.scale[g] : 1.0f, g * all + e, n, v);
}

template <typename F>
hipError_t by_type(int dtype, F&& f) {
  return dtype == 1 ? f(uint16_t{}) : f(float{});
}

}  // namespace

namespace {

// How the work is split, from sizes alone (the types change the tile, so that the
// same shares may be of another length).
struct LoraPlan {
  bool rows;   // the row kernels
  int splits;  // workgroups along the contraction
};
constexpr int64_t kFar = int64_t(1) << 21;  // elements of a row with which a tile's byte offsets stay below 2^31
LoraPlan lora_plan(int64_t rows, int64_t segments, int64_t c_x, int64_t c_y, int64_t rank) {
  // The row kernels read a row's adapter for every row; the tile kernels take some 11 to
  // 18 us for any few rows, and go through a tile's adapters one by one.  bf16, row and
  // tile kernels in us, one segment:
  //   rank 16: 1024 -> 1024   64 rows 7.1 and 10.9, 256 rows 8.5 and 11.1, 512 rows 11.7 and 11.2
  //            4096 -> 12288  64 rows 9.9 and 12.8, 128 rows 14.5 and 14.1, 256 rows 21 and 16
  //            17408 -> 5120  64 rows 11.2 and 16.8, 256 rows 19.8 and 18.7, 512 rows 33 and 21
  //   rank 64: 4096 -> 12288  64 rows 14.7 and 17.3, 128 rows 23.5 and 18.1
  // and in segments of four rows, 4096 -> 12288, rank 16: 256 rows of 8 adapters 21.5 and
  // 25, of 64 adapters 22 and 30, 512 rows 44 and 37, 1024 rows 86 and 57.  The bound does
  // not know widths, and segments of four rows take the row kernels at any number of rows.
  LoraPlan p{rows * ((rank + 15) / 16) <= 256 || rows <= 4 * segments || c_y < 8 || c_x >= kFar || c_y >= kFar, 1};
  if (p.rows) {  // two pieces of 512 elements a wave while the card is not full
    const int64_t units = rows * ((rank + kRowRanks - 1) / kRowRanks), most = (c_x + 4095) / 4096;
    const int64_t splits = units > 0 ? 512 / units : 1;
    p.splits = (int)(splits < 1 ? 1 : splits < most ? splits : most < 1 ? 1 : most);
    if (p.splits > 16) p.splits = 16;
    return p;
  }
  const int64_t tiles = (rows + 31) / 32, steps = (c_x + 31) / 32;
  int64_t splits = (512 + tiles - 1) / tiles;  // some two workgroups a CU
  const int64_t most = steps / 16;             // and 512 elements each at least
  splits = splits < most ? splits : most;
  p.splits = splits < 1 ? 1 : splits > 16 ? 16 : (int)splits;
  return p;
}

template <typename F>
hipError_t by_rank(int64_t rank, F&& f) {
  const int64_t g = (rank + 15) / 16;
  if (g <= 1) return f(std::integral_constant<int, 1>{});
  if (g <= 2) return f(std::integral_constant<int, 2>{});
  if (g <= 4) return f(std::integral_constant<int, 4>{});
  if (g <= 8) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

hipError_t launch_rows(const LoraArgs& a, int splits, float* part, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.rank > 0) {
    const int64_t groups = (a.rank + kRowRanks - 1) / kRowRanks, span = ((a.c_x + 511) / 512 + splits - 1) / splits * 512;
    e = by_type(a.x_dtype, [&](auto x) {
      return by_type(a.w_dtype, [&](auto w) {
        lora_row_in_kernel<decltype(x), decltype(w)>
            <<<grid_of(a.rows * groups * splits), dim3(kThreads), 0, stream>>>(a, groups, splits, span, part);
        return hipGetLastError();
      });
    });
    if (e != hipSuccess) return e;
  }
  const int64_t spans = a.c_y > 512 ? (a.c_y + 511) / 512 : 1;  // (without outputs: for s)
  return by_type(a.w_dtype, [&](auto w) {
    return by_type(a.y_dtype, [&](auto y) {
      lora_row_out_kernel<decltype(w), decltype(y)>
          <<<grid_of(a.rows * spans), dim3(kThreads), 0, stream>>>(a, spans, part, splits);
      return hipGetLastError();
    });
  });
}

hipError_t launch_tiles(const LoraArgs& a, int splits, float* part, hipStream_t stream) {
  const hipError_t e = by_type(a.x_dtype, [&](auto x) {
    return by_type(a.w_dtype, [&](auto w) {
      return by_rank(a.rank, [&](auto r) {
        using TX = decltype(x);
        using TW = decltype(w);
        const dim3 grid = grid_of((a.rows + kInRows - 1) / kInRows * splits);
        if constexpr (sizeof(TX) == 2 && sizeof(TW) == 2) {
          static_assert(LineShape<r>::kRows == kInRows);
          lora_line_in_kernel<r><<<grid, dim3(64 * LineShape<r>::kWaves), 0, stream>>>(a, splits, part);
        } else {
          const int64_t waves = (int64_t)kInWaves * splits, k_wave = ((a.c_x + 31) / 32 + waves - 1) / waves * 32;
          lora_tile_in_kernel<TX, TW, r><<<grid, dim3(64 * kInWaves), 0, stream>>>(a, splits, k_wave, part);
        }
        return hipGetLastError();
      });
    });
  });
  if (e != hipSuccess) return e;
  return by_type(a.w_dtype, [&](auto w) {
    return by_type(a.y_dtype, [&](auto y) {
      return by_rank(a.rank, [&](auto r) {
        using TW = decltype(w);
        using TY = decltype(y);
        constexpr int kOut = out_run<TW, r>, kPlanes = out_planes<TW>;
        const int64_t col_tiles = (a.c_y + 64 * kOut - 1) / (64 * kOut);
        // bytes of a row in LDS: below 26 KiB for 16 rows of any rank
        constexpr size_t kRowBytes = kPlanes ? kPlanes * (16 * r + 8) * 2 : (16 * r + 4) * 4;
        int row_tile = kOutRows;
        while (row_tile > 16 &&
               ((a.rows + row_tile - 1) / row_tile * col_tiles < 512 || row_tile * kRowBytes > 56 * 1024))
          row_tile /= 2;
        const size_t lds = row_tile * kRowBytes;
        lora_tile_out_kernel<TW, TY, r><<<grid_of((a.rows + row_tile - 1) / row_tile * col_tiles), dim3(kThreads), lds,
                                          stream>>>(a, part, splits, row_tile, col_tiles);
        return hipGetLastError();
      });
    });
  });
}

// Whether one launch does it: for many rows, unless most of the work is the way
// out (8192 rows, rank 16, 4096 -> 4096: 47 us, two launches 59; 12288 -> 4096: 73
// and 86; 4096 -> 12288: 107 and 101; 32768 rows, 2048 -> 1024: 63 and 71; larger
// ranks leave room for one workgroup a CU, 32768 rows of rank 32: 88 and 75).  At the
// bounds: 2048 rows, 4096 -> 4096 22 and 24 us, 1024 rows 17 and 17, but 2048 -> 1024 is
// 9 and 13 at 1024 rows too; with twice as many columns out, 4096 -> 8192, 8192 rows take
// 75 and 77, 2048 rows 36 and 33, and 2048 -> 4096 39 and 53 at 8192, 18 and 19 at 2048.
bool both_ways(const LoraArgs& a) {
  return a.x_dtype == 1 && a.w_dtype == 1 && a.rank <= 16 && a.rows >= 2048 && a.c_y <= 2 * a.c_x;
}

hipError_t launch_both(const LoraArgs& a, hipStream_t stream) {
  return by_type(a.y_dtype, [&](auto y) {
    lora_both_kernel<decltype(y)><<<grid_of((a.rows + 15) / 16), dim3(64 * kBothWaves), 0, stream>>>(a);
    return hipGetLastError();
  });
}

}  // namespace

size_t lora_ws_bytes(int64_t rows, int64_t segments, int64_t c_x, int64_t c_y, int64_t rank) {
  return (size_t)lora_plan(rows, segments, c_x, c_y, rank).splits * (size_t)rows * (size_t)rank * sizeof(float);
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t stream) {
  const LoraPlan p = lora_plan(a.rows, a.seg.n, a.c_x, a.c_y, a.rank);
  float* ws = static_cast<float*>(a.ws);
  if (p.rows || a.rank == 0 || a.ld_x >= kFar || a.ld_base >= kFar || a.ld_y >= kFar) {
    const int splits = p.rows ? p.splits : 1;
    return launch_rows(a, splits, splits == 1 && a.s ? a.s : ws, stream);
  }
  if (both_ways(a)) return launch_both(a, stream);
  int splits = p.splits;
  if (a.x_dtype == 1 && a.w_dtype == 1) {  // workgroups of eight waves, two a CU or one
    const int64_t tiles = (a.rows + kInRows - 1) / kInRows, most = ((a.rank <= 32 ? 512 : 256) + tiles - 1) / tiles;
    splits = splits < most ? splits : (int)most;
  }
  return launch_tiles(a, splits, splits == 1 && a.s ? a.s : ws, stream);
}

namespace {

int rank_groups(int64_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : rank <= 128 ? 8 : 16; }

// Rows of a slot: 256 to 2048, so that some 512 workgroups have work.
int64_t weight_chunk(int64_t rows, int64_t rank, int64_t c_in, int64_t c_out) {
  const int64_t tile = 16 * weight_run(rank_groups(rank), 1), tiles = (c_in + tile - 1) / tile + (c_out + tile - 1) / tile;
  int64_t chunk = kMostChunk;
  while (chunk > 256 && (rows + chunk - 1) / chunk * tiles < 512) chunk /= 2;
  return chunk;
}
// Parts: the slots of adapters that have several, at most two for every chunk of rows (no row
// is counted twice, and k full chunks and a rest are k + 1 <= 2 k slots).
int64_t weight_parts(int64_t rows, int64_t chunk) { return rows > chunk ? 2 * (rows / chunk) : 0; }

template <int kDx, int kDy>
hipError_t launch_weights(const LoraWeightArgs& a, WeightWork w, hipStream_t stream) {
  return by_rank(a.rank, [&](auto r) {
    constexpr int kX = 16 * weight_run(r, kDx), kY = 16 * weight_run(r, kDy);
    w.tiles[0] = a.f[0].out ? (a.f[0].cols + kX - 1) / kX : 0;
    w.tiles[1] = a.f[1].out ? (a.f[1].cols + kY - 1) / kY : 0;
    const int64_t blocks = w.slots * (w.tiles[0] + w.tiles[1]);
    if (blocks == 0) return hipSuccess;
    lora_weight_kernel<kDx, kDy, r><<<grid_of(blocks), dim3(kThreads), 0, stream>>>(a, w);
    return hipGetLastError();
  });
}

}  // namespace

size_t lora_weight_ws_bytes(int64_t rows, int64_t segments, int64_t n_adapters, int64_t rank, int64_t c_in,
                            int64_t c_out) {
  (void)segments;
  (void)n_adapters;
  return (size_t)weight_parts(rows, weight_chunk(rows, rank, c_in, c_out)) * (size_t)rank * (size_t)(c_in + c_out) *
         sizeof(float);
}

hipError_t launch_lora_weight_grad(const LoraWeightArgs& a, hipStream_t stream) {
  WeightWork w{};
  w.chunk = weight_chunk(a.rows, a.rank, a.f[0].cols, a.f[1].cols);
  w.slots = a.seg.n_adapters + a.rows / w.chunk;
  const int64_t parts = weight_parts(a.rows, w.chunk);
  w.part[0] = static_cast<float*>(a.ws);
  w.part[1] = w.part[0] + parts * a.rank * a.f[0].cols;
  const int dx = a.f[0].dtype, dy = a.f[1].dtype;
  hipError_t e;
  if (dx == dy) {
    e = dx == 0 ? launch_weights<0, 0>(a, w, stream) : launch_weights<1, 1>(a, w, stream);
  } else if (dx == 2 && dy == 1) {
    e = launch_weights<2, 1>(a, w, stream);
  } else {  // one after the other
    LoraWeightArgs x = a, y = a;
    x.f[1].out = y.f[0].out = nullptr;
    e = dx == 0 ? launch_weights<0, 0>(x, w, stream) : dx == 1 ? launch_weights<1, 1>(x, w, stream) : launch_weights<2, 1>(x, w, stream);
    if (e != hipSuccess) return e;
    e = dy == 0 ? launch_weights<0, 0>(y, w, stream) : launch_weights<1, 1>(y, w, stream);
  }
  if (e != hipSuccess || parts == 0) return e;
  const auto spans_of = [&](const LoraFactor& f) { return f.out ? (a.rank * f.cols + kThreads * kSumRun - 1) / (kThreads * kSumRun) : 0; };
  const int64_t spans0 = spans_of(a.f[0]), spans = spans0 + spans_of(a.f[1]);
  if (spans == 0) return e;
  lora_weight_sum_kernel<<<grid_of(a.seg.n_adapters * spans), dim3(kThreads), 0, stream>>>(a, w, spans0, spans);
  return hipGetLastError();
}

}  // namespace lh
