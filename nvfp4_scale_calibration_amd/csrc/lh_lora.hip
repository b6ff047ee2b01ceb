// lh_lora.hip - low-rank adapters beside a frozen projection, for many
// requests at once, and their gradients.
//
//   s[t][r] = sum_c x[t][c] in[g][r][c]            (the row into the rank)
//   y[t][o] = base[t][o] + scale[g] sum_r s[t][r] out[g][r][o]
// with g the adapter of t's segment.  Both factors are stored with the rank
// first, so the gradient to the input (dy for x, b for in, a for out) is the
// same two kernels.  The gradients to the factors are sums over an adapter's
// rows, out[g][r][c] = scale[g] sum_t p[t][r] x[t][c].
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

// Row t's adapter, -1 for none, -2 where t is in no segment.  All lanes of the
// wave ask for the same row.
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
__device__ __forceinline__ void store8(uint16_t* p, int64_t n, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  if (n >= 8) {
    __builtin_memcpy(p, w, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store8(float* p, int64_t n, const float (&v)[8]) {
  if (n >= 8) {
    __builtin_memcpy(p, v, 32);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}

// ---------------------------------------------------------------------------
// The row kernels: a wave per row and group of ranks, a thread per row and
// eight outputs.
// ---------------------------------------------------------------------------
constexpr int kRowRanks = 4;

template <typename TX, typename TW>
__global__ __launch_bounds__(64) void lora_row_in_kernel(LoraArgs a, int64_t groups, float* __restrict__ s) {
  const int64_t unit = block_id(), t = unit / groups, r0 = (unit - t * groups) * kRowRanks;
  if (t >= a.rows) return;
  const int lane = threadIdx.x & 63;
  const int64_t g = adapter_of_row(a.seg, t);
  if (g == -2) return;
  float acc[kRowRanks] = {};
  if (g >= 0) {
    const TX* x = static_cast<const TX*>(a.x) + t * a.ld_x;
    const TW* w = static_cast<const TW*>(a.in) + (g * a.rank + r0) * a.c_x;
    for (int64_t c = lane * 8; c < a.c_x; c += 512) {
      float xv[8];
      load8(x + c, a.c_x - c, xv);
#pragma unroll
      for (int r = 0; r < kRowRanks; ++r) {
        if (r0 + r >= a.rank) break;
        float wv[8];
        load8(w + r * a.c_x + c, a.c_x - c, wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[r] = __builtin_fmaf(xv[i], wv[i], acc[r]);
      }
    }
  }
  const float v = wave_sums(acc);
  const int r = lane / (64 / kRowRanks);
  if (lane % (64 / kRowRanks) == 0 && r0 + r < a.rank) s[t * a.rank + r0 + r] = v;
}

template <typename TW, typename TY>
__global__ __launch_bounds__(64) void lora_row_out_kernel(LoraArgs a, int64_t spans, const float* __restrict__ s) {
  const int64_t unit = block_id(), t = unit / spans;
  if (t >= a.rows) return;
  const int64_t g = adapter_of_row(a.seg, t);
  const int64_t c = (unit - t * spans) * 512 + threadIdx.x * 8;
  if (g == -2 || c >= a.c_y) return;
  const int64_t n = a.c_y - c;
  TY* y = static_cast<TY*>(a.y) + t * a.ld_y + c;
  float acc[8] = {}, v[8] = {};
  if (a.base) load8(static_cast<const TY*>(a.base) + t * a.ld_base + c, n, v);
  if (g >= 0) {
    const TW* w = static_cast<const TW*>(a.out) + g * a.rank * a.c_y + c;
    for (int64_t r = 0; r < a.rank; ++r) {
      float wv[8];
      load8(w + r * a.c_y, n, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(s[t * a.rank + r], wv[i], acc[i]);
    }
    const float scale = a.scale ? a.scale[g] : 1.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(scale, acc[i], v[i]);
  }
  store8(y, n, v);
}

// ---------------------------------------------------------------------------
// Gradients to the factors: a thread per column, eight ranks at a time.
// ---------------------------------------------------------------------------
constexpr int kGradRanks = 8;

template <int kDtype>
__device__ __forceinline__ float value_at(const LoraFactor& f, int64_t t, int64_t c) {
  if constexpr (kDtype == 0) return static_cast<const float*>(f.x)[t * f.ld + c];
  if constexpr (kDtype == 1) return bf16_bits_to_f32(static_cast<const uint16_t*>(f.x)[t * f.ld + c]);
  const uint32_t v = static_cast<const uint8_t*>(f.x)[t * f.cols + c];
  return e4m3_to_f32<0>(v) * e8m0_to_f32(f.x_scale[t * ((f.cols + 31) / 32) + c / 32]);
}

template <int kDtype, typename TO>
__global__ __launch_bounds__(kThreads) void lora_weight_kernel(LoraWeightArgs a, LoraFactor f, int64_t col_tiles,
                                                               int64_t rank_tiles) {
  const int64_t unit = block_id(), per = col_tiles * rank_tiles, g = unit / per, in = unit - g * per;
  if (g >= a.seg.n_adapters) return;
  const int64_t r0 = in / col_tiles * kGradRanks, c = in % col_tiles * kThreads + threadIdx.x;
  if (c >= f.cols) return;
  float acc[kGradRanks] = {};
  for (int64_t i = 0; i < a.seg.n; ++i) {
    if (adapter_of(a.seg, i) != g) continue;
    int64_t t0, t1;
    if (a.seg.offsets) {
      t0 = min(max(a.seg.offsets[i], (int64_t)0), a.rows);
      t1 = min(max(a.seg.offsets[i + 1], (int64_t)0), a.rows);
    } else {
      t0 = a.seg.n == 1 ? 0 : i;
      t1 = a.seg.n == 1 ? a.rows : i + 1;
    }
    for (int64_t t = t0; t < t1; ++t) {
      const float v = value_at<kDtype>(f, t, c);
#pragma unroll
      for (int r = 0; r < kGradRanks; ++r)
        if (r0 + r < a.rank) acc[r] = __builtin_fmaf(f.p[t * a.rank + r0 + r], v, acc[r]);
    }
  }
  const float scale = a.scale ? a.scale[g] : 1.0f;
  TO* out = static_cast<TO*>(f.out) + (g * a.rank + r0) * f.cols + c;
#pragma unroll
  for (int r = 0; r < kGradRanks; ++r) {
    if (r0 + r >= a.rank) break;
    float v = scale * acc[r];
    if (a.beta != 0.0f) v = __builtin_fmaf(a.beta, load_as_f32<TO>(out, r * f.cols), v);
    if constexpr (sizeof(TO) == 2) out[r * f.cols] = f32_to_bf16_bits(v);
    else out[r * f.cols] = v;
  }
}

template <typename F>
hipError_t by_type(int dtype, F&& f) {
  return dtype == 1 ? f(uint16_t{}) : f(float{});
}

}  // namespace

size_t lora_ws_bytes(int64_t rows, int64_t segments, int64_t c_x, int64_t c_y, int64_t rank) {
  (void)segments;
  (void)c_x;
  (void)c_y;
  return (size_t)rows * (size_t)rank * sizeof(float);
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t stream) {
  const bool adds = a.rank > 0;
  float* s = a.s ? a.s : static_cast<float*>(a.ws);
  hipError_t e = hipSuccess;
  if (adds) {
    const int64_t groups = (a.rank + kRowRanks - 1) / kRowRanks;
    e = by_type(a.x_dtype, [&](auto x) {
      return by_type(a.w_dtype, [&](auto w) {
        lora_row_in_kernel<decltype(x), decltype(w)><<<grid_of(a.rows * groups), dim3(64), 0, stream>>>(a, groups, s);
        return hipGetLastError();
      });
    });
    if (e != hipSuccess) return e;
  }
  if (a.c_y == 0) return e;
  const int64_t spans = (a.c_y + 511) / 512;
  return by_type(a.w_dtype, [&](auto w) {
    return by_type(a.y_dtype, [&](auto y) {
      lora_row_out_kernel<decltype(w), decltype(y)><<<grid_of(a.rows * spans), dim3(64), 0, stream>>>(a, spans, s);
      return hipGetLastError();
    });
  });
}

size_t lora_weight_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_lora_weight_grad(const LoraWeightArgs& a, hipStream_t stream) {
  for (const LoraFactor& f : a.f) {
    if (!f.out || f.cols == 0) continue;
    const int64_t cols = (f.cols + kThreads - 1) / kThreads, ranks = (a.rank + kGradRanks - 1) / kGradRanks;
    const dim3 grid = grid_of(a.seg.n_adapters * cols * ranks);
    const hipError_t e = by_type(a.out_dtype, [&](auto o) {
      using TO = decltype(o);
      if (f.dtype == 0) lora_weight_kernel<0, TO><<<grid, dim3(kThreads), 0, stream>>>(a, f, cols, ranks);
      else if (f.dtype == 1) lora_weight_kernel<1, TO><<<grid, dim3(kThreads), 0, stream>>>(a, f, cols, ranks);
      else lora_weight_kernel<2, TO><<<grid, dim3(kThreads), 0, stream>>>(a, f, cols, ranks);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace lh
