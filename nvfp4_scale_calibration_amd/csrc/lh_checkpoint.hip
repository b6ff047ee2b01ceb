// lh_checkpoint.hip - activations kept in 8 bits for a backward pass, and back.
//
// 32 values of a row share a power of two 2^e, the smallest with e >= -127 and
// no value beyond 448 2^e (448 is E4M3's largest number), and are rounded to
// E4M3 after an exact division by it.  With amax = 1.m 2^k, e = k - 8 where 1.m
// <= 1.75 and k - 7 above: one integer sum on amax's bits carries into the
// exponent exactly where the mantissa passes 0x600000, so E8M0's byte is
// max(0, ((bits + 0x1fffff) >> 23) - 8).
//
// HBM-bound: a lane moves 16 values, two lanes share a block and exchange its
// maximum once; rows of any length and alignment.  16384 x 17408 bf16: 147 us
// either way, 5.9 TB/s (2 bytes one way for 1 the other; a copy, 1 for 1, reaches
// 5.2, a fill 6.9).
#include "lh_internal.h"
#include "lh_rows.h"

namespace lh {
namespace {

constexpr int kPer = 16;     // values a lane
constexpr int kShared = 32;  // values that share a power of two

// 16 values of a row from p on, the first n of them inside it (others zero).
__device__ __forceinline__ void load16(const uint16_t* p, int n, float (&v)[kPer]) {
  uint32_t w[8] = {};
  if (n >= kPer) {
    __builtin_memcpy(w, p, 32);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load16(const float* p, int n, float (&v)[kPer]) {
  if (n >= kPer) {
    __builtin_memcpy(v, p, 64);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
}
__device__ __forceinline__ void store16(uint16_t* p, int n, const float (&v)[kPer]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  if (n >= kPer) {
    __builtin_memcpy(p, w, 32);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store16(float* p, int n, const float (&v)[kPer]) {
  if (n >= kPer) {
    __builtin_memcpy(p, v, 64);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < n) p[i] = v[i];
  }
}

// A wave takes 64 * 16 values of a row: its row and this lane's first column.
__device__ __forceinline__ bool wave_place(int64_t rows, int64_t spans, int64_t& row, int64_t& col) {
  const uint32_t w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t unit = block_id() * (kThreads / 64) + w;
  row = unit / spans;
  col = (unit - row * spans) * (64 * kPer) + (threadIdx.x & 63) * kPer;
  return row < rows;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void checkpoint_pack_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                                   int64_t ld, int64_t spans,
                                                                   uint8_t* __restrict__ values,
                                                                   uint8_t* __restrict__ scales) {
  int64_t row, col;
  if (!wave_place(rows, spans, row, col)) return;
  const int n = (int)min((int64_t)kPer, cols - col);  // <= 0: a lane past the row, which takes part in the exchange
  float v[kPer];
  load16(x + row * ld + min(col, cols), n, v);
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint32_t b = __float_as_uint(v[i]) & 0x7fffffffu;
    const bool finite = b < 0x7f800000u;
    most = max(most, finite ? b : 0u);
    if (!finite) v[i] = __uint_as_float(0x7fc00000u);  // E4M3FN has no infinity
  }
  most = max(most, (uint32_t)__shfl_xor((int)most, 1));
  const int code = max(0, (int)((most + 0x1fffffu) >> 23) - 8);
  if (n <= 0) return;
  const float down = __uint_as_float((uint32_t)(254 - code) << 23);  // 2^-e
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * down, v[4 * i + 1] * down, 0, false);
    w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * down, v[4 * i + 3] * down, p, true);
  }
  uint8_t* d = values + row * cols + col;
  if (n >= kPer) {
    __builtin_memcpy(d, w, 16);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < n) d[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
  if ((threadIdx.x & 1) == 0) scales[row * ((cols + kShared - 1) / kShared) + col / kShared] = (uint8_t)code;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void checkpoint_unpack_kernel(const uint8_t* __restrict__ values,
                                                                     const uint8_t* __restrict__ scales, int64_t rows,
                                                                     int64_t cols, int64_t spans, T* __restrict__ x,
                                                                     int64_t ld) {
  int64_t row, col;
  if (!wave_place(rows, spans, row, col) || col >= cols) return;
  const int n = (int)min((int64_t)kPer, cols - col);
  const uint8_t* p = values + row * cols + col;
  uint32_t w[4] = {};
  if (n >= kPer) {
    __builtin_memcpy(w, p, 16);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < n) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  }
  const float up = e8m0_to_f32(scales[row * ((cols + kShared - 1) / kShared) + col / kShared]);
  float v[kPer];
  static_for<4>([&](auto i) {
    v[4 * i] = e4m3_to_f32<0>(w[i]) * up;
    v[4 * i + 1] = e4m3_to_f32<1>(w[i]) * up;
    v[4 * i + 2] = e4m3_to_f32<2>(w[i]) * up;
    v[4 * i + 3] = e4m3_to_f32<3>(w[i]) * up;
  });
  store16(x + row * ld + col, n, v);
}

dim3 span_grid(int64_t rows, int64_t cols, int64_t& spans) {
  spans = (cols + 64 * kPer - 1) / (64 * kPer);
  return grid_of((rows * spans + kThreads / 64 - 1) / (kThreads / 64));
}

template <typename T>
hipError_t pack_typed(const CheckpointArgs& a, hipStream_t stream) {
  int64_t spans;
  const dim3 grid = span_grid(a.rows, a.cols, spans);
  checkpoint_pack_kernel<T><<<grid, dim3(kThreads), 0, stream>>>(static_cast<const T*>(a.x), a.rows, a.cols, a.ld,
                                                                 spans, a.values, a.scales);
  return hipGetLastError();
}
template <typename T>
hipError_t unpack_typed(const CheckpointArgs& a, hipStream_t stream) {
  int64_t spans;
  const dim3 grid = span_grid(a.rows, a.cols, spans);
  checkpoint_unpack_kernel<T><<<grid, dim3(kThreads), 0, stream>>>(a.values_in, a.scales_in, a.rows, a.cols, spans,
                                                                   static_cast<T*>(a.out), a.ld);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_checkpoint_pack(const CheckpointArgs& a, hipStream_t stream) {
  return a.dtype == 1 ? pack_typed<uint16_t>(a, stream) : pack_typed<float>(a, stream);
}
hipError_t launch_checkpoint_unpack(const CheckpointArgs& a, hipStream_t stream) {
  return a.dtype == 1 ? unpack_typed<uint16_t>(a, stream) : unpack_typed<float>(a, stream);
}

}  // namespace lh
