// lh_rows.h - row access of any alignment and the exact conversions shared by
// the kernels that multiply, quantise and move rows (lh_linear.hip,
// lh_moe.hip, lh_quant.hip).
#pragma once

#include <utility>

#include "lh_device.h"

namespace lh {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// f(integral_constant 0), ..., f(integral_constant N - 1): a loop whose index
// is a constant for the front end, so that what it indexes is never memory.
template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// A grid of `blocks` > 0 workgroups, numbered by block_id().  A launch takes fewer
// than 2^32 threads along a dimension (what is more wraps around, without an
// error), so workgroups past 2^20 go on along y.  The last ones may lie past
// `blocks`.
inline dim3 grid_of(int64_t blocks) {
  const int64_t x = blocks < (1 << 20) ? blocks : 1 << 20;
  return dim3((unsigned)x, (unsigned)((blocks + x - 1) / x));
}
__device__ __forceinline__ int64_t block_id() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// A wave-uniform value into scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Sums over the wave of kN values (a power of two): lane l gets the sum of
// value l / (64 / kN).  Each of the first steps exchanges half of the values
// with the other half of the lanes, so 2 kN shuffles do instead of 6 kN.
template <int kN>
__device__ __forceinline__ float wave_sums(float (&v)[kN]) {
  const int lane = threadIdx.x & 63;
  static_for<6>([&](auto S) {
    constexpr int off = 32 >> S, live = kN >> S;  // values a lane still carries
    if constexpr (live > 1) {
      const bool upper = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < live / 2; ++i) {
        const float give = upper ? v[i] : v[i + live / 2], keep = upper ? v[i + live / 2] : v[i];
        v[i] = keep + __shfl_xor(give, off);
      }
    } else {
      v[0] += __shfl_xor(v[0], off);
    }
  });
  return v[0];
}

// 16 and 8 bytes from any address (global memory takes unaligned accesses;
// memcpy says so to the compiler, which emits one wide load).
__device__ __forceinline__ uint4 load_u128(const void* p) {
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ uint2 load_u64(const void* p) {
  uint2 v;
  __builtin_memcpy(&v, p, 8);
  return v;
}
__device__ __forceinline__ uint32_t load_u32(const void* p) {
  uint32_t v;
  __builtin_memcpy(&v, p, 4);
  return v;
}

// Round to nearest even, two at a time (v_cvt_pk_bf16_f32); a in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2_t v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint16_t f32_to_bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// E4M3 byte `i` of v as fp32 (v_cvt_f32_fp8: OCP E4M3FN on gfx950).
template <int i>
__device__ __forceinline__ float e4m3_to_f32(uint32_t v) {
  return __builtin_amdgcn_cvt_f32_fp8((int)v, i);
}

// Eight E2M1 nibbles (low nibble first) times c: exact, since r has 2
// significant bits and c 4.
__device__ __forceinline__ void units8(uint32_t pk, float c, float (&u)[8]) {
  const f32x2_t r0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(pk, 1.0f, 0);
  const f32x2_t r1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(pk, 1.0f, 1);
  const f32x2_t r2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(pk, 1.0f, 2);
  const f32x2_t r3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(pk, 1.0f, 3);
  u[0] = r0.x * c; u[1] = r0.y * c; u[2] = r1.x * c; u[3] = r1.y * c;
  u[4] = r2.x * c; u[5] = r2.y * c; u[6] = r3.x * c; u[7] = r3.y * c;
}

// The same as bf16, which holds r c (6 significant bits, 2^-10 .. 2688)
// exactly: one MFMA operand of eight consecutive weights.
__device__ __forceinline__ uint4 units8_bf16(uint32_t pk, float c) {
  float u[8];
  units8(pk, c, u);
  return make_uint4(pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]), pack_bf16(u[4], u[5]), pack_bf16(u[6], u[7]));
}

// x = h + m + l with three bf16 values, exactly (24 significant bits cut into
// 8 + 8 + 8; the remainders are exact differences, none for an infinity): bits
// of two values packed per plane, a in the low half.  Where |x| < 2^-110 the
// low bits reach below 2^-133, a subnormal bf16's last place, and are dropped.
__device__ __forceinline__ void split3(float a, float b, uint32_t (&p)[3]) {
  const uint32_t ha = __float_as_uint(a) & 0xffff0000u, hb = __float_as_uint(b) & 0xffff0000u;
  const float ra = isinf(a) ? 0.0f : a - __uint_as_float(ha), rb = isinf(b) ? 0.0f : b - __uint_as_float(hb);
  const uint32_t ma = __float_as_uint(ra) & 0xffff0000u, mb = __float_as_uint(rb) & 0xffff0000u;
  const float la = ra - __uint_as_float(ma), lb = rb - __uint_as_float(mb);
  p[0] = (ha >> 16) | hb;
  p[1] = (ma >> 16) | mb;
  p[2] = (__float_as_uint(la) >> 16) | (__float_as_uint(lb) & 0xffff0000u);
}

}  // namespace lh
