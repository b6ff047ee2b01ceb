// lh_quant.hip - NVFP4 fake-quant / packing with chosen block scales, and
// the per-group global amax.
//
// "Local-Hessian weight-scale guide" (xxmr.cn/news/266017):
//   "What is Local-Hessian": NVFP4 = E2M1 elements, one FP8 E4M3 scale per 16
//     weights, an FP32 per-tensor scale on top; the block scale maps the block
//     into [-6, 6]; max scaling takes the block's largest |w|.
//   "Algorithm principle": Q(W, s) = Cast(W / s) * s; the kernel receives the
//     global FP32 amax; candidate scales are bit-consistent with fake-quant.
// All kernels here are HBM-bound streaming passes.
#include <math.h>

#include "lh_internal.h"
#include "lh_rows.h"

namespace lh {
namespace {

template <typename T, bool kVec>
__device__ __forceinline__ void load16(const T* p, float (&w)[16]) {
  if constexpr (sizeof(T) == 2) {
    if (kVec) {
      const uint4 u0 = reinterpret_cast<const uint4*>(p)[0];
      const uint4 u1 = reinterpret_cast<const uint4*>(p)[1];
      const uint32_t v[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[2 * i] = __uint_as_float(v[i] << 16);
        w[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = bf16_bits_to_f32(p[i]);
    }
  } else {
    if (kVec) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 f = reinterpret_cast<const float4*>(p)[q];
        w[4 * q] = f.x;
        w[4 * q + 1] = f.y;
        w[4 * q + 2] = f.z;
        w[4 * q + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = p[i];
    }
  }
}

// One thread per 16-weight block.  Outputs are dense and each optional; the
// cast is nvfp4_cast_block, which the fused sweep uses too.  s == 0 (amax 0)
// gives x = 0 for every weight.  The workgroup's fp32 Q (256 blocks, 64
// contiguous bytes each) leaves through LDS, so that every store instruction
// writes 1 KiB of consecutive bytes: written from each thread, a wave's store
// put 16 of every 64 bytes over 4 KiB.  The nibbles and codes are
// consecutive per wave as they are.  In LDS the four 16-byte quarters of
// block i sit in the order rotated by i/2, so neither the writes (64-byte
// stride) nor the reads (16-byte stride) meet a bank twice in 8 lanes.
template <typename T, bool kVec>
__global__ __launch_bounds__(kThreads) void fake_quant_kernel(const T* __restrict__ wt, int64_t c_out,
                                                              int64_t ld_w, int64_t gstride_w, int64_t nb,
                                                              int64_t total, const uint8_t* __restrict__ idx,
                                                              const float* __restrict__ amax,
                                                              float* __restrict__ wq,
                                                              uint8_t* __restrict__ packed,
                                                              uint8_t* __restrict__ codes,
                                                              float* __restrict__ gscale, int64_t n_groups) {
  __shared__ float4 stage[kThreads * 4];
  const int tid = threadIdx.x;
  const int64_t f0 = (int64_t)blockIdx.x * kThreads;
  const int64_t f = f0 + tid;
  if (gscale && f < n_groups) gscale[f] = amax[f] / kAmaxDivisor;  // S_g, written once per group
  if (f < total) {
    const int64_t b = f % nb;
    const int64_t rg = f / nb;  // grp * c_out + row
    const int64_t grp = rg / c_out, row = rg - grp * c_out;
    const int k = idx[f];
    const float Sg = amax[grp] / kAmaxDivisor;
    const float s = e4m3_candidate(k) * Sg;
    float w[16];
    load16<T, kVec>(wt + grp * gstride_w + row * ld_w + 16 * b, w);
    uint32_t pk[2];
    nvfp4_cast_block(w, s, pk);
    nvfp4_emit_at(pk, s, k, f, nullptr, packed, codes);  // block f = rg * nb + b: nibbles and code
    if (wq) {
      float q[16];
      nvfp4_decode_block(pk, s, q);
#pragma unroll
      for (int qd = 0; qd < 4; ++qd)
        stage[4 * tid + ((qd + (tid >> 1)) & 3)] = make_float4(q[4 * qd], q[4 * qd + 1], q[4 * qd + 2], q[4 * qd + 3]);
    }
  }
  if (wq == nullptr) return;  // the same for every thread
  __syncthreads();
  const int64_t live = total - f0 < kThreads ? total - f0 : kThreads;  // this workgroup's blocks
  float4* dst = reinterpret_cast<float4*>(wq + 16 * f0);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = tid + kThreads * r;  // 16-byte piece i of the workgroup's Q
    const int blk = i >> 2;
    if (blk < live) dst[i] = stage[4 * blk + (((i & 3) + (blk >> 1)) & 3)];
  }
}

__global__ void global_scale_kernel(const float* __restrict__ amax, float* __restrict__ out, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) out[i] = amax[i] / kAmaxDivisor;
}

template <typename T, bool kVec>
hipError_t launch_fq_typed(const FakeQuantArgs& a, hipStream_t stream) {
  const int64_t nb = a.c_in / 16;
  const int64_t total = a.n_groups * a.c_out * nb;
  if (total > 0 && (a.wq || a.packed || a.codes)) {
    // threads f < n_groups also write S_g, so the grid covers both
    const int64_t n = total > a.n_groups ? total : a.n_groups;
    const int64_t grid = (n + kThreads - 1) / kThreads;
    fake_quant_kernel<T, kVec><<<dim3((unsigned)grid), dim3(kThreads), 0, stream>>>(
        static_cast<const T*>(a.w), a.c_out, a.ld_w, a.gstride_w, nb, total, a.idx, a.amax, a.wq, a.packed,
        a.codes, a.gscale, a.n_groups);
    return hipGetLastError();
  }
  if (a.gscale && a.n_groups > 0) {
    global_scale_kernel<<<dim3((unsigned)((a.n_groups + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream>>>(
        a.amax, a.gscale, a.n_groups);
    return hipGetLastError();
  }
  return hipSuccess;
}

// ---------------------------------------------------------------------------
// Activations to NVFP4 in one pass: per 16-value block the max rule's scale
// t = fl32(fl32(a / 6) / S_g) as the nearest positive E4M3 value c, then the
// cast of fake_quant_kernel with s = fl32(c S_g), bit for bit what
// lh_select_scales (max) followed by lh_fake_quant_nvfp4 writes.  The values
// leave as r c, in units of S_g, which bf16 and fp32 both hold exactly.
// A lane takes 16 bytes (8 bf16 or 4 fp32 values), so two or four
// neighbouring lanes share a block and find its maximum by xor shuffles;
// every load and store instruction covers consecutive bytes of the wave, and
// a thread has kQVecs of them in flight.
//
// IEEE divisions (some ten operations each) would take most of the vector
// unit's time, so quotients are formed with the reciprocal first, within
// 2^-21 of the exact one, and rounded to the grid a little above and a little
// below (2^-20): where both land on the same point, so does the exact
// quotient, and only where they differ is the division done.  Measured: 16384
// x 17408 bf16 to values and codes 198 us, 5.8 TB/s (with divisions alone 290);
// 4096 x 4096 fp32 23 us, 6.0 TB/s.
// ---------------------------------------------------------------------------
constexpr int kQVecs = 4;
constexpr float kAbove = 1.0f + 0x1p-20f, kBelow = 1.0f - 0x1p-20f;

// E2M1 nibbles of the kE quotients q, low nibble first.
template <int kE>
__device__ __forceinline__ uint32_t nibbles_of(const float (&q)[kE]) {
  uint32_t pk = 0u;
  pk = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(pk, q[0], q[1], 1.0f, 0);
  pk = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(pk, q[2], q[3], 1.0f, 1);
  if constexpr (kE == 8) {
    pk = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(pk, q[4], q[5], 1.0f, 2);
    pk = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(pk, q[6], q[7], 1.0f, 3);
  }
  return pk;
}

// The code of t = fl32(fl32(m / 6) / Sg): the nearest positive E4M3 value
// (ties to even), clamped below the conversion's overflow, never the zero
// code.  inv: about 1 / (6 Sg), or 0 where that is not a normal number.
__device__ __forceinline__ uint32_t max_rule_code(float m, float Sg, float inv) {
  if (!(Sg > 0.0f)) return 1u;
  const float y = fminf(m * inv, 448.0f);
  uint32_t two = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fminf(y * kAbove, 448.0f), y * kBelow, 0, false);
  if (inv == 0.0f || ((two ^ (two >> 8)) & 0xffu)) {
    const float t = fminf((m / 6.0f) / Sg, 448.0f);
    two = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t, t, 0, false);
  }
  const uint32_t code = two & 0x7fu;
  return code > 0u ? code : 1u;
}

template <typename T, typename TV>
__global__ __launch_bounds__(kThreads) void quantize_kernel(QuantizeArgs a, int64_t rows, int64_t cols, int64_t ld) {
  constexpr int kE = 16 / sizeof(T);   // values per lane
  constexpr int kP = kBlock / kE;      // lanes per block
  const int64_t vecs = cols / kE;      // lanes' shares per row; a multiple of kP
  const T* x = static_cast<const T*>(a.x);
  TV* values = static_cast<TV*>(a.values);
  for (int64_t g = blockIdx.z; g < a.n_groups; g += gridDim.z) {
    const float Sg = a.amax[g] / kAmaxDivisor;
    const float six = 6.0f * Sg;
    const float inv6 = six > 0x1p-100f && six < 0x1p100f ? __builtin_amdgcn_rcpf(six) : 0.0f;
    if (a.gscale && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) a.gscale[g] = Sg;
    for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
      const T* row = x + g * a.gstride + r * ld;
      for (int64_t v0 = (int64_t)blockIdx.x * (kThreads * kQVecs) + threadIdx.x; v0 < vecs;
           v0 += (int64_t)gridDim.x * (kThreads * kQVecs)) {
        uint4 raw[kQVecs];
#pragma unroll
        for (int j = 0; j < kQVecs; ++j)
          if (v0 + j * kThreads < vecs) raw[j] = load_u128(row + (v0 + j * kThreads) * kE);
#pragma unroll
        for (int j = 0; j < kQVecs; ++j) {
          const int64_t v = v0 + j * kThreads;
          if (v >= vecs) break;  // the lanes of a block leave together
          const uint32_t in[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
          float w[kE];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (kE == 8) {
              w[2 * i] = __uint_as_float(in[i] << 16);
              w[2 * i + 1] = __uint_as_float(in[i] & 0xffff0000u);
            } else {
              w[i] = __uint_as_float(in[i]);
            }
          }
          float m = 0.0f;
#pragma unroll
          for (int i = 0; i < kE; ++i) m = fmaxf(m, fabsf(w[i]));
#pragma unroll
          for (int off = 1; off < kP; off <<= 1) m = fmaxf(m, __shfl_xor(m, off));
          const uint32_t code = max_rule_code(m, Sg, inv6);
          const float c = e4m3_to_f32<0>(code);
          const float s = c * Sg;
          const bool near = s > 0x1p-100f && s < 0x1p100f;
          const float inv = __builtin_amdgcn_rcpf(s);
          float above[kE], below[kE];
#pragma unroll
          for (int i = 0; i < kE; ++i) {
            const float y = w[i] * inv;
            above[i] = y * kAbove;
            below[i] = y * kBelow;
          }
          uint32_t pk = nibbles_of(above);
          if (!near || pk != nibbles_of(below)) {
            float q[kE];
#pragma unroll
            for (int i = 0; i < kE; ++i) q[i] = (s == 0.0f) ? 0.0f : w[i] / s;  // IEEE division
            pk = nibbles_of(q);
          }
          const uint32_t nz = (pk | (pk >> 1) | (pk >> 2)) & 0x11111111u;  // -0 is written as +0
          pk &= 0x77777777u | (nz << 3);
          const int64_t at = (g * rows + r) * vecs + v;  // dense outputs
          if (values) {
            float u[8];
            units8(pk, c, u);
            if constexpr (sizeof(TV) == 2 && kE == 8) {
              const uint32_t b[4] = {pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3]), pack_bf16(u[4], u[5]),
                                     pack_bf16(u[6], u[7])};
              __builtin_memcpy(values + at * kE, b, 16);
            } else if constexpr (sizeof(TV) == 2) {
              const uint32_t b[2] = {pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3])};
              __builtin_memcpy(values + at * kE, b, 8);
            } else {
              __builtin_memcpy(values + at * kE, u, 4 * kE);
            }
          }
          if (a.packed) {
            if constexpr (kE == 8) *reinterpret_cast<uint32_t*>(a.packed + 4 * at) = pk;
            else *reinterpret_cast<uint16_t*>(a.packed + 2 * at) = (uint16_t)pk;
          }
          if (a.codes && (v & (kP - 1)) == 0) a.codes[at / kP] = (uint8_t)code;
        }
      }
    }
  }
}

template <typename T, typename TV>
hipError_t launch_quantize_typed(const QuantizeArgs& a, hipStream_t stream) {
  int64_t rows = a.rows, cols = a.c_in;
  if (a.ld == a.c_in || rows == 1) {  // a group is one flat row
    cols *= rows;
    rows = 1;
  }
  const int64_t per = kThreads * kQVecs * (16 / (int64_t)sizeof(T));
  const int64_t gx = (cols + per - 1) / per;
  const dim3 grid((unsigned)(gx < 1 ? 1 : gx > (1 << 20) ? (1 << 20) : gx), (unsigned)(rows < 1 ? 1 : rows > 65535 ? 65535 : rows),
                  (unsigned)(a.n_groups > 65535 ? 65535 : a.n_groups));
  quantize_kernel<T, TV><<<grid, dim3(kThreads), 0, stream>>>(a, rows, cols, a.ld);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Global amax: |w| as fp32 bits is monotone in |w|, so the reduction is an
// unsigned max; each workgroup folds its rows, then one atomicMax per
// workgroup into the zero-initialised output (order-independent, exact).
// ---------------------------------------------------------------------------
__global__ void absmax_init_kernel(float* __restrict__ out, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < n) out[i] = 0.0f;
}

// Contiguous groups (ld == cols): the group is one flat array of n16 16-byte
// vectors; grid-stride loop with four loads in flight per thread.
// Otherwise rows are walked one by one (kFlat == false), vectorised when the
// row length and strides allow (kVec).
template <typename T, bool kVec, bool kFlat>
__global__ __launch_bounds__(kThreads) void absmax_kernel(const T* __restrict__ w, int64_t rows, int64_t cols,
                                                          int64_t ld, int64_t gstride, int64_t per_group,
                                                          float* __restrict__ out) {
  const int64_t grp = (int64_t)blockIdx.x / per_group;
  const int64_t chunk = (int64_t)blockIdx.x - grp * per_group;
  const T* base = w + grp * gstride;
  constexpr bool kBf16 = sizeof(T) == 2;
  uint32_t t;
  if (kFlat) {
    t = absmax_flat_share<kBf16>(reinterpret_cast<const uint4*>(base), rows * cols * (int64_t)sizeof(T) / 16, chunk,
                                 per_group);
  } else {
    __shared__ uint32_t part[kThreads / 64];
    uint32_t m = 0;
    constexpr int kV = 16 / sizeof(T);
    for (int64_t r = chunk; r < rows; r += per_group) {
      const T* rp = base + r * ld;
      if (kVec) {
        for (int64_t c = (int64_t)threadIdx.x * kV; c < cols; c += (int64_t)kThreads * kV)
          m = absbits_max(m, *reinterpret_cast<const uint4*>(rp + c), kBf16);
      } else {
        for (int64_t c = threadIdx.x; c < cols; c += kThreads) {
          uint32_t bits;
          if constexpr (kBf16) bits = (uint32_t)rp[c] << 16;
          else bits = __float_as_uint(rp[c]);
          m = max(m, bits & 0x7FFFFFFFu);
        }
      }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
    __syncthreads();
    t = part[0];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) t = max(t, part[i]);
  }
  if (threadIdx.x == 0) {
    // Atomics on one address serialise in L2; the stored value only grows, so
    // a workgroup whose maximum does not exceed what it reads (possibly a
    // stale, smaller value) has nothing to add.
    unsigned int* o = reinterpret_cast<unsigned int*>(out + grp);
    if (t > __atomic_load_n(o, __ATOMIC_RELAXED)) atomicMax(o, t);
  }
}

template <typename T, bool kVec, bool kFlat>
hipError_t launch_absmax_typed(const AbsmaxArgs& a, hipStream_t stream) {
  int64_t per_group;
  if (kFlat) {
    const int64_t n16 = a.rows * a.cols * (int64_t)sizeof(T) / 16;
    per_group = (1024 + a.n_groups - 1) / a.n_groups;              // ~4 workgroups per CU in total
    const int64_t need = (n16 + 4 * kThreads - 1) / (4 * kThreads);  // >= 4 vectors per thread
    if (per_group > need) per_group = need;
  } else {
    per_group = (2048 + a.n_groups - 1) / a.n_groups;
    if (per_group > a.rows) per_group = a.rows;
  }
  if (per_group < 1) per_group = 1;
  absmax_kernel<T, kVec, kFlat><<<dim3((unsigned)(per_group * a.n_groups)), dim3(kThreads), 0, stream>>>(
      static_cast<const T*>(a.w), a.rows, a.cols, a.ld, a.gstride, per_group, a.out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fake_quant(const FakeQuantArgs& a, hipStream_t stream) {
  const int64_t esz = a.dtype == 1 ? 2 : 4;
  const int64_t epv = 16 / esz;
  const bool aligned = (reinterpret_cast<uintptr_t>(a.w) % 16 == 0) && (a.ld_w % epv == 0) &&
                       (a.gstride_w % epv == 0);
  if (a.dtype == 1)
    return aligned ? launch_fq_typed<uint16_t, true>(a, stream) : launch_fq_typed<uint16_t, false>(a, stream);
  return aligned ? launch_fq_typed<float, true>(a, stream) : launch_fq_typed<float, false>(a, stream);
}

hipError_t launch_quantize(const QuantizeArgs& a, hipStream_t stream) {
  if (a.dtype == 1)
    return a.v_dtype == 1 ? launch_quantize_typed<uint16_t, uint16_t>(a, stream)
                          : launch_quantize_typed<uint16_t, float>(a, stream);
  return a.v_dtype == 1 ? launch_quantize_typed<float, uint16_t>(a, stream)
                        : launch_quantize_typed<float, float>(a, stream);
}

hipError_t launch_absmax(const AbsmaxArgs& a, hipStream_t stream) {
  if (a.n_groups == 0) return hipSuccess;
  absmax_init_kernel<<<dim3((unsigned)((a.n_groups + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream>>>(
      a.out, a.n_groups);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.rows == 0 || a.cols == 0) return e;
  const int64_t esz = a.dtype == 1 ? 2 : 4;
  const int64_t epv = 16 / esz;
  const bool aligned = (reinterpret_cast<uintptr_t>(a.w) % 16 == 0) && (a.ld % epv == 0) &&
                       (a.gstride % epv == 0) && (a.cols % epv == 0);
  const bool flat = aligned && (a.ld == a.cols || a.rows == 1);
  if (a.dtype == 1) {
    if (flat) return launch_absmax_typed<uint16_t, true, true>(a, stream);
    return aligned ? launch_absmax_typed<uint16_t, true, false>(a, stream)
                   : launch_absmax_typed<uint16_t, false, false>(a, stream);
  }
  if (flat) return launch_absmax_typed<float, true, true>(a, stream);
  return aligned ? launch_absmax_typed<float, true, false>(a, stream) : launch_absmax_typed<float, false, false>(a, stream);
}

}  // namespace lh
