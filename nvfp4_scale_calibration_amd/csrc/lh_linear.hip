// lh_linear.hip - products with NVFP4 weights as the calibration leaves them
// (E2M1 nibbles, one E4M3 code per 16 weights, FP32 global scale), and their
// gradient to the input.
//
//   y[t][o]  = S_w [S_x] sum_c x[t][c] u[o][c],    u[o][c] = r[o][c] c[o][c/16]
//   dx[t][c] = S_w       sum_o dy[t][o] u[o][c]
//
// u is exact in bf16: r has 2 significant bits and the block scale 4, so
// their product has at most 6, between 2^-10 and 2688.  The products
// therefore run on bf16 MFMA with fp32 accumulation without any loss on the
// weights' side, and the global scale is one multiplication per output.
// (The matrix cores' own block scales are powers of two per 32 elements and
// cannot hold an E4M3 scale per 16.)  fp32 activations are cut into three
// bf16 values that add up to them exactly, so their products are exact too.
//
// MFMA orientation: operand A = weights (rows = outputs), operand B =
// activations (columns = tokens), so that a lane's accumulators are
// consecutive outputs of one token and leave in one store.
#include "lh_internal.h"
#include "lh_rows.h"

namespace lh {
namespace {

// Rows [row0, row1) of group g that tile `t` of the ragged rows covers, with
// kBT rows per tile and tiles counted group by group; false past the last
// tile.  Offsets are clamped into [0, n_rows]; a decreasing pair is an empty
// group.  Every wave computes it for itself (64 groups per step).
template <int kBT>
__device__ __forceinline__ bool ragged_tile(const int64_t* __restrict__ offsets, int64_t n_groups, int64_t n_rows,
                                            int64_t t, int64_t& g, int64_t& row0, int64_t& row1) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int64_t g0 = 0; g0 < n_groups; g0 += 64) {
    int64_t a = 0, b = 0;
    if (g0 + lane < n_groups) {
      a = min(max(offsets[g0 + lane], (int64_t)0), n_rows);
      b = min(max(offsets[g0 + lane + 1], (int64_t)0), n_rows);
    }
    const int64_t tiles = b > a ? (b - a + kBT - 1) / kBT : 0;
    int64_t incl = tiles;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t u = __shfl_up(incl, off);
      if (lane >= off) incl += u;
    }
    const unsigned long long hit = __ballot(before + incl > t);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int64_t first = before + __shfl(incl - tiles, l);
      g = g0 + l;
      row0 = __shfl(a, l) + (t - first) * kBT;
      row1 = min(row0 + kBT, __shfl(b, l));
      return true;
    }
    before += __shfl(incl, 63);
  }
  return false;
}

// Where one workgroup works: a tile of tokens of one group.
struct Place {
  int64_t g, row0, row1;   // rows of x and y relative to the group's first row (dense) or the buffer (ragged)
  const char* x;           // the group's x
  char* y;
};

template <int kBT>
__device__ __forceinline__ bool place_of(const LinearArgs& a, int64_t tile, Place& p) {
  const int64_t ex = a.x_dtype == 1 ? 2 : 4, ey = a.y_dtype == 1 ? 2 : 4;
  p.x = static_cast<const char*>(a.x);
  p.y = static_cast<char*>(a.y);
  if (a.ragged) return ragged_tile<kBT>(a.offsets, a.n_groups, a.rows, tile, p.g, p.row0, p.row1);
  const int64_t per = (a.rows + kBT - 1) / kBT;
  p.g = tile / per;
  if (p.g >= a.n_groups) return false;
  p.row0 = (tile - p.g * per) * kBT;
  p.row1 = min(p.row0 + kBT, a.rows);
  p.x += p.g * a.gstride_x * ex;
  p.y += p.g * a.gstride_y * ey;
  return true;
}

__device__ __forceinline__ float out_scale(const LinearArgs& a, int64_t g) {
  return a.x_scale ? a.gscale[g] * a.x_scale[g] : a.gscale[g];
}

// Four consecutive outputs of one token, the first n of them inside the row.
__device__ __forceinline__ void store4(float* p, int64_t n, const float (&v)[4]) {
  if (n >= 4) {
    __builtin_memcpy(p, v, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store4(uint16_t* p, int64_t n, const float (&v)[4]) {
  const uint32_t b[2] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  if (n >= 4) {
    __builtin_memcpy(p, b, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = (uint16_t)(b[i >> 1] >> (16 * (i & 1)));
  }
}

// ---------------------------------------------------------------------------
// The general kernel: 64 outputs x 64 tokens per workgroup, four waves of
// 32 x 32 quadrants (2 x 2 v_mfma_f32_16x16x32_bf16 tiles), K in steps of 64
// through LDS.  Any size, stride and alignment.
// ---------------------------------------------------------------------------
constexpr int kT = 64;           // outputs and tokens per tile
constexpr int kK = 64;           // contraction step
constexpr int kPitch = kK + 8;   // bf16 elements per LDS row

// 16 activations of a row from element k (past k_len: zero) into the LDS
// planes at element `at`.
template <int kPlanes>
__device__ __forceinline__ void stage_x(const char* row, int64_t k, int64_t k_len, bool live,
                                        uint16_t (*planes)[kT * kPitch], int at) {
  if constexpr (kPlanes == 1) {
    uint32_t v[8] = {};
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + k;
    if (live && k + 16 <= k_len) {
      __builtin_memcpy(v, p, 32);
    } else if (live) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (k + i < k_len) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    }
    uint4* d = reinterpret_cast<uint4*>(&planes[0][at]);
    d[0] = make_uint4(v[0], v[1], v[2], v[3]);
    d[1] = make_uint4(v[4], v[5], v[6], v[7]);
  } else {
    float f[16] = {};
    const float* p = reinterpret_cast<const float*>(row) + k;
    if (live && k + 16 <= k_len) {
      __builtin_memcpy(f, p, 64);
    } else if (live) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (k + i < k_len) f[i] = p[i];
    }
    uint32_t b[8][3];
#pragma unroll
    for (int i = 0; i < 8; ++i) split3(f[2 * i], f[2 * i + 1], b[i]);
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      uint4* d = reinterpret_cast<uint4*>(&planes[q][at]);
      d[0] = make_uint4(b[0][q], b[1][q], b[2][q], b[3][q]);
      d[1] = make_uint4(b[4][q], b[5][q], b[6][q], b[7][q]);
    }
  }
}

template <bool kGrad, typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void linear_tile_kernel(LinearArgs a, int64_t m_tiles) {
  constexpr int kPlanes = sizeof(TX) == 4 ? 3 : 1;
  __shared__ __attribute__((aligned(16))) uint16_t as[kT * kPitch];
  __shared__ __attribute__((aligned(16))) uint16_t bs[kPlanes][kT * kPitch];
  const int64_t tile = blockIdx.x / m_tiles, m0 = (blockIdx.x - tile * m_tiles) * kT;
  Place p;
  if (!place_of<kT>(a, tile, p)) return;  // the whole workgroup
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int wm = wave >> 1, wn = wave & 1, r16 = lane & 15, kg = lane >> 4;
  const int64_t m_len = kGrad ? a.c_in : a.c_out, k_len = kGrad ? a.c_out : a.c_in;
  const uint8_t* wq = a.packed + p.g * a.c_out * (a.c_in / 2);
  const uint8_t* wc = a.codes + p.g * a.c_out * (a.c_in / 16);
  const int xr = tid >> 2, xq = 16 * (tid & 3);
  const bool x_live = p.row0 + xr < p.row1;
  const char* x_row = p.x + (x_live ? (p.row0 + xr) * a.ld_x * (int64_t)sizeof(TX) : 0);

  f32x4_t acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  for (int64_t k0 = 0; k0 < k_len; k0 += kK) {
    if constexpr (!kGrad) {
      // one 16-weight block per thread: row tid / 4, block tid % 4
      const int64_t o = m0 + (tid >> 2), k = k0 + 16 * (tid & 3);
      uint2 pk = make_uint2(0u, 0u);
      uint32_t code = 0;
      if (o < a.c_out && k < a.c_in) {
        pk = load_u64(wq + (o * a.c_in + k) / 2);
        code = wc[o * (a.c_in / 16) + k / 16];
      }
      const float c = e4m3_to_f32<0>(code);
      uint4* d = reinterpret_cast<uint4*>(&as[(tid >> 2) * kPitch + 16 * (tid & 3)]);
      d[0] = units8_bf16(pk.x, c);
      d[1] = units8_bf16(pk.y, c);
    } else {
      // two output rows (consecutive k) x eight columns per thread
      const int64_t c0 = m0 + 8 * (tid & 7), o = k0 + 2 * (tid >> 3);
      float u[2][8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pk = 0, code = 0;
        if (c0 < a.c_in && o + h < a.c_out) {
          pk = load_u32(wq + ((o + h) * a.c_in + c0) / 2);
          code = wc[(o + h) * (a.c_in / 16) + c0 / 16];
        }
        units8(pk, e4m3_to_f32<0>(code), u[h]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint32_t*>(&as[(8 * (tid & 7) + j) * kPitch + 2 * (tid >> 3)]) = pack_bf16(u[0][j], u[1][j]);
    }
    stage_x<kPlanes>(x_row, k0 + xq, k_len, x_live, bs, xr * kPitch + xq);
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < kK; ks += 32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bf16x8_t fa = __builtin_bit_cast(
            bf16x8_t, *reinterpret_cast<const uint4*>(&as[(32 * wm + 16 * i + r16) * kPitch + ks + 8 * kg]));
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = kPlanes - 1; q >= 0; --q) {  // the smallest part first
            const bf16x8_t fb = __builtin_bit_cast(
                bf16x8_t, *reinterpret_cast<const uint4*>(&bs[q][(32 * wn + 16 * j + r16) * kPitch + ks + 8 * kg]));
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa, fb, acc[i][j], 0, 0, 0);
          }
      }
    }
    __syncthreads();
  }

  // lane holds outputs m0 + 32 wm + 16 i + 4 kg + 0..3 of token row0 + 32 wn + 16 j + r16
  const float s = out_scale(a, p.g);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t t = p.row0 + 32 * wn + 16 * j + r16;
    if (t >= p.row1) continue;
    TY* y = reinterpret_cast<TY*>(p.y) + t * a.ld_y;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t m = m0 + 32 * wm + 16 * i + 4 * kg;
      if (m >= m_len) continue;
      const float v[4] = {s * acc[i][j][0], s * acc[i][j][1], s * acc[i][j][2], s * acc[i][j][3]};
      store4(y + m, m_len - m, v);
    }
  }
}

// Tiles of kBT tokens the grid needs: exact for dense rows, an upper bound
// for ragged ones (a group of n rows has n / kBT full tiles and at most one more).
int64_t token_tiles(const LinearArgs& a, int64_t bt) {
  if (!a.ragged) return (a.rows + bt - 1) / bt * a.n_groups;
  return a.rows / bt + (a.n_groups < a.rows ? a.n_groups : a.rows);
}

template <bool kGrad, typename TX, typename TY>
hipError_t launch_tile(const LinearArgs& a, hipStream_t stream) {
  const int64_t m = kGrad ? a.c_in : a.c_out;
  const int64_t m_tiles = (m + kT - 1) / kT;
  linear_tile_kernel<kGrad, TX, TY><<<dim3((unsigned)(m_tiles * token_tiles(a, kT))), dim3(kThreads), 0, stream>>>(
      a, m_tiles);
  return hipGetLastError();
}

template <bool kGrad, typename TX>
hipError_t launch_x(const LinearArgs& a, hipStream_t stream) {
  return a.y_dtype == 1 ? launch_tile<kGrad, TX, uint16_t>(a, stream) : launch_tile<kGrad, TX, float>(a, stream);
}

}  // namespace

size_t linear_ws_bytes(const LinearArgs& a) {
  (void)a;
  return 0;
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t stream) {
  if (a.grad) return a.x_dtype == 1 ? launch_x<true, uint16_t>(a, stream) : launch_x<true, float>(a, stream);
  return a.x_dtype == 1 ? launch_x<false, uint16_t>(a, stream) : launch_x<false, float>(a, stream);
}

}  // namespace lh
