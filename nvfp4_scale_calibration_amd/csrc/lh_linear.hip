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
// bf16 values that add up to them exactly (from 2^-110 on; split3 says what
// tinier ones lose), so their products are exact too.
//
// MFMA orientation: operand A = weights (rows = outputs), operand B =
// activations (columns = tokens), so that a lane's accumulators are
// consecutive outputs of one token and leave in one store.
#include <math.h>

#include "lh_internal.h"
#include "lh_rows.h"

namespace lh {
namespace {

// f(0) && ... && f(N - 1), up to the first false.
template <typename F, int... I>
__device__ __forceinline__ bool static_all_impl(F&& f, std::integer_sequence<int, I...>) {
  return (f(std::integral_constant<int, I>{}) && ...);
}
template <int N, typename F>
__device__ __forceinline__ bool static_all(F&& f) {
  return static_all_impl(f, std::make_integer_sequence<int, N>{});
}

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
      g = uniform(g0 + l);
      row0 = uniform(__shfl(a, l) + (t - first) * kBT);
      row1 = uniform(min(row0 + kBT, (int64_t)__shfl(b, l)));
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
// through LDS.  Any size, stride and alignment: rows of bf16 that are not
// 16-byte aligned, fp32 or odd rows for which the caller gave no workspace,
// row strides past 32-bit offsets.  It decodes a weight once per 64 tokens,
// through LDS, with a barrier per 64 weights, and is bound by that: 8192 x
// (12288 x 4096) 1.6 ms, 0.52 PFLOP/s, against 0.68 ms of the kernels below.
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

// ---------------------------------------------------------------------------
// The large product: kNT * 32 tokens x 32 kRF kMW outputs per workgroup of kMW
// waves: 256 x 256 (four waves, one per SIMD), 128 x 256, 64 x 128, and 64 x 256
// of eight waves.
//
// Each wave owns 32 kRF outputs alone (kRF x kNT tiles of
// v_mfma_f32_32x32x16_bf16, 16 kRF kNT accumulators per lane), so every weight
// is decoded once per workgroup, in registers, straight into the MFMA operand:
// the packed bytes never pass through LDS.  The contraction index may be walked
// in any order as long as both operands agree: in a chunk of 128 weights of a
// row, the lanes of half h (l / 32) take weights 64 h .. 64 h + 63, two 16-byte
// loads, and MFMA step i (of 8) takes weights 64 h + 8 i ..  + 7 of both halves.
//
// Activations come through LDS, one chunk of 256 bytes a token in each of
// kDepth + 1 buffers, filled by direct global -> LDS loads (16 bytes a lane,
// four tokens an instruction, whole lines).  Slot q ^ (token & 15) holds
// 16-byte piece q, so that the 16 lanes which LDS serves together read one
// piece of 16 tokens from distinct banks.
//
// kP = 3: the three planes of fp32 rows side by side, three times the rows in
// LDS and three MFMAs for a decoded operand, into the same accumulators; else
// the planes follow one another along the contraction, the weights walked
// three times.
//
// Per step a wave issues kRF kNT kP MFMAs, and between them reads a later step's
// kNT kP activation operands, decodes its kRF weight operands (16 vector
// operations each) and issues its share of the next chunk's loads: with one wave
// per SIMD the matrix pipe is covered only by what is interleaved by hand
// (sched_barrier keeps each group where it is written).  The barrier of a
// chunk stands before its last step, whose operands are in registers by then,
// so that step's MFMAs cover the first reads of the next chunk.
//
// Measured: 8192 tokens x (12288 x 4096) 682 to 692 us, 1.2 PFLOP/s (a library's
// bf16 product of that size 637 us); 32768 ragged rows on 64 experts of 1024 x
// 2048 174 us, 0.79 PFLOP/s, of which the rows that fill up the experts' last
// tiles are an eighth; 48 tokens x (12288 x 4096), 64 x 256 tiles in four parts,
// 15.9 us and 4.0 for their sum (traced).  Bound by the issue of vector instructions
// between the MFMAs (decoding and LDS reads), the small tiles by the latency
// of their few chunks, the fp32 one (kP = 3) by its LDS reads, which take as
// long as its MFMAs: 333 x (4096 x 4096) fp32 48 us with packing and the sum of
// two parts (planes one after the other: 128 x 256 in five parts 57), 1000 rows
// 95 (114); four waves of 64 outputs, half the LDS reads, 53 and 100; 4096 rows
// 379, here 256 x 256 with the planes in a row is better, 358.
// Eight waves of 32 outputs instead of four: 64
// tokens x 256 outputs 40.4 us at 1024 x (4096 x 4096), where 64 x 128 takes
// 45.7; with 256 tokens 683 against 689 us, with 128 820 against 712: not kept.
// ---------------------------------------------------------------------------
constexpr int kChunk = 128;   // contraction elements per chunk

struct BigArgs {
  LinearArgs a;
  const uint16_t* x;       // bf16 rows, 16-byte aligned, a multiple of kChunk elements each
  int64_t ld, gstride;
  int chunks, w_chunks;    // chunks of x per row (1 or 3 planes) and of a weight row
  int64_t m_tiles, t_tiles;  // output tiles, token tiles (all groups)
  int splits;              // > 1: workgroups per tile, each over its share of the chunks, into part
  float* part;             // [splits][n_groups * rows][c_out]
};

// Workgroups go to the 8 XCDs in turn, and each XCD has its own L2.  Dense
// rows: the tiles are dealt so that an XCD works through a run of neighbours,
// walked in columns of 8 output tiles.  Ragged rows: how many token tiles
// there are is known on the device alone, so an XCD takes every eighth token
// tile with all its outputs (the tiles past the last one then spread evenly;
// t_tiles is a multiple of 8).
__device__ __forceinline__ void big_tile(int64_t b, bool ragged, int64_t m_tiles, int64_t t_tiles, int64_t& tile,
                                         int64_t& mt) {
  if (ragged) {
    const int64_t q = b / 8;
    tile = q / m_tiles * 8 + b % 8;
    mt = q % m_tiles;
    return;
  }
  const int64_t tiles = t_tiles * m_tiles;
  const int64_t per = tiles / 8, rest = tiles % 8, xcd = b % 8;
  const int64_t t = xcd * per + min(xcd, rest) + b / 8;
  const int64_t col = t / (8 * t_tiles), in = t - col * 8 * t_tiles;
  const int64_t width = min((int64_t)8, m_tiles - 8 * col);
  tile = in / width;
  mt = 8 * col + in - tile * width;
}

// 16 bytes per lane from base + off straight into LDS (lane l at lds + 16 l);
// the kernel waits with s_waitcnt vmcnt before the barrier that publishes the
// data.  No register is written; M0 carries the LDS address, and s_nop is the
// wait state that the ISA asks for between a scalar write of M0 and the load
// that takes its address from it (no interlock; the compiler does not look
// into asm).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
// The same for 4 bytes, 2 bytes and 1 byte (zero-extended to 4) per lane: lane l at lds + 4 l.
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void dma2(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ushort %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void dma1(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
#pragma clang diagnostic pop
// A barrier that waits for this wave's LDS reads but for none of its loads
// from global memory (which __syncthreads would drain).
__device__ __forceinline__ void block_sync() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Weights 2 i, 2 i + 1 of the eight nibbles pk times c, as packed bf16.
template <int i>
__device__ __forceinline__ uint32_t units2(uint32_t pk, float c) {
  const f32x2_t r = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(pk, 1.0f, i);
  return pack_bf16(r.x * c, r.y * c);
}

// A lane's share of one weight row's chunk: 64 weights and their 4 codes.
// kPart: rows end inside their last chunk (`whole`: this is not it); blocks
// past the end are replaced by the row's first, finite values that meet the
// zeros behind the activations' row.
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x8_t __attribute__((ext_vector_type(8)));
struct RawW {
  u32x8_t w;
  uint32_t c;
};
template <bool kPart>
__device__ __forceinline__ RawW load_raw(const uint8_t* row_q, const uint8_t* row_c, int64_t k, int64_t c_in,
                                         bool whole) {
  RawW r;
  if (!kPart || whole) {
    const uint4 u = load_u128(row_q + k / 2), v = load_u128(row_q + k / 2 + 16);
    r.w = u32x8_t{u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    r.c = load_u32(row_c + k / 16);
  } else {
    r.c = 0;
    static_for<4>([&](auto e) {
      const int64_t at = k + 16 * e < c_in ? k + 16 * e : 0;
      const uint2 v = load_u64(row_q + at / 2);
      r.w[2 * e] = v.x;
      r.w[2 * e + 1] = v.y;
      r.c |= (uint32_t)row_c[at / 16] << (8 * e);
    });
  }
  return r;
}

// A wave's corner of LDS for 32 rows of kRow bytes (padded by 16).
template <int kRow>
__device__ __forceinline__ uint8_t* lds_corner(uint8_t* lds, int wave) {
  return lds + wave * 32 * (kRow + 16);
}

// Rows row0 + 32 t + (0..31) < row1, outputs m0 .. m0 + 32 kRF - 1 < m_len of
// y = s * acc, acc as v_mfma_f32_32x32x16 leaves it (lane: token l % 32,
// outputs 32 f + 8 q + 4 (l / 32) + r).  All LDS traffic is the wave's own.
template <int kNT, int kRF, typename TY>
__device__ __forceinline__ void store_rows(const f32x16_t (&acc)[kRF][kNT], float s, uint8_t* corner,
                                           TY* __restrict__ y, int64_t ld, int64_t row0, int64_t row1, int64_t m0,
                                           int64_t m_len) {
  constexpr int kRow = 32 * kRF * (int)sizeof(TY), kPitch = kRow + 16, kE = 16 / (int)sizeof(TY);
  constexpr int kLanes = kRow / 16, kTok = 64 / kLanes;  // lanes per row, rows per instruction
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int64_t m = m0 + (lane % kLanes) * kE;
#pragma unroll
  for (int t = 0; t < kNT; ++t) {
#pragma unroll
    for (int f = 0; f < kRF; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v[4] = {s * acc[f][t][4 * q], s * acc[f][t][4 * q + 1], s * acc[f][t][4 * q + 2],
                            s * acc[f][t][4 * q + 3]};
        uint8_t* d = corner + l32 * kPitch + (32 * f + 8 * q + 4 * h) * sizeof(TY);
        if constexpr (sizeof(TY) == 2)
          *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        else
          *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < 32 / kTok; ++i) {
      const int r = i * kTok + lane / kLanes;
      const int64_t tok = row0 + 32 * t + r;
      const uint4 u = *reinterpret_cast<const uint4*>(corner + r * kPitch + (lane % kLanes) * 16);
      if (tok < row1 && m < m_len) {
        TY* d = y + tok * ld + m;
        TY w[kE];
        __builtin_memcpy(w, &u, 16);
        if (m + kE <= m_len) {
          __builtin_memcpy(d, w, 16);
        } else {
#pragma unroll
          for (int e = 0; e < kE; ++e)
            if (m + e < m_len) d[e] = w[e];
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

template <int kNT, int kRF, int kMW, int kDepth, int kWaves, int kP, bool kPart>
__global__ __launch_bounds__(64 * kMW, kWaves) void linear_big_kernel(BigArgs b) {
  constexpr int kBT = 32 * kNT;              // tokens
  constexpr int kWM = 32 * kRF;              // outputs per wave
  constexpr int kB = kNT * kP;               // activation operands of a step
  constexpr int kBuf = kP * kBT * 256;       // bytes of an LDS buffer
  constexpr int kBufs = kDepth + 1;
  constexpr int kLoads = 8 * kB / kMW;       // direct loads per wave and chunk
  // steps by which activation operands are read ahead: one step of 8 or 16
  // MFMAs covers the way through LDS, one of 1 or 2 does not
  constexpr int kR = kB >= 4 ? 1 : 3;
  // loads issued behind the next chunk's by its barrier, at least (the counter holds 63)
  constexpr int kAheadAll = (kDepth - 1) * (kLoads + 3 * kRF), kAhead = kAheadAll < 63 ? kAheadAll : 63;
  __shared__ __attribute__((aligned(1024))) uint8_t xs[kBufs * kBuf];
  int64_t tile, mt;
  big_tile(blockIdx.x, b.a.ragged, b.m_tiles, b.t_tiles, tile, mt);
  Place p;
  if (!place_of<kBT>(b.a, tile, p)) return;  // the whole workgroup
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t c_in = b.a.c_in, c_out = b.a.c_out;
  const int64_t m0 = (mt * kMW + wave) * kWM;  // the wave's first output
  // this workgroup's share of the chunks
  const int c_first = (int)((int64_t)b.chunks * blockIdx.y / b.splits);
  const int end = (int)((int64_t)b.chunks * (blockIdx.y + 1) / b.splits) - 1;  // its last one

  // direct loads: instruction i of a wave fills LDS rows 4 (wave + kMW i) .. + 3
  // (token t of plane q: row kBT q + t); slot lane & 15 of row t holds piece
  // (lane & 15) ^ (t & 15)
  const uint16_t* xg = b.x + uniform((b.a.ragged ? 0 : p.g * b.gstride) + p.row0 * b.ld);
  const int last = (int)(p.row1 - p.row0) - 1;
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int t = 4 * (wave + kMW * i) + (lane >> 4);
    off[i] = (uint32_t)min(t % kBT, last) * (uint32_t)(b.ld * 2) + (uint32_t)(t / kBT * b.w_chunks) * (2 * kChunk) +
             (uint32_t)(((lane & 15) ^ (t & 15)) * 16);
  }
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)xs) + 1024 * wave;
  auto dload = [&](int chunk, int buf, int i) {
    dma16(xg + uniform((int64_t)chunk * kChunk), off[i], lds0 + buf * kBuf + i * (1024 * kMW));
  };

  // weights: row 32 f + l32 of the wave's outputs (past the last one: the last)
  const uint8_t* wq[kRF];
  const uint8_t* wc[kRF];
#pragma unroll
  for (int f = 0; f < kRF; ++f) {
    const int64_t o = p.g * c_out + min(m0 + 32 * f + l32, c_out - 1);
    wq[f] = b.a.packed + o * (c_in / 2);
    wc[f] = b.a.codes + o * (c_in / 16);
  }
  RawW ring[kBufs][kRF];  // this chunk's weights, the next ones'
  auto wload = [&](auto d, int chunk) {
    const int w = chunk % b.w_chunks;
    static_for<kRF>([&](auto f) {
      ring[d][f] = load_raw<kPart>(wq[f], wc[f], (int64_t)w * kChunk + 64 * h, c_in, w + 1 < b.w_chunks);
    });
  };

  uint4 fa[2][kRF];
  uint4 fb[kR + 1][kB];
  f32x16_t acc[kRF][kNT];
#pragma unroll
  for (int f = 0; f < kRF; ++f)
#pragma unroll
    for (int t = 0; t < kNT; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[f][t][e] = 0.0f;

  // operand of step i, tokens 32 t + l32: piece 8 h + i of the token's buffer row
  const uint32_t rd0 = l32 * 256 + (((8 * h) ^ (l32 & 15)) * 16);
  auto bread = [&](auto set, uint32_t rd, auto i, auto t) {
    fb[set][t] = *reinterpret_cast<const uint4*>(xs + (rd ^ (16 * i)) + 8192 * t);
  };
  // pair e (of 4) of weight operand f for step s of the chunk in ring slot u (8: the next chunk's first step)
  auto decode = [&](auto set, auto u, auto s, auto f, auto e) {
    constexpr int i = s & 7;
    const RawW& r = ring[(u + (s >> 3)) % kBufs][f];
    const uint32_t v = units2<e>(r.w[i], e4m3_to_f32<(i >> 1)>(r.c));
    if constexpr (e == 0) fa[set][f].x = v;
    else if constexpr (e == 1) fa[set][f].y = v;
    else if constexpr (e == 2) fa[set][f].z = v;
    else fa[set][f].w = v;
  };
  // Step s of the chunk in slot u: its MFMAs; between them the weight operand
  // of step s + 1, the activation operands of step s + kR (LDS row address rd)
  // and the direct loads d0 .. d1 - 1 of chunk dst into buffer dbuf.
  auto step = [&](auto u, auto s, uint32_t rd, int dst, int dbuf, auto d0, auto d1) {
    constexpr int set = s & 1, bset = s % (kR + 1), rset = (s + kR) % (kR + 1);
    static_for<kRF * kB>([&](auto N) {
      constexpr int n = N;
      if constexpr (n % 4 == 0 && d0 + n / 4 < d1) dload(dst, dbuf, d0 + n / 4);
      if constexpr (kRF * kB < 4 && n == 1 && d0 + 1 < d1) dload(dst, dbuf, d0 + 1);
      if constexpr (n < kB)
        bread(std::integral_constant<int, rset>{}, rd, std::integral_constant<int, (s + kR) & 7>{}, N);
      constexpr int per = 4 / kB > 0 ? 4 / kB : 1;  // pairs per MFMA (kB = 8: every other one)
      if constexpr (kB < 8 || n % 2 == 0)
        static_for<per>([&](auto E) {
          constexpr int k = kB < 8 ? n * per + E : n / 2;  // of 4 kRF pairs
          if constexpr (k < 4 * kRF)
            decode(std::integral_constant<int, set ^ 1>{}, u, std::integral_constant<int, s + 1>{},
                   std::integral_constant<int, (k >> 2)>{}, std::integral_constant<int, (k & 3)>{});
        });
      constexpr int f = n / kB, q = n % kB, t = q % kNT;
      acc[f][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, fa[set][f]),
                                                          __builtin_bit_cast(bf16x8_t, fb[bset][q]), acc[f][t], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // Chunk c sits in buffer (c - c_first) % kBufs and is loaded kDepth chunks
  // ahead, in four steps: the last step of chunk c - kBufs (whose buffer it
  // takes: that chunk's last reads precede its barrier) and the first three of
  // the chunk after that.  Past the end the final
  // chunk is loaded again, into buffers that are read no more, so that no
  // branch breaks the schedule and the counted waits hold.
  static_for<kDepth>([&](auto d) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) dload(min(c_first + d, end), d, i);
    wload(d, min(c_first + d, end));
  });
#pragma unroll
  for (int i = 0; i < kLoads / 4; ++i) dload(min(c_first + kDepth, end), kDepth, i);
  constexpr int kStart = kAheadAll + kLoads / 4;
  wait_loads<kStart < 63 ? kStart : 63>();  // the first chunk has landed
  block_sync();
  static_for<kR>([&](auto i) {
    static_for<kB>([&](auto t) { bread(i, rd0, i, t); });
  });
  static_for<4 * kRF>([&](auto K) {
    decode(std::integral_constant<int, 0>{}, std::integral_constant<int, 0>{}, std::integral_constant<int, 0>{},
           std::integral_constant<int, (K >> 2)>{}, std::integral_constant<int, (K & 3)>{});
  });
  // chunk c, its weights in ring slot u and its activations in LDS buffer
  // buf; returns whether another one follows
  auto chunk = [&](auto u, int c, int buf) {
    const int dst1 = min(c + kDepth, end), dst2 = min(c + kDepth + 1, end);
    const int nbuf = buf + 1 == kBufs ? 0 : buf + 1, pbuf = buf == 0 ? kBufs - 1 : buf - 1;
    const uint32_t rd = rd0 + buf * kBuf, rd_next = rd0 + nbuf * kBuf;
    wload(std::integral_constant<int, (u + kDepth) % kBufs>{}, dst1);
    static_for<8>([&](auto s) {
      if constexpr (s == 8 - kR) {
        wait_loads<kAhead>();  // the next chunk has landed; this one's last operands are in registers
        block_sync();
      }
      // loads: quarters, from the last step on
      constexpr int q0 = s < 3 ? (s + 1) * kLoads / 4 : 0, q1 = s < 3 ? (s + 2) * kLoads / 4 : s == 7 ? kLoads / 4 : 0;
      step(u, s, s < 8 - kR ? rd : rd_next, s == 7 ? dst2 : dst1, s == 7 ? buf : pbuf,
           std::integral_constant<int, q0>{}, std::integral_constant<int, q1>{});
    });
    return c < end;
  };
  if constexpr (kDepth == 1) {
    int buf = 0;
    for (int c = c_first; c <= end; ++c) {
      chunk(std::integral_constant<int, 0>{}, c, buf);
      static_for<kRF>([&](auto f) { ring[0][f] = ring[1][f]; });  // loaded a chunk ago
      buf ^= 1;
    }
  } else {
    // the ring turns by unrolling: to copy a register that a load has yet to
    // fill would wait for that load
    for (int c = c_first; static_all<kBufs>([&](auto u) { return chunk(u, c + u, u); }); c += kBufs) {
    }
  }
  wait_loads<0>();  // the repeated loads have landed
  __syncthreads();  // in every wave: LDS is free

  // The wave's outputs leave through its own corner of LDS, 32 tokens at a
  // time, as whole rows of kWM outputs: a lane's four neighbouring outputs
  // alone would put 8 bytes on each of 32 lines per store instruction.
  const float sc = out_scale(b.a, p.g);
  float* const part = b.splits > 1 ? b.part + (blockIdx.y * b.a.n_groups + p.g) * b.a.rows * c_out : nullptr;
  if (part) store_rows<kNT, kRF>(acc, sc, lds_corner<kWM * 4>(xs, wave), part, c_out, p.row0, p.row1, m0, c_out);
  else if (b.a.y_dtype == 1)
    store_rows<kNT, kRF>(acc, sc, lds_corner<kWM * 4>(xs, wave), reinterpret_cast<uint16_t*>(p.y), b.a.ld_y, p.row0,
                         p.row1, m0, c_out);
  else
    store_rows<kNT, kRF>(acc, sc, lds_corner<kWM * 4>(xs, wave), reinterpret_cast<float*>(p.y), b.a.ld_y, p.row0,
                         p.row1, m0, c_out);
}

// ---------------------------------------------------------------------------
// 32 tokens a tile (2 x 16): 128 outputs per workgroup of eight waves, 16
// outputs each, v_mfma_f32_16x16x32_bf16.
//
// Here the time is the latency of the packed weights, and what counts is how
// many bytes are under way.  So nothing is loaded into registers (the
// compiler's waits for such loads know nothing of the direct ones beside them
// and drain those too): activations, packed weights and codes all go to LDS
// directly, kBufs pairs of chunks, with every wait counted.  A wave's weights
// are its own, so the barrier of a chunk is for the activations alone.
//
// Per chunk of 128 weights lane group g (l / 16) takes weights 32 g .. 32 g + 31
// of its row and MFMA step i (of 4) weights 32 g + 8 i .. + 7.  Activations as
// in linear_big_kernel; weights 64 bytes a row, the wave's 1 KiB in one
// instruction; codes one 32-bit word per lane, its two codes (kW4: one word
// each).  kW4: rows that are not 16-byte aligned, in 4-byte pieces.
//
// Measured: 128 rows on 64 experts of 1024 x 2048 14.5 to 16.7 us (tiles of 64
// tokens by linear_big_kernel 15.1, of 16 by linear_skinny_kernel 19.2, where
// this took 14.5), 18.1 where the weights are not in the last-level cache.  Bound
// by latency: 26 to 36 experts have rows in these routings, whose 31 to 43 MB of
// weights would take 6 to 9 us at a copy's rate.  More pairs of chunks in flight
// gave nothing, nor did tiles of 64 tokens in this manner.
// ---------------------------------------------------------------------------
constexpr int kSmallM = 128;

template <int kBufs, bool kW4>
__global__ __launch_bounds__(512, 2) void linear_small_kernel(BigArgs b) {
  constexpr int kNT = 2, kBT = 16 * kNT;
  constexpr int kXBytes = kBT * 256, kWBytes = 8192, kCBytes = kW4 ? 4096 : 2048;
  constexpr int kBuf = kXBytes + kWBytes + kCBytes;   // of one chunk
  constexpr int kWLoads = kW4 ? 4 : 1, kCLoads = kW4 ? 2 : 1;
  constexpr int kLoads = 1 + kWLoads + kCLoads;         // per wave and chunk
  constexpr int kAheadAll = (kBufs - 2) * 2 * kLoads, kAhead = kAheadAll < 63 ? kAheadAll : 63;
  constexpr int kR = 3;                                 // steps by which activation operands are read ahead
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kBufs * 2 * kBuf];
  int64_t tile, mt;
  big_tile(blockIdx.x, b.a.ragged, b.m_tiles, b.t_tiles, tile, mt);
  Place p;
  if (!place_of<kBT>(b.a, tile, p)) return;  // the whole workgroup
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c_in = b.a.c_in, c_out = b.a.c_out;
  const int64_t m0 = mt * kSmallM + 16 * wave;
  const int c_first = (int)((int64_t)b.chunks * blockIdx.y / b.splits);
  const int end = (int)((int64_t)b.chunks * (blockIdx.y + 1) / b.splits) - 1;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);

  const uint16_t* const xg = b.x + uniform((b.a.ragged ? 0 : p.g * b.gstride) + p.row0 * b.ld);
  const int last = (int)(p.row1 - p.row0) - 1;
  const int xt = 4 * wave + (lane >> 4);  // the token this lane loads from
  const uint32_t xoff = (uint32_t)min(xt, last) * (uint32_t)(b.ld * 2) + (uint32_t)(((lane & 15) ^ (xt & 15)) * 16);
  // the wave's rows from its first one on (rows past the last one are the last one)
  const int64_t w_row = c_in / 2, c_row = c_in / 16, o0 = min(m0, c_out - 1);
  const uint8_t* const wg = b.a.packed + uniform((p.g * c_out + o0) * w_row);
  const uint8_t* const cg = b.a.codes + uniform((p.g * c_out + o0) * c_row);
  auto row_of = [&](int r) { return (uint32_t)(min(m0 + r, c_out - 1) - o0); };
  // weights: row lane / 4, 16-byte piece lane % 4; or (kW4) rows 4 i + lane / 16, 4-byte piece lane % 16
  uint32_t woff[kWLoads];
#pragma unroll
  for (int i = 0; i < kWLoads; ++i) woff[i] = row_of(kW4 ? 4 * i + (lane >> 4) : lane >> 2) * (uint32_t)w_row;
  const uint32_t coff = row_of(l16) * (uint32_t)c_row;
  const int w_last = b.w_chunks - 1;
  const uint32_t left = (uint32_t)(c_in - (int64_t)w_last * kChunk);  // weights of a row's last chunk
  // the loads of a chunk into buffer `at`; a piece past the row's end is the
  // chunk's first one (finite weights that meet the zeros behind the
  // activations' row)
  int ld_c = c_first, ld_w = c_first % b.w_chunks;  // the next chunk to load, and that chunk of W (which repeats)
  auto dload = [&](uint32_t at) {
    dma16(xg + ld_c * kChunk, xoff, lds0 + at + 1024 * wave);
    const uint32_t n = ld_w == w_last ? left : (uint32_t)kChunk;
    const uint8_t* const wb = wg + ld_w * (kChunk / 2);
    const uint8_t* const cb = cg + ld_w * (kChunk / 16);
    if (ld_c < end) {
      ++ld_c;
      ld_w = ld_w == w_last ? 0 : ld_w + 1;
    }
    const uint32_t wd = lds0 + at + kXBytes + 1024 * wave, cd = lds0 + at + kXBytes + kWBytes + (kCBytes / 8) * wave;
    if constexpr (!kW4) {
      const uint32_t q = (lane & 3) * 32u < n ? (lane & 3) * 16u : 0u;
      dma16(wb, woff[0] + q, wd);
      dma2(cb, coff + (g * 32u < n ? g * 2u : 0u), cd);
    } else {
      const uint32_t q = l16 * 8u < n ? l16 * 4u : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) dma4(wb, woff[i] + q, wd + 256 * i);
#pragma unroll
      for (int i = 0; i < 2; ++i) dma1(cb, coff + (g * 32u + i * 16u < n ? g * 2u + i : 0u), cd + 256 * i);
    }
  };

  uint4 fa[2], fb[kR + 1][kNT], raw, raw_next;
  uint32_t code[2], code_next[2];
  f32x4_t acc[kNT];
#pragma unroll
  for (int t = 0; t < kNT; ++t) acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  // activations: token 16 t + l16, piece 4 g + i; weights: row l16, piece g
  const uint32_t rd0 = l16 * 256 + (((4 * g) ^ l16) * 16);
  const uint32_t wrd = kXBytes + 1024 * wave + l16 * 64 + g * 16;
  const uint32_t crd = kXBytes + kWBytes + (kCBytes / 8) * wave + lane * 4;
  auto bread = [&](auto set, uint32_t at, auto i) {
#pragma unroll
    for (int t = 0; t < kNT; ++t)
      fb[set][t] = *reinterpret_cast<const uint4*>(lds + at + (rd0 ^ (16 * i)) + 4096 * t);
  };
  auto wread = [&](uint32_t at) {
    raw_next = *reinterpret_cast<const uint4*>(lds + at + wrd);
    code_next[0] = *reinterpret_cast<const uint32_t*>(lds + at + crd);
    if constexpr (kW4) code_next[1] = *reinterpret_cast<const uint32_t*>(lds + at + crd + 256);
  };
  auto decode = [&](auto set, const uint4& r, const uint32_t (&cc)[2], auto i) {
    const uint32_t w = i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
    const float c = kW4 ? e4m3_to_f32<0>(i < 2 ? cc[0] : cc[1]) : e4m3_to_f32<(i >> 1)>(cc[0]);
    fa[set] = units8_bf16(w, c);
  };

  for (int d = 0; d < 2 * kBufs; ++d) dload(d * kBuf);
  constexpr int kStart = (kBufs - 1) * 2 * kLoads;
  wait_loads<kStart < 63 ? kStart : 63>();  // the first two chunks have landed
  block_sync();
  std::integral_constant<int, 0> i0;
  static_for<kR>([&](auto i) { bread(i, 0u, i); });
  wread(0u);
  auto take = [&]() {
    raw = raw_next;
    code[0] = code_next[0];
    if constexpr (kW4) code[1] = code_next[1];
  };
  take();
  decode(i0, raw, code, i0);
  auto multiply = [&](auto s) {
#pragma unroll
    for (int t = 0; t < kNT; ++t)
      acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, fa[s & 1]),
                                                       __builtin_bit_cast(bf16x8_t, fb[s & 3][t]), acc[t], 0, 0, 0);
  };
  uint32_t at = 0;
  for (int c = c_first; c < end; c += 2) {  // two chunks, eight steps
    const uint32_t second = at + kBuf, next = at + 2 * kBuf == kBufs * 2 * kBuf ? 0u : at + 2 * kBuf;
    static_for<8>([&](auto s) {
      if constexpr (s == 1) wread(second);
      constexpr int rs = s + kR, ns = s + 1;
      bread(std::integral_constant<int, rs & 3>{}, rs >= 8 ? next : rs >= 4 ? second : at,
            std::integral_constant<int, rs & 3>{});
      if constexpr (s == 4) {
        // the last operands of these two chunks are on their way to registers
        // and the next two chunks have landed: past the barrier, in every
        // wave, and these two's buffers can be loaded again
        wait_loads<kAhead>();
        wread(next);
        block_sync();
        dload(at);
        dload(second);
      }
      std::integral_constant<int, ns & 1> nset;
      std::integral_constant<int, ns & 3> ni;
      if constexpr ((ns & 3) == 0) take();
      decode(nset, raw, code, ni);
      multiply(s);
      __builtin_amdgcn_sched_barrier(0);
    });
    at = next;
  }
  if ((end - c_first) % 2 == 0)  // an odd chunk out, in LDS and its first operands in registers
    static_for<4>([&](auto s) {
      if constexpr (s + kR < 4) bread(std::integral_constant<int, s + kR>{}, at, std::integral_constant<int, s + kR>{});
      if constexpr (s < 3)
        decode(std::integral_constant<int, (s + 1) & 1>{}, raw, code, std::integral_constant<int, s + 1>{});
      multiply(s);
    });
  wait_loads<0>();  // the repeated loads: nothing lands after the workgroup has ended

  const float sc = out_scale(b.a, p.g);
  float* const part = b.splits > 1 ? b.part + (blockIdx.y * b.a.n_groups + p.g) * b.a.rows * c_out : nullptr;
  const int64_t m = m0 + 4 * g;
#pragma unroll
  for (int t = 0; t < kNT; ++t) {
    const int64_t tok = p.row0 + 16 * t + l16;
    if (tok >= p.row1 || m >= c_out) continue;
    const float v[4] = {sc * acc[t][0], sc * acc[t][1], sc * acc[t][2], sc * acc[t][3]};
    if (part) store4(part + tok * c_out + m, c_out - m, v);
    else if (b.a.y_dtype == 1) store4(reinterpret_cast<uint16_t*>(p.y) + tok * b.a.ld_y + m, c_out - m, v);
    else store4(reinterpret_cast<float*>(p.y) + tok * b.a.ld_y + m, c_out - m, v);
  }
}

// ---------------------------------------------------------------------------
// Up to 16 tokens a tile: 32 outputs per workgroup, the contraction split over
// its kW waves, v_mfma_f32_16x16x32_bf16.
//
// What counts is how many bytes of weights are under way and that nothing
// stands still for anything else: every wave streams its own chunks of
// activations (4 KiB), packed weights (2 KiB) and codes to its own part of LDS
// by direct loads, kBufs chunks ahead, with counted waits, and no barrier is
// met before the end, where the waves' sums are added in order.  (The
// activations' repeated way to LDS is twice the weights' bytes, from L2.)
//
// Per chunk of 128 weights lane group g (l / 16) takes weights 32 g .. 32 g + 31
// of its row and MFMA step i (of 4) weights 32 g + 8 i .. + 7.  LDS: 256 bytes a
// token, slot q ^ (token & 15) holding 16-byte piece q; 64 bytes a row of
// weights; one 32-bit word per lane and operand for its two codes (kW4: one
// word each).  kW4: rows that are not 16-byte aligned, in 4-byte pieces.
//
// Measured: 16 tokens x (4096 x 4096) 8.0 to 9.4 us (launch, one chunk's latency and
// the join alone are 5), 8 tokens x (12288 x 4096) 13.1 us, 2.2 TB/s of weights;
// linear_small_kernel 13.3 and 16.6.
// ---------------------------------------------------------------------------
constexpr int kSkinnyM = 32;

template <int kW, int kBufs, bool kW4>
__global__ __launch_bounds__(64 * kW, 2) void linear_skinny_kernel(BigArgs b) {
  constexpr int kXBytes = 4096, kWBytes = 2048, kCBytes = kW4 ? 1024 : 512;
  constexpr int kBuf = kXBytes + kWBytes + kCBytes;
  constexpr int kWLoads = kW4 ? 8 : 2, kCLoads = kW4 ? 4 : 2, kLoads = 4 + kWLoads + kCLoads;
  static_assert((kBufs - 1) * kLoads < 64, "the load counter");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kW * kBufs * kBuf];
  int64_t tile, mt;
  big_tile(blockIdx.x, b.a.ragged, b.m_tiles, b.t_tiles, tile, mt);
  Place p;
  if (!place_of<16>(b.a, tile, p)) return;  // the whole workgroup
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t c_in = b.a.c_in, c_out = b.a.c_out, m0 = mt * kSkinnyM;
  const int64_t share = (int64_t)blockIdx.y * kW + wave, shares = (int64_t)b.splits * kW;
  const int c_first = (int)(b.chunks * share / shares);
  const int end = (int)(b.chunks * (share + 1) / shares) - 1;  // < c_first: nothing to do

  const uint16_t* const xg = b.x + uniform((b.a.ragged ? 0 : p.g * b.gstride) + p.row0 * b.ld);
  const int last = (int)(p.row1 - p.row0) - 1;
  uint32_t xoff[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 4 * i + (lane >> 4);
    xoff[i] = (uint32_t)min(t, last) * (uint32_t)(b.ld * 2) + (uint32_t)(((lane & 15) ^ t) * 16);
  }
  const int64_t w_row = c_in / 2, c_row = c_in / 16;
  const uint8_t* const wg = b.a.packed + uniform((p.g * c_out + m0) * w_row);
  const uint8_t* const cg = b.a.codes + uniform((p.g * c_out + m0) * c_row);
  auto row_of = [&](int r) { return (uint32_t)(min(m0 + r, c_out - 1) - m0); };
  // weights: rows 16 i + lane / 4, piece lane % 4; or (kW4) rows 4 i + lane / 16, 4-byte piece lane % 16
  uint32_t woff[kWLoads], coff[2];
#pragma unroll
  for (int i = 0; i < kWLoads; ++i)
    woff[i] = row_of(kW4 ? 4 * i + (lane >> 4) : 16 * i + (lane >> 2)) * (uint32_t)w_row;
#pragma unroll
  for (int f = 0; f < 2; ++f) coff[f] = row_of(16 * f + l16) * (uint32_t)c_row;
  const int w_last = b.w_chunks - 1;
  const uint32_t left = (uint32_t)(c_in - (int64_t)w_last * kChunk);  // weights of a row's last chunk
  uint8_t* const mine = lds + wave * (kBufs * kBuf);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)mine);
  int ld_c = c_first, ld_w = c_first % b.w_chunks;  // the next chunk to load, and that chunk of W (which repeats)
  // that chunk into buffer `at`; a piece past the row's end is the chunk's
  // first one (finite weights that meet the zeros behind the activations' row)
  auto dload = [&](uint32_t at) {
    const uint16_t* const xb = xg + ld_c * kChunk;
#pragma unroll
    for (int i = 0; i < 4; ++i) dma16(xb, xoff[i], lds0 + at + 1024 * i);
    const uint32_t n = ld_w == w_last ? left : (uint32_t)kChunk;
    const uint8_t* const wb = wg + ld_w * (kChunk / 2);
    const uint8_t* const cb = cg + ld_w * (kChunk / 16);
    const uint32_t wd = lds0 + at + kXBytes, cd = wd + kWBytes;
    const uint32_t q = kW4 ? (l16 * 8u < n ? l16 * 4u : 0u) : ((lane & 3) * 32u < n ? (lane & 3) * 16u : 0u);
#pragma unroll
    for (int i = 0; i < kWLoads; ++i) {
      if constexpr (kW4) dma4(wb, woff[i] + q, wd + 256 * i);
      else dma16(wb, woff[i] + q, wd + 1024 * i);
    }
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      if constexpr (!kW4) {
        dma2(cb, coff[f] + (g * 32u < n ? g * 2u : 0u), cd + 256 * f);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          dma1(cb, coff[f] + (g * 32u + i * 16u < n ? g * 2u + i : 0u), cd + 512 * f + 256 * i);
      }
    }
    if (ld_c < end) {  // past the end the last chunk again, into buffers that are read no more
      ++ld_c;
      ld_w = ld_w == w_last ? 0 : ld_w + 1;
    }
  };

  // a chunk's operands in registers
  struct Regs {
    uint4 x[4], w[2];
    uint32_t c[2], c1[2];
  };
  auto lread = [&](uint32_t at) {
    Regs r;
    const uint8_t* const q = mine + at;
    static_for<4>([&](auto i) {
      r.x[i] = *reinterpret_cast<const uint4*>(q + l16 * 256 + (((4 * g + i) ^ l16) * 16));
    });
    static_for<2>([&](auto f) {
      r.w[f] = *reinterpret_cast<const uint4*>(q + kXBytes + 1024 * f + l16 * 64 + g * 16);
      const uint8_t* const c = q + kXBytes + kWBytes + (kW4 ? 512 : 256) * f + lane * 4;
      r.c[f] = *reinterpret_cast<const uint32_t*>(c);
      if constexpr (kW4) r.c1[f] = *reinterpret_cast<const uint32_t*>(c + 256);
    });
    return r;
  };
  f32x4_t acc[2] = {f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}};
  if (c_first <= end) {
    for (int d = 0; d < kBufs; ++d) dload(d * kBuf);
    wait_loads<(kBufs - 1) * kLoads>();
    Regs r = lread(0);
    uint32_t at = 0;
    for (int c = c_first; c <= end; ++c) {
      const uint32_t next = at + kBuf == kBufs * kBuf ? 0u : at + kBuf;
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this chunk's operands are in registers:
      dload(at);                                          // its buffer is free
      wait_loads<(kBufs - 1) * kLoads>();                 // the next chunk has landed
      const Regs n = lread(next);
      static_for<4>([&](auto i) {
        static_for<2>([&](auto f) {
          const uint32_t w = i == 0 ? r.w[f].x : i == 1 ? r.w[f].y : i == 2 ? r.w[f].z : r.w[f].w;
          const float s = kW4 ? e4m3_to_f32<0>(i < 2 ? r.c[f] : r.c1[f]) : e4m3_to_f32<(i >> 1)>(r.c[f]);
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, units8_bf16(w, s)),
                                                           __builtin_bit_cast(bf16x8_t, r.x[i]), acc[f], 0, 0, 0);
        });
      });
      r = n;
      at = next;
    }
    wait_loads<0>();  // the repeated loads have landed
  }

  // the waves' sums, added in their order: output row 16 f + 4 g + e of token l16 at [f][lane]
  __syncthreads();
  float4* const sums = reinterpret_cast<float4*>(lds);
#pragma unroll
  for (int f = 0; f < 2; ++f)
    sums[(wave * 2 + f) * 64 + lane] = make_float4(acc[f][0], acc[f][1], acc[f][2], acc[f][3]);
  __syncthreads();
  if (wave >= 2) return;
  const int f = wave;
  float v[4] = {};
#pragma unroll
  for (int q = 0; q < kW; ++q) {
    const float4 u = sums[(q * 2 + f) * 64 + lane];
    v[0] = q == 0 ? u.x : v[0] + u.x;
    v[1] = q == 0 ? u.y : v[1] + u.y;
    v[2] = q == 0 ? u.z : v[2] + u.z;
    v[3] = q == 0 ? u.w : v[3] + u.w;
  }
  const float sc = out_scale(b.a, p.g);
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] *= sc;
  const int64_t tok = p.row0 + l16, m = m0 + 16 * f + 4 * g;
  if (tok >= p.row1 || m >= c_out) return;
  if (b.splits > 1)
    store4(b.part + (blockIdx.y * b.a.n_groups + p.g) * b.a.rows * c_out + tok * c_out + m, c_out - m, v);
  else if (b.a.y_dtype == 1)
    store4(reinterpret_cast<uint16_t*>(p.y) + tok * b.a.ld_y + m, c_out - m, v);
  else
    store4(reinterpret_cast<float*>(p.y) + tok * b.a.ld_y + m, c_out - m, v);
}

// ---------------------------------------------------------------------------
// The large gradient: 64 kNT tokens x 256 columns per workgroup, four waves
// of 32 kNT tokens x 128 columns.
//
// The contraction runs down the weights' rows, so an MFMA operand needs the
// same column of eight rows.  Nothing is transposed for that: operand f (of
// four) of a wave stands for columns 4 m + f (m its row 0..31), so lane m
// needs the same two bytes of eight rows, four neighbouring columns, and the
// rounding to bf16, which packs two values a register, pairs the rows.  The
// accumulators of a lane are then 16 consecutive columns of its token.
//
// A stage is 64 rows of W (o) for all tokens and columns of the workgroup.
// Everything comes by direct global -> LDS loads: dy 128 bytes a token (slot
// q ^ (token / 2 % 8) holds 16-byte piece q, so 16 tokens' reads of one piece
// meet no bank twice), the packed rows 128 bytes each, and the codes, one
// 32-bit word each, four rows of a block side by side, so that a lane reads
// its eight rows' codes in two 16-byte reads.  With no load into registers in
// the loop every wait is counted by hand, kDepth stages ahead.
//
// Per step (16 rows) a wave issues 4 kNT MFMAs and between them reads the next
// step's operands in the first slots and decodes them in the later ones (72
// vector operations; a weight is decoded by the two waves that share its
// columns).
//
// Measured: 4096 tokens x (12288 x 4096) 389 to 396 us, 1.05 PFLOP/s; 32768
// ragged rows on 64 experts of 1024 x 2048 209 us, 0.66 PFLOP/s.  Bound by vector
// issue as the product, with the pairing of rows on top (72 operations for 4
// kNT MFMAs, against 64 for as many there).
// ---------------------------------------------------------------------------
constexpr int kGradK = 64;      // rows of W per stage
constexpr int kGradM = 256;     // columns per workgroup

struct GradArgs {
  LinearArgs a;
  const uint16_t* x;       // dy: bf16 rows, 16-byte aligned, a multiple of kGradK elements each
  int64_t ld, gstride;
  int stages, w_stages;    // stages of an x row (1 or 3 planes) and of W
  int64_t m_tiles, t_tiles;
  int splits;
  float* part;
};

// kW4: the packed rows are not 16-byte aligned and come in 4-byte pieces.
template <int kNT, int kDepth, int kWaves, bool kW4>
__global__ __launch_bounds__(kThreads, kWaves) void grad_big_kernel(GradArgs b) {
  constexpr int kBT = 64 * kNT;
  constexpr int kXBytes = kBT * 2 * kGradK, kWBytes = kGradK * kGradM / 2, kCBytes = kGradK * kGradM / 16 * 4;
  constexpr int kBuf = kXBytes + kWBytes + kCBytes;
  constexpr int kBufs = kDepth + 1;
  constexpr int kXLoads = kXBytes / 4096, kWLoads = kW4 ? 8 : 2, kCLoads = 4;  // per wave and stage
  constexpr int kLoads = kXLoads + kWLoads + kCLoads;
  constexpr int kAhead = (kDepth - 1) * kLoads;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kBufs * kBuf];
  int64_t tile, mt;
  big_tile(blockIdx.x, b.a.ragged, b.m_tiles, b.t_tiles, tile, mt);
  Place p;
  if (!place_of<kBT>(b.a, tile, p)) return;  // the whole workgroup
  const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t c_in = b.a.c_in, c_out = b.a.c_out, m0 = mt * kGradM;
  const int s_first = (int)((int64_t)b.stages * blockIdx.y / b.splits);
  const int end = (int)((int64_t)b.stages * (blockIdx.y + 1) / b.splits) - 1;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);

  // dy: instruction i of a wave fills tokens 8 (wave + 4 i) .. + 7
  const uint16_t* xg = b.x + uniform((b.a.ragged ? 0 : p.g * b.gstride) + p.row0 * b.ld);
  const int last = (int)(p.row1 - p.row0) - 1;
  const int xrow = 8 * wave + (lane >> 3);
  uint32_t xoff[kXLoads];
#pragma unroll
  for (int i = 0; i < kXLoads; ++i) {
    const int t = xrow + 32 * i;
    xoff[i] = (uint32_t)min(t, last) * (uint32_t)(b.ld * 2) + (uint32_t)(((lane & 7) ^ ((t >> 1) & 7)) * 16);
  }
  // packed rows: 16-byte pieces, 8 rows an instruction, or 4-byte pieces, 2
  // rows; a piece past the row's end is the row's first one (columns that are
  // not stored)
  const int64_t w_row = c_in / 2, c_row = c_in / 16;
  constexpr int kWRows = kW4 ? 2 : 8;  // rows an instruction
  const int wrow = kW4 ? lane >> 5 : lane >> 3;
  int64_t wcol = m0 / 2 + (kW4 ? 4 * (lane & 31) : 16 * (lane & 7));
  if (wcol >= w_row) wcol = 0;
  // codes: block lane / 4, rows lane % 4 of an instruction's four
  const int crow = lane & 3;
  int64_t ccol = m0 / 16 + (lane >> 2);
  if (ccol >= c_row) ccol = 0;
  const uint8_t* wg = b.a.packed + uniform(p.g * c_out * w_row);
  const uint8_t* cg = b.a.codes + uniform(p.g * c_out * c_row);
  // load n of a stage's kLoads of this wave into buffer buf
  auto dload = [&](int st, int buf, auto N) {
    constexpr int n = N;
    const uint32_t at = lds0 + buf * kBuf;
    if constexpr (n < kXLoads) {
      dma16(xg + uniform((int64_t)st * kGradK), xoff[n], at + 1024 * (wave + 4 * n));
    } else {
      // row o0 of the stage; rows past the last one are the last one (their dy is zero)
      const int64_t o0 = (int64_t)(st % b.w_stages) * kGradK;
      if constexpr (n < kXLoads + kWLoads) {
        constexpr int i = n - kXLoads;
        const int base = kWRows * (wave + 4 * i);
        const int64_t o = min(o0 + base + wrow, c_out - 1);
        const int64_t first = min(o0 + base, c_out - 1);  // wave-uniform
        const uint32_t off = (uint32_t)((o - first) * w_row + wcol);
        const uint32_t dst = at + kXBytes + base * (kGradM / 2);
        if constexpr (kW4) dma4(wg + uniform(first * w_row), off, dst);
        else dma16(wg + uniform(first * w_row), off, dst);
      } else {
        constexpr int i = n - kXLoads - kWLoads;
        const int base = 4 * (wave + 4 * i);
        const int64_t o = min(o0 + base + crow, c_out - 1);
        const int64_t first = min(o0 + base, c_out - 1);
        dma1(cg + uniform(first * c_row), (uint32_t)((o - first) * c_row + ccol),
             at + kXBytes + kWBytes + base * (kGradM / 16) * 4);
      }
    }
  };

  // operand addresses within a buffer
  const uint32_t xrd = (32 * kNT * wn + l32) * 128;            // + 4096 t, piece 2 i + h
  const uint32_t xsw = (l32 >> 1) & 7;
  const uint32_t wrd = kXBytes + 8 * h * (kGradM / 2) + 64 * wm + 2 * l32;                // + 128 (16 i + e)
  const uint32_t crd = kXBytes + kWBytes + ((2 * h) * (kGradM / 16) + 8 * wm + (l32 >> 2)) * 16;  // + 1024 i

  f32x16_t acc[4][kNT];
#pragma unroll
  for (int f = 0; f < 4; ++f)
#pragma unroll
    for (int t = 0; t < kNT; ++t)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[f][t][e] = 0.0f;
  u32x4_t fa[2][4];
  uint4 fb[2][kNT];
  uint32_t raw[4];   // rows 2 e, 2 e + 1 of the step: two bytes each
  uint4 code[2];

  auto bread = [&](auto set, int base, auto i, auto t) {
    fb[set][t] = *reinterpret_cast<const uint4*>(lds + base + xrd + 4096 * t + (((2 * i + h) ^ xsw) * 16));
  };
  auto wread = [&](int base, auto i, auto e) {
    const uint8_t* r = lds + base + wrd + (16 * i + 2 * e) * (kGradM / 2);
    const uint32_t lo = *reinterpret_cast<const uint16_t*>(r);
    const uint32_t hi = *reinterpret_cast<const uint16_t*>(r + kGradM / 2);
    raw[e] = lo | (hi << 16);
  };
  auto cread = [&](int base, auto i, auto j) {
    code[j] = *reinterpret_cast<const uint4*>(lds + base + crd + (16 * i + 4 * j) / 4 * (kGradM / 16) * 16);
  };
  // rows 2 e, 2 e + 1, columns 2 q, 2 q + 1 of the four
  auto decode = [&](auto set, auto U) {
    constexpr int e = U >> 1, q = U & 1;
    const uint4 cc = code[e >> 1];
    const float s0 = e4m3_to_f32<0>(e & 1 ? cc.z : cc.x), s1 = e4m3_to_f32<0>(e & 1 ? cc.w : cc.y);
    const f32x2_t r0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(raw[e], 1.0f, q);
    const f32x2_t r1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(raw[e], 1.0f, 2 + q);
    fa[set][2 * q][e] = pack_bf16(r0.x * s0, r1.x * s1);
    fa[set][2 * q + 1][e] = pack_bf16(r0.y * s0, r1.y * s1);
  };
  // Step s (of 4): the MFMAs of operand set s & 1; the operands of the next
  // step from LDS buffer `base`; direct loads d0 .. d1 - 1 of stage dst.
  auto step = [&](auto s, int base, int dst, int dbuf, auto d0, auto d1) {
    constexpr int set = s & 1, slots = 4 * kNT;
    static_for<slots>([&](auto N) {
      constexpr int n = N;
      std::integral_constant<int, set ^ 1> nset;
      std::integral_constant<int, (s + 1) & 3> ni;
      // reads first: codes and packed rows in slots 0, 1 (kNT = 2) or 0 .. 3, activations over the step
      constexpr int rs = slots / 4;
      if constexpr (n < rs) {
        static_for<4 / rs>([&](auto K) { wread(base, ni, std::integral_constant<int, n * (4 / rs) + K>{}); });
        if constexpr (n < 2) cread(base, ni, N);
        if constexpr (rs == 1) cread(base, ni, std::integral_constant<int, 1>{});
      } else if constexpr (n - rs < kNT) {
        bread(nset, base, ni, std::integral_constant<int, n - rs>{});
      }
      // direct loads, dealt over the slots
      static_for<(d1 - d0 + slots - 1) / slots>([&](auto K) {
        constexpr int per = (d1 - d0 + slots - 1) / slots, i = d0 + n * per + K;
        if constexpr (i < d1) dload(dst, dbuf, std::integral_constant<int, i>{});
      });
      // decoding from slot slots / 2 on
      constexpr int u0 = n < slots / 2 ? 0 : (n - slots / 2) * 8 / (slots / 2),
                    u1 = n < slots / 2 ? 0 : (n + 1 - slots / 2) * 8 / (slots / 2);
      static_for<u1 - u0>([&](auto K) { decode(nset, std::integral_constant<int, u0 + K>{}); });
      constexpr int f = n / kNT, t = n % kNT;
      acc[f][t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, fa[set][f]),
                                                          __builtin_bit_cast(bf16x8_t, fb[set][t]), acc[f][t], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // Stage S sits in buffer (S - s_first) % kBufs.  Its loads go out in three
  // steps: the last step of stage S - kBufs (after the barrier that ends that
  // stage's reads) and the first two of the next stage; past the end the
  // final stage is loaded again into buffers that are read no more.
  constexpr int kQ0 = kLoads / 3, kQ1 = 2 * kLoads / 3;
  static_for<kDepth>([&](auto d) {
    static_for<kLoads>([&](auto n) { dload(min(s_first + d, end), d, n); });
  });
  static_for<kQ0>([&](auto n) { dload(min(s_first + kDepth, end), kDepth, n); });
  wait_loads<kAhead + kQ0>();  // the first stage has landed
  block_sync();
  {
    std::integral_constant<int, 0> zero;
    static_for<4>([&](auto e) { wread(0, zero, e); });
    static_for<2>([&](auto j) { cread(0, zero, j); });
    static_for<kNT>([&](auto t) { bread(zero, 0, zero, t); });
    static_for<8>([&](auto u) { decode(zero, u); });
  }
  int buf = 0;
  for (int st = s_first; st <= end; ++st) {
    const int dst1 = min(st + kDepth, end), dst2 = min(st + kDepth + 1, end);
    const int nbuf = buf + 1 == kBufs ? 0 : buf + 1, pbuf = buf == 0 ? kBufs - 1 : buf - 1;
    const int base = buf * kBuf, nbase = nbuf * kBuf;
    std::integral_constant<int, 0> i0;
    std::integral_constant<int, 1> i1;
    std::integral_constant<int, 2> i2;
    std::integral_constant<int, 3> i3;
    std::integral_constant<int, kQ0> q0;
    std::integral_constant<int, kQ1> q1;
    std::integral_constant<int, kLoads> q2;
    step(i0, base, dst1, pbuf, q0, q1);
    step(i1, base, dst1, pbuf, q1, q2);
    step(i2, base, dst1, pbuf, i0, i0);
    wait_loads<kAhead>();  // the next stage has landed; this one's last operands are in registers
    block_sync();
    step(i3, nbase, dst2, buf, i0, q0);
    buf = nbuf;
  }
  wait_loads<0>();  // the repeated loads: nothing lands after the workgroup has ended

  // lane: token 32 kNT wn + 32 t + l32, columns m0 + 128 wm + 32 q + 16 h + 4 r + f
  const float sc = out_scale(b.a, p.g);
  float* part = b.splits > 1 ? b.part + (blockIdx.y * b.a.n_groups + p.g) * b.a.rows * c_in : nullptr;
#pragma unroll
  for (int t = 0; t < kNT; ++t) {
    const int64_t tok = p.row0 + 32 * kNT * wn + 32 * t + l32;
    if (tok >= p.row1) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t c = m0 + 128 * wm + 32 * q + 16 * h;
      if (c >= c_in) continue;  // c_in is a multiple of 16: all sixteen or none
      float v[16];
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int f = 0; f < 4; ++f) v[4 * r + f] = sc * acc[f][t][4 * q + r];
      if (part || b.a.y_dtype == 0) {
        float* d = part ? part + tok * c_in + c : reinterpret_cast<float*>(p.y) + tok * b.a.ld_y + c;
        __builtin_memcpy(d, v, 64);
      } else {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        __builtin_memcpy(reinterpret_cast<uint16_t*>(p.y) + tok * b.a.ld_y + c, o, 32);
      }
    }
  }
}

// y = the splits' sums, added in split order (so results do not change from
// run to run, as they would with atomics).  Memory-bound: 333 x 4096 in two
// parts, 16 MB, 5.3 us.
template <typename TY>
__global__ __launch_bounds__(kThreads) void split_sum_kernel(const float* __restrict__ part, int splits, int64_t rows,
                                                             int64_t n_groups, int64_t cols, TY* __restrict__ y,
                                                             int64_t ld_y, int64_t gstride_y) {
  const int64_t vecs = (cols + 3) / 4;
  const int64_t i = block_id() * kThreads + threadIdx.x;
  const int64_t r = i / vecs, c = 4 * (i - r * vecs);
  if (r >= rows * n_groups) return;
  const int64_t n = cols - c, step = n_groups * rows * cols;
  const float* p = part + r * cols + c;
  float v[4] = {};
  for (int s = 0; s < splits; ++s, p += step) {
    float u[4] = {};
    if (n >= 4) {
      __builtin_memcpy(u, p, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < n) u[e] = p[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = s == 0 ? u[e] : v[e] + u[e];
  }
  const int64_t g = r / rows;
  store4(y + g * gstride_y + (r - g * rows) * ld_y + c, n, v);
}

// Rows of any alignment and length to bf16 rows of kp elements (zeros past
// k), fp32 as three planes of kp elements behind each other: the sum of the
// planes' products is the product.
// Memory-bound: 333 x 4096 fp32 5.6 us, launch included.
template <typename TX>
__global__ __launch_bounds__(kThreads) void pack_rows_kernel(const TX* __restrict__ x, int64_t rows, int64_t k,
                                                             int64_t ld, int64_t n_groups, int64_t gstride, int64_t kp,
                                                             uint16_t* __restrict__ out) {
  constexpr int kPlanes = sizeof(TX) == 4 ? 3 : 1;
  const int64_t i = block_id() * kThreads + threadIdx.x;
  const int64_t vecs = kp / 8, r = i / vecs, c = 8 * (i - r * vecs);
  if (r >= rows * n_groups) return;
  const int64_t g = r / rows;
  const TX* p = x + g * gstride + (r - g * rows) * ld + c;
  TX v[8] = {};
  if (c + 8 <= k) {
    __builtin_memcpy(v, p, 8 * sizeof(TX));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < k) v[e] = p[e];
  }
  uint4* d = reinterpret_cast<uint4*>(out + r * kPlanes * kp + c);
  if constexpr (kPlanes == 1) {
    uint4 o;
    __builtin_memcpy(&o, v, 16);
    *d = o;
  } else {
    uint32_t b[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) split3(v[2 * e], v[2 * e + 1], b[e]);
#pragma unroll
    for (int q = 0; q < 3; ++q) d[q * (kp / 8)] = make_uint4(b[0][q], b[1][q], b[2][q], b[3][q]);
  }
}

// ---------------------------------------------------------------------------
// A few tokens (decoding): kTok tokens x kRows outputs per wave, no matrix
// cores.  The packed weights are read once and everything else is made small
// against them: lane l takes weights 32 l .. 32 l + 31 of a 2048-weight span
// of each row (one 16-byte load, consecutive over the wave), keeps the same
// span of the activations in registers for all its rows, and multiplies in
// pairs: E2M1 values are exact in bf16, so v_dot2_f32_bf16 adds two exact
// products to an fp32 sum, and the E4M3 scale multiplies the 16-weight sums,
// not the weights (1.1 vector operations per weight and token, against 2 to
// build an MFMA operand).  fp32 activations take fused multiply-adds instead.
// The lanes' sums are added by xor shuffles at the end, in a fixed order.
//
// Measured: one token x (5120 x 17408) 12.7 us, 3.9 TB/s of weights and codes, with
// three such layers in turn, which the last-level cache holds; 14.8 us, 3.4
// TB/s, with sixteen, which it does not (a copy of 2 GiB reaches 4.9).  Bound by
// that read and the launch.
// ---------------------------------------------------------------------------
constexpr int kSpan = 2048;

template <int i>
__device__ __forceinline__ bf16x2_t nibbles2(uint32_t pk) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(pk, 1.0f, i);
}

template <int kTok, int kRows, typename TX, typename TY>
__global__ __launch_bounds__(kThreads) void linear_few_kernel(LinearArgs a, int64_t row_groups) {
  constexpr bool kBf16 = sizeof(TX) == 2;
  constexpr int kXw = kBf16 ? 16 : 32;  // 32-bit words of a lane's 32 activations
  const int64_t tile = blockIdx.x / row_groups;
  const int lane = threadIdx.x & 63;
  Place p;
  if (!place_of<kTok>(a, tile, p)) return;  // the whole workgroup
  const int64_t o0 = ((blockIdx.x - tile * row_groups) * (kThreads / 64) + (threadIdx.x >> 6)) * kRows;
  if (o0 >= a.c_out) return;                // the whole wave (no barrier follows)
  const uint8_t* wq = a.packed + p.g * a.c_out * (a.c_in / 2) + 16 * lane;
  const uint8_t* wc = a.codes + p.g * a.c_out * (a.c_in / 16) + 2 * lane;
  const TX* x = reinterpret_cast<const TX*>(p.x) + 32 * lane;

  struct Span {
    uint4 w[kRows];
    uint32_t c[kRows];
  };
  const int64_t spans = (a.c_in + kSpan - 1) / kSpan;
  auto wload = [&](int64_t s) {
    Span v;
    const int64_t n = a.c_in - s * kSpan - 32 * lane;  // a multiple of 16
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t o = min(o0 + r, a.c_out - 1);
      const uint8_t* q = wq + o * (a.c_in / 2) + s * (kSpan / 2);
      const uint8_t* c = wc + o * (a.c_in / 16) + s * (kSpan / 16);
      v.w[r] = make_uint4(0u, 0u, 0u, 0u);
      v.c[r] = 0;
      if (n >= 32) {
        v.w[r] = load_u128(q);
        uint16_t h;
        __builtin_memcpy(&h, c, 2);
        v.c[r] = h;
      } else if (n >= 16) {
        const uint2 u = load_u64(q);
        v.w[r].x = u.x;
        v.w[r].y = u.y;
        v.c[r] = c[0];
      }
    }
    return v;
  };

  float acc[kRows * kTok] = {};
  Span cur = wload(0);
  for (int64_t s = 0; s < spans; ++s) {
    uint32_t xv[kTok][kXw];
    const int64_t n = a.c_in - s * kSpan - 32 * lane;
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      const TX* xp = x + min(p.row0 + t, p.row1 - 1) * a.ld_x + s * kSpan;
#pragma unroll
      for (int q = 0; q < kXw / 4; ++q) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (n >= (q + 1) * (kBf16 ? 8 : 4)) u = load_u128(xp + q * (kBf16 ? 8 : 4));
        xv[t][4 * q] = u.x; xv[t][4 * q + 1] = u.y; xv[t][4 * q + 2] = u.z; xv[t][4 * q + 3] = u.w;
      }
    }
    const Span next = wload(min(s + 1, spans - 1));
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const uint32_t w[4] = {cur.w[r].x, cur.w[r].y, cur.w[r].z, cur.w[r].w};
      const float c[2] = {e4m3_to_f32<0>(cur.c[r]), e4m3_to_f32<1>(cur.c[r])};
      static_for<2>([&](auto B) {  // the lane's two blocks
        float sum[kTok] = {};
        static_for<2>([&](auto D) {
          constexpr int d = 2 * B + D;  // word of eight weights
          static_for<4>([&](auto P) {
            if constexpr (kBf16) {
              const bf16x2_t u = nibbles2<P>(w[d]);
#pragma unroll
              for (int t = 0; t < kTok; ++t)
                sum[t] = __builtin_amdgcn_fdot2_f32_bf16(u, __builtin_bit_cast(bf16x2_t, xv[t][4 * d + P]), sum[t],
                                                         false);
            } else {
              const f32x2_t u = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[d], 1.0f, P);
#pragma unroll
              for (int t = 0; t < kTok; ++t) {
                sum[t] = __builtin_fmaf(u.x, __uint_as_float(xv[t][8 * d + 2 * P]), sum[t]);
                sum[t] = __builtin_fmaf(u.y, __uint_as_float(xv[t][8 * d + 2 * P + 1]), sum[t]);
              }
            }
          });
        });
#pragma unroll
        for (int t = 0; t < kTok; ++t) acc[r * kTok + t] = __builtin_fmaf(c[B], sum[t], acc[r * kTok + t]);
      });
    }
    cur = next;
  }
  const float v = wave_sums(acc) * out_scale(a, p.g);
  constexpr int kShare = 64 / (kRows * kTok);  // lanes that hold the same sum
  const int r = lane / kShare / kTok, t = lane / kShare % kTok;
  if (lane % kShare == 0 && o0 + r < a.c_out && p.row0 + t < p.row1) {
    TY* y = reinterpret_cast<TY*>(p.y) + (p.row0 + t) * a.ld_y + o0 + r;
    if constexpr (sizeof(TY) == 2) *y = f32_to_bf16_bits(v);
    else *y = v;
  }
}

// Tiles of kBT tokens the grid needs: exact for dense rows, an upper bound
// for ragged ones (a group of n rows has n / kBT full tiles and at most one more).
int64_t token_tiles(const LinearArgs& a, int64_t bt) {
  if (!a.ragged) return (a.rows + bt - 1) / bt * a.n_groups;
  return a.rows / bt + (a.n_groups < a.rows ? a.n_groups : a.rows);
}

// Whether that many workgroups fit one launch, which takes fewer than 2^32
// threads along x (more would wrap around, without an error).
bool one_launch(int64_t m_tiles, int64_t t_tiles, int threads) {
  return (double)m_tiles * (double)t_tiles * threads < 0x1p32;
}

template <bool kGrad, typename TX, typename TY>
hipError_t launch_tile(const LinearArgs& a, hipStream_t stream) {
  const int64_t m = kGrad ? a.c_in : a.c_out;
  const int64_t m_tiles = (m + kT - 1) / kT;
  const int64_t t_tiles = token_tiles(a, kT);
  if (!one_launch(m_tiles, t_tiles, kThreads)) return hipErrorInvalidConfiguration;
  linear_tile_kernel<kGrad, TX, TY><<<dim3((unsigned)(m_tiles * t_tiles)), dim3(kThreads), 0, stream>>>(a, m_tiles);
  return hipGetLastError();
}

template <bool kGrad, typename TX>
hipError_t launch_x(const LinearArgs& a, hipStream_t stream) {
  return a.y_dtype == 1 ? launch_tile<kGrad, TX, uint16_t>(a, stream) : launch_tile<kGrad, TX, float>(a, stream);
}

// ---------------------------------------------------------------------------
// Which kernel, from sizes and types alone.
// ---------------------------------------------------------------------------
struct Plan {
  int few = 0;             // > 0: linear_few_kernel with that many tokens per wave
  int tok = 0, outs = 0;   // tok > 0: the kernel with tiles of that many tokens and outputs
  bool together = false;   // the planes of fp32 rows side by side, not one after the other
  int splits = 1;
  int64_t kp = 0;          // packed row length (one plane), chunks * kChunk / planes
  bool pack = false;       // x goes through pack_rows_kernel
  size_t pack_bytes = 0, part_bytes = 0;
};

// Time of a launch in microseconds, from what its parts measured on MI355X.
// Workgroups that share a CU share its issue slots, so a CU with r of them takes
// `start` + r * (`each` + `more` per chunk or stage), one alone `one` per chunk;
// a split adds a launch and its partial sums' way to memory and back.  The
// constants are fitted to timings of every kernel that comes near, up to 16
// parts, 3 to 32768 tokens (all of them in profiles/product_tiles.md).  What
// they pick is slower than the fastest by 0.8% on the mean of 44 products, 1.2%
// of 19 gradients, 1.7% of 9 experts' products and 2.8% of as many gradients
// (at worst 25%: 2048 rows on 64 experts).  The line of the planes side by side
// is set by hand from a dozen calls.  Some of both sides (weights of 4096 x
// 4096 unless named):
//   product, 16 tokens: 16 x 32 tiles 8.1, 32 x 128 in 6 parts 11.8; 64 tokens on
//     5120 x 17408: 64 x 128 in 6 parts 25.7, in 8 33.6, 64 x 256 in 10 27.0; 512
//     tokens: 64 x 128 25.9, 64 x 256 in 2 parts 29.6; 1024 tokens: 64 x 256
//     40.4, 64 x 128 45.7, 128 x 256 in 2 parts 48.0; 2048 tokens: 128 x 256
//     69.4, 64 x 256 79.8; 4096 tokens: 256 x 256 115, 128 x 256 123; 8192 tokens
//     on 12288 x 4096: 692, 715
//   64 experts of 1024 x 2048, 512 rows: 32 x 128 21.8, 64 x 256 22.1, 64 x 128
//     25.5; 8192 rows: 128 x 256 69, 64 x 256 73, 256 x 256 116; 32768 rows: 178,
//     209, 191
//   gradient (n x 256), 64 tokens on 5120 x 17408: 64 in 6 parts 42.0, 128 in 6
//     43.9, 64 in 16 51; 1024 tokens: 256 in 4 parts 66.5, 128 in 4 68.1, 64 in 2
//     77.9; 4096 tokens: 256 132, 128 155, 64 239; experts, 8192 rows: 128 80, 64
//     99, 256 109
struct TileCost {
  int tok, outs;
  double start, each, one, more;
  bool together = false;  // fp32 rows: a chunk is that of all planes
};
constexpr TileCost kProductCosts[] = {{256, 256, 3.66, 0.22, 2.98, 3.45}, {128, 256, 2.36, 0.16, 1.88, 1.75},
                                      {64, 256, 3.27, 0.17, 0.94, 1.06},  {64, 256, 4.0, 0.2, 2.2, 2.6, true},
                                      {64, 128, 3.43, 0.96, 0.60, 0.61},
                                      {32, kSmallM, 3.77, 1.58, 0.52, 0.53}, {16, kSkinnyM, 3.46, 0.43, 0.11, 0.16}};
constexpr TileCost kGradCosts[] = {{256, kGradM, 4.64, 3.64, 1.80, 1.94},
                                   {128, kGradM, 5.26, 0.34, 1.47, 1.04},
                                   {64, kGradM, 6.15, 0.19, 1.23, 0.83}};
constexpr int kCUs = 256;

double tile_cost(const TileCost& k, double tiles, bool ragged, int64_t chunks, int splits, double part_values) {
  double r = tiles * splits / kCUs;
  // small workgroups even out; of large ones the fullest CU counts, and how
  // ragged rows fill their tiles is only estimated
  if (k.tok > 32) r = ragged ? r + 0.25 : ceil(r);
  const double per = (double)((chunks + splits - 1) / splits);
  double t = k.start + (r <= 1.0 ? k.each + k.one * per : r * (k.each + k.more * per));
  if (splits > 1) t += 2.5 + splits * part_values * 8e-6 / 4.0;
  return t;
}

// The cheapest kernel and number of parts for a.  parts: whether there is a
// place for partial sums (up to 16 parts then; 32 tokens on 4096 x 17408 weights
// without one: 16 x 32 tiles 22.5 us, the 64 x 256 chosen with parts 125).
template <int kN>
void cheapest(Plan& p, const LinearArgs& a, const TileCost (&costs)[kN], int planes, int64_t plane_chunks, bool parts) {
  const int64_t all = a.ragged ? a.rows : a.rows * a.n_groups, m = a.grad ? a.c_in : a.c_out;
  double best = 0.0;
  for (const TileCost& k : costs) {
    if (k.together && planes == 1) continue;
    const int64_t chunks = k.together ? plane_chunks : planes * plane_chunks;
    const int64_t m_tiles = (m + k.outs - 1) / k.outs;
    // ragged: about half of a tile more per group that has rows than the rows
    // fill, and a tile at least; with a bound on a group's rows the groups that
    // have any are taken half way between as few and as many as there can be
    double used = (double)(a.n_groups < a.rows ? a.n_groups : a.rows);
    if (a.ragged && a.max_group_rows > 0 && a.max_group_rows < a.rows)
      used = 0.5 * used + 0.5 * fmin(used, (double)a.rows / a.max_group_rows);
    const double t_tiles = a.ragged ? fmax(used, (double)a.rows / k.tok + 0.5 * used)
                                    : (double)((a.rows + k.tok - 1) / k.tok * a.n_groups);
    for (int splits = 1; splits <= (parts && !a.ragged ? 16 : 1) && splits <= chunks; ++splits) {
      const double t = tile_cost(k, t_tiles * m_tiles, a.ragged, chunks, splits, (double)all * m);
      if (p.tok == 0 || t < best) {
        best = t;
        p.tok = k.tok;
        p.outs = k.outs;
        p.together = k.together;
        p.splits = splits;
      }
    }
  }
}

// parts: whether the call has a workspace, as linear_ws_bytes has it for its answer.
Plan plan_of(const LinearArgs& a, bool parts) {
  Plan p;
  if (a.rows <= 0 || a.c_in <= 0 || a.c_out <= 0) return p;
  // Up to two tokens, or eight ragged rows: linear_few_kernel (5120 x 17408
  // weights, one token: 12.9 us against 21.5; 12288 x 4096, two tokens: 9.6
  // against 13.0, four tokens 13.1 against 13.0; eight rows on 64 experts of
  // 1024 x 2048: 4.7 against 6.0).
  if (!a.grad && a.rows <= (a.ragged ? 8 : 2)) {
    p.few = a.ragged ? 1 : (int)a.rows;
    return p;
  }
  const int planes = a.x_dtype == 1 ? 1 : 3;
  const int64_t k = a.grad ? a.c_out : a.c_in, step = a.grad ? kGradK : kChunk;
  const int64_t all = a.ragged ? a.rows : a.rows * a.n_groups;
  p.kp = (k + step - 1) / step * step;
  p.pack = planes == 3 || k % step != 0;
  if (a.grad) cheapest(p, a, kGradCosts, planes, p.kp / step, parts);
  else cheapest(p, a, kProductCosts, planes, p.kp / step, parts);
  if (p.pack) p.pack_bytes = ((size_t)all * planes * p.kp * 2 + 255) / 256 * 256;
  if (p.splits > 1) p.part_bytes = (size_t)p.splits * all * (a.grad ? a.c_in : a.c_out) * 4;
  return p;
}

template <int kTok, int kRows, typename TX, typename TY>
hipError_t launch_few_typed(const LinearArgs& a, hipStream_t stream) {
  const int64_t per = kRows * (kThreads / 64);
  const int64_t row_groups = (a.c_out + per - 1) / per;
  const int64_t t_tiles = token_tiles(a, kTok);
  if (!one_launch(row_groups, t_tiles, kThreads)) return hipErrorInvalidConfiguration;
  linear_few_kernel<kTok, kRows, TX, TY><<<dim3((unsigned)(row_groups * t_tiles)), dim3(kThreads), 0, stream>>>(
      a, row_groups);
  return hipGetLastError();
}
// Rows per wave: two for one bf16 token (5120 x 17408: 12.9 us, four rows
// 14.6), four where the activations in registers weigh more (two tokens,
// 12288 x 4096: 9.6, two rows 10.5; one fp32 token: 11.8 and 15.2).
template <int kTok, typename TX>
hipError_t launch_few_y(const LinearArgs& a, hipStream_t stream) {
  constexpr int kRows = kTok == 1 && sizeof(TX) == 2 ? 2 : 4;
  return a.y_dtype == 1 ? launch_few_typed<kTok, kRows, TX, uint16_t>(a, stream)
                        : launch_few_typed<kTok, kRows, TX, float>(a, stream);
}
template <int kTok>
hipError_t launch_few_x(const LinearArgs& a, hipStream_t stream) {
  return a.x_dtype == 1 ? launch_few_y<kTok, uint16_t>(a, stream) : launch_few_y<kTok, float>(a, stream);
}
hipError_t launch_few(const LinearArgs& a, int tok, hipStream_t stream) {
  switch (tok) {
    case 1: return launch_few_x<1>(a, stream);
    default: return launch_few_x<2>(a, stream);
  }
}

template <int kNT, int kRF, int kMW, int kDepth, int kWaves, int kP = 1>
hipError_t launch_big_nt(const BigArgs& b, hipStream_t stream) {
  const dim3 grid((unsigned)(b.m_tiles * b.t_tiles), (unsigned)b.splits), block(64 * kMW);
  if (b.a.c_in % kChunk == 0)
    linear_big_kernel<kNT, kRF, kMW, kDepth, kWaves, kP, false><<<grid, block, 0, stream>>>(b);
  else
    linear_big_kernel<kNT, kRF, kMW, kDepth, kWaves, kP, true><<<grid, block, 0, stream>>>(b);
  return hipGetLastError();
}


// Whether rows of packed weights are whole 16-byte pieces and the codes whole pairs.
bool whole_pieces(const LinearArgs& a) {
  return a.c_in % 32 == 0 && reinterpret_cast<uintptr_t>(a.packed) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(a.codes) % 2 == 0;
}

template <int kW, int kBufs>
hipError_t launch_skinny(const BigArgs& b, hipStream_t stream) {
  const dim3 grid((unsigned)(b.m_tiles * b.t_tiles), (unsigned)b.splits);
  if (whole_pieces(b.a)) linear_skinny_kernel<kW, kBufs, false><<<grid, dim3(64 * kW), 0, stream>>>(b);
  else linear_skinny_kernel<kW, 2, true><<<grid, dim3(64 * kW), 0, stream>>>(b);
  return hipGetLastError();
}

template <int kBufs>
hipError_t launch_small(const BigArgs& b, hipStream_t stream) {
  const dim3 grid((unsigned)(b.m_tiles * b.t_tiles), (unsigned)b.splits);
  if (whole_pieces(b.a)) linear_small_kernel<kBufs, false><<<grid, dim3(512), 0, stream>>>(b);
  else linear_small_kernel<kBufs, true><<<grid, dim3(512), 0, stream>>>(b);
  return hipGetLastError();
}

template <int kNT, int kDepth, int kWaves>
hipError_t launch_grad_nt(const GradArgs& b, hipStream_t stream) {
  const dim3 grid((unsigned)(b.m_tiles * b.t_tiles), (unsigned)b.splits);
  if (b.a.c_in % 32 == 0 && reinterpret_cast<uintptr_t>(b.a.packed) % 16 == 0)
    grad_big_kernel<kNT, kDepth, kWaves, false><<<grid, dim3(kThreads), 0, stream>>>(b);
  else
    grad_big_kernel<kNT, kDepth, kWaves, true><<<grid, dim3(kThreads), 0, stream>>>(b);
  return hipGetLastError();
}

// The rows of x as the large kernels take them: themselves, or packed into the workspace.
struct Rows {
  const uint16_t* x;
  int64_t ld, gstride;
};
hipError_t pack_rows(const LinearArgs& a, const Plan& p, Rows& r, hipStream_t stream) {
  if (!p.pack) {
    r = Rows{static_cast<const uint16_t*>(a.x), a.ld_x, a.gstride_x};
    return hipSuccess;
  }
  const int planes = a.x_dtype == 1 ? 1 : 3;
  const int64_t groups = a.ragged ? 1 : a.n_groups, k = a.grad ? a.c_out : a.c_in;
  uint16_t* out = static_cast<uint16_t*>(a.ws);
  r = Rows{out, planes * p.kp, a.rows * planes * p.kp};
  const dim3 grid = grid_of((a.rows * groups * (p.kp / 8) + kThreads - 1) / kThreads);
  if (planes == 3)
    pack_rows_kernel<float><<<grid, dim3(kThreads), 0, stream>>>(static_cast<const float*>(a.x), a.rows, k, a.ld_x,
                                                                 groups, a.gstride_x, p.kp, out);
  else
    pack_rows_kernel<uint16_t><<<grid, dim3(kThreads), 0, stream>>>(static_cast<const uint16_t*>(a.x), a.rows, k,
                                                                    a.ld_x, groups, a.gstride_x, p.kp, out);
  return hipGetLastError();
}

hipError_t sum_splits(const LinearArgs& a, const Plan& p, const float* part, hipStream_t stream) {
  const int64_t groups = a.ragged ? 1 : a.n_groups, cols = a.grad ? a.c_in : a.c_out;
  const dim3 grid = grid_of((a.rows * groups * ((cols + 3) / 4) + kThreads - 1) / kThreads);
  if (a.y_dtype == 1)
    split_sum_kernel<uint16_t><<<grid, dim3(kThreads), 0, stream>>>(
        part, p.splits, a.rows, groups, cols, static_cast<uint16_t*>(a.y), a.ld_y, a.gstride_y);
  else
    split_sum_kernel<float><<<grid, dim3(kThreads), 0, stream>>>(part, p.splits, a.rows, groups, cols,
                                                                 static_cast<float*>(a.y), a.ld_y, a.gstride_y);
  return hipGetLastError();
}

hipError_t launch_big(const LinearArgs& a, const Plan& p, hipStream_t stream) {
  const int planes = a.x_dtype == 1 ? 1 : 3;
  const int64_t m_tiles = ((a.grad ? a.c_in : a.c_out) + p.outs - 1) / p.outs;
  int64_t t_tiles = token_tiles(a, p.tok);
  if (a.ragged) t_tiles = (t_tiles + 7) / 8 * 8;
  if (!one_launch(m_tiles, t_tiles, 512)) return hipErrorInvalidConfiguration;  // 512: the most threads of any tile
  Rows r;
  hipError_t e = pack_rows(a, p, r, stream);
  if (e != hipSuccess) return e;
  float* const part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + p.pack_bytes);
  if (a.grad) {
    const int w_stages = (int)(p.kp / kGradK);
    const GradArgs b{a, r.x, r.ld, r.gstride, planes * w_stages, w_stages, m_tiles, t_tiles, p.splits, part};
    switch (p.tok) {
      case 256: e = launch_grad_nt<4, 2, 1>(b, stream); break;
      case 128: e = launch_grad_nt<2, 1, 2>(b, stream); break;
      default: e = launch_grad_nt<1, 2, 2>(b, stream); break;
    }
  } else {
    const int w_chunks = (int)(p.kp / kChunk);
    const BigArgs b{a, r.x, r.ld, r.gstride, p.together ? w_chunks : planes * w_chunks, w_chunks, m_tiles, t_tiles,
                    p.splits, part};
    switch (p.tok) {
      case 256: e = launch_big_nt<8, 2, 4, 1, 1>(b, stream); break;
      case 128: e = launch_big_nt<4, 2, 4, 1, 2>(b, stream); break;
      case 64:
        e = p.together      ? launch_big_nt<2, 1, 8, 1, 2, 3>(b, stream)
            : p.outs == 256 ? launch_big_nt<2, 1, 8, 2, 2>(b, stream)
                            : launch_big_nt<2, 1, 4, 4, 2>(b, stream);
        break;
      case 32: e = launch_small<2>(b, stream); break;
      default: e = launch_skinny<4, 3>(b, stream); break;
    }
  }
  if (e != hipSuccess || p.splits == 1) return e;
  return sum_splits(a, p, part, stream);
}

// Whether the kernels with direct loads take a: rows that they can load
// themselves (or packed ones), and offsets within a tile in 32 bits.  The
// general kernel takes the rest.
bool direct_rows(const LinearArgs& a, const Plan& p) {
  const int planes = a.x_dtype == 1 ? 1 : 3;
  if ((p.pack ? planes * p.kp : a.ld_x) >= (1 << 22) || a.c_in >= (1 << 28)) return false;
  if (p.pack) return a.ws != nullptr;
  return reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (a.ld_x % 8 == 0 || a.rows == 1) && a.gstride_x % 8 == 0;
}

}  // namespace

size_t linear_ws_bytes(const LinearArgs& a) {
  const Plan p = plan_of(a, true);
  return p.pack_bytes + p.part_bytes;
}

hipError_t launch_linear(const LinearArgs& a, hipStream_t stream) {
  const Plan p = plan_of(a, a.ws != nullptr);
  if (p.few > 0) return launch_few(a, p.few, stream);
  if (p.tok > 0 && direct_rows(a, p)) return launch_big(a, p, stream);
  if (a.grad) return a.x_dtype == 1 ? launch_x<true, uint16_t>(a, stream) : launch_x<true, float>(a, stream);
  return a.x_dtype == 1 ? launch_x<false, uint16_t>(a, stream) : launch_x<false, float>(a, stream);
}

}  // namespace lh
