// gfx950 matrix-vector products with 4-bit weights and group scales.
//
// Per (row n, group g) of W, with codes c, scale d, zero z and a row x:
//     sum_k d (c_k - z) x_k = d ( sum_k (16 + c_k) x_k  -  (16 + z) sum_k x_k )
// A code planted below the exponent of 16.0 is the 16-bit float 16 + c, one
// shift and one and-or per two codes, with no conversion; the matrix
// instruction multiplies them by x exactly and sums in fp32, starting from
// -(16 + z) sum x, so what is scaled by d is the difference itself (16, the
// smallest base that leaves four mantissa bits, keeps the cancellation small).
// The 16 weight rows of a tile are the instruction's rows and up to 16 rows of
// x its columns: with one row of x 15 columns are idle, but the instruction is
// not what bounds the product -- the bytes of W are, then the unpacking.
//
// Measured (bf16 x; bytes of codes, scales and zeros):
//     131072 x 5120, group 32, 1 row                 74 us   5.1 TB/s
//     the same, group 64 and zeros, 8 rows           94 us   3.9 TB/s
//     384 of 4608 x 5120, group 64 and zeros, SwiGLU,
//       8 rows of 6 ids (45 matrices chosen)        118 us   4.6 TB/s
//     5120 x 5120, group 32, 1 row                  8.9 us   latency: one load's
//       round trip, the sum across waves, the launch
//     32768 x 5120, group 64 and zeros, 16 | 64 rows   37 | 133 us: unpacking
//       and matrix instructions
#include <hip/hip_runtime.h>

#include <cstdint>

#include "dev_common.h"
#include "group.h"

namespace moe {
namespace grp {

typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
using dev::u32x2;
using dev::u32x4;
#define MOE_Q4_LDS __attribute__((address_space(3)))

// A workgroup of eight waves takes a few row tiles of one matrix.  The waves
// split the columns, in tiles of 128 dealt in turn (with fewer than eight
// column tiles, they split the row tiles too).  For a column tile a wave reads
// its piece of x from LDS once and multiplies T row tiles by it; loads for T
// row tiles times D column tiles ahead are in flight in a ring of registers,
// the first of them issued before the rows of x are staged in LDS.  Partial
// sums meet in LDS once, at the end, and are added in a fixed order.
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
// LDS for x and for partial sums: together with the list of rows 80 KB, so
// that two workgroups share a compute unit (128 KB for the 64-row form).  The
// sums take 64 bytes a row of x, row tile, half of a SwiGLU and wave.
constexpr int kLds = (80 << 10) - 256, kLdsMany = 128 << 10;
struct Q4 {
  const uint16_t* x;
  const int32_t* idx;
  const uint8_t* codes;
  const uint8_t* scales;
  const uint8_t* zeros;
  void* y;
  int64_t ldx, ldy;
  int n, k, rows, x_div, n_mats, out_type;
  int tn, tk;               // tiles of a matrix; with SwiGLU tn counts the gate's
  int split, split_log2;    // waves along the columns (a power of two)
  int x_bytes;              // LDS for x; the rest is for partial sums
};

template <bool BF>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Codes 0 .. 7 of a word as 16 + c, in the order (0,4) (1,5) (2,6) (3,7).
// `base` holds the exponent bits of 16.0 twice, in a register that the compiler
// cannot see through: with two literals it would split each and-or in two.
// (Written as inline assembly, the and-or escapes the compiler's count of the
// cycles that a matrix instruction goes on reading its addend, and may
// overwrite it: seen as wrong sums where two products share one addend.)
template <bool BF>
__device__ __forceinline__ uint32_t opaque_base() {
  uint32_t b = BF ? 0x41804180u : 0x4C004C00u;
  asm("" : "+v"(b));
  return b;
}
template <bool BF>
__device__ __forceinline__ u32x4 unpack8(uint32_t w, uint32_t base) {
  constexpr int at = BF ? 3 : 6;                     // lowest of the top four mantissa bits
  constexpr uint32_t mask = 0x000F000Fu << at;
  return u32x4{((w << at) & mask) | base, ((BF ? w >> 1 : w << 2) & mask) | base, ((w >> (8 - at)) & mask) | base,
               ((w >> (12 - at)) & mask) | base};
}

// Eight values of x in the same order.
__device__ __forceinline__ u32x4 order8(u32x4 x) {
  return u32x4{(x[0] & 0xFFFFu) | x[2] << 16, x[0] >> 16 | (x[2] & 0xFFFF0000u), (x[1] & 0xFFFFu) | x[3] << 16,
               x[1] >> 16 | (x[3] & 0xFFFF0000u)};
}

// -(16 + z) in every element: its product with x is what the codes' base and
// zero add to the sum, exact in 16 bits for z = 0 .. 15.
template <bool BF>
__device__ __forceinline__ u32x4 offset8(uint32_t z) {
  // bf16: 16 + z = 0x41800000 + z * 2^19 as fp32 bits; f16: 0x4C00 + z * 2^6
  const uint32_t h = BF ? 0xC180u + (z << 3) : 0xCC00u + (z << 6);
  const uint32_t w = h | h << 16;
  return u32x4{w, w, w, w};
}

// The value that lane g (0 .. 3) of each row of 16 lanes holds, in all of them.
__device__ __forceinline__ f16x4 lane_of_row(u32x2 v, int g) {
  u32x2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r[i] = g == 0   ? __builtin_amdgcn_mov_dpp(v[i], 0x150, 0xF, 0xF, true)
           : g == 1 ? __builtin_amdgcn_mov_dpp(v[i], 0x151, 0xF, 0xF, true)
           : g == 2 ? __builtin_amdgcn_mov_dpp(v[i], 0x152, 0xF, 0xF, true)
                    : __builtin_amdgcn_mov_dpp(v[i], 0x153, 0xF, 0xF, true);
  return __builtin_bit_cast(f16x4, r);
}

__device__ __forceinline__ void put(void* y, int64_t at, float v, int type) {
  if (type == MOE_T_F32) static_cast<float*>(y)[at] = v;
  else if (type == MOE_T_BF16) static_cast<uint16_t*>(y)[at] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else static_cast<uint16_t*>(y)[at] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

// The rows of y that workgroup row `lead` computes (a bit each) and their
// matrix: with idx, the rows that chose the matrix of row `lead`, or none if
// an earlier row leads them.
__device__ __forceinline__ uint64_t rows_of(const Q4& a, int lead, int& mat) {
  if (!a.idx) {
    mat = 0;
    return a.rows >= 64 ? ~0ull : (1ull << a.rows) - 1;
  }
  const int lane = threadIdx.x & 63;
  const int id = lane < a.rows ? a.idx[lane] : INT32_MIN;
  mat = __builtin_amdgcn_readlane(id, lead);
  const uint64_t same = __ballot(lane < a.rows && id == mat);
  return (same & ((1ull << lead) - 1)) ? 0 : same;
}

// The c-th set bit of m, or -1.
__device__ __forceinline__ int nth_row(uint64_t m, int c) {
  for (int i = 0; i < c && m; ++i) m &= m - 1;
  return m ? __ffsll(static_cast<unsigned long long>(m)) - 1 : -1;
}

// CT: column tiles of 16 rows of x.  (Rows that chose one matrix: 16 at a
// time.)  T row tiles a wave, D column tiles ahead.  Four row tiles a wave (two
// with SwiGLU) against one: 131072 x 5120 95 -> 78 us, as a piece of x is read and
// its base summed once for all; six or eight spill registers.  64 rows of 32768 x
// 5120, two row tiles a wave against one: 218 -> 134 us.
template <bool BF, int G, bool Z, bool SW, int CT, int T, int D>
__global__ __launch_bounds__(kThreads, CT > 1 ? 2 : 4) void k_q4(Q4 a) {
  constexpr int H = SW ? 2 : 1;
  constexpr int kPer = 128 / G;          // groups of a tile
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int member[CT * 16];        // the row of y in each column
  const int tid = threadIdx.x, lane = tid & 63, wave = dev::uniform(tid >> 6), col = lane & 15, q = lane >> 4;
  const uint32_t unit = opaque_base<BF>();
  int mat;
  const uint64_t all = rows_of(a, blockIdx.y, mat);
  if (!all) return;
  const int out_n = SW ? a.n / 2 : a.n;
  const int per_wg = T * kWaves >> a.split_log2;
  const int tile0 = blockIdx.x * per_wg, tiles = a.tn - tile0 < per_wg ? a.tn - tile0 : per_wg;
  if (mat < 0 || mat >= a.n_mats) {                 // no matrix: zeros for -1, else NaN
    for (uint64_t m = all; m; m &= m - 1) {
      const int p = __ffsll(static_cast<unsigned long long>(m)) - 1;
      for (int i = tid; i < tiles * 16; i += kThreads)
        if (tile0 * 16 + i < out_n) put(a.y, p * a.ldy + tile0 * 16 + i, mat == -1 ? 0.0f : __builtin_nanf(""), a.out_type);
    }
    return;
  }
  const int64_t mat_tiles = static_cast<int64_t>(a.tn) * H * a.tk;
  const u32x4* codes = reinterpret_cast<const u32x4*>(a.codes + mat * mat_tiles * 1024) + lane;
  // lane g of a row of 16 lanes loads the scales of group g for the row's four outputs
  const uint8_t* scales = a.scales + mat * mat_tiles * kPer * 32 + (col & (kPer - 1)) * 32 + q * 8;
  const uint8_t* zeros = Z ? a.zeros + mat * mat_tiles * kPer * 16 + col : nullptr;
  const int ks = wave & (a.split - 1), first_tile = (wave >> a.split_log2) * T;
  MOE_Q4_LDS uint8_t* xl = (MOE_Q4_LDS uint8_t*)lds;
  MOE_Q4_LDS f32x4* part = (MOE_Q4_LDS f32x4*)(lds + a.x_bytes);

  for (uint64_t rest = all; rest;) {
    const uint64_t rows = rest;
    const int left = __popcll(rows), count = left < CT * 16 ? left : CT * 16;
    // x chunk (eight columns) c of column j lies at (c * held + j) * 16; lanes
    // past the last column repeat one (their products belong to no row)
    const int log_held = CT > 1 ? 6 : count <= 1 ? 0 : count <= 2 ? 1 : count <= 4 ? 2 : count <= 8 ? 3 : 4, held = 1 << log_held;
    const int span = a.x_bytes >> (log_held + 8) >> a.split_log2 << a.split_log2;   // column tiles of x at a time
    if (rest != all) __syncthreads();
    if (tid < CT * 16) member[tid] = nth_row(rows, tid);
    for (int i = 0; i < CT * 16; ++i) rest &= rest - 1;

    f32x4 out[T][H][CT] = {};
    for (int k0 = 0; k0 < a.tk; k0 += span) {
      const int kn = a.tk - k0 < span ? a.tk - k0 : span;        // column tiles of this pass
      const int each = (kn - ks + a.split - 1) >> a.split_log2;  // of which this wave's

      u32x4 w[D][T][H];
      u32x2 d[D][T][H];
      uint8_t z[D][T][H][kPer];
      // Column tile `i` of this wave's; past the last the loads repeat it, as
      // row tiles past the matrix repeat its last: without a branch around
      // them the compiler knows how many are in flight and waits for the
      // oldest only.
      const auto load = [&](int s, int t, int i) {
        const int kt = k0 + ks + (i < each ? i : each - 1) * a.split;
        const int row = tile0 + first_tile + t;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const int64_t at = static_cast<int64_t>((row < a.tn ? row : a.tn - 1) + h * a.tn) * a.tk + kt;
          w[s][t][h] = codes[at * 64];
          d[s][t][h] = *reinterpret_cast<const u32x2*>(scales + at * kPer * 32);
          if constexpr (Z)
#pragma unroll
            for (int g = 0; g < kPer; ++g) z[s][t][h][g] = zeros[(at * kPer + g) * 16];
        }
      };
      if (each > 0) {
#pragma unroll
        for (int s = 0; s < D; ++s)
#pragma unroll
          for (int t = 0; t < T; ++t) load(s, t, s);
      }

      __syncthreads();                                           // x of the last pass is used, member is there
      for (int c = tid; c < kn * 16 << log_held; c += kThreads) {
        const int k = (k0 * 16 + (c >> log_held)) * 8, p = member[c & (held - 1)];
        if (p < 0) continue;
        u32x4 v{0, 0, 0, 0};
        if (k < a.k) __builtin_memcpy(&v, a.x + (a.x_div == 1 ? p : p / a.x_div) * a.ldx + k, 16);
        *reinterpret_cast<MOE_Q4_LDS u32x4*>(xl + c * 16) = order8(v);
      }
      __syncthreads();

      const MOE_Q4_LDS uint8_t* xq = xl + ((q << log_held) + (CT > 1 ? col : col & (held - 1))) * 16;
      for (int i0 = 0; i0 < each; i0 += D) {
#pragma unroll
        for (int s = 0; s < D; ++s) {
          if (i0 + s >= each) break;
          const MOE_Q4_LDS uint8_t* xt = xq + ((ks + (i0 + s) * a.split) * 256 << log_held);
          u32x4 xv[4][CT];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int c = 0; c < CT; ++c)
              xv[j][c] = *reinterpret_cast<const MOE_Q4_LDS u32x4*>(xt + ((j * 64 << log_held) + c * 256));
          // symmetric: what base and zero add is the same for every row tile
          f32x4 start[kPer][CT];
#pragma unroll
          for (int g = 0; g < kPer; ++g)
#pragma unroll
            for (int c = 0; c < CT; ++c) {
              start[g][c] = f32x4{0, 0, 0, 0};
              if constexpr (!Z)
#pragma unroll
                for (int j = 0; j < G / 32; ++j) start[g][c] = mma<BF>(offset8<BF>(8), xv[g * (G / 32) + j][c], start[g][c]);
            }
#pragma unroll
          for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int h = 0; h < H; ++h) {
#pragma unroll
              for (int g = 0; g < kPer; ++g) {
                f32x4 acc[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[c] = start[g][c];
#pragma unroll
                for (int j = 0; j < G / 32; ++j) {
                  const u32x4 code = unpack8<BF>(w[s][t][h][g * (G / 32) + j], unit);
#pragma unroll
                  for (int c = 0; c < CT; ++c) {
                    if constexpr (Z) acc[c] = mma<BF>(offset8<BF>(z[s][t][h][g]), xv[g * (G / 32) + j][c], acc[c]);
                    acc[c] = mma<BF>(code, xv[g * (G / 32) + j][c], acc[c]);
                  }
                }
                const f16x4 scale = lane_of_row(d[s][t][h], g);
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                  for (int i = 0; i < 4; ++i) out[t][h][c][i] += static_cast<float>(scale[i]) * acc[c][i];
              }
            }
            load(s, t, i0 + s + D);
          }
        }
      }
    }
    // [row tile][half][wave along the columns][quarter][column]
    if (CT > 1 || col < held) {
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int c = 0; c < CT; ++c)
            part[((((((first_tile + t) * H + h) << a.split_log2) | ks) * 4 + q) << log_held) + c * 16 + col] = out[t][h][c];
    }
    __syncthreads();

    // one thread per output: row r of a tile, column j
    const MOE_Q4_LDS float* sums = reinterpret_cast<const MOE_Q4_LDS float*>(part);
    for (int i = tid; i < tiles * 16 << log_held; i += kThreads) {
      const int r = i & 15, j = (i >> 4) & (held - 1), t = i >> (4 + log_held);
      if (j >= count) continue;
      float v[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        v[h] = 0.0f;
        for (int s = 0; s < a.split; ++s)
          v[h] += sums[((((((t * H + h) << a.split_log2) | s) * 4 + (r >> 2)) << log_held) + j) * 4 + (r & 3)];
      }
      float o = v[0];
      if constexpr (SW) o = o / (1.0f + __expf(-o)) * v[1];
      const int c = (tile0 + t) * 16 + r, p = member[j];
      if (c < out_n) put(a.y, p * a.ldy + c, o, a.out_type);
    }
  }
}

namespace {

// Waves along the columns: as many as there are column tiles, and as a column
// tile each of x fits in LDS (`held` rows take held * 256 bytes).
int split_of(int tk, int held, int x_bytes) {
  const int fit = x_bytes / (held * 256);
  return tk >= 8 && fit >= 8 ? 3 : tk >= 4 && fit >= 4 ? 2 : tk >= 2 && fit >= 2 ? 1 : 0;
}

template <bool BF, int G, bool Z, bool SW, int CT, int T, int D>
void run(Q4 a, int held, int lds, hipStream_t s) {
  constexpr int H = SW ? 2 : 1;
  a.split_log2 = split_of(a.tk, held, a.x_bytes);
  a.split = 1 << a.split_log2;
  const int per_wg = T * kWaves >> a.split_log2;
  // the sums of the workgroup: always kWaves * T * H KB at most for 16 rows
  static_assert(CT * kWaves * T * H <= 64, "the partial sums fit");
  (void)H;
  const dim3 grid((a.tn + per_wg - 1) / per_wg, a.idx ? a.rows : 1);
  hipLaunchKernelGGL((k_q4<BF, G, Z, SW, CT, T, D>), grid, dim3(kThreads), lds, s, a);
}

template <bool BF, int G, bool Z, bool SW>
void go(Q4 a, hipStream_t s) {
  constexpr int H = SW ? 2 : 1;
  if (SW) a.tn /= 2;
  // rows of one matrix: 16 columns of the instruction, or four times 16
  const bool many = !a.idx && a.rows > 16;
  int held = many ? 64 : 1;
  while (held < 16 && held < a.rows) held *= 2;
  if (many) {
    a.x_bytes = 64 << 10;
    run<BF, G, Z, SW, 4, 2 / H, 1>(a, held, kLdsMany, s);
    return;
  }
  // several row tiles a wave as long as every compute unit has two workgroups
  constexpr int T = 4 / H;
  const int64_t mats = a.idx ? (a.rows < a.n_mats ? a.rows : a.n_mats) : 1;
  const int sums = kWaves * H * held * 64;        // bytes, times the row tiles of a wave
  a.x_bytes = (kLds - T * sums) & ~255;
  const int waves_tile = kWaves >> split_of(a.tk, held, a.x_bytes);
  if (mats * a.tn >= 512 * T * waves_tile) {
    run<BF, G, Z, SW, 1, T, 1>(a, held, kLds, s);
  } else {
    a.x_bytes = (kLds - sums) & ~255;
    run<BF, G, Z, SW, 1, 1, Z && SW && G == 32 ? 1 : T>(a, held, kLds, s);   // (registers)
  }
}

template <bool BF, int G>
void go(const Q4& a, bool swiglu, hipStream_t s) {
  if (a.zeros) {
    if (swiglu) go<BF, G, true, true>(a, s);
    else go<BF, G, true, false>(a, s);
  } else {
    if (swiglu) go<BF, G, false, true>(a, s);
    else go<BF, G, false, false>(a, s);
  }
}

template <bool BF>
void go(const Q4& a, int group, bool swiglu, hipStream_t s) {
  if (group == 32) go<BF, 32>(a, swiglu, s);
  else if (group == 64) go<BF, 64>(a, swiglu, s);
  else go<BF, 128>(a, swiglu, s);
}

}  // namespace
}  // namespace grp
}  // namespace moe

extern "C" int moe_q4_matvec(const moe_q4_dims* d, const void* x, const int32_t* idx, const void* codes,
                             const void* scales, const void* zeros, void* y, void* stream) {
  using namespace moe::grp;
  if (int st = check_q4(d)) return st;
  if (d->rows == 0) return MOE_OK;
  if (!x || !codes || !scales || !y) return MOE_EINVAL;
  for (const void* p : {codes, scales, zeros})
    if (reinterpret_cast<uintptr_t>(p) % 16) return MOE_EINVAL;
  Q4 a{};
  a.x = static_cast<const uint16_t*>(x);
  a.idx = idx;
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = static_cast<const uint8_t*>(scales);
  a.zeros = static_cast<const uint8_t*>(zeros);
  a.y = y;
  a.ldx = d->ldx;
  a.ldy = d->ldy;
  a.n = d->n;
  a.k = d->k;
  a.rows = d->rows;
  a.x_div = d->x_div;
  a.n_mats = d->n_mats;
  a.out_type = d->out_type;
  a.tn = static_cast<int>(q4_tiles_n(d->n));
  a.tk = static_cast<int>(q4_tiles_k(d->k));
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (d->type == MOE_T_BF16) go<true>(a, d->group, d->swiglu, s);
  else go<false>(a, d->group, d->swiglu, s);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EDEVICE;
}
