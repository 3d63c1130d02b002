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
using dev::u32x4;

constexpr int kQ4Waves = 4;

struct Q4 {
  const uint16_t* x;
  const int32_t* idx;
  const uint8_t* codes;
  const uint8_t* scales;
  const uint8_t* zeros;
  void* y;
  int64_t ldx, ldy;
  int n, k, rows, x_div, n_mats, out_type;
  int tn, tk;               // tiles of a matrix
};

template <bool BF>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Codes 0 .. 7 of a word as 16 + c, in the order (0,4) (1,5) (2,6) (3,7).
template <bool BF>
__device__ __forceinline__ u32x4 unpack8(uint32_t w) {
  constexpr int at = BF ? 3 : 6;                     // lowest of the top four mantissa bits
  constexpr uint32_t mask = 0x000F000Fu << at, base = BF ? 0x41804180u : 0x4C004C00u;
  u32x4 v;
  v[0] = dev::andor(w << at, mask, base);
  v[1] = BF ? dev::andor(w >> 1, mask, base) : dev::andor(w << 2, mask, base);
  v[2] = dev::andor(w >> (8 - at), mask, base);
  v[3] = dev::andor(w >> (12 - at), mask, base);
  return v;
}

// Eight values of x in the same order, and their sum.
template <bool BF>
__device__ __forceinline__ u32x4 order8(u32x4 x, float& sum) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF) s += dev::bf16_bits_to_f32(x[i] & 0xFFFFu) + dev::bf16_bits_to_f32(x[i] >> 16);
    else s += dev::h2_lo(x[i]) + dev::h2_hi(x[i]);
  }
  sum = s;
  return u32x4{(x[0] & 0xFFFFu) | x[2] << 16, x[0] >> 16 | (x[2] & 0xFFFF0000u), (x[1] & 0xFFFFu) | x[3] << 16,
               x[1] >> 16 | (x[3] & 0xFFFF0000u)};
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

template <bool BF, int G, bool Z, bool SW>
__global__ __launch_bounds__(64 * kQ4Waves) void k_q4(Q4 a) {
  constexpr int H = SW ? 2 : 1;
  __shared__ f32x4 part[kQ4Waves][H][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = dev::uniform(tid >> 6), col = lane & 15, q = lane >> 4;
  int mat;
  uint64_t rows = rows_of(a, blockIdx.y, mat);
  if (!rows) return;
  const int out_n = SW ? a.n / 2 : a.n;
  if (mat < 0 || mat >= a.n_mats) {                 // no matrix: zeros for -1, else NaN
    for (; rows; rows &= rows - 1) {
      const int p = __ffsll(static_cast<unsigned long long>(rows)) - 1, c = blockIdx.x * 16 + tid;
      if (tid < 16 && c < out_n) put(a.y, p * a.ldy + c, mat == -1 ? 0.0f : __builtin_nanf(""), a.out_type);
    }
    return;
  }
  const int64_t tiles = static_cast<int64_t>(a.tn) * a.tk;
  constexpr int kPer = 128 / G;                     // groups of a tile
  const u32x4* codes = reinterpret_cast<const u32x4*>(a.codes + mat * tiles * 1024);
  const uint8_t* scales = a.scales + mat * tiles * kPer * 32;
  const uint8_t* zeros = Z ? a.zeros + mat * tiles * kPer * 16 : nullptr;
  for (; rows;) {
    const int p = nth_row(rows, col);
    const uint16_t* x = a.x + (p < 0 ? 0 : p / a.x_div) * a.ldx;
    f32x4 out[H] = {};
    for (int kt = wave; kt < a.tk; kt += kQ4Waves) {
      u32x4 xv[4];
      float sum[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = kt * 128 + j * 32 + q * 8;
        u32x4 v{0, 0, 0, 0};
        if (p >= 0 && k < a.k) __builtin_memcpy(&v, x + k, 16);
        xv[j] = order8<BF>(v, sum[j]);
        sum[j] += __shfl_xor(sum[j], 16, 64);
        sum[j] += __shfl_xor(sum[j], 32, 64);
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int64_t t = static_cast<int64_t>(blockIdx.x + h * (a.tn / 2)) * a.tk + kt;
        const u32x4 w = codes[t * 64 + lane];
#pragma unroll
        for (int g = 0; g < kPer; ++g) {
          float s = 0.0f;
#pragma unroll
          for (int j = 0; j < G / 32; ++j) s += sum[g * (G / 32) + j];
          uint32_t z4 = 0x08080808u;
          if constexpr (Z) z4 = *reinterpret_cast<const uint32_t*>(zeros + (t * kPer + g) * 16 + q * 4);
          const f16x4 d = *reinterpret_cast<const f16x4*>(scales + (t * kPer + g) * 32 + q * 8);
          f32x4 acc;
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = -static_cast<float>(16 + (z4 >> (8 * i) & 255u)) * s;
#pragma unroll
          for (int j = 0; j < G / 32; ++j) acc = mma<BF>(unpack8<BF>(w[g * (G / 32) + j]), xv[g * (G / 32) + j], acc);
#pragma unroll
          for (int i = 0; i < 4; ++i) out[h][i] += static_cast<float>(d[i]) * acc[i];
        }
      }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) part[wave][h][lane] = out[h];
    __syncthreads();
    if (wave == 0 && p >= 0) {
      f32x4 v[H] = {};
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int w = 0; w < kQ4Waves; ++w) v[h] += part[w][h][lane];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = blockIdx.x * 16 + q * 4 + i;
        float o = v[0][i];
        if constexpr (SW) o = o / (1.0f + __expf(-o)) * v[1][i];
        if (c < out_n) put(a.y, p * a.ldy + c, o, a.out_type);
      }
    }
    __syncthreads();
    for (int i = 0; i < 16; ++i) rows &= rows - 1;
  }
}

namespace {

template <bool BF, int G, bool Z>
void go(const Q4& a, bool swiglu, hipStream_t s) {
  const dim3 block(64 * kQ4Waves);
  const uint32_t y = a.idx ? a.rows : 1;
  if (swiglu) hipLaunchKernelGGL((k_q4<BF, G, Z, true>), dim3(a.tn / 2, y), block, 0, s, a);
  else hipLaunchKernelGGL((k_q4<BF, G, Z, false>), dim3(a.tn, y), block, 0, s, a);
}

template <bool BF, int G>
void go(const Q4& a, bool swiglu, hipStream_t s) {
  if (a.zeros) go<BF, G, true>(a, swiglu, s);
  else go<BF, G, false>(a, swiglu, s);
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
