// gfx950 products of rows grouped by expert (ragged groups), in bf16 or f16
// with fp32 sums:
//
//   matmul, swiglu    y[i, :]  = x[src(i), :] W_g^T           contraction over k
//   matmul_t, ..grad  dx[i, :] = dy[src(i), :] W_g            contraction over n
//   wgrad             dW_g     = sum_i dy[i, :]^T x[src(i), :]  over the group's rows
//
// One kernel computes them all as D[p][q] = sum_r P[p][r] Q[q][r]: p runs along
// the output's contiguous dimension (the matrix instruction's rows, of which a
// lane holds four in a row: one vector store), q along its rows.  An operand
// is "straight" when r is contiguous in memory (x, W for matmul) and "across"
// when p or q is (W for matmul_t, both for wgrad): a straight tile lies in LDS
// as [p][64 r], an across tile as [64 r][p], read with the transposing LDS
// read, so no operand is transposed in memory first.
//
// Bound by the matrix cores with many rows a group, by the weights' bytes with
// few.  Measured, bf16:
//     8192^3, one group: y 898 us (1224 TFLOP/s), SwiGLU 806, dx 827 (1330), fp32
//       dW 844 (1302); the same operations in a library's product: 772 (another
//       card of the same model ran all of ours 5 % faster)
//     16 groups of 1024 rows, n 4608, k 5120: y 681 us (1135), dx 691 (1119), fp32
//       dW 864 (895, 1.5 GB written)
//     384 groups of 32 rows, the same matrices: y 3150 us, 5.8 TB/s; dx 3274
#include <hip/hip_runtime.h>

#include <cstdint>

#include "dev_common.h"
#include "group.h"

namespace moe {
namespace grp {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
using dev::u32x2;
using dev::u32x4;
#define MOE_LDS __attribute__((address_space(3)))

using ConstInts = const int32_t __attribute__((address_space(4)))*;   // read through scalar loads

constexpr int kRed = 64;   // contraction per step: whole 128-byte lines of a straight row

enum Epilogue { kStore, kSwigluOut, kSwigluBack };

struct Gemm {
  const uint16_t *p, *q;          // the two operands
  void* y;
  const uint16_t* pre_in;         // kSwigluBack: (g | u)
  uint16_t* pre_out;              // kSwigluOut: (g | u), or null
  const int32_t* offsets;         // [groups + 1]
  const int32_t* src;             // rows of the gathered operand, or null
  int64_t ldp, ldq, ldy, ld_pre;
  int64_t p_stride, y_stride;     // per group: of P (weights), of y (wgrad)
  int groups, rows;
  int np, nq, nr;                 // extents (nq: wgrad; nr: the products)
  int half;                       // I of the SwiGLU calls
  int src_rows;                   // rows that src selects from
  uint32_t div_mul;               // floor(s / src_div) = (s * div_mul) >> 32 >> div_shift; 0: src_div is 1
  int div_shift;
  int tiles_p, tiles_q;           // tiles of an output (tiles_q: wgrad)
  int out_type, accumulate;
};

// ---------------------------------------------------------------------------
// types
// ---------------------------------------------------------------------------
template <bool BF>
__device__ __forceinline__ f32x4 mma(s16x8 a, s16x8 b, f32x4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <bool BF>
__device__ __forceinline__ uint16_t to_half(float v) {
  if constexpr (BF) return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}
template <bool BF>
__device__ __forceinline__ float from_half(uint16_t v) {
  if constexpr (BF) return static_cast<float>(__builtin_bit_cast(__bf16, v));
  else return static_cast<float>(__builtin_bit_cast(_Float16, v));
}

// Vectors at any element boundary.  Outputs are stored past the caches' usual
// order: kept in it, a large output pushes out the operands that other tiles
// will read again (the fp32 weight gradients of 16 experts of 4608 x 5120: 1024
// us, 930 so).
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

// Four consecutive outputs, of which `n` exist.
__device__ __forceinline__ void store4(void* y, int64_t at, f32x4 v, int n, int type, bool add) {
  if (type == MOE_T_F32) {
    float* o = static_cast<float*>(y) + at;
    if (n >= 4) {
      if (add) {
        f32x4 held;
        __builtin_memcpy(&held, o, 16);
        v += held;
      }
      __builtin_nontemporal_store(v, reinterpret_cast<f32x4_any*>(o));
    } else {
      for (int i = 0; i < 4; ++i)
        if (i < n) o[i] = add ? o[i] + v[i] : v[i];
    }
    return;
  }
  uint16_t* o = static_cast<uint16_t*>(y) + at;
  if (add)
    for (int i = 0; i < 4; ++i)
      if (i < n) v[i] += type == MOE_T_BF16 ? from_half<true>(o[i]) : from_half<false>(o[i]);
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = type == MOE_T_BF16 ? to_half<true>(v[i]) : to_half<false>(v[i]);
  if (n >= 4) {
    u32x2 w;
    __builtin_memcpy(&w, h, 8);
    __builtin_nontemporal_store(w, reinterpret_cast<u32x2_any*>(o));
  } else {
    for (int i = 0; i < 4; ++i)
      if (i < n) o[i] = h[i];
  }
}

// Eight, added to nothing: 16 bytes of a 16-bit type at once.
__device__ __forceinline__ void store8(void* y, int64_t at, const f32x4 (&v)[2], int n, int type) {
  if (type != MOE_T_F32 && n >= 8) {
    uint16_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = type == MOE_T_BF16 ? to_half<true>(v[i / 4][i % 4]) : to_half<false>(v[i / 4][i % 4]);
    u32x4 w;
    __builtin_memcpy(&w, h, 16);
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4_any*>(static_cast<uint16_t*>(y) + at));
  } else {
    store4(y, at, v[0], n, type, false);
    store4(y, at + 4, v[1], n - 4, type, false);
  }
}

// ---------------------------------------------------------------------------
// work items
// ---------------------------------------------------------------------------
struct Item {
  int group, begin, end;   // the group's rows
  int p0, q0;              // first column / row of the output tile (products: q0 a pair row)
  bool any;
};

// Workgroup ids go to the eight XCDs in turn: XCD x takes the x-th eighth of
// the items, so tiles that share an operand share an L2.
__device__ __forceinline__ int xcd_item(int items) {
  const int per = (items + 7) / 8, b = blockIdx.x;
  return (b >> 3) < per ? (b & 7) * per + (b >> 3) : items;
}

__device__ __forceinline__ int wave_id() { return dev::uniform(static_cast<int>(threadIdx.x >> 6)); }

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// Sums over lanes 0 .. own, and over the wave, through in-register moves.
template <int CTRL, int ROWMASK>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWMASK, 0xF, false);
}
__device__ __forceinline__ int scan_wave(int v) {
  v = dpp_add<0x111, 0xF>(v);   // row_shr 1, 2, 4, 8: sums along each row of 16
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);   // row_bcast 15 into rows 1 and 3
  v = dpp_add<0x143, 0xC>(v);   // row_bcast 31 into rows 2 and 3
  return v;
}

// Products: group g has ceil(rows of g / BQ) row tiles, each tiles_p items.
// Every wave finds its workgroup's item by itself, 64 groups at a time, one a
// lane: the offsets of all of them are loaded first, then a scan over the
// lanes gives the group that holds the item.  Each dependent load here is a
// memory round trip before the tile's first byte is asked for.
template <int BP, int BQ>
__device__ __forceinline__ Item find_rows(const Gemm& a) {
  constexpr int kMost = MOE_MAX_GROUPS / 64;
  const int lane = threadIdx.x & 63, parts = (a.groups + 63) / 64;
  int begin[kMost], end[kMost];
#pragma unroll
  for (int c = 0; c < kMost; ++c) {
    if (c >= parts) break;
    const int g = c * 64 + lane < a.groups ? c * 64 + lane : a.groups;   // past the last: begin = end
    begin[c] = a.offsets[g];
    end[c] = a.offsets[g < a.groups ? g + 1 : g];
  }
  int upto[kMost], total = 0;
#pragma unroll
  for (int c = 0; c < kMost; ++c) {
    if (c >= parts) break;
    begin[c] = clampi(begin[c], 0, a.rows);
    end[c] = clampi(end[c], begin[c], a.rows);
    upto[c] = total + scan_wave((end[c] - begin[c] + BQ - 1) / BQ);
    total = __builtin_amdgcn_readlane(upto[c], 63);
  }
  Item it{};
  const int at = xcd_item(total * a.tiles_p);
  const int tile = at / a.tiles_p;
  if (tile >= total) return it;
#pragma unroll
  for (int c = 0; c < kMost; ++c) {
    if (c >= parts) break;
    const uint64_t over = __ballot(upto[c] > tile);
    if (!over) continue;
    const int holder = __ffsll(static_cast<unsigned long long>(over)) - 1;
    it.group = c * 64 + holder;
    it.begin = __builtin_amdgcn_readlane(begin[c], holder);
    it.end = __builtin_amdgcn_readlane(end[c], holder);
    const int tq = (it.end - it.begin + BQ - 1) / BQ;
    const int in = at - (__builtin_amdgcn_readlane(upto[c], holder) - tq) * a.tiles_p;
    // bands of eight row tiles: the tiles in flight on an XCD are then a
    // block of rows by columns, which shares both operands
    const int band = in / (8 * a.tiles_p), rest = in - band * 8 * a.tiles_p;
    const int wide = tq - 8 * band < 8 ? tq - 8 * band : 8;
    it.p0 = rest / wide * BP;
    it.q0 = it.begin + (8 * band + rest % wide) * BQ;
    // offsets that do not ascend can make more items than the grid was made
    // for, past 32 bits too: whatever such a count gives writes nothing
    it.any = at >= 0 && in >= 0 && it.q0 >= it.begin && it.q0 < it.end;
    break;
  }
  return it;
}

// wgrad: every group has the same tiles; each XCD takes an eighth of every
// group's, so unequal groups do not make unequal XCDs.
template <int BP, int BQ>
__device__ __forceinline__ Item find_matrix(const Gemm& a) {
  const int tiles = a.tiles_p * a.tiles_q, per = (tiles + 7) / 8, b = blockIdx.x;
  const int x = b & 7, j = b >> 3, g = j / per, t = x * per + j % per;
  Item it{};
  it.any = t < tiles;
  it.group = g;
  it.begin = clampi(a.offsets[g], 0, a.rows);
  it.end = clampi(a.offsets[g + 1], it.begin, a.rows);
  const int band = t / (8 * a.tiles_p), in = t - band * 8 * a.tiles_p;
  const int wide = a.tiles_q - 8 * band < 8 ? a.tiles_q - 8 * band : 8;
  it.p0 = in / wide * BP;
  it.q0 = (8 * band + in % wide) * BQ;
  return it;
}

// Row that a src entry names, or -1.
__device__ __forceinline__ int named_row(const Gemm& a, int32_t s) {
  const uint32_t u = static_cast<uint32_t>(s);
  const int r = static_cast<int>(a.div_mul ? __umulhi(u, a.div_mul) >> a.div_shift : u);
  return s >= 0 && r < a.src_rows ? r : -1;
}
// Row of the gathered operand for pair row i, or -1.
__device__ __forceinline__ int source_row(const Gemm& a, int i) { return a.src ? named_row(a, a.src[i]) : i; }

// ---------------------------------------------------------------------------
// LDS tiles.  Straight: [rows][64], 128-byte rows of eight 16-byte chunks,
// chunk c of row r at place c ^ (r & 7).  Across: [64][cols], chunks of 32
// bytes (one 16-column unit), unit u of row r at u ^ spread(r).  Both let the
// lanes of one read touch different banks.
// ---------------------------------------------------------------------------
template <int B>
__device__ __forceinline__ int spread(int r) {
  return B >= 128 ? (r & 3) | ((r >> 3) & 1) << 2 : r & 3;
}

template <bool ACROSS, int B>
__device__ __forceinline__ s16x8 fragment(const MOE_LDS uint8_t* tile, int at, int kk) {
  const int l = threadIdx.x & 63;
  if constexpr (!ACROSS) {
    const int r = at + (l & 15), c = kk * 4 + (l >> 4);
    return *reinterpret_cast<const MOE_LDS s16x8*>(tile + r * 128 + ((c ^ (r & 7)) * 16));
  } else {
    // per 16 lanes: four rows of 16 columns in, four rows of one column out
    const int r = kk * 32 + (l >> 4) * 8 + ((l & 15) >> 2), u = at >> 4;
    const MOE_LDS uint8_t* lo = tile + r * (B * 2) + ((u ^ spread<B>(r)) * 32) + (l & 3) * 8;
    const int r4 = r + 4;
    const MOE_LDS uint8_t* hi = tile + r4 * (B * 2) + ((u ^ spread<B>(r4)) * 32) + (l & 3) * 8;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)lo);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS s16x4*)hi);
    return s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
}

// Eight elements at `ptr`, of which the first `n` are wanted and the rest read
// as 0.  One load from any 2-byte boundary: what follows the wanted ones lies
// inside the operand, except at its very end (`end`), where the elements are
// read one by one.
__device__ __forceinline__ u32x4 load8(const uint16_t* ptr, const uint16_t* end, int n) {
  u32x4 v{0, 0, 0, 0};
  if (n > 0 && ptr + 8 <= end) {
    __builtin_memcpy(&v, ptr, 16);
    if (n < 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = n >= 2 * i + 2 ? v[i] : n == 2 * i + 1 ? v[i] & 0xFFFFu : 0u;
    }
  } else if (n > 0) {
    for (int i = 0; i < 8; ++i)
      if (i < n) v[i / 2] |= static_cast<uint32_t>(ptr[i]) << 16 * (i & 1);
  }
  return v;
}

// Row of W for slot s of a P tile at column p0.  With the SwiGLU epilogue a
// wave's slots are half gate rows, half the up rows of the same channels.
template <int EPI, int TP>
__device__ __forceinline__ int p_row(const Gemm& a, int p0, int s) {
  if constexpr (EPI != kSwigluOut) return p0 + s;
  const int ch = p0 / 2 + s / TP * (TP / 2) + s % (TP / 2);
  if (ch >= a.half) return a.np;
  return s % TP < TP / 2 ? ch : a.half + ch;
}

// Rows of 16 outputs by TP columns that a wave holds as fragments (a lane: one
// row, four columns of each 16) go through LDS, from where a lane takes 16
// bytes of output in a row: a wave then writes whole lines.  Storing the
// fragments as they are writes 32-byte pieces of 16 rows at a time: 8192^3 took
// 963 us so, and 854 with half the output (SwiGLU); through LDS 884 and 803.
template <int C>
struct Rows {
  static constexpr int kPitch = C * 4 + 16;   // bytes; the odd 16 spread the rows over the banks
  static constexpr int kBytes = 16 * kPitch;
  MOE_LDS uint8_t* at;

  __device__ __forceinline__ void put(int i, f32x4 v) const {
    const int l = threadIdx.x & 63;
    *reinterpret_cast<MOE_LDS f32x4*>(at + (l & 15) * kPitch + i * 64 + (l >> 4) * 16) = v;
  }
  // Columns [c0, c0 + C) of `cols` of rows q0 .. of y, as far as q_end.
  __device__ __forceinline__ void flush(void* y, int64_t ld, int q0, int q_end, int c0, int cols, int type, bool add) const {
    const int l = threadIdx.x & 63;
    if (type == MOE_T_F32) {
#pragma unroll
      for (int s = 0; s < C / 16; ++s) {
        const int r = (s * 64 + l) / (C / 4), c = (s * 64 + l) % (C / 4) * 4;
        const f32x4 v = *reinterpret_cast<const MOE_LDS f32x4*>(at + r * kPitch + c * 4);
        if (q0 + r < q_end) store4(y, (q0 + r) * ld + c0 + c, v, cols - c0 - c, type, add);
      }
    } else {
#pragma unroll
      for (int s = 0; s < (C + 31) / 32; ++s) {   // the lanes past row 15 (C = 16) rest
        const int r = (s * 64 + l) / (C / 8), c = (s * 64 + l) % (C / 8) * 8;
        if (C < 32 && r >= 16) continue;
        const MOE_LDS uint8_t* p = at + r * kPitch + c * 4;
        const f32x4 lo = *reinterpret_cast<const MOE_LDS f32x4*>(p), hi = *reinterpret_cast<const MOE_LDS f32x4*>(p + 16);
        if (q0 + r >= q_end) continue;
        const int64_t o = (q0 + r) * ld + c0 + c;
        if (!add) {
          store8(y, o, {lo, hi}, cols - c0 - c, type);
        } else {
          store4(y, o, lo, cols - c0 - c, type, add);
          store4(y, o + 4, hi, cols - c0 - c - 4, type, add);
        }
      }
    }
  }
};

// The SwiGLU gradient's epilogue.  dh goes through LDS, 16 rows at a time; a lane
// then holds eight columns of a row.  Their gate and up are asked for two such
// pieces ahead, and without a branch when the tile is whole: the compiler then
// waits for those loads alone, not for the stores behind them.
template <bool BF, int TP, int TQ, bool WHOLE>
__device__ __forceinline__ void swiglu_back(const Gemm& a, f32x4 (&acc)[TP / 16][TQ / 16], int c0, int q_first, int q_end,
                                            void* y, const Rows<TP>& rows) {
  constexpr int kPieces = TP / 32, kAhead = TQ / 16 < 2 ? 1 : 2;
  static_assert(TP % 32 == 0, "whole pieces of 16 rows by 32 columns");
  const int l = threadIdx.x & 63;
  uint8_t* y2 = static_cast<uint8_t*>(y) + static_cast<int64_t>(a.np) * (a.out_type == MOE_T_F32 ? 4 : 2);
  u32x4 gate[kAhead][kPieces], up[kAhead][kPieces];
  const auto ask = [&](int j) {
#pragma unroll
    for (int s = 0; s < kPieces; ++s) {
      const int r = q_first + j * 16 + (s * 64 + l) / (TP / 8), c = c0 + (s * 64 + l) % (TP / 8) * 8;
      u32x4 &g = gate[j % kAhead][s], &u = up[j % kAhead][s];
      if constexpr (!WHOLE) {
        g = u = u32x4{0, 0, 0, 0};
        if (r >= q_end || c >= a.np) continue;
      }
      const uint16_t* at = a.pre_in + r * a.ld_pre + c;
      if (WHOLE || c + 8 <= a.np) {
        __builtin_memcpy(&g, at, 16);
        __builtin_memcpy(&u, at + a.np, 16);
      } else {
        for (int e = 0; e < 8; ++e)
          if (c + e < a.np) {
            g[e / 2] |= static_cast<uint32_t>(at[e]) << 16 * (e & 1);
            u[e / 2] |= static_cast<uint32_t>(at[a.np + e]) << 16 * (e & 1);
          }
      }
    }
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) ask(j);
#pragma unroll
  for (int j = 0; j < TQ / 16; ++j) {
    if (!WHOLE && q_first + j * 16 >= q_end) break;
#pragma unroll
    for (int i = 0; i < TP / 16; ++i) rows.put(i, acc[i][j]);
#pragma unroll
    for (int s = 0; s < kPieces; ++s) {
      const int rl = (s * 64 + l) / (TP / 8), cl = (s * 64 + l) % (TP / 8) * 8, r = q_first + j * 16 + rl, c = c0 + cl;
      if (!WHOLE && (r >= q_end || c >= a.np)) continue;
      const MOE_LDS uint8_t* at = rows.at + rl * rows.kPitch + cl * 4;
      f32x4 dh[2], dg[2], du[2];
      dh[0] = *reinterpret_cast<const MOE_LDS f32x4*>(at);
      dh[1] = *reinterpret_cast<const MOE_LDS f32x4*>(at + 16);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = from_half<BF>(static_cast<uint16_t>(gate[j % kAhead][s][e / 2] >> 16 * (e & 1)));
        const float u = from_half<BF>(static_cast<uint16_t>(up[j % kAhead][s][e / 2] >> 16 * (e & 1)));
        const float sg = 1.0f / (1.0f + __expf(-g)), d = dh[e / 4][e % 4];
        dg[e / 4][e % 4] = d * u * sg * (1.0f + g * (1.0f - sg));
        du[e / 4][e % 4] = d * g * sg;
      }
      const int64_t o = r * a.ldy + c;
      const int n = WHOLE ? 8 : a.np - c;
      store8(y, o, dg, n, a.out_type);
      store8(y2, o, du, n, a.out_type);
    }
    if (j + kAhead < TQ / 16) ask(j + kAhead);
  }
}

// `lds`: room for a Rows<TP> a wave; every wave's tile reads are done.
template <bool BF, int EPI, int TP, int TQ>
__device__ __forceinline__ void epilogue(const Gemm& a, const Item& it, f32x4 (&acc)[TP / 16][TQ / 16], int wp, int wq,
                                         int q_end, void* y, MOE_LDS uint8_t* lds) {
  constexpr int C = EPI == kSwigluOut ? TP / 2 : TP;   // columns of an output that a wave holds
  const int type = BF ? MOE_T_BF16 : MOE_T_F16;
  const Rows<C> rows{lds + wave_id() * Rows<C>::kBytes};
  const int c0 = (EPI == kSwigluOut ? it.p0 / 2 : it.p0) + wp * C;
  if constexpr (EPI == kSwigluBack) {
    const int q0 = it.q0 + wq * TQ;
    if (q0 + TQ <= q_end && c0 + TP <= a.np) swiglu_back<BF, TP, TQ, true>(a, acc, c0, q0, q_end, y, rows);
    else if (q0 < q_end) swiglu_back<BF, TP, TQ, false>(a, acc, c0, q0, q_end, y, rows);
    return;
  }
#pragma unroll
  for (int j = 0; j < TQ / 16; ++j) {
    const int q0 = it.q0 + wq * TQ + j * 16;
    if (q0 >= q_end) break;
    if constexpr (EPI == kStore) {
#pragma unroll
      for (int i = 0; i < TP / 16; ++i) rows.put(i, acc[i][j]);
      rows.flush(y, a.ldy, q0, q_end, c0, a.np, a.out_type, a.accumulate);
    } else if constexpr (EPI == kSwigluOut) {
      // gate and up of a channel are TP / 32 fragments apart
#pragma unroll
      for (int i = 0; i < TP / 32; ++i) {
        const f32x4 g = acc[i][j], u = acc[i + TP / 32][j];
        f32x4 h;
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = g[e] / (1.0f + __expf(-g[e])) * u[e];
        rows.put(i, h);
      }
      rows.flush(y, a.ldy, q0, q_end, c0, a.half, a.out_type, false);
      if (a.pre_out) {
#pragma unroll
        for (int i = 0; i < TP / 32; ++i) rows.put(i, acc[i][j]);
        rows.flush(a.pre_out, a.ld_pre, q0, q_end, c0, a.half, type, false);
#pragma unroll
        for (int i = 0; i < TP / 32; ++i) rows.put(i, acc[i + TP / 32][j]);
        rows.flush(a.pre_out + a.half, a.ld_pre, q0, q_end, c0, a.half, type, false);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Any alignment, any span: tiles go through registers.  The next step's chunks
// (eight elements, loaded from any 2-byte boundary) are in flight while the
// present step is multiplied.
// ---------------------------------------------------------------------------
template <bool BF, bool PA, bool QA, int EPI, int BP, int BQ, int WP, int WQ>
__global__ __launch_bounds__(64 * WP * WQ) void k_group_any(Gemm a) {
  constexpr int TP = BP / WP, TQ = BQ / WQ, NT = 64 * WP * WQ;
  constexpr int NP = BP * 8 / NT, NQ = BQ * 8 / NT;   // chunks a thread
  constexpr bool kWeight = PA && QA;                  // wgrad
  constexpr int kTiles = (BP + BQ) * 128, kOut = WP * WQ * Rows<TP>::kBytes;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kTiles > kOut ? kTiles : kOut];
  const Item it = kWeight ? find_matrix<BP, BQ>(a) : find_rows<BP, BQ>(a);
  if (!it.any) return;
  const int tid = threadIdx.x, wave = wave_id(), wp = wave % WP, wq = wave / WP;
  const int red = kWeight ? it.end - it.begin : a.nr;
  const int q_end = kWeight ? a.nq : it.end;
  MOE_LDS uint8_t* lp = (MOE_LDS uint8_t*)lds;
  MOE_LDS uint8_t* lq = lp + BP * 128;
  f32x4 acc[TP / 16][TQ / 16] = {};

  const bool gather = kWeight && a.src;   // of P
  // one past the operands' last elements
  const uint16_t* pbase = kWeight ? a.p : a.p + it.group * a.p_stride;
  const uint16_t* pend = pbase + (kWeight ? static_cast<int64_t>(a.src_rows) - 1 : PA ? a.nr - 1 : a.np - 1) * a.ldp + (PA ? a.np : a.nr);
  const uint16_t* qend = a.q + (static_cast<int64_t>(kWeight ? a.rows : a.src_rows) - 1) * a.ldq + (QA ? a.nq : a.nr);
  if constexpr (kWeight) {
    if (!gather) pbase += it.begin * a.ldp;
  }
  const uint16_t* qbase = QA ? a.q + it.begin * a.ldq : a.q;

  // Each chunk's place in the first step.  Straight: rows past the tile's last
  // read another row instead (they belong to no output), entries that name no
  // row read as zeros.
  const uint16_t *ps[NP], *qs[NQ];
  uint32_t none = 0;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int c = tid + i * NT;
    if constexpr (!PA) {
      const int row = p_row<EPI, TP>(a, it.p0, c >> 3);
      ps[i] = pbase + (row < a.np ? row : 0) * a.ldp + (c & 7) * 8;
    } else {
      ps[i] = pbase + c / (BP / 8) * a.ldp + it.p0 + c % (BP / 8) * 8;
    }
  }
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int c = tid + i * NT;
    if constexpr (!QA) {
      const int q = it.q0 + (c >> 3), row = source_row(a, q < q_end ? q : it.q0);
      none |= row < 0 ? 1u << i : 0u;
      qs[i] = qbase + (row < 0 ? 0 : row) * a.ldq + (c & 7) * 8;
    } else {
      qs[i] = qbase + c / (BQ / 8) * a.ldq + it.q0 + c % (BQ / 8) * 8;
    }
  }

  u32x4 vp[NP], vq[NQ];
  [[maybe_unused]] int from[NP];   // gathered: the chunks' rows of the next step to fetch, -1 for none
  const auto look_up = [&](int r0) {
    if constexpr (kWeight) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int r = r0 + (tid + i * NT) / (BP / 8);
        from[i] = r < red ? source_row(a, it.begin + r) : -1;
      }
    }
  };
  const auto fetch = [&](int r0) {
    // A step whose chunks all lie inside their operands needs no care.  An
    // across chunk may run past its row there: the columns past the last
    // belong to no output.
    const bool inner = r0 + kRed <= red &&
                       (!PA || (gather ? it.p0 + BP <= a.np : pbase + (r0 + kRed - 1) * a.ldp + it.p0 + BP <= pend)) &&
                       (!QA || qbase + (r0 + kRed - 1) * a.ldq + it.q0 + BQ <= qend);
    const int64_t po = PA ? r0 * a.ldp : r0, qo = QA ? r0 * a.ldq : r0;
    if (inner) {
      if (gather) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
          __builtin_memcpy(&vp[i], pbase + (from[i] < 0 ? 0 : from[i]) * a.ldp + it.p0 + (tid + i * NT) % (BP / 8) * 8, 16);
      } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) __builtin_memcpy(&vp[i], ps[i] + po, 16);
      }
#pragma unroll
      for (int i = 0; i < NQ; ++i) __builtin_memcpy(&vq[i], qs[i] + qo, 16);
      if (gather) {
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (from[i] < 0) vp[i] = u32x4{0, 0, 0, 0};
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int c = tid + i * NT;
        if constexpr (!PA) {
          vp[i] = load8(ps[i] + po, pend, red - r0 - (c & 7) * 8);
        } else {
          const int r = r0 + c / (BP / 8), cols = a.np - it.p0 - c % (BP / 8) * 8;
          const uint16_t* s = ps[i] + po;
          bool in = r < red;
          if (gather) {
            in = from[i] >= 0;
            s = pbase + from[i] * a.ldp + a.np - cols;
          }
          vp[i] = load8(s, pend, !in ? 0 : s + 8 <= pend ? 8 : cols);
        }
      }
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int c = tid + i * NT;
        if constexpr (!QA) {
          vq[i] = load8(qs[i] + qo, qend, red - r0 - (c & 7) * 8);
        } else {
          const uint16_t* s = qs[i] + qo;
          vq[i] = load8(s, qend, r0 + c / (BQ / 8) >= red ? 0 : s + 8 <= qend ? 8 : a.nq - it.q0 - c % (BQ / 8) * 8);
        }
      }
    }
    if constexpr (!QA) {
      if (a.src) {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
          if (none >> i & 1) vq[i] = u32x4{0, 0, 0, 0};
      }
    }
    if (gather) look_up(r0 + kRed);
  };

  if (gather) look_up(0);
  fetch(0);
  for (int r0 = 0; r0 < red; r0 += kRed) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int c = tid + i * NT, r = c / (PA ? BP / 8 : 8), ch = c % (PA ? BP / 8 : 8);
      const int at = PA ? r * (BP * 2) + (((ch >> 1) ^ spread<BP>(r)) * 32) + (ch & 1) * 16 : r * 128 + ((ch ^ (r & 7)) * 16);
      *reinterpret_cast<MOE_LDS u32x4*>(lp + at) = vp[i];
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int c = tid + i * NT, r = c / (QA ? BQ / 8 : 8), ch = c % (QA ? BQ / 8 : 8);
      const int at = QA ? r * (BQ * 2) + (((ch >> 1) ^ spread<BQ>(r)) * 32) + (ch & 1) * 16 : r * 128 + ((ch ^ (r & 7)) * 16);
      *reinterpret_cast<MOE_LDS u32x4*>(lq + at) = vq[i];
    }
    __syncthreads();
    if (r0 + kRed < red) fetch(r0 + kRed);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      s16x8 fp[TP / 16], fq[TQ / 16];
#pragma unroll
      for (int i = 0; i < TP / 16; ++i) fp[i] = fragment<PA, BP>(lp, wp * TP + i * 16, kk);
#pragma unroll
      for (int j = 0; j < TQ / 16; ++j) fq[j] = fragment<QA, BQ>(lq, wq * TQ + j * 16, kk);
#pragma unroll
      for (int i = 0; i < TP / 16; ++i)
#pragma unroll
        for (int j = 0; j < TQ / 16; ++j) acc[i][j] = mma<BF>(fp[i], fq[j], acc[i][j]);
    }
  }
  __syncthreads();
  void* y = a.y;
  if constexpr (kWeight) y = static_cast<uint8_t*>(y) + it.group * a.y_stride * (a.out_type == MOE_T_F32 ? 4 : 2);
  epilogue<BF, EPI, TP, TQ>(a, it, acc, wp, wq, q_end, y, lp);
}

// ---------------------------------------------------------------------------
// Aligned operands: tiles go from memory to LDS without passing registers.
// A buffer load writes LDS in lane order, 16 bytes a lane, so the swizzles of
// the tiles are applied to the lanes' source addresses (with them no LDS read
// has a bank conflict, by the counters).  Reads outside an
// operand (a row of no group, a row past the contraction) return zeros by the
// buffer's bounds; kOutside is past every buffer (all are below 2 GiB).
// ---------------------------------------------------------------------------
constexpr uint32_t kOutside = 0x7ffffff0u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint16_t* base, int64_t rows, int64_t ld, int64_t cols) {
  const int64_t bytes = rows > 0 ? ((rows - 1) * ld + cols) * 2 : 0;
  void* u = reinterpret_cast<void*>(dev::uniform(reinterpret_cast<uint64_t>(base)));
  return __builtin_amdgcn_make_buffer_rsrc(u, 0, dev::uniform(static_cast<int>(bytes)), 0x00020000);
}

__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t b, MOE_LDS uint8_t* at, uint32_t lane_off, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (MOE_LDS void*)at, 16, static_cast<int>(lane_off), static_cast<int>(off), 0, 0);
}

// The loads of one operand's tile: N of them a wave, 64 chunks of 16 bytes each.
template <bool ACROSS, int B, int WAVES>
struct Feed {
  static constexpr int N = B / (8 * WAVES);
  static constexpr int kRowsPerLoad = ACROSS ? 512 / B : 8;
  __amdgpu_buffer_rsrc_t buf;
  uint32_t lane[N];        // byte offset of each load's chunk in the first step
  int chunk;               // straight: this lane's chunk of a row
  int red;                 // contraction length
  uint32_t step;           // bytes a step

  // Tile row (straight: of the tile, across: of the step) that load i of this lane fetches.
  static __device__ __forceinline__ int row(int i) {
    const int l = threadIdx.x & 63, w = wave_id() % WAVES;
    return (w * N + i) * kRowsPerLoad + (ACROSS ? l / (B / 8) : l >> 3);
  }
  // Across: the column of the chunk that load i of this lane fetches.
  static __device__ __forceinline__ int col(int i) {
    const int place = (threadIdx.x & 63) % (B / 8), u = (place >> 1) ^ spread<B>(row(i));
    return u * 16 + (place & 1) * 8;
  }
  __device__ __forceinline__ void set_chunk() { chunk = (threadIdx.x & 7) ^ ((threadIdx.x >> 3) & 7); }

  // Straight operands and across operands without a gather.
  __device__ __forceinline__ void load(MOE_LDS uint8_t* tile, int t) const {
    const int w = wave_id() % WAVES, left = red - t * kRed;
    MOE_LDS uint8_t* at = tile + w * N * 1024;
    if (ACROSS || left >= kRed) {
#pragma unroll
      for (int i = 0; i < N; ++i) to_lds(buf, at + i * 1024, lane[i], t * step);
    } else {
      // a straight row ends inside the step: what follows it must not be read
#pragma unroll
      for (int i = 0; i < N; ++i) to_lds(buf, at + i * 1024, chunk * 8 < left ? lane[i] : kOutside, t * step);
    }
  }
};

template <int LOADS>
__device__ __forceinline__ void step_barrier() {
  // this wave's loads of the step have landed and its reads of the last one
  // are done; behind the barrier that holds for every wave
  if constexpr (LOADS == 0) asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LOADS) : "memory");
}

// SPLIT > 1: few tiles with a long contraction.  SPLIT groups of WP x WQ waves
// take the steps in turn, each with its own part of a stage, and the groups'
// sums are added in order at the end.
template <bool BF, bool PA, bool QA, int EPI, int BP, int BQ, int WP, int WQ, int STAGES, int SPLIT>
__global__ __launch_bounds__(64 * WP * WQ * SPLIT) void k_group_tiles(Gemm a) {
  constexpr int TP = BP / WP, TQ = BQ / WQ, NW = WP * WQ;
  constexpr bool kWeight = PA && QA;   // wgrad
  constexpr int kStep = (BP + BQ) * 128, kStage = SPLIT * kStep;
  constexpr bool kPhased = STAGES == 2 && NW == 8 && SPLIT == 1;   // two groups of waves, a phase apart
  constexpr int kLds = STAGES * kStage + (kPhased ? BP * 128 : 0);
  static_assert(SPLIT == 1 || (SPLIT - 1) * BP * BQ * 4 <= STAGES * kStage, "the groups' sums use the tiles' memory");
  static_assert(NW * Rows<TP>::kBytes + (SPLIT - 1) * BP * BQ * 4 <= STAGES * kStage, "the epilogue's rows use the tiles' memory");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const Item it = kWeight ? find_matrix<BP, BQ>(a) : find_rows<BP, BQ>(a);
  if (!it.any) return;
  const int wave = wave_id() % NW, turn = wave_id() / NW, wp = wave % WP, wq = wave / WP;
  const int red = kWeight ? it.end - it.begin : a.nr;
  const int q_end = kWeight ? a.nq : it.end;
  MOE_LDS uint8_t* base = (MOE_LDS uint8_t*)lds + turn * kStep;   // stages are kStage apart

  Feed<PA, BP, NW> fp;
  Feed<QA, BQ, NW> fq;
  fp.red = fq.red = red;
  fp.set_chunk();
  fq.set_chunk();
  if constexpr (!PA) {
    fp.buf = buffer_of(a.p + it.group * a.p_stride, a.np, a.ldp, a.nr);
    fp.step = kRed * 2;
#pragma unroll
    for (int i = 0; i < fp.N; ++i) {
      const int row = p_row<EPI, TP>(a, it.p0, fp.row(i));
      fp.lane[i] = row < a.np ? static_cast<uint32_t>(row) * static_cast<uint32_t>(a.ldp * 2) + fp.chunk * 16 : kOutside;
    }
  } else {
    const bool gather = kWeight && a.src;
    fp.buf = kWeight ? (gather ? buffer_of(a.p, a.src_rows, a.ldp, a.np) : buffer_of(a.p + it.begin * a.ldp, red, a.ldp, a.np))
                     : buffer_of(a.p + it.group * a.p_stride, a.nr, a.ldp, a.np);
    fp.step = static_cast<uint32_t>(kRed * 2 * a.ldp);
#pragma unroll
    for (int i = 0; i < fp.N; ++i)
      fp.lane[i] = (gather ? 0u : fp.row(i) * static_cast<uint32_t>(a.ldp * 2)) + (it.p0 + fp.col(i)) * 2;
  }
  if constexpr (!QA) {
    const bool gather = a.src != nullptr;
    // of a group, only the tile's rows: all of them may pass 4 GiB
    fq.buf = gather ? buffer_of(a.q, a.src_rows, a.ldq, a.nr)
                    : buffer_of(a.q + it.q0 * a.ldq, it.end - it.q0 < BQ ? it.end - it.q0 : BQ, a.ldq, a.nr);
    fq.step = kRed * 2;
#pragma unroll
    for (int i = 0; i < fq.N; ++i) {
      const int r = fq.row(i);
      int row = r;
      if (gather) row = it.q0 + r < it.end ? source_row(a, it.q0 + r) : -1;
      fq.lane[i] = it.q0 + r < it.end && row >= 0 ? static_cast<uint32_t>(row) * static_cast<uint32_t>(a.ldq * 2) + fq.chunk * 16 : kOutside;
    }
  } else {
    fq.buf = buffer_of(a.q + it.begin * a.ldq, red, a.ldq, a.nq);
    fq.step = static_cast<uint32_t>(kRed * 2 * a.ldq);
#pragma unroll
    for (int i = 0; i < fq.N; ++i) fq.lane[i] = fq.row(i) * static_cast<uint32_t>(a.ldq * 2) + (it.q0 + fq.col(i)) * 2;
  }

  // wgrad: the rows of x follow src.  A load covers kR of them, the same for
  // the whole wave, so their entries come through scalar loads (which no
  // vector-memory count waits for), a phase or more before they are used.
  constexpr int kR = PA ? Feed<PA, BP, NW>::kRowsPerLoad : 1, kNext = decltype(fp)::N * kR;
  [[maybe_unused]] int32_t next[kNext];
  const auto fetch = [&](int m) {
    if constexpr (kWeight) {
      if (!a.src) return;
      const int t = m * SPLIT + turn;
      const int first = it.begin + t * kRed + wave * kNext;
      const ConstInts src = reinterpret_cast<ConstInts>(reinterpret_cast<uintptr_t>(a.src));
      if (first + kNext <= it.end) {
#pragma unroll
        for (int i = 0; i < kNext; ++i) next[i] = src[first + i];
      } else {
#pragma unroll
        for (int i = 0; i < kNext; ++i) next[i] = first + i < it.end ? src[first + i] : -1;
      }
    }
  };
  fetch(0);

  // stage m holds steps m * SPLIT .. ; this group's is `turn` of them
  const auto issue_p = [&](int m, MOE_LDS uint8_t* tp) {
    const int t = m * SPLIT + turn;
    if (kWeight && a.src) {
      const int sub = (threadIdx.x & 63) / (BP / 8);   // which of a load's rows
#pragma unroll
      for (int i = 0; i < fp.N; ++i) {
        uint32_t off = 0;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const int row = named_row(a, next[i * kR + r]);
          const uint32_t at = row >= 0 ? static_cast<uint32_t>(row) * static_cast<uint32_t>(a.ldp * 2) : kOutside;
          off = r == 0 || sub == r ? at : off;
        }
        to_lds(fp.buf, tp + (wave * fp.N + i) * 1024, off + fp.lane[i], 0);
      }
    } else {
      fp.load(tp, t);
    }
  };
  const auto issue = [&](int m) {
    MOE_LDS uint8_t* tp = base + m % STAGES * kStage;
    issue_p(m, tp);
    fq.load(tp + BP * 128, m * SPLIT + turn);
  };

  f32x4 acc[TP / 16][TQ / 16] = {};
  s16x8 vp[TP / 16], vq[TQ / 16];
  const auto read = [&](const MOE_LDS uint8_t* lp, const MOE_LDS uint8_t* lq, int kk) {
#pragma unroll
    for (int i = 0; i < TP / 16; ++i) vp[i] = fragment<PA, BP>(lp, wp * TP + i * 16, kk);
#pragma unroll
    for (int j = 0; j < TQ / 16; ++j) vq[j] = fragment<QA, BQ>(lq, wq * TQ + j * 16, kk);
  };
  const auto multiply = [&] {
#pragma unroll
    for (int i = 0; i < TP / 16; ++i)
#pragma unroll
      for (int j = 0; j < TQ / 16; ++j) acc[i][j] = mma<BF>(vp[i], vq[j], acc[i][j]);
  };
  const int steps = (red + kRed * SPLIT - 1) / (kRed * SPLIT);
  if constexpr (kPhased) {
    // Two waves share a SIMD, and four of the eight run one phase behind the
    // other four: while one wave of a SIMD multiplies, the other one reads its
    // next fragments and issues loads, so the matrix cores see no gap.  A step
    // is four phases (read and multiply each half of the 64), with a barrier
    // after each.  Step t loads Q of step t + 1 and then P of step t + 2, both
    // over tiles of step t - 1, whose last reader was done a phase before step t
    // began.  Q and P of step t + 1 have landed at the end of the fourth phase
    // of step t, when only the last loads, of P, may be in flight: the leading
    // waves wait there, the others in their third phase, which ends at the same
    // barrier.  8192^3 went from 1141 to 1230 TFLOP/s with the phases, its input
    // gradient from 1017 to 1291, its weight gradient from 972 to 1268.  Five
    // stages of half the length for both operands were 8 - 15 % slower than two.
    // P (the weights, in the products) a step earlier takes the LDS that is
    // left: 16 groups of 1024 rows, n 4608, k 5120 724 -> 681 us, 128 of 192
    // 1539 -> 1448, its weight gradient 2308 -> 2189; 8192^3, whose operands the
    // last cache holds, 885 -> 898.
    const bool behind = wave >= 4;
    constexpr int kTileP = BP * 128, kTileQ = BQ * 128, kLate = decltype(fp)::N;
    MOE_LDS uint8_t *p0 = base, *p1 = base + kTileP, *p2 = base + 2 * kTileP;   // of P: this step's, the next two
    MOE_LDS uint8_t* const lq = base + 3 * kTileP;
    fq.load(lq, 0);
    issue_p(0, p0);
    fetch(1);
    issue_p(1, p1);
    fetch(2);
    step_barrier<kLate>();
    if (behind) asm volatile("s_barrier" ::: "memory");
    for (int t = 0; t < steps; ++t) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        read(p0, lq + (t & 1) * kTileQ, kk);
        if (kk == 0) {
          fq.load(lq + (~t & 1) * kTileQ, t + 1);
          issue_p(t + 2, p2);
        }
        if (kk == 1 && behind) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLate) : "memory");
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (kk == 0) fetch(t + 3);   // waited for with the next fragments, a phase from here
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        multiply();
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        if (kk == 1 && !behind) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLate) : "memory");
        asm volatile("s_barrier" ::: "memory");
      }
      MOE_LDS uint8_t* done = p0;
      p0 = p1, p1 = p2, p2 = done;
    }
    if (!behind) asm volatile("s_barrier" ::: "memory");
  } else {
    // steps past the last read nothing (every lane is outside), so the number
    // of loads in flight is the same at every barrier
#pragma unroll
    for (int t = 0; t < STAGES - 1; ++t) {
      issue(t);
      fetch(t + 1);
    }
    for (int t = 0; t < steps; ++t) {
      step_barrier<(STAGES - 2) * (decltype(fp)::N + decltype(fq)::N)>();
      issue(t + STAGES - 1);
      fetch(t + STAGES);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        read(base + t % STAGES * kStage, base + t % STAGES * kStage + BP * 128, kk);
        multiply();
      }
    }
  }
  step_barrier<0>();
  base = (MOE_LDS uint8_t*)lds;
  if constexpr (SPLIT > 1) {
    // [group - 1][wave][fragment][lane]
    constexpr int kFragments = TP / 16 * (TQ / 16);
    MOE_LDS f32x4* sums = reinterpret_cast<MOE_LDS f32x4*>(base) + wave * kFragments * 64 + (threadIdx.x & 63);
    if (turn) {
#pragma unroll
      for (int i = 0; i < TP / 16; ++i)
#pragma unroll
        for (int j = 0; j < TQ / 16; ++j) sums[((turn - 1) * NW * kFragments + i * (TQ / 16) + j) * 64] = acc[i][j];
    }
    __syncthreads();
    if (turn) return;
#pragma unroll
    for (int s = 1; s < SPLIT; ++s)
#pragma unroll
      for (int i = 0; i < TP / 16; ++i)
#pragma unroll
        for (int j = 0; j < TQ / 16; ++j) acc[i][j] += sums[((s - 1) * NW * kFragments + i * (TQ / 16) + j) * 64];
    // the epilogue's rows may lie over another wave's sums
    base += (SPLIT - 1) * BP * BQ * 4;
  }
  void* y = a.y;
  if constexpr (kWeight) y = static_cast<uint8_t*>(y) + it.group * a.y_stride * (a.out_type == MOE_T_F32 ? 4 : 2);
  epilogue<BF, EPI, TP, TQ>(a, it, acc, wp, wq, q_end, y, base);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
namespace {

constexpr int64_t kMaxGrid = 0x7fffff00;

// Whether k_group_tiles takes the operands: 16-byte aligned rows, whole
// 16-byte chunks along a straight contraction, every buffer below 2 GiB.
template <bool PA, bool QA>
bool direct(const Gemm& a) {
  constexpr int64_t kMost = 0x7fff0000;
  const auto fits = [](int64_t rows, int64_t ld) { return (rows + 4 * kRed) * ld * 2 < kMost; };
  if (reinterpret_cast<uintptr_t>(a.p) % 16 || reinterpret_cast<uintptr_t>(a.q) % 16) return false;
  if (a.ldp % 8 || a.ldq % 8 || a.p_stride % 8) return false;
  if (!QA && a.nr % 8) return false;
  if (PA && QA) return fits(a.rows, a.ldq) && fits(a.src ? a.src_rows : a.rows, a.ldp);
  return fits(PA ? a.nr : a.np, a.ldp) && fits(a.src ? a.src_rows : 256, a.ldq);
}

// Workgroups of a launch with tiles of BP x BQ (0: too many); fills in the tile counts.
template <bool WEIGHT, int EPI>
int64_t grid_of(Gemm& a, int BP, int BQ) {
  a.tiles_p = EPI == kSwigluOut ? (a.half + BP / 2 - 1) / (BP / 2) : (a.np + BP - 1) / BP;
  int64_t grid;
  if (WEIGHT) {
    a.tiles_q = (a.nq + BQ - 1) / BQ;
    const int64_t tiles = static_cast<int64_t>(a.tiles_p) * a.tiles_q;
    if (tiles > kMaxGrid / 8) return 0;
    grid = (tiles + 7) / 8 * 8 * a.groups;
  } else {
    // a group's last row tile may be partial: at most one more each
    const int64_t tq = a.rows / BQ + (a.rows < a.groups ? a.rows : a.groups);
    grid = (tq * a.tiles_p + 7) / 8 * 8;
  }
  return grid > kMaxGrid ? 0 : grid;
}

template <bool BF, bool PA, bool QA, int EPI, int BP, int BQ, int WP, int WQ, int STAGES, int SPLIT = 1>
int go(Gemm a, hipStream_t s) {
  const int64_t grid = grid_of<PA && QA, EPI>(a, BP, BQ);
  if (!grid) return MOE_ESHAPE;
  const dim3 g(static_cast<uint32_t>(grid)), b(64 * WP * WQ * SPLIT);
  if constexpr (STAGES == 0) hipLaunchKernelGGL((k_group_any<BF, PA, QA, EPI, BP, BQ, WP, WQ>), g, b, 0, s, a);
  else hipLaunchKernelGGL((k_group_tiles<BF, PA, QA, EPI, BP, BQ, WP, WQ, STAGES, SPLIT>), g, b, 0, s, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EDEVICE;
}

// Tile shapes.  A large tile asks least of the caches per product and runs the
// matrix cores best; small ones fill the chip with few rows or columns, keep
// more bytes in flight per compute unit when the weights' bytes bound the
// call, and end a step sooner when one tile's chain of steps does.  The
// shape is chosen by a model of the time:
//     max(compute, bytes) + min(compute, bytes) / 4
//     compute = rounds * fixed + steps * max(rounds * latency, tiles * step)
//     bytes   = touched weights / bandwidth
// with `tiles` per compute unit and `rounds` = tiles / (workgroups that fit).
// Its constants (us, us, us, -, TB/s) are fits to a sweep of every shape over
// 24 sizes, 1 .. 16384 rows in 1 .. 384 groups; measured, us (bf16):
//     rows x n x k (groups)      256x256  128x128  128x64   64x32
//     64 x 4096 x 4096 (1)            78       41      37      19
//     512 x 4096 x 4096 (1)           81       43      39      46
//     8192 x 2304 x 5120 (8)         272      238     283     481
//     16384 x 2304 x 5120 (16)       422      433     556    1028
//     12288 x 2304 x 5120 (384)     2134     1731    1731    1971
// and for weight gradients (64x64 in the last column)
//     8192 x 1024 x 1024 (1)         178      122     100      85
//     16384 x 5120 x 2304 (16)       441      525     587     728
// The last entry of each table is the small tile with its steps dealt to four
// groups of waves: 16 x 512 x 8192 34 -> 20 us, 64 x 4096 x 4096 19 -> 13, the
// weight gradient of 8192 x 1024 x 1024 85 -> 42; with many tiles it loses (512 x
// 4096 x 4096 39 -> 51), one workgroup filling a compute unit.
struct TileCost {
  int bp, bq;
  double fixed, latency, step;
  int fit;
  double bandwidth;
};
enum { kLarge, kMedium, kFlat, kSmall, kDeep };
constexpr TileCost kStraightCost[] = {{256, 256, 10, 1.15, 1.5, 1, 4.4}, {128, 128, 8, 0.58, 0.537, 2, 5.3},
                                      {128, 64, 4, 0.5, 0.33, 3, 5.0}, {64, 32, 3, 0.25, 0.144, 3, 5.3},
                                      {64, 32, 5, 0.12, 0.12, 1, 5.0}};
constexpr TileCost kAcrossCost[] = {{256, 256, 10, 1.25, 1.4, 1, 4.2}, {128, 128, 8, 0.82, 0.62, 2, 5.0},
                                    {128, 64, 4, 0.67, 0.36, 3, 4.8}, {64, 32, 3, 0.5, 0.21, 3, 4.5},
                                    {64, 32, 5, 0.2, 0.2, 1, 4.5}};
constexpr TileCost kWeightCost[] = {{256, 256, 9.2, 1.25, 1.6, 1, 5.0}, {128, 128, 5.2, 0.85, 0.75, 2, 5.0},
                                    {128, 64, 4, 0.75, 0.42, 3, 5.0}, {64, 64, 3.7, 0.63, 0.25, 5, 5.0},
                                    {64, 64, 4, 0.28, 0.28, 1, 5.0}};

// The register path, any operands:
//     8192 x 2303 x 5121 (8)         128x128 353, 64x64 599; gradients 343 / 560 and 317 / 511
//     512 x 4097 x 4097 (1)          69, 67
//     4096 x 511 x 513 (16), wgrad   33, 25
constexpr TileCost kAnyCost[] = {{128, 128, 5, 0.95, 0.87, 2, 3.6}, {64, 64, 3, 0.65, 0.38, 7, 3.6}};

template <bool PA, bool QA, int EPI, int N>
int tile_shape(const Gemm& a, const TileCost (&costs)[N]) {
  constexpr bool kWeight = PA && QA;
  const double held = a.rows < a.groups ? a.rows : a.groups;   // groups with rows, at most
  int best = 0;
  double least = 0;
  for (int i = 0; i < N; ++i) {
    const TileCost& c = costs[i];
    const double tp = EPI == kSwigluOut ? (2 * a.half + c.bp - 1) / c.bp : (a.np + c.bp - 1) / c.bp;
    double tiles, steps, bytes;
    if (kWeight) {
      tiles = a.groups * tp * ((a.nq + c.bq - 1) / c.bq);
      steps = held ? a.rows / held / kRed + 0.5 : 0.0;
      bytes = 0.0;
    } else {
      // a group's last row tile is half empty in the mean; each row tile past
      // a group's first reads its weights again, mostly from the caches
      double tq = a.groups == 1 ? (a.rows + c.bq - 1) / c.bq : a.rows / static_cast<double>(c.bq) + held / 2;
      tq = tq > held ? tq : held;
      tiles = tq * tp;
      steps = (a.nr + kRed - 1) / kRed;
      bytes = held * a.np * a.nr * 2e-6 / c.bandwidth * (0.75 + 0.25 * tq / held);
    }
    const double per_cu = __builtin_ceil(tiles / 256), rounds = __builtin_ceil(per_cu / c.fit);
    const double chain = rounds * c.latency, work = per_cu * c.step;
    double t = rounds * c.fixed + steps * (chain > work ? chain : work);
    // weight gradients: the tiles of a group with four times the mean rows end last
    if (kWeight) t += (a.groups < 4 ? a.groups - 1 : 3) * steps * c.latency;
    t = t > bytes ? t + bytes / 4 : bytes + t / 4;
    if (i == 0 || t < least) {
      best = i;
      least = t;
    }
  }
  return best;
}

template <bool BF, bool PA, bool QA, int EPI>
int launch(const Gemm& a, hipStream_t s) {
  if (!direct<PA, QA>(a)) {
    if (tile_shape<PA, QA, EPI>(a, kAnyCost) == 0) return go<BF, PA, QA, EPI, 128, 128, 2, 2, 0>(a, s);
    return go<BF, PA, QA, EPI, 64, 64, 2, 2, 0>(a, s);
  }
  switch (tile_shape<PA, QA, EPI>(a, PA && QA ? kWeightCost : PA ? kAcrossCost : kStraightCost)) {
    case kLarge: return go<BF, PA, QA, EPI, 256, 256, 2, 4, 2>(a, s);
    case kMedium: return go<BF, PA, QA, EPI, 128, 128, 2, 2, 2>(a, s);
    case kFlat: return go<BF, PA, QA, EPI, 128, 64, 2, 2, 2>(a, s);
    case kSmall:
      if constexpr (PA && QA) return go<BF, PA, QA, EPI, 64, 64, 2, 2, 2>(a, s);
      else return go<BF, PA, QA, EPI, 64, 32, 2, 2, 4>(a, s);
    default:
      if constexpr (PA && QA) return go<BF, PA, QA, EPI, 64, 64, 2, 2, 2, 4>(a, s);
      else return go<BF, PA, QA, EPI, 64, 32, 2, 2, 3, 4>(a, s);
  }
}

template <bool PA, bool QA, int EPI>
int launch_type(const moe_group_dims* d, const Gemm& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  return d->type == MOE_T_BF16 ? launch<true, PA, QA, EPI>(a, s) : launch<false, PA, QA, EPI>(a, s);
}

Gemm common(const moe_group_dims* d, const int32_t* src, const int32_t* offsets) {
  Gemm a{};
  a.offsets = offsets;
  a.src = src;
  a.groups = d->n_groups;
  a.rows = d->rows;
  a.src_rows = d->x_rows;
  // exact for entries below 2^31: with m = ceil(2^(32 + s) / d), the error of
  // u m / 2^(32 + s) is below u / 2^(32 + s) < 1 / d, as d < 2^(s + 1) or is a power of two
  a.div_shift = d->src_div <= 2 ? 0 : d->src_div <= 4 ? 1 : 2;
  a.div_mul = d->src_div == 1 ? 0 : static_cast<uint32_t>(((1ull << (32 + a.div_shift)) + d->src_div - 1) / d->src_div);
  a.ldy = d->ldy;
  a.ld_pre = d->ld_pre;
  a.out_type = d->out_type;
  return a;
}

Gemm products(const moe_group_dims* d, const void* x, const int32_t* src, const int32_t* offsets, const void* w,
              void* y, int np, int nr) {
  Gemm a = common(d, src, offsets);
  a.p = static_cast<const uint16_t*>(w);
  a.q = static_cast<const uint16_t*>(x);
  a.y = y;
  a.ldp = d->ldw;
  a.ldq = d->ldx;
  a.p_stride = d->w_stride;
  a.np = np;
  a.nr = d->x_rows ? nr : 0;   // no row to read: every sum is empty
  return a;
}

}  // namespace
}  // namespace grp
}  // namespace moe

extern "C" {

using namespace moe::grp;

int moe_group_matmul(const moe_group_dims* d, const void* x, const int32_t* src, const int32_t* offsets,
                     const void* w, void* y, void* stream) {
  if (int st = check_group(d, kMatmul, src, false)) return st;
  if (d->rows == 0) return MOE_OK;
  if ((!x && d->x_rows) || !offsets || !w || !y) return MOE_EINVAL;
  return launch_type<false, false, kStore>(d, products(d, x, src, offsets, w, y, d->n, d->k), stream);
}

int moe_group_swiglu(const moe_group_dims* d, const void* x, const int32_t* src, const int32_t* offsets,
                     const void* w, void* h, void* pre, void* stream) {
  if (int st = check_group(d, kSwiglu, src, pre)) return st;
  if (d->rows == 0) return MOE_OK;
  if ((!x && d->x_rows) || !offsets || !w || !h) return MOE_EINVAL;
  Gemm a = products(d, x, src, offsets, w, h, d->n, d->k);
  a.half = d->n / 2;
  a.pre_out = static_cast<uint16_t*>(pre);
  return launch_type<false, false, kSwigluOut>(d, a, stream);
}

int moe_group_matmul_t(const moe_group_dims* d, const void* dy, const int32_t* src, const int32_t* offsets,
                       const void* w, void* dx, void* stream) {
  if (int st = check_group(d, kMatmulT, src, false)) return st;
  if (d->rows == 0) return MOE_OK;
  if ((!dy && d->x_rows) || !offsets || !w || !dx) return MOE_EINVAL;
  return launch_type<true, false, kStore>(d, products(d, dy, src, offsets, w, dx, d->k, d->n), stream);
}

int moe_group_swiglu_grad(const moe_group_dims* d, const void* dy, const int32_t* src, const int32_t* offsets,
                          const void* w, const void* pre, void* dpre, void* stream) {
  if (int st = check_group(d, kSwigluGrad, src, true)) return st;
  if (d->rows == 0) return MOE_OK;
  if ((!dy && d->x_rows) || !offsets || !w || !pre || !dpre) return MOE_EINVAL;
  Gemm a = products(d, dy, src, offsets, w, dpre, d->k, d->n);
  a.pre_in = static_cast<const uint16_t*>(pre);
  return launch_type<true, false, kSwigluBack>(d, a, stream);
}

int moe_group_wgrad(const moe_group_dims* d, const void* dy, const void* x, const int32_t* src,
                    const int32_t* offsets, void* dw, int32_t accumulate, void* stream) {
  if (int st = check_group(d, kWgrad, src, false)) return st;
  if (!offsets || !dw || (d->rows && (!dy || (!x && d->x_rows)))) return MOE_EINVAL;
  Gemm a = common(d, src, offsets);
  if (d->x_rows == 0) a.rows = 0;   // no row to read: every group is empty
  a.p = static_cast<const uint16_t*>(x);
  a.q = static_cast<const uint16_t*>(dy);
  a.y = dw;
  a.ldp = d->ldx;
  a.ldq = d->ldy;
  a.ldy = d->ldw;
  a.y_stride = d->w_stride;
  a.np = d->k;
  a.nq = d->n;
  a.accumulate = accumulate != 0;
  return launch_type<true, true, kStore>(d, a, stream);
}

}  // extern "C"
