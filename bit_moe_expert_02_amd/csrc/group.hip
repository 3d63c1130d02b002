// gfx950 dispatch and combine of the expert-grouped path: routing ids to
// offsets / sorted pairs / positions, the weighted sum over a row's experts,
// and its gradients.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "dev_common.h"
#include "group.h"

namespace moe {
namespace grp {

using dev::u32x2;
using dev::u32x4;
typedef float f32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Dispatch: a stable counting sort of the pairs by expert id.
//
// A workgroup owns kPlanChunk consecutive pairs, a wave 128 of them in two
// rounds of 64.  In a round, the lanes with one id find each other with a
// ballot per bit of the id (no atomics, so the order is fixed): a pair's rank
// among them is the number of such lanes below it, and the lowest one adds
// their count to the wave's counter of that id.  A scan over the waves and
// the earlier workgroups' counts turns ranks into places.  Up to kPlanChunk
// pairs one workgroup does it all; past that, k_plan_count leaves each chunk's
// counts in the workspace and k_plan_place repeats the ranking with the sums of
// the earlier chunks' as bases.  Each workgroup adds those up itself as long
// as that is less reading than a launch takes time (kSumChunks); past it
// k_plan_scan sums along the chunks in between.  196,608 pairs of 384 ids (96
// chunks): 13.1 us with the scan's launch, 12.4 without, of which counting takes
// 4.8 and placing 9.0 (in kernels; the bytes would take 0.5).  48 pairs: 4.2 us.
// Latency bounds both: launch, ids, ballots, sums and stores follow each other.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kRounds = kPlanChunk / kPlanThreads;
constexpr int kNone = 2047;   // past every group id: 11 bits
constexpr int kSumChunks = 256;

struct Plan {
  const int32_t* idx;
  int32_t *offsets, *pairs, *pos;
  int32_t* ws;                  // [chunks + 1][groups]
  int pairs_n, groups, chunks;
};

// Lanes of the wave whose id is this lane's.
__device__ __forceinline__ uint64_t same_id(int id) {
  uint64_t m = ~0ull;
#pragma unroll
  for (int b = 0; b < 11; ++b) {
    const uint64_t v = __ballot(id >> b & 1);
    m &= id >> b & 1 ? v : ~v;
  }
  return m;
}

// Ranks of this thread's pairs among the wave's pairs with the same id, and
// the wave's counts per id in `count` (its own row, zeroed).
__device__ __forceinline__ void rank_pairs(const Plan& a, int chunk, int (&id)[kRounds], int (&rank)[kRounds],
                                           int32_t* count) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t first = static_cast<int64_t>(chunk) * kPlanChunk + wave * 64 * kRounds + lane;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t p = first + 64 * r;
    id[r] = p < a.pairs_n ? a.idx[p] : -1;
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const bool in = id[r] >= 0 && id[r] < a.groups;
    const uint64_t m = same_id(in ? id[r] : kNone);
    const int below = __popcll(m & ((1ull << lane) - 1));
    int held = 0;
    if (in) held = count[id[r]];
    rank[r] = held + below;
    __builtin_amdgcn_wave_barrier();
    if (in && below == 0) count[id[r]] = held + __popcll(m);
    __builtin_amdgcn_wave_barrier();
  }
}

__device__ __forceinline__ int inclusive_wave(int v) {
  const int lane = threadIdx.x & 63;
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}

// Writes this chunk's places.  total(e) / before(e): pairs of id e in all
// chunks / in earlier chunks.  count [kPlanWaves][groups] is the waves'
// counts on entry.
template <class T, class B>
__device__ __forceinline__ void place_pairs(const Plan& a, int chunk, const int (&id)[kRounds], const int (&rank)[kRounds],
                                            int32_t* count, int32_t* part, T total, B before) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  // MOE_MAX_GROUPS is the workgroup's size: one id a thread
  const int tot = tid < a.groups ? total(tid) : 0;
  const int upto = inclusive_wave(tot);
  if (lane == 63) part[wave] = upto;
  __syncthreads();
  int base = upto - tot, all = 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    const int v = part[w];
    if (w < wave) base += v;
    all += v;
  }
  if (chunk == 0) {
    if (tid < a.groups) a.offsets[tid] = base;
    if (tid == 0) a.offsets[a.groups] = all;
  }
  if (tid < a.groups) {
    int at = base + before(tid);
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = count[w * a.groups + tid];
      count[w * a.groups + tid] = at;
      at += c;
    }
  }
  __syncthreads();
  const int64_t first = static_cast<int64_t>(chunk) * kPlanChunk + wave * 64 * kRounds + lane;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int64_t p = first + 64 * r;
    if (p >= a.pairs_n) continue;
    int at = id[r] == -1 ? -1 : -2;
    if (id[r] >= 0 && id[r] < a.groups) {
      at = count[wave * a.groups + id[r]] + rank[r];
      a.pairs[at] = static_cast<int32_t>(p);
    }
    a.pos[p] = at;
    if (p >= all) a.pairs[p] = -1;
  }
}

extern __shared__ int32_t plan_lds[];   // [kPlanWaves][groups] counts, then kPlanWaves partial sums

__device__ __forceinline__ void clear_counts(const Plan& a) {
  for (int i = threadIdx.x; i < kPlanWaves * a.groups; i += kPlanThreads) plan_lds[i] = 0;
  __syncthreads();
}

__global__ __launch_bounds__(kPlanThreads) void k_plan_small(Plan a) {
  int id[kRounds], rank[kRounds];
  clear_counts(a);
  rank_pairs(a, 0, id, rank, plan_lds + (threadIdx.x >> 6) * a.groups);
  __syncthreads();
  place_pairs(
      a, 0, id, rank, plan_lds, plan_lds + kPlanWaves * a.groups,
      [&](int e) {
        int s = 0;
        for (int w = 0; w < kPlanWaves; ++w) s += plan_lds[w * a.groups + e];
        return s;
      },
      [](int) { return 0; });
}

__global__ __launch_bounds__(kPlanThreads) void k_plan_count(Plan a) {
  int id[kRounds], rank[kRounds];
  clear_counts(a);
  rank_pairs(a, blockIdx.x, id, rank, plan_lds + (threadIdx.x >> 6) * a.groups);
  __syncthreads();
  for (int e = threadIdx.x; e < a.groups; e += kPlanThreads) {
    int s = 0;
    for (int w = 0; w < kPlanWaves; ++w) s += plan_lds[w * a.groups + e];
    a.ws[static_cast<int64_t>(blockIdx.x) * a.groups + e] = s;
  }
}

// One wave per id: exclusive sums along the chunks, the total in the last row.
__global__ __launch_bounds__(64) void k_plan_scan(Plan a) {
  const int e = blockIdx.x, lane = threadIdx.x;
  int base = 0;
  for (int c0 = 0; c0 < a.chunks; c0 += 64) {
    const int c = c0 + lane;
    int32_t* at = a.ws + static_cast<int64_t>(c) * a.groups + e;
    const int v = c < a.chunks ? *at : 0;
    const int upto = inclusive_wave(v);
    if (c < a.chunks) *at = base + upto - v;
    base += __shfl(upto, 63, 64);
  }
  if (lane == 0) a.ws[static_cast<int64_t>(a.chunks) * a.groups + e] = base;
}

template <bool SCANNED>
__global__ __launch_bounds__(kPlanThreads) void k_plan_place(Plan a) {
  int id[kRounds], rank[kRounds];
  const int chunk = blockIdx.x, e = threadIdx.x;
  // this thread's id: its pairs in earlier chunks and in all
  int before = 0, total = 0;
  if (e < a.groups) {
    if constexpr (SCANNED) {
      before = a.ws[static_cast<int64_t>(chunk) * a.groups + e];
      total = a.ws[static_cast<int64_t>(a.chunks) * a.groups + e];
    } else {
#pragma unroll 32
      for (int c = 0; c < a.chunks; ++c) {
        const int v = a.ws[c * a.groups + e];
        before += c < chunk ? v : 0;
        total += v;
      }
    }
  }
  clear_counts(a);
  rank_pairs(a, chunk, id, rank, plan_lds + (threadIdx.x >> 6) * a.groups);
  __syncthreads();
  place_pairs(
      a, chunk, id, rank, plan_lds, plan_lds + kPlanWaves * a.groups, [&](int) { return total; }, [&](int) { return before; });
}

// ---------------------------------------------------------------------------
// Combine: bound by bytes (gradients of 8192 x 6 rows of 5120 in bf16: 219 us
// for 1.09 GB, 5.0 TB/s, what a large copy reaches; the sums of 8 x 6 rows: 5 us,
// latency).  A thread takes V consecutive columns of a row (one
// 16-byte load of each operand where alignment allows, V = 8 or 4, else V =
// 1) and loads the row's top_k pieces before it adds the first.
// ---------------------------------------------------------------------------
constexpr int kCombineThreads = 256;

struct Combine {
  const void* o;
  const int32_t* pos;
  const float* wts;
  void* y;                  // forward
  const void* dy;           // backward
  void* d_o;
  float* d_wts;
  int64_t ldo, ldy;
  int rows, top_k, n, o_rows, out_type;
};

template <int T, int V>
__device__ __forceinline__ void load_v(const void* base, int64_t at, float (&v)[V]) {
  if constexpr (T == MOE_T_F32) {
    const float* p = static_cast<const float*>(base) + at;
    if constexpr (V == 4) {
      const float4 q = *reinterpret_cast<const float4*>(p);
      v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
      for (int i = 0; i < V; ++i) v[i] = p[i];
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    uint16_t h[V];
    if constexpr (V == 8) {
      const u32x4 q = *reinterpret_cast<const u32x4*>(p);
      __builtin_memcpy(h, &q, 16);
    } else {
      for (int i = 0; i < V; ++i) h[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      v[i] = T == MOE_T_BF16 ? static_cast<float>(__builtin_bit_cast(__bf16, h[i]))
                             : static_cast<float>(__builtin_bit_cast(_Float16, h[i]));
  }
}

// One rounding to the output's type; V > 1 stores are aligned to their size.
template <int V>
__device__ __forceinline__ void store_v(void* base, int64_t at, const float (&v)[V], int type) {
  if (type == MOE_T_F32) {
    float* p = static_cast<float*>(base) + at;
    if constexpr (V >= 4) {
#pragma unroll
      for (int i = 0; i < V; i += 4)
        __builtin_nontemporal_store(f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]}, reinterpret_cast<f32x4*>(p + i));
    } else {
      p[0] = v[0];
    }
    return;
  }
  uint16_t h[V];
#pragma unroll
  for (int i = 0; i < V; ++i)
    h[i] = type == MOE_T_BF16 ? __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[i]))
                              : __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[i]));
  uint16_t* p = static_cast<uint16_t*>(base) + at;
  if constexpr (V == 8) {
    u32x4 q;
    __builtin_memcpy(&q, h, 16);
    __builtin_nontemporal_store(q, reinterpret_cast<u32x4*>(p));
  } else if constexpr (V == 4) {
    u32x2 q;
    __builtin_memcpy(&q, h, 8);
    __builtin_nontemporal_store(q, reinterpret_cast<u32x2*>(p));
  } else {
    p[0] = h[0];
  }
}

// Place of pair p: -1 none, -2 not a row of o.
__device__ __forceinline__ int64_t place_of(const Combine& a, int64_t p) {
  const int64_t at = a.pos ? a.pos[p] : p;
  return at >= 0 && at < a.o_rows ? at : at == -1 ? -1 : -2;
}

template <int T, int V>
__global__ __launch_bounds__(kCombineThreads) void k_combine_rows(Combine a) {
  const int64_t per = (a.n + V - 1) / V;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kCombineThreads + threadIdx.x;
  if (at >= per * a.rows) return;
  const int64_t r = at / per;
  const int64_t c = (at - r * per) * V;
  float v[MOE_MAX_TOP_K][V], w[MOE_MAX_TOP_K];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < MOE_MAX_TOP_K; ++j) {
    w[j] = 0.0f;
    if (j >= a.top_k) continue;
    const int64_t pl = place_of(a, r * a.top_k + j);
    bad |= pl == -2;
    if (pl < 0) continue;
    w[j] = a.wts ? a.wts[r * a.top_k + j] : 1.0f;
    load_v<T, V>(a.o, pl * a.ldo + c, v[j]);
  }
  float s[V] = {};
#pragma unroll
  for (int j = 0; j < MOE_MAX_TOP_K; ++j) {
    if (j >= a.top_k || place_of(a, r * a.top_k + j) < 0) continue;
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] += w[j] * v[j][i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = bad ? __builtin_nanf("") : s[i];
  store_v<V>(a.y, r * a.ldy + c, s, a.out_type);
}

// One workgroup a row: dy stays in registers for the row's top_k pairs.
template <int T, int V>
__global__ __launch_bounds__(kCombineThreads) void k_combine_back(Combine a) {
  __shared__ float part[kCombineThreads / 64][MOE_MAX_TOP_K];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x;
  int64_t pl[MOE_MAX_TOP_K];
  float w[MOE_MAX_TOP_K], dot[MOE_MAX_TOP_K] = {};
#pragma unroll
  for (int j = 0; j < MOE_MAX_TOP_K; ++j) {
    pl[j] = j < a.top_k ? place_of(a, r * a.top_k + j) : -1;
    w[j] = j < a.top_k && a.wts ? a.wts[r * a.top_k + j] : 1.0f;
  }
  for (int c = tid * V; c < a.n; c += kCombineThreads * V) {
    float g[V];
    load_v<T, V>(a.dy, r * a.ldy + c, g);
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOP_K; ++j) {
      if (pl[j] < 0) continue;
      if (a.d_wts) {
        float v[V];
        load_v<T, V>(a.o, pl[j] * a.ldo + c, v);
#pragma unroll
        for (int i = 0; i < V; ++i) dot[j] += g[i] * v[i];
      }
      if (a.d_o) {
        float v[V];
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = w[j] * g[i];
        store_v<V>(a.d_o, pl[j] * a.ldo + c, v, a.out_type);
      }
    }
  }
  if (!a.d_wts) return;
#pragma unroll
  for (int j = 0; j < MOE_MAX_TOP_K; ++j) {
    const float s = dev::group_sum<64>(dot[j]);
    if ((tid & 63) == 0) part[tid >> 6][j] = s;
  }
  __syncthreads();
  if (tid < a.top_k) {
    float s = 0.0f;
    for (int i = 0; i < kCombineThreads / 64; ++i) s += part[i][tid];
    const int64_t at = place_of(a, r * a.top_k + tid);
    a.d_wts[r * a.top_k + tid] = at >= 0 ? s : at == -1 ? 0.0f : __builtin_nanf("");
  }
}

namespace {

bool aligned(const void* p, int64_t ld, int type) {
  const int64_t bytes = type == MOE_T_F32 ? 4 : 2;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * bytes % 16 == 0;
}

template <int T>
int run_combine(const Combine& a, bool back, bool vec, hipStream_t s) {
  constexpr int V = T == MOE_T_F32 ? 4 : 8;
  if (back) {
    const dim3 grid(a.rows), block(kCombineThreads);
    if (vec) hipLaunchKernelGGL((k_combine_back<T, V>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_combine_back<T, 1>), grid, block, 0, s, a);
  } else {
    const int64_t per = vec ? (a.n + V - 1) / V : a.n;
    const int64_t blocks = (per * a.rows + kCombineThreads - 1) / kCombineThreads;
    if (blocks > INT32_MAX) return MOE_ESHAPE;
    const dim3 grid(static_cast<uint32_t>(blocks)), block(kCombineThreads);
    if (vec) hipLaunchKernelGGL((k_combine_rows<T, V>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_combine_rows<T, 1>), grid, block, 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EDEVICE;
}

int run_combine(const moe_combine_dims* d, const Combine& a, bool back, void* stream) {
  const int V = d->type == MOE_T_F32 ? 4 : 8;
  // vector accesses: whole pieces, every row of every array 16-byte aligned
  bool vec = d->n % V == 0;
  if (a.o) vec = vec && aligned(a.o, d->ldo, d->type);
  if (back) {
    vec = vec && aligned(a.dy, d->ldy, d->type);
    if (a.d_o) vec = vec && aligned(a.d_o, d->ldo, d->out_type);
  } else {
    vec = vec && aligned(a.y, d->ldy, d->out_type);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (d->type) {
    case MOE_T_F32: return run_combine<MOE_T_F32>(a, back, vec, s);
    case MOE_T_BF16: return run_combine<MOE_T_BF16>(a, back, vec, s);
    default: return run_combine<MOE_T_F16>(a, back, vec, s);
  }
}

Combine combine_args(const moe_combine_dims* d, const void* o, const int32_t* pos, const float* wts) {
  Combine a{};
  a.o = o;
  a.pos = pos;
  a.wts = wts;
  a.ldo = d->ldo;
  a.ldy = d->ldy;
  a.rows = d->rows;
  a.top_k = d->top_k;
  a.n = d->n;
  a.o_rows = d->o_rows;
  a.out_type = d->out_type;
  return a;
}

}  // namespace
}  // namespace grp
}  // namespace moe

extern "C" {

using namespace moe::grp;

int moe_group_plan(const int32_t* idx, int32_t rows, int32_t top_k, int32_t n_groups, int32_t* offsets,
                   int32_t* pairs, int32_t* pos, void* ws, size_t ws_bytes, void* stream) {
  if (int st = check_plan(rows, top_k, n_groups)) return st;
  if (!offsets || (rows && (!idx || !pairs || !pos))) return MOE_EINVAL;
  const size_t need = moe_group_plan_bytes(rows, top_k, n_groups);
  if (need && !ws) return MOE_EINVAL;
  if (ws_bytes < need) return MOE_EWORKSPACE;
  if (need && reinterpret_cast<uintptr_t>(ws) % 4) return MOE_EINVAL;
  Plan a{idx, offsets, pairs, pos, static_cast<int32_t*>(ws), rows * top_k, n_groups, 0};
  a.chunks = static_cast<int>((static_cast<int64_t>(a.pairs_n) + kPlanChunk - 1) / kPlanChunk);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t lds = 4 * (static_cast<size_t>(kPlanWaves) * n_groups + kPlanWaves);
  if (!need) {
    hipLaunchKernelGGL(k_plan_small, dim3(1), dim3(kPlanThreads), lds, s, a);
  } else {
    hipLaunchKernelGGL(k_plan_count, dim3(a.chunks), dim3(kPlanThreads), lds, s, a);
    if (a.chunks <= kSumChunks) {
      hipLaunchKernelGGL(k_plan_place<false>, dim3(a.chunks), dim3(kPlanThreads), lds, s, a);
    } else {
      hipLaunchKernelGGL(k_plan_scan, dim3(n_groups), dim3(64), 0, s, a);
      hipLaunchKernelGGL(k_plan_place<true>, dim3(a.chunks), dim3(kPlanThreads), lds, s, a);
    }
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EDEVICE;
}

int moe_group_combine(const moe_combine_dims* d, const void* o, const int32_t* pos, const float* wts, void* y,
                      void* stream) {
  if (int st = check_combine(d)) return st;
  if (d->rows == 0) return MOE_OK;
  if (!y || (!o && d->o_rows)) return MOE_EINVAL;
  if (!pos && d->o_rows < d->rows * d->top_k) return MOE_ESHAPE;
  Combine a = combine_args(d, o, pos, wts);
  a.y = y;
  return run_combine(d, a, false, stream);
}

int moe_group_combine_grad(const moe_combine_dims* d, const void* dy, const void* o, const int32_t* pos,
                           const float* wts, void* d_o, float* d_wts, void* stream) {
  if (int st = check_combine(d)) return st;
  if (d->rows == 0 || (!d_o && !d_wts)) return MOE_OK;
  if (!dy || (d_wts && !o && d->o_rows)) return MOE_EINVAL;
  if (!pos && d->o_rows < d->rows * d->top_k) return MOE_ESHAPE;
  Combine a = combine_args(d, d_wts ? o : nullptr, pos, wts);
  a.dy = dy;
  a.d_o = d_o;
  a.d_wts = d_wts;
  return run_combine(d, a, true, stream);
}

}  // extern "C"
