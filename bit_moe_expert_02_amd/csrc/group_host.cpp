// Host code of the expert-grouped operators and of the 4-bit format: argument
// checks, sizes, packing and unpacking.  Plain C++ with no HIP calls.
#include "group.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <system_error>
#include <thread>
#include <vector>

#include "host_common.h"

namespace moe {
namespace grp {

int check_plan(int rows, int top_k, int n_groups) {
  if (rows < 0) return MOE_EINVAL;
  if (top_k < 1 || top_k > MOE_MAX_TOP_K || n_groups < 1 || n_groups > MOE_MAX_GROUPS) return MOE_ESHAPE;
  if (static_cast<int64_t>(rows) * top_k > INT32_MAX) return MOE_ESHAPE;
  return MOE_OK;
}

namespace {
// the last element of a [rows x cols] array with row stride ld has to lie
// within what a signed 64-bit byte offset reaches
bool span_ok(int64_t rows, int64_t cols, int64_t ld) {
  return ld >= cols && (rows <= 1 || ld <= (INT64_MAX / 16) / rows);
}
}  // namespace

int check_group(const moe_group_dims* d, Call call, bool gathered, bool has_pre) {
  if (!d || d->rows < 0 || d->x_rows < 0) return MOE_EINVAL;
  if (!half_type(d->type) || !known_type(d->out_type)) return MOE_EFORMAT;
  if (d->n_groups < 1 || d->n_groups > MOE_MAX_GROUPS || d->n < 1 || d->k < 1) return MOE_ESHAPE;
  if (d->src_div < 1 || d->src_div > MOE_MAX_TOP_K) return MOE_ESHAPE;
  if (!gathered && d->x_rows < d->rows) return MOE_ESHAPE;
  if (call == kSwiglu && d->n % 2) return MOE_ESHAPE;
  // 2 I columns of dpre, and tile counts, stay within 32 bits
  if (d->n > (1 << 28) || d->k > (1 << 28)) return MOE_ESHAPE;
  const int64_t n = d->n, k = d->k;
  const int64_t x_cols = call == kMatmulT || call == kSwigluGrad ? n : k;
  const int64_t y_cols = call == kMatmul || call == kWgrad ? n : call == kSwiglu ? n / 2 : call == kMatmulT ? k : 2 * k;
  if (!span_ok(d->x_rows, x_cols, d->ldx) || !span_ok(d->rows, y_cols, d->ldy) || !span_ok(n, k, d->ldw))
    return MOE_ESHAPE;
  if (has_pre && !span_ok(d->rows, call == kSwiglu ? n : 2 * k, d->ld_pre)) return MOE_ESHAPE;
  if (d->w_stride < 0 || d->w_stride > INT64_MAX / 16 / MOE_MAX_GROUPS) return MOE_ESHAPE;
  // gradients of different experts may not share memory (a stride of 0 would
  // be one matrix for every group, which only reading can share)
  if (call == kWgrad && d->n_groups > 1 && d->w_stride < (n - 1) * d->ldw + k) return MOE_ESHAPE;
  return MOE_OK;
}

int check_combine(const moe_combine_dims* d) {
  if (!d || d->rows < 0 || d->o_rows < 0) return MOE_EINVAL;
  if (!known_type(d->type) || !known_type(d->out_type)) return MOE_EFORMAT;
  if (d->n < 1 || d->top_k < 1 || d->top_k > MOE_MAX_TOP_K) return MOE_ESHAPE;
  if (static_cast<int64_t>(d->rows) * d->top_k > INT32_MAX || d->n > (1 << 28)) return MOE_ESHAPE;
  if (!span_ok(d->o_rows, d->n, d->ldo) || !span_ok(d->rows, d->n, d->ldy)) return MOE_ESHAPE;
  return MOE_OK;
}

namespace {
int check_q4_shape(int64_t n, int64_t k, int32_t group) {
  if (n < 1 || k < 1 || n > INT32_MAX || k > INT32_MAX) return MOE_ESHAPE;
  if ((group != 32 && group != 64 && group != 128) || k % group) return MOE_ESHAPE;
  return MOE_OK;
}

// Runs body(first, last) over [0, count) on up to nthreads threads; a thread
// that cannot be started has its share run here.
template <class F>
void over_threads(int64_t count, int nthreads, F body) {
  int64_t t = nthreads > 0 ? nthreads : static_cast<int64_t>(std::thread::hardware_concurrency());
  t = std::max<int64_t>(1, std::min<int64_t>(t, count));
  const int64_t per = (count + t - 1) / t;
  std::vector<std::thread> pool;
  int64_t at = per;
  try {
    pool.reserve(static_cast<size_t>(t));
    for (; at < count; at += per) pool.emplace_back(body, at, std::min(count, at + per));
  } catch (const std::exception&) {
  }
  body(0, std::min(count, per));
  for (std::thread& p : pool) p.join();
  for (; at < count; at += per) body(at, std::min(count, at + per));
}

struct Q4View {
  int64_t n, k, kt, ng;   // ng: groups of a padded row
  int group;
  int64_t word(int64_t row, int64_t col) const {   // 32-bit word of codes
    const int64_t in = col % 128;
    return (((row / 16) * kt + col / 128) * 4 + (in % 32) / 8) * 64 + (row % 16) * 4 + in / 32;
  }
  int64_t per_group(int64_t row, int64_t g) const { return ((row / 16) * ng + g) * 16 + row % 16; }
};

Q4View q4_view(int64_t n, int64_t k, int group) {
  const int64_t kt = q4_tiles_k(k);
  return Q4View{n, k, kt, kt * 128 / group, group};
}
}  // namespace

int check_q4(const moe_q4_dims* d) {
  if (!d || d->rows < 0) return MOE_EINVAL;
  if (!half_type(d->type) || !known_type(d->out_type)) return MOE_EFORMAT;
  if (int st = check_q4_shape(d->n, d->k, d->group)) return st;
  if (d->swiglu != 0 && d->swiglu != 1) return MOE_EINVAL;
  if (d->rows > MOE_MAX_Q4_ROWS || d->n_mats < 1 || d->x_div < 1) return MOE_ESHAPE;
  if (d->swiglu && d->n % 32) return MOE_ESHAPE;
  if (d->n > (1 << 26) || d->k > (1 << 24)) return MOE_ESHAPE;
  if (!span_ok(d->rows, d->k, d->ldx) || !span_ok(d->rows, d->swiglu ? d->n / 2 : d->n, d->ldy)) return MOE_ESHAPE;
  return MOE_OK;
}

}  // namespace grp
}  // namespace moe

extern "C" {

size_t moe_group_plan_bytes(int32_t rows, int32_t top_k, int32_t n_groups) {
  if (moe::grp::check_plan(rows, top_k, n_groups)) return 0;
  const int64_t pairs = static_cast<int64_t>(rows) * top_k;
  if (pairs <= moe::grp::kPlanChunk) return 0;
  const int64_t chunks = (pairs + moe::grp::kPlanChunk - 1) / moe::grp::kPlanChunk;
  return static_cast<size_t>(4 * n_groups * (chunks + 1));
}

int moe_q4_bytes(int64_t n, int64_t k, int32_t group, size_t* codes, size_t* scales, size_t* zeros) {
  using namespace moe::grp;
  if (int st = check_q4_shape(n, k, group)) return st;
  const size_t tn = static_cast<size_t>(q4_tiles_n(n)), tk = static_cast<size_t>(q4_tiles_k(k));
  const size_t groups = tn * 16 * (tk * 128 / group);
  if (codes) *codes = tn * tk * 1024;
  if (scales) *scales = groups * 2;
  if (zeros) *zeros = groups;
  return MOE_OK;
}

int moe_q4_pack(const float* w, int64_t n, int64_t k, int32_t group, void* codes, void* scales, void* zeros,
                int32_t nthreads) {
  using namespace moe::grp;
  if (!w || !codes || !scales) return MOE_EINVAL;
  if (int st = check_q4_shape(n, k, group)) return st;
  const Q4View v = q4_view(n, k, group);
  uint32_t* cw = static_cast<uint32_t*>(codes);
  uint16_t* sc = static_cast<uint16_t*>(scales);
  uint8_t* zr = static_cast<uint8_t*>(zeros);
  over_threads(q4_tiles_n(n), nthreads, [=](int64_t t0, int64_t t1) {
    for (int64_t row = t0 * 16; row < t1 * 16; ++row)
      for (int64_t g = 0; g < v.ng; ++g) {
        const int64_t c0 = g * group;
        const bool held = row < n && c0 < k;       // groups divide k: a group is inside or past it
        const float* src = held ? w + row * k + c0 : nullptr;
        float lo = 0.0f, hi = 0.0f;
        for (int i = 0; held && i < group; ++i) {
          lo = std::min(lo, src[i]);
          hi = std::max(hi, src[i]);
        }
        const float step = zr ? (hi - lo) / 15.0f : std::max(-lo, hi) / 7.0f;
        const uint16_t dh = moe::f32_to_f16_sat(step);
        const float d = moe::f16_to_f32(dh);
        float z = zr ? 0.0f : 8.0f;
        if (zr && d > 0.0f) z = std::min(15.0f, std::max(0.0f, std::nearbyint(-lo / d)));
        sc[v.per_group(row, g)] = d > 0.0f ? dh : 0;
        if (zr) zr[v.per_group(row, g)] = static_cast<uint8_t>(z);
        for (int i = 0; i < group; i += 8) {
          uint32_t word = 0;
          for (int e = 0; e < 8; ++e) {
            float c = z;
            if (d > 0.0f) c = std::min(15.0f, std::max(0.0f, std::nearbyint(src[i + e] / d) + z));
            if (!(c >= 0.0f)) c = z;               // NaN input: an unspecified, valid code
            word |= static_cast<uint32_t>(c) << (4 * e);
          }
          cw[v.word(row, c0 + i)] = word;
        }
      }
  });
  return MOE_OK;
}

int moe_q4_unpack(const void* codes, const void* scales, const void* zeros, int64_t n, int64_t k, int32_t group,
                  float* w, int32_t nthreads) {
  using namespace moe::grp;
  if (!w || !codes || !scales) return MOE_EINVAL;
  if (int st = check_q4_shape(n, k, group)) return st;
  const Q4View v = q4_view(n, k, group);
  const uint32_t* cw = static_cast<const uint32_t*>(codes);
  const uint16_t* sc = static_cast<const uint16_t*>(scales);
  const uint8_t* zr = static_cast<const uint8_t*>(zeros);
  over_threads(n, nthreads, [=](int64_t r0, int64_t r1) {
    for (int64_t row = r0; row < r1; ++row)
      for (int64_t c = 0; c < k; c += 8) {
        const uint32_t word = cw[v.word(row, c)];
        const float d = moe::f16_to_f32(sc[v.per_group(row, c / group)]);
        const int z = zr ? zr[v.per_group(row, c / group)] : 8;
        for (int e = 0; e < 8; ++e)
          w[row * k + c + e] = d * static_cast<float>(static_cast<int>(word >> (4 * e) & 15u) - z);
      }
  });
  return MOE_OK;
}

}  // extern "C"
