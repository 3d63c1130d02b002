// Shared by the expert-grouped operators and the 4-bit matrix-vector product:
// host-side argument checks (plain C++, no HIP) and sizes.
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/moe.h"

namespace moe {
namespace grp {

// Pairs per workgroup of the dispatch; up to this many, one workgroup makes
// the whole plan and no workspace is used.
constexpr int kPlanChunk = 2048;

enum Call { kMatmul, kSwiglu, kMatmulT, kSwigluGrad, kWgrad };

inline bool half_type(int t) { return t == MOE_T_BF16 || t == MOE_T_F16; }
inline bool known_type(int t) { return t == MOE_T_F32 || half_type(t); }

int check_plan(int rows, int top_k, int n_groups);
int check_group(const moe_group_dims* d, Call call, bool gathered, bool has_pre);
int check_combine(const moe_combine_dims* d);
int check_q4(const moe_q4_dims* d);

// Whole 16 x 128 tiles of a 4-bit matrix.
inline int64_t q4_tiles_n(int64_t n) { return (n + 15) / 16; }
inline int64_t q4_tiles_k(int64_t k) { return (k + 127) / 128; }

}  // namespace grp
}  // namespace moe
