// delta_device.hpp -- what the gated delta rule's kernels share: the workspace
// of a chunk, operand fragments, and the numbering of their rows.
//
// Per chunk of C = 64 tokens and head, with G_t the running sum of dt A,
// M_tj = exp(G_t - G_j) (0 across a document start) and S0 the state entering:
//     L_tj = beta_t M_tj k_t.k_j  (j < t)      T = (I + L)^-1
//     X = V - e^G K S0        U = T (beta X)   Att_tj = scale M_tj q_t.k_j  (j <= t)
//     Y = scale e^G Q S0 + Att U               S_C = e^{G_C} S0 + (e^{G_C - G} K)^T U
// q and k enter the products as they are in memory; their norms, like the
// decays, multiply rows of the fp32 results.
#pragma once

#include "ssd_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {
namespace delta {

constexpr int C = 64;              // tokens of a chunk

// ------------------------------------------------------------ the workspace
// Unit u = (b * H + h) * nc + c.  Matrices are stored as MFMA operand
// fragments, lane after lane, so that a copy into LDS and a 16-byte read of
// it is conflict-free.  bf16 path: a fragment is one 16-row tile of the rows
// by two 16-wide K blocks (elements 0..3 of a lane: K = 4q..4q+3 of the first,
// 4..7 of the second), as a high and a low half of 1 KB each where the value
// is split.  fp32 path: one 16-row tile by one K block, 1 KB.
// Rows t with K blocks j <= t ("lower", T and Att): fragment (m, s) of row
// tile m and block pair s; rows j with K blocks t >= j ("upper", the transposes):
// fragment (n, s).  Each has 6 fragments (bf16) or 10 tiles (fp32).
__host__ __device__ constexpr int lower_frag(int m, int s) { return m < 2 ? m : 2 + 2 * (m - 2) + s; }
__host__ __device__ constexpr int upper_frag(int n, int s) { return n < 2 ? 2 * n + s : 2 + n; }
__host__ __device__ constexpr int tile_id(int m, int n) { return m * (m + 1) / 2 + n; }   // n <= m

template <bool F32>
struct Bytes {
    static constexpr int split = F32 ? 10 * 1024 : 12 * 1024;   // T, its transpose, the backward's Att
    static constexpr int att = F32 ? 10 * 1024 : 6 * 1024;      // the forward's Att (one bf16 rounding)
};
// per-token scalars of a unit: four arrays of C
enum { kKin = 0, kKout = 1, kQin = 2, kBeta = 3, kScal = 4 };

// ------------------------------------------------------------ sums over the four 16-lane rows
__device__ __forceinline__ float rows_sum(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// ------------------------------------------------------------ operands
union Frag {                       // 8 bf16 of a lane
    uint4 u;
    bf16x8 v;
    uint32_t w[4];
};
__device__ __forceinline__ f32x4 mma(f32x4 acc, const Frag& a, const Frag& b) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, acc, 0, 0, 0);
}
struct Pair { Frag hi, lo; };      // a split operand: value = hi + lo
// two accumulator tiles as the halves of one fragment
__device__ __forceinline__ Frag round2(const f32x4& a, const f32x4& b) {
    Frag f;
    f.w[0] = pack_bf16x2(a[0], a[1]);
    f.w[1] = pack_bf16x2(a[2], a[3]);
    f.w[2] = pack_bf16x2(b[0], b[1]);
    f.w[3] = pack_bf16x2(b[2], b[3]);
    return f;
}
__device__ __forceinline__ Pair split2(const f32x4& a, const f32x4& b) {
    Pair p;
    split_pair(a[0], a[1], p.hi.w[0], p.lo.w[0]);
    split_pair(a[2], a[3], p.hi.w[1], p.lo.w[1]);
    split_pair(b[0], b[1], p.hi.w[2], p.lo.w[2]);
    split_pair(b[2], b[3], p.hi.w[3], p.lo.w[3]);
    return p;
}
__device__ __forceinline__ float4 f4(const f32x4& a) { return make_float4(a[0], a[1], a[2], a[3]); }
__device__ __forceinline__ f32x4 v4(const float4& a) { return f32x4{a.x, a.y, a.z, a.w}; }
constexpr f32x4 kZero4 = {0.0f, 0.0f, 0.0f, 0.0f};

// the real tokens of batch row b
__device__ __forceinline__ int row_len(const DeltaArgs& a, int b) {
    return a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
}

}  // namespace delta
}  // namespace ssd
