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

// The bf16 forward's T is packed: of the two fragments whose second block lies
// above the diagonal only the first halves are kept, 8 bytes a lane.
template <bool F32>
struct Bytes {
    static constexpr int split = F32 ? 10 * 1024 : 12 * 1024;   // T, its transpose, the backward's Att
    static constexpr int packed = 10 * 1024;                    // the bf16 forward's T
    static constexpr int att = F32 ? 10 * 1024 : 6 * 1024;      // the forward's Att (one bf16 rounding)
};
__host__ __device__ constexpr bool packed_half(int m, int s) { return m == 2 * s; }
// where fragment (m, s)'s high part starts, in KB; its low part follows
__host__ __device__ constexpr int packed_at(int m, int s) { return m == 0 ? 0 : m == 1 ? 1 : m == 2 ? 3 + 2 * s : 6 + 2 * s; }
// a fragment from its packed place, the second half 0 where it is not kept
__device__ __forceinline__ uint4 packed_read(const unsigned char* at, bool half, int lane) {
    if (!half) return *reinterpret_cast<const uint4*>(at + lane * 16);
    const uint2 v = *reinterpret_cast<const uint2*>(at + lane * 8);
    return make_uint4(v.x, v.y, 0, 0);
}
__device__ __forceinline__ void packed_write(unsigned char* at, bool half, int lane, const uint4& v) {
    if (half) *reinterpret_cast<uint2*>(at + lane * 8) = make_uint2(v.x, v.y);
    else *reinterpret_cast<uint4*>(at + lane * 16) = v;
}
// per-token scalars of a unit: four arrays of C
enum { kKin = 0, kKout = 1, kQin = 2, kBeta = 3, kScal = 4 };
// the backward's: also the running sum of dt A (log2) as two floats, the document's number within the chunk, and the
// norms' factors of k and of q times the output's scale
enum { kSGhi = 4, kSGlo = 5, kSSeg = 6, kSRk = 7, kSRq = 8, kScalBwd = 9 };
struct PrepOut {
    unsigned char *T, *TT, *att;   // per unit: T, its transpose, Att or Att T
    float* scal;                   // [u][kScal][C]
    float* across;                 // [u]
};


// A 64 x N bf16 matrix in LDS, rows unpadded: the 16-byte piece of row t that
// holds entries 8 x .. 8 x + 7.  Both kinds of read hit every bank once: by
// rows (16 consecutive rows, one x) and transposed (rows 4 q .. 4 q + 3, four
// consecutive x).
template <int N>
__device__ __forceinline__ int row_piece(int t, int x) {
    return x ^ (N == 128 ? (t & 3) << 2 | (t >> 2 & 3) : N == 64 ? (t >> 1 & 1) << 2 | (t >> 2 & 3) : t >> 2 & 3);
}

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

// ------------------------------------------------------------ operands read by rows, K contiguous: 32 of K a fragment
// 8 consecutive entries of a row of the inputs; lane (q, i) holds row i, entries 8 q .. 8 q + 7
template <typename T>
struct Rows;
template <>
struct Rows<uint16_t> {
    Frag f;
    __device__ __forceinline__ void load(const uint16_t* p) { f.u = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void clear() { f.u = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ float sq() const {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = bf16_lo(f.w[i]), hi = bf16_hi(f.w[i]);
            s = fmaf(lo, lo, fmaf(hi, hi, s));
        }
        return s;
    }
    static __device__ __forceinline__ f32x4 mul(f32x4 acc, const Rows& a, const Rows& b) { return mma(acc, a.f, b.f); }
};
template <>
struct Rows<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0, 0, 0, 0); }
    __device__ __forceinline__ float sq() const {
        return a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w + b.x * b.x + b.y * b.y + b.z * b.z + b.w * b.w;
    }
    static __device__ __forceinline__ f32x4 mul(f32x4 acc, const Rows& x, const Rows& y) {
        return mma_f32(mma_f32(acc, x.a, y.a), x.b, y.b);
    }
};

// 8 consecutive entries of a row of fp32 intermediates: two 16-byte words a lane either way
template <typename T>
struct Wide;
template <>
struct Wide<uint16_t> {
    Pair p;
    __device__ __forceinline__ void set(const float4& a, const float4& b) { p = split2(v4(a), v4(b)); }
    __device__ __forceinline__ void put(unsigned char* at) const {
        *reinterpret_cast<uint4*>(at) = p.hi.u;
        *reinterpret_cast<uint4*>(at + 1024) = p.lo.u;
    }
    __device__ __forceinline__ void get(const unsigned char* at) {
        p.hi.u = *reinterpret_cast<const uint4*>(at);
        p.lo.u = *reinterpret_cast<const uint4*>(at + 1024);
    }
    // wide x input, wide x wide
    static __device__ __forceinline__ f32x4 mul(f32x4 acc, const Wide& a, const Rows<uint16_t>& b) {
        return mma(mma(acc, a.p.lo, b.f), a.p.hi, b.f);
    }
    static __device__ __forceinline__ f32x4 mul(f32x4 acc, const Wide& a, const Wide& b) {
        return mma(mma(mma(acc, a.p.lo, b.p.hi), a.p.hi, b.p.lo), a.p.hi, b.p.hi);
    }
};
template <>
struct Wide<float> {
    Rows<float> p;
    __device__ __forceinline__ void set(const float4& a, const float4& b) { p.a = a; p.b = b; }
    __device__ __forceinline__ void put(unsigned char* at) const {
        *reinterpret_cast<float4*>(at) = p.a;
        *reinterpret_cast<float4*>(at + 1024) = p.b;
    }
    __device__ __forceinline__ void get(const unsigned char* at) {
        p.a = *reinterpret_cast<const float4*>(at);
        p.b = *reinterpret_cast<const float4*>(at + 1024);
    }
    static __device__ __forceinline__ f32x4 mul(f32x4 acc, const Wide& a, const Rows<float>& b) { return Rows<float>::mul(acc, a.p, b); }
    static __device__ __forceinline__ f32x4 mul(f32x4 acc, const Wide& a, const Wide& b) { return Rows<float>::mul(acc, a.p, b.p); }
};

// the real tokens of batch row b
__device__ __forceinline__ int row_len(const DeltaArgs& a, int b) {
    return a.lengths ? min(max(a.lengths[b], 0), a.L) : a.L;
}

// a long sequence's superchunks: K of S chunks (K = 1: none), and [b h][K] states from zero and entering, transitions
struct Split {
    int K, S;
    float *loc, *phi, *s0;
};
struct KeepOut {
    float *S, *U;                  // the states entering the chunks [u][N][P], U [u][C][P]
    Split split;
};

// the backward's first launches (delta.hip): every chunk's T, T^T, Att and scalars, then the states and U
hipError_t launch_keep(const DeltaArgs& a, const PrepOut& o, const KeepOut& k, hipStream_t stream);
// the gradients of the states leaving the superchunks (to s0), from those that they have of their own (loc)
hipError_t launch_join_back(const DeltaArgs& a, const Split& s, const float* g_final, hipStream_t stream);
void split_bwd(int B, int L, int H, int P, int N, int dtype, Split& s);

}  // namespace delta
}  // namespace ssd
