// delta.hip -- the gated delta rule over a sequence: what of a chunk does not
// depend on the state (ssd_delta_prep_kernel, all chunks at once), then the
// chunks in turn (ssd_delta_scan_kernel).
#include <hip/hip_runtime.h>
#include <algorithm>
#include <type_traits>

#include "delta_device.hpp"

namespace ssd {
namespace {

using namespace delta;

// ============================================================ prep
// One wave a unit; four heads of a chunk, which mostly share q and k, in a
// workgroup, without a barrier between them.  A row of k is an operand of
// k k^T from either side, so the chunk's k is loaded once, straight into
// fragments (a lane takes 8 consecutive entries of a row: 64-byte pieces of
// memory; which K index an element stands for does not matter while both
// operands agree).
//
// The inverse is taken of I + L^T, whose accumulator tiles [j][t] are T's
// operand fragments as they come: the four diagonal 16 x 16 blocks by back
// substitution, one block to each 16 lanes, a column to a lane, then the
// blocks above them, T_ac^T = -T_cc^T sum_b L_bc^T T_ab^T, on the fp32 MFMA
// (16 products of 16 x 16 x 16).  Substitution, unlike the product form
// (I - L)(I + L^2)..., never forms a power of L, whose entries can reach 1e8
// where keys point the same way and would cancel.
//
// The running sum of dt A is taken in fp64 and kept as two floats: decays
// within a chunk are differences of sums that can reach -12800 (a token's
// dt A is taken as at least -200: e^-200 is 0 in fp32 either way).
constexpr int kLtStride = C + 4;

struct PrepOut {
    unsigned char *T, *TT, *att;   // per unit: T, its transpose (backward), Att (forward: lower; backward: upper, split)
    float* scal;                   // [u][kScal][C]
    float* across;                 // [u]
};

template <typename T>
struct Rows;                       // 8 consecutive entries of a row
template <>
struct Rows<uint16_t> {
    Frag f;
    __device__ __forceinline__ void load(const uint16_t* p, bool on) {
        f.u = on ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
    }
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
    __device__ __forceinline__ void load(const float* p, bool on) {
        a = b = make_float4(0, 0, 0, 0);
        if (on) {
            a = *reinterpret_cast<const float4*>(p);
            b = *reinterpret_cast<const float4*>(p + 4);
        }
    }
    __device__ __forceinline__ float sq() const {
        return a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w + b.x * b.x + b.y * b.y + b.z * b.z + b.w * b.w;
    }
    static __device__ __forceinline__ f32x4 mul(f32x4 acc, const Rows& x, const Rows& y) {
        return mma_f32(mma_f32(acc, x.a, y.a), x.b, y.b);
    }
};

__device__ __forceinline__ double shfl_up_f64(double v, int d) {
    const long long b = __double_as_longlong(v);
    const int lo = __shfl_up((int)b, d), hi = __shfl_up((int)(b >> 32), d);
    return __longlong_as_double(((long long)hi << 32) | (unsigned)lo);
}

template <typename T, int N, bool BWD>
__global__ __launch_bounds__(256) void ssd_delta_prep_kernel(DeltaArgs a, PrepOut o, int nc) {
    constexpr bool F32 = std::is_same<T, float>::value;
    constexpr int KS = N / 32;
    __shared__ float lt_s[4][C][kLtStride];
    __shared__ float tok_s[4][6][C];
    enum { kGhi, kGlo, kSeg, kB, kRk, kRq };

    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, q = lane / 16, i = lane % 16;
    const int64_t id = (int64_t)blockIdx.x * 4 + wave;
    if (id >= (int64_t)a.B * nc * a.H) return;
    const int h = (int)(id % a.H), c = (int)(id / a.H % nc), b = (int)(id / a.H / nc);
    const int t0 = c * C, n_on = min(C, row_len(a, b) - t0);
    if (n_on <= 0) return;
    const size_t u = ((size_t)b * a.H + h) * nc + c;
    const int g = h / (a.H / a.G);
    float(*lt)[kLtStride] = lt_s[wave];
    float(*tok)[C] = tok_s[wave];

    // ---- k's rows as fragments, and their norms
    const T* kp = static_cast<const T*>(a.k) + ((size_t)b * a.L + t0) * a.k_stride + (size_t)g * N + 8 * q;
    const T* qp = static_cast<const T*>(a.q) + ((size_t)b * a.L + t0) * a.q_stride + (size_t)g * N + 8 * q;
    Rows<T> kf[4][KS];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int t = 16 * m + i;
#pragma unroll
        for (int s = 0; s < KS; ++s) kf[m][s].load(kp + (size_t)t * a.k_stride + 32 * s, t < n_on);
    }

    // ---- the token's scalars, one token a lane
    const bool on = lane < n_on;
    const size_t row = (size_t)b * a.L + t0 + (on ? lane : 0);
    float dt = a.dt[row * a.dt_stride + h], beta = a.beta[row * a.beta_stride + h];
    bool start = false;
    if (a.doc && on && t0 + lane > 0) start = a.doc[row] != a.doc[row - 1];
    if (a.dt_softplus) dt = softplus_f(dt + (a.dt_bias ? a.dt_bias[h] : 0.0f));
    if (a.beta_sigmoid) beta = 1.0f / (1.0f + expf(-beta));
    double G = (double)dt * (double)a.A[h];
    G = G < -200.0 ? -200.0 : G;
    if (!on) { G = 0.0; beta = 0.0f; }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const double up = shfl_up_f64(G, d);
        if (lane >= d) G += up;
    }
    G *= 1.4426950408889634074;                      // log2 e
    const uint64_t starts = __ballot(start);
    const int seg = __popcll(starts & (~0ull >> (63 - lane))), last = __popcll(starts);
    const double Gc = __longlong_as_double(((long long)__builtin_amdgcn_readlane((int)(__double_as_longlong(G) >> 32), 63) << 32) |
                                           (unsigned)__builtin_amdgcn_readlane((int)__double_as_longlong(G), 63));
    const float into = seg == 0 ? fast_exp2((float)G) : 0.0f;
    const float out = seg == last ? fast_exp2((float)(Gc - G)) : 0.0f;
    const float ghi = (float)G;
    tok[kGhi][lane] = ghi;
    tok[kGlo][lane] = (float)(G - (double)ghi);
    tok[kSeg][lane] = (float)seg;
    tok[kB][lane] = beta;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) s += kf[m][k].sq();
        s = rows_sum(s);
        if (q == 0) tok[kRk][16 * m + i] = a.qk_norm ? 1.0f / sqrtf(s + kQkEps) : 1.0f;
    }
    lds_wait();

    // ---- L^T, tile by tile, into LDS; column quantities of t = 16 m + i
    float chi[4], clo[4], cseg[4], cb[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        chi[m] = tok[kGhi][16 * m + i];
        clo[m] = tok[kGlo][16 * m + i];
        cseg[m] = tok[kSeg][16 * m + i];
        cb[m] = tok[kB][16 * m + i] * tok[kRk][16 * m + i];
    }
    // decay from j = 16 n + 4 q + r to t = 16 m + i, 0 where it does not apply
    auto decay = [&](int n, int m, int r, float4 jh, float4 jl, float4 js, bool diag) {
        const float h4[4] = {jh.x, jh.y, jh.z, jh.w}, l4[4] = {jl.x, jl.y, jl.z, jl.w}, s4[4] = {js.x, js.y, js.z, js.w};
        const bool use = s4[r] == cseg[m] && (n < m || (diag ? 4 * q + r <= i : 4 * q + r < i));
        return use ? fast_exp2((chi[m] - h4[r]) + (clo[m] - l4[r])) : 0.0f;
    };
    auto row4 = [&](int what, int n) { return *reinterpret_cast<const float4*>(&tok[what][16 * n + 4 * q]); };
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const float4 jh = row4(kGhi, n), jl = row4(kGlo, n), js = row4(kSeg, n), jr = row4(kRk, n);
        const float r4[4] = {jr.x, jr.y, jr.z, jr.w};
#pragma unroll
        for (int m = n; m < 4; ++m) {
            f32x4 acc = kZero4;
#pragma unroll
            for (int s = 0; s < KS; ++s) acc = Rows<T>::mul(acc, kf[n][s], kf[m][s]);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                lt[16 * n + 4 * q + r][16 * m + i] = acc[r] * (cb[m] * r4[r]) * decay(n, m, r, jh, jl, js, false);
        }
    }

    // ---- Att: a row tile of q at a time
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        Rows<T> qf[KS];
        const int t = 16 * m + i;
        float s2 = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            qf[s].load(qp + (size_t)t * a.q_stride + 32 * s, t < n_on);
            s2 += qf[s].sq();
        }
        s2 = rows_sum(s2);
        const float rq = (a.qk_norm ? 1.0f / sqrtf(s2 + kQkEps) : 1.0f) * a.scale;   // of column t
        if (q == 0) tok[kRq][t] = rq;
        if constexpr (!BWD) {
            f32x4 at[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                at[n] = kZero4;
                if (n > m) continue;
                f32x4 acc = kZero4;
#pragma unroll
                for (int s = 0; s < KS; ++s) acc = Rows<T>::mul(acc, kf[n][s], qf[s]);
                const float4 jh = row4(kGhi, n), jl = row4(kGlo, n), js = row4(kSeg, n), jr = row4(kRk, n);
                const float r4[4] = {jr.x, jr.y, jr.z, jr.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) at[n][r] = acc[r] * (rq * r4[r]) * decay(n, m, r, jh, jl, js, true);
            }
            unsigned char* dst = o.att + u * Bytes<F32>::att + lane * 16;
            if constexpr (F32) {
#pragma unroll
                for (int n = 0; n <= m; ++n) *reinterpret_cast<float4*>(dst + tile_id(m, n) * 1024) = f4(at[n]);
            } else {
#pragma unroll
                for (int s = 0; s < m / 2 + 1; ++s)
                    *reinterpret_cast<uint4*>(dst + lower_frag(m, s) * 1024) = round2(at[2 * s], at[2 * s + 1]).u;
            }
        } else {
            // rows t = 16 m + 4 q + r, column j = 16 n + i: the transposed product's operand
            lds_wait();
            const float4 th = row4(kGhi, m), tl = row4(kGlo, m), ts = row4(kSeg, m), tr = row4(kRq, m);
            const float h4[4] = {th.x, th.y, th.z, th.w}, l4[4] = {tl.x, tl.y, tl.z, tl.w};
            const float s4[4] = {ts.x, ts.y, ts.z, ts.w}, r4[4] = {tr.x, tr.y, tr.z, tr.w};
            unsigned char* dst = o.att + u * Bytes<F32>::split + lane * 16;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                f32x4 acc = kZero4;
                if (n <= m) {
#pragma unroll
                    for (int s = 0; s < KS; ++s) acc = Rows<T>::mul(acc, qf[s], kf[n][s]);
                    const float rk = tok[kRk][16 * n + i];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const bool use = s4[r] == cseg[n] && (n < m || i <= 4 * q + r);
                        acc[r] = use ? acc[r] * (rk * r4[r]) * fast_exp2((h4[r] - chi[n]) + (l4[r] - clo[n])) : 0.0f;
                    }
                }
                if constexpr (F32) {
                    if (n <= m) *reinterpret_cast<float4*>(dst + tile_id(m, n) * 1024) = f4(acc);
                } else if (m / 2 >= n / 2) {
                    // half (m & 1) of fragment (n, m / 2)
                    Pair p = split2(acc, kZero4);
                    unsigned char* at = dst + upper_frag(n, m / 2) * 2048 + (m & 1) * 8;
                    *reinterpret_cast<uint2*>(at) = make_uint2(p.hi.w[0], p.hi.w[1]);
                    *reinterpret_cast<uint2*>(at + 1024) = make_uint2(p.lo.w[0], p.lo.w[1]);
                }
            }
        }
    }
    lds_wait();
    {
        float* sc = o.scal + u * kScal * C;
        const float rk = tok[kRk][lane];
        sc[kKin * C + lane] = into * rk;
        sc[kKout * C + lane] = out * rk;
        sc[kQin * C + lane] = into * tok[kRq][lane];
        sc[kBeta * C + lane] = beta;
        if (lane == 0) o.across[u] = last == 0 ? fast_exp2((float)Gc) : 0.0f;
    }

    // ---- the inverse: lane group q takes diagonal block q, lane i its column i
    {
        float x[16];
#pragma unroll
        for (int r = 15; r >= 0; --r) {
            float v = r == i ? 1.0f : 0.0f;
#pragma unroll
            for (int s4 = (r + 1) / 4; s4 < 4; ++s4) {
                const float4 l = *reinterpret_cast<const float4*>(&lt[16 * q + r][16 * q + 4 * s4]);
                if (4 * s4 + 0 > r) v = fmaf(-l.x, x[4 * s4 + 0], v);
                if (4 * s4 + 1 > r) v = fmaf(-l.y, x[4 * s4 + 1], v);
                if (4 * s4 + 2 > r) v = fmaf(-l.z, x[4 * s4 + 2], v);
                if (4 * s4 + 3 > r) v = fmaf(-l.w, x[4 * s4 + 3], v);
            }
            x[r] = v;
        }
        lds_wait();
#pragma unroll
        for (int r = 0; r < 16; ++r) lt[16 * q + r][16 * q + i] = x[r];
    }
    lds_wait();
    f32x4 tt[4][4];                                  // [c][a]: rows j of block c, columns t of block a
    auto lt4 = [&](int rb, int cb) { return *reinterpret_cast<const float4*>(&lt[16 * rb + i][16 * cb + 4 * q]); };
#pragma unroll
    for (int m = 0; m < 4; ++m) {
#pragma unroll
        for (int n = 0; n < 4; ++n) tt[n][m] = kZero4;
#pragma unroll
        for (int r = 0; r < 4; ++r) tt[m][m][r] = lt[16 * m + 4 * q + r][16 * m + i];
#pragma unroll
        for (int n = m - 1; n >= 0; --n) {
            f32x4 y = kZero4;
#pragma unroll
            for (int k = n + 1; k <= m; ++k) y = mma_f32(y, lt4(n, k), f4(tt[k][m]));
            tt[n][m] = -mma_f32(kZero4, lt4(n, n), f4(y));
        }
    }
    unsigned char* dst = o.T + u * Bytes<F32>::split + lane * 16;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if constexpr (F32) {
#pragma unroll
            for (int n = 0; n <= m; ++n) *reinterpret_cast<float4*>(dst + tile_id(m, n) * 1024) = f4(tt[n][m]);
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                    if (s > m / 2) continue;
                const Pair p = split2(tt[2 * s][m], tt[2 * s + 1][m]);
                *reinterpret_cast<uint4*>(dst + lower_frag(m, s) * 2048) = p.hi.u;
                *reinterpret_cast<uint4*>(dst + lower_frag(m, s) * 2048 + 1024) = p.lo.u;
            }
        }
    }
    if constexpr (BWD) {
        lds_wait();
#pragma unroll
        for (int m = 1; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < m; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) lt[16 * n + 4 * q + r][16 * m + i] = tt[n][m][r];
        lds_wait();
        unsigned char* dtt = o.TT + u * Bytes<F32>::split + lane * 16;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if constexpr (F32) {
#pragma unroll
                for (int m = n; m < 4; ++m) *reinterpret_cast<float4*>(dtt + tile_id(m, n) * 1024) = lt4(n, m);
            } else {
#pragma unroll
                for (int s = n / 2; s < 2; ++s) {
                    const Pair p = split2(2 * s >= n ? v4(lt4(n, 2 * s)) : kZero4, v4(lt4(n, 2 * s + 1)));
                    *reinterpret_cast<uint4*>(dtt + upper_frag(n, s) * 2048) = p.hi.u;
                    *reinterpret_cast<uint4*>(dtt + upper_frag(n, s) * 2048 + 1024) = p.lo.u;
                }
            }
        }
    }
}

// ============================================================ scan
// One workgroup of four waves holds 64 of a head's P columns, a wave 16 of
// them: its part of the state, N x 16, stays in accumulator tiles from the
// first chunk to the last, and since an accumulator tile is an operand
// fragment as it stands, the chain K S -> X -> T X -> U -> K^T U -> S never
// leaves the wave's registers.  What the waves share are the chunk's left
// operands, staged in LDS: k (read by rows for K S and, transposed, for
// K^T U), q, T, Att and v.  The next chunk's loads are in flight meanwhile.
// Splits (bf16): S, X and U scaled are hi + lo pairs, T too: K S and K^T U
// take two MFMAs a tile, T X three.  Y is rounded to bf16 in the end, so its
// products take S and U rounded once (relative 2^-9 each before the output's
// own 2^-9).
struct ScanIo {
    const unsigned char *T, *att;
    const float *scal, *across;
    int nc;
};

template <typename T, int N>
struct ScanLds {
    static constexpr bool F32 = std::is_same<T, float>::value;
    static constexpr int es = sizeof(T);
    static constexpr int kRow = N * es + 16;         // bytes of a k or q row: the odd 16 spreads rows over the banks
    static constexpr int vRow = 64 * es + 16;
    static constexpr int k = 0, q = k + C * kRow, v = q + C * kRow, t = v + C * vRow;
    static constexpr int att = t + Bytes<F32>::split, scal = att + Bytes<F32>::att;
    static constexpr int bytes = scal + kScal * C * 4;
};

template <typename T, int N>
__global__ __launch_bounds__(256) void ssd_delta_scan_kernel(DeltaArgs a, ScanIo io) {
    using LD = ScanLds<T, N>;
    constexpr bool F32 = LD::F32;
    constexpr int NT = N / 16, es = LD::es, nc16 = N * es / 16, nv16 = 64 * es / 16;
    extern __shared__ __align__(16) unsigned char lds[];
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64, q = lane / 16, i = lane % 16;
    const int pb = a.P / 64;
    // heads of a group, which read the same q and k, on one XCD (workgroups go round the eight of them)
    int unit = blockIdx.x;
    const int share = a.H / a.G * pb;
    if (a.B * a.G % 8 == 0) unit = (unit / 8 / share * 8 + unit % 8) * share + unit / 8 % share;
    const int p0 = unit % pb * 64, bh = unit / pb, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    const int len = row_len(a, b), nch = (len + C - 1) / C;
    const size_t tok0 = (size_t)b * a.L;

    // the state: tile n of lane (q, i) holds rows state_n(n) .. +3 of column p
    const int p = p0 + 16 * wave + i;
    auto state_n = [&](int n) { return F32 ? 16 * n + 4 * q : 32 * (n / 2) + 8 * q + 4 * (n % 2); };
    const size_t sofs = ((size_t)bh * a.P + p) * N;
    f32x4 S[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        S[n] = a.init_state ? v4(*reinterpret_cast<const float4*>(a.init_state + sofs + state_n(n))) : kZero4;

    // ---- staging: 16-byte pieces, the next chunk's in registers
    constexpr int NK = (C * nc16 + 255) / 256, NVp = (C * nv16 + 255) / 256;
    constexpr int NTp = (Bytes<F32>::split / 16 + 255) / 256, NA = (Bytes<F32>::att / 16 + 255) / 256;
    u32x4_t rk[NK], rq[NK], rv[NVp], rt[NTp], ra[NA];
    float rs = 0.0f, r_across = 0.0f;
    const unsigned char* kb = static_cast<const unsigned char*>(a.k) + (size_t)g * N * es;
    const unsigned char* qb = static_cast<const unsigned char*>(a.q) + (size_t)g * N * es;
    const unsigned char* vb = static_cast<const unsigned char*>(a.v) + ((size_t)h * a.P + p0) * es;
    auto fetch = [&](int c) {
        const size_t u = (size_t)bh * io.nc + c;
        const int t0 = c * C;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int e = tid + 256 * j, t = e / nc16, x = e % nc16;
            const bool on = t0 + t < len;
            const size_t row = tok0 + (on ? t0 + t : 0);
            rk[j] = on ? *reinterpret_cast<const u32x4_t*>(kb + row * a.k_stride * es + x * 16) : u32x4_t{0, 0, 0, 0};
            rq[j] = on ? *reinterpret_cast<const u32x4_t*>(qb + row * a.q_stride * es + x * 16) : u32x4_t{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < NVp; ++j) {
            const int e = tid + 256 * j, t = e / nv16, x = e % nv16;
            const bool on = t0 + t < len;
            const size_t row = tok0 + (on ? t0 + t : 0);
            rv[j] = on ? *reinterpret_cast<const u32x4_t*>(vb + row * a.v_stride * es + x * 16) : u32x4_t{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < NTp; ++j) {
            const int e = min(tid + 256 * j, Bytes<F32>::split / 16 - 1);
            rt[j] = *reinterpret_cast<const u32x4_t*>(io.T + u * Bytes<F32>::split + e * 16);
        }
#pragma unroll
        for (int j = 0; j < NA; ++j) {
            const int e = min(tid + 256 * j, Bytes<F32>::att / 16 - 1);
            ra[j] = *reinterpret_cast<const u32x4_t*>(io.att + u * Bytes<F32>::att + e * 16);
        }
        rs = io.scal[u * kScal * C + tid];
        r_across = io.across[u];
    };
    auto stage = [&]() {
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int e = tid + 256 * j, t = e / nc16, x = e % nc16;
            if (e < C * nc16) {
                *reinterpret_cast<u32x4_t*>(lds + LD::k + t * LD::kRow + x * 16) = rk[j];
                *reinterpret_cast<u32x4_t*>(lds + LD::q + t * LD::kRow + x * 16) = rq[j];
            }
        }
#pragma unroll
        for (int j = 0; j < NVp; ++j) {
            const int e = tid + 256 * j, t = e / nv16, x = e % nv16;
            *reinterpret_cast<u32x4_t*>(lds + LD::v + t * LD::vRow + x * 16) = rv[j];
        }
#pragma unroll
        for (int j = 0; j < NTp; ++j)
            if (tid + 256 * j < Bytes<F32>::split / 16) *reinterpret_cast<u32x4_t*>(lds + LD::t + (tid + 256 * j) * 16) = rt[j];
#pragma unroll
        for (int j = 0; j < NA; ++j)
            if (tid + 256 * j < Bytes<F32>::att / 16) *reinterpret_cast<u32x4_t*>(lds + LD::att + (tid + 256 * j) * 16) = ra[j];
        *reinterpret_cast<float*>(lds + LD::scal + tid * 4) = rs;
    };
    auto scal4 = [&](int what, int m) {
        return *reinterpret_cast<const float4*>(lds + LD::scal + (what * C + 16 * m + 4 * q) * 4);
    };
    auto frag16 = [&](int ofs) { return *reinterpret_cast<const uint4*>(lds + ofs + lane * 16); };

    T* yp = static_cast<T*>(a.y) + tok0 * a.y_stride + (size_t)h * a.P + p0 + 16 * wave + 4 * q;
    if (nch > 0) fetch(0);
    for (int c = 0; c < nch; ++c) {
        __syncthreads();                             // the last chunk's operands have been read
        stage();
        const float across = r_across;
        __syncthreads();
        if (c + 1 < nch) fetch(c + 1);

        f32x4 U[4];
        if constexpr (!F32) {
            Pair sp[NT / 2];
#pragma unroll
            for (int s = 0; s < NT / 2; ++s) sp[s] = split2(S[2 * s], S[2 * s + 1]);
            f32x4 X[4], O[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f32x4 R = kZero4;
                O[m] = kZero4;
#pragma unroll
                for (int s = 0; s < NT / 2; ++s) {
                    Frag kf, qf;
                    kf.u = *reinterpret_cast<const uint4*>(lds + LD::k + (16 * m + i) * LD::kRow + 64 * s + 16 * q);
                    qf.u = *reinterpret_cast<const uint4*>(lds + LD::q + (16 * m + i) * LD::kRow + 64 * s + 16 * q);
                    R = mma(R, kf, sp[s].lo);
                    R = mma(R, kf, sp[s].hi);
                    O[m] = mma(O[m], sp[s].hi, qf);   // [p][t]
                }
                const FragBF vf = tr_read(lds, LD::v + (16 * m + 4 * q + i / 4) * LD::vRow + (16 * wave + 4 * (i % 4)) * 2);
                const float4 kin = scal4(kKin, m), be = scal4(kBeta, m);
                X[m][0] = be.x * (bf16_lo(vf.a) - kin.x * R[0]);
                X[m][1] = be.y * (bf16_hi(vf.a) - kin.y * R[1]);
                X[m][2] = be.z * (bf16_lo(vf.b) - kin.z * R[2]);
                X[m][3] = be.w * (bf16_hi(vf.b) - kin.w * R[3]);
            }
            const Pair xp[2] = {split2(X[0], X[1]), split2(X[2], X[3])};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                U[m] = kZero4;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (s > m / 2) continue;
                    Frag th, tl;
                    th.u = frag16(LD::t + lower_frag(m, s) * 2048);
                    tl.u = frag16(LD::t + lower_frag(m, s) * 2048 + 1024);
                    U[m] = mma(U[m], tl, xp[s].hi);
                    U[m] = mma(U[m], th, xp[s].lo);
                    U[m] = mma(U[m], th, xp[s].hi);
                }
            }
            const Frag ub[2] = {round2(U[0], U[1]), round2(U[2], U[3])};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int t = c * C + 16 * m + i;
                const float qin = *reinterpret_cast<const float*>(lds + LD::scal + (kQin * C + 16 * m + i) * 4);
                O[m] *= qin;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (s > m / 2) continue;
                    Frag af;
                    af.u = frag16(LD::att + lower_frag(m, s) * 1024);
                    O[m] = mma(O[m], ub[s], af);
                }
                if (t < len)
                    *reinterpret_cast<uint2*>(yp + (size_t)t * a.y_stride) =
                        make_uint2(pack_bf16x2(O[m][0], O[m][1]), pack_bf16x2(O[m][2], O[m][3]));
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) U[m] *= v4(scal4(kKout, m));
            const Pair up[2] = {split2(U[0], U[1]), split2(U[2], U[3])};
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                S[n] *= across;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    // k^T: row n of the tile pair's numbering, K index t
                    Frag kt;
                    const int col = 32 * (n / 2) + 8 * (i % 4) + 4 * (n % 2);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const FragBF f = tr_read(lds, LD::k + (32 * s + 16 * e + 4 * q + i / 4) * LD::kRow + col * 2);
                        kt.w[2 * e] = f.a;
                        kt.w[2 * e + 1] = f.b;
                    }
                    S[n] = mma(S[n], kt, up[s].lo);
                    S[n] = mma(S[n], kt, up[s].hi);
                }
            }
        } else {
            f32x4 X[4], O[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                f32x4 R = kZero4;
                O[m] = kZero4;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float4 kf = *reinterpret_cast<const float4*>(lds + LD::k + (16 * m + i) * LD::kRow + (16 * n + 4 * q) * 4);
                    const float4 qf = *reinterpret_cast<const float4*>(lds + LD::q + (16 * m + i) * LD::kRow + (16 * n + 4 * q) * 4);
                    R = mma_f32(R, kf, f4(S[n]));
                    O[m] = mma_f32(O[m], f4(S[n]), qf);
                }
                const float4 kin = scal4(kKin, m), be = scal4(kBeta, m);
                const float k4[4] = {kin.x, kin.y, kin.z, kin.w}, b4[4] = {be.x, be.y, be.z, be.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float v = *reinterpret_cast<const float*>(lds + LD::v + (16 * m + 4 * q + r) * LD::vRow + (16 * wave + i) * 4);
                    X[m][r] = b4[r] * (v - k4[r] * R[r]);
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                U[m] = kZero4;
#pragma unroll
                for (int n = 0; n <= m; ++n)
                    U[m] = mma_f32(U[m], __builtin_bit_cast(float4, frag16(LD::t + tile_id(m, n) * 1024)), f4(X[n]));
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int t = c * C + 16 * m + i;
                const float qin = *reinterpret_cast<const float*>(lds + LD::scal + (kQin * C + 16 * m + i) * 4);
                O[m] *= qin;
#pragma unroll
                for (int n = 0; n <= m; ++n)
                    O[m] = mma_f32(O[m], f4(U[n]), __builtin_bit_cast(float4, frag16(LD::att + tile_id(m, n) * 1024)));
                if (t < len) *reinterpret_cast<float4*>(yp + (size_t)t * a.y_stride) = f4(O[m]);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) U[m] *= v4(scal4(kKout, m));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                S[n] *= across;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const unsigned char* kc = lds + LD::k + (16 * m + 4 * q) * LD::kRow + (16 * n + i) * 4;
                    float4 kt;
                    kt.x = *reinterpret_cast<const float*>(kc);
                    kt.y = *reinterpret_cast<const float*>(kc + LD::kRow);
                    kt.z = *reinterpret_cast<const float*>(kc + 2 * LD::kRow);
                    kt.w = *reinterpret_cast<const float*>(kc + 3 * LD::kRow);
                    S[n] = mma_f32(S[n], kt, f4(U[m]));
                }
            }
        }
    }
    // rows past the sequence are exactly 0
    for (int t = len + i; t < a.L; t += 16) {
        if constexpr (F32) *reinterpret_cast<float4*>(yp + (size_t)t * a.y_stride) = make_float4(0, 0, 0, 0);
        else *reinterpret_cast<uint2*>(yp + (size_t)t * a.y_stride) = make_uint2(0, 0);
    }
    if (a.final_state) {
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<float4*>(a.final_state + sofs + state_n(n)) = f4(S[n]);
    }
}

struct FwdWs {                     // byte offsets
    size_t T, att, scal, across, total;
};
FwdWs fwd_ws(int B, int L, int H, int dtype) {
    const size_t units = (size_t)B * H * ((L + C - 1) / C);
    FwdWs w;
    w.T = 0;
    w.att = w.T + units * (dtype == 0 ? Bytes<true>::split : Bytes<false>::split);
    w.scal = w.att + units * (dtype == 0 ? Bytes<true>::att : Bytes<false>::att);
    w.across = w.scal + units * kScal * C * 4;
    w.total = w.across + (units * 4 + 255) / 256 * 256;
    return w;
}

template <typename T, int N>
hipError_t launch_fwd_n(const DeltaArgs& a, void* ws, hipStream_t stream) {
    const int nc = (a.L + C - 1) / C;
    const FwdWs w = fwd_ws(a.B, a.L, a.H, a.dtype);
    unsigned char* base = static_cast<unsigned char*>(ws);
    PrepOut o{base + w.T, nullptr, base + w.att, reinterpret_cast<float*>(base + w.scal),
              reinterpret_cast<float*>(base + w.across)};
    const int64_t units = (int64_t)a.B * a.H * nc;
    hipLaunchKernelGGL((ssd_delta_prep_kernel<T, N, false>), dim3((unsigned)((units + 3) / 4)), dim3(256), 0, stream, a,
                       o, nc);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    constexpr size_t lds = ScanLds<T, N>::bytes;
    e = prepare_launch(reinterpret_cast<const void*>(&ssd_delta_scan_kernel<T, N>), lds);
    if (e != hipSuccess) return e;
    ScanIo io{o.T, o.att, o.scal, o.across, nc};
    hipLaunchKernelGGL((ssd_delta_scan_kernel<T, N>), dim3(a.B * a.H * (a.P / 64)), dim3(256), lds, stream, a, io);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_fwd_t(const DeltaArgs& a, void* ws, hipStream_t stream) {
    switch (a.N) {
        case 32: return launch_fwd_n<T, 32>(a, ws, stream);
        case 64: return launch_fwd_n<T, 64>(a, ws, stream);
        case 128: return launch_fwd_n<T, 128>(a, ws, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace

size_t delta_fwd_workspace_bytes(int B, int L, int H, int dtype) { return fwd_ws(B, L, H, dtype).total; }

hipError_t launch_delta_fwd(const DeltaArgs& a, void* ws, hipStream_t stream) {
    return a.dtype == 0 ? launch_fwd_t<float>(a, ws, stream) : launch_fwd_t<uint16_t>(a, ws, stream);
}

}  // namespace ssd
