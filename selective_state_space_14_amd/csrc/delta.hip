// delta.hip -- the gated delta rule over a sequence: what of a chunk does not
// depend on the state (ssd_delta_prep_kernel, all chunks at once), then the
// chunks in turn (ssd_delta_chain_kernel in bf16, ssd_delta_scan_kernel in
// fp32).
#include <hip/hip_runtime.h>
#include <algorithm>
#include <type_traits>

#include "delta_device.hpp"

namespace ssd {
namespace {

using namespace delta;

// ============================================================ prep
// One wave a unit, two to a workgroup, without a barrier between them.  A row
// of k is an operand of k k^T from either side, so the chunk's k is loaded
// once, straight into fragments (a lane takes 8 consecutive entries of a row:
// 64-byte pieces of memory; which K index an element stands for does not
// matter while both operands agree).
//
// The inverse is taken of I + L^T, whose accumulator tiles [j][t] are T's
// operand fragments as they come: the four diagonal 16 x 16 blocks by back
// substitution, one block to each 16 lanes, a column to a lane, then the
// blocks above them, T_ac^T = -T_cc^T sum_b L_bc^T T_ab^T, on the fp32 MFMA
// (16 products of 16 x 16 x 16).  Substitution, unlike the product form
// (I - L)(I + L^2)..., never forms a power of L, whose entries can reach 1e8
// where keys point the same way and would cancel.
//
// The running sum of dt A is taken in fp64: within a chunk decays are
// differences of sums that can reach -12800 (a token's dt A is taken as at
// least -200: e^-200 is 0 in fp32 either way).  Between two 16-token blocks a
// decay is the product of one to the later block's first token and one from
// it, both from a table of 16 exponentials a token; inside a block it is taken
// from the sum held as two floats.
//
// What the scan needs of T depends on it (Prep): the bf16 forward multiplies X
// by T only to get U scaled for the state, diag(e^{G_C - G}) T diag(beta), and
// Att T diag(beta) for y, so those two products are formed here, where all
// chunks run at once, and not in the chain of the scan.  (Forming only Att here
// took 122 us in place of 156 at B=5 L=8192 H=32 N=64, but the scan 242 in
// place of 225, both from an idle GPU's lower clocks.)
//
// Measured, bf16: 144 us at B=5 L=8192 H=32 P=N=64 (20480 units, 17 KB written
// each, 357 MB, and 255 MB read: 120 us at a copy's rate), 262 us at B=4 L=4096
// H=128 N=128 (32768 units; 571 MB written and 681 MB read, since a group's 16
// heads are on all eight XCDs: 245 us at a copy's rate, with the matrix pipes
// busy for 85 us and the vector units for 89).
constexpr int kLtRow = 20;                           // floats of an L^T tile's row: 16-byte reads of 16 rows hit all banks
constexpr int kPrepWaves = 2;
enum Prep {
    kPrepScaled = 0,               // bf16 forward: diag(kout) T diag(beta) (split), Att T diag(beta) (rounded)
    kPrepPlain = 1,                // fp32 forward: T, Att
    kPrepBwd = 2,                  // backward: T, its transpose, Att's transposed product's operand (all split)
};


__device__ __forceinline__ double shfl_up_f64(double v, int d) {
    const long long b = __double_as_longlong(v);
    const int lo = __shfl_up((int)b, d), hi = __shfl_up((int)(b >> 32), d);
    return __longlong_as_double(((long long)hi << 32) | (unsigned)lo);
}

template <typename T, int N, int PM>
__global__ __launch_bounds__(64 * kPrepWaves) void ssd_delta_prep_kernel(DeltaArgs a, PrepOut o, int nc) {
    constexpr bool F32 = std::is_same<T, float>::value;
    constexpr int KS = N / 32;
    __shared__ __align__(16) float lt_s[kPrepWaves][10 * 16 * kLtRow];
    enum { kGhi, kGlo, kSeg, kB, kRk, kRq, kF, kOut, kE, kTok = kE + 3 };
    __shared__ __align__(16) float tok_s[kPrepWaves][kTok][C];

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64, q = lane / 16, i = lane % 16;
    const uint32_t id = blockIdx.x * kPrepWaves + wave;   // below 2^31 (api)
    if (id >= (uint32_t)a.B * nc * a.H) return;
    const int h = (int)(id % a.H), b = (int)(id / a.H % a.B), c = (int)(id / a.H / a.B);
    const int t0 = c * C, n_on = min(C, row_len(a, b) - t0);
    if (n_on <= 0) return;
    const size_t u = ((size_t)b * a.H + h) * nc + c;
    const int g = h / (a.H / a.G);
    float* lt = lt_s[wave];
    float(*tok)[C] = tok_s[wave];
    // tile (n, m), n <= m, of an upper triangular matrix: rows j of block n, columns t of block m
    auto ltp = [&](int n, int m, int r, int col) { return lt + (tile_id(m, n) * 16 + r) * kLtRow + col; };
    auto lt4 = [&](int n, int m) { return *reinterpret_cast<const float4*>(ltp(n, m, i, 4 * q)); };

    // ---- k's rows as fragments
    const T* kp = static_cast<const T*>(a.k) + ((size_t)b * a.L + t0) * a.k_stride + (size_t)g * N + 8 * q;
    const T* qp = static_cast<const T*>(a.q) + ((size_t)b * a.L + t0) * a.q_stride + (size_t)g * N + 8 * q;
    // row t = 16 m + i of a tile; rows past the sequence read its last one and become zeros
    auto load_rows = [&](Rows<T>(&f)[KS], const T* p, int64_t stride, int m) {
        const T* at = p + min(16 * m + i, n_on - 1) * stride;
#pragma unroll
        for (int s = 0; s < KS; ++s) f[s].load(at + 32 * s);
        if (n_on < C && 16 * m + i >= n_on) {
#pragma unroll
            for (int s = 0; s < KS; ++s) f[s].clear();
        }
    };
    Rows<T> kf[4][KS], qf[4][KS];
#pragma unroll
    for (int m = 0; m < 4; ++m) load_rows(kf[m], kp, a.k_stride, m);
#pragma unroll
    for (int m = 0; m < 4; ++m) load_rows(qf[m], qp, a.q_stride, m);

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
    auto of_lane = [&](int l) {
        const long long v = __double_as_longlong(G);
        return __longlong_as_double(((long long)__builtin_amdgcn_readlane((int)(v >> 32), l) << 32) |
                                    (unsigned)__builtin_amdgcn_readlane((int)v, l));
    };
    const uint64_t starts = __ballot(start);
    const int seg = __popcll(starts & (~0ull >> (63 - lane))), last = __popcll(starts);
    const double Gc = of_lane(63);
    const float into = seg == 0 ? fast_exp2((float)G) : 0.0f;
    const float out = seg == last ? fast_exp2((float)(Gc - G)) : 0.0f;
    const float ghi = (float)G;
    tok[kGhi][lane] = ghi;
    tok[kGlo][lane] = (float)(G - (double)ghi);
    tok[kSeg][lane] = (float)seg;
    tok[kB][lane] = beta;
    {
        float f = 0.0f;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const double ref = of_lane(16 * m);
            const int rseg = __popcll(starts & (~0ull >> (63 - 16 * m)));
            if (lane / 16 == m && seg == rseg) f = fast_exp2((float)(G - ref));
            if (m > 0) tok[kE + m - 1][lane] = lane < 16 * m && seg == rseg ? fast_exp2((float)(ref - G)) : 0.0f;
        }
        tok[kF][lane] = f;
    }
    float rq[4];                                     // of column t = 16 m + i, with the output's scale
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        // a row's square is the diagonal of its tile's product with itself: entry r = i % 4 of lane (i / 4, i)
        float rk = 1.0f;
        rq[m] = a.scale;
        if (a.qk_norm) {
            f32x4 kk = kZero4, qq = kZero4;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                kk = Rows<T>::mul(kk, kf[m][s], kf[m][s]);
                qq = Rows<T>::mul(qq, qf[m][s], qf[m][s]);
            }
            const bool odd = i & 1, high = i & 2, mine = q == i / 4;
            const float k1 = high ? (odd ? kk[3] : kk[2]) : (odd ? kk[1] : kk[0]);
            const float q1 = high ? (odd ? qq[3] : qq[2]) : (odd ? qq[1] : qq[0]);
            rk = __builtin_amdgcn_rsqf(rows_sum(mine ? k1 : 0.0f) + kQkEps);
            rq[m] *= __builtin_amdgcn_rsqf(rows_sum(mine ? q1 : 0.0f) + kQkEps);
        }
        if (q == 0) {
            tok[kRk][16 * m + i] = rk;
            tok[kRq][16 * m + i] = rq[m];
        }
    }
    lds_wait();
    auto row4 = [&](int what, int n) { return v4(*reinterpret_cast<const float4*>(&tok[what][16 * n + 4 * q])); };
    auto col1 = [&](int what, int m) { return tok[what][16 * m + i]; };
    // the table's decays with k_j's norm.  The bf16 forward wants T diag(beta) and Att T diag(beta): with beta on the
    // columns of L instead of its rows, T' = (I + L')^-1 has T diag(beta) = diag(beta) T', and Att T diag(beta) =
    // (Att diag(beta)) T', so there beta_j joins the table too
    f32x4 rk4[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        rk4[n] = row4(kRk, n);
        if (PM == kPrepScaled) rk4[n] *= row4(kB, n);
#pragma unroll
        for (int m = n + 1; m < 4; ++m) {
            const f32x4 e = row4(kE + m - 1, n) * rk4[n];
            if (i == 0) *reinterpret_cast<float4*>(&tok[kE + m - 1][16 * n + 4 * q]) = f4(e);
        }
    }
    lds_wait();

    // ---- L^T and Att^T, tile by tile: row j = 16 n + 4 q + r, column t = 16 m + i.  L^T goes to LDS, Att^T stays in
    // registers (the backward's Att, whose transpose is wanted, leaves at once)
    f32x4 at[4][4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float ct = col1(kF, m), cb = PM == kPrepScaled ? col1(kRk, m) : col1(kB, m) * col1(kRk, m);
#pragma unroll
        for (int n = 0; n <= m; ++n) {
            f32x4 l = kZero4, d;
#pragma unroll
            for (int s = 0; s < KS; ++s) l = Rows<T>::mul(l, kf[n][s], kf[m][s]);
            if (n < m) {
                d = row4(kE + m - 1, n) * ct;
            } else {
                const f32x4 h4 = row4(kGhi, n), l4 = row4(kGlo, n), s4 = row4(kSeg, n);
                const float th = col1(kGhi, m), tl = col1(kGlo, m), ts = col1(kSeg, m);
#pragma unroll
                for (int r = 0; r < 4; ++r) d[r] = fast_exp2(s4[r] == ts && 4 * q + r <= i ? (th - h4[r]) + (tl - l4[r]) : -INFINITY);
                d *= rk4[n];
            }
            l *= d * cb;
#pragma unroll
            for (int r = 0; r < 4; ++r) *ltp(n, m, 4 * q + r, i) = n == m && 4 * q + r == i ? 0.0f : l[r];
            if constexpr (PM != kPrepBwd) {
                at[n][m] = kZero4;
#pragma unroll
                for (int s = 0; s < KS; ++s) at[n][m] = Rows<T>::mul(at[n][m], kf[n][s], qf[m][s]);
                at[n][m] *= d * rq[m];
            }
        }
    }
    if constexpr (PM == kPrepBwd) {
        unsigned char* da = o.att + u * Bytes<F32>::split + lane * 16;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            // rows t = 16 m + 4 q + r, column j = 16 n + i
            const f32x4 r4 = row4(kRq, m);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                f32x4 acc = kZero4;
                if (n <= m) {
#pragma unroll
                    for (int s = 0; s < KS; ++s) acc = Rows<T>::mul(acc, qf[m][s], kf[n][s]);
                    if (n < m) {
                        acc *= r4 * row4(kF, m) * col1(kE + m - 1, n);
                    } else {
                        acc *= r4 * col1(kRk, n);
                        const f32x4 h4 = row4(kGhi, m), l4 = row4(kGlo, m), s4 = row4(kSeg, m);
                        const float jh = col1(kGhi, n), jl = col1(kGlo, n), js = col1(kSeg, n);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[r] *= fast_exp2(s4[r] == js && i <= 4 * q + r ? (h4[r] - jh) + (l4[r] - jl) : -INFINITY);
                    }
                }
                if constexpr (F32) {
                    if (n <= m) *reinterpret_cast<float4*>(da + tile_id(m, n) * 1024) = f4(acc);
                } else if (m / 2 >= n / 2) {
                    // half (m & 1) of fragment (n, m / 2)
                    const Pair p = split2(acc, kZero4);
                    unsigned char* to = da + upper_frag(n, m / 2) * 2048 + (m & 1) * 8;
                    *reinterpret_cast<uint2*>(to) = make_uint2(p.hi.w[0], p.hi.w[1]);
                    *reinterpret_cast<uint2*>(to + 1024) = make_uint2(p.lo.w[0], p.lo.w[1]);
                }
            }
        }
    }
    {
        constexpr int NS = PM == kPrepBwd ? kScalBwd : kScal;
        float* sc = o.scal + u * NS * C;
        const float rk = tok[kRk][lane];
        if (PM == kPrepBwd) {
            sc[kSGhi * C + lane] = ghi;
            sc[kSGlo * C + lane] = tok[kGlo][lane];
            sc[kSSeg * C + lane] = (float)seg;
            sc[kSRk * C + lane] = rk;
            sc[kSRq * C + lane] = tok[kRq][lane];
        }
        sc[kKin * C + lane] = into * rk;
        sc[kKout * C + lane] = out * rk;
        sc[kQin * C + lane] = into * tok[kRq][lane];
        sc[kBeta * C + lane] = beta;
        if (PM == kPrepScaled) tok[kOut][lane] = out * rk * beta;
        if (lane == 0) o.across[u] = last == 0 ? fast_exp2((float)Gc) : 0.0f;
    }
    lds_wait();

    // ---- the inverse: lane group q takes diagonal block q, lane i its column i
    {
        float x[16];
        const float* dg = lt + tile_id(q, q) * 16 * kLtRow;
#pragma unroll
        for (int r = 15; r >= 0; --r) {
            float v = r == i ? 1.0f : 0.0f;
#pragma unroll
            for (int s4 = (r + 1) / 4; s4 < 4; ++s4) {
                const float4 l = *reinterpret_cast<const float4*>(dg + r * kLtRow + 4 * s4);
                if (4 * s4 + 0 > r) v = fmaf(-l.x, x[4 * s4 + 0], v);
                if (4 * s4 + 1 > r) v = fmaf(-l.y, x[4 * s4 + 1], v);
                if (4 * s4 + 2 > r) v = fmaf(-l.z, x[4 * s4 + 2], v);
                if (4 * s4 + 3 > r) v = fmaf(-l.w, x[4 * s4 + 3], v);
            }
            x[r] = v;
        }
        lds_wait();
        float* dw = lt + tile_id(q, q) * 16 * kLtRow + i;
#pragma unroll
        for (int r = 0; r < 16; ++r) dw[r * kLtRow] = x[r];
    }
    lds_wait();
    f32x4 tt[4][4];                                  // [c][a]: rows j of block c, columns t of block a
#pragma unroll
    for (int m = 0; m < 4; ++m) {
#pragma unroll
        for (int n = 0; n < 4; ++n) tt[n][m] = kZero4;
#pragma unroll
        for (int r = 0; r < 4; ++r) tt[m][m][r] = *ltp(m, m, 4 * q + r, i);
#pragma unroll
        for (int n = m - 1; n >= 0; --n) {
            f32x4 y = kZero4;
#pragma unroll
            for (int k = n + 1; k <= m; ++k) y = mma_f32(y, lt4(n, k), f4(tt[k][m]));
            tt[n][m] = -mma_f32(kZero4, lt4(n, n), f4(y));
        }
    }
    // T^T back to LDS, over L^T, where its transpose is wanted
    if constexpr (PM != kPrepPlain) {
        lds_wait();
#pragma unroll
        for (int m = 1; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < m; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) *ltp(n, m, 4 * q + r, i) = tt[n][m][r];
    }
    unsigned char* dst = o.T + u * (PM == kPrepScaled ? Bytes<F32>::packed : Bytes<F32>::split) + (PM == kPrepScaled ? 0 : lane * 16);
    lds_wait();
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if constexpr (PM == kPrepScaled) {
            const float ko = col1(kOut, m);
#pragma unroll
            for (int n = 0; n <= m; ++n) tt[n][m] *= ko;
        }
        if constexpr (F32) {
#pragma unroll
            for (int n = 0; n <= m; ++n) *reinterpret_cast<float4*>(dst + tile_id(m, n) * 1024) = f4(tt[n][m]);
        } else {
#pragma unroll
            for (int s = 0; s < m / 2 + 1; ++s) {
                const Pair p = split2(tt[2 * s][m], tt[2 * s + 1][m]);
                if constexpr (PM == kPrepScaled) {
                    unsigned char* at = dst + packed_at(m, s) * 1024;
                    packed_write(at, packed_half(m, s), lane, p.hi.u);
                    packed_write(at + (packed_half(m, s) ? 512 : 1024), packed_half(m, s), lane, p.lo.u);
                } else {
                    *reinterpret_cast<uint4*>(dst + lower_frag(m, s) * 2048) = p.hi.u;
                    *reinterpret_cast<uint4*>(dst + lower_frag(m, s) * 2048 + 1024) = p.lo.u;
                }
            }
        }
    }
    if constexpr (PM == kPrepBwd) {
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

    // ---- Att
    if constexpr (PM != kPrepBwd) {
        unsigned char* da = o.att + u * Bytes<F32>::att + lane * 16;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if constexpr (F32) {
#pragma unroll
                for (int n = 0; n <= m; ++n) *reinterpret_cast<float4*>(da + tile_id(m, n) * 1024) = f4(at[n][m]);
            } else {
                // (Att T)^T, tile (n, m) = sum_k T^T(n, k) Att^T(k, m) over k = n .. m; on the fp32 MFMA, since the
                // VALU, which would split the operands, is what this kernel is short of
                f32x4 w[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    w[n] = kZero4;
                    if (n > m) continue;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k >= n && k <= m) w[n] = mma_f32(w[n], lt4(n, k), f4(at[k][m]));
                }
#pragma unroll
                for (int s = 0; s < m / 2 + 1; ++s)
                    *reinterpret_cast<uint4*>(da + lower_frag(m, s) * 1024) = round2(w[2 * s], w[2 * s + 1]).u;
            }
        }
    }
}

// ============================================================ scan
// One workgroup holds 64 of a head's P columns, a wave 16 of them: its part of
// the state, N x 16, stays in accumulator tiles from the first chunk to the
// last, and since an accumulator tile is an operand fragment as it stands, the
// chain K S -> X -> T X -> K^T U -> S never leaves the wave's registers.  The
// chunks' left operands, which the waves share, are staged in LDS in two
// buffers, the next chunk's while this one is computed.
struct ScanIo {
    const unsigned char *T, *att;
    const float *scal, *across;
    int nc;
    float *keepS, *keepU;          // backward: the state entering each chunk [u][N][P] and U [u][C][P]
    // sequence split: K superchunks of S chunks (K = 1: none).  Of each, the end state from a zero state [b h][K][P][N]
    // and the transition [b h][K][N columns][N] (the forward's last has none); the state entering each [b h][K][P][N].
    int K, S;
    float *loc, *phi, *s0;
};

// ---- bf16 forward
// With one sequence's head to a workgroup there is one chain to a SIMD, and
// its latency a chunk is what bounds the kernel.  So four waves do nothing but
// the chain, and four more everything that is not part of it, on the same
// SIMDs: they bring the next chunk's k, v and T from memory to LDS, and compute
// and store the last chunk's y from the S and X fragments that the chain left
// in LDS.  A chunk costs one barrier.  Measured: 1.7 us a chunk at N = 64 (213
// us at B=5 L=8192 H=32, 160 workgroups; 364 us with all of it in four waves),
// 2.6 us at N = 128 (331 us at B=4 L=4096 H=128, two rounds of 64 chunks).  At
// N = 128 a CU's reads in flight bound it (11 bytes a cycle and CU), at N = 64
// the chain's latency.  The chain's LDS reads are issued ahead
// of the products they feed (sched_barrier: left to itself the compiler reads
// each fragment just before its use).
// Splits: S, X, U and T are hi + lo pairs, k is bf16 as it is: K S and K^T U
// take two MFMAs a tile, T X three; the state's error stays near 2^-18.  Y is
// rounded to bf16 in the end, so its products take S and Att T rounded once,
// 2^-8 each at most, as the output's own rounding, and X as a pair.
//
// Few heads and a long sequence leave most CUs without a chain.  A chunk's
// step is linear in the state, S' = Phi S + (a part from v), so the sequence
// is cut into superchunks: one launch (kState) passes over all but the last
// from a zero state, and with N columns more, which start as the identity and
// see v = 0, computes their transitions; ssd_delta_join_kernel puts the states
// entering the superchunks together; the full launch runs them side by side.
// The backward's recomputation is the same chain (kStates) with T and beta apart, each chunk's entering state and U
// going to memory from the chain's waves, and no y.
enum { kFull = 0, kState = 1, kStates = 2, kStateApart = 3 };   // kStateApart: kState for kStates

template <int N, int MODE>
struct ChainLds {
    static constexpr int kRow = N * 2;               // bytes of a k row, its 16-byte pieces permuted (piece())
    static constexpr int vRow = 64 * 2 + 16;
    static constexpr int KS = N / 32;
    static __device__ __forceinline__ int piece(int t, int x) { return row_piece<N>(t, x); }
    static constexpr bool apart = MODE == kStates || MODE == kStateApart;   // T, beta and kout come by themselves
    static constexpr int k = 0, v = k + C * kRow, t = v + C * vRow;
    static constexpr int t_bytes = apart ? Bytes<false>::split : Bytes<false>::packed;
    // kin (apart: all four arrays of scalars), then the decay across the chunk
    static constexpr int kin = t + t_bytes, across = kin + (apart ? kScal : 1) * C * 4;
    static constexpr int buffer = across + 256;
    static constexpr int kept = (KS + 4) * 1024;     // a wave's S (rounded) and X (split) fragments
    static constexpr int bytes = 2 * (buffer + (MODE == kFull ? 4 * kept : 0));
};

template <int N, int MODE>
__global__ __launch_bounds__(512, 2) void ssd_delta_chain_kernel(DeltaArgs a, ScanIo io) {
    using LD = ChainLds<N, MODE>;
    constexpr int NT = N / 16, KS = N / 32, nc16 = N / 8;
    constexpr bool kApart = LD::apart, kPass = MODE == kState || MODE == kStateApart;
    extern __shared__ __align__(16) unsigned char lds_all[];
    const int tid = threadIdx.x % 256, wave = tid / 64, lane = tid % 64, q = lane / 16, i = lane % 16;
    // blocks of 64 columns of a head: P's, and in the state pass the transition's
    const int pb = a.P / 64 + (kPass ? (N + 63) / 64 : 0);
    const int units = a.B * a.H * pb, sk = blockIdx.x / units;
    // heads of a group, which read the same q and k, on one XCD (workgroups go round the eight of them)
    int unit = blockIdx.x % units;
    const int share = a.H / a.G * pb;
    if (a.B * a.G % 8 == 0) unit = (unit / 8 / share * 8 + unit % 8) * share + unit / 8 % share;
    const int blk = unit % pb, bh = unit / pb, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    const bool phi = kPass && blk >= a.P / 64;
    const int p0 = phi ? 0 : blk * 64;
    const int len = row_len(a, b), c0 = sk * io.S;
    const int nch = max(0, min(io.S, (len + C - 1) / C - c0));   // chunks here, counted from c0 below
    const size_t tok0 = (size_t)b * a.L;
    unsigned char* const kept = lds_all + 2 * LD::buffer + wave * LD::kept + lane * 16;   // + 4 LD::kept a parity

    if (threadIdx.x < 256) {
        // ------------------------------------------------ the chain
        // tile n of lane (q, i) holds the state's rows 32 (n / 2) + 8 q + 4 (n % 2) .. +3 of column p
        const size_t sofs = ((size_t)bh * a.P + p0 + 16 * wave + i) * N + 8 * q;
        const int pc = (blk - a.P / 64) * 64 + 16 * wave + i;   // column of the transition
        f32x4 S[NT];
        const float* first = kPass ? nullptr
                             : io.K > 1     ? io.s0 + ((size_t)bh * io.K + sk) * a.P * N + (sofs - (size_t)bh * a.P * N)
                             : a.init_state ? a.init_state + sofs
                                            : nullptr;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            S[n] = first ? v4(*reinterpret_cast<const float4*>(first + 32 * (n / 2) + 4 * (n % 2))) : kZero4;
            if (phi) {
#pragma unroll
                for (int r = 0; r < 4; ++r) S[n][r] = 32 * (n / 2) + 8 * q + 4 * (n % 2) + r == pc ? 1.0f : 0.0f;
            }
        }
        __builtin_amdgcn_s_setprio(3);               // before the other four waves wherever both can issue
        lds_barrier();
        for (int c = 0; c < nch; ++c) {
            const unsigned char* const lds = lds_all + (c & 1) * LD::buffer;
            unsigned char* const keep = kept + (c & 1) * 4 * LD::kept;
            Frag kf[4][KS], th[6], tl[6], kt[NT][2];
            FragBF vf[4];
            f32x4 kin[4];
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    kf[m][s].u = *reinterpret_cast<const uint4*>(lds + LD::k + (16 * m + i) * LD::kRow + LD::piece(i, 4 * s + q) * 16);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                kin[m] = v4(*reinterpret_cast<const float4*>(lds + LD::kin + (16 * m + 4 * q) * 4));
                vf[m] = tr_read(lds, LD::v + (16 * m + 4 * q + i / 4) * LD::vRow + (16 * wave + 4 * (i % 4)) * 2);
            }
            const float across = *reinterpret_cast<const float*>(lds + LD::across);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (MODE == kStates) {
                float* to = io.keepS + ((size_t)bh * io.nc + c0 + c) * N * a.P + p0 + 16 * wave + i;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r) to[(size_t)(32 * (n / 2) + 8 * q + 4 * (n % 2) + r) * a.P] = S[n][r];
            }
            Pair sp[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                sp[s] = split2(S[2 * s], S[2 * s + 1]);
                if (MODE == kFull) *reinterpret_cast<uint4*>(keep + s * 1024) = sp[s].hi.u;
            }
            f32x4 R[4], U[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) R[m] = U[m] = kZero4;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
#pragma unroll
                for (int m = 0; m < 4; ++m) R[m] = mma(R[m], kf[m][s], sp[s].lo);
#pragma unroll
                for (int m = 0; m < 4; ++m) R[m] = mma(R[m], kf[m][s], sp[s].hi);
            }
            f32x4 be[4], kout[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
                for (int s = 0; s < m / 2 + 1; ++s) {
                    const int f = lower_frag(m, s);
                    if constexpr (kApart) {
                        const unsigned char* at = lds + LD::t + f * 2048 + lane * 16;
                        th[f].u = *reinterpret_cast<const uint4*>(at);
                        tl[f].u = *reinterpret_cast<const uint4*>(at + 1024);
                    } else {
                        const unsigned char* at = lds + LD::t + packed_at(m, s) * 1024;
                        th[f].u = packed_read(at, packed_half(m, s), lane);
                        tl[f].u = packed_read(at + (packed_half(m, s) ? 512 : 1024), packed_half(m, s), lane);
                    }
                }
                if constexpr (kApart) {
                    be[m] = v4(*reinterpret_cast<const float4*>(lds + LD::kin + (kBeta * C + 16 * m + 4 * q) * 4));
                    kout[m] = v4(*reinterpret_cast<const float4*>(lds + LD::kin + (kKout * C + 16 * m + 4 * q) * 4));
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            // k^T: row i of the state tiles' numbering, K index t
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int r = 4 * q + i / 4, at = LD::piece(r, 4 * (n / 2) + i % 4) * 16 + 8 * (n % 2);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const FragBF f = tr_read(lds, LD::k + (32 * s + 16 * e + r) * LD::kRow + at);
                        kt[n][s].w[2 * e] = f.a;
                        kt[n][s].w[2 * e + 1] = f.b;
                    }
                }
            f32x4 X[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const f32x4 v = {bf16_lo(vf[m].a), bf16_hi(vf[m].a), bf16_lo(vf[m].b), bf16_hi(vf[m].b)};
                X[m] = v - kin[m] * R[m];
                if constexpr (kApart) X[m] *= be[m];
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) S[n] *= across;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Pair xp = split2(X[2 * s], X[2 * s + 1]);
                if (MODE == kFull) {
                    *reinterpret_cast<uint4*>(keep + (KS + 2 * s) * 1024) = xp.hi.u;
                    *reinterpret_cast<uint4*>(keep + (KS + 2 * s + 1) * 1024) = xp.lo.u;
                }
#pragma unroll
                for (int x = 0; x < 3; ++x)
#pragma unroll
                    for (int m = 2 * s; m < 4; ++m) {
                        const int f = lower_frag(m, s);
                        U[m] = x == 0 ? mma(U[m], tl[f], xp.hi) : mma(U[m], th[f], x == 1 ? xp.lo : xp.hi);
                    }
            }
            if constexpr (MODE == kStates) {
                float* to = io.keepU + ((size_t)bh * io.nc + c0 + c) * C * a.P + p0 + 16 * wave + i;
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r) to[(size_t)(16 * m + 4 * q + r) * a.P] = U[m][r];
            }
            if constexpr (kApart) {
#pragma unroll
                for (int m = 0; m < 4; ++m) U[m] *= kout[m];
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Pair up = split2(U[2 * s], U[2 * s + 1]);
#pragma unroll
                for (int n = 0; n < NT; ++n) S[n] = mma(S[n], kt[n][s], up.lo);
#pragma unroll
                for (int n = 0; n < NT; ++n) S[n] = mma(S[n], kt[n][s], up.hi);
            }
            lds_barrier();
        }
        if (nch & 1) lds_barrier();                  // the other waves go in pairs
        float* last;
        if (MODE == kStates) {
            last = nullptr;
        } else if (kPass) {
            const size_t u = (size_t)bh * io.K + sk;
            last = phi ? (pc < N ? io.phi + (u * N + pc) * N + 8 * q : nullptr) : io.loc + (u * a.P + p0 + 16 * wave + i) * N + 8 * q;
        } else {
            last = a.final_state && sk == io.K - 1 ? a.final_state + sofs : nullptr;
        }
        if (last) {
#pragma unroll
            for (int n = 0; n < NT; ++n) *reinterpret_cast<float4*>(last + 32 * (n / 2) + 4 * (n % 2)) = f4(S[n]);
        }
        return;
    }
    // ---------------------------------------------------- staging and y
    constexpr int NK = C * nc16 / 256, NV = 2, NTp = (LD::t_bytes / 16 + 255) / 256, NS = kApart ? kScalBwd : kScal;
    // two chunks are on their way at any time, in register sets of their parity: one chunk's time is less than
    // the memory's latency under this kernel's own load
    u32x4_t rk[2][NK], rv[2][NV], rt[2][NTp];
    float rs[2], ra[2];
    const unsigned char* kb = static_cast<const unsigned char*>(a.k) + (tok0 * a.k_stride + (size_t)g * N) * 2;
    const unsigned char* qb = static_cast<const unsigned char*>(a.q) + (tok0 * a.q_stride + (size_t)g * N) * 2;
    const unsigned char* vb = static_cast<const unsigned char*>(a.v) + (tok0 * a.v_stride + (size_t)h * a.P + p0) * 2;
    unsigned char* yb = static_cast<unsigned char*>(a.y) + tok0 * a.y_stride * 2;
    const uint32_t k_row = (uint32_t)a.k_stride * 2, q_row = (uint32_t)a.q_stride * 2, v_row = (uint32_t)a.v_stride * 2;
    const uint32_t y_row = (uint32_t)a.y_stride * 2, y_col = (uint32_t)(h * a.P + p0 + 16 * (q & 1) + 8 * (q >> 1)) * 2;
    // No branch stands between the loads, the stores and the waits for them, so
    // that the waits can count: a chunk number past the end is the last one's,
    // rows past the sequence read its last row (k and v of them become zeros on
    // their way to LDS), and their y falls out of the buffer's range.
    auto fetch = [&](int c, auto set) {
        constexpr int Z = decltype(set)::value;
        c = c0 + min(c, nch - 1);
        const size_t u = (size_t)bh * io.nc + c;
        const int n_on = min(C, len - c * C);
        const unsigned char *kc = kb + (size_t)c * C * k_row, *vc = vb + (size_t)c * C * v_row;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int e = tid + 256 * j, t = min(e / nc16, n_on - 1), x = e % nc16;
            rk[Z][j] = *reinterpret_cast<const u32x4_t*>(kc + ((uint32_t)t * k_row + x * 16));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = tid + 256 * j, t = min(e / 8, n_on - 1), x = e % 8;
            rv[Z][j] = *reinterpret_cast<const u32x4_t*>(vc + ((uint32_t)t * v_row + x * 16));
        }
#pragma unroll
        for (int j = 0; j < NTp; ++j) {
            const int e = min(tid + 256 * j, LD::t_bytes / 16 - 1);
            rt[Z][j] = *reinterpret_cast<const u32x4_t*>(io.T + u * LD::t_bytes + e * 16);
        }
        if constexpr (kApart) {
            rs[Z] = io.scal[u * NS * C + tid];
            ra[Z] = io.across[u];
        } else {
            const float* sc = tid < C ? io.scal + (u * NS + kKin) * C + tid : io.across + u;
            rs[Z] = *sc;
        }
    };
    auto stage = [&](int c, auto set) {
        constexpr int Z = decltype(set)::value;
        unsigned char* const lds = lds_all + (c & 1) * LD::buffer;
        const int n_on = len - (c0 + min(c, nch - 1)) * C;
        const u32x4_t zero = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int e = tid + 256 * j, t = e / nc16, x = e % nc16;
            *reinterpret_cast<u32x4_t*>(lds + LD::k + t * LD::kRow + LD::piece(t, x) * 16) = t < n_on ? rk[Z][j] : zero;
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int e = tid + 256 * j, t = e / 8, x = e % 8;
            *reinterpret_cast<u32x4_t*>(lds + LD::v + t * LD::vRow + x * 16) = t < n_on && !phi ? rv[Z][j] : zero;
        }
#pragma unroll
        for (int j = 0; j < NTp; ++j)                // past T's end the last piece again
            *reinterpret_cast<u32x4_t*>(lds + LD::t + min(tid + 256 * j, LD::t_bytes / 16 - 1) * 16) = rt[Z][j];
        if constexpr (kApart) {
            *reinterpret_cast<float*>(lds + LD::kin + tid * 4) = rs[Z];
            if (tid == 0) *reinterpret_cast<float*>(lds + LD::across) = ra[Z];
        } else {
            if (tid < 128) *reinterpret_cast<float*>(lds + LD::kin + min(tid, C) * 4) = rs[Z];
        }
    };
    // y: this wave's 16 tokens of all 64 columns, so that each piece of q and Att T is read by one wave
    Frag qf[2][KS], af[2][2];
    float qin[2];
    auto fetch_q = [&](int c, auto set) {
        constexpr int Z = decltype(set)::value;
        c = c0 + min(c, nch - 1);
        const size_t u = (size_t)bh * io.nc + c;
        const int t = min(16 * wave + i, min(C, len - c * C) - 1);
        const unsigned char* qc = qb + ((size_t)c * C + t) * q_row + 16 * q;
        qin[Z] = io.scal[(u * kScal + kQin) * C + 16 * wave + i];
#pragma unroll
        for (int s = 0; s < KS; ++s) qf[Z][s].u = *reinterpret_cast<const uint4*>(qc + 64 * s);
        const unsigned char* ac = io.att + u * Bytes<false>::att + lane * 16;
        af[Z][0].u = *reinterpret_cast<const uint4*>(ac + lower_frag(wave, 0) * 1024);
        af[Z][1].u = *reinterpret_cast<const uint4*>(ac + lower_frag(wave, wave / 2) * 1024);   // waves 2 and 3: their second
    };
    const std::integral_constant<int, 0> even;
    const std::integral_constant<int, 1> odd;
    // The loads before the loop stand in the loop's own order, stores (dropped, out of range) included: a wait in the
    // loop can then count past as many younger operations on its first round as on the others, and waits for no more.
    auto no_store = [&]() {
        const __amdgpu_buffer_rsrc_t none = __builtin_amdgcn_make_buffer_rsrc(yb, 0, 0, 0x00020000);
        __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{0, 0, 0, 0}, none, 0x80000000u, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{0, 0, 0, 0}, none, 0x80000000u, 64, 0);
    };
    if (nch > 0) {
        fetch(0, even);
        stage(0, even);
        fetch(1, odd);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MODE == kFull) {
            fetch_q(0, even);
            __builtin_amdgcn_sched_barrier(0);
            no_store();
        }
        __builtin_amdgcn_sched_barrier(0);
        fetch(2, even);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (MODE == kFull) {
            fetch_q(1, odd);
            __builtin_amdgcn_sched_barrier(0);
            no_store();
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    lds_barrier();
    // while the chain is at chunk c (of parity Z): chunk c + 1 to LDS, c + 3 on its way; behind the barrier, beside
    // chunk c + 1, y of c
    auto body = [&](int c, auto set, auto other) {
        constexpr int Z = decltype(set)::value;
        stage(c + 1, other);
        fetch(c + 3, other);
        lds_barrier();
        if constexpr (MODE != kFull) return;
        const unsigned char* const keep = lds_all + 2 * LD::buffer + (c & 1) * 4 * LD::kept + lane * 16;
        f32x4 O[4];
#pragma unroll
        for (int w0 = 0; w0 < 4; w0 += 2) {          // the chain's waves, 16 columns each, two at a time
            Frag f[2][KS + 4];
#pragma unroll
            for (int x = 0; x < KS + 4; ++x)
#pragma unroll
                for (int w = 0; w < 2; ++w) f[w][x].u = *reinterpret_cast<const uint4*>(keep + (w0 + w) * LD::kept + x * 1024);
            __builtin_amdgcn_sched_barrier(0);
            O[w0] = O[w0 + 1] = kZero4;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int w = 0; w < 2; ++w) O[w0 + w] = mma(O[w0 + w], f[w][s], qf[Z][s]);   // [p][t]
#pragma unroll
            for (int w = 0; w < 2; ++w) O[w0 + w] *= qin[Z];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int w = 0; w < 2; ++w) O[w0 + w] = mma(O[w0 + w], f[w][KS + x], af[Z][0]);
            if (wave >= 2) {
#pragma unroll
                for (int x = 2; x < 4; ++x)
#pragma unroll
                    for (int w = 0; w < 2; ++w) O[w0 + w] = mma(O[w0 + w], f[w][KS + x], af[Z][1]);
            }
        }
        fetch_q(c + 2, set);
        const __amdgpu_buffer_rsrc_t yr = __builtin_amdgcn_make_buffer_rsrc(yb + (size_t)(c0 + c) * C * y_row, 0, 0x7fffffff, 0x00020000);
        const int t = 16 * wave + i;
        const uint32_t at = c < nch && (c0 + c) * C + t < len ? (uint32_t)t * y_row + y_col : 0x80000000u;
#pragma unroll
        for (int w = 0; w < 4; w += 2) {
            // lanes of neighbouring rows of 16 exchange halves of two tiles: eight columns a lane, 64 bytes a token
            const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16x2(O[w][0], O[w][1]), pack_bf16x2(O[w + 1][0], O[w + 1][1]), false, false);
            const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16x2(O[w][2], O[w][3]), pack_bf16x2(O[w + 1][2], O[w + 1][3]), false, false);
            __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{lo[0], hi[0], lo[1], hi[1]}, yr, at, 32 * w, 0);
        }
    };
    // in pairs, so that the loop has one way round and the waits' counts hold; the chain passes as many barriers
    for (int c = 0; c < nch; c += 2) {
        body(c, even, odd);
        body(c + 1, odd, even);
    }
    if (MODE != kFull) return;
    // rows past the sequence are exactly 0
    const int tend = sk == io.K - 1 ? a.L : min(a.L, (c0 + io.S) * C);
    for (int t = max(len, c0 * C) + i; t < tend; t += 16) if (wave % 2 == 0) *reinterpret_cast<uint4*>(yb + (size_t)t * y_row + y_col + 32 * wave) = make_uint4(0, 0, 0, 0);
}

// The states entering the superchunks, S_{k+1} = Phi_k S_k + loc_k in turn, on the fp32 MFMA.  A workgroup has 16
// columns, its waves every fourth row tile; all of S_k goes round through LDS, whose two halves take turns.  The
// backward's gradients of the states (REV) go the other way, D_{k-1} = Phi_k^T D_k + loc_k.
template <int N, bool REV>
__global__ __launch_bounds__(256) void ssd_delta_join_kernel(DeltaArgs a, ScanIo io, const float* first) {
    constexpr int NT = N / 16, NW = (NT + 3) / 4;
    __shared__ __align__(16) float4 s_all[2][NT][64];
    const int lane = threadIdx.x % 64, q = lane / 16, i = lane % 16;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int pb = a.P / 16, bh = blockIdx.x / pb, p = blockIdx.x % pb * 16 + i;
    f32x4 S[NW];
#pragma unroll
    for (int j = 0; j < NW; ++j) {
        const int n = w + 4 * j;
        S[j] = first && n < NT ? v4(*reinterpret_cast<const float4*>(first + ((size_t)bh * a.P + p) * N + 16 * n + 4 * q)) : kZero4;
    }
    for (int x = 0; x < io.K; ++x) {
        const size_t u = (size_t)bh * io.K + (REV ? io.K - 1 - x : x);
        float* to = io.s0 + (u * a.P + p) * N + 4 * q;
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int n = w + 4 * j;
            if (n < NT) {
                *reinterpret_cast<float4*>(to + 16 * n) = f4(S[j]);
                s_all[x & 1][n][lane] = f4(S[j]);
            }
        }
        if (x == io.K - 1) break;
        __syncthreads();
        const float* loc = io.loc + (u * a.P + p) * N + 4 * q;
        const float* phi = io.phi + u * N * N;                 // [column][row]
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            const int n = w + 4 * j;
            if (n >= NT) continue;
            f32x4 R = v4(*reinterpret_cast<const float4*>(loc + 16 * n));
#pragma unroll
            for (int m = 0; m < NT; ++m) {
                float4 f;                                      // row 16 n + i of Phi or its transpose, columns 16 m + 4 q ..
                if constexpr (REV) {
                    f = *reinterpret_cast<const float4*>(phi + (16 * n + i) * N + 16 * m + 4 * q);
                } else {
                    const float* at = phi + (16 * m + 4 * q) * N + 16 * n + i;
                    f = make_float4(at[0], at[N], at[2 * N], at[3 * N]);
                }
                R = mma_f32(R, f, s_all[x & 1][m][lane]);
            }
            S[j] = R;
        }
    }
}

// ---- fp32: the forward (kY), and the backward's recomputation of S and U (kKeep)
// The same chain on the fp32 MFMA (a 16 x 16 x 4 product takes 32 cycles), which is what bounds it: k, q, Att and T come
// as they are, four waves stage their own chunks, and y is computed in the chain.  Measured: B=3 L=77 H=8 P=N=64 in 14.5
// us, two chunks of 272 products a wave (3.6 us each at 2.4 GHz) and the first chunk's loads; the backward's S and U of
// B=2 L=150 H=4 P=64 N=32 in 11.4 us.
enum { kY = 0, kKeep = 1 };

template <int N, int MODE>
struct ScanLds {
    static constexpr int es = 4;
    static constexpr int kRow = N * es + 16;         // bytes of a k or q row: the odd 16 spreads rows over the banks
    static constexpr int vRow = 64 * es + 16;
    static constexpr int k = 0, v = k + C * kRow, t = v + C * vRow, scal = t + Bytes<true>::split;
    static constexpr int q = scal + kScal * C * 4, att = q + (MODE == kY ? C * kRow : 0);
    static constexpr int bytes = att + (MODE == kY ? Bytes<true>::att : 0);
    static constexpr int buffers = 2 * bytes <= 160 * 1024 ? 2 : 1;
};

template <int N, int MODE>
__global__ __launch_bounds__(256) void ssd_delta_scan_kernel(DeltaArgs a, ScanIo io) {
    using LD = ScanLds<N, MODE>;
    constexpr int NT = N / 16, es = LD::es, nc16 = N * es / 16, nv16 = 64 * es / 16;
    constexpr int NS = MODE == kY ? kScal : kScalBwd;
    extern __shared__ __align__(16) unsigned char lds_all[];
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
    auto state_n = [&](int n) { return 16 * n + 4 * q; };
    const size_t sofs = ((size_t)bh * a.P + p) * N;
    f32x4 S[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        S[n] = a.init_state ? v4(*reinterpret_cast<const float4*>(a.init_state + sofs + state_n(n))) : kZero4;

    // ---- staging: 16-byte pieces, the next chunk's in registers
    constexpr int NK = C * nc16 / 256, NVp = C * nv16 / 256;
    constexpr int NTp = (Bytes<true>::split / 16 + 255) / 256, NA = (Bytes<true>::att / 16 + 255) / 256;
    u32x4_t rk[NK], rq[NK], rv[NVp], rt[NTp], ra[NA];
    float rs = 0.0f, r_across = 0.0f;
    const unsigned char* kb = static_cast<const unsigned char*>(a.k) + (tok0 * a.k_stride + (size_t)g * N) * es;
    const unsigned char* qb = static_cast<const unsigned char*>(a.q) + (tok0 * a.q_stride + (size_t)g * N) * es;
    const unsigned char* vb = static_cast<const unsigned char*>(a.v) + (tok0 * a.v_stride + (size_t)h * a.P + p0) * es;
    const uint32_t k_row = (uint32_t)a.k_stride * es, q_row = (uint32_t)a.q_stride * es, v_row = (uint32_t)a.v_stride * es;
    // rows past the sequence read its last row here and become zeros on their way to LDS
    auto fetch = [&](int c) {
        const size_t u = (size_t)bh * io.nc + c;
        const int n_on = min(C, len - c * C);
        const unsigned char *kc = kb + (size_t)c * C * k_row, *qc = qb + (size_t)c * C * q_row, *vc = vb + (size_t)c * C * v_row;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int e = tid + 256 * j, t = min(e / nc16, n_on - 1), x = e % nc16;
            rk[j] = *reinterpret_cast<const u32x4_t*>(kc + ((uint32_t)t * k_row + x * 16));
            if (MODE == kY) rq[j] = *reinterpret_cast<const u32x4_t*>(qc + ((uint32_t)t * q_row + x * 16));
        }
#pragma unroll
        for (int j = 0; j < NVp; ++j) {
            const int e = tid + 256 * j, t = min(e / nv16, n_on - 1), x = e % nv16;
            rv[j] = *reinterpret_cast<const u32x4_t*>(vc + ((uint32_t)t * v_row + x * 16));
        }
#pragma unroll
        for (int j = 0; j < NTp; ++j) {
            const int e = min(tid + 256 * j, Bytes<true>::split / 16 - 1);
            rt[j] = *reinterpret_cast<const u32x4_t*>(io.T + u * Bytes<true>::split + e * 16);
        }
        if (MODE == kY) {
#pragma unroll
            for (int j = 0; j < NA; ++j) {
                const int e = min(tid + 256 * j, Bytes<true>::att / 16 - 1);
                ra[j] = *reinterpret_cast<const u32x4_t*>(io.att + u * Bytes<true>::att + e * 16);
            }
        }
        rs = io.scal[u * NS * C + tid];
        r_across = io.across[u];
    };
    auto stage = [&](unsigned char* lds, int c) {
        const int n_on = len - c * C;
        const u32x4_t zero = {0, 0, 0, 0};
        if (n_on < C) {
#pragma unroll
            for (int j = 0; j < NK; ++j)
                if ((tid + 256 * j) / nc16 >= n_on) {
                    rk[j] = zero;
                    if (MODE == kY) rq[j] = zero;
                }
#pragma unroll
            for (int j = 0; j < NVp; ++j)
                if ((tid + 256 * j) / nv16 >= n_on) rv[j] = zero;
        }
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int e = tid + 256 * j, t = e / nc16, x = e % nc16;
            *reinterpret_cast<u32x4_t*>(lds + LD::k + t * LD::kRow + x * 16) = rk[j];
            if (MODE == kY) *reinterpret_cast<u32x4_t*>(lds + LD::q + t * LD::kRow + x * 16) = rq[j];
        }
#pragma unroll
        for (int j = 0; j < NVp; ++j) {
            const int e = tid + 256 * j, t = e / nv16, x = e % nv16;
            *reinterpret_cast<u32x4_t*>(lds + LD::v + t * LD::vRow + x * 16) = rv[j];
        }
#pragma unroll
        for (int j = 0; j < NTp; ++j)
            if (tid + 256 * j < Bytes<true>::split / 16) *reinterpret_cast<u32x4_t*>(lds + LD::t + (tid + 256 * j) * 16) = rt[j];
        if (MODE == kY) {
#pragma unroll
            for (int j = 0; j < NA; ++j)
                if (tid + 256 * j < Bytes<true>::att / 16) *reinterpret_cast<u32x4_t*>(lds + LD::att + (tid + 256 * j) * 16) = ra[j];
        }
        *reinterpret_cast<float*>(lds + LD::scal + tid * 4) = rs;
    };

    unsigned char* yb = static_cast<unsigned char*>(a.y) + tok0 * a.y_stride * es;
    const uint32_t y_row = (uint32_t)a.y_stride * es, y_col = (uint32_t)(h * a.P + p0 + 16 * wave + 4 * q) * es;
    float across = 0.0f;
    if (nch > 0) {
        fetch(0);
        stage(lds_all, 0);
        across = r_across;
        if (nch > 1) fetch(1);
        lds_barrier();
    }
    for (int c = 0; c < nch; ++c) {
        unsigned char* const lds = lds_all + (LD::buffers == 2 && c % 2 ? LD::bytes : 0);
        auto scal4 = [&](int what, int m) {
            return v4(*reinterpret_cast<const float4*>(lds + LD::scal + (what * C + 16 * m + 4 * q) * 4));
        };
        auto frag16 = [&](int ofs) { return *reinterpret_cast<const uint4*>(lds + ofs + lane * 16); };
        auto next = [&]() {                          // the next chunk to the other buffer, the one after it on its way
            if (c + 1 < nch) {
                stage(lds_all + (LD::buffers == 2 && c % 2 == 0 ? LD::bytes : 0), c + 1);
                across = r_across;
                if (c + 2 < nch) fetch(c + 2);
            }
        };
        const float keep = across;                   // of this chunk
        if constexpr (MODE == kKeep) {
            float* ks = io.keepS + ((size_t)bh * io.nc + c) * N * a.P + p;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) ks[(size_t)(state_n(n) + r) * a.P] = S[n][r];
        }
        f32x4 R[4], X[4], U[4], O[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            R[m] = O[m] = kZero4;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float4 kf = *reinterpret_cast<const float4*>(lds + LD::k + (16 * m + i) * LD::kRow + (16 * n + 4 * q) * 4);
                R[m] = mma_f32(R[m], kf, f4(S[n]));
                if constexpr (MODE == kY) {
                    const float4 qf = *reinterpret_cast<const float4*>(lds + LD::q + (16 * m + i) * LD::kRow + (16 * n + 4 * q) * 4);
                    O[m] = mma_f32(O[m], f4(S[n]), qf);
                }
            }
            const f32x4 kin = scal4(kKin, m), be = scal4(kBeta, m);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float v = *reinterpret_cast<const float*>(lds + LD::v + (16 * m + 4 * q + r) * LD::vRow + (16 * wave + i) * 4);
                X[m][r] = be[r] * (v - kin[r] * R[m][r]);
            }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            U[m] = kZero4;
#pragma unroll
            for (int n = 0; n <= m; ++n)
                U[m] = mma_f32(U[m], __builtin_bit_cast(float4, frag16(LD::t + tile_id(m, n) * 1024)), f4(X[n]));
        }
        if constexpr (MODE == kY) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                O[m] *= *reinterpret_cast<const float*>(lds + LD::scal + (kQin * C + 16 * m + i) * 4);
#pragma unroll
                for (int n = 0; n <= m; ++n)
                    O[m] = mma_f32(O[m], f4(U[n]), __builtin_bit_cast(float4, frag16(LD::att + tile_id(m, n) * 1024)));
            }
        }
        f32x4 w[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) w[m] = U[m] * scal4(kKout, m);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            S[n] *= keep;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const unsigned char* kc = lds + LD::k + (16 * m + 4 * q) * LD::kRow + (16 * n + i) * 4;
                float4 kt;
                kt.x = *reinterpret_cast<const float*>(kc);
                kt.y = *reinterpret_cast<const float*>(kc + LD::kRow);
                kt.z = *reinterpret_cast<const float*>(kc + 2 * LD::kRow);
                kt.w = *reinterpret_cast<const float*>(kc + 3 * LD::kRow);
                S[n] = mma_f32(S[n], kt, f4(w[m]));
            }
        }
        if constexpr (LD::buffers == 1) lds_barrier();   // this chunk's operands have been read
        next();
        __builtin_amdgcn_sched_barrier(0);
        // Stores come last and without a branch (rows past the sequence are out
        // of the buffer's range and dropped): the next chunk's wait for its
        // loads then counts past them instead of waiting for them.
        if constexpr (MODE == kY) {
            const __amdgpu_buffer_rsrc_t yr =
                __builtin_amdgcn_make_buffer_rsrc(yb + (size_t)c * C * y_row, 0, 0x7fffffff, 0x00020000);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int t = 16 * m + i;
                const uint32_t at = c * C + t < len ? (uint32_t)t * y_row + y_col : 0x80000000u;
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, O[m]), yr, at, 0, 0);
            }
        } else {
            float* ku = io.keepU + ((size_t)bh * io.nc + c) * C * a.P + p;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) ku[(size_t)(16 * m + 4 * q + r) * a.P] = U[m][r];
        }
        lds_barrier();
    }
    if constexpr (MODE == kY) {
        // rows past the sequence are exactly 0
        for (int t = len + i; t < a.L; t += 16) *reinterpret_cast<float4*>(yb + (size_t)t * y_row + y_col) = make_float4(0, 0, 0, 0);
        if (a.final_state) {
#pragma unroll
            for (int n = 0; n < NT; ++n) *reinterpret_cast<float4*>(a.final_state + sofs + state_n(n)) = f4(S[n]);
        }
    }
}

// Superchunks of a sequence, bf16: the K that takes the fewest chunk steps, with one workgroup a CU at a time.  Against
// a step of the full pass the state pass's, without y, is counted as 0.75, and joining one superchunk as 3 (measured: 2.4,
// 1.6 and 3 us at N = P = 128).  B=1 L=32768 H=16 N=P=128 takes 1.07 ms whole and 0.47 ms in the superchunks chosen.
// The backward has two full passes (a step of both: 2.2) and two state passes, the transitions in the first only, and two
// joins: B=2 L=8192 H=32 N=P=64 takes 902 us whole and 722 us in four superchunks.
void delta_split(int B, int L, int H, int P, int N, int dtype, bool bwd, int& K, int& S) {
    const int nc = (L + C - 1) / C;
    const int64_t units = (int64_t)B * H * (P / 64), wide = (int64_t)B * H * (P / 64 + (N + 63) / 64);
    K = 1;
    S = nc;
    if (dtype == 0) return;
    auto rounds = [](int64_t n) { return (double)((n + 255) / 256); };
    const double full = bwd ? 2.2 : 1.0;
    double best = full * rounds(units) * nc;
    for (int k = 2; k <= 32; ++k) {
        const int s = (nc + k - 1) / k, used = (nc + s - 1) / s;
        if (s < 8) break;
        const double ahead = bwd ? rounds(wide * used) + rounds(units * (used - 1)) : rounds(wide * (used - 1));
        const double t = s * (full * rounds(units * used) + 0.75 * ahead) + (bwd ? 6.0 : 3.0) * (used - 1);
        if (t < best) {
            best = t;
            K = used;
            S = s;
        }
    }
}

struct FwdWs {                     // byte offsets
    size_t T, att, scal, across, loc, phi, s0, total;
    int K, S;
};
FwdWs fwd_ws(int B, int L, int H, int P, int N, int dtype) {
    const size_t heads = (size_t)B * H, units = heads * ((L + C - 1) / C);
    FwdWs w;
    delta_split(B, L, H, P, N, dtype, false, w.K, w.S);
    const size_t split = w.K > 1 ? heads * w.K * N * 4 : 0;
    w.T = 0;
    w.att = w.T + units * (dtype == 0 ? Bytes<true>::split : Bytes<false>::packed);
    w.scal = w.att + units * (dtype == 0 ? Bytes<true>::att : Bytes<false>::att);
    w.across = w.scal + units * kScal * C * 4;
    w.loc = w.across + (units * 4 + 255) / 256 * 256;
    w.phi = w.loc + split * P;
    w.s0 = w.phi + split * N;
    w.total = w.s0 + split * P;
    return w;
}

// the states entering the superchunks: the pass over all of them but, in the forward, the last, and the join
template <int N, int MODE>
hipError_t launch_ahead(const DeltaArgs& a, const ScanIo& io, int count, hipStream_t stream) {
    constexpr size_t lds = 2 * ChainLds<N, MODE>::buffer;
    hipError_t e = prepare_launch(reinterpret_cast<const void*>(&ssd_delta_chain_kernel<N, MODE>), lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ssd_delta_chain_kernel<N, MODE>), dim3(a.B * a.H * (a.P / 64 + (N + 63) / 64) * count), dim3(512), lds, stream, a, io);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ssd_delta_join_kernel<N, false>), dim3(a.B * a.H * (a.P / 16)), dim3(256), 0, stream, a, io, a.init_state);
    return hipGetLastError();
}

template <typename T, int N>
hipError_t launch_fwd_n(const DeltaArgs& a, void* ws, hipStream_t stream) {
    constexpr bool F32 = std::is_same<T, float>::value;
    constexpr int PM = F32 ? kPrepPlain : kPrepScaled;
    const int nc = (a.L + C - 1) / C;
    const FwdWs w = fwd_ws(a.B, a.L, a.H, a.P, N, a.dtype);
    unsigned char* base = static_cast<unsigned char*>(ws);
    PrepOut o{base + w.T, nullptr, base + w.att, reinterpret_cast<float*>(base + w.scal),
              reinterpret_cast<float*>(base + w.across)};
    const int64_t units = (int64_t)a.B * a.H * nc;
    hipLaunchKernelGGL((ssd_delta_prep_kernel<T, N, PM>), dim3((unsigned)((units + kPrepWaves - 1) / kPrepWaves)),
                       dim3(64 * kPrepWaves), 0, stream, a, o, nc);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    auto fp = [&](size_t at) { return reinterpret_cast<float*>(base + at); };
    ScanIo io{o.T, o.att, o.scal, o.across, nc, nullptr, nullptr, w.K, w.S, fp(w.loc), fp(w.phi), fp(w.s0)};
    const dim3 grid(a.B * a.H * (a.P / 64) * w.K);
    if constexpr (F32) {
        constexpr size_t lds = (size_t)ScanLds<N, kY>::bytes * ScanLds<N, kY>::buffers;
        e = prepare_launch(reinterpret_cast<const void*>(&ssd_delta_scan_kernel<N, kY>), lds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((ssd_delta_scan_kernel<N, kY>), grid, dim3(256), lds, stream, a, io);
    } else {
        constexpr size_t lds = ChainLds<N, kFull>::bytes;
        if (w.K > 1) {
            e = launch_ahead<N, kState>(a, io, w.K - 1, stream);
            if (e != hipSuccess) return e;
        }
        e = prepare_launch(reinterpret_cast<const void*>(&ssd_delta_chain_kernel<N, kFull>), lds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((ssd_delta_chain_kernel<N, kFull>), grid, dim3(512), lds, stream, a, io);
    }
    return hipGetLastError();
}

template <typename T, int N>
hipError_t launch_keep_n(const DeltaArgs& a, const PrepOut& o, const KeepOut& k, hipStream_t stream) {
    const int nc = (a.L + C - 1) / C;
    const int64_t units = (int64_t)a.B * a.H * nc;
    hipLaunchKernelGGL((ssd_delta_prep_kernel<T, N, kPrepBwd>), dim3((unsigned)((units + kPrepWaves - 1) / kPrepWaves)),
                       dim3(64 * kPrepWaves), 0, stream, a, o, nc);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    ScanIo io{o.T, nullptr, o.scal, o.across, nc, k.S, k.U, k.split.K, k.split.S, k.split.loc, k.split.phi, k.split.s0};
    const dim3 grid(a.B * a.H * (a.P / 64) * k.split.K);
    if constexpr (std::is_same<T, float>::value) {
        constexpr size_t lds = (size_t)ScanLds<N, kKeep>::bytes * ScanLds<N, kKeep>::buffers;
        e = prepare_launch(reinterpret_cast<const void*>(&ssd_delta_scan_kernel<N, kKeep>), lds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((ssd_delta_scan_kernel<N, kKeep>), grid, dim3(256), lds, stream, a, io);
    } else {
        constexpr size_t lds = ChainLds<N, kStates>::bytes;
        if (k.split.K > 1) {                         // the last superchunk's transition is for the gradients
            e = launch_ahead<N, kStateApart>(a, io, k.split.K, stream);
            if (e != hipSuccess) return e;
        }
        e = prepare_launch(reinterpret_cast<const void*>(&ssd_delta_chain_kernel<N, kStates>), lds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((ssd_delta_chain_kernel<N, kStates>), grid, dim3(512), lds, stream, a, io);
    }
    return hipGetLastError();
}
template <typename T>
hipError_t launch_keep_t(const DeltaArgs& a, const PrepOut& o, const KeepOut& k, hipStream_t stream) {
    switch (a.N) {
        case 32: return launch_keep_n<T, 32>(a, o, k, stream);
        case 64: return launch_keep_n<T, 64>(a, o, k, stream);
        case 128: return launch_keep_n<T, 128>(a, o, k, stream);
    }
    return hipErrorInvalidValue;
}

template <int N>
hipError_t launch_join_back_n(const DeltaArgs& a, const Split& s, const float* g_final, hipStream_t stream) {
    ScanIo io{};
    io.K = s.K;
    io.S = s.S;
    io.loc = s.loc;
    io.phi = s.phi;
    io.s0 = s.s0;
    hipLaunchKernelGGL((ssd_delta_join_kernel<N, true>), dim3(a.B * a.H * (a.P / 16)), dim3(256), 0, stream, a, io, g_final);
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

namespace delta {
hipError_t launch_keep(const DeltaArgs& a, const PrepOut& o, const KeepOut& k, hipStream_t stream) {
    return a.dtype == 0 ? launch_keep_t<float>(a, o, k, stream) : launch_keep_t<uint16_t>(a, o, k, stream);
}
hipError_t launch_join_back(const DeltaArgs& a, const Split& s, const float* g_final, hipStream_t stream) {
    switch (a.N) {
        case 32: return launch_join_back_n<32>(a, s, g_final, stream);
        case 64: return launch_join_back_n<64>(a, s, g_final, stream);
        case 128: return launch_join_back_n<128>(a, s, g_final, stream);
    }
    return hipErrorInvalidValue;
}
void split_bwd(int B, int L, int H, int P, int N, int dtype, Split& s) { delta_split(B, L, H, P, N, dtype, true, s.K, s.S); }
}  // namespace delta

size_t delta_fwd_workspace_bytes(int B, int L, int H, int P, int N, int dtype) { return fwd_ws(B, L, H, P, N, dtype).total; }

hipError_t launch_delta_fwd(const DeltaArgs& a, void* ws, hipStream_t stream) {
    return a.dtype == 0 ? launch_fwd_t<float>(a, ws, stream) : launch_fwd_t<uint16_t>(a, ws, stream);
}

}  // namespace ssd
