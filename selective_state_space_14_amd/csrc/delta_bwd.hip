// delta_bwd.hip -- backward of the gated delta rule.
//
// With dS the adjoint of the state leaving a chunk and the forward's T, U and
// S0 (delta_device.hpp), x o y the row-wise products:
//     dU = Att^T dY + e^{G_C - G} o K dS         Z = T^T dU         dV = beta o Z
//     dS0 = e^{G_C} dS + (scale e^G o Q)^T dY - (beta e^G o K)^T Z
// and from dAtt = dY U^T, dL = -Z U^T, W1 = dY S0^T, W2 = Z S0^T, W3 = U dS^T
//     dQ = scale e^G o W1 + (scale M o dAtt) K
//     dK = e^{G_C - G} o W3 - beta e^G o W2 + (scale M o dAtt)^T Q + (D + D^T) K,   D = beta M o dL
//     dbeta_t = Z_t.V_t - e^{G_t} K_t.W2_t + sum_j dL_tj M_tj k_t.k_j
//     dG_t = row sums - column sums of dAtt o Att + dL o L, + scale e^{G_t} Q_t.W1_t - beta_t e^{G_t} K_t.W2_t
//            - e^{G_C - G_t} K_t.W3_t, and at the chunk's end + sum of the last + e^{G_C} <S0, dS>
//     d(dt A)_t = sum of dG behind t in the chunk
// Row and column sums are taken of the same entries, so pairs on one side
// of t cancel to fp32 rounding whatever the products' own error.
//
// Launches: delta.hip's prep (T, T^T, Att, scalars) and forward chain (S0 and U
// of every chunk), the reverse chain here (dS and Z of every chunk), then all
// chunks at once (the gradients), then dA's and ddt_bias's sums.
#include <hip/hip_runtime.h>
#include <algorithm>
#include <type_traits>

#include "delta_device.hpp"

namespace ssd {
namespace {

using namespace delta;

struct BwdIo {
    const unsigned char *TT, *att;
    const float *scal, *across;    // [u][kScalBwd][C], [u]
    const float *S, *U;            // [u][N][P], [u][C][P]
    float *D, *Z;                  // as S and U: the adjoint leaving each chunk, Z
    void* part;                    // [2][B * nc][H] (Sum)
    int nc;
    Split split;
};

// ============================================================ the reverse chain
// As the forward's: a wave holds 16 columns of dS from the last chunk to the
// first, the chunk's left operands (k and q both ways, Att^T, T^T, dY) staged
// in LDS ahead of it.  Bound by the chain's latency, like the forward.

// ---- bf16: four waves are the chain, four more bring the next chunks
// LDS is read in three batches ahead of the products they feed.  2.4 us a chunk
// at N = P = 64, against 4.1 with staging in the chain's own waves: B=2 L=8192
// H=32 took 531 us so, 307 us this way, and in four superchunks side by side
// (AHEAD and the join included) 195 us.
// Splits: dS, dU and Z are hi + lo pairs like Att and T, dY and k, q bf16 as
// they are.
template <int N>
struct BackLds {
    static constexpr int kRow = N * 2, dRow = 64 * 2 + 16;
    static constexpr int k = 0, q = k + C * kRow, d = q + C * kRow, tt = d + C * dRow;
    static constexpr int att = tt + Bytes<false>::split, scal = att + Bytes<false>::split, across = scal + kScal * C * 4;
    static constexpr int buffer = across + 256;
};

// AHEAD: superchunks from a zero gradient, for launch_join_back.
template <int N, bool AHEAD>
__global__ __launch_bounds__(512, 2) void ssd_delta_back_kernel(DeltaBwdArgs ba, BwdIo io) {
    using LD = BackLds<N>;
    constexpr int NT = N / 16, KS = N / 32, nc16 = N / 8, QS = N == 128 ? 1 : 2;   // QS: half of Q^T and K^T at a time where registers run short
    extern __shared__ __align__(16) unsigned char lds_all[];
    const DeltaArgs& a = ba.f;
    const int tid = threadIdx.x % 256, wave = tid / 64, lane = tid % 64, q = lane / 16, i = lane % 16;
    const int pb = a.P / 64;
    const int units = a.B * a.H * pb, sk = blockIdx.x / units + AHEAD;   // the first superchunk hands nothing on
    int unit = blockIdx.x % units;
    const int share = a.H / a.G * pb;                // heads of a group on one XCD
    if (a.B * a.G % 8 == 0) unit = (unit / 8 / share * 8 + unit % 8) * share + unit / 8 % share;
    const int p0 = unit % pb * 64, bh = unit / pb, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    const int len = row_len(a, b), c0 = sk * io.split.S;
    const int nch = max(0, min(io.split.S, (len + C - 1) / C - c0)), last = c0 + nch - 1;   // step e is chunk last - e
    const size_t tok0 = (size_t)b * a.L;

    if (threadIdx.x < 256) {
        const int p = p0 + 16 * wave + i;
        const size_t sofs = ((size_t)bh * a.P + p) * N + 8 * q, kofs = (((size_t)bh * io.split.K + sk) * a.P + p) * N + 8 * q;
        const float* from = AHEAD ? nullptr : io.split.K > 1 ? io.split.s0 + kofs : ba.g_final ? ba.g_final + sofs : nullptr;
        f32x4 D[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
            D[n] = from ? v4(*reinterpret_cast<const float4*>(from + 32 * (n / 2) + 4 * (n % 2))) : kZero4;
        lds_barrier();
        for (int e = 0; e < nch; ++e) {
            const unsigned char* const lds = lds_all + (e & 1) * LD::buffer;
            const size_t u = (size_t)bh * io.nc + last - e;
            auto scal4 = [&](int what, int m) {
                return v4(*reinterpret_cast<const float4*>(lds + LD::scal + (what * C + 16 * m + 4 * q) * 4));
            };
            auto frag = [&](int at) {
                Frag f;
                f.u = *reinterpret_cast<const uint4*>(lds + at + lane * 16);
                return f;
            };
            auto trans = [&](int at, int s, int n) {   // the transposed operand: row i of the state tiles' numbering, K index t
                Frag f;
                const int r = 4 * q + i / 4, x = row_piece<N>(r, 4 * (n / 2) + i % 4) * 16 + 8 * (n % 2);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const FragBF z = tr_read(lds, at + (32 * s + 16 * e + r) * LD::kRow + x);
                    f.w[2 * e] = z.a;
                    f.w[2 * e + 1] = z.b;
                }
                return f;
            };
            Frag kf[4][KS], ah[6], al[6], df[2];
            f32x4 qin[4], kout[4];
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    kf[m][s].u = *reinterpret_cast<const uint4*>(lds + LD::k + (16 * m + i) * LD::kRow + row_piece<N>(i, 4 * s + q) * 16);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const FragBF f = tr_read(lds, LD::d + (16 * m + 4 * q + i / 4) * LD::dRow + (16 * wave + 4 * (i % 4)) * 2);
                df[m / 2].w[2 * (m % 2)] = f.a;
                df[m / 2].w[2 * (m % 2) + 1] = f.b;
            }
            auto scals = [&]() {
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    qin[m] = scal4(kQin, m);
                    kout[m] = scal4(kKout, m);
                }
            };
            if (QS == 2) scals();
#pragma unroll
            for (int f = 0; f < 6; ++f) {
                ah[f] = frag(LD::att + f * 2048);
                al[f] = frag(LD::att + f * 2048 + 1024);
            }
            const float across = *reinterpret_cast<const float*>(lds + LD::across);
            __builtin_amdgcn_sched_barrier(0);
            if (QS == 1) scals();
            if constexpr (!AHEAD) {
                float* kd = io.D + u * N * a.P + p;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 4; ++r) kd[(size_t)(32 * (n / 2) + 8 * q + 4 * (n % 2) + r) * a.P] = D[n][r];
            }
            f32x4 W[4], Z[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) W[m] = Z[m] = kZero4;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const Pair sp = split2(D[2 * s], D[2 * s + 1]);
#pragma unroll
                for (int m = 0; m < 4; ++m) W[m] = mma(W[m], kf[m][s], sp.lo);
#pragma unroll
                for (int m = 0; m < 4; ++m) W[m] = mma(W[m], kf[m][s], sp.hi);
            }
            Pair yp[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint32_t* w = df[s].w;
                const f32x4 y0 = {bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
                const f32x4 y1 = {bf16_lo(w[2]), bf16_hi(w[2]), bf16_lo(w[3]), bf16_hi(w[3])};
                yp[s] = split2(y0 * qin[2 * s], y1 * qin[2 * s + 1]);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m) W[m] *= kout[m];
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int s = m / 2; s < 2; ++s) {
                    W[m] = mma(W[m], al[upper_frag(m, s)], df[s]);
                    W[m] = mma(W[m], ah[upper_frag(m, s)], df[s]);
                }
            Frag th[6], tl[6];
            f32x4 kb[4];
#pragma unroll
            for (int f = 0; f < 6; ++f) {
                th[f] = frag(LD::tt + f * 2048);
                tl[f] = frag(LD::tt + f * 2048 + 1024);
            }
            {
                // the part of dS that does not wait for Z fills in while W is split
#pragma unroll
                for (int n = 0; n < NT; ++n) D[n] *= across;
#pragma unroll
                for (int m = 0; m < 4; ++m) kb[m] = scal4(kKin, m) * scal4(kBeta, m);
#pragma unroll
                for (int s = 0; s < 2; s += QS) {
                    Frag qt[QS][NT];
#pragma unroll
                    for (int x = 0; x < QS; ++x)
#pragma unroll
                        for (int n = 0; n < NT; ++n) qt[x][n] = trans(LD::q, s + x, n);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int x = 0; x < QS; ++x) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) D[n] = mma(D[n], qt[x][n], yp[s + x].lo);
#pragma unroll
                        for (int n = 0; n < NT; ++n) D[n] = mma(D[n], qt[x][n], yp[s + x].hi);
                    }
                }
            }
            const Pair up[2] = {split2(W[0], W[1]), split2(W[2], W[3])};
            Frag kt[NT][2];
            auto read_kt = [&](int s) {
#pragma unroll
                for (int n = 0; n < NT; ++n) kt[n][s] = trans(LD::k, s, n);
            };
            read_kt(0);
            if (QS == 2) read_kt(1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = 1; s >= 0; --s)
#pragma unroll
                for (int x = 0; x < 3; ++x)
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        if (m / 2 > s) continue;
                        const int f = upper_frag(m, s);
                        Z[m] = x == 0 ? mma(Z[m], tl[f], up[s].hi) : mma(Z[m], th[f], x == 1 ? up[s].lo : up[s].hi);
                    }
            float* kz = io.Z + u * C * a.P + p;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!AHEAD) kz[(size_t)(16 * m + 4 * q + r) * a.P] = Z[m][r];
                Z[m] *= -kb[m];
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Pair zp = split2(Z[2 * s], Z[2 * s + 1]);
                if (QS == 1 && s == 1) read_kt(1);
#pragma unroll
                for (int n = 0; n < NT; ++n) D[n] = mma(D[n], kt[n][s], zp.lo);
#pragma unroll
                for (int n = 0; n < NT; ++n) D[n] = mma(D[n], kt[n][s], zp.hi);
            }
            lds_barrier();
        }
        if (nch & 1) lds_barrier();                  // the other waves go in pairs
        float* to = AHEAD ? io.split.loc + kofs : ba.g_init && sk == 0 ? ba.g_init + sofs : nullptr;
        if (to) {
#pragma unroll
            for (int n = 0; n < NT; ++n) *reinterpret_cast<float4*>(to + 32 * (n / 2) + 4 * (n % 2)) = f4(D[n]);
        }
        return;
    }
    // ---- staging: two chunks on their way; a step past the first chunk is that chunk again, rows past the sequence
    // read its last row and become zeros
    constexpr int NK = C * nc16 / 256, NTp = Bytes<false>::split / 4096;
    u32x4_t rk[2][NK], rq[2][NK], rd[2][2], rt[2][NTp], ra[2][NTp];
    float rs[2], rx[2];
    const unsigned char* kb = static_cast<const unsigned char*>(a.k) + (tok0 * a.k_stride + (size_t)g * N) * 2;
    const unsigned char* qb = static_cast<const unsigned char*>(a.q) + (tok0 * a.q_stride + (size_t)g * N) * 2;
    const unsigned char* db = static_cast<const unsigned char*>(ba.gy) + (tok0 * ba.gy_stride + (size_t)h * a.P + p0) * 2;
    const uint32_t k_row = (uint32_t)a.k_stride * 2, q_row = (uint32_t)a.q_stride * 2, d_row = (uint32_t)ba.gy_stride * 2;
    auto fetch = [&](int e, auto set) {
        constexpr int Z = decltype(set)::value;
        const int c = max(last - e, c0);
        const size_t u = (size_t)bh * io.nc + c;
        const int n_on = min(C, len - c * C);
        const unsigned char *kc = kb + (size_t)c * C * k_row, *qc = qb + (size_t)c * C * q_row, *dc = db + (size_t)c * C * d_row;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int x = tid + 256 * j, t = min(x / nc16, n_on - 1);
            rk[Z][j] = *reinterpret_cast<const u32x4_t*>(kc + ((uint32_t)t * k_row + x % nc16 * 16));
            rq[Z][j] = *reinterpret_cast<const u32x4_t*>(qc + ((uint32_t)t * q_row + x % nc16 * 16));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int x = tid + 256 * j, t = min(x / 8, n_on - 1);
            rd[Z][j] = *reinterpret_cast<const u32x4_t*>(dc + ((uint32_t)t * d_row + x % 8 * 16));
        }
#pragma unroll
        for (int j = 0; j < NTp; ++j) {
            rt[Z][j] = *reinterpret_cast<const u32x4_t*>(io.TT + u * Bytes<false>::split + (tid + 256 * j) * 16);
            ra[Z][j] = *reinterpret_cast<const u32x4_t*>(io.att + u * Bytes<false>::split + (tid + 256 * j) * 16);
        }
        rs[Z] = io.scal[u * kScalBwd * C + tid];
        rx[Z] = io.across[u];
    };
    auto stage = [&](int e, auto set) {
        constexpr int Z = decltype(set)::value;
        unsigned char* const lds = lds_all + (e & 1) * LD::buffer;
        const int n_on = len - max(last - e, c0) * C;
        const u32x4_t zero = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int x = tid + 256 * j, t = x / nc16, at = t * LD::kRow + row_piece<N>(t, x % nc16) * 16;
            *reinterpret_cast<u32x4_t*>(lds + LD::k + at) = t < n_on ? rk[Z][j] : zero;
            *reinterpret_cast<u32x4_t*>(lds + LD::q + at) = t < n_on ? rq[Z][j] : zero;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int x = tid + 256 * j, t = x / 8;
            *reinterpret_cast<u32x4_t*>(lds + LD::d + t * LD::dRow + x % 8 * 16) = t < n_on ? rd[Z][j] : zero;
        }
#pragma unroll
        for (int j = 0; j < NTp; ++j) {
            *reinterpret_cast<u32x4_t*>(lds + LD::tt + (tid + 256 * j) * 16) = rt[Z][j];
            *reinterpret_cast<u32x4_t*>(lds + LD::att + (tid + 256 * j) * 16) = ra[Z][j];
        }
        *reinterpret_cast<float*>(lds + LD::scal + tid * 4) = rs[Z];
        if (tid == 0) *reinterpret_cast<float*>(lds + LD::across) = rx[Z];
    };
    const std::integral_constant<int, 0> even;
    const std::integral_constant<int, 1> odd;
    if (nch > 0) {
        fetch(0, even);
        stage(0, even);
        fetch(1, odd);
        __builtin_amdgcn_sched_barrier(0);
        fetch(2, even);
    }
    lds_barrier();
    for (int e = 0; e < nch; e += 2) {
        stage(e + 1, odd);
        fetch(e + 3, odd);
        lds_barrier();
        stage(e + 2, even);
        fetch(e + 4, even);
        lds_barrier();
    }
}

// ---- fp32
template <int N>
struct RevLds {
    static constexpr int es = 4;
    static constexpr int kRow = N * es + 16, dRow = 64 * es + 16;
    static constexpr int k = 0, q = k + C * kRow, d = q + C * kRow, tt = d + C * dRow;
    static constexpr int att = tt + Bytes<true>::split, scal = att + Bytes<true>::split;
    static constexpr int bytes = scal + kScal * C * 4;
    static constexpr int buffers = 2 * bytes <= 160 * 1024 ? 2 : 1;
};

template <int N>
__global__ __launch_bounds__(256) void ssd_delta_reverse_kernel(DeltaBwdArgs ba, BwdIo io) {
    using LD = RevLds<N>;
    constexpr int NT = N / 16, es = LD::es, nc16 = N * es / 16, nv16 = 64 * es / 16;
    extern __shared__ __align__(16) unsigned char lds_all[];
    const DeltaArgs& a = ba.f;
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64, q = lane / 16, i = lane % 16;
    const int pb = a.P / 64;
    int unit = blockIdx.x;
    const int share = a.H / a.G * pb;                // heads of a group on one XCD
    if (a.B * a.G % 8 == 0) unit = (unit / 8 / share * 8 + unit % 8) * share + unit / 8 % share;
    const int p0 = unit % pb * 64, bh = unit / pb, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    const int len = row_len(a, b), nch = (len + C - 1) / C;
    const size_t tok0 = (size_t)b * a.L;
    const int p = p0 + 16 * wave + i;
    auto state_n = [&](int n) { return 16 * n + 4 * q; };
    const size_t sofs = ((size_t)bh * a.P + p) * N;
    f32x4 D[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
        D[n] = ba.g_final ? v4(*reinterpret_cast<const float4*>(ba.g_final + sofs + state_n(n))) : kZero4;

    constexpr int NK = C * nc16 / 256, NVp = C * nv16 / 256, NTp = (Bytes<true>::split / 16 + 255) / 256;
    u32x4_t rk[NK], rq[NK], rd[NVp], rt[NTp], ra[NTp];
    float rs = 0.0f, r_across = 0.0f;
    const unsigned char* kb = static_cast<const unsigned char*>(a.k) + (tok0 * a.k_stride + (size_t)g * N) * es;
    const unsigned char* qb = static_cast<const unsigned char*>(a.q) + (tok0 * a.q_stride + (size_t)g * N) * es;
    const unsigned char* db = static_cast<const unsigned char*>(ba.gy) + (tok0 * ba.gy_stride + (size_t)h * a.P + p0) * es;
    const uint32_t k_row = (uint32_t)a.k_stride * es, q_row = (uint32_t)a.q_stride * es, d_row = (uint32_t)ba.gy_stride * es;
    auto fetch = [&](int c) {
        const size_t u = (size_t)bh * io.nc + c;
        const int n_on = min(C, len - c * C);
        const unsigned char *kc = kb + (size_t)c * C * k_row, *qc = qb + (size_t)c * C * q_row, *dc = db + (size_t)c * C * d_row;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int e = tid + 256 * j, t = min(e / nc16, n_on - 1), x = e % nc16;
            rk[j] = *reinterpret_cast<const u32x4_t*>(kc + ((uint32_t)t * k_row + x * 16));
            rq[j] = *reinterpret_cast<const u32x4_t*>(qc + ((uint32_t)t * q_row + x * 16));
        }
#pragma unroll
        for (int j = 0; j < NVp; ++j) {
            const int e = tid + 256 * j, t = min(e / nv16, n_on - 1), x = e % nv16;
            rd[j] = *reinterpret_cast<const u32x4_t*>(dc + ((uint32_t)t * d_row + x * 16));
        }
#pragma unroll
        for (int j = 0; j < NTp; ++j) {
            const int e = min(tid + 256 * j, Bytes<true>::split / 16 - 1);
            rt[j] = *reinterpret_cast<const u32x4_t*>(io.TT + u * Bytes<true>::split + e * 16);
            ra[j] = *reinterpret_cast<const u32x4_t*>(io.att + u * Bytes<true>::split + e * 16);
        }
        rs = io.scal[u * kScalBwd * C + tid];
        r_across = io.across[u];
    };
    auto stage = [&](unsigned char* lds, int c) {
        const int n_on = len - c * C;
        const u32x4_t zero = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < NK; ++j) {
            const int e = tid + 256 * j, t = e / nc16, x = e % nc16;
            *reinterpret_cast<u32x4_t*>(lds + LD::k + t * LD::kRow + x * 16) = t < n_on ? rk[j] : zero;
            *reinterpret_cast<u32x4_t*>(lds + LD::q + t * LD::kRow + x * 16) = t < n_on ? rq[j] : zero;
        }
#pragma unroll
        for (int j = 0; j < NVp; ++j) {
            const int e = tid + 256 * j, t = e / nv16, x = e % nv16;
            *reinterpret_cast<u32x4_t*>(lds + LD::d + t * LD::dRow + x * 16) = t < n_on ? rd[j] : zero;
        }
#pragma unroll
        for (int j = 0; j < NTp; ++j)
            if (tid + 256 * j < Bytes<true>::split / 16) {
                *reinterpret_cast<u32x4_t*>(lds + LD::tt + (tid + 256 * j) * 16) = rt[j];
                *reinterpret_cast<u32x4_t*>(lds + LD::att + (tid + 256 * j) * 16) = ra[j];
            }
        *reinterpret_cast<float*>(lds + LD::scal + tid * 4) = rs;
    };
    float across = 0.0f;
    if (nch > 0) {
        fetch(nch - 1);
        stage(lds_all + (LD::buffers == 2 && (nch - 1) % 2 ? LD::bytes : 0), nch - 1);
        across = r_across;
        if (nch > 1) fetch(nch - 2);
        lds_barrier();
    }
    for (int c = nch - 1; c >= 0; --c) {
        unsigned char* const lds = lds_all + (LD::buffers == 2 && c % 2 ? LD::bytes : 0);
        auto scal4 = [&](int what, int m) {
            return v4(*reinterpret_cast<const float4*>(lds + LD::scal + (what * C + 16 * m + 4 * q) * 4));
        };
        auto frag16 = [&](int ofs) { return *reinterpret_cast<const uint4*>(lds + ofs + lane * 16); };
        const float keep = across;
        const size_t u = (size_t)bh * io.nc + c;
        f32x4 Z[4], W[4], Y[4];                      // dU then Z; dY times qin, and -beta kin Z
        {
            float* kd = io.D + u * N * a.P + p;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) kd[(size_t)(state_n(n) + r) * a.P] = D[n][r];
        }
        f32x4 d4[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                d4[m][r] = *reinterpret_cast<const float*>(lds + LD::d + (16 * m + 4 * q + r) * LD::dRow + (16 * wave + i) * 4);
            Y[m] = d4[m] * scal4(kQin, m);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            W[m] = kZero4;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                W[m] = mma_f32(W[m], *reinterpret_cast<const float4*>(lds + LD::k + (16 * m + i) * LD::kRow + (16 * n + 4 * q) * 4), f4(D[n]));
            W[m] *= scal4(kKout, m);
#pragma unroll
            for (int t = m; t < 4; ++t)
                W[m] = mma_f32(W[m], __builtin_bit_cast(float4, frag16(LD::att + tile_id(t, m) * 1024)), f4(d4[t]));
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            Z[m] = kZero4;
#pragma unroll
            for (int t = m; t < 4; ++t)
                Z[m] = mma_f32(Z[m], __builtin_bit_cast(float4, frag16(LD::tt + tile_id(t, m) * 1024)), f4(W[t]));
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) W[m] = -Z[m] * scal4(kKin, m) * scal4(kBeta, m);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            D[n] *= keep;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                auto col = [&](int base) {
                    const unsigned char* at = lds + base + (16 * m + 4 * q) * LD::kRow + (16 * n + i) * 4;
                    return make_float4(*reinterpret_cast<const float*>(at), *reinterpret_cast<const float*>(at + LD::kRow),
                                       *reinterpret_cast<const float*>(at + 2 * LD::kRow), *reinterpret_cast<const float*>(at + 3 * LD::kRow));
                };
                D[n] = mma_f32(D[n], col(LD::q), f4(Y[m]));
                D[n] = mma_f32(D[n], col(LD::k), f4(W[m]));
            }
        }
        if constexpr (LD::buffers == 1) lds_barrier();
        if (c > 0) {
            stage(lds_all + (LD::buffers == 2 && c % 2 == 0 ? LD::bytes : 0), c - 1);
            across = r_across;
            if (c > 1) fetch(c - 2);
        }
        float* kz = io.Z + u * C * a.P + p;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int r = 0; r < 4; ++r) kz[(size_t)(16 * m + 4 * q + r) * a.P] = Z[m][r];
        lds_barrier();
    }
    if (ba.g_init) {
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<float4*>(ba.g_init + sofs + state_n(n)) = f4(D[n]);
    }
}

// ============================================================ the gradients
// One workgroup a chunk and group; its heads in turn, dQ and dK of the group
// summed over them in registers, in order.  Wave w has the tokens 16 w .. +15
// as the columns of its tiles, so every token's scalars are one a lane, and
// products come out as [n][t] or [j][t]: W^T = S0 [n][p] x dY, Z, U [t][p], and
// dAtt^T, dL^T [j][t], whose tiles are again operands for dQ^T and dK^T of the
// wave's own tokens; the tiles that other waves' keys need go through LDS.
// U and the state are read once from memory by 16-row tiles, one wave each,
// and shared as fragments (P in halves of 64 columns, S0 and then dS in one
// buffer).
//
// bf16: states, U and Z enter as pairs, and the last products (of dAtt and dL
// with K and Q, whose results are rounded to bf16) with one rounding each.
// Measured, B=2 L=8192 H=32 G=8 P=N=64: 256 us (0.79 GB read and 0.14 GB
// written: 181 us at a copy's rate).  Loads are not ahead of their head (the
// registers are full), so it takes two workgroups a CU to hide them: at one,
// with 280 registers a wave, it took 415 us.
// The sums behind d(dt A), from a row's parts to dA and ddt_bias: fp32 inputs take all of them in fp64, where the terms on
// one side of a token cancel to 2^-47 of their magnitudes (dA and ddt_bias of four seeds at B=2 L=150 H=4 P=64 N=32: up to
// 1.3e-6 and 2.8e-6 off with the chunk's totals and the last sums in fp32, up to 3.5e-7 and 2.6e-7 this way); the products
// of bf16 inputs are off by more than fp32 sums.
template <typename T>
using Sum = std::conditional_t<std::is_same<T, float>::value, double, float>;

template <typename T, int N>
struct GradLds {
    static constexpr int es = sizeof(T);
    static constexpr int kRow = N * es + 16, gRow = C * es + 16;
    static constexpr int k = 0, q = k + C * kRow, s = q + C * kRow;
    static constexpr int s_bytes = std::max(N * 256, 2 * C * gRow);   // a half of S0 or dS; then the two [j][t] matrices
    static constexpr int u = s + s_bytes, scal = u + 16 * 1024;
    static constexpr int col = scal + kScalBwd * C * 4;               // [4][C] column sums
    static constexpr int row = col + 4 * C * sizeof(Sum<T>);          // [3][C]: dG's rows, its W3 part, dbeta
    static constexpr int dot = row + 3 * C * sizeof(Sum<T>);          // [4] <S0, dS>
    static constexpr int bytes = dot + 64;
};

// every lane has it
__device__ __forceinline__ float wave_sum(float v) { return lanes_sum<64>(v); }
__device__ __forceinline__ double of_halves(unsigned lo, unsigned hi) {
    return __longlong_as_double(((long long)(int)hi << 32) | lo);
}
template <int CTRL>
__device__ __forceinline__ double dpp_plus64(double v) {
    const long long b = __double_as_longlong(v);
    return v + of_halves(__builtin_amdgcn_update_dpp(0, (int)b, CTRL, 0xF, 0xF, true),
                         __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ double wave_sum(double v) {   // the moves of lanes_sum, on both halves
    v = dpp_plus64<0xB1>(v);
    v = dpp_plus64<0x4E>(v);
    v = dpp_plus64<0x141>(v);
    v = dpp_plus64<0x140>(v);
    long long b = __double_as_longlong(v);
    auto lo = __builtin_amdgcn_permlane16_swap((unsigned)b, (unsigned)b, false, false);
    auto hi = __builtin_amdgcn_permlane16_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
    v = of_halves(lo[0], hi[0]) + of_halves(lo[1], hi[1]);
    b = __double_as_longlong(v);
    lo = __builtin_amdgcn_permlane32_swap((unsigned)b, (unsigned)b, false, false);
    hi = __builtin_amdgcn_permlane32_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
    return of_halves(lo[0], hi[0]) + of_halves(lo[1], hi[1]);
}
__device__ __forceinline__ float shfl_down(float v, int d) { return __shfl_down(v, d); }
__device__ __forceinline__ double shfl_down(double v, int d) {
    const long long b = __double_as_longlong(v);
    return __longlong_as_double(((long long)__shfl_down((int)(b >> 32), d) << 32) | (unsigned)__shfl_down((int)b, d));
}
// over 16 lanes (the first has it), and over the four rows of 16
__device__ __forceinline__ float sum16(float v) { return lanes_sum<16>(v); }
__device__ __forceinline__ double sum16(double v) {
#pragma unroll
    for (int d = 8; d > 0; d /= 2) v += shfl_down(v, d);
    return v;
}
__device__ __forceinline__ float sum_rows(float v) { return rows_sum(v); }
__device__ __forceinline__ double sum_rows(double v) {
    v += shfl_down(v, 32);
    return v + shfl_down(v, 16);     // the first row has it
}

// four consecutive entries of a row, and their store
__device__ __forceinline__ f32x4 ld4t(const unsigned char* p, uint16_t) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return f32x4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
}
__device__ __forceinline__ f32x4 ld4t(const unsigned char* p, float) { return v4(*reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ void st4t(uint16_t* p, f32x4 v) { *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])); }
__device__ __forceinline__ void st4t(float* p, f32x4 v) { *reinterpret_cast<float4*>(p) = f4(v); }
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) { return fmaf(a[3], b[3], fmaf(a[2], b[2], fmaf(a[1], b[1], a[0] * b[0]))); }

// the sum over 8 entries of z * v
__device__ __forceinline__ float dot8(const float4& a, const float4& b, const Rows<float>& v) {
    return a.x * v.a.x + a.y * v.a.y + a.z * v.a.z + a.w * v.a.w + b.x * v.b.x + b.y * v.b.y + b.z * v.b.z + b.w * v.b.w;
}
__device__ __forceinline__ float dot8(const float4& a, const float4& b, const Rows<uint16_t>& v) {
    const uint32_t* w = v.f.w;
    return a.x * bf16_lo(w[0]) + a.y * bf16_hi(w[0]) + a.z * bf16_lo(w[1]) + a.w * bf16_hi(w[1]) + b.x * bf16_lo(w[2]) +
           b.y * bf16_hi(w[2]) + b.z * bf16_lo(w[3]) + b.w * bf16_hi(w[3]);
}

// two [j][t] tiles (K blocks of 16) as an operand of the last products, rounded to bf16 there: its outputs are bf16
template <typename T>
struct Last;
template <>
struct Last<uint16_t> {
    Frag f;
    __device__ __forceinline__ void set(f32x4 a, f32x4 b) { f = round2(a, b); }
    // row j of a [j][t] matrix, K blocks 2 s and 2 s + 1
    __device__ __forceinline__ void row(const unsigned char* p, int s, int q) {
        const FragBF x = plain_read(p + (32 * s + 4 * q) * 2), y = plain_read(p + (32 * s + 16 + 4 * q) * 2);
        f.w[0] = x.a; f.w[1] = x.b; f.w[2] = y.a; f.w[3] = y.b;
    }
    // column n of rows t of k or q: the transposed operand [n][t], 16-row tile at column n0
    __device__ __forceinline__ void tr(const unsigned char* base, int ofs, int row_bytes, int s, int n0, int q, int i) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const FragBF x = tr_read(base, ofs + (32 * s + 16 * e + 4 * q + i / 4) * row_bytes + (n0 + 4 * (i % 4)) * 2);
            f.w[2 * e] = x.a;
            f.w[2 * e + 1] = x.b;
        }
    }
    static __device__ __forceinline__ f32x4 mul(f32x4 acc, const Last& a, const Last& b) { return mma(acc, a.f, b.f); }
};
template <>
struct Last<float> {
    float4 a, b;
    __device__ __forceinline__ void set(f32x4 x, f32x4 y) { a = f4(x); b = f4(y); }
    __device__ __forceinline__ void row(const unsigned char* p, int s, int q) {
        a = *reinterpret_cast<const float4*>(p + (32 * s + 4 * q) * 4);
        b = *reinterpret_cast<const float4*>(p + (32 * s + 16 + 4 * q) * 4);
    }
    __device__ __forceinline__ void tr(const unsigned char* base, int ofs, int row_bytes, int s, int n0, int q, int i) {
        const unsigned char* p = base + ofs + (32 * s + 4 * q) * row_bytes + (n0 + i) * 4;
        auto at = [&](int t) { return *reinterpret_cast<const float*>(p + t * row_bytes); };
        a = make_float4(at(0), at(1), at(2), at(3));
        b = make_float4(at(16), at(17), at(18), at(19));
    }
    static __device__ __forceinline__ f32x4 mul(f32x4 acc, const Last& x, const Last& y) { return mma_f32(mma_f32(acc, x.a, y.a), x.b, y.b); }
};

// two workgroups a CU where a wave's registers allow it (fp32 N = 32: 242)
template <typename T, int N>
__global__ __launch_bounds__(256, N <= (sizeof(T) == 2 ? 64 : 32) ? 2 : 1) void ssd_delta_grad_kernel(DeltaBwdArgs ba, BwdIo io) {
    using LD = GradLds<T, N>;
    constexpr int NT = N / 16, KS = N / 32, es = LD::es, nc16 = N * es / 16;
    constexpr bool kLate = es == 4 && N == 128;      // dS only when S0 has been used: registers
    extern __shared__ __align__(16) unsigned char lds[];
    const DeltaArgs& a = ba.f;
    const int tid = threadIdx.x, lane = tid % 64, q = lane / 16, i = lane % 16;
    const int w = __builtin_amdgcn_readfirstlane(tid / 64);
    const int g = blockIdx.x % a.G, c = blockIdx.x / a.G % io.nc, b = blockIdx.x / a.G / io.nc;
    const int hg = a.H / a.G, t0 = c * C, n_on = min(C, row_len(a, b) - t0), n_rows = min(C, a.L - t0);
    const size_t tok0 = (size_t)b * a.L + t0;
    const size_t bc = (size_t)b * io.nc + c, parts = (size_t)a.B * io.nc * a.H;
    using SumT = Sum<T>;
    SumT* part = static_cast<SumT*>(io.part);
    T* dq = static_cast<T*>(ba.dq) + tok0 * ba.dq_stride + (size_t)g * N;
    T* dk = static_cast<T*>(ba.dk) + tok0 * ba.dk_stride + (size_t)g * N;
    T* dv = static_cast<T*>(ba.dv) + tok0 * ba.dv_stride + (size_t)g * hg * a.P;
    if (n_on <= 0) {                                 // nothing real in the chunk: zero gradients
        for (int e = tid; e < n_rows * N / 4; e += 256) {
            st4t(dq + (size_t)(e / (N / 4)) * ba.dq_stride + e % (N / 4) * 4, kZero4);
            st4t(dk + (size_t)(e / (N / 4)) * ba.dk_stride + e % (N / 4) * 4, kZero4);
        }
        const int wide = hg * a.P / 4;
        for (int e = tid; e < n_rows * wide; e += 256) st4t(dv + (size_t)(e / wide) * ba.dv_stride + e % wide * 4, kZero4);
        for (int e = tid; e < n_rows * hg; e += 256) {
            ba.ddt[(tok0 + e / hg) * ba.ddt_stride + g * hg + e % hg] = 0.0f;
            ba.dbeta[(tok0 + e / hg) * ba.dbeta_stride + g * hg + e % hg] = 0.0f;
        }
        for (int e = tid; e < hg; e += 256) part[bc * a.H + g * hg + e] = part[parts + bc * a.H + g * hg + e] = 0;
        return;
    }
    // ---- k and q of the chunk
    {
        const unsigned char* kc = static_cast<const unsigned char*>(a.k) + (tok0 * a.k_stride + (size_t)g * N) * es;
        const unsigned char* qc = static_cast<const unsigned char*>(a.q) + (tok0 * a.q_stride + (size_t)g * N) * es;
        const u32x4_t zero = {0, 0, 0, 0};
        for (int e = tid; e < C * nc16; e += 256) {
            const int t = e / nc16, x = e % nc16, r = min(t, n_on - 1);
            const u32x4_t vk = *reinterpret_cast<const u32x4_t*>(kc + (size_t)r * a.k_stride * es + x * 16);
            const u32x4_t vq = *reinterpret_cast<const u32x4_t*>(qc + (size_t)r * a.q_stride * es + x * 16);
            *reinterpret_cast<u32x4_t*>(lds + LD::k + t * LD::kRow + x * 16) = t < n_on ? vk : zero;
            *reinterpret_cast<u32x4_t*>(lds + LD::q + t * LD::kRow + x * 16) = t < n_on ? vq : zero;
        }
    }
    const int t = 16 * w + i;                        // this lane's token
    const bool on = t < n_on;
    const uint32_t row = min(t, n_on - 1);           // offsets within a chunk fit 32 bits
    f32x4 dQ[NT], dK[NT];                            // [n][t]
#pragma unroll
    for (int n = 0; n < NT; ++n) dQ[n] = dK[n] = kZero4;
    SumT* colp = reinterpret_cast<SumT*>(lds + LD::col);
    SumT* rowp = reinterpret_cast<SumT*>(lds + LD::row);
    SumT* dotp = reinterpret_cast<SumT*>(lds + LD::dot);

    for (int hh = 0; hh < hg; ++hh) {
        const int h = g * hg + hh;
        const size_t u = ((size_t)b * a.H + h) * io.nc + c;
        for (int e = tid; e < kScalBwd * C; e += 256) *reinterpret_cast<float*>(lds + LD::scal + e * 4) = io.scal[u * kScalBwd * C + e];
        const float beta = io.scal[(u * kScalBwd + kBeta) * C + t];
        f32x4 W1[NT], W2[NT], W3[NT], EA[4], EL[4];
#pragma unroll
        for (int n = 0; n < NT; ++n) W1[n] = W2[n] = W3[n] = kZero4;
#pragma unroll
        for (int n = 0; n < 4; ++n) EA[n] = EL[n] = kZero4;
        float zv = 0.0f;
        SumT sd = 0.0f;
        for (int p0 = 0; p0 < a.P; p0 += 64) {
            // the wave's own rows t: dY, Z, U as operands; dV; U's tile for everyone
            Rows<T> dy[2];
            Wide<T> z[2], ds[(NT + 3) / 4][2];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const uint32_t col = p0 + 32 * s + 8 * q;
                Rows<T> v;
                dy[s].load(static_cast<const T*>(ba.gy) + tok0 * ba.gy_stride + (size_t)h * a.P + (row * (uint32_t)ba.gy_stride + col));
                v.load(static_cast<const T*>(a.v) + tok0 * a.v_stride + (size_t)h * a.P + (row * (uint32_t)a.v_stride + col));
                if (!on) {
                    dy[s].clear();
                    v.clear();
                }
                const float* zp = io.Z + u * C * a.P + ((uint32_t)t * a.P + col);
                const float* up = io.U + u * C * a.P + ((uint32_t)t * a.P + col);
                const float4 z0 = *reinterpret_cast<const float4*>(zp), z1 = *reinterpret_cast<const float4*>(zp + 4);
                z[s].set(z0, z1);
                Wide<T> f;
                f.set(*reinterpret_cast<const float4*>(up), *reinterpret_cast<const float4*>(up + 4));
                f.put(lds + LD::u + (w * 2 + s) * 2048 + lane * 16);
                zv += dot8(z0, z1, v);
                if (t < n_rows) {
                    T* dst = dv + (size_t)hh * a.P + ((uint32_t)t * (uint32_t)ba.dv_stride + col);
                    st4t(dst, v4(z0) * beta);
                    st4t(dst + 4, v4(z1) * beta);
                }
            }
#pragma unroll
            for (int j = 0; j < (NT + 3) / 4; ++j) {
                const int n = w + 4 * j;
                if (n < NT) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t at = (uint32_t)(16 * n + i) * a.P + p0 + 32 * s + 8 * q;
                        const float *sp = io.S + u * N * a.P + at, *dp = io.D + u * N * a.P + at;
                        const float4 s0 = *reinterpret_cast<const float4*>(sp), s1 = *reinterpret_cast<const float4*>(sp + 4);
                        if constexpr (!kLate) {
                            const float4 d0 = *reinterpret_cast<const float4*>(dp), d1 = *reinterpret_cast<const float4*>(dp + 4);
                            sd += dot4(v4(s0), v4(d0)) + dot4(v4(s1), v4(d1));
                            ds[j][s].set(d0, d1);
                        }
                        Wide<T> f;
                        f.set(s0, s1);
                        f.put(lds + LD::s + (n * 2 + s) * 2048 + lane * 16);
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                if (n > w) continue;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    Wide<T> f;
                    f.get(lds + LD::u + (n * 2 + s) * 2048 + lane * 16);
                    EA[n] = Wide<T>::mul(EA[n], f, dy[s]);
                    EL[n] = Wide<T>::mul(EL[n], f, z[s]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    Wide<T> f;
                    f.get(lds + LD::s + (n * 2 + s) * 2048 + lane * 16);
                    W1[n] = Wide<T>::mul(W1[n], f, dy[s]);
                    W2[n] = Wide<T>::mul(W2[n], f, z[s]);
                }
            __syncthreads();
            float late = 0.0f;                       // kLate: 32 products of <S0, dS>
#pragma unroll
            for (int j = 0; j < (NT + 3) / 4; ++j) {
                const int n = w + 4 * j;
                if (n < NT) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        unsigned char* to = lds + LD::s + (n * 2 + s) * 2048 + lane * 16;
                        if constexpr (kLate) {
                            const float* dp = io.D + u * N * a.P + (uint32_t)(16 * n + i) * a.P + p0 + 32 * s + 8 * q;
                            const float4 d0 = *reinterpret_cast<const float4*>(dp), d1 = *reinterpret_cast<const float4*>(dp + 4);
                            Wide<T> f;
                            f.get(to);
                            late += dot4(v4(f.p.a), v4(d0)) + dot4(v4(f.p.b), v4(d1));
                            ds[j][s].set(d0, d1);
                        }
                        ds[j][s].put(to);
                    }
                }
            }
            if constexpr (kLate) {                   // not held over the products, for the registers' sake
                const SumT all = wave_sum((SumT)late);
                if (lane == 0) dotp[w] = p0 == 0 ? all : dotp[w] + all;
            }
            __syncthreads();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                Wide<T> own;
                own.get(lds + LD::u + (w * 2 + s) * 2048 + lane * 16);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    Wide<T> f;
                    f.get(lds + LD::s + (n * 2 + s) * 2048 + lane * 16);
                    W3[n] = Wide<T>::mul(W3[n], f, own);
                }
            }
            __syncthreads();
        }
        auto sc1 = [&](int what) { return *reinterpret_cast<const float*>(lds + LD::scal + (what * C + t) * 4); };
        auto sc4 = [&](int what, int n) { return v4(*reinterpret_cast<const float4*>(lds + LD::scal + (what * C + 16 * n + 4 * q) * 4)); };
        const float kin = sc1(kKin), kout = sc1(kKout), qin = sc1(kQin), rk = sc1(kSRk), rq = sc1(kSRq);
        const float th = sc1(kSGhi), tl = sc1(kSGlo), ts = sc1(kSSeg);
        // ---- the state's parts, and their row products
        float r1 = 0.0f, r2 = 0.0f, r3 = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const f32x4 k4 = ld4t(lds + LD::k + t * LD::kRow + (16 * n + 4 * q) * es, T()), q4 = ld4t(lds + LD::q + t * LD::kRow + (16 * n + 4 * q) * es, T());
            W1[n] *= qin;
            W2[n] *= kin;
            W3[n] *= kout;
            r1 += dot4(W1[n], q4);
            r2 += dot4(W2[n], k4);
            r3 += dot4(W3[n], k4);
            dQ[n] += W1[n];
            dK[n] += W3[n] - beta * W2[n];
        }
        // ---- the chunk's own pairs: [j][t], j = 16 n + 4 q + r <= t
        Rows<T> ko[KS], qo[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            ko[s].load(reinterpret_cast<const T*>(lds + LD::k + t * LD::kRow) + 32 * s + 8 * q);
            qo[s].load(reinterpret_cast<const T*>(lds + LD::q + t * LD::kRow) + 32 * s + 8 * q);
        }
        SumT rsum = 0.0f;
        float bsum = 0.0f;
        unsigned char *g1 = lds + LD::s, *g2 = g1 + C * LD::gRow;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            f32x4 x1 = kZero4, x2 = kZero4, cs = kZero4;
            if (n <= w) {
                f32x4 kk = kZero4, qk = kZero4;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    Rows<T> kf;
                    kf.load(reinterpret_cast<const T*>(lds + LD::k + (16 * n + i) * LD::kRow) + 32 * s + 8 * q);
                    kk = Rows<T>::mul(kk, kf, ko[s]);
                    qk = Rows<T>::mul(qk, kf, qo[s]);
                }
                const f32x4 h4 = sc4(kSGhi, n), l4 = sc4(kSGlo, n), s4 = sc4(kSSeg, n), rk4 = sc4(kSRk, n);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 16 * n + 4 * q + r;
                    const float m = fast_exp2(s4[r] == ts && j <= t ? (th - h4[r]) + (tl - l4[r]) : -INFINITY) * rk4[r];
                    const bool before = j < t;
                    x1[r] = EA[n][r] * (m * rq);
                    x2[r] = before ? -EL[n][r] * (m * rk) : 0.0f;   // without beta
                    const float ea = before ? x1[r] * qk[r] : 0.0f, el = x2[r] * kk[r];
                    bsum += el;
                    cs[r] = fmaf(beta, el, ea);
                    rsum += cs[r];
                    x2[r] *= beta;
                }
            }
            EA[n] = x1;
            EL[n] = x2;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = 16 * n + 4 * q + r;
                const SumT all = sum16((SumT)cs[r]);
                if (i == 0) colp[w * C + j] = all;
                if constexpr (es == 2) {
                    *reinterpret_cast<uint16_t*>(g1 + j * LD::gRow + t * 2) = (uint16_t)f32_to_bf16_bits(x1[r]);
                    *reinterpret_cast<uint16_t*>(g2 + j * LD::gRow + t * 2) = (uint16_t)f32_to_bf16_bits(x2[r]);
                } else {
                    *reinterpret_cast<float*>(g1 + j * LD::gRow + t * 4) = x1[r];
                    *reinterpret_cast<float*>(g2 + j * LD::gRow + t * 4) = x2[r];
                }
            }
        }
        {
            float all[5] = {r1, r2, r3, bsum, zv};
#pragma unroll
            for (int x = 0; x < 5; ++x) all[x] = rows_sum(all[x]);
            rsum = sum_rows(rsum);
            if constexpr (!kLate) sd = wave_sum(sd);
            if (q == 0) {
                rowp[t] = rsum + all[0] - (SumT)beta * all[1] - all[2];
                rowp[C + t] = all[2];
                rowp[2 * C + t] = all[4] - all[1] + all[3];
            }
            if (!kLate && lane == 0) dotp[w] = sd;
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            Last<T> own1, own2, far1, far2;
            own1.set(EA[2 * s], EA[2 * s + 1]);      // queries and keys of this wave's tokens: K index j
            own2.set(EL[2 * s], EL[2 * s + 1]);
            far1.row(g1 + t * LD::gRow, s, q);       // this wave's tokens as keys j: K index t
            far2.row(g2 + t * LD::gRow, s, q);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                Last<T> kt, qt;
                kt.tr(lds, LD::k, LD::kRow, s, 16 * n, q, i);
                qt.tr(lds, LD::q, LD::kRow, s, 16 * n, q, i);
                dQ[n] = Last<T>::mul(dQ[n], kt, own1);
                dK[n] = Last<T>::mul(dK[n], kt, own2);
                dK[n] = Last<T>::mul(dK[n], qt, far1);
                dK[n] = Last<T>::mul(dK[n], kt, far2);
            }
        }
        if (w == 0) {
            // one token a lane: d(dt A) is the sum of dG behind it
            SumT dG = rowp[lane] - ((colp[lane] + colp[C + lane]) + (colp[2 * C + lane] + colp[3 * C + lane]));
            const SumT r3s = wave_sum(rowp[C + lane]), dot = (dotp[0] + dotp[1]) + (dotp[2] + dotp[3]);
            if (lane == 63) dG += fma((SumT)io.across[u], dot, r3s);
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const SumT dn = shfl_down(dG, d);
                if (lane + d < 64) dG += dn;
            }
            const size_t at = tok0 + min(lane, n_on - 1);
            float dt = a.dt[at * a.dt_stride + h], chain = 1.0f;
            const float be = *reinterpret_cast<const float*>(lds + LD::scal + (kBeta * C + lane) * 4);
            float db = (float)rowp[2 * C + lane];
            if (a.dt_softplus) {
                dt += a.dt_bias ? a.dt_bias[h] : 0.0f;
                chain = 1.0f / (1.0f + expf(-dt));
                dt = softplus_f(dt);
            }
            if (a.beta_sigmoid) db *= be * (1.0f - be);
            // Every pair across t carries the factor exp(dt A): below e^-30 the true sum is far under the rounding
            // that the row and column sums leave behind (2^-24 of them), which a large dt would carry into dA.
            if (dt * a.A[h] < -30.0f) dG = 0.0f;
            // Nothing passes into a document's first token, nor into a row's that has no state before it: exactly 0.
            const float* seg = reinterpret_cast<const float*>(lds + LD::scal) + kSSeg * C;
            const bool none = seg[lane] != (lane ? seg[lane - 1] : 0.0f) || (t0 + lane == 0 && !a.init_state);
            if (none) dG = 0.0f;
            const bool live = lane < n_on;
            const float dd = live ? (float)dG * a.A[h] * chain : 0.0f;
            if (lane < n_rows) {
                ba.ddt[(tok0 + lane) * ba.ddt_stride + h] = dd;
                ba.dbeta[(tok0 + lane) * ba.dbeta_stride + h] = live ? db : 0.0f;
            }
            const SumT pa = wave_sum(live && dG != 0.0f ? dG * dt : SumT(0)), pd = wave_sum((SumT)dd);   // dt may be infinite
            if (lane == 0) {
                part[bc * a.H + h] = pa;
                part[parts + bc * a.H + h] = pd;
            }
        }
        __syncthreads();
    }
    // ---- through the norms, and out
    float sq = 0.0f, sk = 0.0f, dotq = 0.0f, dotk = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const f32x4 k4 = ld4t(lds + LD::k + t * LD::kRow + (16 * n + 4 * q) * es, T()), q4 = ld4t(lds + LD::q + t * LD::kRow + (16 * n + 4 * q) * es, T());
        sq += dot4(q4, q4);
        sk += dot4(k4, k4);
        dotq += dot4(q4, dQ[n]);
        dotk += dot4(k4, dK[n]);
    }
    const float fq = a.qk_norm ? rows_sum(dotq) / (rows_sum(sq) + kQkEps) : 0.0f;
    const float fk = a.qk_norm ? rows_sum(dotk) / (rows_sum(sk) + kQkEps) : 0.0f;
    if (t < n_rows) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const f32x4 k4 = ld4t(lds + LD::k + t * LD::kRow + (16 * n + 4 * q) * es, T()), q4 = ld4t(lds + LD::q + t * LD::kRow + (16 * n + 4 * q) * es, T());
            st4t(dq + (size_t)t * ba.dq_stride + 16 * n + 4 * q, dQ[n] - fq * q4);
            st4t(dk + (size_t)t * ba.dk_stride + 16 * n + 4 * q, dK[n] - fk * k4);
        }
    }
}

// dA and ddt_bias: the chunks' parts of a head, added in a fixed order
template <typename S>
__global__ __launch_bounds__(256) void ssd_delta_sum_kernel(const S* part, size_t rows, int H, float* dA, float* ddt_bias) {
    __shared__ S s[256];
    const int h = blockIdx.x % H, k = blockIdx.x / H;
    S v = 0.0f;
    for (size_t r = threadIdx.x; r < rows; r += 256) v += part[(k * rows + r) * H + h];
    s[threadIdx.x] = v;
    __syncthreads();
#pragma unroll
    for (int d = 128; d > 0; d /= 2) {
        if (threadIdx.x < d) s[threadIdx.x] += s[threadIdx.x + d];
        __syncthreads();
    }
    float* out = k ? ddt_bias : dA;
    if (threadIdx.x == 0 && out) out[h] = (float)s[0];
}

struct BwdWs {
    size_t T, TT, att, scal, across, S, U, D, Z, part, loc, phi, s0, total;
    Split split;
};
BwdWs bwd_ws(int B, int L, int H, int P, int N, int dtype) {
    const size_t nc = (L + C - 1) / C, units = (size_t)B * H * nc;
    const size_t split = dtype == 0 ? Bytes<true>::split : Bytes<false>::split;
    BwdWs w;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t o = at;
        at += (n + 255) / 256 * 256;
        return o;
    };
    w.T = take(units * split);
    w.TT = take(units * split);
    w.att = take(units * split);
    w.scal = take(units * kScalBwd * C * 4);
    w.across = take(units * 4);
    w.S = take(units * N * P * 4);
    w.U = take(units * C * P * 4);
    w.D = take(units * N * P * 4);
    w.Z = take(units * C * P * 4);
    w.part = take(2 * units * (dtype == 0 ? sizeof(Sum<float>) : sizeof(Sum<uint16_t>)));
    split_bwd(B, L, H, P, N, dtype, w.split);
    const size_t states = w.split.K > 1 ? (size_t)B * H * w.split.K * N * 4 : 0;
    w.loc = take(states * P);
    w.phi = take(states * N);
    w.s0 = take(states * P);
    w.total = at;
    return w;
}

template <typename T, int N>
hipError_t launch_bwd_n(const DeltaBwdArgs& ba, void* ws, hipStream_t stream) {
    const DeltaArgs& a = ba.f;
    const int nc = (a.L + C - 1) / C;
    const BwdWs w = bwd_ws(a.B, a.L, a.H, a.P, N, a.dtype);
    unsigned char* base = static_cast<unsigned char*>(ws);
    auto fp = [&](size_t o) { return reinterpret_cast<float*>(base + o); };
    PrepOut o{base + w.T, base + w.TT, base + w.att, fp(w.scal), fp(w.across)};
    const Split split{w.split.K, w.split.S, fp(w.loc), fp(w.phi), fp(w.s0)};
    hipError_t e = launch_keep(a, o, KeepOut{fp(w.S), fp(w.U), split}, stream);
    if (e != hipSuccess) return e;
    BwdIo io{o.TT, o.att, o.scal, o.across, fp(w.S), fp(w.U), fp(w.D), fp(w.Z), base + w.part, nc, split};
    constexpr size_t grad = GradLds<T, N>::bytes;
    const dim3 chains(a.B * a.H * (a.P / 64));
    if constexpr (std::is_same<T, float>::value) {
        constexpr size_t rev = (size_t)RevLds<N>::bytes * RevLds<N>::buffers;
        e = prepare_launch(reinterpret_cast<const void*>(&ssd_delta_reverse_kernel<N>), rev);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((ssd_delta_reverse_kernel<N>), chains, dim3(256), rev, stream, ba, io);
    } else {
        constexpr size_t rev = 2 * BackLds<N>::buffer;
        if (split.K > 1) {
            e = prepare_launch(reinterpret_cast<const void*>(&ssd_delta_back_kernel<N, true>), rev);
            if (e != hipSuccess) return e;
            hipLaunchKernelGGL((ssd_delta_back_kernel<N, true>), dim3(chains.x * (split.K - 1)), dim3(512), rev, stream, ba, io);
            e = hipGetLastError();
            if (e != hipSuccess) return e;
            e = launch_join_back(a, split, ba.g_final, stream);
            if (e != hipSuccess) return e;
        }
        e = prepare_launch(reinterpret_cast<const void*>(&ssd_delta_back_kernel<N, false>), rev);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((ssd_delta_back_kernel<N, false>), dim3(chains.x * split.K), dim3(512), rev, stream, ba, io);
    }
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    e = prepare_launch(reinterpret_cast<const void*>(&ssd_delta_grad_kernel<T, N>), grad);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ssd_delta_grad_kernel<T, N>), dim3((unsigned)((size_t)a.B * nc * a.G)), dim3(256), grad, stream, ba, io);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ssd_delta_sum_kernel<Sum<T>>), dim3(2 * a.H), dim3(256), 0, stream, static_cast<const Sum<T>*>(io.part), (size_t)a.B * nc, a.H, ba.dA, ba.ddt_bias);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_bwd_t(const DeltaBwdArgs& a, void* ws, hipStream_t stream) {
    switch (a.f.N) {
        case 32: return launch_bwd_n<T, 32>(a, ws, stream);
        case 64: return launch_bwd_n<T, 64>(a, ws, stream);
        case 128: return launch_bwd_n<T, 128>(a, ws, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace

size_t delta_bwd_workspace_bytes(int B, int L, int H, int P, int N, int dtype) { return bwd_ws(B, L, H, P, N, dtype).total; }

hipError_t launch_delta_bwd(const DeltaBwdArgs& a, void* ws, hipStream_t stream) {
    return a.f.dtype == 0 ? launch_bwd_t<float>(a, ws, stream) : launch_bwd_t<uint16_t>(a, ws, stream);
}

}  // namespace ssd
