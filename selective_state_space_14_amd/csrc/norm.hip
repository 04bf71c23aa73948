// norm.hip -- the row norm that ends a mixer, forward and backward.
//
//   layer: xhat = (x - mean(x)) * rstd,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)
//   rms:   xhat = x * rstd,              rstd = 1 / sqrt(mean(x^2) + eps)
//   y = (xhat * w + b) * silu(z)         (w, b and the gate z optional)
// and with g = dy * silu(z):
//   dw = sum_rows g xhat,  db = sum_rows g,  dz = dy (xhat w + b) silu'(z)
//   dx = rstd (g w - mean(g w) - xhat mean(g w xhat))      (rms: no mean(g w))
//
// Both passes are bound by HBM: every operand is read once and every result
// written once, the row staying in registers between the statistics (two
// passes over the registers, so a large mean costs no digits) and the output.
// A row belongs to TPR threads, each holding NV vectors of VEC elements; TPR
// is a part of a wave for short rows (several rows a wave), one wave, or a
// workgroup.  VEC is 8 where every row starts on a 16-byte boundary and W is
// a multiple of 8, else 1.  Workgroups walk the rows with w and b in
// registers; the backward also keeps its columns' dw and db there, adds a
// workgroup's rows up in LDS, and a second launch adds the workgroups' sums
// in their order, so results do not change from run to run.
//
// Measured: 40960 rows of 2048, fp32 to bf16, 91 us (5.5 TB/s; a large copy
// reaches 5.1); 1.3 million gated rows of 64 in bf16, 98 us (5.1 TB/s); the
// gated backward of 40960 rows of 2048 in bf16, 172 us and 5 us of sums
// (4.9 TB/s), 200 us before it loaded the next row's operands a row ahead.
// The threads of a row: at 2048 columns a wave of four vectors a thread takes
// 91 us forward and 256 threads of one 99, while backward, with more live a
// column, they take 201 and 172; rows of 64 take 98 us with eight threads each
// and 428 with a wave each.  Loads that go past the last-level cache take 84 us
// in place of 91 where the same 336 MB are read call after call, but 96 where
// the inputs are new.
#include <hip/hip_runtime.h>
#include <algorithm>

#include "ssd_device.hpp"
#include "ssd_launch.hpp"

namespace ssd {
namespace {

// ------------------------------------------------------------ vectors of a row
template <int VEC>
__device__ __forceinline__ void ldv(const float* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        v[0] = *p;
    }
}
template <int VEC>
__device__ __forceinline__ void ldv(const uint16_t* p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
        v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
    } else {
        v[0] = bf16_to_f32(*p);
    }
}
template <int VEC>
__device__ __forceinline__ void stv(float* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *p = v[0];
    }
}
template <int VEC>
__device__ __forceinline__ void stv(uint16_t* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
        *p = (uint16_t)f32_to_bf16_bits(v[0]);
    }
}

// A vector as it is in memory: loaded a row ahead, widened when its row comes.
template <typename T, int VEC>
struct Raw {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void clear() { v = 0; }
    __device__ __forceinline__ void get(float (&o)[VEC]) const { ldv<VEC>(&v, o); }
};
template <>
struct Raw<uint16_t, 8> {
    u32x4_t v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const u32x4_t*>(p); }
    __device__ __forceinline__ void clear() { v = u32x4_t{0, 0, 0, 0}; }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = bf16_lo(v[i]);
            o[2 * i + 1] = bf16_hi(v[i]);
        }
    }
};
template <>
struct Raw<float, 8> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const f32x4*>(p);
        b = *reinterpret_cast<const f32x4*>(p + 4);
    }
    __device__ __forceinline__ void clear() { a = b = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; }
    __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[i] = a[i];
            o[4 + i] = b[i];
        }
    }
};

// ------------------------------------------------------------ sums over a row's threads
// two sums at once; over a workgroup they meet in `red`, whose two halves are
// used in turn, so one barrier a call is enough: a wave reads its half before
// it comes to the next call's barrier, behind which the half is written again
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float (*red)[2][16], int& turn) {
    a = lanes_sum<(TPR > 64 ? 64 : TPR)>(a);
    b = lanes_sum<(TPR > 64 ? 64 : TPR)>(b);
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x / 64;
        if (threadIdx.x % 64 == 0) {
            red[turn][0][wave] = a;
            red[turn][1][wave] = b;
        }
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) {
            a += red[turn][0][i];
            b += red[turn][1][i];
        }
        turn ^= 1;
    }
}

template <int TPR, int NV, int VEC>
struct Shape {
    static constexpr int threads = TPR > 256 ? TPR : 256;
    static constexpr int rows = threads / TPR;      // rows of a workgroup at a time
};

// mean (0 for rms) and rstd of the row in x; x becomes xhat.  Threads without a
// row (not live) hold zeros: their rstd is 0, since with eps = 0 it would be
// infinite and their xhat, which enters the weights' sums, NaN
template <int TPR, int NV, int VEC>
__device__ __forceinline__ float to_hat(float (&x)[NV][VEC], const bool (&on)[NV], bool live, int W, int rms, float eps,
                                        float (*red)[2][16], int& turn) {
    const float inv = 1.0f / (float)W;
    float s = 0.0f, unused = 0.0f;
    if (!rms) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += x[j][e];
        row_sum2<TPR>(s, unused, red, turn);
        const float mean = s * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[j][e] = on[j] ? x[j][e] - mean : 0.0f;
    }
    s = unused = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s = fmaf(x[j][e], x[j][e], s);
    row_sum2<TPR>(s, unused, red, turn);
    const float rstd = live ? 1.0f / sqrtf(s * inv + eps) : 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) x[j][e] *= rstd;
    return rstd;
}

template <int TPR, int NV, int VEC>
__device__ __forceinline__ void load_params(const float* w, const float* b, const bool (&on)[NV], int lane,
                                            float (&wv)[NV][VEC], float (&bv)[NV][VEC]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            wv[j][e] = 1.0f;
            bv[j][e] = 0.0f;
        }
        const int c = (lane + j * TPR) * VEC;
        if (on[j] && w) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) wv[j][e] = w[c + e];
        }
        if (on[j] && b) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) bv[j][e] = b[c + e];
        }
    }
}

// group r as row `row` of memory and the columns before it; r < 2^31
__device__ __forceinline__ void locate(const NormArgs& a, int64_t r, int64_t& row, int& col) {
    row = r;
    col = 0;
    if (a.groups > 1) {
        const uint32_t o = (uint32_t)r / (uint32_t)a.groups;
        row = o;
        col = (int)((uint32_t)r - o * (uint32_t)a.groups) * a.W;
    }
}

template <typename X, typename T, int TPR, int NV, int VEC>
__global__ __launch_bounds__((Shape<TPR, NV, VEC>::threads)) void ssd_norm_fwd_kernel(NormArgs a) {
    using SH = Shape<TPR, NV, VEC>;
    __shared__ float red[2][2][16];
    int turn = 0;
    const int lane = threadIdx.x % TPR, sub = SH::rows == 1 ? 0 : threadIdx.x / TPR;
    bool on[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) on[j] = (lane + j * TPR) * VEC < a.W;
    float wv[NV][VEC], bv[NV][VEC];
    load_params<TPR, NV, VEC>(a.w, a.b, on, lane, wv, bv);
    const X* xp = static_cast<const X*>(a.x);
    const T* zp = static_cast<const T*>(a.z);
    T* yp = static_cast<T*>(a.y);
    for (int64_t r0 = (int64_t)blockIdx.x * SH::rows; r0 < a.R; r0 += (int64_t)gridDim.x * SH::rows) {
        const bool live = r0 + sub < a.R;           // TPR > 64: rows = 1, uniform
        int64_t r;
        int col;
        locate(a, r0 + sub, r, col);
        float x[NV][VEC], z[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (lane + j * TPR) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[j][e] = z[j][e] = 0.0f;
            if (live && on[j]) {
                ldv<VEC>(xp + r * a.x_stride + col + c, x[j]);
                if (zp) ldv<VEC>(zp + r * a.z_stride + col + c, z[j]);
            }
        }
        to_hat<TPR, NV, VEC>(x, on, live, a.W, a.rms, a.eps, red, turn);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (lane + j * TPR) * VEC;
            float y[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                y[e] = fmaf(x[j][e], wv[j][e], bv[j][e]);
                if (zp) y[e] *= silu_f(z[j][e]);
            }
            if (live && on[j]) stv<VEC>(yp + r * a.y_stride + col + c, y);
        }
    }
}

template <typename X, typename T, int TPR, int NV, int VEC>
__global__ __launch_bounds__((Shape<TPR, NV, VEC>::threads)) void ssd_norm_bwd_kernel(NormArgs a) {
    using SH = Shape<TPR, NV, VEC>;
    __shared__ float red[2][2][16];
    int turn = 0;
    const int lane = threadIdx.x % TPR, sub = SH::rows == 1 ? 0 : threadIdx.x / TPR;
    bool on[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) on[j] = (lane + j * TPR) * VEC < a.W;
    constexpr bool kHeld = NV * VEC <= 8;           // w and b stay in registers, else they are read again a row (L1, L2)
    // 1024 threads have 128 registers each: there the sums stand in LDS, every
    // thread's own column of it, so that nothing spills
    constexpr bool kLds = TPR == 1024;
    __shared__ float sums[2][kLds ? NV * VEC : 1][kLds ? TPR : 1];
    float wv[NV][VEC], bv[NV][VEC], dw[kLds ? 1 : NV][VEC], db[kLds ? 1 : NV][VEC];
    if (kHeld) load_params<TPR, NV, VEC>(a.w, a.b, on, lane, wv, bv);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if constexpr (kLds) sums[0][j * VEC + e][lane] = sums[1][j * VEC + e][lane] = 0.0f;
            else dw[j][e] = db[j][e] = 0.0f;
        }
    const X* xp = static_cast<const X*>(a.x);
    const T* zp = static_cast<const T*>(a.z);
    const T* gp = static_cast<const T*>(a.gy);
    X* dxp = static_cast<X*>(a.dx);
    T* dzp = static_cast<T*>(a.dz);
    const float inv = 1.0f / (float)a.W;
    // the next row's operands are on their way while this row is computed
    Raw<X, VEC> nx[NV];
    Raw<T, VEC> nz[NV], ng[NV];
    auto fetch = [&](int64_t at) {
        const bool live = at < a.R;
        int64_t r;
        int col;
        locate(a, at, r, col);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (lane + j * TPR) * VEC;
            nx[j].clear();
            nz[j].clear();
            ng[j].clear();
            if (live && on[j]) {
                nx[j].load(xp + r * a.x_stride + col + c);
                ng[j].load(gp + r * a.gy_stride + col + c);
                if (zp) nz[j].load(zp + r * a.z_stride + col + c);
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * SH::rows;
    int64_t at = (int64_t)blockIdx.x * SH::rows + sub;
    constexpr bool kAhead = !kLds;                   // 1024 threads have no registers for it
    if (kAhead) fetch(at);
    for (; at - sub < a.R; at += step) {
        if (!kAhead) fetch(at);
        const bool live = at < a.R;
        int64_t r;
        int col;
        locate(a, at, r, col);
        float x[NV][VEC], z[NV][VEC], g[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            nx[j].get(x[j]);
            nz[j].get(z[j]);
            ng[j].get(g[j]);
        }
        if (kAhead) fetch(at + step);
        const float rstd = to_hat<TPR, NV, VEC>(x, on, live, a.W, a.rms, a.eps, red, turn);
        if (!kHeld) load_params<TPR, NV, VEC>(a.w, a.b, on, lane, wv, bv);
        float m1 = 0.0f, m2 = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (lane + j * TPR) * VEC;
            if (zp) {
                float d[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float s = fast_rcp(1.0f + fast_exp2(-z[j][e] * kLog2e));
                    const float n = fmaf(x[j][e], wv[j][e], bv[j][e]);
                    d[e] = g[j][e] * n * s * fmaf(z[j][e], 1.0f - s, 1.0f);
                    g[j][e] *= z[j][e] * s;
                }
                if (dzp && live && on[j]) stv<VEC>(dzp + r * a.dz_stride + col + c, d);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                if constexpr (kLds) {
                    sums[0][j * VEC + e][lane] += g[j][e] * x[j][e];
                    sums[1][j * VEC + e][lane] += g[j][e];
                } else {
                    dw[j][e] = fmaf(g[j][e], x[j][e], dw[j][e]);
                    db[j][e] += g[j][e];
                }
                g[j][e] *= wv[j][e];
                m1 += g[j][e];
                m2 = fmaf(g[j][e], x[j][e], m2);
            }
        }
        row_sum2<TPR>(m1, m2, red, turn);
        m1 = a.rms ? 0.0f : m1 * inv;
        m2 *= inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (lane + j * TPR) * VEC;
            float d[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) d[e] = rstd * (g[j][e] - m1 - x[j][e] * m2);
            if (live && on[j]) stv<VEC>(dxp + r * a.dx_stride + col + c, d);
        }
    }
    // the workgroup's sums: [block][2][W], rows of the workgroup added in order
    if (!a.part) return;
    float* out = a.part + (size_t)blockIdx.x * 2 * a.W;
    if constexpr (kLds) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (lane + j * TPR) * VEC;
            if (on[j]) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    out[c + e] = sums[0][j * VEC + e][lane];
                    out[a.W + c + e] = sums[1][j * VEC + e][lane];
                }
            }
        }
    } else if constexpr (SH::rows == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (lane + j * TPR) * VEC;
            if (on[j]) {
                stv<VEC>(out + c, dw[j]);
                stv<VEC>(out + a.W + c, db[j]);
            }
        }
    } else {
        __shared__ float acc[SH::rows][TPR * NV * VEC];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[sub][(lane + j * TPR) * VEC + e] = k ? db[j][e] : dw[j][e];
            __syncthreads();
            for (int c = threadIdx.x; c < a.W; c += SH::threads) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < SH::rows; ++i) s += acc[i][c];
                out[(size_t)k * a.W + c] = s;
            }
        }
    }
}

// dw and db: the sum of the workgroups' partial rows.  32 columns a workgroup,
// 32 threads a column each adding every 32nd row, four loads at a time, then
// the 32 sums in order.
__global__ __launch_bounds__(1024) void ssd_norm_sum_kernel(const float* part, int nblk, int W, float* dw, float* db) {
    __shared__ float s[32][33];
    const int x = threadIdx.x % 32, k = threadIdx.x / 32, c = blockIdx.x * 32 + x;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (c < 2 * W) {
        const float* p = part + c;
        int i = k;
        for (; i + 96 < nblk; i += 128) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += p[(size_t)(i + 32 * j) * 2 * W];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + 32 * j < nblk) v[j] += p[(size_t)(i + 32 * j) * 2 * W];
    }
    s[k][x] = (v[0] + v[1]) + (v[2] + v[3]);
    __syncthreads();
    if (k == 0 && c < 2 * W) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += s[i][x];
        if (c < W) {
            if (dw) dw[c] = t;
        } else if (db) {
            db[c - W] = t;
        }
    }
}

template <typename X, typename T, int TPR, int NV, int VEC>
hipError_t launch_fwd(const NormArgs& a, hipStream_t stream) {
    using SH = Shape<TPR, NV, VEC>;
    const int64_t blocks = std::min<int64_t>((a.R + SH::rows - 1) / SH::rows, kNormGrid);
    hipLaunchKernelGGL((ssd_norm_fwd_kernel<X, T, TPR, NV, VEC>), dim3((unsigned)blocks), dim3(SH::threads), 0, stream, a);
    return hipGetLastError();
}
template <typename X, typename T, int TPR, int NV, int VEC>
hipError_t launch_bwd(const NormArgs& a, hipStream_t stream) {
    using SH = Shape<TPR, NV, VEC>;
    const int n = (int)std::min<int64_t>((a.R + SH::rows - 1) / SH::rows, kNormBwdGrid);
    hipLaunchKernelGGL((ssd_norm_bwd_kernel<X, T, TPR, NV, VEC>), dim3(n), dim3(SH::threads), 0, stream, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.part) return e;
    hipLaunchKernelGGL(ssd_norm_sum_kernel, dim3((2 * a.W + 31) / 32), dim3(1024), 0, stream, a.part, n, a.W, a.dw, a.db);
    return hipGetLastError();
}

// Threads and vectors of a row: the forward holds up to 32 columns a thread,
// the backward, with five values a column live, up to 16.
template <typename X, typename T>
hipError_t launch_fwd_t(const NormArgs& a, hipStream_t s) {
    if (a.vec) {
        const int n = a.W / 8;
        if (n <= 8) return launch_fwd<X, T, 8, 1, 8>(a, s);
        if (n <= 16) return launch_fwd<X, T, 16, 1, 8>(a, s);
        if (n <= 32) return launch_fwd<X, T, 32, 1, 8>(a, s);
        if (n <= 64) return launch_fwd<X, T, 64, 1, 8>(a, s);
        if (n <= 128) return launch_fwd<X, T, 64, 2, 8>(a, s);
        if (n <= 256) return launch_fwd<X, T, 64, 4, 8>(a, s);
        if (n <= 512) return launch_fwd<X, T, 256, 2, 8>(a, s);
        if (n <= 1024) return launch_fwd<X, T, 256, 4, 8>(a, s);
        return launch_fwd<X, T, 512, 4, 8>(a, s);
    }
    if (a.W <= 16) return launch_fwd<X, T, 16, 1, 1>(a, s);
    if (a.W <= 64) return launch_fwd<X, T, 64, 1, 1>(a, s);
    if (a.W <= 256) return launch_fwd<X, T, 64, 4, 1>(a, s);
    if (a.W <= 1024) return launch_fwd<X, T, 64, 16, 1>(a, s);
    if (a.W <= 4096) return launch_fwd<X, T, 256, 16, 1>(a, s);
    return launch_fwd<X, T, 512, 16, 1>(a, s);
}
template <typename X, typename T>
hipError_t launch_bwd_t(const NormArgs& a, hipStream_t s) {
    if (a.vec) {
        const int n = a.W / 8;
        if (n <= 8) return launch_bwd<X, T, 8, 1, 8>(a, s);
        if (n <= 16) return launch_bwd<X, T, 16, 1, 8>(a, s);
        if (n <= 32) return launch_bwd<X, T, 32, 1, 8>(a, s);
        if (n <= 64) return launch_bwd<X, T, 64, 1, 8>(a, s);
        if (n <= 128) return launch_bwd<X, T, 64, 2, 8>(a, s);
        if (n <= 256) return launch_bwd<X, T, 256, 1, 8>(a, s);
        if (n <= 512) return launch_bwd<X, T, 256, 2, 8>(a, s);
        if (n <= 1024) return launch_bwd<X, T, 512, 2, 8>(a, s);
        return launch_bwd<X, T, 1024, 2, 8>(a, s);
    }
    if (a.W <= 16) return launch_bwd<X, T, 16, 1, 1>(a, s);
    if (a.W <= 64) return launch_bwd<X, T, 64, 1, 1>(a, s);
    if (a.W <= 256) return launch_bwd<X, T, 64, 4, 1>(a, s);
    if (a.W <= 1024) return launch_bwd<X, T, 256, 4, 1>(a, s);
    if (a.W <= 4096) return launch_bwd<X, T, 512, 8, 1>(a, s);
    return launch_bwd<X, T, 1024, 8, 1>(a, s);
}
template <typename X, typename T>
hipError_t launch_norm_t(const NormArgs& a, hipStream_t s) {
    return a.gy ? launch_bwd_t<X, T>(a, s) : launch_fwd_t<X, T>(a, s);
}

}  // namespace

size_t norm_bwd_workspace_bytes(int64_t R, int W) {
    return (size_t)std::min<int64_t>(R, kNormBwdGrid) * 2 * W * sizeof(float);
}

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    if (a.x_dtype == 0) return a.dtype == 0 ? launch_norm_t<float, float>(a, s) : launch_norm_t<float, uint16_t>(a, s);
    return a.dtype == 0 ? launch_norm_t<uint16_t, float>(a, s) : launch_norm_t<uint16_t, uint16_t>(a, s);
}

}  // namespace ssd
