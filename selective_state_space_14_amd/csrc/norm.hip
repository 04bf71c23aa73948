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

#include <type_traits>

#include "layer_launch.hpp"
#include "norm_device.hpp"

namespace ssd {
namespace {

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

// ADD: dx also takes gs, the gradient that reaches the norm's input past it (a residual stream's), or null with ODD: rows off
// the 16-byte grid, or cut inside a thread's eight columns
template <typename X, typename T, int TPR, int NV, int VEC, bool ADD, bool ODD>
__global__ __launch_bounds__((Shape<TPR, NV, VEC>::threads)) void ssd_norm_bwd_kernel(
    std::conditional_t<ADD, AddNormBwdArgs, NormArgs> a) {
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
    constexpr bool kAddAhead = ADD && !kLds;         // and gs is read where it is used
    __shared__ float sums[2][kLds ? NV * VEC : 1][kLds ? TPR : 1];
    float wv[NV][VEC], bv[NV][VEC], dw[kLds ? 1 : NV][VEC], db[kLds ? 1 : NV][VEC];
    if (kHeld) load_params<TPR, NV, VEC, ODD>(a.w, a.b, on, lane, wv, bv, a.W);
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
    const X* sp = nullptr;
    int64_t sp_stride = 0;
    if constexpr (ADD) {
        sp = static_cast<const X*>(a.gs);
        sp_stride = a.gs_stride;
    }
    X* dxp = static_cast<X*>(a.dx);
    T* dzp = static_cast<T*>(a.dz);
    const float inv = 1.0f / (float)a.W;
    // the next row's operands are on their way while this row is computed
    Raw<X, VEC> nx[NV], ns[kAddAhead ? NV : 1];
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
            if constexpr (kAddAhead) ns[j].clear();
            if (live && on[j]) {
                if constexpr (ODD) {
                    if constexpr (kAddAhead) {
                        if (sp) ns[j].load_odd(sp + r * sp_stride + c, a.W - c, a.W < 8);
                    }
                    nx[j].load_odd(xp + r * a.x_stride + c, a.W - c, a.W < 8);
                    ng[j].load_odd(gp + r * a.gy_stride + c, a.W - c, a.W < 8);
                    if (zp) nz[j].load_odd(zp + r * a.z_stride + c, a.W - c, a.W < 8);
                } else {
                    if constexpr (kAddAhead) ns[j].load(sp + r * sp_stride + col + c);
                    nx[j].load(xp + r * a.x_stride + col + c);
                    ng[j].load(gp + r * a.gy_stride + col + c);
                    if (zp) nz[j].load(zp + r * a.z_stride + col + c);
                }
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * SH::rows;
    int64_t at = (int64_t)blockIdx.x * SH::rows + sub;
    // 1024 threads have no registers for it, nor have 512 with what the ends of rows take
    constexpr bool kAhead = !kLds && !(ODD && TPR == 512);
    if (kAhead) fetch(at);
    for (; at - sub < a.R; at += step) {
        if (!kAhead) fetch(at);
        const bool live = at < a.R;
        int64_t r;
        int col;
        locate(a, at, r, col);
        float x[NV][VEC], z[NV][VEC], g[NV][VEC], past[kAddAhead ? NV : 1][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            nx[j].get(x[j]);
            nz[j].get(z[j]);
            ng[j].get(g[j]);
            if constexpr (kAddAhead) ns[j].get(past[j]);
            if constexpr (ODD) {
                const int k = on[j] && a.W >= 8 ? before(a.W - (lane + j * TPR) * VEC) : 0;
                shift_out(x[j], k);
                shift_out(z[j], k);
                shift_out(g[j], k);
                if constexpr (kAddAhead) shift_out(past[j], k);
            }
        }
        if (kAhead) fetch(at + step);
        const float rstd = to_hat<TPR, NV, VEC, ODD>(x, on, live, a.W, a.rms, a.eps, red, turn, lane);
        if (!kHeld) load_params<TPR, NV, VEC, ODD>(a.w, a.b, on, lane, wv, bv, a.W);
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
                if (dzp && live && on[j]) st_row<VEC, ODD>(dzp + r * a.dz_stride + col + c, a.W - c, d);
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
            for (int e = 0; e < VEC; ++e) {
                d[e] = rstd * (g[j][e] - m1 - x[j][e] * m2);
                if constexpr (kAddAhead) d[e] += past[j][e];
            }
            if constexpr (ADD && !kAddAhead) {
                float p[VEC];
                if (live && on[j]) {
                    ldv<VEC>(sp + r * sp_stride + col + c, p);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) d[e] += p[e];
                }
            }
            if (live && on[j]) st_row<VEC, ODD>(dxp + r * a.dx_stride + col + c, a.W - c, d);
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
                st_row<VEC, ODD>(out + c, a.W - c, dw[j]);
                st_row<VEC, ODD>(out + a.W + c, a.W - c, db[j]);
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
template <typename X, typename T, int TPR, int NV, int VEC, bool ODD = false, typename Args>
hipError_t launch_bwd(const Args& a, hipStream_t stream) {
    using SH = Shape<TPR, NV, VEC>;
    const int n = (int)std::min<int64_t>((a.R + SH::rows - 1) / SH::rows, kNormBwdGrid);
    hipLaunchKernelGGL((ssd_norm_bwd_kernel<X, T, TPR, NV, VEC, std::is_same_v<Args, AddNormBwdArgs>, ODD>), dim3(n), dim3(SH::threads), 0, stream, a);
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
// every row in vectors, ODD: at the alignment of their elements
template <typename X, typename T, bool ODD, typename Args>
hipError_t launch_bwd_vec(const Args& a, hipStream_t s) {
    const int n = (a.W + 7) / 8;
    if (n <= 8) return launch_bwd<X, T, 8, 1, 8, ODD>(a, s);
    if (n <= 16) return launch_bwd<X, T, 16, 1, 8, ODD>(a, s);
    if (n <= 32) return launch_bwd<X, T, 32, 1, 8, ODD>(a, s);
    if (n <= 64) return launch_bwd<X, T, 64, 1, 8, ODD>(a, s);
    if (n <= 128) return launch_bwd<X, T, 64, 2, 8, ODD>(a, s);
    if (n <= 256) return launch_bwd<X, T, 256, 1, 8, ODD>(a, s);
    if (n <= 512) return launch_bwd<X, T, 256, 2, 8, ODD>(a, s);
    if (n <= 1024) return launch_bwd<X, T, 512, 2, 8, ODD>(a, s);
    return launch_bwd<X, T, 1024, 2, 8>(a, s);       // rows of more than 8192 are on the grid
}
template <typename X, typename T>
hipError_t launch_bwd_t(const NormArgs& a, hipStream_t s) {
    if (a.vec) return launch_bwd_vec<X, T, false>(a, s);
    if (a.W <= 16) return launch_bwd<X, T, 16, 1, 1>(a, s);
    if (a.W <= 64) return launch_bwd<X, T, 64, 1, 1>(a, s);
    if (a.W <= 256) return launch_bwd<X, T, 64, 4, 1>(a, s);
    if (a.W <= 1024) return launch_bwd<X, T, 256, 4, 1>(a, s);
    if (a.W <= 4096) return launch_bwd<X, T, 512, 8, 1>(a, s);
    return launch_bwd<X, T, 1024, 8, 1>(a, s);
}
template <typename X, typename T>
hipError_t launch_bwd_t(const AddNormBwdArgs& a, hipStream_t s) {
    return a.vec ? launch_bwd_vec<X, T, false>(a, s) : launch_bwd_vec<X, T, true>(a, s);
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

hipError_t launch_add_norm_bwd(const AddNormBwdArgs& a, hipStream_t s) {
    if (a.vec && !a.gs) return launch_norm(a, s);
    if (a.x_dtype == 0) return a.dtype == 0 ? launch_bwd_t<float, float>(a, s) : launch_bwd_t<float, uint16_t>(a, s);
    return a.dtype == 0 ? launch_bwd_t<uint16_t, float>(a, s) : launch_bwd_t<uint16_t, uint16_t>(a, s);
}

}  // namespace ssd
