// add_norm.hip -- the norm at a layer's entry and end: the residual's addition before it, 8-bit output behind it.
//
//   s = x + residual, rounded to the residual's type and stored (or s = x)
//   n = norm(s) as in norm.hip,  y = (n w + b) silu(z)
//   q = e4m3(y / scale),  scale = max|y| / 448 over every 128 columns of the row
//
// The statistics are those of the stored sum, so that the backward pass (norm.hip's, with the stream's gradient added)
// and a second forward see the same row.  q is rounded from fp32, not from a y that was rounded before.
//
// One pass over HBM: a row stays in its threads' registers from the sum to the last output.  Threads and vectors of a row
// are norm.hip's, but that every row is read in vectors of 8: one that does not start on 16 bytes, or ends inside a vector, at
// the alignment of its elements.  128 columns are 16 neighbouring lanes, so their maximum is four lane exchanges.
//
// Bound by HBM.  Measured: 32768 rows of 4096, bf16 plus bf16 to e4m3, 182 us (944 MB, 5.2 TB/s, the rate of a large copy);
// 16 rows of 2048 6 us, a launch and a row's latency.  Odd rows to e4m3: 16228 of 3646 in bf16 113 us (a copy of as much 80), 20000
// of 1001 in fp32 54 (50); read element by element the first took 436.  The backward, 40960 rows of 2048 in bf16 with the stream's
// gradient: 124 us and 5 us of sums (671 MB, 5.2 TB/s).  The large ones with inputs that the last-level cache does not hold: 20000 x 1001 over
// the same 160 MB of inputs takes 47.
#include <hip/hip_runtime.h>
#include <algorithm>

#include "layer_launch.hpp"
#include "norm_device.hpp"

namespace ssd {
namespace {

constexpr float kE4m3Max = 448.0f;

template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true)));
}
// the maximum of an aligned group of W lanes (8 or 16), v >= 0
template <int W>
__device__ __forceinline__ float lanes_max(float v) {
    v = dpp_max<0xB1>(v);
    v = dpp_max<0x4E>(v);
    v = dpp_max<0x141>(v);
    if (W >= 16) v = dpp_max<0x140>(v);
    return v;
}

// |v|, and 0 for NaN: a NaN quantises to NaN and does not choose the scale
__device__ __forceinline__ float size_of(float v) { return v == v ? fabsf(v) : 0.0f; }
// Infinities take the largest finite scale; below 2^-100 the reciprocal would leave fp32.
__device__ __forceinline__ float scale_of(float top) {
    return top > 0.0f ? fminf(fmaxf(top, 0x1p-100f), 0x1.fffffep127f) / kE4m3Max : 1.0f;
}
__device__ __forceinline__ float into_range(float v) { return v == v ? fminf(fmaxf(v, -kE4m3Max), kE4m3Max) : v; }

// a row's values rounded to the stream's type
__device__ __forceinline__ float round_to(const float*, float v) { return v; }
__device__ __forceinline__ float round_to(const uint16_t*, float v) { return __uint_as_float(f32_to_bf16_bits(v) << 16); }

// S: the type of the row that is normalised (the residual's, or x's where there is none); T: y's and z's
// ODD: rows off the 16-byte grid, or cut inside a thread's eight columns
template <typename S, typename T, int TPR, int NV, bool ODD>
__global__ __launch_bounds__((Shape<TPR, NV, 8>::threads)) void ssd_add_norm_kernel(AddNormArgs a) {
    constexpr int VEC = 8;
    using SH = Shape<TPR, NV, VEC>;
    __shared__ float red[2][2][16];
    int turn = 0;
    const int lane = threadIdx.x % TPR, sub = SH::rows == 1 ? 0 : threadIdx.x / TPR;
    bool on[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) on[j] = (lane + j * TPR) * VEC < a.W;
    float wv[NV][VEC], bv[NV][VEC];
    load_params<TPR, NV, VEC, ODD>(a.w, a.b, on, lane, wv, bv, a.W);
    const S* rp = static_cast<const S*>(a.residual);
    S* sp = static_cast<S*>(a.sum);
    const T* zp = static_cast<const T*>(a.z);
    T* yp = static_cast<T*>(a.y);
    for (int64_t r0 = (int64_t)blockIdx.x * SH::rows; r0 < a.R; r0 += (int64_t)gridDim.x * SH::rows) {
        const int64_t r = r0 + sub;
        const bool live = r < a.R;                  // TPR > 64: rows = 1, uniform
        float x[NV][VEC], z[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (lane + j * TPR) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) x[j][e] = z[j][e] = 0.0f;
            if (live && on[j]) {
                if (rp) {
                    float f[VEC];
                    ld_row<VEC, ODD>(rp + r * a.residual_stride + c, a.W - c, a.W < 8, f);
                    if (a.x_dtype == 0) ld_row<VEC, ODD>(static_cast<const float*>(a.x) + r * a.x_stride + c, a.W - c, a.W < 8, x[j]);
                    else ld_row<VEC, ODD>(static_cast<const uint16_t*>(a.x) + r * a.x_stride + c, a.W - c, a.W < 8, x[j]);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) x[j][e] = round_to(rp, x[j][e] + f[e]);
                } else {
                    ld_row<VEC, ODD>(static_cast<const S*>(a.x) + r * a.x_stride + c, a.W - c, a.W < 8, x[j]);
                }
                if (zp) ld_row<VEC, ODD>(zp + r * a.z_stride + c, a.W - c, a.W < 8, z[j]);
            }
        }
        if (sp) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (lane + j * TPR) * VEC;
                if (live && on[j]) st_row<VEC, ODD>(sp + r * a.sum_stride + c, a.W - c, x[j]);
            }
        }
        to_hat<TPR, NV, VEC, ODD>(x, on, live, a.W, a.rms, a.eps, red, turn, lane);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                x[j][e] = fmaf(x[j][e], wv[j][e], bv[j][e]);
                if (zp) x[j][e] *= silu_f(z[j][e]);
            }
        if (yp) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = (lane + j * TPR) * VEC;
                if (live && on[j]) st_row<VEC, ODD>(yp + r * a.y_stride + c, a.W - c, x[j]);
            }
        }
        if (!a.q) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, size_of(on[j] ? x[j][e] : 0.0f));
            const float scale = scale_of(lanes_max<(TPR < 16 ? TPR : 16)>(top)), inv = 1.0f / scale;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = into_range(x[j][e] * inv);
            uint2 o;
            int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
            o.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], p, true);
            p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
            o.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], p, true);
            const int c = lane + j * TPR;
            if (live && on[j]) {
                uint8_t* q = a.q + r * a.q_stride + c * 8;
                if (!ODD) {
                    *reinterpret_cast<uint2*>(q) = o;
                } else if (a.W - c * 8 >= 8) {
                    __builtin_memcpy(q, &o, 8);
                } else {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (e < a.W - c * 8) q[e] = (uint8_t)((e < 4 ? o.x : o.y) >> 8 * (e % 4));
                }
                if (c % 16 == 0) a.scale[r * a.scale_stride + c / 16] = scale;
            }
        }
    }
}

template <typename S, typename T, int TPR, int NV, bool ODD>
hipError_t launch(const AddNormArgs& a, hipStream_t stream) {
    using SH = Shape<TPR, NV, 8>;
    const int64_t blocks = std::min<int64_t>((a.R + SH::rows - 1) / SH::rows, kNormGrid);
    hipLaunchKernelGGL((ssd_add_norm_kernel<S, T, TPR, NV, ODD>), dim3((unsigned)blocks), dim3(SH::threads), 0, stream, a);
    return hipGetLastError();
}

// Threads and vectors of a row: norm.hip's up to 32 columns a thread, where they are measured.
template <typename S, typename T, bool ODD>
hipError_t launch_t(const AddNormArgs& a, hipStream_t s) {
    const int n = (a.W + 7) / 8;
    if (n <= 8) return launch<S, T, 8, 1, ODD>(a, s);
    if (n <= 16) return launch<S, T, 16, 1, ODD>(a, s);
    if (n <= 32) return launch<S, T, 32, 1, ODD>(a, s);
    if (n <= 64) return launch<S, T, 64, 1, ODD>(a, s);
    if (n <= 128) return launch<S, T, 64, 2, ODD>(a, s);
    if (n <= 256) return launch<S, T, 64, 4, ODD>(a, s);
    if (n <= 512) return launch<S, T, 256, 2, ODD>(a, s);
    if (n <= 1024) return launch<S, T, 256, 4, ODD>(a, s);
    return launch<S, T, 512, 4, false>(a, s);        // rows of more than 8192 are on the grid
}
template <typename S, typename T>
hipError_t launch_s(const AddNormArgs& a, hipStream_t s) {
    return a.vec ? launch_t<S, T, false>(a, s) : launch_t<S, T, true>(a, s);
}

}  // namespace

hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t s) {
    if (a.s_dtype == 0) return a.dtype == 0 ? launch_s<float, float>(a, s) : launch_s<float, uint16_t>(a, s);
    return a.dtype == 0 ? launch_s<uint16_t, float>(a, s) : launch_s<uint16_t, uint16_t>(a, s);
}

}  // namespace ssd
