// norm_device.hpp -- what the row norms share: vectors of a row, sums over a row's threads, the normalised row.
#pragma once

#include "ssd_device.hpp"

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

// Eight elements at any alignment of theirs, which the hardware reads and writes in one instruction too.  Of a row's last ones
// only `left` are the thread's: the vector that ends with the row is read, and what stands before the thread's own shifted
// out (so no thread waits for single elements; what a neighbour may be writing there is not used).  Rows of fewer than eight
// columns (few) are read one by one.  Elements that the row does not have read as 0.
template <typename V>
__device__ __forceinline__ V load_any(const void* p) {
    V v;
    __builtin_memcpy(&v, p, sizeof(V));
    return v;
}
__device__ __forceinline__ int before(int left) { return left < 8 ? 8 - left : 0; }
__device__ __forceinline__ void shift_out(float (&v)[8], int k) {
    if (!k) return;
#pragma unroll
    for (int s = 4; s; s >>= 1) {
        const bool by = k & s;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = by ? (e + s < 8 ? v[e + s < 8 ? e + s : 0] : 0.0f) : v[e];
    }
}
__device__ __forceinline__ void ld_odd(const float* p, int left, bool few, float (&v)[8]) {
    if (few) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < left ? p[e] : 0.0f;
        return;
    }
    const int k = before(left);
    const f32x4 a = load_any<f32x4>(p - k), b = load_any<f32x4>(p - k + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
    }
    shift_out(v, k);
}
__device__ __forceinline__ void ld_odd(const uint16_t* p, int left, bool few, float (&v)[8]) {
    if (few) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < left ? bf16_to_f32(p[e]) : 0.0f;
        return;
    }
    const int k = before(left);
    const u32x4_t a = load_any<u32x4_t>(p - k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(a[i]);
        v[2 * i + 1] = bf16_hi(a[i]);
    }
    shift_out(v, k);
}
__device__ __forceinline__ void st_odd(float* p, int left, const float (&v)[8]) {
    if (left >= 8) {
        const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
        __builtin_memcpy(static_cast<void*>(p), &a, 16);
        __builtin_memcpy(static_cast<void*>(p + 4), &b, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < left) p[e] = v[e];
    }
}
__device__ __forceinline__ void st_odd(uint16_t* p, int left, const float (&v)[8]) {
    if (left >= 8) {
        const u32x4_t a = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
        __builtin_memcpy(static_cast<void*>(p), &a, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < left) p[e] = (uint16_t)f32_to_bf16_bits(v[e]);
    }
}
// a thread's vector, ODD: as above
template <int VEC, bool ODD, typename T>
__device__ __forceinline__ void ld_row(const T* p, int left, bool few, float (&v)[VEC]) {
    if constexpr (ODD) ld_odd(p, left, few, v);
    else ldv<VEC>(p, v);
}
template <int VEC, bool ODD, typename T>
__device__ __forceinline__ void st_row(T* p, int left, const float (&v)[VEC]) {
    if constexpr (ODD) st_odd(p, left, v);
    else stv<VEC>(p, v);
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
    __device__ __forceinline__ void load_odd(const uint16_t* p, int left, bool few) {
        if (!few) {
            v = load_any<u32x4_t>(p - before(left));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = (2 * i < left ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < left ? (uint32_t)p[2 * i + 1] << 16 : 0u);
        }
    }
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
    __device__ __forceinline__ void load_odd(const float* p, int left, bool few) {
        if (!few) {
            p -= before(left);
            a = load_any<f32x4>(p);
            b = load_any<f32x4>(p + 4);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = i < left ? p[i] : 0.0f;
                b[i] = 4 + i < left ? p[4 + i] : 0.0f;
            }
        }
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
template <int TPR, int NV, int VEC, bool ODD = false>
__device__ __forceinline__ float to_hat(float (&x)[NV][VEC], const bool (&on)[NV], bool live, int W, int rms, float eps,
                                        float (*red)[2][16], int& turn, int lane = 0) {
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
            for (int e = 0; e < VEC; ++e)
                x[j][e] = (ODD ? (lane + j * TPR) * VEC + e < W : on[j]) ? x[j][e] - mean : 0.0f;
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

template <int TPR, int NV, int VEC, bool ODD = false>
__device__ __forceinline__ void load_params(const float* w, const float* b, const bool (&on)[NV], int lane,
                                            float (&wv)[NV][VEC], float (&bv)[NV][VEC], int W = 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            wv[j][e] = 1.0f;
            bv[j][e] = 0.0f;
        }
        const int c = (lane + j * TPR) * VEC;
        if constexpr (ODD) {
            if (on[j] && w) ld_odd(w + c, W - c, W < 8, wv[j]);
            if (on[j] && b) ld_odd(b + c, W - c, W < 8, bv[j]);
        } else {
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
}

}  // namespace
}  // namespace ssd
